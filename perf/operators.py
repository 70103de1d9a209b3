"""Workloads of the library's linear-attention and 4-bit cache operators.

Four kinds of case, each a call (or the pair of calls) that a serving program makes:

* ``linear_prefill``  gdn_linear_prefill: linear attention with a decay for each head,
                      packed prompts.
* ``linear_decode``   gdn_linear_decode: one token per sequence on a pool of states.
* ``kv_append``       gdn_kv_append, then gdn_kv_read of the rows it wrote: rotation of q
                      and k, 4-bit storage of k and v in a paged cache.
* ``kv_attention``    gdn_kv_attention: attention over such a cache.

``run`` computes a case through the library when ``own`` is true, and in elementary torch
operations (32-bit arithmetic, one rounding at the end) when it is false.  ``exact`` gives
the same outputs from the definitions in 64 bits.

The cache is one uint8 tensor [pages, 2 (k, v), Hkv, page, D/2 + D/8].  A record (one token
of one head) is D/2 bytes of codes followed by D/32 pairs (scale, minimum) of fp16, one for
each 32 consecutive elements; element d stands for minimum + scale * code.  The codes are
nibbles (low first) in this order: nibble 8 W + i of a key record holds
d = 32 (W mod D/32) + 8 (W div D/32) + i, and nibble 8 W + i of a value record holds
d = 64 (W div 8) + 32 (i div 4) + 4 (W mod 8) + i mod 4.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_GROUP = 32


# ------------------------------------------------------------------------------- cases

def listed():
    lp = dict(kind="linear_prefill", dtype="bf16", D=128, Hk=16, Hv=32, n=1, lo=1, hi=1,
              decay="token", start=False)
    ld = dict(kind="linear_decode", dtype="bf16", D=128, Hk=16, Hv=48, n=1, pool=1,
              decay="token")
    ap = dict(kind="kv_append", dtype="bf16", D=128, Hq=32, Hkv=8, page=16, n=1, q_lo=1,
              q_hi=1, past=0, rot=128, interleaved=False)
    at = dict(kind="kv_attention", dtype="bf16", D=128, Hq=32, Hkv=8, page=16, n=1, m=1,
              lo=1, hi=1)
    return [
        # a short prompt alone: launch and pipeline latency
        dict(lp, name="linear prefill, 100 tokens", lo=100, hi=100),
        # one layer of a 4096-token prompt over the library's 48 v-heads, fixed decays
        dict(lp, name="linear prefill, 4096 tokens", Hv=48, lo=4096, hi=4096, decay="head"),
        # a packed batch of continued prompts of ragged lengths, about 32k tokens
        dict(lp, name="linear prefill, packed", Hv=48, n=8, lo=1, hi=8192, start=True),
        # fp32 activations over narrow heads, two prompts
        dict(lp, name="linear prefill, fp32", dtype="fp32", D=64, Hk=4, Hv=8, n=2, lo=700,
             hi=900),
        # fp32 activations, two sequences answering at once
        dict(ld, name="linear decode, fp32", dtype="fp32", D=64, Hk=4, Hv=8, n=2, pool=4),
        # a full decode batch: 256 states of 48 heads, 805 MB
        dict(ld, name="linear decode, 256 sequences", n=256, pool=256),
        # the cache write of a decode step of eight sequences
        dict(ap, name="append, 8 tokens", n=8, past=1000),
        # the cache write of ragged prompts, about 8k tokens
        dict(ap, name="append, prompts", n=4, q_lo=1500, q_hi=2600, past=77),
        # one sequence answering over a short context: latency
        dict(at, name="attention, 777 keys", lo=777, hi=777),
        # a decode batch over ragged contexts
        dict(at, name="attention, 64 sequences", n=64, lo=1, hi=16384, page=32),
        # four drafted tokens checked over one very long context, wide heads
        dict(at, name="attention, long context", D=256, Hq=24, Hkv=4, page=64, m=4,
             lo=131072, hi=131072),
        # a 2048-token piece of a prompt over the 8k tokens before it and itself
        dict(at, name="attention, prompt piece", m=2048, lo=10240, hi=10240),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["linear_prefill", "linear_decode", "kv_append", "kv_attention"])
    len_seed = rng.randrange(1 << 20)
    if kind in ("linear_prefill", "linear_decode"):
        dtype, D = rng.choice([("bf16", 128), ("bf16", 128), ("bf16", 128), ("fp32", 64)])
        Hk, Hv = rng.choice([(1, 1), (2, 6), (4, 8), (16, 16), (16, 32), (16, 48)])
        c = dict(kind=kind, dtype=dtype, D=D, Hk=Hk, Hv=Hv, len_seed=len_seed,
                 decay=rng.choice(["token", "head"]))
        if kind == "linear_decode":
            n = _log_int(rng, 1, 256)
            return dict(c, n=n, pool=n + rng.randrange(0, 3))
        n = rng.choice([1, 1, 2, 3, 5, 8])
        hi = _log_int(rng, 1, (32768 if dtype == "bf16" else 4096) // n)
        return dict(c, n=n, lo=rng.randrange(1, hi + 1), hi=hi, start=rng.random() < 0.5)
    D = rng.choice([64, 128, 128, 256])
    Hq, Hkv = rng.choice([(8, 8), (16, 2), (24, 4), (32, 8), (8, 1)])
    page = rng.choice([16, 32, 64, 128])
    c = dict(kind=kind, dtype="bf16", D=D, Hq=Hq, Hkv=Hkv, page=page, len_seed=len_seed)
    if kind == "kv_append":
        n = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 8192 // n)
        return dict(c, n=n, q_lo=rng.randrange(1, hi + 1), q_hi=hi, past=_log_int(rng, 1, 4096),
                    rot=rng.choice([D, D // 2]), interleaved=rng.random() < 0.5)
    if rng.random() < 0.25:     # a piece of a prompt
        m = _log_int(rng, 16, 2048)
        hi = m + _log_int(rng, 1, 8192)
        return dict(c, n=1, m=m, lo=hi, hi=hi)
    n = _log_int(rng, 1, 64)
    hi = _log_int(rng, 1, min(131072, (1 << 20) // n))
    hi = min(hi, (1 << 32) // (n * Hkv * D * 4))
    return dict(c, n=n, m=rng.choice([1, 1, 1, 2, 5]), lo=rng.randrange(1, hi + 1), hi=hi)


def _lens(case, lo="lo", hi="hi"):
    r = random.Random(case.get("len_seed", 7))
    lens = [r.randint(case[lo], case[hi]) for _ in range(case["n"])]
    lens[0] = case[hi]
    return lens


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _offsets(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return torch.tensor(cu, dtype=torch.int32)


def _log_decay(gen, case, T):
    """Log decays: fixed per head, from half-lives of one token to hundreds, or drawn per
    token and head around e^g = 0.95."""
    Hv = case["Hv"]
    if case["decay"] == "head":
        slope = torch.exp2(-8.0 * torch.arange(1, Hv + 1, device="cuda") / Hv)
        return -(slope * (1 + 0.1 * torch.rand(Hv, generator=gen, device="cuda"))).float()
    return -torch.nn.functional.softplus(_randn(gen, T, Hv) - 3.0)


def _pages(gen, lens, page):
    """A block table whose pages lie anywhere in the cache, and the page count."""
    need = [-(-x // page) for x in lens]
    total = sum(need) + 3
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), max(max(need), 1)), dtype=torch.int32, device="cuda")
    at = 0
    for n, c in enumerate(need):
        table[n, :c] = perm[at:at + c]
        at += c
    return table, total


def prepare(case, seed):
    gen = _gen(seed)
    dt, D, kind = _DT[case["dtype"]], case["D"], case["kind"]
    s = dict(case=case)
    if kind in ("linear_prefill", "linear_decode"):
        Hk, Hv, n = case["Hk"], case["Hv"], case["n"]
        lens = _lens(case) if kind == "linear_prefill" else [1] * n
        T = sum(lens)
        unit = torch.nn.functional.normalize
        s["q"] = unit(_randn(gen, T, Hk, D), dim=-1).to(dt)
        s["k"] = unit(_randn(gen, T, Hk, D), dim=-1).to(dt)
        s["v"] = _randn(gen, T, Hv, D).to(dt)
        s["g"] = _log_decay(gen, case, T)
        if kind == "linear_prefill":
            s["lens"] = lens
            s["cu_host"] = _offsets(lens)
            s["cu"] = s["cu_host"].cuda()
            s["h0"] = 0.2 * _randn(gen, n, Hv, D, D) if case["start"] else None
        else:
            s["state"] = 0.2 * _randn(gen, case["pool"], Hv, D, D)
            s["idx"] = torch.randperm(case["pool"], generator=gen, device="cuda")[:n].int()
        return s
    Hq, Hkv, page, n = case["Hq"], case["Hkv"], case["page"], case["n"]
    if kind == "kv_append":
        m = _lens(case, "q_lo", "q_hi")
        lens = [x + case["past"] for x in m]
    else:
        m = [case["m"]] * n
        lens = [max(x, case["m"]) for x in _lens(case)]
    s["m"], s["lens"] = m, lens
    s["cu_host"] = _offsets(m)
    s["cu"] = s["cu_host"].cuda()
    s["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["table"], pages = _pages(gen, lens, page)
    T, ng = sum(m), D // _GROUP
    s["q"] = _randn(gen, T, Hq, D).to(dt)
    if kind == "kv_append":
        s["k"] = (_randn(gen, T, Hkv, D) * (1 + 3 * torch.rand(Hkv, D, generator=gen, device="cuda") ** 8)).to(dt)
        s["v"] = _randn(gen, T, Hkv, D).to(dt)
        half = case["rot"] // 2
        ang = torch.arange(max(lens), device="cuda")[:, None].double() \
            * (1e6 ** (-torch.arange(half, device="cuda").double() / half))
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        s["cache"] = torch.zeros((pages, 2, Hkv, page, D // 2 + 4 * ng), dtype=torch.uint8,
                                 device="cuda")
        return s
    # a cache as appended keys and values leave it: near-Gaussian codes, group ranges of
    # about five standard deviations
    cache = torch.empty((pages, 2, Hkv, page, D // 2 + 4 * ng), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (2 * Hkv * page * D))
    for at in range(0, pages, step):
        part = cache[at:at + step]
        codes = torch.randn(part.shape[:-1] + (D,), generator=gen, device="cuda")
        codes = codes.mul_(3.0).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        part[..., :D // 2] = codes[..., 0::2] | (codes[..., 1::2] << 4)
        sc = 0.28 + 0.1 * torch.rand(part.shape[:-1] + (ng,), generator=gen, device="cuda")
        mn = -sc * (7.5 + 0.5 * torch.randn(sc.shape, generator=gen, device="cuda"))
        part[..., D // 2:] = torch.stack((sc, mn), -1).half().flatten(-2).view(torch.uint8)
    s["cache"] = cache
    return s


# --------------------------------------------------------------------------------- run

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _OWN[kind](state)
    return _PLAIN[kind](state)


def _own_linear_prefill(s):
    import gated_deltanet_linear_11_gb300 as gdn
    o, h = gdn.gdn_linear_prefill(s["q"], s["k"], s["v"], s["g"], s["cu"],
                                  initial_state=s["h0"], cu_seqlens_host=s["cu_host"])
    return {"o": o, "state": h}


def _own_linear_decode(s):
    import gated_deltanet_linear_11_gb300 as gdn
    o = gdn.gdn_linear_decode(s["q"], s["k"], s["v"], s["g"], s["state"], state_idx=s["idx"])
    return {"o": o, "state": s["state"]}


def _own_kv_append(s):
    import gated_deltanet_linear_11_gb300 as gdn
    q = gdn.gdn_kv_append(s["k"], s["v"], s["cache"], s["table"], s["kv_lens"], s["cu"],
                          cos=s["cos"], sin=s["sin"], q=s["q"],
                          interleaved=s["case"]["interleaved"], cu_seqlens_host=s["cu_host"])
    k, v = gdn.gdn_kv_read(s["cache"], s["table"], s["kv_lens"], s["cu"],
                           head_dim=s["case"]["D"], dtype=torch.float32,
                           cu_seqlens_host=s["cu_host"])
    return {"q": q, "k": k, "v": v}


def _own_kv_attention(s):
    import gated_deltanet_linear_11_gb300 as gdn
    return gdn.gdn_kv_attention(s["q"], s["cache"], s["table"], s["kv_lens"], s["cu"],
                                max_kv_len=max(s["lens"]), cu_seqlens_host=s["cu_host"])


_OWN = {"linear_prefill": _own_linear_prefill, "linear_decode": _own_linear_decode,
        "kv_append": _own_kv_append, "kv_attention": _own_kv_attention}


# ----------------------------------------------------------------- the plain forms

def _decay_rows(g, T):
    return g if g.dim() == 2 else g.expand(T, g.shape[0])


def _plain_linear_prefill(s):
    """Chunks of 64 tokens: the masked products inside a chunk, each chunk's own state, and
    every start state as a decayed sum of the states of the chunks before it."""
    C, D, Hk, Hv, n = 64, s["case"]["D"], s["case"]["Hk"], s["case"]["Hv"], s["case"]["n"]
    T, nc = s["q"].shape[0], -(-max(s["lens"]) // C)
    cu = s["cu"].long()
    pos = torch.arange(nc * C, device="cuda")
    at = (cu[:-1, None] + pos).clamp_(max=T - 1)                        # [n, nc C]
    real = pos < (cu[1:] - cu[:-1])[:, None]

    def chunks(x, width):       # packed [T, H, width] -> fp32 [n, nc, Hv, C, width]
        x = x.float()[at] * real[..., None, None]
        if x.shape[2] != Hv:
            x = x.repeat_interleave(Hv // x.shape[2], 2)
        return x.view(n, nc, C, Hv, width).transpose(2, 3)

    q, k, v = chunks(s["q"], D), chunks(s["k"], D), chunks(s["v"], D)
    g = chunks(_decay_rows(s["g"], T)[..., None], 1)[..., 0]            # [n, nc, Hv, C]
    upto = g.cumsum(-1)
    after = g.flip(-1).cumsum(-1).flip(-1) - g
    low = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    w = (upto[..., :, None] - upto[..., None, :]).masked_fill(~low, -math.inf).exp()
    o = ((q @ k.transpose(-1, -2)) * w) @ v
    own_state = (k * after.exp()[..., None]).transpose(-1, -2) @ v      # [n, nc, Hv, D, D]
    # sums of the chunks' log decays over the chunks c' < m < c, for starts c = 0 .. nc
    total = upto[..., -1].transpose(1, 2)                               # [n, Hv, nc]
    c = torch.arange(nc, device="cuda")
    seg = (total[..., :, None] * (c[:, None] > c[None, :])).cumsum(-2)  # over c' < m <= row
    seg = seg.masked_fill(c[:, None] < c[None, :], -math.inf).exp()
    part = seg @ own_state.transpose(1, 2).reshape(n, Hv, nc, D * D)    # starts 1 .. nc
    if s["h0"] is not None:
        part = part + total.cumsum(-1).exp()[..., None] * s["h0"].reshape(n, Hv, 1, D * D)
        first = s["h0"].reshape(n, Hv, 1, D * D)
    else:
        first = torch.zeros_like(part[:, :, :1])
    start = torch.cat((first, part[:, :, :-1]), 2).view(n, Hv, nc, D, D).transpose(1, 2)
    o = o + (q * upto.exp()[..., None]) @ start
    o = o.transpose(2, 3).reshape(n, nc * C, Hv, D)[real]
    return {"o": o.to(s["q"].dtype), "state": part[:, :, -1].reshape(n, Hv, D, D)}


def _plain_linear_decode(s):
    n, Hv = s["case"]["n"], s["case"]["Hv"]
    G = Hv // s["case"]["Hk"]
    q, k = (s[x].float().repeat_interleave(G, 1) for x in "qk")
    a = _decay_rows(s["g"], n).exp()
    idx = s["idx"].long()
    h = s["state"][idx] * a[..., None, None] + k[..., :, None] * s["v"].float()[..., None, :]
    s["state"][idx] = h
    o = (q[..., None, :] @ h)[..., 0, :]
    return {"o": o.to(s["q"].dtype), "state": s["state"]}


def _orders(D):
    """Element held by each nibble of a key record and of a value record."""
    x = torch.arange(D, device="cuda")
    W, i, ng = x // 8, x % 8, D // _GROUP
    return (32 * (W % ng) + 8 * (W // ng) + i,
            64 * (W // 8) + 32 * (i // 4) + 4 * (W % 8) + i % 4)


def _rotate(x, cos, sin, interleaved):
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    r = x[..., :2 * half]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def _quantize(x, order):
    """Records of x [T, H, D]: codes in storage order, then the scales and minima."""
    T, H, D = x.shape
    x = x.clamp(-65504.0, 65504.0).view(T, H, D // _GROUP, _GROUP)
    mn = x.amin(-1, keepdim=True).half()
    sc = ((x.amax(-1, keepdim=True) - mn.float()) * (1.0 / 15.0)).half()
    inv = torch.where(sc > 0, 1.0 / sc.float(), torch.zeros_like(sc, dtype=torch.float32))
    u = ((x - mn.float()) * inv).round().clamp(0, 15).to(torch.uint8).view(T, H, D)[..., order]
    codes = u[..., 0::2] | (u[..., 1::2] << 4)
    return torch.cat((codes, torch.cat((sc, mn), -1).flatten(-2).view(torch.uint8)), -1)


def _values(rec, order):
    """fp32 values of records [..., D/2 + D/8]."""
    D = order.numel()
    codes = rec[..., :D // 2]
    u = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)[..., order.argsort()].float()
    sm = rec[..., D // 2:].contiguous().view(torch.float16).float()
    u = u.unflatten(-1, (D // _GROUP, _GROUP))
    return (sm[..., 0::2, None] * u + sm[..., 1::2, None]).flatten(-2)


def _row_positions(s):
    """Sequence and position of each of the packed new tokens."""
    cu, T = s["cu"].long(), s["q"].shape[0]
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu[1:], t, right=True)
    return seq, s["kv_lens"].long()[seq] - (cu[1:][seq] - t)


def _plain_kv_append(s):
    page, D = s["case"]["page"], s["case"]["D"]
    seq, pos = _row_positions(s)
    cos, sin = s["cos"][pos], s["sin"][pos]
    inter = s["case"]["interleaved"]
    order_k, order_v = _orders(D)
    at, slot = s["table"][seq, pos // page].long(), pos % page
    s["cache"][at, 0, :, slot] = _quantize(_rotate(s["k"].float(), cos, sin, inter), order_k)
    s["cache"][at, 1, :, slot] = _quantize(s["v"].float(), order_v)
    q = _rotate(s["q"].float(), cos, sin, inter).to(s["q"].dtype)
    return {"q": q, "k": _values(s["cache"][at, 0, :, slot], order_k),
            "v": _values(s["cache"][at, 1, :, slot], order_v)}


def _plain_kv_attention(s):
    D, Hq, Hkv, n, m = (s["case"][x] for x in ("D", "Hq", "Hkv", "n", "m"))
    G, page = Hq // Hkv, s["case"]["page"]
    order_k, order_v = _orders(D)
    used = -(-max(s["lens"]) // page)
    rec = s["cache"][s["table"][:, :used].long()]               # [n, used, 2, Hkv, page, rec]
    k = _values(rec[:, :, 0], order_k).transpose(1, 2).reshape(n, Hkv, used * page, D)
    v = _values(rec[:, :, 1], order_v).transpose(1, 2).reshape(n, Hkv, used * page, D)
    q = s["q"].float().view(n, m, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(n, Hkv, G * m, D)
    sc = (q @ k.transpose(-1, -2)) * D ** -0.5
    i, j = torch.arange(m, device="cuda"), torch.arange(used * page, device="cuda")
    hidden = j > (s["kv_lens"].long()[:, None, None] - m + i[:, None])      # [n, m, keys]
    sc = sc.view(n, Hkv, G, m, -1).masked_fill_(hidden[:, None, None], -math.inf)
    p = sc.sub_(sc.amax(-1, keepdim=True)).exp_()
    o = (p.view(n, Hkv, G * m, -1) @ v).view(n, Hkv, G, m, D) / p.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).reshape(n * m, Hq, D).to(s["q"].dtype)


_PLAIN = {"linear_prefill": _plain_linear_prefill, "linear_decode": _plain_linear_decode,
          "kv_append": _plain_kv_append, "kv_attention": _plain_kv_attention}


# -------------------------------------------------------------------------------- work

def work(case):
    e, D, kind = (2 if case["dtype"] == "bf16" else 4), case["D"], case["kind"]
    if kind in ("linear_prefill", "linear_decode"):
        Hk, Hv, n = case["Hk"], case["Hv"], case["n"]
        T = sum(_lens(case)) if kind == "linear_prefill" else n
        states = 2 if kind == "linear_decode" or case["start"] else 1
        gate = 4 * (T * Hv if case["decay"] == "token" else Hv)
        return {"bytes": e * T * (2 * Hk + 2 * Hv) * D + gate + states * n * Hv * D * D * 4,
                "flops": 4 * T * Hv * D * D}
    Hq, Hkv, rec = case["Hq"], case["Hkv"], case["D"] // 2 + case["D"] // 8
    if kind == "kv_append":
        T = sum(_lens(case, "q_lo", "q_hi"))
        # q and k, v in; q and the records out; the records in again, their values out
        return {"bytes": T * (2 * e * (Hq + Hkv) * D + 4 * case["rot"]
                              + 2 * 2 * Hkv * rec + 2 * 4 * Hkv * D),
                "flops": T * (3 * (Hq + Hkv) * case["rot"] + 10 * Hkv * D)}
    m, lens = case["m"], [max(x, case["m"]) for x in _lens(case)]
    seen = sum(m * x - m * (m - 1) // 2 for x in lens)
    return {"bytes": sum(lens) * 2 * Hkv * rec + 2 * e * case["n"] * m * Hq * D,
            "flops": 4 * seen * Hq * D}


# ------------------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["kind"]](s, case)


def _exact_linear_prefill(s, case):
    """The recurrence, token by token, over all sequences and heads at once."""
    lens, Hv, D, n = s["lens"], case["Hv"], case["D"], case["n"]
    G, T = Hv // case["Hk"], sum(lens)
    h = torch.zeros(n, Hv, D, D, dtype=torch.float64, device="cuda")
    if s["h0"] is not None:
        h += s["h0"]
    a = torch.exp(s["g"].double())
    a = a if a.dim() == 2 else a.expand(T, Hv)
    first = s["cu_host"][:-1].tolist()
    o = torch.empty(T, Hv, D, dtype=torch.float64, device="cuda")
    by_len = sorted(range(n), key=lambda i: -lens[i])
    h = h[by_len]
    rows = torch.tensor([first[i] for i in by_len], device="cuda")
    q, k, v = s["q"], s["k"], s["v"]
    live = n
    for t in range(max(lens)):
        while lens[by_len[live - 1]] <= t:
            live -= 1
        r, hl = rows[:live] + t, h[:live]
        kt = k[r].double().repeat_interleave(G, 1)
        qt = q[r].double().repeat_interleave(G, 1)
        hl.mul_(a[r][..., None, None]).addcmul_(kt[..., :, None], v[r].double()[..., None, :])
        o[r] = torch.matmul(qt[..., None, :], hl)[..., 0, :]
    back = torch.empty_like(h)
    back[by_len] = h
    return {"o": o, "state": back}


def _exact_linear_decode(s, case):
    G = case["Hv"] // case["Hk"]
    st, o = s["state"].double(), []
    for i, at in enumerate(s["idx"].tolist()):
        a = torch.exp((s["g"][i] if s["g"].dim() == 2 else s["g"]).double())
        k = s["k"][i].double().repeat_interleave(G, 0)
        q = s["q"][i].double().repeat_interleave(G, 0)
        st[at] = a[:, None, None] * st[at] + torch.einsum("hi,hj->hij", k, s["v"][i].double())
        o.append(torch.einsum("hi,hij->hj", q, st[at]))
    return {"o": torch.stack(o), "state": st}


def _exact_kv_append(s, case):
    """Rotation in 64 bits; stored values by the format's definition (fp16 minimum and
    scale of each 32 elements, nearest of 16 levels)."""
    half, inter, D = case["rot"] // 2, case["interleaved"], case["D"]
    pos = torch.cat([torch.arange(L - m, L) for L, m in zip(s["lens"], s["m"])]).cuda()
    z = torch.complex(s["cos"][pos].double(), s["sin"][pos].double())[:, None]

    def turn(x):
        x = x.double().clone()
        if inter:
            y = torch.complex(x[..., 0:2 * half:2], x[..., 1:2 * half:2]) * z
            x[..., 0:2 * half:2], x[..., 1:2 * half:2] = y.real, y.imag
        else:
            y = torch.complex(x[..., :half], x[..., half:2 * half]) * z
            x[..., :half], x[..., half:2 * half] = y.real, y.imag
        return x

    def stored(x):
        g = x.reshape(-1, 32)
        low = g.min(1, keepdim=True).values.float().half().double()
        step = ((g.max(1, keepdim=True).values - low) / 15).float().half().double()
        level = torch.where(step > 0, torch.round((g - low) / step), 0.0).clamp(0, 15)
        return (low + step * level).reshape(x.shape)

    return {"q": turn(s["q"]), "k": stored(turn(s["k"])), "v": stored(s["v"].double())}


def _exact_kv_attention(s, case):
    D, Hkv, m, page = case["D"], case["Hkv"], case["m"], case["page"]
    G = case["Hq"] // Hkv
    place_k = [32 * ((x // 8) % (D // 32)) + 8 * ((x // 8) // (D // 32)) + x % 8 for x in range(D)]
    place_v = [64 * (x // 64) + 32 * ((x % 8) // 4) + 4 * ((x // 8) % 8) + x % 4 for x in range(D)]
    out = []
    for i, L in enumerate(s["lens"]):
        rec = s["cache"][s["table"][i, :-(-L // page)].long()]
        rec = rec.permute(1, 2, 0, 3, 4).reshape(2, Hkv, -1, rec.shape[-1])[:, :, :L]
        q = s["q"][i * m:(i + 1) * m].double()
        heads = []
        for h in range(Hkv):
            kv = []
            for which, place in ((0, place_k), (1, place_v)):
                b = rec[which, h]
                x = torch.empty(L, D, dtype=torch.float64, device="cuda")
                x[:, place[0::2]] = (b[:, :D // 2] % 16).double()
                x[:, place[1::2]] = (b[:, :D // 2] // 16).double()
                p = b[:, D // 2:].contiguous().view(torch.float16).double().view(L, D // 32, 2)
                kv.append(x * p[..., 0].repeat_interleave(32, 1) + p[..., 1].repeat_interleave(32, 1))
            sc = torch.einsum("mgd,ld->gml", q[:, h * G:(h + 1) * G], kv[0]) / math.sqrt(D)
            last = torch.arange(L - m, L, device="cuda")[:, None]
            sc[:, torch.arange(L, device="cuda")[None] > last] = -math.inf
            heads.append(torch.einsum("gml,ld->mgd", torch.softmax(sc, -1), kv[1]))
        out.append(torch.cat(heads, 1))
    return torch.cat(out)


_EXACT = {"linear_prefill": _exact_linear_prefill, "linear_decode": _exact_linear_decode,
          "kv_append": _exact_kv_append, "kv_attention": _exact_kv_attention}
