"""Workloads of the library's operators around the token mixers: norms and products in 8 bits.

Five kinds of case, each a call (or the run of calls) that a serving program makes:

* ``add_rmsnorm``    gdn_add_rmsnorm: residual addition and root-mean-square norm, out in the
                     activations' type or in 8 bits with a scale for each row.
* ``gated_rmsnorm``  gdn_gated_rmsnorm: the Gated DeltaNet layer's output norm (per head) times
                     silu(z), likewise.
* ``quantize_rows``  gdn_quantize_rows: rows to 8 bits with a scale each.
* ``matmul_i8``      gdn_matmul_i8: product of 8-bit integers with a scale for each token and
                     channel.
* ``project``        gdn_add_rmsnorm in 8 bits, then gdn_matmul_i8 of its rows.

``run`` computes a case through the library when ``own`` is true, and in elementary torch
operations (32-bit arithmetic, one rounding at the end) when it is false.  ``exact`` gives
the same outputs from the definitions in 64 bits.  Rows in 8 bits are returned as the values
they stand for, code times scale, in bf16 (which holds more digits than a code has); over a
row, scale = max|y| / 127 and code = 127 y / max|y| rounded to the nearest integer (even at
ties).
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_TINY = 2.0 ** -126         # the smallest scale: of a row of zeros
_EPS = 1e-6


# ------------------------------------------------------------------------------- cases

def listed():
    nr = dict(kind="add_rmsnorm", dtype="bf16", T=1, D=5120, residual=True, offset=1.0,
              eight=False)
    gt = dict(kind="gated_rmsnorm", dtype="bf16", T=1, H=48, D=128, eight=True)
    qr = dict(kind="quantize_rows", dtype="bf16", T=1, D=5120)
    mm = dict(kind="matmul_i8", dtype="bf16", M=1, N=5120, K=6144, bias=False)
    return [
        # the norm in front of a decode step's projections, four sequences: latency
        dict(nr, name="norm, 4 tokens to 8 bits", T=4, eight=True),
        # the norm of a 4096-token prompt, kept in the activations' type
        dict(nr, name="norm, 4096 tokens", T=4096),
        # fp32 activations of an odd width, ragged tokens, no residual yet (the first layer)
        dict(nr, name="norm, fp32", dtype="fp32", T=777, D=2047, residual=False, offset=0.0),
        # the layer's output norm in a decode batch, for an 8-bit output projection
        dict(gt, name="gated norm, 64 tokens to 8 bits", T=64),
        # the same for a 4096-token prompt, kept in the activations' type
        dict(gt, name="gated norm, 4096 tokens", T=4096, eight=False),
        # outputs of an attention layer, a ragged batch
        dict(qr, name="rows to 8 bits, 300 tokens", T=300, D=6144),
        # the input projection's weights, when a model is loaded
        dict(qr, name="rows to 8 bits, weights", T=10240),
        # the output projection of one token: reading the weights
        dict(mm, name="product, 1 token"),
        # the input projections (q, k, v, z and gates together) of a decode batch
        dict(mm, name="product, 64 tokens", M=64, N=16480, K=5120),
        # odd sizes in fp32 with a bias
        dict(mm, name="product, odd sizes", dtype="fp32", M=333, N=515, K=1001, bias=True),
        # the input projections of a 4096-token prompt
        dict(mm, name="product, 4096 tokens", M=4096, N=16480, K=5120),
        # norm and q, k, v projection of ragged short prompts
        dict(kind="project", name="norm and product, 500 tokens", dtype="bf16", M=500, N=10240,
             K=5120),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _width(rng, lo, hi):
    """A row's length: mostly a multiple of 64, else any."""
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.3 else max(64, n // 64 * 64)


def draw(rng):
    kind = rng.choice(["add_rmsnorm", "gated_rmsnorm", "quantize_rows", "matmul_i8",
                       "matmul_i8", "matmul_i8", "project"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    c = dict(kind=kind, dtype=dtype)
    most = 4096 * 5120 // (2 if dtype == "fp32" else 1)       # elements of a norm
    if kind == "add_rmsnorm":
        D = _width(rng, 17, 16384)
        return dict(c, D=D, T=_log_int(rng, 1, min(8192, most // D)),
                    residual=rng.random() < 0.7, offset=rng.choice([0.0, 1.0]),
                    eight=rng.random() < 0.5)
    if kind == "gated_rmsnorm":
        H, D = rng.choice([(1, 64), (8, 64), (6, 128), (32, 128), (48, 128), (16, 256)])
        return dict(c, H=H, D=D, T=_log_int(rng, 1, min(8192, most // (H * D))),
                    eight=rng.random() < 0.5)
    if kind == "quantize_rows":
        D = _width(rng, 17, 16384)
        return dict(c, D=D, T=_log_int(rng, 1, min(16384, 2 * most // D)))
    M, N, K = _log_int(rng, 1, 4096), _width(rng, 16, 16480), _width(rng, 64, 8192)
    K = min(K, 4096 * 16480 * 5120 // (M * N))
    if kind == "project":       # bf16 as served: a code next to a border may fall either way
        return dict(c, dtype="bf16", M=M, N=N, K=K)
    return dict(c, M=M, N=N, K=K, bias=rng.random() < 0.3)


# ------------------------------------------------------------------------------ inputs

def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _residual_stream(gen, T, D):
    """Activations between layers: a few channels far larger than the rest, and rows of
    different sizes."""
    channels = 1 + 30 * torch.rand(D, generator=gen, device="cuda") ** 24
    return _randn(gen, T, D) * channels * torch.exp(0.5 * _randn(gen, T, 1))


def _eight_bit(x):
    """Rows in 8 bits as a program holds them."""
    scale = x.abs().amax(-1).clamp_min(127 * _TINY) / 127
    return (x / scale[:, None]).round_().to(torch.int8), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, kind = _DT[case["dtype"]], case["kind"]
    s = dict(case=case)
    if kind == "add_rmsnorm":
        T, D = case["T"], case["D"]
        s["x"] = _randn(gen, T, D).to(dt)
        s["residual"] = _residual_stream(gen, T, D).to(dt) if case["residual"] else None
        s["weight"] = (1 - case["offset"] + 0.2 * _randn(gen, D)).to(dt)
    elif kind == "gated_rmsnorm":
        T, H, D = case["T"], case["H"], case["D"]
        s["x"] = (_randn(gen, T, H, D) * torch.exp(_randn(gen, T, H, 1))).to(dt)
        # z is a part of the input projection's rows
        rows = _randn(gen, T, 2 * H * D).to(dt)
        s["z"] = rows[:, H * D:].view(T, H, D)
        s["weight"] = (1 + 0.2 * _randn(gen, D)).to(dt)
    elif kind == "quantize_rows":
        s["x"] = _residual_stream(gen, case["T"], case["D"]).to(dt)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        if kind == "project":
            s["x"] = _randn(gen, M, K).to(dt)
            s["residual"] = _residual_stream(gen, M, K).to(dt)
            s["weight"] = (0.2 * _randn(gen, K)).to(dt)
            s["bias"] = None
        else:
            s["a"], s["a_scale"] = _eight_bit(_randn(gen, M, K))
            s["bias"] = _randn(gen, N) if case["bias"] else None
        s["w"], s["w_scale"] = _eight_bit(_randn(gen, N, K) * K ** -0.5)
    return s


# --------------------------------------------------------------------------------- run

def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["kind"]](state)


def _values(code, scale):
    out = torch.empty(code.shape, dtype=torch.bfloat16, device=code.device)
    return torch.mul(code, scale[:, None], out=out)


def _own_add_rmsnorm(s):
    import gated_deltanet_linear_11_gb300 as gdn
    c = s["case"]
    y, residual = gdn.gdn_add_rmsnorm(s["x"], s["weight"], s["residual"], eps=_EPS,
                                      weight_offset=c["offset"], eight_bit=c["eight"])
    if c["eight"]:
        y = _values(*y)
    return {"y": y, "residual": residual} if c["residual"] else {"y": y}


def _own_gated_rmsnorm(s):
    import gated_deltanet_linear_11_gb300 as gdn
    y = gdn.gdn_gated_rmsnorm(s["x"], s["z"], s["weight"], eps=_EPS,
                              eight_bit=s["case"]["eight"])
    return {"y": _values(*y) if s["case"]["eight"] else y}


def _own_quantize_rows(s):
    import gated_deltanet_linear_11_gb300 as gdn
    return {"values": _values(*gdn.gdn_quantize_rows(s["x"]))}


def _own_matmul_i8(s):
    import gated_deltanet_linear_11_gb300 as gdn
    return {"out": gdn.gdn_matmul_i8(s["a"], s["a_scale"], s["w"], s["w_scale"], bias=s["bias"],
                                     dtype=_DT[s["case"]["dtype"]])}


def _own_project(s):
    import gated_deltanet_linear_11_gb300 as gdn
    (q, scale), residual = gdn.gdn_add_rmsnorm(s["x"], s["weight"], s["residual"], eps=_EPS,
                                               weight_offset=1.0, eight_bit=True)
    return {"out": gdn.gdn_matmul_i8(q, scale, s["w"], s["w_scale"],
                                     dtype=_DT[s["case"]["dtype"]]),
            "residual": residual}


_OWN = {"add_rmsnorm": _own_add_rmsnorm, "gated_rmsnorm": _own_gated_rmsnorm,
        "quantize_rows": _own_quantize_rows, "matmul_i8": _own_matmul_i8,
        "project": _own_project}


# ----------------------------------------------------------------- the plain forms

def _plain_codes(y):
    largest = y.abs().amax(-1, keepdim=True).clamp_min(127 * _TINY)
    return (127 * y / largest).round(), largest / 127


def _values_of(y):
    code, scale = _plain_codes(y)
    return (code * scale).bfloat16()


def _plain_norm(s, offset):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + _EPS)
    return y * (offset + s["weight"].float()), h.to(s["x"].dtype)


def _plain_add_rmsnorm(s):
    c = s["case"]
    y, h = _plain_norm(s, c["offset"])
    if c["eight"]:
        y = _values_of(y)
    else:
        y = y.to(s["x"].dtype)
    return {"y": y, "residual": h} if c["residual"] else {"y": y}


def _plain_gated_rmsnorm(s):
    x, z = s["x"].float(), s["z"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * s["weight"].float()
    y = (y * (z / (1 + torch.exp(-z)))).flatten(1)
    return {"y": _values_of(y) if s["case"]["eight"] else y.to(s["x"].dtype)}


def _plain_quantize_rows(s):
    return {"values": _values_of(s["x"].float())}


def _plain_product(a, a_scale, s):
    out = (a @ s["w"].float().t()) * a_scale * s["w_scale"]
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(_DT[s["case"]["dtype"]])


def _plain_matmul_i8(s):
    return {"out": _plain_product(s["a"].float(), s["a_scale"][:, None], s)}


def _plain_project(s):
    y, h = _plain_norm(s, 1.0)
    return {"out": _plain_product(*_plain_codes(y), s), "residual": h}


_PLAIN = {"add_rmsnorm": _plain_add_rmsnorm, "gated_rmsnorm": _plain_gated_rmsnorm,
          "quantize_rows": _plain_quantize_rows, "matmul_i8": _plain_matmul_i8,
          "project": _plain_project}


# -------------------------------------------------------------------------------- work

def work(case):
    e, kind = (2 if case["dtype"] == "bf16" else 4), case["kind"]
    if kind in ("add_rmsnorm", "gated_rmsnorm", "quantize_rows"):
        T, D = case["T"], case["D"] * case.get("H", 1)
        # a row in 8 bits is written, read again, and written as values
        eight = kind == "quantize_rows" or case["eight"]
        out = 1 + 1 + 2 if eight else e
        reads = {"add_rmsnorm": 1 + case.get("residual", 0), "gated_rmsnorm": 2,
                 "quantize_rows": 1}[kind]
        writes = case.get("residual", 0)
        return {"bytes": T * D * (e * (reads + writes) + out), "flops": 8 * T * D}
    M, N, K = case["M"], case["N"], case["K"]
    moved = K * (M + N) + 4 * (M + N) + e * M * N
    if kind == "project":       # x, residual in, residual and the codes out
        moved += M * K * (3 * e + 1)
    return {"bytes": moved, "flops": 2 * M * N * K}


# ------------------------------------------------------------------------------- exact

def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) else v
         for k, v in prepare(case, seed).items()}
    kind = case["kind"]
    if kind == "quantize_rows":
        return {"values": _nearest_codes(s["x"])}
    if kind == "gated_rmsnorm":
        rms = (s["x"].pow(2).sum(-1) / case["D"] + _EPS).sqrt()
        y = s["x"] / rms[..., None] * s["weight"] * s["z"] * torch.sigmoid(s["z"])
        y = y.reshape(case["T"], -1)
        return {"y": _nearest_codes(y) if case["eight"] else y}
    if kind == "matmul_i8":
        out = torch.einsum("mk,nk->mn", s["a"], s["w"])
        out = torch.outer(s["a_scale"], s["w_scale"]) * out
        return {"out": out if s["bias"] is None else s["bias"] + out}
    h = s["x"] if s["residual"] is None else s["x"] + s["residual"]
    rms = (h.pow(2).sum(-1) / h.shape[-1] + _EPS).sqrt()
    y = (s["weight"] + case.get("offset", 1.0)) * h / rms[:, None]
    if kind == "project":
        out = torch.einsum("mk,nk->mn", _nearest_codes(y), s["w"]) * s["w_scale"]
        return {"out": out, "residual": h}
    out = {"y": _nearest_codes(y) if case["eight"] else y}
    return dict(out, residual=h) if case["residual"] else out


def _nearest_codes(y):
    largest = y.abs().max(-1).values[:, None]
    steps = torch.round(127 * y / torch.where(largest > 0, largest, 1.0))
    return steps * largest / 127
