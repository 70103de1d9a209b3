"""The paged 4-bit cache: what is stored, what is read back, and attention over it.

Bounds: stored bytes are exact (the format's arithmetic is fixed).  Attention, with
A = sum p |v| / sum p in 64 bits over the stored values: bf16 o within its own rounding
(2^-8 |o|) plus 2^-9 A (weights rounded twice to fp16, 2 * 2^-11, and the rest for fp32
scores below 64 in size, whose error of about 2^-24 * 64 * 4 passes through exp); fp32 o
within 2^-16 A (the same scores in fp32 and sums of up to 5000 terms); lse within 1e-4.
"""
import numpy as np
import pytest
import torch

import linear_ref as ref
from gpu_util import assert_bits_equal, np64

pytestmark = pytest.mark.gpu

gdn = pytest.importorskip("gated_deltanet_linear_11_gb300")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load()


def tables(rng, lens, page, extra=2):
    need = [max(1, -(-int(x) // page)) for x in lens]
    perm = rng.permutation(sum(need) + extra).astype(np.int32)
    table = np.full((len(lens), max(need) + 1), -7, np.int32)     # unused entries are never read
    at = 0
    for n, c in enumerate(need):
        table[n, :c] = perm[at:at + c]
        at += c
    return table, sum(need) + extra


def offsets(ms):
    return torch.tensor(np.concatenate(([0], np.cumsum(ms))), dtype=torch.int32)


def append_case(seed, D, Hq, Hkv, page, ms, lens, dtype, rot, interleaved):
    rng = np.random.default_rng(seed)
    T = sum(ms)
    table, pages = tables(rng, lens, page)

    def rnd(h):
        return torch.from_numpy(rng.standard_normal((T, h, D)).astype(np.float32)).to(dtype)
    c = dict(q=rnd(Hq), k=rnd(Hkv) * 3, v=rnd(Hkv), table=table, pages=pages, ms=ms, lens=lens,
             page=page, D=D, Hkv=Hkv, interleaved=interleaved, cos=None, sin=None)
    if rot:
        ang = np.arange(max(lens))[:, None] * 100.0 ** (-np.arange(rot // 2) / (rot // 2))
        c["cos"] = torch.from_numpy(np.cos(ang).astype(np.float32))
        c["sin"] = torch.from_numpy(np.sin(ang).astype(np.float32))
    return c


def positions(c):
    seq = np.concatenate([np.full(m, n) for n, m in enumerate(c["ms"])]).astype(int)
    pos = np.concatenate([np.arange(L - m, L) for m, L in zip(c["ms"], c["lens"])]).astype(int)
    return seq, pos


def run_append(c, cache=None, **kw):
    if cache is None:
        cache = gdn.gdn_kv_cache(c["pages"], c["page"], c["Hkv"], c["D"])
        cache.fill_(0xAB)
    one = all(m == 1 for m in c["ms"])
    cu = offsets(c["ms"])
    q_out = gdn.gdn_kv_append(
        c["k"].cuda(), c["v"].cuda(), cache, torch.from_numpy(c["table"]).cuda(),
        torch.tensor(c["lens"], dtype=torch.int32).cuda(), None if one else cu.cuda(),
        cos=None if c["cos"] is None else c["cos"].cuda(),
        sin=None if c["sin"] is None else c["sin"].cuda(), q=c["q"].cuda(),
        interleaved=c["interleaved"], cu_seqlens_host=None if one else cu, **kw)
    return cache, q_out


@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (128, 128, False), (128, 32, True),
                                               (256, 256, True), (256, 64, False), (128, 0, False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,ms,lens", [(16, [1, 1, 1], [1, 17, 40]),
                                          (32, [5, 0, 33, 1], [5, 3, 70, 64])])
def test_append_stores_exactly(D, rot, interleaved, dtype, page, ms, lens):
    c = append_case(1, D, 6, 2, page, ms, lens, dtype, rot, interleaved)
    cache, q_out = run_append(c)
    seq, pos = positions(c)
    want = np.full(tuple(cache.shape), 0xAB, np.uint8)
    k, v, q = (c[x].float().numpy() for x in "kvq")
    if rot:
        k, q = (ref.rotate32(x, c["cos"].numpy()[pos], c["sin"].numpy()[pos], interleaved)
                for x in (k, q))
    at = c["table"][seq, pos // page]
    want[at, 0, :, pos % page] = ref.records(k, ref.key_order(D))
    want[at, 1, :, pos % page] = ref.records(v, ref.value_order(D))
    got = cache.cpu().numpy()
    assert np.array_equal(got, want), "%d bytes differ" % int((got != want).sum())
    assert_bits_equal(q_out, torch.from_numpy(q).to(dtype).cuda(), "rotated q")
    for out in (torch.float32, torch.bfloat16):
        cu = offsets(ms)
        rk, rv = gdn.gdn_kv_read(cache, torch.from_numpy(c["table"]).cuda(),
                                 torch.tensor(lens, dtype=torch.int32).cuda(), cu.cuda(),
                                 head_dim=D, dtype=out, cu_seqlens_host=cu)
        for name, x, order in (("k", rk, ref.key_order(D)), ("v", rv, ref.value_order(D))):
            val = ref.values(got[at, 0 if name == "k" else 1, :, pos % page], order)
            # scale * code has 15 bits, so the sum's one rounding is the exact value's
            assert_bits_equal(x, torch.from_numpy(val).float().to(out).cuda(), "read " + name)


def test_append_special_values():
    """Constant groups, subnormal ranges, values past fp16, infinities and NaN."""
    D = 128
    c = append_case(2, D, 2, 1, 16, [6], [6], torch.float32, 0, False)
    k = c["k"]
    k[0] = 3.25
    k[1] = 0.0
    k[2] *= 1e-7
    k[3] *= 1e6
    k[4, 0, 5] = float("inf")
    k[4, 0, 40] = -float("inf")
    k[5, 0, 70] = float("nan")
    cache, _ = run_append(c)
    rk, _ = gdn.gdn_kv_read(cache, torch.from_numpy(c["table"]).cuda(),
                            torch.tensor([6], dtype=torch.int32).cuda(), offsets([6]).cuda(),
                            head_dim=D, dtype=torch.float32)
    got = cache.cpu().numpy()
    page = c["table"][0, 0]
    assert np.array_equal(got[page, 0, 0, :6], ref.records(k[:, 0].numpy(), ref.key_order(D)))
    rk = rk[:, 0].cpu()
    assert bool((rk[0] == 3.25).all()) and not bool(rk[1].any())
    # the scale's rounding (2^-11 of at most 131008) may carry the top level past 65504
    assert bool(rk[:5].isfinite().all()) and float(rk[3].abs().max()) <= 65504 + 64
    nan = rk[5].isnan()
    assert bool(nan[64:96].all()) and not bool(nan[:64].any()) and not bool(nan[96:].any())


def test_append_skips_and_reports_rows_without_a_place():
    D = 64
    for what in ("page", "position", "table", "angles"):
        c = append_case(3, D, 2, 2, 16, [3, 2], [20, 30], torch.bfloat16, 64, False)
        good, _ = run_append(c)
        if what == "page":
            c["table"][1, 1] = c["pages"]
        elif what == "position":
            c["lens"] = [20, 1]                    # the first of two rows lies before 0
        elif what == "table":
            c["lens"] = [20, 16 * c["table"].shape[1] + 1]
        else:
            c["cos"], c["sin"] = c["cos"][:25].contiguous(), c["sin"][:25].contiguous()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        cache, _ = run_append(c, status=status)
        assert int(status) == 10, what
        pages = c["table"][0, :2]
        assert_bits_equal(cache[pages.tolist()], good[pages.tolist()], "the other sequence")


def test_append_from_strided_views_and_its_refusals():
    c = append_case(4, 128, 4, 2, 16, [7], [7], torch.bfloat16, 128, False)
    good, q1 = run_append(c)
    T = 7
    y = torch.cat([c[x].reshape(T, -1) for x in "qkv"], 1).cuda()
    table, lens = torch.from_numpy(c["table"]).cuda(), torch.tensor([7], dtype=torch.int32).cuda()
    q, k, v = y[:, :512].unflatten(1, (4, 128)), y[:, 512:768].unflatten(1, (2, 128)), \
        y[:, 768:].unflatten(1, (2, 128))
    cache = torch.full_like(good, 0xAB)
    cos, sin = c["cos"].cuda(), c["sin"].cuda()
    cu = offsets([7]).cuda()
    q2 = gdn.gdn_kv_append(k, v, cache, table, lens, cu, cos=cos, sin=sin, q=q)
    assert_bits_equal(cache, good, "cache from views")
    assert_bits_equal(q1, q2, "q from views")

    def code(**kw):
        a = dict(k=k, v=v, cache=cache, block_table=table, kv_lens=lens, cu_seqlens=cu, cos=cos,
                 sin=sin, q=q)
        a.update(kw)
        with pytest.raises((gdn.GdnError, ValueError)) as e:
            gdn.gdn_kv_append(**a)
        return getattr(e.value, "code", "value")
    assert code(q_out=q) == 3                                     # in place
    assert code(v=v.float()) == 4
    assert code(cos=cos[:, :12].contiguous(), sin=sin[:, :12].contiguous()) == 6
    assert code(sin=None) == "value"
    assert code(cache=cache[:, :, :, :8].contiguous()) == 6       # pages of 8 tokens
    assert code(cache=cache[..., :40].contiguous()) == "value"
    assert code(kv_lens=lens.long()) == "value"
    assert code(cu_seqlens=None) == "value"
    assert code(k=k[:, :1]) in (2, 3)


# ------------------------------------------------------------------------- attention

def attention_case(seed, D, Hq, Hkv, page, ms, lens, dtype=torch.bfloat16, spread=1.0):
    rng = np.random.default_rng(seed)
    table, pages = tables(rng, lens, page)
    rec = D // 2 + D // 8
    cache = rng.integers(0, 256, (pages, 2, Hkv, page, rec)).astype(np.uint8)
    sc = (0.2 + 0.2 * rng.random((pages, 2, Hkv, page, D // 32))).astype(np.float16)
    mn = (-sc * (7.5 + rng.standard_normal(sc.shape))).astype(np.float16)
    cache[..., D // 2:] = np.ascontiguousarray(np.stack((sc, mn), -1)).reshape(
        sc.shape[:-1] + (-1,)).view(np.uint8)
    # what lies past a sequence's end holds NaN and infinities
    for n, L in enumerate(lens):
        for p in range(max(int(L), 0), max(1, -(-int(L) // page)) * page):
            cache[table[n, p // page], :, :, p % page] = 0xFF if p % 2 else 0x7C
    q = torch.from_numpy((spread * rng.standard_normal((sum(ms), Hq, D))).astype(np.float32)).to(dtype)
    return dict(q=q, cache=cache, table=table, lens=np.array(lens, np.int32), ms=ms, D=D)


def run_attention(c, simt=False, **kw):
    cu = offsets(c["ms"])
    one = all(m == 1 for m in c["ms"])
    T, Hq, D = c["q"].shape
    lse = torch.full((T, Hq), 7.0, device="cuda")
    o = gdn.gdn_kv_attention(c["q"].cuda(), torch.from_numpy(c["cache"]).cuda(),
                             torch.from_numpy(c["table"]).cuda(),
                             torch.from_numpy(c["lens"]).cuda(), None if one else cu.cuda(),
                             lse=lse, simt=simt, cu_seqlens_host=None if one else cu, **kw)
    return o, lse


def check_attention(c, o, lse, scale=None):
    scale = c["D"] ** -0.5 if scale is None else scale
    ro, rl, oa = ref.attention(np64(c["q"]), c["cache"], c["table"], c["lens"],
                               offsets(c["ms"]).tolist(), scale)
    lim = 2.0 ** -16 * oa if c["q"].dtype == torch.float32 else \
        ref.U_BF16 * np.abs(ro) + 2.0 ** -9 * oa
    err = np.abs(np64(o) - ro)
    assert np.all(err <= lim), "o: %.3g of its bound" % float(np.nanmax(err / (lim + 1e-30)))
    got = np64(lse)
    empty = np.isinf(rl)
    assert np.array_equal(empty, np.isinf(got)) and np.all(got[empty] < 0)
    assert np.all(np.abs(got[~empty] - rl[~empty]) <= 1e-4)


HEADS = [(64, 4, 4), (64, 8, 1), (128, 2, 2), (128, 12, 2), (128, 16, 2), (128, 20, 1),
         (256, 6, 1), (256, 2, 2)]


@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
def test_attention_one_token(D, Hq, Hkv):
    lens = [1, 15, 16, 17, 0, 63, 64, 65, 255, 256, 257, 1000]
    c = attention_case(5, D, Hq, Hkv, 16, [1] * len(lens), lens)
    check_attention(c, *run_attention(c))


@pytest.mark.parametrize("D,Hq,Hkv", HEADS)
@pytest.mark.parametrize("page", [16, 128])
def test_attention_several_tokens(D, Hq, Hkv, page):
    ms, lens = [2, 5, 1, 0, 17, 3], [2, 77, 500, 9, 300, 130]
    c = attention_case(6, D, Hq, Hkv, page, ms, lens)
    check_attention(c, *run_attention(c))


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 1), (128, 8, 2), (256, 4, 2)])
def test_attention_prompt_pieces(D, Hq, Hkv):
    ms, lens = [130, 64, 33], [130, 700, 290]
    c = attention_case(7, D, Hq, Hkv, 32, ms, lens)
    check_attention(c, *run_attention(c))


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 1), (128, 6, 2), (256, 2, 1)])
def test_attention_long(D, Hq, Hkv):
    """Contexts of many splits, peaked scores, and a scale of the caller's."""
    c = attention_case(8, D, Hq, Hkv, 64, [1, 3], [5000, 3333], spread=3.0)
    check_attention(c, *run_attention(c, scale=0.11), scale=0.11)


# sequences of many rows (heads times new tokens from 5120 on), alone and beside others
MANY = [(64, 32, 8), (64, 40, 40), (128, 32, 8), (128, 48, 2)]


@pytest.mark.parametrize("D,Hq,Hkv", MANY)
def test_attention_many_rows(D, Hq, Hkv):
    ms, lens = [200, 1, 129, 161], [200, 400, 300, 777]
    c = attention_case(18, D, Hq, Hkv, 32, ms, lens)
    check_attention(c, *run_attention(c))


@pytest.mark.parametrize("D,Hq,Hkv,ms,lens", [(64, 1, 1, [257], [20000]), (128, 1, 1, [257], [20000]),
                                              (256, 1, 1, [257], [20000]),
                                              (256, 24, 4, [4], [100000])])
def test_attention_long_runs_stay_exact(D, Hq, Hkv, ms, lens):
    """Outputs over many keys are small against the sums of codes they come from.  Rounding to
    bf16 leaves 0.0017 of their norm, weights and values in fp16 another 2^-12 at most: together
    under 0.002, however long the run of keys."""
    c = attention_case(38, D, Hq, Hkv, 64, ms, lens)
    o, _ = run_attention(c)
    ro, _, _ = ref.attention(np64(c["q"]), c["cache"], c["table"], c["lens"],
                             offsets(c["ms"]).tolist(), D ** -0.5)
    assert np.linalg.norm(np64(o) - ro) <= 0.002 * np.linalg.norm(ro)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 2), (128, 2, 2), (256, 4, 2)])
def test_attention_unsplit_beside_split(D, Hq, Hkv):
    """Sequences of so many rows that their keys stay whole, in a grid made for another's
    splits."""
    ms, lens = [257, 1, 300, 2], [600, 1500, 301, 2500]
    c = attention_case(28, D, Hq, Hkv, 32, ms, lens)
    check_attention(c, *run_attention(c))


def test_attention_many_rows_peaked_and_scaled():
    """Large scores of both signs of the scale, so that the running maximum moves often."""
    for scale in (0.3, -0.25):
        c = attention_case(19, 128, 32, 4, 16, [170], [600], spread=2.0)
        check_attention(c, *run_attention(c, scale=scale), scale=scale)


def test_attention_many_rows_without_keys():
    for m, L in ((200, 150), (200, 0), (180, 1)):
        c = attention_case(20, 128, 32, 8, 16, [m], [L])
        o, lse = run_attention(c)
        check_attention(c, o, lse)
        assert not bool(o[:m - L].any())


@pytest.mark.parametrize("ms,Hq", [([4, 1], 8), ([180, 1], 32)])
def test_attention_nan_values_reach_only_rows_that_see_them(ms, Hq):
    """A value group holding a NaN at a late position: earlier rows do not see it."""
    L = ms[0] + 30
    c = attention_case(21, 128, Hq, 2, 16, ms, [L, 40])
    o1, l1 = run_attention(c)
    at, g = L - 2, 2                       # the row before last sees it, and the last
    rec = c["cache"][c["table"][0, at // 16], 1, 1, at % 16]
    rec[64 + 4 * g + 2:64 + 4 * g + 4] = (0xFF, 0x7F)
    o2, l2 = run_attention(c)
    h = slice(Hq // 2, Hq)                 # the second kv-head's query heads
    assert bool(o2[ms[0] - 2:ms[0], h, 32 * g:32 * g + 32].isnan().all())
    keep = torch.ones(o1.shape, dtype=torch.bool)
    keep[ms[0] - 2:ms[0], h, 32 * g:32 * g + 32] = False
    assert_bits_equal(o1[keep], o2[keep], "outputs that the NaN does not reach")
    assert_bits_equal(l1, l2, "lse")


def test_attention_many_rows_bad_page_strides_and_batch():
    c = attention_case(22, 128, 32, 8, 16, [170, 165], [300, 280])
    o, lse = run_attention(c)
    for n in range(2):
        cu = offsets(c["ms"]).tolist()
        one = dict(c, q=c["q"][cu[n]:cu[n + 1]], table=c["table"][n:n + 1], lens=c["lens"][n:n + 1],
                   ms=[c["ms"][n]])
        o1, l1 = run_attention(one)
        assert_bits_equal(o[cu[n]:cu[n + 1]], o1, "o of sequence %d" % n)
        assert_bits_equal(lse[cu[n]:cu[n + 1]], l1, "lse of sequence %d" % n)
    # a page outside the cache: its keys are left out
    bad = dict(c, table=c["table"].copy())
    bad["table"][1, 3] = -5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o2, _ = run_attention(bad, status=status)
    assert int(status) == 10
    assert_bits_equal(o2[:170], o[:170], "the other sequence")
    keys = [p for p in range(280) if not 48 <= p < 64]
    kk = ref.values(ref.gather(c["cache"], c["table"][1], 280, 0)[keys], ref.key_order(128))
    vv = ref.values(ref.gather(c["cache"], c["table"][1], 280, 1)[keys], ref.value_order(128))
    s = np.einsum("hd,lhd->hl", np64(c["q"])[-1], np.repeat(kk, 4, 1)) * 128 ** -0.5
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    ro = np.einsum("hl,lhd->hd", p, np.repeat(vv, 4, 1))
    oa = np.einsum("hl,lhd->hd", p, np.abs(np.repeat(vv, 4, 1)))
    assert np.all(np.abs(np64(o2[-1]) - ro) <= ref.U_BF16 * np.abs(ro) + 2.0 ** -9 * oa)
    # lengths past the bound
    status.zero_()
    run_attention(c, status=status, max_kv_len=290)
    assert int(status) == 5


@pytest.mark.parametrize("m", [3, 40])
def test_attention_rows_without_keys(m):
    """Lengths below the new rows: the first rows see nothing and give zeros."""
    c = attention_case(9, 128, 8, 2, 16, [m, m, m], [m - 2, 0, 1])
    o, lse = run_attention(c)
    check_attention(c, o, lse)
    assert not bool(o[:2].any()) and not bool(o[m:2 * m].any())


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 8, 2), (256, 3, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_attention_cuda_cores(D, Hq, Hkv, dtype):
    ms, lens = [1, 4, 1, 9], [300, 130, 0, 3]
    c = attention_case(10, D, Hq, Hkv, 16, ms, lens, dtype)
    check_attention(c, *run_attention(c, simt=True))
    if dtype == torch.float32:
        check_attention(c, *run_attention(c))


def test_attention_large_and_small_queries():
    """Rows of very different size in one group; a zero row; scores that saturate."""
    c = attention_case(11, 128, 8, 1, 16, [1, 1], [200, 90])
    c["q"][0, 0] *= 1e-6
    c["q"][0, 1] = 0.0
    c["q"][0, 2] *= 1e4
    c["q"][1, 3] *= 1e-30
    o, lse = run_attention(c)
    ro, rl, oa = ref.attention(np64(c["q"]), c["cache"], c["table"], c["lens"], [0, 1, 2], 128 ** -0.5)
    err = np.abs(np64(o) - ro)
    # scores of size 1e4 * 40: 2^-24 of 4e5 is 0.03 in the exponent; that row is one-hot
    # or nearly, so it is held to 1 part in 16 and the others to the usual bound
    lim = ref.U_BF16 * np.abs(ro) + 2.0 ** -9 * oa
    lim[0, 2] = oa[0, 2] / 16
    assert np.all(err <= lim)


def test_attention_nan_stays_in_its_row():
    c = attention_case(12, 128, 8, 2, 16, [4, 1], [90, 40])
    o1, _ = run_attention(c)
    c["q"][1, 2] = float("nan")
    o2, _ = run_attention(c)
    assert bool(o2[1, 2].isnan().all())
    same = torch.ones(5, 8, dtype=torch.bool)
    same[1, 2] = False
    assert_bits_equal(o1[same], o2[same], "rows next to a NaN row")


def test_attention_batch_invariance():
    lens = [3000, 17, 1, 900]
    for ms in ([1] * 4, [5] * 4):
        c = attention_case(13, 128, 8, 2, 32, ms, [max(a, b) for a, b in zip(lens, ms)])
        o, lse = run_attention(c)
        cu = offsets(ms).tolist()
        for n in range(4):
            one = dict(c, q=c["q"][cu[n]:cu[n + 1]], table=c["table"][n:n + 1],
                       lens=c["lens"][n:n + 1], ms=[ms[n]])
            o1, l1 = run_attention(one)
            assert_bits_equal(o[cu[n]:cu[n + 1]], o1, "o of sequence %d" % n)
            assert_bits_equal(lse[cu[n]:cu[n + 1]], l1, "lse of sequence %d" % n)


def test_attention_bad_lengths_and_pages():
    c = attention_case(14, 128, 4, 2, 16, [1, 1, 1], [40, 50, 60])
    good, _ = run_attention(c)
    for lens, max_len in (([40, 50, 1000], None), ([40, 50, -3], None), ([40, 50, 60], 55)):
        bad = dict(c, lens=np.array(lens, np.int32))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = torch.full((3, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        run_attention(bad, o=o, status=status, max_kv_len=max_len)
        assert int(status) == 5
        assert bool((o[2] == 7.0).all())
        if max_len is None:
            assert_bits_equal(o[:2], good[:2], "other sequences")
    # keys of a page outside the cache are left out
    bad = dict(c, table=c["table"].copy())
    bad["table"][2, 1] = 9999
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, _ = run_attention(bad, status=status)
    assert int(status) == 10
    k = [p for p in range(60) if not 16 <= p < 32]
    cache = torch.from_numpy(c["cache"]).cuda()
    rec = ref.gather(c["cache"], c["table"][2], 60, 0)[k], ref.gather(c["cache"], c["table"][2], 60, 1)[k]
    kk, vv = ref.values(rec[0], ref.key_order(128)), ref.values(rec[1], ref.value_order(128))
    q = np64(c["q"])[2]
    s = np.einsum("hd,lhd->hl", q, np.repeat(kk, 2, 1)) * 128 ** -0.5
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    ro = np.einsum("hl,lhd->hd", p, np.repeat(vv, 2, 1))
    oa = np.einsum("hl,lhd->hd", p, np.abs(np.repeat(vv, 2, 1)))
    assert np.all(np.abs(np64(o[2]) - ro) <= ref.U_BF16 * np.abs(ro) + 2.0 ** -9 * oa)
    assert_bits_equal(o[:2], good[:2], "other sequences")


def test_attention_streams_graphs_and_dirty_workspace():
    c = attention_case(15, 128, 8, 2, 16, [1, 1], [2000, 70])
    o1, l1 = run_attention(c)
    q, cache, table, lens = c["q"].cuda(), torch.from_numpy(c["cache"]).cuda(), \
        torch.from_numpy(c["table"]).cuda(), torch.from_numpy(c["lens"]).cuda()
    ws = torch.empty(max(16, gdn.gdn_kv_attention_workspace_size(128, 8, 2, 2, 2, 1, 2000)),
                     dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(o1), torch.empty_like(l1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_kv_attention(q, cache, table, lens, max_kv_len=2000, o=o, lse=lse, workspace=ws)
    for _ in range(2):
        o.fill_(float("nan"))
        lse.fill_(float("nan"))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert_bits_equal(o, o1, "o of a replay")
        assert_bits_equal(lse, l1, "lse of a replay")


def test_attention_strided_queries_and_refusals():
    c = attention_case(16, 128, 8, 2, 16, [3], [50])
    o1, _ = run_attention(c)
    y = torch.full((3, 8 * 128 + 256), float("nan"), dtype=torch.bfloat16)
    y[:, :1024] = c["q"].reshape(3, -1)
    q = y.cuda()[:, :1024].unflatten(1, (8, 128))
    cache, table, lens = torch.from_numpy(c["cache"]).cuda(), torch.from_numpy(c["table"]).cuda(), \
        torch.from_numpy(c["lens"]).cuda()
    cu = offsets([3]).cuda()
    assert_bits_equal(gdn.gdn_kv_attention(q, cache, table, lens, cu), o1, "o from a view")

    def code(**kw):
        a = dict(q=q, cache=cache, block_table=table, kv_lens=lens, cu_seqlens=cu)
        a.update(kw)
        with pytest.raises((gdn.GdnError, ValueError, TypeError)) as e:
            gdn.gdn_kv_attention(**a)
        return getattr(e.value, "code", "value")
    assert code(q=q[:, :7]) in (2, 3)
    assert code(q=q.half()) == "value"
    assert code(o=torch.empty(3, 8, 128, device="cuda")) == 4
    assert code(cache=cache.cpu()) == "value"
    assert code(cache=cache[:, :1]) == "value"
    assert code(max_kv_len=-1) == 2
    assert code(lse=torch.empty(8, 3, device="cuda")) == "value"
    assert code(cu_seqlens=offsets([4]).cuda()) == 5


def test_attention_over_what_append_stored():
    """The two together: prompt and token, against attention on the values read back."""
    c = append_case(17, 128, 8, 2, 16, [37, 5], [37, 60], torch.bfloat16, 64, False)
    cache, q = run_append(c)
    page0 = dict(c, ms=[37, 60])
    cache.view(-1)  # positions 0..54 of the second sequence hold the fill pattern 0xAB
    host = cache.cpu().numpy()
    table, lens = torch.from_numpy(c["table"]).cuda(), torch.tensor(c["lens"], dtype=torch.int32).cuda()
    cu = offsets(c["ms"])
    o = gdn.gdn_kv_attention(q, cache, table, lens, cu.cuda(), cu_seqlens_host=cu)
    ro, _, oa = ref.attention(np64(q), host, c["table"], np.array(c["lens"]), cu.tolist(), 128 ** -0.5)
    assert np.all(np.abs(np64(o) - ro) <= ref.U_BF16 * np.abs(ro) + 2.0 ** -9 * oa)
    assert page0["ms"][0] == 37
