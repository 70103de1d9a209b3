"""gdn_quantize_rows, gdn_add_rmsnorm and gdn_gated_rmsnorm against their formulas in 64 bits,
at the bounds of eight_bit_ref."""
import numpy as np
import pytest
import torch

import eight_bit_ref as ref
from gpu_util import assert_bits_equal

pytestmark = pytest.mark.gpu

gdn = pytest.importorskip("gated_deltanet_linear_11_gb300")

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load()


def rnd(seed, *shape, dtype=BF):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=gen).to(dtype).cuda()


def strided(x, pad):
    """The same rows inside wider ones, `pad` elements in."""
    wide = torch.full((x.shape[0], x.shape[1] + 2 * pad), 7.0, dtype=x.dtype, device=x.device)
    wide[:, pad:pad + x.shape[1]] = x
    return wide[:, pad:pad + x.shape[1]]


# lengths on both sides of every split: part of a vector, a warp's one and four vectors, a CTA's
# two and four, and the longest row
WIDTHS = [1, 7, 8, 255, 256, 264, 1024, 1025, 2047, 5120, 16384, 16392, 32768]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", WIDTHS)
def test_quantize_rows(D, dtype):
    x = rnd(D, 5, D, dtype=dtype) * torch.tensor([1.0, 1e-30, 1e30, 3.0, 1.0]).to(dtype).cuda()[:, None]
    x[3] = 0
    q, scale = gdn.gdn_quantize_rows(x)
    assert q.shape == x.shape and q.dtype is torch.int8 and scale.shape == (5,)
    ref.assert_codes(q, scale, ref.f64(x), 2 * ref.U)
    assert scale[3] == 2.0 ** -126 and not q[3].any()
    assert (q.int().abs().amax(-1)[[0, 1, 2, 4]] == 127).all()


def test_bf16_codes_are_exact():
    """Every pair of significands, a few octaves apart: ties go to the even code, and no other
    quotient changes sides."""
    sig = torch.arange(128, 256).float()
    rows = []
    for s in range(0, 9):
        x = (sig * 2.0 ** -s).repeat(128, 1)
        x = torch.where(x <= sig[:, None], x, torch.zeros(()))
        rows.append(torch.cat((sig[:, None], x, -x), 1))
    x = torch.cat(rows).to(BF).cuda()
    q, scale = gdn.gdn_quantize_rows(x)
    want, s = ref.quotients(ref.f64(x))
    assert (np.abs(want - np.floor(want) - 0.5) == 0).any()
    assert (ref.f64(q) == np.rint(want)).all()
    assert (np.abs(ref.f64(scale) - s) <= ref.U * s).all()


def test_rows_that_are_not_finite():
    for dtype in (BF, F32):
        x = rnd(1, 6, 300, dtype=dtype)
        x[1, 7], x[2, 299], x[4, 0] = float("nan"), float("inf"), float("-inf")
        q, scale = gdn.gdn_quantize_rows(x)
        bad = torch.tensor([1, 2, 4], device="cuda")
        good = torch.tensor([0, 3, 5], device="cuda")
        assert scale[bad].isnan().all() and not q[bad].any()
        ref.assert_codes(q[good], scale[good], ref.f64(x[good]), 2 * ref.U)
        w = torch.ones(300, device="cuda")
        (q, scale), _ = gdn.gdn_add_rmsnorm(x, w, eight_bit=True)
        assert scale[bad].isnan().all() and not q[bad].any() and scale[good].isfinite().all()
        y, _ = gdn.gdn_add_rmsnorm(x, w)
        assert not y[bad].isfinite().all(-1).any() and y[good].isfinite().all()


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dtype,wt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("D", WIDTHS)
def test_add_rmsnorm(D, dtype, wt, eight):
    for res, offset, eps in ((True, 1.0, 1e-6), (False, 0.0, 1e-5)):
        x, w = rnd(D, 3, D, dtype=dtype), rnd(D + 1, D, dtype=wt)
        r = rnd(D + 2, 3, D, dtype=dtype) * 5 if res else None
        y, out = gdn.gdn_add_rmsnorm(x, w, r, eps=eps, weight_offset=offset, eight_bit=eight)
        want, h = ref.add_rmsnorm(x, w, r, eps, offset)
        if eight:
            ref.assert_codes(*y, want, ref.NORM)
        else:
            ref.assert_close(y, want, ref.NORM, dtype)
        if res:
            assert out.dtype is dtype
            assert_bits_equal(out, (x.float() + r.float()).to(dtype), "residual")
        else:
            assert out is None


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norms_of_extreme_rows(dtype):
    """Squares past fp32, zeros, and rows so small that eps rules."""
    size = torch.tensor([1e25, 3e37, 0.0, 1e-25, 1e-12, 1.0], device="cuda")
    x = (rnd(5, 6, 640, dtype=F32) * size[:, None]).to(dtype)
    w = rnd(6, 640, dtype=F32) * 20
    want, _ = ref.add_rmsnorm(x, w, None, 1e-6, 0.0)
    y, _ = gdn.gdn_add_rmsnorm(x, w)
    ref.assert_close(y, want, ref.NORM, dtype)
    (q, scale), _ = gdn.gdn_add_rmsnorm(x, w, eight_bit=True)
    keep = [0, 1, 2, 4, 5]              # 1e-25 of x gives y of 1e-22: fp32 holds it
    ref.assert_codes(q, scale, want, ref.NORM)
    assert scale[2] == 2.0 ** -126 and not q[2].any() and keep
    x3, z = x.view(6, 5, 128), rnd(7, 6, 5, 128, dtype=dtype)
    z[0, 0, :4] = torch.tensor([100.0, -100.0, -80.0, 0.0])
    w3 = w[:128].contiguous()
    want = ref.gated_rmsnorm(x3, z, w3, 1e-6)
    got = gdn.gdn_gated_rmsnorm(x3, z, w3)
    # silu(-100) = -3.7e-42 is under the fp32 range, where the kernel gives a zero
    want = np.where(np.abs(want) < 1e-36, ref.f64(got) * (np.abs(ref.f64(got)) < 1e-36), want)
    # the exponent -80 log2 e is rounded before e^-z: 116 half steps of it times ln 2
    ref.assert_close(got, want, ref.GATED[dtype] + 116 * ref.U, dtype)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,D", [(1, 16), (3, 16), (5, 32), (7, 64), (48, 128), (9, 128), (16, 256),
                                 (128, 256)])
def test_gated_rmsnorm(H, D, dtype, eight):
    T = 5
    x = rnd(H, T, H, D, dtype=dtype) * torch.arange(1, H + 1, device="cuda").to(dtype)[:, None]
    rows = rnd(H + 1, T, 2 * H * D, dtype=dtype)
    z = rows[:, H * D:].view(T, H, D)
    w = rnd(H + 2, D, dtype=F32)
    y = gdn.gdn_gated_rmsnorm(x, z, w, eps=1e-5, eight_bit=eight)
    want = ref.gated_rmsnorm(x, z, w, 1e-5)
    if eight:
        ref.assert_codes(*y, want, ref.GATED[dtype])
    else:
        assert y.shape == (T, H * D)
        ref.assert_close(y, want, ref.GATED[dtype], dtype)
    assert_bits_equal(gdn.gdn_gated_rmsnorm(x[None], z[None], w, eps=1e-5),
                      gdn.gdn_gated_rmsnorm(x, z, w, eps=1e-5), "[1, T, H, D]")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [40, 1000, 1031, 6144])
def test_bits_do_not_depend_on_batch_or_layout(D, dtype):
    x, r, w = rnd(1, 37, D, dtype=dtype), rnd(2, 37, D, dtype=dtype), rnd(3, D, dtype=dtype)
    (q, s), h = gdn.gdn_add_rmsnorm(x, w, r, eight_bit=True)
    y, _ = gdn.gdn_add_rmsnorm(x, w, r)
    for rows in (slice(0, 1), slice(36, 37), slice(5, 9)):
        (q1, s1), h1 = gdn.gdn_add_rmsnorm(x[rows], w, r[rows], eight_bit=True)
        assert_bits_equal(q1, q[rows], "codes")
        assert_bits_equal(s1, s[rows], "scale")
        assert_bits_equal(h1, h[rows], "residual")
    for pad in (1, 3, 8):
        wide = torch.zeros(37, D + pad, dtype=torch.int8, device="cuda")
        ws = torch.zeros(D + 1, dtype=dtype, device="cuda")
        ws[1:] = w
        (q1, s1), h1 = gdn.gdn_add_rmsnorm(strided(x, pad), ws[1:], strided(r, pad),
                                           eight_bit=True, y=wide[:, pad:])
        assert_bits_equal(q1, q, "codes")
        assert_bits_equal(s1, s, "scale")
        assert_bits_equal(h1, h, "residual")
        assert not wide[:, :pad].any()
        out = strided(x, pad)
        gdn.gdn_add_rmsnorm(out, ws[1:], strided(r, pad), y=out)        # in place
        assert_bits_equal(out.contiguous(), y, "y")
    # the residual updated in place
    r2 = r.clone()
    y2, h2 = gdn.gdn_add_rmsnorm(x, w, r2, residual_out=r2)
    assert h2 is r2
    assert_bits_equal(r2, h, "residual")
    assert_bits_equal(y2, y, "y")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [512, 1000, 1001, 6144])
def test_many_rows_in_place(D, dtype):
    """More rows than run at once, each written where rows still to come are read ahead."""
    T = 3000
    x, r, w = rnd(1, T, D, dtype=dtype), rnd(2, T, D, dtype=dtype), rnd(3, D, dtype=dtype)
    y, h = gdn.gdn_add_rmsnorm(x, w, r)
    x2, r2 = x.clone(), r.clone()
    gdn.gdn_add_rmsnorm(x2, w, r2, y=x2, residual_out=r2)
    assert_bits_equal(x2, y, "y")
    assert_bits_equal(r2, h, "residual")
    assert_bits_equal(gdn.gdn_add_rmsnorm(x[2990:], w, r[2990:])[0], y[2990:], "last rows")
    if D % 128 == 0:
        z = rnd(4, T, D, dtype=dtype)
        g = gdn.gdn_gated_rmsnorm(x.view(T, -1, 128), z.view(T, -1, 128), w[:128].contiguous())
        gdn.gdn_gated_rmsnorm(x.view(T, -1, 128), z.view(T, -1, 128), w[:128].contiguous(), y=x)
        assert_bits_equal(x, g, "gated")


def test_no_rows_and_many():
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    q, s = gdn.gdn_quantize_rows(e)
    assert q.shape == (0, 64) and s.shape == (0,)
    y, h = gdn.gdn_add_rmsnorm(e, torch.ones(64, device="cuda"), e)
    assert y.shape == h.shape == (0, 64)
    assert gdn.gdn_gated_rmsnorm(e.view(0, 4, 16), e.view(0, 4, 16),
                                 torch.ones(16, device="cuda")).shape == (0, 64)
    x = rnd(3, 100001, 8)
    q, s = gdn.gdn_quantize_rows(x)
    ref.assert_codes(q[-3:], s[-3:], ref.f64(x[-3:]), 2 * ref.U)
    ref.assert_codes(q[:3], s[:3], ref.f64(x[:3]), 2 * ref.U)


def test_rows_far_apart():
    """Row offsets past 2^31 elements."""
    st = (1 << 30) + 8
    wide = torch.empty(2 * st + 64, dtype=BF, device="cuda")
    x = wide.as_strided((3, 64), (st, 1))
    x.copy_(rnd(4, 3, 64))
    q, s = gdn.gdn_quantize_rows(x)
    ref.assert_codes(q, s, ref.f64(x), 2 * ref.U)
    y, h = gdn.gdn_add_rmsnorm(x, torch.ones(64, device="cuda"), x, residual_out=x, y=None)
    assert h is x and y.isfinite().all()


def test_norm_in_a_graph():
    """A captured pass, replayed on new values, gives what the plain calls give."""
    x, r, w = rnd(1, 9, 700), rnd(2, 9, 700), rnd(3, 700)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gdn.gdn_add_rmsnorm(x, w, r, eight_bit=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (q, s), h = gdn.gdn_add_rmsnorm(x, w, r, eight_bit=True)
    for seed in (5, 6):
        x.copy_(rnd(seed, 9, 700))
        graph.replay()
        (q1, s1), h1 = gdn.gdn_add_rmsnorm(x, w, r, eight_bit=True)
        assert_bits_equal(q, q1, "codes")
        assert_bits_equal(s, s1, "scale")
        assert_bits_equal(h, h1, "residual")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [256, 640, 2047, 5120, 20000])
def test_weights_and_rows_far_from_one(D, dtype):
    """Sizes of rows and weights whose products leave fp32's range, or its normal numbers, though
    the norm stays inside; eps as small as it may be.  The largest of 20000 normal numbers is
    about 4, so results stay under 1e38."""
    sizes = [(30.0, 1e37, 1e-6), (100.0, 1e37, 1e-6), (1e3, 1e36, 1e-6), (3e37, 1e34, 1e-6),
             (3e37, 1e-38, 1e-6), (1e-10, 1e-35, 1e-6), (1e-18, 1e-24, 2.0 ** -126),
             (1e-20, 1e-20, 2.0 ** -126), (1e-20, 1e-28, 2.0 ** -126)]
    for size, weight, eps in sizes:
        x = (rnd(D, 4, D, dtype=F32) * size).to(dtype)
        x[2] = 0
        w = (1 + torch.rand(D, generator=torch.Generator().manual_seed(D))).cuda() * weight
        want, _ = ref.add_rmsnorm(x, w, None, eps, 0.0)
        (q, scale), _ = gdn.gdn_add_rmsnorm(x, w, eps=eps, eight_bit=True)
        ref.assert_codes(q, scale, want, ref.NORM)
        y, _ = gdn.gdn_add_rmsnorm(x, w, eps=eps)
        ref.assert_close(y, want, ref.NORM, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [256, 640, 5120])
def test_small_elements_of_large_rows(D, dtype):
    """Elements far under the others of a row whose squares pass fp32: their results are normal
    numbers."""
    x = rnd(1, 4, D, dtype=F32) * 1e19
    x[:, ::7] *= 1e-37
    x = x.to(dtype)
    w = rnd(2, D, dtype=F32) * 20
    want, _ = ref.add_rmsnorm(x, w, None, 1e-6, 0.0)
    ref.assert_close(gdn.gdn_add_rmsnorm(x, w)[0], want, ref.NORM, dtype)
    x3, z, w3 = x.view(4, -1, 128), rnd(3, 4, D // 128, 128, dtype=dtype) + 3, w[:128].contiguous()
    want = ref.gated_rmsnorm(x3, z, w3, 1e-6)
    ref.assert_close(gdn.gdn_gated_rmsnorm(x3, z, w3), want, ref.GATED[dtype], dtype)


def odd_rows(x):
    """Among x's rows some of zeros, some whose squares pass fp32, some with a NaN."""
    x[5::11] = 0
    x[3::7] *= 1e25
    x[6::13, x.shape[1] // 3] = float("nan")
    return x


def assert_rows(got, want, rel):
    """8-bit rows against `want`; those of NaN are marked."""
    q, scale = got
    bad = torch.from_numpy(~np.isfinite(want).all(-1)).cuda()
    assert scale[bad].isnan().all() and not q[bad].any()
    ref.assert_codes(q[~bad], scale[~bad], want[~bad.cpu().numpy()], rel)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [512, 1000, 1001, 6144])
def test_many_rows_in_eight_bits(D, dtype):
    """More rows than run at once, so that every CTA makes several, ordinary and odd ones in turn:
    all of them against 64 bits, and some against calls of a few rows."""
    T = 3000
    x, r, w = odd_rows(rnd(1, T, D, dtype=dtype)), rnd(2, T, D, dtype=dtype), rnd(3, D, dtype=dtype)
    few = slice(1490, 1500)
    with np.errstate(invalid="ignore"):
        got = gdn.gdn_quantize_rows(x)
        assert_rows(got, ref.f64(x), 2 * ref.U)
        for a, b in zip(got, gdn.gdn_quantize_rows(x[few])):
            assert_bits_equal(a[few], b, "rows to 8 bits")
        got, h = gdn.gdn_add_rmsnorm(x, w, r, eight_bit=True)
        assert_rows(got, ref.add_rmsnorm(x, w, r, 1e-6, 0.0)[0], ref.NORM)
        one, _ = gdn.gdn_add_rmsnorm(x[few], w, r[few], eight_bit=True)
        for a, b in zip(got, one):
            assert_bits_equal(a[few], b, "norm")
        if D % 128 == 0:
            x3, z, w3 = x.view(T, -1, 128), r.view(T, -1, 128), w[:128].contiguous()
            got = gdn.gdn_gated_rmsnorm(x3, z, w3, eight_bit=True)
            assert_rows(got, ref.gated_rmsnorm(x3, z, w3, 1e-6), ref.GATED[dtype])
            for a, b in zip(got, gdn.gdn_gated_rmsnorm(x3[few], z[few], w3, eight_bit=True)):
                assert_bits_equal(a[few], b, "gated norm")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,D", [(4, 16), (8, 128), (48, 128), (4, 256)])
def test_gated_rows_that_are_not_finite_and_heads_that_overflow(H, D, dtype):
    x, z, w = rnd(1, 7, H, D, dtype=dtype), rnd(2, 7, H, D, dtype=dtype), rnd(3, D, dtype=F32)
    x[0, 1] *= 1e25                         # heads beside ordinary ones in the same warp
    x[1, 0], x[1, H - 1] = 0, x[1, H - 1] * 3e37
    want = ref.gated_rmsnorm(x, z, w, 1e-6)
    y = gdn.gdn_gated_rmsnorm(x, z, w)
    ref.assert_close(y, want, ref.GATED[dtype], dtype)
    ref.assert_codes(*gdn.gdn_gated_rmsnorm(x, z, w, eight_bit=True), want, ref.GATED[dtype])
    inf = float("inf")
    for t, row, value in ((x, 2, float("nan")), (x, 3, inf), (x, 4, -inf), (z, 5, float("nan")), (z, 6, -inf)):
        t[row, H - 1, D // 2] = value
    q, scale = gdn.gdn_gated_rmsnorm(x, z, w, eight_bit=True)
    assert scale[2:].isnan().all() and not q[2:].any() and scale[:2].isfinite().all()
    ref.assert_codes(q[:2], scale[:2], want[:2], ref.GATED[dtype])
    # the other heads are what they were
    bad = gdn.gdn_gated_rmsnorm(x, z, w)
    assert_bits_equal(bad[:, :(H - 1) * D].contiguous(), y[:, :(H - 1) * D].contiguous(), "other heads")
    assert not bad[2:, (H - 1) * D:].isfinite().all(-1).any()


def test_gated_rows_repeat_themselves():
    """The same bits at every pass, other inputs in between, over memory that held other values;
    codes that are not the nearest lie within 2^-10 of a border."""
    H, D = 48, 128
    w = 1 + 0.2 * rnd(1, D)
    sets = []
    for seed in (2, 3):
        x = (rnd(seed, 64, H, D, dtype=F32) * rnd(seed + 5, 64, H, 1, dtype=F32).exp()).to(BF)
        sets.append((x, rnd(seed + 9, 64, 2 * H * D)[:, H * D:].view(64, H, D)))
    first = [gdn.gdn_gated_rmsnorm(x, z, w, eight_bit=True) for x, z in sets]
    off = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(100):
        junk = torch.full((64, H * D), 255, dtype=torch.uint8, device="cuda")
        del junk
        for (x, z), (q, scale) in zip(sets, first):
            q2, scale2 = gdn.gdn_gated_rmsnorm(x, z, w, eight_bit=True)
            off += (q != q2).sum() + (scale != scale2).sum()
            del q2, scale2
    assert int(off) == 0
    for (x, z), (q, _) in zip(sets, first):
        want, _ = ref.quotients(ref.gated_rmsnorm(x, z, w, 1e-6))
        away = np.abs(want - np.floor(want) - 0.5)[ref.f64(q) != np.rint(want)]
        assert (away <= 2.0 ** -10).all(), float(away.max())
