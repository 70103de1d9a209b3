"""gdn_matmul_i8 against the exact sum and the documented fp32 steps after it, to the bit."""
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


def codes(seed, rows, cols, lo=-128, hi=127, pad=0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randint(lo, hi + 1, (rows, cols + pad), generator=gen, dtype=torch.int8)
    return x.cuda()[:, :cols]


def scales(seed, n):
    gen = torch.Generator().manual_seed(seed)
    return (torch.rand(n, generator=gen) * 0.01 + 1e-4).cuda()


def check(a, w, bias=None, dtype=BF, simt=False, **kw):
    M, N = a.shape[0], w.shape[0]
    sa, sw = scales(1, M), scales(2, N)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gdn.gdn_matmul_i8(a, sa, w, sw, bias=bias, dtype=dtype, simt=simt, status=status, **kw)
    want = ref.product(a, sa, w, sw, bias, dtype)
    assert int(status) == 0
    assert_bits_equal(out.cpu().contiguous(), want, "out %s" % (tuple(out.shape),))
    return out


SIZES = [(1, 1, 1), (1, 16, 16), (1, 128, 64), (2, 130, 100), (3, 5, 1001), (8, 64, 48),
         (9, 257, 2064), (16, 1000, 512), (17, 96, 5120), (33, 300, 1040), (64, 515, 1024),
         (65, 128, 1025), (100, 1024, 4096), (128, 129, 272), (129, 640, 3200), (200, 200, 200),
         (256, 256, 1088), (257, 384, 2048), (333, 515, 1001), (512, 130, 96), (700, 900, 1536)]


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(M, N, K, dtype, simt):
    gen = torch.Generator().manual_seed(M)
    bias = None if M % 2 else torch.randn(N, generator=gen).to(dtype).cuda()
    check(codes(M + K, M, K), codes(N + K, N, K), bias, dtype, simt)


@pytest.mark.parametrize("M", [1, 4, 16, 64, 300])
@pytest.mark.parametrize("lo,hi", [(-128, -128), (127, 127), (-128, -120), (120, 127)])
def test_largest_sums(M, lo, hi):
    """All products of one sign: sums far past 2^24, where fp32 no longer holds every integer."""
    for K in (1024, 1040, 5120, 131071):
        a, w = codes(1, M, K, lo, hi, pad=-K % 16), codes(2, 40, K, lo, hi, pad=-K % 16)
        check(a, w, dtype=F32)


def test_cancelling_sums():
    """Large partial sums that cancel to small ones."""
    K = 8192
    a, w = codes(1, 70, K, 100, 127), codes(2, 150, K, 100, 127)
    w[:, K // 2:] = -w[:, :K // 2]
    a[:, K // 2:] = a[:, :K // 2]
    a[:, 0] += 1 * (a[:, 0] < 127).to(torch.int8)
    check(a, w, dtype=F32)


@pytest.mark.parametrize("M", [1, 12, 80, 400])
@pytest.mark.parametrize("pad_a,pad_w", [(0, 0), (5, 0), (0, 3), (16, 32), (1, 1)])
def test_strides(M, pad_a, pad_w):
    """Rows with any distance between them; what lies behind a row is not read into sums."""
    K, N = 528, 200
    a, w = codes(1, M, K, pad=pad_a), codes(2, N, K, pad=pad_w)
    wide = torch.full((M, N + 7), 3.0, device="cuda", dtype=BF)
    out = check(a, w, out=wide[:, 2:2 + N])
    assert out.data_ptr() == wide[:, 2:].data_ptr()
    assert (wide[:, :2] == 3).all() and (wide[:, 2 + N:] == 3).all()
    # rows whose length is not a multiple of 16 bytes, on 16-byte starts
    check(codes(3, M, 500, pad=12), codes(4, N, 500, pad=12))
    # views that start inside their storage
    check(codes(5, M, 560)[:, 16:], codes(6, N, 560)[:, 16:])
    check(codes(5, M, 560)[:, 3:], codes(6, N, 560)[:, 3:])


def test_bits_do_not_depend_on_the_batch():
    a, w = codes(1, 300, 1200, pad=0), codes(2, 333, 1200)
    sa, sw = scales(3, 300), scales(4, 333)
    full = gdn.gdn_matmul_i8(a, sa, w, sw, dtype=F32)
    for rows in (slice(0, 1), slice(7, 11), slice(299, 300), slice(100, 230)):
        part = gdn.gdn_matmul_i8(a[rows], sa[rows].contiguous(), w, sw, dtype=F32)
        assert_bits_equal(part, full[rows].contiguous(), "rows")
    part = gdn.gdn_matmul_i8(a, sa, w[50:51], sw[50:51].contiguous(), dtype=F32)
    assert_bits_equal(part, full[:, 50:51].contiguous(), "channel")


def test_nothing_to_do_and_scales_that_are_not_finite():
    a, w = codes(1, 5, 64), codes(2, 7, 64)
    sa, sw = scales(1, 5), scales(2, 7)
    assert gdn.gdn_matmul_i8(a[:0], sa[:0], w, sw).shape == (0, 7)
    assert gdn.gdn_matmul_i8(a, sa, w[:0], sw[:0]).shape == (5, 0)
    sa[2], sw[3] = float("nan"), float("inf")
    out = gdn.gdn_matmul_i8(a, sa, w, sw)
    assert out[2].isnan().all() and not out[:, 3].isfinite().any()
    keep = out[[0, 1, 3, 4]][:, [0, 1, 2, 4, 5, 6]]
    assert keep.isfinite().all()


@pytest.mark.parametrize("K", [2048, 4096])
def test_leading_dimension_and_given_scratch(K):
    """[1, T, K] operands, a workspace of the stated size, and one that is too small."""
    a, w = codes(1, 400, K), codes(2, 2304, K)
    sa, sw = scales(1, 400), scales(2, 2304)
    want = gdn.gdn_matmul_i8(a, sa, w, sw)
    size = gdn.gdn_matmul_i8_workspace_size(a, w)
    assert (size > 0) == (K == 4096)            # the longer rows go by pairs of CTAs
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")     # fp16 NaN, counts of -1
    got = gdn.gdn_matmul_i8(a[None], sa, w[None], sw, workspace=ws)
    assert got.shape == (1, 400, 2304)
    assert_bits_equal(got[0], want, "out")
    # shifted by a byte: rows off 16 bytes, so copies of both
    b = torch.empty(400 * K + 1, dtype=torch.int8, device="cuda")[1:].view(400, K)
    v = torch.empty(2304 * K + 1, dtype=torch.int8, device="cuda")[1:].view(2304, K)
    b.copy_(a)
    v.copy_(w)
    assert gdn.gdn_matmul_i8_workspace_size(b, v) > size
    assert_bits_equal(gdn.gdn_matmul_i8(b, sa, v, sw), want, "out")
    assert gdn.gdn_matmul_i8_workspace_size(a, w, simt=True) == 0


@pytest.mark.parametrize("shapes", [[(1, 5120, 5120), (200, 1000, 2048), (40, 4000, 3000)],
                                    [(700, 2048, 2048), (600, 2048, 2048), (64, 9000, 1024)]])
def test_products_on_streams_at_once(shapes):
    """Kernels of every form side by side on three streams, many times over."""
    cases = []
    for i, (M, N, K) in enumerate(shapes):
        a, w, sa, sw = codes(i, M, K, -90, 90), codes(9 + i, N, K, -90, 90), scales(i, M), scales(i, N)
        cases.append((a, sa, w, sw, ref.product(a, sa, w, sw, None, BF), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for a, sa, w, sw, want, stream in cases:
            with torch.cuda.stream(stream):
                outs.append((gdn.gdn_matmul_i8(a, sa, w, sw), want))
    torch.cuda.synchronize()
    for got, want in outs:
        assert_bits_equal(got.cpu(), want, "out")


def test_outputs_past_2_31():
    M, N, K = 70000, 32768, 16
    a, w = codes(1, M, K), codes(2, N, K)
    sa, sw = scales(1, M), scales(2, N)
    out = gdn.gdn_matmul_i8(a, sa, w, sw)
    for m in (0, 65535, 65536, M - 1):
        want = ref.product(a[m:m + 1], sa[m:m + 1], w, sw, None, BF)
        assert_bits_equal(out[m:m + 1].cpu(), want, "row %d" % m)


@pytest.mark.parametrize("M", [1, 40, 500])
def test_graphs_and_streams(M):
    """Two captured products with scratch of their own, and one on another stream, at once."""
    K, N = 5120, 640
    a = [codes(i, M, K) for i in range(3)]
    w, sa, sw = codes(9, N, K), scales(1, M), scales(2, N)
    want = [ref.product(x, sa, w, sw, None, BF) for x in a]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gdn.gdn_matmul_i8(a[0], sa, w, sw)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gdn.gdn_matmul_i8(a[i], sa, w, sw))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
            third = gdn.gdn_matmul_i8(a[2], sa, w, sw)
        torch.cuda.synchronize()
        for got, exp in zip(outs + [third], want):
            assert_bits_equal(got.cpu(), exp, "out")
            got.zero_()
        torch.cuda.synchronize()


@pytest.mark.parametrize("M", [70, 128, 200, 300, 600])
def test_some_tiles_with_large_sums(M):
    """Ordinary codes but for a few tokens or channels whose sums pass 2^24 on the way, alone
    and together; 700 channels are more than one tile of them."""
    K, N = 6144, 700
    a, w = codes(1, M, K, -30, 30), codes(2, N, K, -30, 30)
    check(a, w, dtype=F32)
    w[130:140], w[699] = 127, -128
    check(a, w, dtype=F32)
    a[M // 2], a[M - 1] = -128, 127
    check(a, w, dtype=F32)
    w[:] = codes(2, N, K, -30, 30)
    check(a, w, dtype=F32)


# Many channels or long rows: pairs of CTAs from 65 tokens on, tiles whole, in parts and both.
PAIRS = [(65, 5130, 6144), (128, 5120, 6160), (129, 5200, 6145), (300, 2600, 12288), (500, 10240, 2048),
         (700, 5131, 3008), (1500, 2311, 2048)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", PAIRS)
def test_sizes_of_pairs(M, N, K, dtype):
    a, w = codes(M + K, M, K, pad=-K % 16), codes(N + K, N, K, pad=-K % 16)
    assert gdn.gdn_matmul_i8_workspace_size(a, w) > 0
    gen = torch.Generator().manual_seed(M)
    bias = None if M % 2 else torch.randn(N, generator=gen).to(dtype).cuda()
    out = torch.zeros(M + 1, N + 24, dtype=dtype, device="cuda")
    check(a, w, bias, dtype, out=out[:M, 8:8 + N])
    assert not out[M].any() and not out[:, :8].any() and not out[:, 8 + N:].any()


@pytest.mark.parametrize("M", [70, 300])
@pytest.mark.parametrize("lo,hi", [(-128, -128), (120, 127)])
def test_largest_sums_of_pairs(M, lo, hi):
    a, w = codes(1, M, 6144, lo, hi), codes(2, 5130, 6144, lo, hi)
    assert gdn.gdn_matmul_i8_workspace_size(a, w) > 0
    check(a, w)


@pytest.mark.parametrize("M", [70, 128, 300])
def test_some_pairs_with_large_sums(M):
    """As above, for tiles that are made a second time beside ones that are not."""
    K, N = 6144, 5400
    a, w = codes(1, M, K, -30, 30), codes(2, N, K, -30, 30)
    assert gdn.gdn_matmul_i8_workspace_size(a, w) > 0
    w[130:140], w[4000], w[5399] = 127, 127, -128
    check(a, w, dtype=F32)
    a[M // 2], a[M - 1] = -128, 127
    check(a, w)


@pytest.mark.parametrize("M,N,K,shift", [(128, 5120, 6144, 0), (300, 5131, 2049, 1), (64, 700, 1001, 1),
                                         (4, 700, 1001, 3)])
def test_calls_one_after_the_other_in_one_workspace(M, N, K, shift):
    """Tokens written just before each product, small and large ones in turn, all through the same
    buffers: nothing of the call before is seen."""
    sets = [codes(1, M, K, -30, 30), codes(2, M, K, 100, 127), codes(3, M, K)]
    room = torch.empty(M * K + shift, dtype=torch.int8, device="cuda")
    a, w = room[shift:].view(M, K), codes(4, N, K)
    sa, sw = scales(1, M), scales(2, N)
    ws = torch.full((gdn.gdn_matmul_i8_workspace_size(a, w),), 255, dtype=torch.uint8, device="cuda")
    assert (ws.numel() > 0) == (M > 64 or shift > 0)
    torch.cuda.synchronize()
    outs = []
    for i in range(24):
        a.copy_(sets[i % 3])
        outs.append(gdn.gdn_matmul_i8(a, sa, w, sw, dtype=F32, workspace=ws))
    want = [ref.product(x, sa, w, sw, None, F32) for x in sets]
    for i, out in enumerate(outs):
        assert_bits_equal(out.cpu(), want[i % 3], "call %d" % i)


# Tiles of pairs of CTAs whose sums turn out to be too large for one run along K, which are then
# made again: tokens stay under the size at which tiles are made with moves from the start.
CAREFUL, FAR = 15_000_000, 2 ** 48


def squares(x):
    return x.int().square().sum(-1, dtype=torch.int64)


def large_tokens(a, rows):
    """Tokens whose codes are large in one third of a row each, or of medium size all along:
    |a|^2 just under the border, sums with channels of 127 above 2^24, their low bits at random."""
    K = a.shape[1]
    gen = torch.Generator().manual_seed(K)
    for i, row in enumerate(rows):
        if i % 4 == 3:
            a[row] = torch.randint(47, 49, (K,), generator=gen, dtype=torch.int8).cuda()
        else:
            at = K // 3 * (i % 4)
            a[row] = torch.randint(0, 2, (K,), generator=gen, dtype=torch.int8).cuda()
            a[row, at:at + K // 3] = torch.randint(83, 85, (K // 3,), generator=gen, dtype=torch.int8).cuda()


# whole tiles (76 of them fill 152 SMs once) of 128 and of 256 tokens, tiles in two and three parts,
# both kinds in one launch
AGAIN = [(128, 19456), (300, 9728), (300, 4864), (70, 5130), (700, 9000)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N", AGAIN)
def test_tiles_made_again(M, N, dtype):
    K = 6144
    a, w = codes(1, M, K, -30, 30), codes(2, N, K, -30, 30)
    large_tokens(a, [0, 1, 2, 3, M // 2, M - 3, M - 2, M - 1])
    gen = torch.Generator().manual_seed(3)
    channels = [3, 256 + 130, N - 1, N - 300]           # in the first and the second CTA of a pair
    w[channels] = torch.randint(126, 128, (4, K), generator=gen, dtype=torch.int8).cuda()
    assert gdn.gdn_matmul_i8_workspace_size(a, w) > 0
    most, far = int(squares(a).max()), squares(w).cpu().double() * int(squares(a).max())
    assert most <= CAREFUL and (far > FAR).nonzero().flatten().tolist() == sorted(channels)
    assert int((a.double() @ w[3].double()).max()) > 2 ** 24
    check(a, w, dtype=dtype)


@pytest.mark.parametrize("M", [128, 250])
def test_sums_at_the_border(M):
    """Every sum just under 2^24 in some tiles and just over it in others, with odd sums of both."""
    K, N = 6144, 19456
    a, w = torch.full((M, K), 41, dtype=torch.int8, device="cuda"), codes(2, N, K, -20, 20)
    a[M // 3, 9] = 40
    w[256:512], w[1024:1280] = 66, 67
    w[300:400, 0], w[1100:1200, 0] = 65, 66
    assert gdn.gdn_matmul_i8_workspace_size(a, w) > 0
    sums = a.double() @ w.double().t()
    assert 16_600_000 < sums[:, 256:512].min() and sums[:, 256:512].max() < 2 ** 24
    assert sums[:, 1024:1280].min() > 2 ** 24
    assert (sums[:, [300, 1100]] % 2 == 1).any(0).all() and int(squares(a).max()) <= CAREFUL
    far = squares(w).cpu().double() * int(squares(a).max()) > FAR
    assert not far[:1024].any() and far[1024:1280].all() and not far[1280:].any()
    check(a, w, dtype=F32)


def test_tiles_made_again_of_very_many():
    """More than a thousand tiles a pair of CTAs: those behind share one mark."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    M, N, K = 65, pairs * 1026 * 256, 1280
    if torch.cuda.mem_get_info()[0] < 2 * N * (K + 6 * M):
        pytest.skip("not enough memory")
    a, kinds = codes(1, M, K, -30, 30), codes(2, 64, K, -30, 30)
    gen = torch.Generator().manual_seed(5)
    a[[0, 64]] = torch.randint(107, 109, (2, K), generator=gen, dtype=torch.int8).cuda()
    w = kinds.repeat(N // 64, 1)
    tiles = [0, pairs * 500 + 3, pairs * 1022 + 1, pairs * 1023 + 5, pairs * 1024 + 5, pairs * 1026 - 1]
    channels = [256 * t + (7 if t % 2 else 200) for t in tiles]
    w[channels] = torch.randint(-128, -126, (len(channels), K), generator=gen, dtype=torch.int8).cuda()
    assert gdn.gdn_matmul_i8_workspace_size(a, w) > 0
    assert int(squares(a).max()) <= CAREFUL and int(squares(a).max()) * int(squares(w[channels]).max()) > FAR
    assert int((a.double() @ w[channels].double().t()).abs().max()) > 2 ** 24
    sa, sw = scales(1, M), scales(2, 64).repeat(N // 64)
    out = gdn.gdn_matmul_i8(a, sa, w, sw, dtype=F32)
    want = ref.product(a, sa, kinds, sw[:64], None, F32).cuda()
    large = ref.product(a, sa, w[channels], sw[channels], None, F32)
    assert_bits_equal(out[:, channels].cpu(), large, "large sums")
    out[:, channels] = want[:, [c % 64 for c in channels]]
    for m in range(M):
        assert (out[m].view(-1, 64) == want[m]).all(), m


@pytest.mark.parametrize("M,N", [(70, 2600), (70, 19456), (140, 2600), (140, 19456)])
def test_longest_rows_of_pairs(M, N):
    """K as long as it may be: sums and sums of squares up to 2^31, tiles in parts and whole."""
    K = 131071
    a, kinds = codes(1, M, K, pad=1), codes(2, 8, K)
    a[0], a[1], a[M - 1] = -128, 127, -128
    kinds[0], kinds[1], kinds[2, K // 2:] = -128, 127, -128
    w = torch.empty(N, K + 1, dtype=torch.int8, device="cuda")
    w.view(-1, 8, K + 1)[:, :, :K] = kinds
    w = w[:, :K]
    assert gdn.gdn_matmul_i8_workspace_size(a, w) > 0
    sa, sw = scales(1, M), scales(2, 8)
    out = gdn.gdn_matmul_i8(a, sa, w, sw.repeat(N // 8), dtype=F32)
    want = ref.product(a, sa, kinds, sw, None, F32).cuda()
    assert (out.view(M, -1, 8) == want[:, None]).all()
