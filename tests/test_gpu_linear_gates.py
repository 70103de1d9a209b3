"""Linear attention: decays over their whole range, values and gates that are not finite, and
the accuracy of final states, against 64 bits.

Bounds: a decay factor from expf is within 2 ulps, 2 * 2^-23, and the product with the state
rounds once more, so a step leaves at most 8 * 2^-24 of |e^g S| where nothing is added.
"""
import numpy as np
import pytest
import torch

import linear_ref as ref
from gpu_util import assert_bits_equal, np64
from test_gpu_linear import call, make

pytestmark = pytest.mark.gpu

gdn = pytest.importorskip("gated_deltanet_linear_11_gb300")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load()


# one head for each of these log decays
DECAYS = [-0.01, -0.3, -0.49, -0.51, -0.7] + [-float(x) for x in range(1, 41)]


def decayed_case(D, dtype, lens):
    """Tokens without keys, so that a state is its decays times what it was."""
    T, Hv = sum(lens), len(DECAYS)
    d = make(31, lens, 5, Hv, D, dtype, True, True)
    d["k"].zero_()
    d["h0"] += torch.sign(d["h0"])         # nothing near zero
    return d


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_decays(D, dtype):
    N = 3
    d = decayed_case(D, dtype, [1] * N)
    g = torch.tensor(DECAYS).expand(N, -1).contiguous()
    for gg in (g, g[0].contiguous()):
        state = d["h0"].cuda()
        gdn.gdn_linear_decode(d["q"].cuda(), d["k"].cuda(), d["v"].cuda(), gg.cuda(), state)
        want = np.exp(np64(g))[:, :, None, None] * np64(d["h0"])
        err = np.abs(np64(state) - want) / np.abs(want)
        assert err.max() <= 8 * ref.U_F32, "%.3g at g = %g" % (
            err.max(), DECAYS[int(err.max((0, 2, 3)).argmax())])


@pytest.mark.parametrize("D,dtype", [(16, torch.bfloat16), (32, torch.float32),
                                     (64, torch.float32), (64, torch.bfloat16),
                                     (128, torch.float32), (128, torch.bfloat16)])
@pytest.mark.parametrize("T", [2, 300])
@pytest.mark.parametrize("simt", [True, False])
def test_prefill_decays(D, dtype, T, simt):
    """One strong decay or two among tokens that keep the state."""
    d = decayed_case(D, dtype, [T])
    g = torch.zeros(T, len(DECAYS))
    g[T // 2] = g[T - 1] = torch.tensor(DECAYS)
    d["g"] = g
    _, h = call(d, simt=simt)
    want = np.exp(np64(g).sum(0))[:, None, None] * np64(d["h0"][0])
    err = np.abs(np64(h)[0] - want) / np.abs(want)
    # g of up to 40 is summed in fp32 before the tensor cores' and the ranges' exp: 80 * 2^-24
    lim = (16 + 80) * ref.U_F32
    assert err.max() <= lim, "%.3g at g = %g" % (err.max(), DECAYS[int(err.max((1, 2)).argmax())])


# where a value or a gate is not finite: inside a block of 32 tokens, at the start and the end of
# one, in a last chunk that is not full, in a sequence cut into ranges
PLACES = [([150], 5), ([150], 32), ([150], 127), ([150], 149), ([150], 0), ([60, 90], 100),
          ([300, 128], 200), ([2100], 1000), ([2100], 2090)]


def upto(lens, j):
    """(first token, end, index) of the sequence of token j."""
    cu = np.concatenate(([0], np.cumsum(lens))).tolist()
    n = max(i for i in range(len(lens)) if cu[i] <= j)
    return cu[n], cu[n + 1], n


@pytest.mark.parametrize("lens,j", PLACES)
@pytest.mark.parametrize("simt", [False, True])
def test_prefill_gate_nan_reaches_only_later_tokens(lens, j, simt):
    d = make(34, lens, 1, 2, 128, torch.bfloat16, True, True)
    o1, h1 = call(d, simt=simt)
    d["g"][j, 1] = float("nan")
    o2, h2 = call(d, simt=simt)
    a, b, n = upto(lens, j)
    assert bool(o2[j:b, 1].isnan().all()) and bool(h2[n, 1].isnan().all())
    assert_bits_equal(o1[:, 0], o2[:, 0], "the other head")
    rest = [i for i in range(len(lens)) if i != n]
    assert_bits_equal(h1[rest], h2[rest], "other sequences' states")
    before = [i for i in range(sum(lens)) if not a <= i or i >= b or i < j]
    if simt:
        assert_bits_equal(o1[before], o2[before], "earlier tokens")
    # (the tensor-core form takes the weights of that block of 32 from their exponents)
    _, _, oa, _ = ref.linear_scan(np64(d["q"]), np64(d["k"]), np64(d["v"]),
                                  np.nan_to_num(np64(d["g"])),
                                  np.concatenate(([0], np.cumsum(lens))).tolist(), np64(d["h0"]))
    assert np.all(np.abs(np64(o1[before]) - np64(o2[before])) <= 4 * ref.U_BF16 * oa[before])


@pytest.mark.parametrize("lens,j", PLACES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("simt", [False, True])
def test_prefill_values_reach_only_later_tokens(lens, j, bad, simt):
    """A value that is not finite makes its column so from its token on, and nothing else."""
    d = make(32, lens, 1, 2, 128, torch.bfloat16, True, True, slow=True)
    o1, h1 = call(d, simt=simt)
    d["v"][j, 1, 70] = bad
    d["v"][j, 0, 3] = bad
    o2, h2 = call(d, simt=simt)
    a, b, n = upto(lens, j)
    keep, keep_h = torch.ones(o1.shape, dtype=torch.bool), torch.ones(h1.shape, dtype=torch.bool)
    for h, c in ((1, 70), (0, 3)):
        assert not bool(o2[j:b, h, c].isfinite().any())
        assert not bool(h2[n, h, :, c].isfinite().any())
        keep[j:b, h, c] = False
        keep_h[n, h, :, c] = False
    assert_bits_equal(o1[keep], o2[keep], "outputs that the value does not reach")
    assert_bits_equal(h1[keep_h], h2[keep_h], "state columns that the value does not reach")


@pytest.mark.parametrize("simt", [False, True])
def test_prefill_many_values_not_finite(simt):
    """Several of them in one column and chunk, in all columns of a token, and in every token
    of a chunk; the first counts."""
    d = make(33, [400], 1, 3, 128, torch.bfloat16, True, False, slow=True)
    o1, h1 = call(d, simt=simt)
    d["v"][[40, 90, 200], 0, 9] = float("nan")
    d["v"][77, 1] = float("inf")
    d["v"][256:384, 2] = float("nan")
    o2, h2 = call(d, simt=simt)
    keep = torch.ones(o1.shape, dtype=torch.bool)
    keep[40:, 0, 9] = False
    keep[77:, 1] = False
    keep[256:, 2] = False
    assert_bits_equal(o1[keep], o2[keep], "outputs that no value reaches")
    assert not bool(o2[~keep.to(o2.device)].isfinite().any())
    assert not bool(h2[0, 1:].isfinite().any()) and not bool(h2[0, 0, :, 9].isfinite().any())


@pytest.mark.parametrize("lens,j", [([150], 40), ([2100], 700), ([2100, 90], 2150)])
def test_prefill_value_not_finite_with_the_state_in_place(lens, j):
    """The state that such a call starts from is still there where it runs again."""
    d = make(37, lens, 1, 2, 128, torch.bfloat16, True, True, slow=True)
    d["v"][j, 1, 70] = float("nan")
    o1, h1 = call(d)
    state = d["h0"].cuda()
    dev = {x: d[x].cuda() for x in ("q", "k", "v", "g", "cu")}
    o2, h2 = gdn.gdn_linear_prefill(dev["q"], dev["k"], dev["v"], dev["g"], dev["cu"],
                                    initial_state=state, final_state=state,
                                    cu_seqlens_host=d["cu"])
    assert_bits_equal(o1, o2, "o with the state in place")
    assert_bits_equal(h1, state, "state in place")
    assert bool(o2.isnan().any()) and int(h2.isnan().sum()) == 128


def test_debug_checks_take_cleared_states(monkeypatch):
    """g = -inf clears a state: a valid gate, with and without the debug checks."""
    d = make(36, [9], 2, 4, 128, torch.bfloat16)
    d["g"][3, 1] = d["g"][0, 0] = -float("inf")
    o1, h1 = call(d)
    dec = [d[x][:1].cuda() for x in "qkvg"]
    state = torch.ones(1, 4, 128, 128, device="cuda")
    monkeypatch.setenv("GDN_DEBUG", "1")
    o2, h2 = call(d)
    assert_bits_equal(o1, o2, "o")
    assert_bits_equal(h1, h2, "state")
    gdn.gdn_linear_decode(*dec, state)
    for bad in (float("inf"), float("nan")):
        d["g"][3, 1] = bad
        with pytest.raises(gdn.GdnError) as e:
            call(d)
        assert e.value.code == 11
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_linear_decode(*dec[:3], torch.full((4,), bad, device="cuda"), state)
        assert e.value.code == 11


def test_debug_checks_reach_the_last_word(monkeypatch):
    """More gates and more offsets than one step of the checks copies."""
    T, N = 6000, 5000
    d = make(38, [2] * 1000 + [1] * 4000, 1, 2, 16, torch.float32)
    dev = {x: d[x].cuda() for x in ("q", "k", "v", "g", "cu")}
    monkeypatch.setenv("GDN_DEBUG", "1")

    def prefill():
        return gdn.gdn_linear_prefill(dev["q"], dev["k"], dev["v"], dev["g"], dev["cu"],
                                      cu_seqlens_host=d["cu"])
    assert prefill()[0].shape[0] == T and d["cu"].numel() == N + 1
    dev["cu"][N - 1] -= 1
    with pytest.raises(gdn.GdnError) as e:
        prefill()
    assert e.value.code == 5
    dev["cu"][N - 1] += 1
    dev["g"][T - 1, 1] = float("nan")
    with pytest.raises(gdn.GdnError) as e:
        prefill()
    assert e.value.code == 11


@pytest.mark.parametrize("lens,Hv", [([500], 2), ([2500, 1600], 2), ([4096], 48)])
@pytest.mark.parametrize("slow", [True, False])
def test_prefill_state_accuracy(lens, Hv, slow):
    """Final states of the tensor-core form, whole and in ranges, by norm: keys as three bf16
    terms leave 2^-24 of a product, the sums of 128 products in fp32 and one rounding a chunk
    some more, together under 1.2e-6; with two terms the state is off by 3e-6."""
    d = make(35, lens, 1, Hv, 128, torch.bfloat16, True, True, slow=slow)
    if Hv > 2:                             # the same heads again: the 64-bit form is slow
        for x in ("v", "g"):
            d[x] = d[x][:, :2].repeat(*([1, Hv // 2] + [1] * (d[x].dim() - 2)))
        d["h0"] = d["h0"][:, :2].repeat(1, Hv // 2, 1, 1)
    _, h = call(d)
    _, rh, _, _ = ref.linear_scan(np64(d["q"]), np64(d["k"]), np64(d["v"][:, :2]),
                                  np64(d["g"][:, :2]),
                                  np.concatenate(([0], np.cumsum(lens))).tolist(),
                                  np64(d["h0"][:, :2]))
    for i in range(Hv):
        err = np.linalg.norm(np64(h[:, i]) - rh[:, i % 2]) / np.linalg.norm(rh[:, i % 2])
        assert err <= 1.2e-6, (i, err)


def test_prefill_values_not_finite_in_long_ranges():
    """Ranges of many chunks, some heads with such values and some without."""
    T, Hv = 4096, 48
    d = make(39, [T - 700, 700], 16, Hv, 128, torch.bfloat16, True, True, slow=True)
    o1, h1 = call(d)
    keep, keep_h = torch.ones(o1.shape, dtype=torch.bool), torch.ones(h1.shape, dtype=torch.bool)
    for t, h, c in ((0, 3, 0), (1300, 3, 127), (1407, 20, 64), (3000, 47, 31), (3395, 11, 90),
                    (3396, 12, 7), (4095, 5, 5)):
        d["v"][t, h, c] = float("nan")
        n, end = (0, T - 700) if t < T - 700 else (1, T)
        keep[t:end, h, c] = False
        keep_h[n, h, :, c] = False
    o2, h2 = call(d)
    assert_bits_equal(o1[keep], o2[keep], "outputs that no value reaches")
    assert_bits_equal(h1[keep_h], h2[keep_h], "state columns that no value reaches")
    assert bool(o2[~keep].isnan().all()) and bool(h2[~keep_h].isnan().all())
