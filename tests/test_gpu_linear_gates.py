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
