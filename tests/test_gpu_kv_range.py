"""Attention over the 4-bit cache across the format's range: groups of large and of small scale,
rows that one key dominates, and bad entries of the block table.  Bounds as in
test_gpu_kv_cache.py: q or the values are scaled by powers of two, which changes no rounding.
"""
import numpy as np
import pytest
import torch

import linear_ref as ref
from gpu_util import assert_bits_equal, np64
from test_gpu_kv_cache import attention_case, check_attention, offsets, run_attention

pytestmark = pytest.mark.gpu

gdn = pytest.importorskip("gated_deltanet_linear_11_gb300")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load()


def scale_records(c, which, f, every=1):
    """Scales and minima of every `every`-th slot of the keys (0) or values (1) times f, within
    the format's range."""
    D = c["D"]
    par = c["cache"][:, which, :, ::every, D // 2:]
    with np.errstate(invalid="ignore"):    # NaN past the sequences' ends
        x = np.ascontiguousarray(par).view(np.float16).astype(np.float32) * np.float32(f)
        x = np.clip(x, -65504, 65504).astype(np.float16)
    c["cache"][:, which, :, ::every, D // 2:] = x.view(np.uint8)
    return c


# a few rows (split and whole), and pieces of prompts with many
ROWS = [([1, 3], [700, 40]), ([40, 1], [300, 700]), ([200, 161], [400, 170])]


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 32, 8), (128, 32, 8), (256, 8, 2)])
@pytest.mark.parametrize("ms,lens", ROWS)
@pytest.mark.parametrize("every", [1, 5, 16])
def test_attention_keys_of_large_scale(D, Hq, Hkv, ms, lens, every):
    """Key groups with scales up to 6550 (codes times scales past the fp16 range), alone and
    among others, against queries as much smaller."""
    c = attention_case(41, D, Hq, Hkv, 16, ms, lens)
    scale_records(c, 0, 2.0 ** 14, every)
    c["q"] *= 2.0 ** -14
    check_attention(c, *run_attention(c))


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 32, 8), (128, 32, 8), (256, 8, 2)])
@pytest.mark.parametrize("ms,lens", ROWS)
@pytest.mark.parametrize("simt", [False, True])
def test_attention_over_clamped_keys(D, Hq, Hkv, ms, lens, simt):
    """Keys as append stores them, with infinities and values past fp16 clamped to +-65504."""
    c = attention_case(42, D, Hq, Hkv, 16, ms, lens)
    rng = np.random.default_rng(43)
    k = rng.standard_normal(c["cache"][:, 0].shape[:-1] + (D,)).astype(np.float32)
    k[:, :, ::7, 5] = np.inf
    k[:, :, ::11, 40] = -np.inf
    k[:, :, 3, 32:64] *= np.float32(1e6)
    c["cache"][:, 0] = ref.records(k, ref.key_order(D))
    c["q"] *= 2.0 ** -15
    check_attention(c, *run_attention(c, simt=simt))


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (64, 8, 1), (128, 8, 2), (128, 12, 1), (256, 2, 2),
                                      (256, 12, 1), (256, 24, 1)])
@pytest.mark.parametrize("ms,lens", [([1, 2], [1500, 90]), ([260], [700])])
@pytest.mark.parametrize("f", [2.0 ** -8, 2.0 ** -11, 2.0 ** 10, 2.0 ** 14])
def test_attention_values_of_any_scale(D, Hq, Hkv, ms, lens, f):
    c = attention_case(44, D, Hq, Hkv, 16, ms, lens)
    check_attention(c, *run_attention(scale_records(c, 1, f)))


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 1), (128, 8, 2), (256, 8, 1), (256, 24, 1)])
@pytest.mark.parametrize("big", ["late", "early", "rows"])
def test_attention_values_of_mixed_scale(D, Hq, Hkv, big):
    """Groups of very different scales: each is held to its own size."""
    c = attention_case(45, D, Hq, Hkv, 16, [2, 1], [1500, 600])
    with np.errstate(invalid="ignore"):    # NaN past the sequences' ends
        par = c["cache"][:, 1, :, :, D // 2:].copy().view(np.float16).astype(np.float32)
    par = par.reshape(par.shape[:-1] + (D // 32, 2))
    f = np.ones(par.shape[:-1], np.float32)
    if big == "rows":                      # groups of one record
        f[..., 1] = 4096.0
    else:                                  # blocks of a sequence
        for n, L in enumerate(c["lens"]):
            pages = c["table"][n, :-(-int(L) // 16)]
            half = len(pages) // 2
            for x, p in enumerate(pages[half:] if big == "late" else pages[:half]):
                f[p] = 2.0 ** (4 + 2 * (x % 5))
    par = np.clip(par * f[..., None], -65504, 65504).astype(np.float16)
    c["cache"][:, 1, :, :, D // 2:] = np.ascontiguousarray(par).reshape(
        par.shape[:-2] + (-1,)).view(np.uint8)
    check_attention(c, *run_attention(c))


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 1), (128, 4, 1), (256, 2, 1), (256, 12, 1)])
@pytest.mark.parametrize("ms,L", [([1], 30000), ([260], 12000)])
@pytest.mark.parametrize("down", [13, 18, 21])
def test_attention_one_key_dominates(D, Hq, Hkv, ms, L, down):
    """Every other key weighs about 2^-down of the first; together they still count."""
    c = dominated_case(D, Hq, Hkv, ms, L, down)
    check_attention(c, *run_attention(c))


def dominated_case(D, Hq, Hkv, ms, L, down):
    c = attention_case(46, D, Hq, Hkv, 64, ms, [L])
    scale_records(c, 0, 2.0 ** -4)         # the others' scores lie close together
    scale_records(c, 1, 2.0 ** -3)
    q = c["q"].float()
    q[..., :32] = q[..., :32] * 0.1 + 1.0
    c["q"] = q.to(torch.bfloat16)
    at = c["cache"][c["table"][0, 0], 0, :, 0]
    at[:, :D // 2] = 0
    x = down * np.log(2.0) * D ** 0.5 / 32
    pair = np.zeros((D // 32, 2), np.float16)
    pair[0, 1] = x
    at[:, D // 2:] = pair.reshape(-1).view(np.uint8)
    # values that do not cancel over the keys
    par = c["cache"][:, 1, :, :, D // 2:].copy().view(np.float16)
    par[..., 1::2] = 0.25 * par[..., 0::2]
    c["cache"][:, 1, :, :, D // 2:] = par.view(np.uint8)
    return c


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("down", [13, 21])
def test_attention_one_key_dominates_many_rows(D, down):
    """The same for a piece of a prompt; its last rows are looked at."""
    c = dominated_case(D, 32, 1, [170], 30000, down)
    o, lse = run_attention(c)
    end = dict(c, q=c["q"][-3:], ms=[3])
    check_attention(end, o[-3:], lse[-3:])


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 2), (128, 8, 2), (256, 8, 2)])
def test_attention_long_runs_beside_splits(D, Hq, Hkv):
    """Sequences beside one whose keys stay in a long run: the bits that they give beside one of
    as many new tokens and a short run."""
    ms, lens = [260, 1, 2], [9500, 1900, 700]
    c = attention_case(48, D, Hq, Hkv, 32, ms, lens)
    o, lse = run_attention(c)
    check_attention(c, o, lse)
    short = dict(c, lens=np.array([300, 1900, 700], np.int32))
    o1, l1 = run_attention(short, max_kv_len=1900)
    assert_bits_equal(o[260:], o1[260:], "o beside a long run")
    assert_bits_equal(lse[260:], l1[260:], "lse beside a long run")


@pytest.mark.parametrize("D,Hq,ms,simt", [(128, 8, [1], False), (256, 24, [2], False),
                                          (128, 32, [170], False), (64, 32, [170], False),
                                          (128, 8, [3], True)])
@pytest.mark.parametrize("page", [-1, -2, -(1 << 31), 1 << 30])
def test_attention_reports_every_bad_page(D, Hq, ms, simt, page):
    """Any entry outside the cache within a sequence's length is left out and reported, the last
    one too; entries past its length are not looked at."""
    c = attention_case(47, D, Hq, 1, 16, ms, [ms[0] + 130])
    last = (ms[0] + 129) // 16
    for at in (2, last, last + 1):
        bad = dict(c, table=c["table"].copy())
        bad["table"][0, at] = page
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, _ = run_attention(bad, simt=simt, status=status)
        assert int(status) == (10 if at <= last else 0), (at, int(status))
        assert bool(o.isfinite().all())


def test_attention_with_nothing_to_join():
    """Short sequences under a bound that allows splits: the join has no row of its own, and what
    comes next in the stream sees the outputs."""
    c = attention_case(49, 128, 8, 2, 16, [1] * 40, [100] * 40)
    want, _ = run_attention(c, max_kv_len=100)
    q, cache, table, lens = c["q"].cuda(), torch.from_numpy(c["cache"]).cuda(), \
        torch.from_numpy(c["table"]).cuda(), torch.from_numpy(c["lens"]).cuda()
    o, got = torch.empty_like(want), []
    for _ in range(50):
        o.fill_(float("nan"))
        gdn.gdn_kv_attention(q, cache, table, lens, max_kv_len=100000, o=o)
        got.append(o.clone())
    for x in got:
        assert_bits_equal(x, want, "a copy of the outputs")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("f", [2.0 ** -11, 2.0 ** 10])
def test_attention_many_rows_values_of_any_scale(D, f):
    c = attention_case(50, D, 32, 8, 16, [170], [300])
    check_attention(c, *run_attention(scale_records(c, 1, f)))


@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 2), (256, 2), (256, 12)])
def test_attention_scales_that_grow_along_a_long_run(D, Hq):
    """Sums that have been stowed before the first scales that the lift has no room for."""
    c = attention_case(51, D, Hq, 1, 64, [258], [9000])
    par = c["cache"][:, 1, :, :, D // 2:].copy()
    with np.errstate(invalid="ignore"):
        x = par.view(np.float16).astype(np.float32)
    for i, f in ((70, 2.0 ** 8), (100, 2.0 ** 9), (120, 2.0 ** 12)):
        x[c["table"][0, i]] *= f
    x = np.clip(x, -65504, 65504).astype(np.float16)
    c["cache"][:, 1, :, :, D // 2:] = x.view(np.uint8)
    end = dict(c, q=c["q"][-4:], ms=[4])
    o, lse = run_attention(c)
    check_attention(end, o[-4:], lse[-4:])
