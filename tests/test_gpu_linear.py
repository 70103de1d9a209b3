"""Linear attention with a decay for each head against its recurrence in 64 bits.

Bounds, from the roundings that each path makes (A: the same sums over absolute values):
* bf16 o: its own rounding (2^-8 |o|), and at most two of the factors of a term rounded to
  bf16 (2 * 2^-8 A), with half of one more for everything in fp32.
* fp32 o and all states: (T + D) roundings of 2^-24 A at most, and 2^-16 A for states whose
  keys go through the tensor cores in bf16 terms (twice the 2^-17 that two of them leave
  out).
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


def make(seed, lens, Hk, Hv, D, dtype, per_token=True, start=False, slow=False):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)

    def rnd(*s):
        return torch.randn(*s, generator=gen)
    d = dict(q=(rnd(T, Hk, D) * D ** -0.5).to(dtype), k=(rnd(T, Hk, D) * D ** -0.5).to(dtype),
             v=rnd(T, Hv, D).to(dtype))
    g = -torch.nn.functional.softplus(rnd(T, Hv) - (5.0 if slow else 2.0))
    d["g"] = g if per_token else g[0] * 0.1 if T else -torch.ones(Hv)
    d["h0"] = rnd(N, Hv, D, D) * 0.3 if start else None
    d["cu"] = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32)
    return d


def call(d, **kw):
    dev = {x: None if d[x] is None else d[x].cuda() for x in ("q", "k", "v", "g", "h0", "cu")}
    return gdn.gdn_linear_prefill(dev["q"], dev["k"], dev["v"], dev["g"], dev["cu"],
                                  initial_state=dev["h0"], cu_seqlens_host=d["cu"], **kw)


def check(d, o, hT, simt, scale=1.0):
    cu = d["cu"].tolist()
    with np.errstate(over="ignore"):
        ro, rh, oa, ha = ref.linear_scan(np64(d["q"]), np64(d["k"]), np64(d["v"]), np64(d["g"]),
                                         cu, None if d["h0"] is None else np64(d["h0"]), scale)
    T, D = d["q"].shape[0], d["q"].shape[2]
    f32 = (T + D) * ref.U_F32
    lim = f32 * oa if d["q"].dtype == torch.float32 else \
        ref.U_BF16 * np.abs(ro) + 2.5 * ref.U_BF16 * oa
    err = np.abs(np64(o) - ro)
    assert np.all(err <= lim + 1e-30), "o: %.3g of its bound" % float((err / (lim + 1e-30)).max())
    if hT is not None:
        err = np.abs(np64(hT) - rh)
        lim = (f32 + (0 if simt or d["q"].dtype == torch.float32 else 2.0 ** -16)) * ha
        assert np.all(err <= lim + 1e-30), "state: %.3g of its bound" % float((err / (lim + 1e-30)).max())


LENS = [[1], [64], [100], [0, 1, 2, 63, 64, 65, 0, 127, 128, 129], [513], [300, 700]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("per_token,start", [(True, True), (False, False)])
def test_prefill_bf16_128(lens, per_token, start):
    d = make(1, lens, 2, 6, 128, torch.bfloat16, per_token, start)
    o, h = call(d)
    check(d, o, h, False)


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill_cuda_cores(D, dtype):
    d = make(2, [5, 0, 33, 64, 130], 2, 4, D, dtype, True, True)
    o, h = call(d, simt=True, scale=0.5)
    check(d, o, h, True, 0.5)
    o, h = call(d, scale=0.5)
    check(d, o, h, dtype == torch.float32 or D != 128, 0.5)


@pytest.mark.parametrize("D,dtype", [(16, torch.float32), (32, torch.bfloat16),
                                     (64, torch.float32), (64, torch.bfloat16),
                                     (128, torch.float32)])
def test_prefill_cuda_cores_ranges(D, dtype):
    """Sequences cut into ranges beside short ones: a memory of hundreds of tokens, cleared
    states, the state in place, and the bits that each sequence gives alone."""
    lens = [700, 255, 1, 256, 0, 1000]
    d = make(12, lens, 1, 2, D, dtype, True, True, slow=True)
    d["g"][300, 1] = -float("inf")
    d["g"][1500:1510, 0] = -300.0
    o, h = call(d, simt=True)
    check(d, o, h, True)
    state = d["h0"].cuda()
    o2, _ = gdn.gdn_linear_prefill(d["q"].cuda(), d["k"].cuda(), d["v"].cuda(), d["g"].cuda(),
                                   d["cu"].cuda(), initial_state=state, final_state=state,
                                   simt=True, cu_seqlens_host=d["cu"])
    assert_bits_equal(o, o2, "o with the state in place")
    assert_bits_equal(h, state, "state in place")
    cu = d["cu"].tolist()
    for n in (0, 1, 5):
        sl = slice(cu[n], cu[n + 1])
        one = dict(q=d["q"][sl], k=d["k"][sl], v=d["v"][sl], g=d["g"][sl], h0=d["h0"][n:n + 1],
                   cu=torch.tensor([0, lens[n]], dtype=torch.int32))
        o1, h1 = call(one, simt=True)
        assert_bits_equal(o[sl], o1, "o of sequence %d" % n)
        assert_bits_equal(h[n:n + 1], h1, "state of sequence %d" % n)
    # per-head decays, no state to start from
    d = make(13, [511, 257], 1, 2, D, dtype, False, False)
    check(d, *call(d, simt=True), True)


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (3, 3), (1, 5), (4, 8)])
def test_prefill_head_layouts(Hk, Hv):
    d = make(3, [200, 17], Hk, Hv, 128, torch.bfloat16, True, True)
    o, h = call(d)
    check(d, o, h, False)


def test_prefill_long_slow_decay():
    """Many ranges and a memory of hundreds of tokens: the start states matter."""
    for per_token in (True, False):
        d = make(4, [2500, 1111], 1, 2, 128, torch.bfloat16, per_token, True, slow=True)
        o, h = call(d)
        check(d, o, h, False)


@pytest.mark.parametrize("simt", [False, True])
def test_prefill_extreme_gates(simt):
    """No decay, a decay that underflows, and -inf (a cleared state) at scattered tokens."""
    d = make(5, [260, 140], 1, 3, 128, torch.bfloat16, True, True)
    g = d["g"]
    g[:, 0] = 0.0
    g[::7, 1] = -300.0
    g[5::50, 2] = -float("inf")
    g[261, 2] = -float("inf")
    o, h = call(d, simt=simt)
    check(d, o, h, simt)
    # g = -inf everywhere: o_t = (q.k) v of the token alone
    d["g"] = torch.full((400, 3), -float("inf"))
    o, h = call(d, simt=simt)
    check(d, o, h, simt)


@pytest.mark.parametrize("simt", [False, True])
def test_prefill_keeps_sequences_apart(simt):
    """NaN and infinities in one sequence stay out of its neighbours, before and after."""
    lens = [70, 90, 200, 1]
    clean = make(6, lens, 1, 2, 128, torch.bfloat16, True, True)
    dirty = {k: (x.clone() if isinstance(x, torch.Tensor) else x) for k, x in clean.items()}
    for name in ("q", "k", "v"):
        dirty[name][70:160] = float("nan")
        dirty[name][80:100] = float("inf")
    dirty["g"][70:160] = float("nan")
    o1, h1 = call(clean, simt=simt)
    o2, h2 = call(dirty, simt=simt)
    keep = [i for i in range(361) if not 70 <= i < 160]
    assert_bits_equal(o1[keep], o2[keep], "o next to a NaN sequence")
    assert_bits_equal(h1[[0, 2, 3]], h2[[0, 2, 3]], "states next to a NaN sequence")
    assert bool(torch.isnan(o2[80:160]).all()) and bool(torch.isnan(h2[1]).all())


def test_prefill_batch_invariance():
    lens = [700, 1, 2050, 64, 0, 515]
    d = make(7, lens, 2, 4, 128, torch.bfloat16, True, True, slow=True)
    o, h = call(d)
    cu = d["cu"].tolist()
    for n, L in enumerate(lens):
        sl = slice(cu[n], cu[n + 1])
        one = dict(q=d["q"][sl], k=d["k"][sl], v=d["v"][sl], g=d["g"][sl], h0=d["h0"][n:n + 1],
                   cu=torch.tensor([0, L], dtype=torch.int32))
        o1, h1 = call(one)
        assert_bits_equal(o[sl], o1, "o of sequence %d" % n)
        assert_bits_equal(h[n:n + 1], h1, "state of sequence %d" % n)


def test_prefill_views_streams_and_in_place_state():
    """q, k, v as strided views of one packed tensor, on a stream of the caller's, with
    final_state over initial_state; the same bits as from contiguous copies."""
    lens, Hk, Hv, D = [150, 333], 2, 4, 128
    d = make(8, lens, Hk, Hv, D, torch.bfloat16, True, True)
    o1, h1 = call(d)
    T = sum(lens)
    packed = torch.cat((d["q"].reshape(T, -1), d["k"].reshape(T, -1), d["v"].reshape(T, -1)), 1)
    y = torch.full((T, packed.shape[1] + 64), float("nan"), dtype=torch.bfloat16)
    y[:, :packed.shape[1]] = packed
    y = y.cuda()
    q, k, v = gdn.split_qkv(y, Hk, Hv, D, D)
    st = torch.cuda.Stream()
    h, g, cu = d["h0"].cuda(), d["g"].cuda(), d["cu"].cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        o2, h2 = gdn.gdn_linear_prefill(q, k, v, g, cu, initial_state=h, final_state=h,
                                        cu_seqlens_host=d["cu"])
    st.synchronize()
    assert h2.data_ptr() == h.data_ptr()
    assert_bits_equal(o1, o2, "o from strided views")
    assert_bits_equal(h1, h2, "state in place")


def test_prefill_no_tokens():
    d = make(9, [0, 0], 1, 2, 128, torch.bfloat16, True, True)
    o, h = call(d)
    assert o.shape[0] == 0
    assert_bits_equal(h, d["h0"].cuda(), "state without tokens")
    d["h0"] = None
    _, h = call(d)
    assert not bool(h.any())


def test_prefill_graph_replay():
    d = make(10, [640, 77], 1, 2, 128, torch.bfloat16, True, True)
    dev = {x: d[x].cuda() for x in ("q", "k", "v", "g", "h0", "cu")}
    o1, h1 = call(d)
    ws = torch.empty(max(16, gdn.gdn_linear_prefill_workspace_size(d["cu"], 717, 1, 2, 128)),
                     dtype=torch.uint8, device="cuda")
    o, h = torch.empty_like(o1), torch.empty_like(h1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_linear_prefill(dev["q"], dev["k"], dev["v"], dev["g"], dev["cu"],
                               initial_state=dev["h0"], o=o, final_state=h, workspace=ws,
                               cu_seqlens_host=d["cu"])
    for _ in range(2):
        o.fill_(float("nan"))
        h.fill_(float("nan"))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert_bits_equal(o, o1, "o of a replay")
        assert_bits_equal(h, h1, "state of a replay")


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode(D, dtype):
    N, Hk, Hv, P = 5, 2, 6, 9
    d = make(11, [1] * N, Hk, Hv, D, dtype)
    gen = torch.Generator().manual_seed(12)
    pool = torch.randn(P, Hv, D, D, generator=gen)
    idx = torch.randperm(P, generator=gen)[:N].int()
    for g in (d["g"], d["g"][0].contiguous()):
        state = pool.cuda()
        o = gdn.gdn_linear_decode(d["q"].cuda(), d["k"].cuda(), d["v"].cuda(), g.cuda(), state,
                                  state_idx=idx.cuda(), scale=0.7)
        sel = idx.long()
        ro, rh, oa, ha = ref.linear_scan(np64(d["q"]), np64(d["k"]), np64(d["v"]), np64(g),
                                         list(range(N + 1)), np64(pool[sel]), 0.7)
        lim = (D + 4) * ref.U_F32 * oa + (ref.U_BF16 * np.abs(ro) if dtype == torch.bfloat16 else 0)
        assert np.all(np.abs(np64(o) - ro) <= lim)
        assert np.all(np.abs(np64(state)[sel.numpy()] - rh) <= 4 * ref.U_F32 * ha)
        rest = [i for i in range(P) if i not in idx.tolist()]
        assert_bits_equal(state[rest], pool[rest].cuda(), "untouched slots")


def test_decode_many_steps_slow_decay():
    """Decode after a prompt, token by token, equals the prompt run to the end."""
    T, P0 = 400, 300
    d = make(13, [T], 1, 2, 128, torch.bfloat16, False, True, slow=True)
    o, h = call(d)
    head = {k: (x[:P0] if k in "qkv" else x) for k, x in d.items()}
    head["cu"] = torch.tensor([0, P0], dtype=torch.int32)
    _, state = call(head)
    q, k, v, g = (d[x].cuda() for x in "qkvg")
    outs = [gdn.gdn_linear_decode(q[t:t + 1], k[t:t + 1], v[t:t + 1], g, state)
            for t in range(P0, T)]
    ro, rh, oa, ha = ref.linear_scan(np64(d["q"]), np64(d["k"]), np64(d["v"]), np64(d["g"]),
                                     [0, T], np64(d["h0"]))
    assert np.all(np.abs(np64(torch.cat(outs)) - ro[P0:]) <=
                  ref.U_BF16 * np.abs(ro[P0:]) + 2.0 ** -15 * oa[P0:])
    assert np.all(np.abs(np64(state) - rh) <= ((T + 128) * ref.U_F32 + 2.0 ** -16) * ha)


def test_decode_bad_index_is_reported_and_skipped():
    d = make(14, [1] * 4, 1, 2, 128, torch.bfloat16)
    pool = torch.randn(3, 2, 128, 128).cuda()
    before = pool.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.tensor([2, -1, 3, 0], dtype=torch.int32, device="cuda")
    o = torch.full((4, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_linear_decode(d["q"].cuda(), d["k"].cuda(), d["v"].cuda(), d["g"].cuda(), pool,
                          state_idx=idx, o=o, status=status)
    assert int(status) == 10
    assert bool((o[1:3] == 7.0).all()) and not bool((o[0] == 7.0).all())
    assert_bits_equal(pool[1], before[1], "slot that no index names")


def test_refusals():
    d = make(15, [8], 2, 4, 128, torch.bfloat16)
    q, k, v, g, cu = (d[x].cuda() for x in ("q", "k", "v", "g", "cu"))
    with pytest.raises(ValueError):
        gdn.gdn_linear_prefill(q, k, v, g[:, :3], cu)
    with pytest.raises(TypeError):
        gdn.gdn_linear_prefill(q, k, v, g.double(), cu)
    with pytest.raises(ValueError):
        gdn.gdn_linear_prefill(q, k, v, g, cu, initial_state=torch.zeros(1, 4, 64, 128, device="cuda"))
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_linear_prefill(q, k.float(), v, g, cu)
    assert e.value.code == 4
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_linear_prefill(q[..., :96], k[..., :96], v[..., :96], g, cu)
    assert e.value.code in (3, 6)
    hf = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_linear_prefill(hf, hf, v, g, cu)
    assert e.value.code == 3
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_linear_prefill(q, k, v, g, torch.tensor([0, 7], dtype=torch.int32))
    assert e.value.code == 5


def test_debug_checks_refuse_bad_gates(monkeypatch):
    monkeypatch.setenv("GDN_DEBUG", "1")
    d = make(16, [8], 2, 4, 128, torch.bfloat16)
    d["g"][3, 1] = float("nan")
    with pytest.raises(gdn.GdnError) as e:
        call(d)
    assert e.value.code == 11
