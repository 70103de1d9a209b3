"""Host-side checks of the linear-attention and cache entries (no GPU): refusals come back
before anything is launched, and the reference forms of the tests agree with themselves."""
import ctypes

import numpy as np
import pytest
import torch

import linear_ref as ref
from gated_deltanet_linear_11_gb300 import _lib, build
from test_abi_cpu import FAKE, desc, no_gpu


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def offsets(*cu):
    return ctypes.cast((ctypes.c_int32 * len(cu))(*cu), ctypes.c_void_p)


def cache(**kw):
    c = _lib.GdnKvCache()
    c.data = c.block_table = c.kv_lens = FAKE
    c.pages, c.page_size, c.Hkv, c.head_dim, c.table_width, c.N = 4, 16, 2, 128, 2, 1
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


@no_gpu
def test_linear_prefill_refusals(lib):
    def call(q=None, k=None, v=None, o=None, g=FAKE, cu=(0, 8), N=1, h0=None):
        args = [ctypes.byref(x) for x in (q or desc(8, 2, 128), k or desc(8, 2, 128),
                                          v or desc(8, 4, 128))]
        return lib.gdn_linear_prefill(*args, g, 1, FAKE, offsets(*cu), N, 1.0, 0, h0,
                                      ctypes.byref(o or desc(8, 4, 128)), None, None, 0, None,
                                      None)
    assert call(g=None) == 1
    assert call(v=desc(8, 3, 128), o=desc(8, 3, 128)) == 2
    assert call(k=desc(7, 2, 128)) == 2
    assert call(q=desc(8, 2, 128, stride=(128, 8 * 128, 1))) == 3
    assert call(q=desc(8, 2, 128, ptr=FAKE + 2)) == 3
    assert call(h0=FAKE + 4) == 3
    assert call(o=desc(8, 4, 128, dtype=_lib.GDN_F32)) == 4
    assert call(cu=(0, 9)) == 5
    assert call(cu=(0, 9, 8), N=2) == 5
    assert call(q=desc(8, 2, 96), k=desc(8, 2, 96), v=desc(8, 4, 96), o=desc(8, 4, 96)) == 6
    assert call(cu=(0,), N=0, q=desc(0, 2, 128), k=desc(0, 2, 128), v=desc(0, 4, 128),
                o=desc(0, 4, 128)) == 0


@no_gpu
def test_linear_decode_refusals(lib):
    def call(T=4, P=4, state=FAKE, idx=None, g=FAKE, D=128):
        a, b = desc(T, 2, D), desc(T, 4, D)
        r = ctypes.byref
        return lib.gdn_linear_decode(r(a), r(a), r(b), g, 0, state, P, idx, 1.0, 0, r(b), None,
                                     None)
    assert call(P=3) == 2
    assert call(state=None) == 1
    assert call(state=FAKE + 4) == 3
    assert call(g=None) == 1
    assert call(D=256) == 6
    assert call(T=0) == 0


@no_gpu
def test_kv_refusals(lib):
    r = ctypes.byref

    def append(c=None, T=8, cu=(0, 8), k=None, v=None, q=None, qo=None, cos=None, sin=None, rot=0,
               rows=100):
        return lib.gdn_kv_append(c or cache(), FAKE if cu else None, offsets(*cu) if cu else None,
                                 r(k or desc(T, 2, 128)), r(v or desc(T, 2, 128)),
                                 r(q) if q else None, r(qo) if qo else None, cos, sin, rows, rot,
                                 0, None, None)
    assert append(c=cache(data=None)) == 1
    assert append(c=cache(kv_lens=None)) == 1
    assert append(c=cache(data=FAKE + 4)) == 3
    assert append(c=cache(page_size=24)) == 6
    assert append(c=cache(page_size=8)) == 6
    assert append(c=cache(head_dim=96)) == 6
    assert append(c=cache(Hkv=3)) == 2
    assert append(c=cache(pages=-1)) == 2
    assert append(cu=(0, 7)) == 5
    assert append(cu=None) == 5                        # eight rows, one sequence
    assert append(v=desc(8, 2, 128, dtype=_lib.GDN_F32)) == 4
    assert append(q=desc(8, 4, 128)) == 1              # no q_out
    assert append(q=desc(8, 4, 128), qo=desc(8, 4, 128)) == 3      # in place
    assert append(cos=FAKE) == 1
    assert append(cos=FAKE, sin=FAKE, rot=24) == 6
    assert append(cos=FAKE, sin=FAKE, rot=256) == 6
    assert append(cos=FAKE, sin=FAKE, rot=64, rows=0) == 2

    def attend(q=None, o=None, max_len=32, c=None):
        return lib.gdn_kv_attention(c or cache(), FAKE, offsets(0, 8), max_len,
                                    r(q or desc(8, 4, 128)), 1.0, 0, r(o or desc(8, 4, 128)), None,
                                    None, 0, None, None)
    assert attend(q=desc(8, 3, 128), o=desc(8, 3, 128)) == 2
    assert attend(o=desc(8, 4, 128, dtype=_lib.GDN_F32)) == 4
    assert attend(max_len=-1) == 2
    assert attend(q=desc(8, 4, 64), o=desc(8, 4, 64)) == 2
    assert [lib.gdn_kv_record_bytes(d) for d in (64, 128, 256, 96, 0)] == [40, 80, 160, 0, 0]


@no_gpu
def test_limits_and_missing_workspaces(lib):
    r = ctypes.byref

    def attend(T=8, Hq=4, max_len=32):
        x = desc(T, Hq, 128)
        return lib.gdn_kv_attention(cache(), FAKE, offsets(0, T), max_len, r(x), 1.0, 0, r(x), None,
                                    None, 0, None, None)
    assert attend(max_len=(1 << 30) + 1) == 2
    assert attend(T=1 << 26, Hq=32) == 2
    assert attend(max_len=1000) == 9                   # splits need a workspace
    x = desc(300, 2, 64, dtype=_lib.GDN_F32)
    size = lib.gdn_linear_prefill_workspace_size(offsets(0, 300), 1, 300, 2, 2, 64, _lib.GDN_F32, 0)
    assert size >= 3 * 2 * 64 * 64 * 4                 # three ranges begin from a state each

    def prefill(ws, nbytes):
        return lib.gdn_linear_prefill(r(x), r(x), r(x), FAKE, 1, FAKE, offsets(0, 300), 1, 1.0, 0,
                                      None, r(x), None, ws, nbytes, None, None)
    assert prefill(None, size) == 9
    assert prefill(FAKE, size - 1) == 9
    assert prefill(FAKE + 16, size) == 9


def test_forced_errors_reach_the_new_entries(monkeypatch):
    gdn = pytest.importorskip("gated_deltanet_linear_11_gb300")
    z = torch.zeros(1)
    for name, nargs in (("gdn_linear_prefill", 5), ("gdn_linear_decode", 5), ("gdn_kv_append", 5),
                        ("gdn_kv_read", 3), ("gdn_kv_attention", 4)):
        monkeypatch.setenv("GDN_FORCE_ERROR", name + "=7")
        with pytest.raises(gdn.GdnError) as e:
            getattr(gdn, name)(*[z] * nargs)
        assert e.value.code == 7
        monkeypatch.delenv("GDN_FORCE_ERROR")
        with pytest.raises(ValueError):
            getattr(gdn, name)(*[z] * nargs)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_reference_format_round_trip(D):
    """The orders are permutations, and stored values lie within half a step of x (plus the
    fp16 rounding of the minimum, which shifts the levels)."""
    for order in (ref.key_order(D), ref.value_order(D)):
        assert sorted(order) == list(range(D))
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, D)).astype(np.float32)
    for order in (ref.key_order(D), ref.value_order(D)):
        rec = ref.records(x, order)
        assert rec.shape[-1] == D // 2 + D // 8
        g = x.reshape(5, 3, D // 32, 32)
        step = (g.max(-1) - g.min(-1)) / 15
        err = np.abs(ref.values(rec, order).reshape(g.shape) - g).max(-1)
        assert np.all(err <= 0.5 * step * (1 + 2.0 ** -10) + 2.0 ** -10 * np.abs(g).max(-1))


def test_reference_recurrence_closed_form():
    """With one head and a constant decay, o_t is the decayed sum over earlier tokens."""
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((7, 1, 4)) for _ in range(3))
    o, h, _, _ = ref.linear_scan(q, k, v, np.array([-0.3]), [0, 7], None, 2.0)
    for t in range(7):
        want = sum(np.exp(-0.3 * (t - j)) * (q[t, 0] @ k[j, 0]) * v[j, 0] for j in range(t + 1))
        assert np.allclose(o[t, 0], 2 * want)
    assert np.allclose(h[0, 0], sum(np.exp(-0.3 * (6 - j)) * np.outer(k[j, 0], v[j, 0]) for j in range(7)))
