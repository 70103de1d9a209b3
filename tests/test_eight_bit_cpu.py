"""Refusals of the operators around the mixers, before anything is launched (no GPU)."""
import ctypes

import pytest
import torch

from gated_deltanet_linear_11_gb300 import _lib, build, eight_bit
from test_abi_cpu import FAKE, desc, no_gpu

BF, F32, I8 = _lib.GDN_BF16, _lib.GDN_F32, _lib.GDN_I8


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def mat(rows, cols, dtype=BF, stride=None, ptr=FAKE):
    m = _lib.GdnMatrix()
    m.ptr, m.rows, m.cols, m.dtype = ptr, rows, cols, dtype
    m.stride = cols if stride is None else stride
    return m


def ref(x):
    return None if x is None else ctypes.byref(x)


@no_gpu
def test_quantize_rows_refusals(lib):
    def call(x=mat(4, 64), q=mat(4, 64, I8), scale=FAKE):
        return lib.gdn_quantize_rows(ref(x), ref(q), scale, None)
    assert call(x=None) == 1 and call(q=None) == 1 and call(scale=None) == 1
    assert call(x=mat(4, 64, ptr=None)) == 1
    assert call(q=mat(3, 64, I8)) == 2 and call(q=mat(4, 63, I8)) == 2
    assert call(x=mat(-1, 64)) == 2
    assert call(x=mat(4, 64, stride=63)) == 3 and call(x=mat(4, 64, ptr=FAKE + 1)) == 3
    assert call(scale=FAKE + 2) == 3
    assert call(x=mat(4, 64, I8)) == 4 and call(q=mat(4, 64)) == 4 and call(x=mat(4, 64, 9)) == 4
    assert call(x=mat(4, 32776), q=mat(4, 32776, I8)) == 6
    assert call(x=mat(0, 64, ptr=None), q=mat(0, 64, I8, ptr=None), scale=None) == 0


@no_gpu
def test_add_rmsnorm_refusals(lib):
    def call(x=mat(4, 64), r=mat(4, 64), o=mat(4, 64), w=mat(1, 64), eps=1e-6, y=mat(4, 64),
             scale=None):
        return lib.gdn_add_rmsnorm(ref(x), ref(r), ref(o), ref(w), 0.0, eps, ref(y), scale, None)
    assert call(x=None) == 1 and call(w=None) == 1 and call(y=None) == 1
    assert call(r=None) == 1 and call(o=None) == 1
    assert call(y=mat(4, 64, I8)) == 1                  # codes without scales
    assert call(scale=FAKE) == 1                        # scales without codes
    assert call(r=mat(3, 64)) == 2 and call(o=mat(4, 65)) == 2 and call(w=mat(1, 63)) == 2
    assert call(y=mat(5, 64)) == 2
    assert call(o=mat(4, 64, stride=8)) == 3
    assert call(r=mat(4, 64, F32)) == 4 and call(y=mat(4, 64, F32)) == 4
    assert call(w=mat(1, 64, I8)) == 4
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert call(eps=eps) == 6
    big = [mat(4, 40000) for _ in range(4)]
    assert call(big[0], big[1], big[2], mat(1, 40000), y=big[3]) == 6
    none = [mat(0, 64, ptr=None) for _ in range(4)]
    assert call(none[0], none[1], none[2], y=none[3]) == 0


@no_gpu
def test_gated_rmsnorm_refusals(lib):
    def call(x=desc(4, 2, 64), z=desc(4, 2, 64), w=mat(1, 64), eps=1e-6, y=mat(4, 128),
             scale=None):
        return lib.gdn_gated_rmsnorm(ref(x), ref(z), ref(w), eps, ref(y), scale, None)
    assert call(x=None) == 1 and call(z=None) == 1 and call(w=None) == 1 and call(y=None) == 1
    assert call(y=mat(4, 128, I8)) == 1
    assert call(z=desc(4, 3, 64)) == 2 and call(w=mat(1, 128)) == 2 and call(y=mat(4, 64)) == 2
    assert call(x=desc(4, 2, 64, stride=(64, 4 * 64, 1))) == 3
    assert call(x=desc(4, 2, 64, ptr=FAKE + 8)) == 3
    assert call(z=desc(4, 2, 64, dtype=F32)) == 4
    for D in (8, 48, 96, 512):
        assert call(desc(4, 2, D), desc(4, 2, D), mat(1, D), y=mat(4, 2 * D)) == 6
    assert call(desc(4, 200, 256), desc(4, 200, 256), mat(1, 256), y=mat(4, 200 * 256)) == 6
    assert call(eps=0.0) == 6


@no_gpu
def test_matmul_i8_refusals(lib):
    def call(a=mat(4, 64, I8), sa=FAKE, w=mat(8, 64, I8), sw=FAKE, bias=None, out=mat(4, 8),
             flags=_lib.GDN_PREFILL_SIMT):
        return lib.gdn_matmul_i8(ref(a), sa, ref(w), sw, ref(bias), ref(out), flags, None, 0,
                                 None, None)
    assert call(a=None) == 1 and call(w=None) == 1 and call(out=None) == 1
    assert call(sa=None) == 1 and call(sw=None) == 1
    assert call(w=mat(8, 63, I8)) == 2 and call(out=mat(4, 9)) == 2 and call(out=mat(3, 8)) == 2
    assert call(bias=mat(1, 7)) == 2 and call(bias=mat(2, 8)) == 2
    assert call(a=mat(4, 0, I8), w=mat(8, 0, I8)) == 2
    assert call(a=mat(4, 64, I8, stride=32)) == 3 and call(sa=FAKE + 1) == 3
    assert call(a=mat(4, 64)) == 4 and call(w=mat(8, 64, F32)) == 4 and call(out=mat(4, 8, I8)) == 4
    assert call(bias=mat(1, 8, I8)) == 4
    assert call(a=mat(4, 131072, I8), w=mat(8, 131072, I8)) == 6
    assert call(a=mat(0, 64, I8, ptr=None), sa=None, out=mat(0, 8, ptr=None)) == 0
    # rows off 16 bytes, and many tokens, need scratch
    assert call(a=mat(4, 65, I8), w=mat(8, 65, I8), flags=0) == 9
    assert call(a=mat(300, 64, I8), w=mat(8, 64, I8), out=mat(300, 8), flags=0) == 9


def test_matmul_i8_workspace(lib):
    """fp16 tokens and a sum of squares each for more than 64 tokens, and copies of rows that
    do not start on 16 bytes."""
    def f(a, w, flags=0):
        return lib.gdn_matmul_i8_workspace_size(ref(a), ref(w), flags)
    w = mat(8, 64, I8)
    assert f(mat(0, 64, I8), w) == f(mat(4, 64, I8), mat(0, 64, I8)) == 0
    assert f(mat(4, 0, I8), mat(8, 0, I8)) == f(mat(4, 64, I8), mat(8, 63, I8)) == 0
    assert f(mat(64, 64, I8), w) == 0
    assert f(mat(100, 64, I8), w) == 100 * 128 + 512            # 400 bytes, to 256
    assert f(mat(100, 64, I8), w, _lib.GDN_PREFILL_SIMT) == 0
    odd = mat(8, 65, I8)
    assert f(mat(1, 65, I8), odd) == 768                        # 8 rows of 80, to 256 bytes
    assert f(mat(3, 65, I8), odd) == 256 + 768
    assert f(mat(3, 65, I8, stride=80), mat(8, 65, I8, stride=80)) == 0
    assert f(mat(100, 65, I8), odd) == 768 + (100 * 72 * 2 + 255) // 256 * 256 + 512
    assert f(mat(3, 64, I8, ptr=FAKE + 1), w) == 256


def on_device(*shape, dtype=torch.bfloat16):
    """What the binding's checks look at, without a device."""
    class Tensor:
        is_cuda = True

        def __init__(self, inner):
            self.inner, self.dtype, self.shape = inner, inner.dtype, inner.shape

        def get_device(self):
            return 0

        def __getitem__(self, i):
            return Tensor(self.inner[i])

        def t(self):
            return Tensor(self.inner.t())

        def __getattr__(self, name):
            return getattr(self.inner, name)
    return Tensor(torch.zeros(*shape, dtype=dtype))


def test_binding_refusals(lib, monkeypatch):
    import gated_deltanet_linear_11_gb300 as gdn
    monkeypatch.setattr(gdn, "_current_device", lambda: 0)
    z = on_device
    for name in eight_bit.__all__:
        assert getattr(gdn, name) is getattr(eight_bit, name)
        if not name.endswith("_size"):
            assert hasattr(getattr(gdn, name), "__wrapped__"), name
    with pytest.raises(ValueError, match="CUDA device"):
        gdn.gdn_quantize_rows(torch.zeros(2, 4))
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        gdn.gdn_quantize_rows(z(2, 4, dtype=torch.float16))
    with pytest.raises(ValueError, match="rows, cols"):
        gdn.gdn_quantize_rows(z(2, 2, 4))
    with pytest.raises(ValueError, match="next to each other"):
        gdn.gdn_quantize_rows(z(4, 2).t())
    with pytest.raises(ValueError, match="x's shape"):
        gdn.gdn_add_rmsnorm(z(2, 4), z(4), z(3, 4), residual_out=z(2, 4))
    with pytest.raises(ValueError, match="residual_out"):
        gdn.gdn_add_rmsnorm(z(2, 4), z(4), residual_out=z(2, 4))
    with pytest.raises(ValueError, match="eight_bit"):
        gdn.gdn_add_rmsnorm(z(2, 4), z(4), scale=z(2, dtype=torch.float32))
    with pytest.raises(ValueError, match="y must be"):
        gdn.gdn_add_rmsnorm(z(2, 4), z(4), y=z(2, 4, dtype=torch.float32))
    with pytest.raises(ValueError, match="weight"):
        gdn.gdn_add_rmsnorm(z(2, 4), z(5), y=z(2, 4))
    with pytest.raises(ValueError, match="weight"):
        gdn.gdn_gated_rmsnorm(z(2, 3, 16), z(2, 3, 16), z(48), y=z(2, 48))
    i8 = torch.int8
    with pytest.raises(ValueError, match="rows of 16 codes"):
        gdn.gdn_matmul_i8(z(2, 16, dtype=i8), None, z(3, 8, dtype=i8), None)
    with pytest.raises(ValueError, match="a_scale"):
        gdn.gdn_matmul_i8(z(2, 16, dtype=i8), z(3, dtype=torch.float32), z(3, 16, dtype=i8),
                          z(3, dtype=torch.float32))
    with pytest.raises(TypeError, match="a must be int8"):
        gdn.gdn_matmul_i8(z(2, 16), None, z(3, 16, dtype=i8), None)
    monkeypatch.setenv("GDN_FORCE_ERROR", "gdn_matmul_i8=7")
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_matmul_i8(z(2, 16, dtype=i8), None, z(3, 16, dtype=i8), None)
    assert e.value.code == 7


@no_gpu
def test_smallest_eps(lib):
    """Beside an eps under 2^-126 the squares of small rows would lack digits: 3e-22 squared is 64
    of fp32's smallest steps."""
    x, z, w, g = mat(4, 64), desc(4, 1, 64), mat(1, 64), mat(4, 64)
    for eps in (1e-45, 1e-40, 1.17e-38):
        assert lib.gdn_add_rmsnorm(ref(x), None, None, ref(w), 0.0, eps, ref(g), None, None) == 6
        assert lib.gdn_gated_rmsnorm(ref(z), ref(z), ref(w), eps, ref(g), None, None) == 6
    none = mat(0, 64, ptr=None)
    assert lib.gdn_add_rmsnorm(ref(none), None, None, ref(w), 0.0, 2.0 ** -126, ref(none), None,
                               None) == 0
