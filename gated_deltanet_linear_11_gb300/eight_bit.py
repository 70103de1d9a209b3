"""The operators around the mixers: norms, rows in 8 bits and their products.

Part of the package's namespace, like every other entry (``gdn.gdn_add_rmsnorm``, ...).
"""
from __future__ import annotations

import torch

from . import (GDN_PREFILL_SIMT, _DT, _entry, _need_cuda, _on_device, _ptr, _raw_stream,
               _scratch, _view)
from . import _lib

__all__ = ["gdn_quantize_rows", "gdn_add_rmsnorm", "gdn_gated_rmsnorm", "gdn_matmul_i8",
           "gdn_matmul_i8_workspace_size"]


# Called once per layer and token, as the entries of the package's own module: descriptors are
# packed in one go, and the checks of the usual case come first.
_PACK = _lib.GDN_MATRIX_PACK.pack


def _names(dtypes):
    return " or ".join(str(x).replace("torch.", "") for x in dtypes)


def _matrix(name, t, dtypes):
    """gdn_matrix_t of a view [rows, cols] or [1, rows, cols], packed."""
    dt = dtypes.get(t.dtype)
    if dt is None:
        raise TypeError("%s must be %s, got %s" % (name, _names(dtypes), t.dtype))
    strides = t.stride()
    if len(strides) == 2:
        rows, cols = t.shape
        stride, unit = strides
    elif len(strides) == 3 and t.shape[0] == 1:
        _, rows, cols = t.shape
        _, stride, unit = strides
    else:
        raise ValueError("%s must be [rows, cols] or [1, rows, cols], got %s"
                         % (name, tuple(t.shape)))
    if unit != 1 and cols > 1 and rows > 0:
        raise ValueError("%s must have its rows' elements next to each other" % name)
    return _PACK(t.data_ptr(), rows, cols, stride, dt)


def _vector(name, t, n, dtypes):
    """gdn_matrix_t of a contiguous vector [n], packed (None for None)."""
    if t is None:
        return None
    dt = dtypes.get(t.dtype)
    if dt is None or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous vector of %d elements (%s), got %s %s"
                         % (name, n, _names(dtypes), t.dtype, tuple(t.shape)))
    return _PACK(t.data_ptr(), 1, n, n, dt)


_F32 = {torch.float32: _lib.GDN_F32}
_I8 = {torch.int8: _lib.GDN_I8}


def _eight_bit_rows(shape, like, q, scale):
    """Codes (rows on 16 bytes, so that products read them fastest) and scales."""
    D = shape[-1]
    if q is None:
        if D % 16 == 0:
            q = torch.empty(shape, dtype=torch.int8, device=like.device)
        else:
            q = torch.empty((*shape[:-1], -(-D // 16) * 16), dtype=torch.int8,
                            device=like.device)[..., :D]
    elif q.shape != shape:
        raise ValueError("8-bit rows must be of shape %s, got %s" % (tuple(shape), tuple(q.shape)))
    if scale is None:
        scale = torch.empty(shape[-2], dtype=torch.float32, device=like.device)
    else:
        _vector("scale", scale, shape[-2], _F32)
    return q, scale


def _norm_output(shape, like, eight_bit, y, scale):
    if eight_bit:
        y, scale = _eight_bit_rows(shape, like, y, scale)
        return y, scale, _matrix("y", y, _I8)
    if scale is not None:
        raise ValueError("scale comes with eight_bit=True")
    if y is None:
        y = torch.empty(shape, dtype=like.dtype, device=like.device)
    elif y.shape != shape or y.dtype is not like.dtype:
        raise ValueError("y must be %s of shape %s" % (like.dtype, tuple(shape)))
    return y, None, _matrix("y", y, _DT)


@_on_device
def gdn_quantize_rows(x, q=None, scale=None):
    """Rows x [T, D] (bf16 or fp32 views) in 8 bits.  Returns (q, scale): q int8 [T, D] codes,
    scale fp32 [T] = max|row| / 127; an element stands for scale * code."""
    lib, _ = _entry("gdn_quantize_rows")
    _need_cuda(x, q, scale)
    mx = _matrix("x", x, _DT)
    q, scale = _eight_bit_rows(x.shape, x, q, scale)
    rc = lib.gdn_quantize_rows(mx, _matrix("q", q, _I8), scale.data_ptr(), _raw_stream(x))
    if rc:
        _lib.check(rc, "gdn_quantize_rows")
    return q, scale


@_on_device
def gdn_add_rmsnorm(x, weight, residual=None, eps=1e-6, weight_offset=0.0, eight_bit=False,
                    y=None, scale=None, residual_out=None):
    """h = x + residual and its root-mean-square norm, h (weight_offset + weight) /
    sqrt(mean h^2 + eps).  Returns (y, h rounded to x's type), h None without a residual; y is
    a pair (int8 codes, fp32 scales of the rows) with ``eight_bit``.

    x, residual [T, D] bf16 or fp32 views; weight [D] bf16 or fp32; residual_out may be the
    residual itself; eps at least 2^-126.
    """
    lib, _ = _entry("gdn_add_rmsnorm")
    _need_cuda(x, weight, residual, y, scale, residual_out)
    mx = _matrix("x", x, _DT)
    res = out = None
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out comes with a residual")
    else:
        shape = x.shape
        if residual.shape != shape or (residual_out is not None and residual_out.shape != shape):
            raise ValueError("residual and residual_out must have x's shape %s" % (tuple(shape),))
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=x.dtype, device=x.device)
        res, out = _matrix("residual", residual, _DT), _matrix("residual_out", residual_out, _DT)
    y, scale, my = _norm_output(x.shape, x, eight_bit, y, scale)
    rc = lib.gdn_add_rmsnorm(mx, res, out, _vector("weight", weight, x.shape[-1], _DT),
                             weight_offset, eps, my, _ptr(scale), _raw_stream(x))
    if rc:
        _lib.check(rc, "gdn_add_rmsnorm")
    return (y, scale) if eight_bit else y, residual_out


@_on_device
def gdn_gated_rmsnorm(x, z, weight, eps=1e-6, eight_bit=False, y=None, scale=None):
    """The Gated DeltaNet layer's output norm: per head, x weight / sqrt(mean x^2 + eps) *
    silu(z).  Returns y [T, H D] of x's type, or (int8 codes, fp32 scales of the tokens).

    x, z [T, H, D] bf16 or fp32 views (token-major); weight [D] bf16 or fp32; eps at least
    2^-126.
    """
    lib, _ = _entry("gdn_gated_rmsnorm")
    _need_cuda(x, z, weight, y, scale)
    dx, dz = _view(x), _view(z)
    T, H, D = x.shape[-3:]
    y, scale, my = _norm_output(torch.Size((T, H * D)), x, eight_bit, y, scale)
    rc = lib.gdn_gated_rmsnorm(dx, dz, _vector("weight", weight, D, _DT), eps, my, _ptr(scale),
                               _raw_stream(x))
    if rc:
        _lib.check(rc, "gdn_gated_rmsnorm")
    return (y, scale) if eight_bit else y


@_on_device
def gdn_matmul_i8_workspace_size(a, w, simt=False):
    """Workspace bytes of gdn_matmul_i8 (by the sizes and the alignment of a and w and by their
    device)."""
    return int(_lib.load().gdn_matmul_i8_workspace_size(
        _matrix("a", a, _I8), _matrix("w", w, _I8), GDN_PREFILL_SIMT if simt else 0))


@_on_device
def gdn_matmul_i8(a, a_scale, w, w_scale, bias=None, dtype=torch.bfloat16, out=None, simt=False,
                  workspace=None, status=None):
    """out[m, n] = a_scale[m] w_scale[n] sum_k a[m, k] w[n, k] + bias[n], the sum exact.

    a [M, K] and w [N, K] int8 views; a_scale fp32 [M]; w_scale fp32 [N]; bias [N] bf16 or
    fp32; out [M, N] of ``dtype``, bf16 or fp32.
    """
    lib, debug = _entry("gdn_matmul_i8")
    _need_cuda(a, a_scale, w, w_scale, bias, out, workspace, status)
    ma, mw = _matrix("a", a, _I8), _matrix("w", w, _I8)
    lead = a.shape
    M, K = lead[-2:]
    N, Kw = w.shape[-2:]
    if Kw != K:
        raise ValueError("a has rows of %d codes and w of %d" % (K, Kw))
    _vector("a_scale", a_scale, M, _F32)
    _vector("w_scale", w_scale, N, _F32)
    shape = (M, N) if len(lead) == 2 else (1, M, N)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=a.device)
    elif out.shape != shape:
        raise ValueError("out must be of shape %s, got %s" % (tuple(shape), tuple(out.shape)))
    flags = (GDN_PREFILL_SIMT if simt else 0) | debug
    ws_bytes = lib.gdn_matmul_i8_workspace_size(ma, mw, flags)
    workspace = _scratch(workspace, ws_bytes, a)
    rc = lib.gdn_matmul_i8(ma, a_scale.data_ptr(), mw, w_scale.data_ptr(),
                           _vector("bias", bias, N, _DT), _matrix("out", out, _DT), flags,
                           _ptr(workspace), ws_bytes, _ptr(status), _raw_stream(a))
    if rc:
        _lib.check(rc, "gdn_matmul_i8")
    return out
