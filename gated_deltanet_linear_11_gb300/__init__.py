"""GB300-native (sm_103a) Gated DeltaNet layer hot path.

Thin Python binding over the C ABI of ``libgdn.so`` (declared in ``include/gdn.h``).
PyTorch supplies device memory and the current CUDA stream; every step of the layer runs
in this package's CUDA kernels.  The functions keep the C entry points' names:

* :func:`gdn_conv1d_fwd`       -- prefill conv1d + SiLU over packed sequences
* :func:`gdn_conv1d_update`    -- decode conv step on a pool of conv states
* :func:`gdn_chunk_prefill`    -- chunked gated delta rule over packed sequences
* :func:`gdn_recurrent_decode` -- one-token gated delta rule step on a state pool
* :func:`gdn_fused_decode`     -- conv update + gates from raw logits + recurrent step,
  one call

* :func:`gdn_linear_prefill`, :func:`gdn_linear_decode` -- linear attention with a plain
  decay for each head, over packed prompts and one token at a time
* :func:`gdn_kv_append`, :func:`gdn_kv_read`, :func:`gdn_kv_attention` -- a paged
  key/value cache held in 4 bits: rotate and store, read back, attend
  (:func:`gdn_kv_cache` allocates one)

plus :func:`gdn_layer_prefill` / :func:`gdn_layer_decode`, which chain the conv and the
scan over the packed q||k||v channels (q, k, v are strided views of the conv output;
nothing is copied).

There is no CPU fallback: without the built library every call raises.

Two environment variables serve debugging and callers' failure tests, read at each call:

* ``GDN_DEBUG=1`` adds ``GDN_CHECK_INPUTS`` to every call that takes flags. Before
  launching anything (it waits for the stream), the library copies the gate inputs to the
  host and fails with ``GDN_ERR_NONFINITE`` (11) on a NaN or an infinity. It also fails
  with ``GDN_ERR_SEQLENS`` (5) if a prefill's device ``cu_seqlens`` differs from its host
  copy.
* ``GDN_FORCE_ERROR="gdn_chunk_prefill=7,gdn_fused_decode=10"`` makes each named entry
  raise :class:`GdnError` with that status code at once, without calling the library:
  host-side fault injection for code that handles this package's errors.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os

import torch

from . import _lib
from ._lib import (GDN_CHECK_INPUTS, GDN_KV_INTERLEAVED, GDN_LAYER_FUSED_VCONV,  # noqa: F401
                   GDN_PREFILL_SIMT, GDN_PREFILL_TILES2, GDN_PREFILL_TILES3, GDN_QK_L2NORM,
                   GdnError)

__all__ = ["gdn_conv1d_fwd", "gdn_conv1d_update", "gdn_chunk_prefill",
           "gdn_chunk_prefill_noalloc", "gdn_chunk_prefill_cp",
           "gdn_chunk_prefill_cp_workspace_size", "gdn_chunk_prefill_cp_range_hint",
           "gdn_recurrent_decode", "gdn_fused_decode", "gdn_chunk_prefill_workspace_size",
           "gdn_layer_prefill", "gdn_layer_decode", "gdn_linear_prefill",
           "gdn_linear_prefill_workspace_size", "gdn_linear_decode", "gdn_kv_cache",
           "gdn_kv_append", "gdn_kv_read", "gdn_kv_attention",
           "gdn_kv_attention_workspace_size", "GdnError", "load"]

_DT = {torch.bfloat16: _lib.GDN_BF16, torch.float32: _lib.GDN_F32}


def load():
    """Load the CUDA library (raises when it is not built)."""
    return _lib.load()


def _vp(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _desc(t):
    if t.dtype not in _DT:
        raise TypeError("activations must be bf16 or fp32, got %s" % t.dtype)
    if t.dim() not in (3, 4):
        raise ValueError("activations must be [T,H,D] or [1,T,H,D]")
    d = _lib.GdnTensor()
    d.ptr = t.data_ptr()
    d.ndim = t.dim()
    d.dtype = _DT[t.dtype]
    for i in range(t.dim()):
        d.shape[i] = t.shape[i]
        d.stride[i] = t.stride(i)
    return d


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _debug_flags():
    """GDN_CHECK_INPUTS when GDN_DEBUG is set (to anything but "" or "0")."""
    return GDN_CHECK_INPUTS if os.environ.get("GDN_DEBUG", "") not in ("", "0") else 0


def _forced(name):
    """Raise the status GDN_FORCE_ERROR assigns to entry `name`, if any."""
    spec = os.environ.get("GDN_FORCE_ERROR", "")
    for item in filter(None, (x.strip() for x in spec.split(","))):
        entry, sep, code = item.partition("=")
        if not sep or not code.strip().lstrip("-").isdigit():
            raise ValueError("GDN_FORCE_ERROR items are name=code, got %r" % item)
        if entry.strip() == name:
            raise GdnError(int(code), name + " (GDN_FORCE_ERROR)")


def _need_cuda(*ts):
    device = ts[0].get_device()              # -1 on the host
    for t in ts:
        if t is not None and (t.get_device() != device or device < 0):
            raise ValueError("tensor must live on a CUDA device" if not t.is_cuda or device < 0
                             else "tensors live on different devices")


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on_device(fn):
    """Entries that launch: run with the device of the first tensor as the current one, since
    the C side launches on the current device and the stream is that device's."""
    first = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, **kw):
        t = args[0] if args else kw.get(first)
        d = -1 if t is None else t.get_device()
        if d < 0 or d == _current_device():
            return fn(*args, **kw)
        with torch.cuda.device(d):
            return fn(*args, **kw)
    return call


def _same_offsets(cu_seqlens, cu_seqlens_host):
    """The kernels read as many device offsets as the host copy has."""
    if cu_seqlens_host is not None and cu_seqlens.numel() < cu_seqlens_host.numel():
        raise ValueError("cu_seqlens has %d entries and cu_seqlens_host %d"
                         % (cu_seqlens.numel(), cu_seqlens_host.numel()))


def _seqlens(cu_seqlens, cu_seqlens_host):
    """Device and host int32 copies of the offsets (a host copy avoids a sync)."""
    _same_offsets(cu_seqlens, cu_seqlens_host)
    if cu_seqlens_host is None:
        cu_seqlens_host = cu_seqlens.detach().to("cpu", torch.int32).contiguous()
    else:
        cu_seqlens_host = cu_seqlens_host.to(torch.int32).contiguous()
    if not cu_seqlens.is_cuda:
        cu_seqlens = cu_seqlens.to(torch.int32).cuda()
    cu_seqlens = cu_seqlens.to(torch.int32).contiguous()
    return cu_seqlens, cu_seqlens_host


@_on_device
def gdn_conv1d_fwd(x, w, bias, cu_seqlens, conv_state_in=None, conv_state_out=None,
                   y=None, cu_seqlens_host=None):
    """y = silu(conv1d(cat(conv_state, x_seq))) per sequence; returns (y, conv_state_out).

    x [T, C] bf16; w [C, 4] (or [C, 1, 4]) bf16; bias [C] or None; cu_seqlens [N+1] int32;
    conv_state_in [N, 3, C] or None (zeros); conv_state_out may be conv_state_in.
    """
    _forced("gdn_conv1d_fwd")
    lib = _lib.load()
    _need_cuda(x, w, bias, conv_state_in, conv_state_out, y)
    T, C = x.shape
    w = w.reshape(C, 4).contiguous()
    cu, cu_h = _seqlens(cu_seqlens, cu_seqlens_host)
    N = cu_h.numel() - 1
    if y is None:
        y = torch.empty_like(x)
    if conv_state_out is None:
        conv_state_out = torch.empty((N, 3, C), dtype=x.dtype, device=x.device)
    rc = lib.gdn_conv1d_fwd(_vp(x), T, C, _vp(w), _vp(bias), _vp(cu),
                            ctypes.c_void_p(cu_h.data_ptr()), N, _vp(conv_state_in),
                            _vp(conv_state_out), _vp(y), _stream())
    _lib.check(rc, "gdn_conv1d_fwd")
    return y, conv_state_out


@_on_device
def gdn_conv1d_update(x, w, bias, conv_state, state_idx=None, y=None, status=None):
    """One-token conv step; conv_state [P, 3, C] is shifted in place.  Returns y [N, C]."""
    _forced("gdn_conv1d_update")
    lib = _lib.load()
    _need_cuda(x, w, bias, conv_state, state_idx, y, status)
    N, C = x.shape
    w = w.reshape(C, 4).contiguous()
    if y is None:
        y = torch.empty_like(x)
    rc = lib.gdn_conv1d_update(_vp(x), N, C, _vp(w), _vp(bias), _vp(conv_state),
                               conv_state.shape[0], _vp(state_idx), _vp(y), _vp(status),
                               _stream())
    _lib.check(rc, "gdn_conv1d_update")
    return y


def gdn_chunk_prefill_workspace_size(N, T, Hk, Hv, dk, dv, chunk=64, simt=False):
    lib = _lib.load()
    return int(lib.gdn_chunk_prefill_workspace_size(N, T, Hk, Hv, dk, dv, chunk,
                                                    GDN_PREFILL_SIMT if simt else 0))


def _tile_flag(tiles):
    if tiles is None:
        return 0
    if tiles not in (2, 3):
        raise ValueError("tiles must be 2, 3 or None")
    return GDN_PREFILL_TILES2 if tiles == 2 else GDN_PREFILL_TILES3


@_on_device
def gdn_chunk_prefill(q, k, v, g, beta, cu_seqlens, chunk=64, scale=1.0, l2norm=False,
                      initial_state=None, output_final_state=True, o=None,
                      final_state=None, simt=False, cu_seqlens_host=None, workspace=None,
                      status=None, tiles=None):
    """Chunked gated delta rule over packed sequences.  Returns (o, final_state).

    q, k [T, Hk, dk]; v [T, Hv, dv] (token-major views; head-first is rejected);
    g, beta [T, Hv] fp32; cu_seqlens [N+1]; initial_state [N, Hv, dk, dv] fp32 or None.
    tiles: None (chosen from N and the SM count), 2 or 3 dv tiles per head in the
    tensor-core state pass; the bits are the same under every choice.
    """
    _forced("gdn_chunk_prefill")
    lib = _lib.load()
    _need_cuda(q, k, v, g, beta, initial_state, o, final_state, workspace, status)
    cu, cu_h = _seqlens(cu_seqlens, cu_seqlens_host)
    N = cu_h.numel() - 1
    T, Hk, dk = q.shape[-3:]
    Hv, dv = v.shape[-2:]
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, Hv, dk, dv), dtype=torch.float32, device=q.device)
    flags = ((GDN_QK_L2NORM if l2norm else 0) | (GDN_PREFILL_SIMT if simt else 0) |
             _tile_flag(tiles) | _debug_flags())
    ws_bytes = int(lib.gdn_chunk_prefill_workspace_size(N, T, Hk, Hv, dk, dv, chunk, flags))
    if ws_bytes and (workspace is None or workspace.numel() * workspace.element_size() < ws_bytes):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    g = g.contiguous()
    beta = beta.contiguous()
    dq, dk_, dv_, do = _desc(q), _desc(k), _desc(v), _desc(o)
    rc = lib.gdn_chunk_prefill(
        ctypes.byref(dq), ctypes.byref(dk_), ctypes.byref(dv_), _vp(g), _vp(beta), _vp(cu),
        ctypes.c_void_p(cu_h.data_ptr()), N, chunk, float(scale), flags,
        _vp(initial_state), ctypes.byref(do), _vp(final_state), _vp(workspace),
        ws_bytes, _vp(status), _stream())
    _lib.check(rc, "gdn_chunk_prefill")
    return o, final_state


def gdn_chunk_prefill_cp_workspace_size(cu_seqlens_host, T, Hk, Hv, dk, dv, range_chunks,
                                        chunk=64):
    """Workspace bytes of gdn_chunk_prefill_cp (0 for a shape it does not take)."""
    lib = _lib.load()
    cu_h = cu_seqlens_host.to(torch.int32).contiguous()
    return int(lib.gdn_chunk_prefill_cp_workspace_size(
        ctypes.c_void_p(cu_h.data_ptr()), cu_h.numel() - 1, T, Hk, Hv, dk, dv, chunk,
        range_chunks))


def gdn_chunk_prefill_cp_range_hint(seq_len, Hv, sm_count=None):
    """range_chunks for one sequence of ``seq_len`` tokens over ``Hv`` v-heads alone on
    the current device (or on one with ``sm_count`` SMs), or 0 when the plain scan is
    expected to be as fast (C entries gdn_chunk_prefill_cp_range_hint and
    gdn_chunk_prefill_cp_range_hint_for; depends on the sequence's own length only)."""
    lib = _lib.load()
    if sm_count is None:
        return int(lib.gdn_chunk_prefill_cp_range_hint(int(seq_len), int(Hv)))
    return int(lib.gdn_chunk_prefill_cp_range_hint_for(int(seq_len), int(Hv), int(sm_count)))


@_on_device
def gdn_chunk_prefill_cp(q, k, v, g, beta, cu_seqlens, range_chunks, chunk=64, scale=1.0,
                         l2norm=False, initial_state=None, output_final_state=True, o=None,
                         final_state=None, cu_seqlens_host=None, workspace=None, status=None,
                         tiles=None):
    """gdn_chunk_prefill with every sequence split into ranges of ``range_chunks`` chunks
    run side by side (the context-parallel scan; tensor-core path only).  Returns
    (o, final_state)."""
    _forced("gdn_chunk_prefill_cp")
    lib = _lib.load()
    _need_cuda(q, k, v, g, beta, initial_state, o, final_state, workspace, status)
    cu, cu_h = _seqlens(cu_seqlens, cu_seqlens_host)
    N = cu_h.numel() - 1
    T, Hk, dk = q.shape[-3:]
    Hv, dv = v.shape[-2:]
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, Hv, dk, dv), dtype=torch.float32, device=q.device)
    flags = (GDN_QK_L2NORM if l2norm else 0) | _tile_flag(tiles) | _debug_flags()
    ws_bytes = int(lib.gdn_chunk_prefill_cp_workspace_size(
        ctypes.c_void_p(cu_h.data_ptr()), N, T, Hk, Hv, dk, dv, chunk, range_chunks))
    if ws_bytes and (workspace is None or workspace.numel() * workspace.element_size() < ws_bytes):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    dq, dk_, dv_, do = _desc(q), _desc(k), _desc(v), _desc(o)
    rc = lib.gdn_chunk_prefill_cp(
        ctypes.byref(dq), ctypes.byref(dk_), ctypes.byref(dv_), _vp(g.contiguous()),
        _vp(beta.contiguous()), _vp(cu), ctypes.c_void_p(cu_h.data_ptr()), N, chunk,
        float(scale), flags, int(range_chunks), _vp(initial_state), ctypes.byref(do),
        _vp(final_state), _vp(workspace), ws_bytes, _vp(status), _stream())
    _lib.check(rc, "gdn_chunk_prefill_cp")
    return o, final_state


@_on_device
def gdn_chunk_prefill_noalloc(q, k, v, g, beta, cu_seqlens, chunk=64, scale=1.0,
                              l2norm=False, initial_state=None, output_final_state=True,
                              o=None, final_state=None, simt=False, cu_seqlens_host=None,
                              status=None):
    """gdn_chunk_prefill for callers that cannot allocate device scratch: the library
    uses its own fixed 128 MiB device array instead of a workspace.  Output tensors are
    still the caller's; pass ``o``/``final_state`` (and the device ``cu_seqlens``, ``g`` and
    ``beta`` as contiguous tensors) to avoid any allocation on the Python side as well.
    Returns (o, final_state)."""
    _forced("gdn_chunk_prefill_noalloc")
    lib = _lib.load()
    _need_cuda(q, k, v, g, beta, initial_state, o, final_state, status)
    cu, cu_h = _seqlens(cu_seqlens, cu_seqlens_host)
    N = cu_h.numel() - 1
    T, Hk, dk = q.shape[-3:]
    Hv, dv = v.shape[-2:]
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, Hv, dk, dv), dtype=torch.float32, device=q.device)
    flags = ((GDN_QK_L2NORM if l2norm else 0) | (GDN_PREFILL_SIMT if simt else 0) |
             _debug_flags())
    dq, dk_, dv_, do = _desc(q), _desc(k), _desc(v), _desc(o)
    rc = lib.gdn_chunk_prefill_noalloc(
        ctypes.byref(dq), ctypes.byref(dk_), ctypes.byref(dv_), _vp(g.contiguous()),
        _vp(beta.contiguous()), _vp(cu), ctypes.c_void_p(cu_h.data_ptr()), N, chunk,
        float(scale), flags, _vp(initial_state), ctypes.byref(do), _vp(final_state),
        _vp(status), _stream())
    _lib.check(rc, "gdn_chunk_prefill_noalloc")
    return o, final_state


@_on_device
def gdn_recurrent_decode(q, k, v, g, beta, state, state_idx=None, scale=1.0, l2norm=False,
                         o=None, status=None):
    """One token per sequence; state [P, Hv, dk, dv] fp32 updated in place.  Returns o."""
    _forced("gdn_recurrent_decode")
    lib = _lib.load()
    _need_cuda(q, k, v, g, beta, state, state_idx, o, status)
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    dq, dk_, dv_, do = _desc(q), _desc(k), _desc(v), _desc(o)
    rc = lib.gdn_recurrent_decode(
        ctypes.byref(dq), ctypes.byref(dk_), ctypes.byref(dv_), _vp(g.contiguous()),
        _vp(beta.contiguous()), _vp(state), state.shape[0], _vp(state_idx), float(scale),
        (GDN_QK_L2NORM if l2norm else 0) | _debug_flags(), ctypes.byref(do), _vp(status),
        _stream())
    _lib.check(rc, "gdn_recurrent_decode")
    return o


@_on_device
def gdn_fused_decode(x_qkv, conv_w, conv_bias, a_raw, b_raw, conv_state, state, Hk, Hv, dk,
                     dv, state_idx=None, scale=1.0, l2norm=True, o=None, status=None):
    """The whole one-token decode step in one call: conv update (conv_state shifted in
    place), q/k/v split, optional q/k L2 norm, beta = sigmoid(b_raw), g = -softplus(a_raw),
    recurrent step (state updated in place).  x_qkv [N, C] bf16; a_raw, b_raw [N, Hv] fp32.
    Returns o [N, Hv, dv] bf16."""
    _forced("gdn_fused_decode")
    lib = _lib.load()
    _need_cuda(x_qkv, conv_w, conv_bias, a_raw, b_raw, conv_state, state, state_idx, o, status)
    N = x_qkv.shape[0]
    if o is None:
        o = torch.empty((N, Hv, dv), dtype=torch.bfloat16, device=x_qkv.device)
    for t in (x_qkv, conv_w, conv_state, state, o):
        if not t.is_contiguous():
            raise ValueError("gdn_fused_decode takes contiguous tensors")
    rc = lib.gdn_fused_decode(
        _vp(x_qkv), N, Hk, Hv, dk, dv, _vp(conv_w), _vp(conv_bias), _vp(conv_state),
        _vp(a_raw.contiguous()), _vp(b_raw.contiguous()), _vp(state), state.shape[0],
        _vp(state_idx), float(scale), (GDN_QK_L2NORM if l2norm else 0) | _debug_flags(),
        _vp(o), _vp(status), _stream())
    _lib.check(rc, "gdn_fused_decode")
    return o


def split_qkv(y, Hk, Hv, dk, dv):
    """Strided [T, H, D] views of the packed q||k||v conv output (no copy)."""
    T = y.shape[0]
    q = y[:, : Hk * dk].unflatten(1, (Hk, dk))
    k = y[:, Hk * dk: 2 * Hk * dk].unflatten(1, (Hk, dk))
    v = y[:, 2 * Hk * dk: 2 * Hk * dk + Hv * dv].unflatten(1, (Hv, dv))
    assert q.shape[0] == T
    return q, k, v


@_on_device
def gdn_layer_prefill(x_qkv, conv_w, conv_bias, g, beta, cu_seqlens, Hk, Hv, dk, dv,
                      conv_state_in=None, conv_state_out=None, initial_state=None,
                      final_state=None, scale=1.0, chunk=64, l2norm=True, y=None, o=None,
                      cu_seqlens_host=None, workspace=None, status=None, side_stream=None,
                      fused_vconv=False, tiles=None):
    """conv1d + SiLU over packed q||k||v, then the chunked scan with in-kernel q/k L2 norm,
    in one call of the C entry gdn_layer_prefill.  With ``side_stream`` (a second
    torch.cuda.Stream) the v channels' conv runs on it, overlapping the chunk preparation;
    without one everything runs on the current stream.  ``fused_vconv`` instead convolves
    the v channels inside the scan's state pass (GDN_LAYER_FUSED_VCONV).  Every path gives
    the bits of the two calls in sequence (y included, when passed).

    Returns (o [T, Hv, dv], final_state [N, Hv, dk, dv], conv_state_out [N, 3, C]).
    """
    _forced("gdn_layer_prefill")
    if chunk != 64:
        raise ValueError("gdn_layer_prefill runs the 64-token chunk scan")
    lib = _lib.load()
    _need_cuda(x_qkv, conv_w, conv_bias, g, beta, conv_state_in, conv_state_out,
               initial_state, final_state, y, o, workspace, status)
    T, C = x_qkv.shape
    if C != 2 * Hk * dk + Hv * dv:
        raise ValueError("x_qkv has %d channels, not 2*Hk*dk + Hv*dv" % C)
    conv_w = conv_w.reshape(C, 4).contiguous()
    cu, cu_h = _seqlens(cu_seqlens, cu_seqlens_host)
    N = cu_h.numel() - 1
    dev = x_qkv.device
    if y is None:
        y = torch.empty_like(x_qkv)
    if conv_state_out is None:
        conv_state_out = torch.empty((N, 3, C), dtype=x_qkv.dtype, device=dev)
    if o is None:
        o = torch.empty((T, Hv, dv), dtype=torch.bfloat16, device=dev)
    if final_state is None:
        final_state = torch.empty((N, Hv, dk, dv), dtype=torch.float32, device=dev)
    flags = (GDN_QK_L2NORM if l2norm else 0) | (GDN_LAYER_FUSED_VCONV if fused_vconv else 0)
    flags |= _tile_flag(tiles) | _debug_flags()
    ws_bytes = int(lib.gdn_chunk_prefill_workspace_size(N, T, Hk, Hv, dk, dv, 64, flags))
    if ws_bytes and (workspace is None or workspace.numel() * workspace.element_size() < ws_bytes):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    for t in (x_qkv, y, o):
        if not t.is_contiguous():
            raise ValueError("gdn_layer_prefill takes contiguous x_qkv, y and o")
    rc = lib.gdn_layer_prefill(
        _vp(x_qkv), T, Hk, Hv, dk, dv, _vp(conv_w), _vp(conv_bias), _vp(cu),
        ctypes.c_void_p(cu_h.data_ptr()), N, _vp(conv_state_in), _vp(conv_state_out), _vp(y),
        _vp(g.contiguous()), _vp(beta.contiguous()), float(scale), flags, _vp(initial_state),
        _vp(o), _vp(final_state), _vp(workspace), ws_bytes, _vp(status),
        None if side_stream is None else ctypes.c_void_p(side_stream.cuda_stream), _stream())
    _lib.check(rc, "gdn_layer_prefill")
    return o, final_state, conv_state_out


@_on_device
def gdn_layer_decode(x_qkv, conv_w, conv_bias, g, beta, conv_state, state, Hk, Hv, dk, dv,
                     state_idx=None, scale=1.0, l2norm=True, y=None, o=None, status=None):
    """One-token layer step: conv update, then the recurrent step (states in place)."""
    y = gdn_conv1d_update(x_qkv, conv_w, conv_bias, conv_state, state_idx, y, status)
    q, k, v = split_qkv(y, Hk, Hv, dk, dv)
    return gdn_recurrent_decode(q, k, v, g, beta, state, state_idx, scale, l2norm, o,
                                status)


# The entries below are called once per layer and token, so their host side is kept short:
# descriptors are filled in one go, pointers go to ctypes as plain integers and offsets that
# are already int32 on the right device are used as they are.

_PACK = _lib.GDN_TENSOR_PACK.pack
# os.environ without its per-lookup key encoding: most calls find neither variable set
_ENV = getattr(os.environ, "_data", os.environ)
_ENV_FORCE, _ENV_DEBUG = (getattr(os.environ, "encodekey", str)(x)
                          for x in ("GDN_FORCE_ERROR", "GDN_DEBUG"))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _entry(name):
    """What every call starts with: forced errors, the library, the debug flags."""
    if _ENV_FORCE in _ENV:
        _forced(name)
    return _lib.load(), _debug_flags() if _ENV_DEBUG in _ENV else 0


def _view(t):
    """gdn_tensor_t of an activation view (as _desc), packed."""
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError("activations must be bf16 or fp32, got %s" % t.dtype)
    if t.dim() == 3:
        a, b, c = t.shape
        x, y, z = t.stride()
        return _PACK(t.data_ptr(), 3, dt, a, b, c, 0, x, y, z, 0)
    if t.dim() == 4:
        return _PACK(t.data_ptr(), 4, dt, *t.shape, *t.stride())
    raise ValueError("activations must be [T,H,D] or [1,T,H,D]")


def _raw_stream(t):
    """The current stream of t's device, as the integer that ctypes passes on."""
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _offsets(cu_seqlens, cu_seqlens_host):
    """_seqlens without conversions where none are needed."""
    if cu_seqlens_host is not None and cu_seqlens_host.dtype is torch.int32 and \
            cu_seqlens.dtype is torch.int32 and cu_seqlens.is_cuda and \
            cu_seqlens.is_contiguous() and cu_seqlens_host.is_contiguous() and \
            not cu_seqlens_host.is_cuda:
        _same_offsets(cu_seqlens, cu_seqlens_host)
        return cu_seqlens, cu_seqlens_host
    return _seqlens(cu_seqlens, cu_seqlens_host)


def _gates(g, T, Hv):
    """(contiguous fp32 log decays, per-token flag) of g [Hv] or [T, Hv]."""
    if g.dtype is not torch.float32:
        raise TypeError("g must be fp32, got %s" % g.dtype)
    if g.dim() == 1 and g.shape[0] == Hv:
        return g.contiguous(), 0
    if g.dim() >= 2 and tuple(g.shape[-2:]) == (T, Hv) and g.numel() == T * Hv:
        return g.contiguous(), 1
    raise ValueError("g must be [Hv] or [T, Hv] = [%d, %d], got %s" % (T, Hv, tuple(g.shape)))


def _states(name, t, shape):
    if t is not None and (t.dtype is not torch.float32 or t.shape != shape or
                          not t.is_contiguous()):
        raise ValueError("%s must be a contiguous fp32 tensor of shape %s" % (name, tuple(shape)))


def _int32(name, t, shape):
    if t is not None and (t.dtype is not torch.int32 or t.shape != shape or
                          not t.is_contiguous()):
        raise ValueError("%s must be a contiguous int32 tensor of shape %s" % (name, tuple(shape)))


def _scratch(workspace, size, like):
    if size and (workspace is None or workspace.numel() * workspace.element_size() < size):
        return torch.empty(size, dtype=torch.uint8, device=like.device)
    return workspace


def gdn_linear_prefill_workspace_size(cu_seqlens_host, T, Hk, Hv, D, dtype=torch.bfloat16,
                                      simt=False):
    """Workspace bytes of gdn_linear_prefill."""
    lib = _lib.load()
    cu_h = cu_seqlens_host.to(torch.int32).contiguous()
    return int(lib.gdn_linear_prefill_workspace_size(
        cu_h.data_ptr(), cu_h.numel() - 1, T, Hk, Hv, D, _DT[dtype],
        GDN_PREFILL_SIMT if simt else 0))


@_on_device
def gdn_linear_prefill(q, k, v, g, cu_seqlens, scale=1.0, initial_state=None,
                       output_final_state=True, o=None, final_state=None, simt=False,
                       cu_seqlens_host=None, workspace=None, status=None):
    """Linear attention with a decay for each head over packed sequences,
    S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.  Returns (o, final_state).

    q, k [T, Hk, D]; v [T, Hv, D], all bf16 or all fp32 (token-major views); g fp32 log
    decays, [Hv] or [T, Hv]; cu_seqlens [N+1]; initial_state [N, Hv, D, D] fp32 or None.
    """
    lib, debug = _entry("gdn_linear_prefill")
    _need_cuda(q, k, v, g, initial_state, o, final_state, workspace, status)
    cu, cu_h = _offsets(cu_seqlens, cu_seqlens_host)
    N = cu_h.numel() - 1
    T, Hk, D = q.shape[-3:]
    Hv = v.shape[-2]
    g, per_token = _gates(g, T, Hv)
    _states("initial_state", initial_state, (N, Hv, D, D))
    _states("final_state", final_state, (N, Hv, D, D))
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, Hv, D, D), dtype=torch.float32, device=q.device)
    flags = (GDN_PREFILL_SIMT if simt else 0) | debug
    cu_hp = cu_h.data_ptr()
    ws_bytes = lib.gdn_linear_prefill_workspace_size(cu_hp, N, T, Hk, Hv, D,
                                                     _DT.get(v.dtype, 0), flags)
    workspace = _scratch(workspace, ws_bytes, q)
    rc = lib.gdn_linear_prefill(_view(q), _view(k), _view(v), g.data_ptr(), per_token,
                                cu.data_ptr(), cu_hp, N, scale, flags, _ptr(initial_state),
                                _view(o), _ptr(final_state), _ptr(workspace), ws_bytes,
                                _ptr(status), _raw_stream(q))
    if rc:
        _lib.check(rc, "gdn_linear_prefill")
    return o, final_state


@_on_device
def gdn_linear_decode(q, k, v, g, state, state_idx=None, scale=1.0, o=None, status=None):
    """One token per sequence of gdn_linear_prefill's recurrence; state [P, Hv, D, D] fp32
    updated in place.  g [Hv] or [N, Hv].  Returns o."""
    lib, debug = _entry("gdn_linear_decode")
    _need_cuda(q, k, v, g, state, state_idx, o, status)
    N, _, D = q.shape[-3:]
    Hv = v.shape[-2]
    g, per_token = _gates(g, N, Hv)
    P = state.shape[0]
    _states("state", state, (P, Hv, D, D))
    _int32("state_idx", state_idx, (N,))
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    rc = lib.gdn_linear_decode(_view(q), _view(k), _view(v), g.data_ptr(), per_token,
                               state.data_ptr(), P, _ptr(state_idx), scale, debug,
                               _view(o), _ptr(status), _raw_stream(q))
    if rc:
        _lib.check(rc, "gdn_linear_decode")
    return o


def gdn_kv_cache(pages, page_size, Hkv, head_dim, device="cuda"):
    """A zeroed paged 4-bit cache: uint8 [pages, 2, Hkv, page_size, record bytes] (the
    layout is described in include/gdn.h)."""
    rec = int(_lib.load().gdn_kv_record_bytes(head_dim))
    if rec == 0:
        raise GdnError(6, "gdn_kv_cache (head_dim %d)" % head_dim)
    return torch.zeros((pages, 2, Hkv, page_size, rec), dtype=torch.uint8, device=device)


def _kv_cache(cache, block_table, kv_lens, head_dim):
    """(N, Hkv, packed gdn_kv_cache_t) of a cache tensor with its table and lengths."""
    if cache.dtype is not torch.uint8 or cache.dim() != 5 or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous uint8 tensor of five dimensions")
    pages, two, Hkv, page, rec = cache.shape
    if two != 2 or rec != head_dim // 2 + head_dim // 8:
        raise ValueError("cache of shape %s does not hold keys and values of head_dim %d"
                         % (tuple(cache.shape), head_dim))
    if block_table.dim() != 2:
        raise ValueError("block_table must be [N, pages of a sequence]")
    N, width = block_table.shape
    _int32("block_table", block_table, (N, width))
    _int32("kv_lens", kv_lens, (N,))
    return N, Hkv, _lib.GDN_KV_CACHE_PACK.pack(
        cache.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr(), pages, page, Hkv,
        head_dim, width, N)


def _kv_offsets(cu_seqlens, cu_seqlens_host, T, N):
    """Device and host offsets of the new tokens (None, None: one per sequence)."""
    if cu_seqlens is None:
        if T != N:
            raise ValueError("%d new tokens for %d sequences need cu_seqlens" % (T, N))
        return None, None
    cu, cu_h = _offsets(cu_seqlens, cu_seqlens_host)
    if cu_h.numel() != N + 1 or cu.numel() != N + 1:
        raise ValueError("cu_seqlens must have %d entries" % (N + 1))
    return cu, cu_h


@_on_device
def gdn_kv_append(k, v, cache, block_table, kv_lens, cu_seqlens=None, cos=None, sin=None,
                  q=None, q_out=None, interleaved=False, cu_seqlens_host=None, status=None):
    """Store new tokens' keys (rotated) and values in a paged 4-bit cache; with ``q``,
    return q rotated.

    k, v [T, Hkv, D] and q [T, Hq, D], bf16 or fp32 views; cache as gdn_kv_cache gives it;
    block_table int32 [N, W]; kv_lens int32 [N], the new tokens included; cu_seqlens [N+1]
    offsets of the new tokens, or None for one per sequence; cos, sin fp32
    [positions, rot / 2] or None for no rotation (rot = twice their width).
    """
    lib, debug = _entry("gdn_kv_append")
    _need_cuda(k, v, cache, block_table, kv_lens, cos, sin, q, q_out, status)
    T, _, D = k.shape[-3:]
    N, Hkv, c = _kv_cache(cache, block_table, kv_lens, D)
    cu, cu_h = _kv_offsets(cu_seqlens, cu_seqlens_host, T, N)
    rows = rot = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is not None:
        if cos.dtype is not torch.float32 or sin.dtype is not torch.float32 or cos.dim() != 2 or \
                cos.shape != sin.shape or not cos.is_contiguous() or not sin.is_contiguous():
            raise ValueError("cos and sin must be contiguous fp32 [positions, rot / 2]")
        rows, rot = cos.shape[0], 2 * cos.shape[1]
    dq = do = None
    if q is not None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        dq, do = _view(q), _view(q_out)
    rc = lib.gdn_kv_append(c, _ptr(cu), _ptr(cu_h), _view(k), _view(v), dq, do, _ptr(cos),
                           _ptr(sin), rows, rot,
                           (GDN_KV_INTERLEAVED if interleaved else 0) | debug,
                           _ptr(status), _raw_stream(k))
    if rc:
        _lib.check(rc, "gdn_kv_append")
    return q_out


@_on_device
def gdn_kv_read(cache, block_table, kv_lens, cu_seqlens=None, head_dim=128,
                dtype=torch.bfloat16, k=None, v=None, cu_seqlens_host=None, status=None):
    """The last tokens' keys and values (as many per sequence as cu_seqlens says; None:
    one) of a paged 4-bit cache, as values.  Returns (k, v), each [T, Hkv, head_dim]."""
    lib, debug = _entry("gdn_kv_read")
    _need_cuda(cache, block_table, kv_lens, k, v, status)
    N, Hkv, c = _kv_cache(cache, block_table, kv_lens, head_dim)
    cu, cu_h = _kv_offsets(cu_seqlens, cu_seqlens_host, N, N)
    T = N if cu_h is None else int(cu_h[-1])
    if k is None:
        k = torch.empty((T, Hkv, head_dim), dtype=dtype, device=cache.device)
    if v is None:
        v = torch.empty((T, Hkv, head_dim), dtype=k.dtype, device=cache.device)
    rc = lib.gdn_kv_read(c, _ptr(cu), _ptr(cu_h), _view(k), _view(v), debug,
                         _ptr(status), _raw_stream(cache))
    if rc:
        _lib.check(rc, "gdn_kv_read")
    return k, v


def gdn_kv_attention_workspace_size(head_dim, Hq, Hkv, T, N, max_q_len, max_kv_len,
                                    dtype=torch.bfloat16, simt=False):
    """Workspace bytes of gdn_kv_attention for T new tokens of N sequences."""
    return int(_lib.load().gdn_kv_attention_workspace_size(
        head_dim, Hq, Hkv, T, N, max_q_len, max_kv_len, _DT[dtype],
        GDN_PREFILL_SIMT if simt else 0))


@_on_device
def gdn_kv_attention(q, cache, block_table, kv_lens, cu_seqlens=None, max_kv_len=None,
                     scale=None, o=None, lse=None, simt=False, cu_seqlens_host=None,
                     workspace=None, status=None):
    """Softmax attention of the new tokens over a paged 4-bit cache that already holds
    them: the row at position p sees keys 0 .. p.  Returns o [T, Hq, D].

    q [T, Hq, D] bf16 or fp32, Hq a multiple of the cache's Hkv; cu_seqlens [N+1], or None
    for one new token per sequence; max_kv_len: an upper bound of kv_lens (default: what
    block_table can hold; a tighter one means a smaller grid and workspace); scale
    defaults to D^-1/2; lse: an fp32 [T, Hq] tensor that receives the log-sum-exp.
    """
    lib, debug = _entry("gdn_kv_attention")
    _need_cuda(q, cache, block_table, kv_lens, o, lse, workspace, status)
    T, Hq, D = q.shape[-3:]
    N, Hkv, c = _kv_cache(cache, block_table, kv_lens, D)
    cu, cu_h = _kv_offsets(cu_seqlens, cu_seqlens_host, T, N)
    if max_kv_len is None:
        max_kv_len = min(block_table.shape[1] * cache.shape[3], 1 << 30)
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (T, Hq) or
                            not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 tensor of shape [T, Hq]")
    if o is None:
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    flags = (GDN_PREFILL_SIMT if simt else 0) | debug
    max_q = 1 if cu_h is None else T if N == 1 else _longest(cu_h)
    dq = _view(q)
    ws_bytes = lib.gdn_kv_attention_workspace_size(D, Hq, Hkv, T, N, max_q, max_kv_len,
                                                   _DT[q.dtype], flags)
    workspace = _scratch(workspace, ws_bytes, q)
    rc = lib.gdn_kv_attention(c, _ptr(cu), _ptr(cu_h), max_kv_len, dq,
                              D ** -0.5 if scale is None else scale, flags, _view(o), _ptr(lse),
                              _ptr(workspace), ws_bytes, _ptr(status), _raw_stream(q))
    if rc:
        _lib.check(rc, "gdn_kv_attention")
    return o


def _longest(cu_h):
    cu = cu_h.tolist()
    return max((b - a for a, b in zip(cu, cu[1:])), default=0)


def gdn_selftest_bounded_wait(status=None):
    """The failure path of the kernels' bounded waits, without a GPU fault: one CTA waits
    on an mbarrier phase that nothing completes, gives up after about 2 s and writes
    GDN_ERR_TIMEOUT to the status word.  Returns the status tensor (int32 [1])."""
    lib = _lib.load()
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _need_cuda(status)
    _lib.check(lib.gdn_selftest_bounded_wait(_vp(status), _stream()),
               "gdn_selftest_bounded_wait")
    return status
