"""Binding of the operators around the scan: the short causal convolution, the
channel scan and the block norm.

Token-major operands (x, y, gradients) may be strided views whose last
dimension is contiguous, such as column slices of a projection's rows; states
and parameters are contiguous.  ``cu_seqlens`` is a host sequence of
nseq + 1 offsets as for ssd_fwd_varlen; without it every batch row is one
sequence.  Operands are on the current device; every function takes
``stream`` (the current one by default).
Argument marshalling only, as everywhere in this package.
"""
from __future__ import annotations

import ctypes
import functools

import torch

_F32 = torch.float32
_CODE = {torch.float32: 0, torch.bfloat16: 1}
_MAX_PARTS = 4
_Parts = ctypes.c_int64 * _MAX_PARTS


class _rows_t(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64)]


class _conv_shape_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("width", ctypes.c_int64), ("nparts", ctypes.c_int64), ("part", ctypes.c_int64 * _MAX_PARTS),
                ("dtype", ctypes.c_int), ("silu", ctypes.c_int)]


class _channel_shape_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("dt_softplus", ctypes.c_int)]


class _channel_inputs_t(ctypes.Structure):
    _fields_ = [("x", _rows_t), ("dt", _rows_t), ("z", _rows_t), ("B", _rows_t), ("C", _rows_t),
                ("A", ctypes.c_void_p), ("D", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("init_state", ctypes.c_void_p)]


class _channel_grads_t(ctypes.Structure):
    _fields_ = [("dx", _rows_t), ("ddt", _rows_t), ("dz", _rows_t), ("dB", _rows_t), ("dC", _rows_t),
                ("dA", ctypes.c_void_p), ("dD", ctypes.c_void_p), ("ddt_bias", ctypes.c_void_p),
                ("dinit_state", ctypes.c_void_p)]


class _norm_shape_t(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("group_size", ctypes.c_int64),
                ("eps", ctypes.c_float), ("dtype", ctypes.c_int), ("residual_dtype", ctypes.c_int),
                ("gate_after", ctypes.c_int)]


_RowsOf = [None] + [_rows_t * n for n in range(1, _MAX_PARTS + 1)]


def declare(lib):
    """Declare this module's entry points on the loaded library."""
    vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64
    lib.ssd_conv_fwd.argtypes = [vp, vp, i64] + [vp] * 7
    lib.ssd_conv_bwd_workspace_size.argtypes = [vp, vp, i64]
    lib.ssd_conv_bwd_workspace_size.restype = sz
    lib.ssd_conv_bwd.argtypes = [vp, vp, i64] + [vp] * 11 + [sz, vp]
    lib.ssd_conv_step.argtypes = [vp] * 7
    for name in ("ssd_channel_scan_workspace_size", "ssd_channel_scan_bwd_workspace_size"):
        getattr(lib, name).argtypes = [vp, vp, i64]
        getattr(lib, name).restype = sz
    lib.ssd_block_norm_fwd.argtypes = [vp] * 9
    lib.ssd_block_norm_bwd_workspace_size.argtypes = [vp]
    lib.ssd_block_norm_bwd_workspace_size.restype = sz
    lib.ssd_block_norm_bwd.argtypes = [vp] * 14 + [sz, vp]
    lib.ssd_channel_scan_fwd.argtypes = [vp, vp, i64] + [vp] * 4 + [sz, vp]
    lib.ssd_channel_scan_bwd.argtypes = [vp, vp, i64] + [vp] * 5 + [sz, vp]
    lib.ssd_channel_scan_step.argtypes = [vp] * 5
    for name in ("ssd_conv_fwd", "ssd_conv_bwd", "ssd_conv_step", "ssd_channel_scan_fwd", "ssd_channel_scan_bwd",
                 "ssd_channel_scan_step", "ssd_block_norm_fwd", "ssd_block_norm_bwd"):
        getattr(lib, name).restype = i32


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        from . import load_library
        _LIB = load_library()
    return _LIB


def _fail(fn, status):
    from . import _check
    _check(fn, status)


def _on_stream(fn):
    """Adds ``stream``: the whole call, its allocations included, then belongs
    to that stream instead of the current one."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _current_device():
    return torch._C._cuda_getDevice()


# These run several times a call, and a call for one token takes a few
# microseconds on the GPU: the checks that pass are few and plain.
def _code(x, name="x"):
    """(dtype code, device index)"""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    code = _CODE.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {x.dtype}")
    idx, current = x.get_device(), _current_device()
    if idx != current:  # kernels run on the current device, whatever the stream
        raise ValueError(f"{name} is on cuda:{idx}, the current device is cuda:{current}")
    return code, idx


def _refuse(t, name, dtype, shape, idx):
    if not isinstance(t, torch.Tensor) or t.get_device() != idx:
        raise TypeError(f"{name} must be a CUDA tensor on cuda:{idx}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _is(t, dtype, shape, idx):
    return isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == idx


def _rows(t, name, dtype, shape, idx):
    """ssd_rows_t of a [b, L, C] or [b, L, G, N] tensor whose trailing
    dimensions are contiguous."""
    if not _is(t, dtype, shape, idx):
        _refuse(t, name, dtype, shape, idx)
    st = t.stride()
    if (st[-1] != 1 and shape[-1] > 1) or (len(st) == 4 and st[2] != shape[3] and shape[2] > 1):
        raise ValueError(f"{name} must be contiguous in its trailing dimensions")
    return _rows_t(t.data_ptr(), st[0], st[1])


def _rows2(t, name, dtype, shape, idx):
    """The same for one token per sequence: [b, C] or [b, G, N]."""
    if not _is(t, dtype, shape, idx):
        _refuse(t, name, dtype, shape, idx)
    st = t.stride()
    if (st[-1] != 1 and shape[-1] > 1) or (len(st) == 3 and st[1] != shape[2] and shape[1] > 1):
        raise ValueError(f"{name} must be contiguous in its trailing dimensions")
    return _rows_t(t.data_ptr(), st[0], 0)


def _flat(t, name, dtype, shape, idx):
    """data pointer of a contiguous tensor; None for None."""
    if t is None:
        return None
    if not _is(t, dtype, shape, idx):
        _refuse(t, name, dtype, shape, idx)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _offsets(cu_seqlens, batch):
    """(ctypes array or None, number of sequences)."""
    if cu_seqlens is None:
        return None, batch
    cu = cu_seqlens.tolist() if isinstance(cu_seqlens, torch.Tensor) else cu_seqlens
    if len(cu) == 0:
        raise ValueError("cu_seqlens needs at least one offset")
    return (ctypes.c_int64 * len(cu))(*cu), len(cu) - 1


def _empty(shape, dtype, x):
    return torch.empty(shape, dtype=dtype, device=x.device)


def _workspace(workspace, need, x):
    """The given workspace where it is large enough, else a new one."""
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.get_device() != x.get_device():
            raise TypeError(f"workspace must be a CUDA tensor on {x.device}")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if workspace.numel() * workspace.element_size() >= need:
            return workspace
    return _empty((max(need, 16),), torch.uint8, x)


# ---------------------------------------------------------------------------
# short causal convolution
# ---------------------------------------------------------------------------
def _conv_shape(x, weight, parts, silu, code):
    if x.dim() != 3 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x must be [b, L, C] and weight [C, W]")
    if not 1 <= len(parts) <= _MAX_PARTS:
        raise ValueError(f"1 to {_MAX_PARTS} parts, got {len(parts)}")
    b, L, C = x.shape
    return _conv_shape_t(b, L, C, weight.shape[1], len(parts), _Parts(*parts), code,
                         1 if silu else 0)


@_on_stream
def ssd_conv_fwd(x, weight, bias=None, init_state=None, *, silu=True, cu_seqlens=None, split=None, y=None,
                 final_state=None, return_final_state=True):
    """Causal depthwise convolution over the last W tokens with bias and SiLU.

    x [b, L, C], weight [C, W] fp32 (W 2 to 4), bias [C] fp32; the rows before
    a sequence come from ``init_state`` [nseq, W-1, C] (zeros without it).
    Returns ``(y, final_state)``, the final state being each sequence's last
    W-1 rows of x.  With ``split``, widths that sum to C, y is a list of
    contiguous tensors [b, L, width]: the x, B and C a scan takes.  ``y`` and
    ``final_state`` may be given; they must not overlap the inputs."""
    lib = _lib()
    code, dev = _code(x)
    dt = x.dtype
    parts = [x.shape[-1]] if split is None else [int(v) for v in split]
    shape = _conv_shape(x, weight, parts, silu, code)
    b, L, C = x.shape
    W = weight.shape[1]
    cu, nseq = _offsets(cu_seqlens, b)
    xr = _rows(x, "x", dt, (b, L, C), dev)
    wp = _flat(weight, "weight", _F32, (C, W), dev)
    bp = _flat(bias, "bias", _F32, (C,), dev)
    ip = _flat(init_state, "init_state", dt, (nseq, W - 1, C), dev)
    if y is None:
        ys = [_empty((b, L, p), dt, x) for p in parts]
        yr = _RowsOf[len(parts)](*[_rows_t(t.data_ptr(), L * p, p) for t, p in zip(ys, parts)])
    else:
        ys = [y] if split is None else list(y)
        if len(ys) != len(parts):
            raise ValueError(f"y must hold {len(parts)} tensors")
        yr = _RowsOf[len(parts)](*[_rows(t, "y", dt, (b, L, p), dev) for t, p in zip(ys, parts)])
    fp = None
    if final_state is not None:
        fp = _flat(final_state, "final_state", dt, (nseq, W - 1, C), dev)
        if fp and fp == ip:
            raise ValueError("final_state must not be init_state")
    elif return_final_state:
        final_state = _empty((nseq, W - 1, C), dt, x)
        fp = final_state.data_ptr()
    st = lib.ssd_conv_fwd(ctypes.byref(shape), cu, nseq, ctypes.byref(xr), wp, bp, ip, yr, fp,
                          torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _fail("ssd_conv_fwd", st)
    return (ys[0] if split is None else ys), final_state


@_on_stream
def ssd_conv_bwd(dy, x, weight, bias=None, init_state=None, *, silu=True, cu_seqlens=None, dfinal_state=None, dx=None,
                 workspace=None):
    """Gradient of ssd_conv_fwd.  ``dy`` is a tensor [b, L, C] or the list of
    parts' gradients; ``dfinal_state`` [nseq, W-1, C] that of the final state
    (zero without it).  Returns ``(dx, dweight, dbias, dinit_state)``: dbias
    and dinit_state None where the input was None; dweight and dbias fp32."""
    lib = _lib()
    code, dev = _code(x)
    dt = x.dtype
    dys = [dy] if isinstance(dy, torch.Tensor) else list(dy)
    parts = [t.shape[-1] for t in dys]
    shape = _conv_shape(x, weight, parts, silu, code)
    b, L, C = x.shape
    W = weight.shape[1]
    cu, nseq = _offsets(cu_seqlens, b)
    xr = _rows(x, "x", dt, (b, L, C), dev)
    gr = _RowsOf[len(parts)](*[_rows(t, "dy", dt, (b, L, p), dev) for t, p in zip(dys, parts)])
    wp = _flat(weight, "weight", _F32, (C, W), dev)
    bp = _flat(bias, "bias", _F32, (C,), dev)
    ip = _flat(init_state, "init_state", dt, (nseq, W - 1, C), dev)
    gp = _flat(dfinal_state, "dfinal_state", dt, (nseq, W - 1, C), dev)
    if dx is None:
        dx = _empty((b, L, C), dt, x)
        dxr = _rows_t(dx.data_ptr(), L * C, C)
    else:
        dxr = _rows(dx, "dx", dt, (b, L, C), dev)
    dweight = _empty((C, W), _F32, x)
    dbias = None if bias is None else _empty((C,), _F32, x)
    dinit = None if init_state is None else _empty((nseq, W - 1, C), x.dtype, x)
    workspace = _workspace(workspace, lib.ssd_conv_bwd_workspace_size(ctypes.byref(shape), cu, nseq), x)
    st = lib.ssd_conv_bwd(
        ctypes.byref(shape), cu, nseq, gr, ctypes.byref(xr), wp, bp, ip, gp, ctypes.byref(dxr), dweight.data_ptr(),
        None if dbias is None else dbias.data_ptr(), None if dinit is None else dinit.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _fail("ssd_conv_bwd", st)
    return dx, dweight, dbias, dinit


@_on_stream
def ssd_conv_step(x, weight, bias=None, *, state, silu=True, y=None):
    """One token per sequence: x [b, C]; ``state`` [b, W-1, C], the rows before
    it, moves up by one in place.  Returns y [b, C]."""
    lib = _lib()
    code, dev = _code(x)
    if x.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x must be [b, C] and weight [C, W]")
    dt = x.dtype
    b, C = x.shape
    W = weight.shape[1]
    xr = _rows2(x, "x", dt, (b, C), dev)
    wp = _flat(weight, "weight", _F32, (C, W), dev)
    bp = _flat(bias, "bias", _F32, (C,), dev)
    if state is None:
        raise TypeError("state must be a CUDA tensor")
    sp = _flat(state, "state", dt, (b, W - 1, C), dev)
    if y is None:
        y = _empty((b, C), dt, x)
        yr = _rows_t(y.data_ptr(), C, 0)
    else:
        yr = _rows2(y, "y", dt, (b, C), dev)
    shape = _conv_shape_t(b, 1, C, W, 1, _Parts(C), code, 1 if silu else 0)
    st = lib.ssd_conv_step(ctypes.byref(shape), ctypes.byref(xr), wp, bp, sp, ctypes.byref(yr),
                           torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _fail("ssd_conv_step", st)
    return y


# ---------------------------------------------------------------------------
# channel scan
# ---------------------------------------------------------------------------
def _channel_inputs(x, dt, A, B, C, D, z, dt_bias, init_state, nseq, rows, tok, dev):
    """(inputs struct, channels, states, groups); ``rows`` is _rows or _rows2
    and ``tok`` the leading dimensions (b, L) or (b,)."""
    ty = x.dtype
    if x.dim() != len(tok) + 1 or not isinstance(B, torch.Tensor) or B.dim() != len(tok) + 2:
        raise ValueError("x must be [b, L, Ch] and B, C [b, L, G, N] (without L for one token)")
    ch = x.shape[-1]
    G, N = B.shape[-2], B.shape[-1]
    full, bc = (*tok, ch), (*tok, G, N)
    return _channel_inputs_t(
        rows(x, "x", ty, full, dev), rows(dt, "dt", ty, full, dev),
        _rows_t(None, 0, 0) if z is None else rows(z, "z", ty, full, dev),
        rows(B, "B", ty, bc, dev), rows(C, "C", ty, bc, dev), _flat(A, "A", _F32, (ch, N), dev),
        _flat(D, "D", _F32, (ch,), dev), _flat(dt_bias, "dt_bias", _F32, (ch,), dev),
        _flat(init_state, "init_state", _F32, (nseq, ch, N), dev)), ch, N, G


@_on_stream
def ssd_channel_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, init_state=None, *, dt_softplus=True,
                         cu_seqlens=None, y=None, final_state=None, return_final_state=True, workspace=None):
    """Selective scan with a decay per channel and state:

        delta = softplus(dt + dt_bias)   (dt + dt_bias with dt_softplus=False)
        h <- exp(delta A) h + delta x B,   y = (sum_n h C + D x) * silu(z)

    x, dt, z [b, L, Ch]; A [Ch, N] fp32 (N 8, 16 or 32); B, C [b, L, G, N];
    D, dt_bias [Ch] fp32; states [nseq, Ch, N] fp32.  Returns
    ``(y, final_state)``."""
    lib = _lib()
    code, dev = _code(x)
    if x.dim() != 3:
        raise ValueError("x must be [b, L, Ch]")
    b, L = x.shape[0], x.shape[1]
    cu, nseq = _offsets(cu_seqlens, b)
    ins, ch, N, G = _channel_inputs(x, dt, A, B, C, D, z, dt_bias, init_state, nseq, _rows, (b, L), dev)
    if y is None:
        y = _empty((b, L, ch), x.dtype, x)
        yr = _rows_t(y.data_ptr(), L * ch, ch)
    else:
        yr = _rows(y, "y", x.dtype, (b, L, ch), dev)
    fp = None
    if final_state is not None:
        fp = _flat(final_state, "final_state", _F32, (nseq, ch, N), dev)
        if fp and fp == ins.init_state:
            raise ValueError("final_state must not be init_state")
    elif return_final_state:
        final_state = _empty((nseq, ch, N), _F32, x)
        fp = final_state.data_ptr()
    shape = _channel_shape_t(b, L, ch, N, G, code, 1 if dt_softplus else 0)
    need = lib.ssd_channel_scan_workspace_size(ctypes.byref(shape), cu, nseq)
    ws = _workspace(workspace, need, x) if need else None
    st = lib.ssd_channel_scan_fwd(
        ctypes.byref(shape), cu, nseq, ctypes.byref(ins), ctypes.byref(yr), fp, None if ws is None else ws.data_ptr(),
        0 if ws is None else ws.numel() * ws.element_size(), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _fail("ssd_channel_scan_fwd", st)
    return y, final_state


@_on_stream
def ssd_channel_scan_bwd(dy, x, dt, A, B, C, D=None, z=None, dt_bias=None, init_state=None, *, dt_softplus=True,
                         cu_seqlens=None, dfinal_state=None, workspace=None):
    """Gradient of ssd_channel_scan_fwd from its inputs and dy (and that of the
    final state, zero without it).  Returns ``(dx, ddt, dA, dB, dC, dD, dz,
    ddt_bias, dinit_state)``, None where the input was None; dA, dD, ddt_bias
    and dinit_state in fp32, the others in x's type."""
    lib = _lib()
    code, dev = _code(x)
    if x.dim() != 3:
        raise ValueError("x must be [b, L, Ch]")
    b, L = x.shape[0], x.shape[1]
    ty = x.dtype
    cu, nseq = _offsets(cu_seqlens, b)
    ins, ch, N, G = _channel_inputs(x, dt, A, B, C, D, z, dt_bias, init_state, nseq, _rows, (b, L), dev)
    gr = _rows(dy, "dy", ty, (b, L, ch), dev)
    fp = _flat(dfinal_state, "dfinal_state", _F32, (nseq, ch, N), dev)
    dx, ddt = (_empty((b, L, ch), x.dtype, x) for _ in range(2))
    dz = None if z is None else _empty((b, L, ch), x.dtype, x)
    dB, dC = (_empty((b, L, G, N), x.dtype, x) for _ in range(2))
    dA = _empty((ch, N), _F32, x)
    dD = None if D is None else _empty((ch,), _F32, x)
    dbias = None if dt_bias is None else _empty((ch,), _F32, x)
    dinit = None if init_state is None else _empty((nseq, ch, N), _F32, x)
    row = lambda t, w: _rows_t(None, 0, 0) if t is None else _rows_t(t.data_ptr(), L * w, w)
    ptr = lambda t: None if t is None else t.data_ptr()
    grads = _channel_grads_t(row(dx, ch), row(ddt, ch), row(dz, ch), row(dB, G * N), row(dC, G * N), ptr(dA), ptr(dD),
                             ptr(dbias), ptr(dinit))
    shape = _channel_shape_t(b, L, ch, N, G, code, 1 if dt_softplus else 0)
    ws = _workspace(workspace, lib.ssd_channel_scan_bwd_workspace_size(ctypes.byref(shape), cu, nseq), x)
    st = lib.ssd_channel_scan_bwd(
        ctypes.byref(shape), cu, nseq, ctypes.byref(gr), ctypes.byref(ins), fp, ctypes.byref(grads), ws.data_ptr(),
        ws.numel() * ws.element_size(), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _fail("ssd_channel_scan_bwd", st)
    return dx, ddt, dA, dB, dC, dD, dz, dbias, dinit


@_on_stream
def ssd_channel_scan_step(x, dt, A, B, C, D=None, z=None, dt_bias=None, *, state, dt_softplus=True, y=None):
    """One token per sequence: x, dt, z [b, Ch], B, C [b, G, N]; ``state``
    [b, Ch, N] fp32 is advanced in place.  Returns y [b, Ch]."""
    lib = _lib()
    code, dev = _code(x)
    if x.dim() != 2:
        raise ValueError("x must be [b, Ch]")
    b = x.shape[0]
    ins, ch, N, G = _channel_inputs(x, dt, A, B, C, D, z, dt_bias, None, b, _rows2, (b,), dev)
    if state is None:
        raise TypeError("state must be a CUDA tensor")
    sp = _flat(state, "state", _F32, (b, ch, N), dev)
    if y is None:
        y = _empty((b, ch), x.dtype, x)
        yr = _rows_t(y.data_ptr(), ch, 0)
    else:
        yr = _rows2(y, "y", x.dtype, (b, ch), dev)
    shape = _channel_shape_t(b, 1, ch, N, G, code, 1 if dt_softplus else 0)
    st = lib.ssd_channel_scan_step(ctypes.byref(shape), ctypes.byref(ins), sp,
                                   ctypes.byref(yr), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _fail("ssd_channel_scan_step", st)
    return y


# ---------------------------------------------------------------------------
# block norm
# ---------------------------------------------------------------------------
def _norm_rows(t, name, dtype, shape, idx):
    """ssd_rows_t of a [..., dim] tensor whose rows lie at one stride; None
    for None."""
    if t is None:
        return None
    if not _is(t, dtype, shape, idx):
        _refuse(t, name, dtype, shape, idx)
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if len(st) == 2:
        return _rows_t(t.data_ptr(), 0, st[0])
    if 0 in shape:  # no rows
        return _rows_t(t.data_ptr(), 0, shape[-1])
    rs, span = 0, None  # span: the stride that the next dimension out has to have (None: none seen yet)
    for i in range(len(shape) - 2, -1, -1):
        if shape[i] == 1:
            continue
        if span is None:
            rs = st[i]
        elif st[i] != span:
            raise ValueError(f"{name}'s rows must lie at one stride, got strides {st}")
        span = st[i] * shape[i]
    return _rows_t(t.data_ptr(), 0, rs)


def _ref(r):
    return None if r is None else ctypes.byref(r)


def _norm_shape(x, group_size, eps, residual, gate_after):
    code, dev = _code(x)
    if x.dim() < 2:
        raise ValueError("x must be [..., dim]")
    dim = x.shape[-1]
    rcode = code if residual is None else _code(residual, "residual")[0]
    return _norm_shape_t(x.numel() // dim if dim else 0, dim, dim if group_size is None else group_size, eps, code, rcode,
                         1 if gate_after else 0), dev


@_on_stream
def ssd_block_norm_fwd(x, weight, *, z=None, residual=None, scale=None, eps=1e-5, group_size=None, gate_after=False,
                       out=None, residual_out=None):
    """RMS norm before or after a block, with its gate and scaled residual:

        v = x * silu(z)  (x without z or with gate_after)
        s = residual + scale * v
        out = s / sqrt(mean(s^2) + eps) * weight  (* silu(z) with gate_after)

    the mean over groups of ``group_size`` columns (all by default).  x, z
    [..., dim], all rows of an operand at one stride (0: one row for all);
    residual the same shape in x's type or fp32; weight, scale [dim] fp32.  Returns ``(out, residual_out)``, residual_out = s in the
    residual's type (None without a residual)."""
    lib = _lib()
    shape, dev = _norm_shape(x, group_size, eps, residual, gate_after)
    ty, full, dim = x.dtype, x.shape, x.shape[-1]
    xr = _norm_rows(x, "x", ty, full, dev)
    zr = _norm_rows(z, "z", ty, full, dev)
    wp, sp = _flat(weight, "weight", _F32, (dim,), dev), _flat(scale, "scale", _F32, (dim,), dev)
    if out is None:
        out = _empty(full, ty, x)
        outr = _rows_t(out.data_ptr(), 0, dim)
    else:
        outr = _norm_rows(out, "out", ty, full, dev)
    rr = ror = None
    if residual is not None:
        rr = _norm_rows(residual, "residual", residual.dtype, full, dev)
        if residual_out is None:
            residual_out = _empty(full, residual.dtype, x)
            ror = _rows_t(residual_out.data_ptr(), 0, dim)
        else:
            ror = _norm_rows(residual_out, "residual_out", residual.dtype, full, dev)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    st = lib.ssd_block_norm_fwd(ctypes.byref(shape), _ref(xr), wp, _ref(zr), _ref(rr), sp,
                                _ref(outr), _ref(ror), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _fail("ssd_block_norm_fwd", st)
    return out, residual_out


@_on_stream
def ssd_block_norm_bwd(dout, x, weight, *, z=None, scale=None, residual_out=None, dresidual_out=None, eps=1e-5,
                       group_size=None, gate_after=False, workspace=None):
    """Gradient of ssd_block_norm_fwd.  ``residual_out`` is the sum the forward
    call returned (where it had a residual) and ``dresidual_out`` the gradient
    of its other uses (zero without it).  Returns ``(dx, dweight, dz,
    dresidual, dscale)``, None where the input was None."""
    lib = _lib()
    shape, dev = _norm_shape(x, group_size, eps, residual_out, gate_after)
    ty, full, dim = x.dtype, x.shape, x.shape[-1]
    gr, xr = _norm_rows(dout, "dout", ty, full, dev), _norm_rows(x, "x", ty, full, dev)
    if gr is None:
        raise TypeError("dout must be a CUDA tensor")
    zr = _norm_rows(z, "z", ty, full, dev)
    wp, sp = _flat(weight, "weight", _F32, (dim,), dev), _flat(scale, "scale", _F32, (dim,), dev)
    dx = _empty(full, ty, x)
    dz = None if z is None else _empty(full, ty, x)
    dweight = _empty((dim,), _F32, x)
    dscale = None if scale is None else _empty((dim,), _F32, x)
    sr = dsr = drr = dres = None
    if residual_out is not None:
        sr = _norm_rows(residual_out, "residual_out", residual_out.dtype, full, dev)
        dsr = _norm_rows(dresidual_out, "dresidual_out", residual_out.dtype, full, dev)
        dres = _empty(full, residual_out.dtype, x)
        drr = _rows_t(dres.data_ptr(), 0, dim)
    elif dresidual_out is not None:
        raise ValueError("dresidual_out needs residual_out")
    dxr = _rows_t(dx.data_ptr(), 0, dim)
    dzr = None if z is None else _rows_t(dz.data_ptr(), 0, dim)
    ws = _workspace(workspace, lib.ssd_block_norm_bwd_workspace_size(ctypes.byref(shape)), x)
    st = lib.ssd_block_norm_bwd(
        ctypes.byref(shape), _ref(gr), _ref(xr), wp, _ref(zr), sp, _ref(sr), _ref(dsr), _ref(dxr),
        dweight.data_ptr(), _ref(dzr), _ref(drr), None if dscale is None else dscale.data_ptr(), ws.data_ptr(),
        ws.numel() * ws.element_size(), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _fail("ssd_block_norm_bwd", st)
    return dx, dweight, dz, dres, dscale
