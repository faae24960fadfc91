"""Binding of the operators around the scan: the short causal convolution, the
channel scan and the block norm.

Token-major operands (x, y, gradients) may be strided views whose last
dimension is contiguous, such as column slices of a projection's rows; states
and parameters are contiguous.  ``cu_seqlens`` is a host sequence of
nseq + 1 offsets as for ssd_fwd_varlen; without it every batch row is one
sequence.  Argument marshalling only, as everywhere in this package.
"""
from __future__ import annotations

import ctypes

import torch

_F32 = torch.float32
_CODE = {torch.float32: 0, torch.bfloat16: 1}
_MAX_PARTS = 4


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


def _lib():
    from . import load_library
    return load_library()


def _raise(fn, status):
    from . import _check
    _check(fn, status)


def _stream_of(x, stream):
    return (torch.cuda.current_stream(x.device) if stream is None else stream).cuda_stream


def _code(x, name="x"):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    code = _CODE.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {x.dtype}")
    return code


def _rows(t, name, dtype, shape, dev):
    """ssd_rows_t of a [b, L, ...] tensor whose trailing dimensions are
    contiguous; of [b, ...] where ``shape`` has no token dimension."""
    if not isinstance(t, torch.Tensor) or t.device != dev:
        raise TypeError(f"{name} must be a CUDA tensor on {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    want = 1
    for i in range(len(shape) - 1, 1, -1):
        if st[i] != want and shape[i] > 1:
            raise ValueError(f"{name} must be contiguous in its trailing dimensions")
        want *= shape[i]
    return _rows_t(t.data_ptr(), st[0], st[1])


def _rows2(t, name, dtype, shape, dev):
    """The same for one token per sequence, [b, ...] (no token dimension)."""
    if not isinstance(t, torch.Tensor) or t.device != dev:
        raise TypeError(f"{name} must be a CUDA tensor on {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    want = 1
    for i in range(len(shape) - 1, 0, -1):
        if st[i] != want and shape[i] > 1:
            raise ValueError(f"{name} must be contiguous in its trailing dimensions")
        want *= shape[i]
    return _rows_t(t.data_ptr(), st[0], 0)


def _flat(t, name, dtype, shape, dev):
    """data pointer of a contiguous tensor; None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device != dev:
        raise TypeError(f"{name} must be a CUDA tensor on {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
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


def _workspace(workspace, need, dev):
    if workspace is not None and workspace.numel() * workspace.element_size() >= need:
        return workspace
    return torch.empty(max(need, 16), device=dev, dtype=torch.uint8)


# ---------------------------------------------------------------------------
# short causal convolution
# ---------------------------------------------------------------------------
def _conv_shape(x, weight, parts, silu):
    if x.dim() != 3 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x must be [b, L, C] and weight [C, W]")
    if not 1 <= len(parts) <= _MAX_PARTS:
        raise ValueError(f"1 to {_MAX_PARTS} parts, got {len(parts)}")
    b, L, C = x.shape
    return _conv_shape_t(b, L, C, weight.shape[1], len(parts), (ctypes.c_int64 * _MAX_PARTS)(*parts), _code(x),
                         1 if silu else 0)


def ssd_conv_fwd(x, weight, bias=None, init_state=None, *, silu=True, cu_seqlens=None, split=None, y=None,
                 final_state=None, return_final_state=True, stream=None):
    """Causal depthwise convolution over the last W tokens with bias and SiLU.

    x [b, L, C], weight [C, W] fp32 (W 2 to 4), bias [C] fp32; the rows before
    a sequence come from ``init_state`` [nseq, W-1, C] (zeros without it).
    Returns ``(y, final_state)``, the final state being each sequence's last
    W-1 rows of x.  With ``split``, widths that sum to C, y is a list of
    contiguous tensors [b, L, width]: the x, B and C a scan takes.  ``y`` and
    ``final_state`` may be given; they must not overlap the inputs."""
    lib = _lib()
    code = _code(x)
    dev, dt = x.device, x.dtype
    parts = [x.shape[-1]] if split is None else [int(v) for v in split]
    shape = _conv_shape(x, weight, parts, silu)
    b, L, C = x.shape
    W = weight.shape[1]
    cu, nseq = _offsets(cu_seqlens, b)
    xr = _rows(x, "x", dt, (b, L, C), dev)
    wp = _flat(weight, "weight", _F32, (C, W), dev)
    bp = _flat(bias, "bias", _F32, (C,), dev)
    ip = _flat(init_state, "init_state", dt, (nseq, W - 1, C), dev)
    if y is None:
        ys = [torch.empty((b, L, p), device=dev, dtype=dt) for p in parts]
    else:
        ys = [y] if split is None else list(y)
        if len(ys) != len(parts):
            raise ValueError(f"y must hold {len(parts)} tensors")
    yr = (_rows_t * len(parts))(*[_rows(t, "y", dt, (b, L, p), dev) for t, p in zip(ys, parts)])
    if final_state is None and return_final_state:
        final_state = torch.empty((nseq, W - 1, C), device=dev, dtype=dt)
    fp = _flat(final_state, "final_state", dt, (nseq, W - 1, C), dev)
    if fp is not None and fp == ip:
        raise ValueError("final_state must not be init_state")
    with torch.cuda.device(dev):
        _raise("ssd_conv_fwd", lib.ssd_conv_fwd(ctypes.byref(shape), cu, nseq, ctypes.byref(xr), wp, bp, ip, yr, fp,
                                                _stream_of(x, stream)))
    return (ys[0] if split is None else ys), final_state


def ssd_conv_bwd(dy, x, weight, bias=None, init_state=None, *, silu=True, cu_seqlens=None, dfinal_state=None, dx=None,
                 workspace=None, stream=None):
    """Gradient of ssd_conv_fwd.  ``dy`` is a tensor [b, L, C] or the list of
    parts' gradients; ``dfinal_state`` [nseq, W-1, C] that of the final state
    (zero without it).  Returns ``(dx, dweight, dbias, dinit_state)``: dbias
    and dinit_state None where the input was None; dweight and dbias fp32."""
    lib = _lib()
    _code(x)
    dev, dt = x.device, x.dtype
    dys = [dy] if isinstance(dy, torch.Tensor) else list(dy)
    parts = [t.shape[-1] for t in dys]
    shape = _conv_shape(x, weight, parts, silu)
    b, L, C = x.shape
    W = weight.shape[1]
    cu, nseq = _offsets(cu_seqlens, b)
    xr = _rows(x, "x", dt, (b, L, C), dev)
    gr = (_rows_t * len(parts))(*[_rows(t, "dy", dt, (b, L, p), dev) for t, p in zip(dys, parts)])
    wp = _flat(weight, "weight", _F32, (C, W), dev)
    bp = _flat(bias, "bias", _F32, (C,), dev)
    ip = _flat(init_state, "init_state", dt, (nseq, W - 1, C), dev)
    gp = _flat(dfinal_state, "dfinal_state", dt, (nseq, W - 1, C), dev)
    if dx is None:
        dx = torch.empty((b, L, C), device=dev, dtype=dt)
    dxr = _rows(dx, "dx", dt, (b, L, C), dev)
    dweight = torch.empty((C, W), device=dev, dtype=_F32)
    dbias = None if bias is None else torch.empty((C,), device=dev, dtype=_F32)
    dinit = None if init_state is None else torch.empty((nseq, W - 1, C), device=dev, dtype=dt)
    workspace = _workspace(workspace, lib.ssd_conv_bwd_workspace_size(ctypes.byref(shape), cu, nseq), dev)
    with torch.cuda.device(dev):
        _raise("ssd_conv_bwd", lib.ssd_conv_bwd(
            ctypes.byref(shape), cu, nseq, gr, ctypes.byref(xr), wp, bp, ip, gp, ctypes.byref(dxr), dweight.data_ptr(),
            None if dbias is None else dbias.data_ptr(), None if dinit is None else dinit.data_ptr(),
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream_of(x, stream)))
    return dx, dweight, dbias, dinit


def ssd_conv_step(x, weight, bias=None, *, state, silu=True, y=None, stream=None):
    """One token per sequence: x [b, C]; ``state`` [b, W-1, C], the rows before
    it, moves up by one in place.  Returns y [b, C]."""
    lib = _lib()
    code = _code(x)
    if x.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x must be [b, C] and weight [C, W]")
    dev, dt = x.device, x.dtype
    b, C = x.shape
    W = weight.shape[1]
    xr = _rows2(x, "x", dt, (b, C), dev)
    wp = _flat(weight, "weight", _F32, (C, W), dev)
    bp = _flat(bias, "bias", _F32, (C,), dev)
    if state is None:
        raise TypeError("state must be a CUDA tensor")
    sp = _flat(state, "state", dt, (b, W - 1, C), dev)
    if y is None:
        y = torch.empty((b, C), device=dev, dtype=dt)
    yr = _rows2(y, "y", dt, (b, C), dev)
    shape = _conv_shape_t(b, 1, C, W, 1, (ctypes.c_int64 * _MAX_PARTS)(C), code, 1 if silu else 0)
    with torch.cuda.device(dev):
        _raise("ssd_conv_step", lib.ssd_conv_step(ctypes.byref(shape), ctypes.byref(xr), wp, bp, sp, ctypes.byref(yr),
                                                  _stream_of(x, stream)))
    return y


# ---------------------------------------------------------------------------
# channel scan
# ---------------------------------------------------------------------------
def _channel_inputs(x, dt, A, B, C, D, z, dt_bias, init_state, nseq, rows, tok):
    """(inputs struct, channels, states, groups); ``rows`` is _rows or _rows2
    and ``tok`` the leading dimensions (b, L) or (b,)."""
    dev, ty = x.device, x.dtype
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


def ssd_channel_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, init_state=None, *, dt_softplus=True,
                         cu_seqlens=None, y=None, final_state=None, return_final_state=True, workspace=None,
                         stream=None):
    """Selective scan with a decay per channel and state:

        delta = softplus(dt + dt_bias)   (dt + dt_bias with dt_softplus=False)
        h <- exp(delta A) h + delta x B,   y = (sum_n h C + D x) * silu(z)

    x, dt, z [b, L, Ch]; A [Ch, N] fp32 (N 8, 16 or 32); B, C [b, L, G, N];
    D, dt_bias [Ch] fp32; states [nseq, Ch, N] fp32.  Returns
    ``(y, final_state)``."""
    lib = _lib()
    code = _code(x)
    if x.dim() != 3:
        raise ValueError("x must be [b, L, Ch]")
    b, L = x.shape[0], x.shape[1]
    dev = x.device
    cu, nseq = _offsets(cu_seqlens, b)
    ins, ch, N, G = _channel_inputs(x, dt, A, B, C, D, z, dt_bias, init_state, nseq, _rows, (b, L))
    if y is None:
        y = torch.empty((b, L, ch), device=dev, dtype=x.dtype)
    yr = _rows(y, "y", x.dtype, (b, L, ch), dev)
    if final_state is None and return_final_state:
        final_state = torch.empty((nseq, ch, N), device=dev, dtype=_F32)
    fp = _flat(final_state, "final_state", _F32, (nseq, ch, N), dev)
    if fp is not None and fp == ins.init_state:
        raise ValueError("final_state must not be init_state")
    shape = _channel_shape_t(b, L, ch, N, G, code, 1 if dt_softplus else 0)
    with torch.cuda.device(dev):
        need = lib.ssd_channel_scan_workspace_size(ctypes.byref(shape), cu, nseq)
        ws = _workspace(workspace, need, dev) if need else None
        _raise("ssd_channel_scan_fwd", lib.ssd_channel_scan_fwd(
            ctypes.byref(shape), cu, nseq, ctypes.byref(ins), ctypes.byref(yr), fp, None if ws is None else ws.data_ptr(),
            0 if ws is None else ws.numel() * ws.element_size(), _stream_of(x, stream)))
    return y, final_state


def ssd_channel_scan_bwd(dy, x, dt, A, B, C, D=None, z=None, dt_bias=None, init_state=None, *, dt_softplus=True,
                         cu_seqlens=None, dfinal_state=None, workspace=None, stream=None):
    """Gradient of ssd_channel_scan_fwd from its inputs and dy (and that of the
    final state, zero without it).  Returns ``(dx, ddt, dA, dB, dC, dD, dz,
    ddt_bias, dinit_state)``, None where the input was None; dA, dD, ddt_bias
    and dinit_state in fp32, the others in x's type."""
    lib = _lib()
    code = _code(x)
    if x.dim() != 3:
        raise ValueError("x must be [b, L, Ch]")
    b, L = x.shape[0], x.shape[1]
    dev, ty = x.device, x.dtype
    cu, nseq = _offsets(cu_seqlens, b)
    ins, ch, N, G = _channel_inputs(x, dt, A, B, C, D, z, dt_bias, init_state, nseq, _rows, (b, L))
    gr = _rows(dy, "dy", ty, (b, L, ch), dev)
    fp = _flat(dfinal_state, "dfinal_state", _F32, (nseq, ch, N), dev)
    dx, ddt = (torch.empty((b, L, ch), device=dev, dtype=ty) for _ in range(2))
    dz = None if z is None else torch.empty((b, L, ch), device=dev, dtype=ty)
    dB, dC = (torch.empty((b, L, G, N), device=dev, dtype=ty) for _ in range(2))
    dA = torch.empty((ch, N), device=dev, dtype=_F32)
    dD = None if D is None else torch.empty((ch,), device=dev, dtype=_F32)
    dbias = None if dt_bias is None else torch.empty((ch,), device=dev, dtype=_F32)
    dinit = None if init_state is None else torch.empty((nseq, ch, N), device=dev, dtype=_F32)
    row = lambda t, w: _rows_t(None, 0, 0) if t is None else _rows_t(t.data_ptr(), L * w, w)
    ptr = lambda t: None if t is None else t.data_ptr()
    grads = _channel_grads_t(row(dx, ch), row(ddt, ch), row(dz, ch), row(dB, G * N), row(dC, G * N), ptr(dA), ptr(dD),
                             ptr(dbias), ptr(dinit))
    shape = _channel_shape_t(b, L, ch, N, G, code, 1 if dt_softplus else 0)
    with torch.cuda.device(dev):
        ws = _workspace(workspace, lib.ssd_channel_scan_bwd_workspace_size(ctypes.byref(shape), cu, nseq), dev)
        _raise("ssd_channel_scan_bwd", lib.ssd_channel_scan_bwd(
            ctypes.byref(shape), cu, nseq, ctypes.byref(gr), ctypes.byref(ins), fp, ctypes.byref(grads), ws.data_ptr(),
            ws.numel() * ws.element_size(), _stream_of(x, stream)))
    return dx, ddt, dA, dB, dC, dD, dz, dbias, dinit


def ssd_channel_scan_step(x, dt, A, B, C, D=None, z=None, dt_bias=None, *, state, dt_softplus=True, y=None,
                          stream=None):
    """One token per sequence: x, dt, z [b, Ch], B, C [b, G, N]; ``state``
    [b, Ch, N] fp32 is advanced in place.  Returns y [b, Ch]."""
    lib = _lib()
    code = _code(x)
    if x.dim() != 2:
        raise ValueError("x must be [b, Ch]")
    b = x.shape[0]
    dev = x.device
    ins, ch, N, G = _channel_inputs(x, dt, A, B, C, D, z, dt_bias, None, b, _rows2, (b,))
    if state is None:
        raise TypeError("state must be a CUDA tensor")
    sp = _flat(state, "state", _F32, (b, ch, N), dev)
    if y is None:
        y = torch.empty((b, ch), device=dev, dtype=x.dtype)
    yr = _rows2(y, "y", x.dtype, (b, ch), dev)
    shape = _channel_shape_t(b, 1, ch, N, G, code, 1 if dt_softplus else 0)
    with torch.cuda.device(dev):
        _raise("ssd_channel_scan_step", lib.ssd_channel_scan_step(ctypes.byref(shape), ctypes.byref(ins), sp,
                                                                  ctypes.byref(yr), _stream_of(x, stream)))
    return y


# ---------------------------------------------------------------------------
# block norm
# ---------------------------------------------------------------------------
def _norm_rows(t, name, dtype, shape, dev):
    """ssd_rows_t of a [..., dim] tensor whose rows lie at one stride; None
    for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device != dev:
        raise TypeError(f"{name} must be a CUDA tensor on {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    rs = want = 0
    for i in range(len(shape) - 2, -1, -1):
        if shape[i] == 1:
            continue
        if want == 0:
            rs, want = st[i], st[i] * shape[i]
        elif st[i] != want:
            raise ValueError(f"{name}'s rows must lie at one stride")
        else:
            want *= shape[i]
    return _rows_t(t.data_ptr(), 0, rs)


def _ref(r):
    return None if r is None else ctypes.byref(r)


def _norm_shape(x, group_size, eps, residual, gate_after):
    code = _code(x)
    if x.dim() < 2:
        raise ValueError("x must be [..., dim]")
    dim = x.shape[-1]
    rcode = code if residual is None else _code(residual, "residual")
    return _norm_shape_t(x.numel() // dim if dim else 0, dim, group_size or dim, eps, code, rcode, 1 if gate_after else 0)


def ssd_block_norm_fwd(x, weight, *, z=None, residual=None, scale=None, eps=1e-5, group_size=None, gate_after=False,
                       out=None, residual_out=None, stream=None):
    """RMS norm before or after a block, with its gate and scaled residual:

        v = x * silu(z)  (x without z or with gate_after)
        s = residual + scale * v
        out = s / sqrt(mean(s^2) + eps) * weight  (* silu(z) with gate_after)

    the mean over groups of ``group_size`` columns (all by default).  x, z
    [..., dim]; residual the same shape in x's type or fp32; weight, scale
    [dim] fp32.  Returns ``(out, residual_out)``, residual_out = s in the
    residual's type (None without a residual)."""
    lib = _lib()
    shape = _norm_shape(x, group_size, eps, residual, gate_after)
    dev, ty, full, dim = x.device, x.dtype, x.shape, x.shape[-1]
    xr = _norm_rows(x, "x", ty, full, dev)
    zr = _norm_rows(z, "z", ty, full, dev)
    wp, sp = _flat(weight, "weight", _F32, (dim,), dev), _flat(scale, "scale", _F32, (dim,), dev)
    if out is None:
        out = torch.empty(full, device=dev, dtype=ty)
    outr = _norm_rows(out, "out", ty, full, dev)
    rr = ror = None
    if residual is not None:
        rr = _norm_rows(residual, "residual", residual.dtype, full, dev)
        if residual_out is None:
            residual_out = torch.empty(full, device=dev, dtype=residual.dtype)
        ror = _norm_rows(residual_out, "residual_out", residual.dtype, full, dev)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    with torch.cuda.device(dev):
        _raise("ssd_block_norm_fwd", lib.ssd_block_norm_fwd(ctypes.byref(shape), _ref(xr), wp, _ref(zr), _ref(rr), sp,
                                                            _ref(outr), _ref(ror), _stream_of(x, stream)))
    return out, residual_out


def ssd_block_norm_bwd(dout, x, weight, *, z=None, scale=None, residual_out=None, dresidual_out=None, eps=1e-5,
                       group_size=None, gate_after=False, workspace=None, stream=None):
    """Gradient of ssd_block_norm_fwd.  ``residual_out`` is the sum the forward
    call returned (where it had a residual) and ``dresidual_out`` the gradient
    of its other uses (zero without it).  Returns ``(dx, dweight, dz,
    dresidual, dscale)``, None where the input was None."""
    lib = _lib()
    shape = _norm_shape(x, group_size, eps, residual_out, gate_after)
    dev, ty, full, dim = x.device, x.dtype, x.shape, x.shape[-1]
    gr, xr = _norm_rows(dout, "dout", ty, full, dev), _norm_rows(x, "x", ty, full, dev)
    if gr is None:
        raise TypeError("dout must be a CUDA tensor")
    zr = _norm_rows(z, "z", ty, full, dev)
    wp, sp = _flat(weight, "weight", _F32, (dim,), dev), _flat(scale, "scale", _F32, (dim,), dev)
    dx = torch.empty(full, device=dev, dtype=ty)
    dz = None if z is None else torch.empty(full, device=dev, dtype=ty)
    dweight = torch.empty((dim,), device=dev, dtype=_F32)
    dscale = None if scale is None else torch.empty((dim,), device=dev, dtype=_F32)
    sr = dsr = drr = dres = None
    if residual_out is not None:
        sr = _norm_rows(residual_out, "residual_out", residual_out.dtype, full, dev)
        dsr = _norm_rows(dresidual_out, "dresidual_out", residual_out.dtype, full, dev)
        dres = torch.empty(full, device=dev, dtype=residual_out.dtype)
        drr = _norm_rows(dres, "dresidual", residual_out.dtype, full, dev)
    elif dresidual_out is not None:
        raise ValueError("dresidual_out needs residual_out")
    dxr, dzr = _norm_rows(dx, "dx", ty, full, dev), _norm_rows(dz, "dz", ty, full, dev)
    with torch.cuda.device(dev):
        ws = _workspace(workspace, lib.ssd_block_norm_bwd_workspace_size(ctypes.byref(shape)), dev)
        _raise("ssd_block_norm_bwd", lib.ssd_block_norm_bwd(
            ctypes.byref(shape), _ref(gr), _ref(xr), wp, _ref(zr), sp, _ref(sr), _ref(dsr), _ref(dxr),
            dweight.data_ptr(), _ref(dzr), _ref(drr), None if dscale is None else dscale.data_ptr(), ws.data_ptr(),
            ws.numel() * ws.element_size(), _stream_of(x, stream)))
    return dx, dweight, dz, dres, dscale
