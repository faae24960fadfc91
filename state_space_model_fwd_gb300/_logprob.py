"""Binding of the end of a language model: log-probabilities of given tokens,
the log of the sum, entropies and the top alternatives, from logits or from
hidden states and the output weights.

Rows of an operand lie at one stride.  Column slices are fine, from hidden
states on 16-byte boundaries; one row for all is, for logits.  Operands are on the current device; every function takes ``stream``
(the current one by default).  Argument marshalling only.
"""
from __future__ import annotations

import ctypes

import torch

from ._layer import _F32, _code, _empty, _fail, _flat, _given, _lib, _norm_rows, _on_stream, _rows_t, _workspace


_MAX_TOP = 64


class _logprob_shape_t(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("top", ctypes.c_int64), ("dtype", ctypes.c_int)]


class _head_shape_t(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("dim", ctypes.c_int64), ("dtype", ctypes.c_int)]


def declare(lib):
    """Declare this module's entry points on the loaded library."""
    vp = ctypes.c_void_p
    lib.ssd_token_logprob_fwd.argtypes = [vp] * 9
    lib.ssd_token_logprob_bwd.argtypes = [vp] * 10
    for name in ("ssd_head_logprob_workspace_size", "ssd_head_logprob_bwd_workspace_size"):
        getattr(lib, name).argtypes = [vp]
        getattr(lib, name).restype = ctypes.c_size_t
    lib.ssd_head_logprob_fwd.argtypes = [vp] * 8 + [ctypes.c_size_t, vp]
    lib.ssd_head_logprob_bwd.argtypes = [vp] * 12 + [ctypes.c_size_t, vp]
    for name in ("ssd_token_logprob_fwd", "ssd_token_logprob_bwd", "ssd_head_logprob_fwd", "ssd_head_logprob_bwd"):
        getattr(lib, name).restype = ctypes.c_int


def _shape_of(logits, top):
    code, dev = _code(logits, "logits")
    if logits.dim() < 2:
        raise ValueError("logits must be [..., vocab]")
    vocab, lead = logits.shape[-1], logits.shape[:-1]
    return _logprob_shape_t(logits.numel() // vocab if vocab else 0, vocab, top, code), dev, lead


def _ptr(t):
    return None if t is None else t.data_ptr()


def _row_outputs(lead, like, targets, return_entropy):
    """(logprob or None, lse, entropy or None)"""
    return (None if targets is None else _empty(lead, _F32, like), _empty(lead, _F32, like),
            _empty(lead, _F32, like) if return_entropy else None)


@_on_stream
def ssd_token_logprob_fwd(logits, targets=None, *, top=0, return_entropy=True):
    """Log-probabilities of the given tokens, entropy and top alternatives:

        lse = log(sum(exp(z))),  logprob = z[target] - lse
        entropy = lse - sum(p z),  p = exp(z - lse)

    logits [..., vocab]; targets [...] int64 (negative: no token, its
    log-probability 0; past the vocabulary: NaN).  Returns ``(logprob, lse,
    entropy, top_logprob, top_index)``, the latter two [..., top] (at most 64),
    the most probable first, equal ones by index; None for what was not asked
    for."""
    lib = _lib()
    shape, dev, lead = _shape_of(logits, top)
    zr = _norm_rows(logits, "logits", logits.dtype, logits.shape, dev)
    tp = _flat(targets, "targets", torch.int64, lead, dev)
    logprob, lse, entropy = _row_outputs(lead, logits, targets, return_entropy)
    value = index = None
    if 0 < top <= _MAX_TOP:  # (others are refused by the call)
        value, index = _empty((*lead, top), _F32, logits), _empty((*lead, top), torch.int64, logits)
    st = lib.ssd_token_logprob_fwd(ctypes.byref(shape), ctypes.byref(zr), tp, _ptr(logprob), lse.data_ptr(), _ptr(entropy),
                                   _ptr(value), _ptr(index), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _fail("ssd_token_logprob_fwd", st)
    return logprob, lse, entropy, value, index


@_on_stream
def ssd_token_logprob_bwd(logits, targets, lse, entropy=None, *, dlogprob=None, dlse=None, dentropy=None, dlogits=None):
    """Gradient of ssd_token_logprob_fwd from its logits, what it returned and
    the gradients of logprob, lse and entropy (zero without them; ``entropy``
    is needed with ``dentropy`` only).  ``dlogits`` may be given, the logits
    themselves included.  Returns dlogits."""
    lib = _lib()
    shape, dev, lead = _shape_of(logits, 0)
    zr = _norm_rows(logits, "logits", logits.dtype, logits.shape, dev)
    tp = _flat(targets, "targets", torch.int64, lead, dev)
    lp = _given(lse, "lse", _F32, lead, dev)
    ep = _flat(entropy, "entropy", _F32, lead, dev)
    g = [_flat(v, n, _F32, lead, dev) for v, n in ((dlogprob, "dlogprob"), (dlse, "dlse"), (dentropy, "dentropy"))]
    if dlogprob is not None and targets is None:
        raise ValueError("dlogprob needs targets")
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs entropy")
    if dlogits is None:
        dlogits = _empty(logits.shape, logits.dtype, logits)
        dr = _rows_t(dlogits.data_ptr(), 0, logits.shape[-1])
    else:
        dr = _norm_rows(dlogits, "dlogits", logits.dtype, logits.shape, dev)
    st = lib.ssd_token_logprob_bwd(ctypes.byref(shape), ctypes.byref(zr), tp, lp, ep, *g, ctypes.byref(dr),
                                   torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _fail("ssd_token_logprob_bwd", st)
    return dlogits


# ---------------------------------------------------------------------------
# from hidden states
# ---------------------------------------------------------------------------
def _head(hidden, weight):
    """(shape, rows of hidden, rows of weight, device, leading dimensions)"""
    code, dev = _code(hidden, "hidden")
    if hidden.dim() < 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("hidden must be [..., dim] and weight [vocab, dim]")
    dim, lead = hidden.shape[-1], hidden.shape[:-1]
    hr = _norm_rows(hidden, "hidden", hidden.dtype, hidden.shape, dev)
    wr = _norm_rows(weight, "weight", hidden.dtype, (weight.shape[0], dim), dev)
    return _head_shape_t(hidden.numel() // dim if dim else 0, weight.shape[0], dim, code), hr, wr, dev, lead


@_on_stream
def ssd_head_logprob_fwd(hidden, weight, targets=None, *, return_entropy=True, workspace=None):
    """ssd_token_logprob_fwd of the logits hidden @ weight.T, which are formed
    on the tensor cores and not stored.

    hidden [..., dim], weight [vocab, dim] bf16 with rows on 16-byte
    boundaries (dim a multiple of 8); targets [...] int64.  Returns
    ``(logprob, lse, entropy)``, None for what was not asked for."""
    lib = _lib()
    shape, hr, wr, dev, lead = _head(hidden, weight)
    tp = _flat(targets, "targets", torch.int64, lead, dev)
    logprob, lse, entropy = _row_outputs(lead, hidden, targets, return_entropy)
    ws = _workspace(workspace, lib.ssd_head_logprob_workspace_size(ctypes.byref(shape)), hidden)
    st = lib.ssd_head_logprob_fwd(ctypes.byref(shape), ctypes.byref(hr), ctypes.byref(wr), tp, _ptr(logprob), lse.data_ptr(),
                                  _ptr(entropy), ws.data_ptr(), ws.numel() * ws.element_size(),
                                  torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _fail("ssd_head_logprob_fwd", st)
    return logprob, lse, entropy


@_on_stream
def ssd_head_logprob_bwd(hidden, weight, targets, lse, entropy=None, *, dlogprob=None, dlse=None, dentropy=None,
                         need_dhidden=True, need_dweight=True, workspace=None):
    """Gradient of ssd_head_logprob_fwd from its inputs, what it returned and
    the gradients of logprob, lse and entropy (zero without them; ``entropy``
    is needed with ``dentropy`` only).  Returns ``(dhidden, dweight)`` in
    bf16, None for what is not needed.  The workspace holds the logits'
    gradient, 2 bytes each."""
    lib = _lib()
    shape, hr, wr, dev, lead = _head(hidden, weight)
    tp = _flat(targets, "targets", torch.int64, lead, dev)
    lp = _given(lse, "lse", _F32, lead, dev)
    ep = _flat(entropy, "entropy", _F32, lead, dev)
    g = [_flat(v, n, _F32, lead, dev) for v, n in ((dlogprob, "dlogprob"), (dlse, "dlse"), (dentropy, "dentropy"))]
    if dlogprob is not None and targets is None:
        raise ValueError("dlogprob needs targets")
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs entropy")
    dim = hidden.shape[-1]
    dhidden = _empty(hidden.shape, hidden.dtype, hidden) if need_dhidden else None
    dweight = _empty(weight.shape, hidden.dtype, hidden) if need_dweight else None
    dhr = None if dhidden is None else ctypes.byref(_rows_t(dhidden.data_ptr(), 0, dim))
    dwr = None if dweight is None else ctypes.byref(_rows_t(dweight.data_ptr(), 0, dim))
    ws = _workspace(workspace, lib.ssd_head_logprob_bwd_workspace_size(ctypes.byref(shape)), hidden)
    st = lib.ssd_head_logprob_bwd(ctypes.byref(shape), ctypes.byref(hr), ctypes.byref(wr), tp, lp, ep, *g, dhr, dwr,
                                  ws.data_ptr(), ws.numel() * ws.element_size(), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _fail("ssd_head_logprob_bwd", st)
    return dhidden, dweight
