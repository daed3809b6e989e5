"""Operators on given tokens' log-probabilities (include/sv_logprobs.h) on torch tensors:
the log-probabilities with the rows' entropies and largest alternatives, and the gradient
of the logits from theirs.

Argument marshalling only, as in head.py: every step runs in the HIP library, and scratch
memory comes from torch's allocator, one piece per call on the stream of the call.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

from .head import _check, _code, _fits, _float, _int32, _lib, _on, _rows, _scratch

MAX_TOP = 32


class sv_logprobs_shape_t(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("V", ctypes.c_int32), ("dtype", ctypes.c_int32), ("top", ctypes.c_int32),
                ("row_stride", ctypes.c_int64), ("temperature", ctypes.c_float), ("ignore_index", ctypes.c_int32)]


class sv_logprobs_grad_shape_t(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("V", ctypes.c_int32), ("dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("row_stride", ctypes.c_int64), ("grad_stride", ctypes.c_int64), ("temperature", ctypes.c_float),
                ("ignore_index", ctypes.c_int32)]


#: logp, entropy, lse and status [...]; norm [2, ...]: the rows' largest logits and the logarithms
#: of their sums beyond them; top_logp and top_idx [..., top], None without alternatives
LogprobsResult = namedtuple("LogprobsResult", "logp entropy lse norm status top_logp top_idx")


def bind(lib):
    """Declare the operators' C entry points on a loaded library."""
    P = ctypes.c_void_p
    S, G = ctypes.POINTER(sv_logprobs_shape_t), ctypes.POINTER(sv_logprobs_grad_shape_t)
    for name, args, res in (("sv_logprobs_workspace_bytes", [S], ctypes.c_size_t),
                            ("sv_logprobs", [S] + [P] * 10 + [ctypes.c_size_t, P], ctypes.c_int),
                            ("sv_logprobs_grad", [G] + [P] * 8, ctypes.c_int)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res


def _logits(logits):
    """(dtype code, vocabulary, leading shape) of logits [..., V]."""
    dt, shape = _code(logits.dtype, "logits"), logits.shape
    if not shape or shape[-1] < 1:
        raise ValueError("logits must be [..., V]")
    V, lead = shape[-1], shape[:-1]
    _fits(V | logits.numel() // V)
    return dt, V, lead


def _index(ignore_index):
    ignore = int(ignore_index)
    if not -(1 << 31) <= ignore < (1 << 31):
        raise ValueError("ignore_index must fit in 32 bits")
    return ignore


def logprobs(logits, tokens, temperature: float = 1.0, *, top: int = 0, ignore_index: int = -1, workspace=None,
             stream=None) -> LogprobsResult:
    """Log-probabilities of one given token a row under softmax(logits / temperature), with
    the rows' entropies and their `top` (0 .. 32) largest alternatives.

    logits [..., V] float32 or bfloat16, tokens [...] int32 or int64.  Alternatives come by
    value, equal ones by index; tokens of probability 0 (logits of -inf) are none, and what a
    row lacks is (-inf, -1).  Rows whose token is ignore_index are left out, whatever they hold: 0,
    and no alternatives.  A row with a data error (its token outside the vocabulary, a logit
    NaN or +inf, or all -inf) has its HEAD_* bits in status and NaN results.  Each result is a
    tensor of its own, which may be changed in place; the rows' (24 bytes a row) share one
    piece of memory, which the last of them frees.  workspace: uint8 scratch of at least
    sv_logprobs_workspace_bytes, 256-byte aligned."""
    import torch
    dt, V, lead = _logits(logits)
    top, ignore, dev = int(top), _index(ignore_index), logits.device
    if not 0 <= top <= MAX_TOP:
        raise ValueError(f"top must be 0 .. {MAX_TOP}")
    here, st = _on(dev, stream)
    with here:
        r, ld = _rows(logits, V, "logits")
        t = _int32(tokens, dev, "tokens", lead, ignore)
        # One piece of memory for the rows' results: a tensor of its own costs the host three of
        # the pieces that this split gives, which autograd takes for tensors of their own too
        # (views of one, it refuses to change in place).
        n = r.shape[0]
        f = torch.empty(6 * n, dtype=torch.float32, device=dev)
        logp, entropy, lse, norm, status = torch.unsafe_split_with_sizes(f, (n, n, n, 2 * n, n))
        p, tv, ti = f.data_ptr(), None, None
        if top:
            tv = torch.empty((*lead, top), dtype=torch.float32, device=dev)
            ti = torch.empty((*lead, top), dtype=torch.int32, device=dev)
        shape = sv_logprobs_shape_t(n, V, dt, top, ld, float(temperature), ignore)
        lib, at = _lib(), ctypes.byref(shape)
        need = lib.sv_logprobs_workspace_bytes(at)
        buf = _scratch(workspace, need, dev) if need or workspace is not None else None
        _check(lib.sv_logprobs(at, r.data_ptr(), t.data_ptr(), p, p + 4 * n, p + 8 * n, p + 12 * n, p + 20 * n,
                               tv.data_ptr() if top else None, ti.data_ptr() if top else None,
                               None if buf is None else buf.data_ptr(), 0 if buf is None else buf.numel(), st))
    # (.data: the tensor as it is shaped here, no view of the one before)
    if len(lead) != 1:
        logp, entropy, lse, status = (x.view(lead).data for x in (logp, entropy, lse, status))
    norm, status = norm.view(2, *lead).data, status.view(torch.int32).data
    return LogprobsResult(logp, entropy, lse, norm, status, tv, ti)


def _shared(a, lda, b, ldb):
    """Whether rows a [N, V] and b [N, V], lda and ldb elements apart, share memory otherwise than
    element by element."""
    n, V = a.shape
    ea, eb, d = a.element_size(), b.element_size(), b.data_ptr() - a.data_ptr()
    if not n or d >= ((n - 1) * lda + V) * ea or -d >= ((n - 1) * ldb + V) * eb:
        return False
    step = lda * ea
    if n == 1 or step != ldb * eb:
        return d != 0 or a.dtype is not b.dtype or n > 1
    if d == 0 and a.dtype is b.dtype:
        return False
    d %= step                                         # b's rows lie in the gaps of a's, or meet them
    return d < V * ea or d + V * eb > step


def logprobs_grad(logits, tokens, result: LogprobsResult, grad_logp, grad_entropy=None, temperature: float = 1.0, *,
                  ignore_index: int = -1, out=None, out_dtype=None, stream=None):
    """The gradient of the logits [..., V] from those of the log-probabilities (grad_logp) and
    entropies (grad_entropy, or None for zeros), float32 [...] each.

    logits, tokens, temperature and ignore_index as logprobs was given them, result what it
    returned.  Rows left out and rows with a data error get zeros.  out_dtype: the logits'
    unless given.  out: memory for the gradient, of its shape and type with unit element
    stride, the logits themselves among it (they are then lost); it may not overlap them
    otherwise."""
    import torch
    dt, V, lead = _logits(logits)
    ignore, dev = _index(ignore_index), logits.device
    norm = result.norm
    if norm.dtype is not torch.float32 or tuple(norm.shape) != (2, *lead) or norm.device != dev:
        raise ValueError("result must be logprobs' of these logits")
    odt = out_dtype if out_dtype is not None else out.dtype if out is not None else logits.dtype
    gt = _code(odt, "out_dtype")
    if out is not None and (out.dtype is not odt or out.shape != logits.shape or out.device != dev):
        raise ValueError("out must have the logits' shape and device, and the gradient's type")
    here, st = _on(dev, stream)
    with here:
        r, ld = _rows(logits, V, "logits")
        t = _int32(tokens, dev, "tokens", lead, ignore)
        g = _float(grad_logp, dev, "grad_logp", lead)
        h = None if grad_entropy is None else _float(grad_entropy, dev, "grad_entropy", lead)
        e = None if h is None else _float(result.entropy, dev, "entropy", lead)
        norm = norm.contiguous()
        if out is None:
            grad = o = torch.empty(logits.shape, dtype=odt, device=dev)
            old = V
        else:
            grad = out
            o, old = _rows(out, V, "out")
            if o.data_ptr() != out.data_ptr():
                raise ValueError("out must have unit element stride and rows one stride apart")
            if _shared(r, ld, o, old):
                raise ValueError("out must be the logits' own memory, element by element, or lie apart from it")
        shape = sv_logprobs_grad_shape_t(r.shape[0], V, dt, gt, ld, old, float(temperature), ignore)
        _check(_lib().sv_logprobs_grad(ctypes.byref(shape), r.data_ptr(), t.data_ptr(), norm.data_ptr(),
                                       None if e is None else e.data_ptr(), g.data_ptr(),
                                       None if h is None else h.data_ptr(), o.data_ptr(), st))
    return grad
