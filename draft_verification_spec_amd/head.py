"""Vocabulary-head operators (include/sv_head.h) on torch tensors: 8-bit hidden
rows, logits of a head held in 8-bit integers, and the cross-entropy and
distillation losses from hidden rows.

Argument marshalling only, as in the package's front end: every step runs in the
HIP library.  Scratch memory comes from torch's allocator, one piece per call on
the stream of the call, so calls on several streams, and captured ones, never
share it; `workspace` replaces it with the caller's own.
"""
from __future__ import annotations

import contextlib
import ctypes
from collections import namedtuple

SV_I8 = 2
GRAD_HIDDEN, GRAD_WEIGHT, GRAD_TWO_TERMS = 1, 2, 4
HEAD_BAD_TARGET, HEAD_NAN, HEAD_POSINF, HEAD_EMPTY, HEAD_BAD_WEIGHT = 1, 2, 4, 8, 16
MAX_H, MAX_N, MAX_V = 131072, 1048576, 16777216


class sv_logits_shape_t(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("H", ctypes.c_int32), ("V", ctypes.c_int32), ("hidden_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("hidden_stride", ctypes.c_int64), ("weight_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64)]


class sv_head_shape_t(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("H", ctypes.c_int32), ("V", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("hidden_dtype", ctypes.c_int32), ("grads", ctypes.c_int32), ("hidden_stride", ctypes.c_int64),
                ("weight_stride", ctypes.c_int64), ("temperature", ctypes.c_float), ("ignore_index", ctypes.c_int32),
                ("S", ctypes.c_int32), ("group", ctypes.c_int32), ("w_max", ctypes.c_float)]


#: hidden rows (or a head's rows) in 8 bits: codes int8 [..., H], scale float32 [...]
Act8 = namedtuple("Act8", "codes scale")
HeadCEResult = namedtuple("HeadCEResult", "loss nll lse status grad_hidden grad_weight")
HeadKDResult = namedtuple("HeadKDResult", "loss kl weight status grad_hidden grad_weight")


def bind(lib):
    """Declare the operators' C entry points on a loaded library."""
    P, i32, i64, size = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L, H = ctypes.POINTER(sv_logits_shape_t), ctypes.POINTER(sv_head_shape_t)
    for name, args, res in (
            ("sv_act8_pack", [i32, i32, i32, P, i64, P, i64, P, P], ctypes.c_int),
            ("sv_act8_unpack", [i32, i32, P, i64, P, i32, P, P], ctypes.c_int),
            ("sv_head_logits_workspace_bytes", [L], size),
            ("sv_head_logits", [L, P, P, P, P, P, P, size, P], ctypes.c_int),
            ("sv_head_ce_workspace_bytes", [H], size),
            ("sv_head_kd_workspace_bytes", [H], size),
            ("sv_head_ce", [H] + [P] * 12 + [size, P], ctypes.c_int),
            ("sv_head_kd", [H] + [P] * 14 + [size, P], ctypes.c_int)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res


_library = None


def _lib():
    global _library
    if _library is None:
        from . import load_library
        _library = load_library()
    return _library


def _check(rc):
    if rc != 0:
        from . import SpecVerifyError
        raise SpecVerifyError(rc)


def _code(dtype, what):
    import torch
    if dtype is torch.bfloat16:
        return 1
    if dtype is torch.float32:
        return 0
    raise TypeError(f"{what} must be float32 or bfloat16")


_HERE = contextlib.nullcontext()


def _on(dev, stream):
    """(context, stream handle): in the context the tensors' device and the call's
    stream are the current ones (conversions and allocations of the call belong to
    that stream)."""
    import torch
    if dev.type != "cuda":
        raise ValueError("tensors must live on the GPU")
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # (a tenth of current_stream's time)
    cur = raw(dev.index) if raw else torch.cuda.current_stream(dev).cuda_stream
    if stream is None or stream == cur:
        return (_HERE if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)), cur
    both = contextlib.ExitStack()
    both.enter_context(torch.cuda.device(dev))
    both.enter_context(torch.cuda.stream(torch.cuda.ExternalStream(stream, device=dev)))
    return both, stream


def _fits(size):
    """A size (or several joined by |, none negative) that the C structures hold; ctypes
    would keep the low 32 bits of another."""
    if not -0x80000000 <= size < 0x80000000:
        _check(-2)                                    # SV_ERR_SHAPE


def _rows(t, H, what):
    """A tensor [..., H] as rows with unit element stride: (tensor, row stride)."""
    if t.dim() < 1 or t.shape[-1] != H:
        raise ValueError(f"{what} must be [..., {H}]")
    t = t.reshape(-1, H) if t.dim() != 2 else t
    ld, one = t.stride()
    if H > 1 and one != 1 or ld < H and t.shape[0] > 1:
        t, ld = t.contiguous(), H
    return t, ld if t.shape[0] > 1 else H


def _scales(s, shape, dev, what):
    import torch
    if s.device != dev or tuple(s.shape) != tuple(shape):
        raise ValueError(f"{what} must be one scale per row on the rows' device")
    if s.dtype is torch.float32 and s.is_contiguous():
        return s
    return s.to(dtype=torch.float32).contiguous()


def _scratch(workspace, nbytes, dev):
    import torch
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous uint8 memory on the tensors' device")
    return workspace


def act8_pack(x, *, stream=None) -> Act8:
    """Rows [..., H] (float32 or bfloat16) in 8 bits: scale = max|x| / 127 of the
    row, codes = x / scale rounded to even.  A row of zeros has scale 0, a row
    with a NaN or an infinity scale NaN.  The rows of codes lie 128 bytes apart
    or a multiple, so that head_logits reads a head in place (hidden rows it copies,
    as it does those that it packs itself)."""
    import torch
    dt = _code(x.dtype, "rows")
    if x.dim() < 1 or not 1 <= x.shape[-1] <= MAX_H:
        raise ValueError(f"rows must be [..., H] with H of 1 .. {MAX_H}")
    lead, H, dev = x.shape[:-1], x.shape[-1], x.device
    _fits(x.numel() // H)
    here, st = _on(dev, stream)
    with here:
        r, ld = _rows(x, H, "rows")
        Hp = -(-H // 128) * 128
        steps, ones, n = [1], [], 1              # strides: rows of codes Hp apart, scales without gaps
        for k in reversed(lead):
            steps.append(n * Hp)
            ones.append(n)
            n *= max(k, 1)
        codes = torch.empty_strided(x.shape, steps[::-1], dtype=torch.int8, device=dev)
        scale = torch.empty_strided(lead, ones[::-1], dtype=torch.float32, device=dev)
        _check(_lib().sv_act8_pack(r.shape[0], H, dt, r.data_ptr(), ld, codes.data_ptr(), Hp, scale.data_ptr(), st))
    return Act8(codes, scale)


def act8_unpack(a: Act8, dtype=None, *, stream=None):
    """The rows that 8-bit codes stand for, codes * scale, in dtype (bfloat16
    unless given)."""
    import torch
    dtype = torch.bfloat16 if dtype is None else dtype
    dt = _code(dtype, "dtype")
    codes, dev = a.codes, a.codes.device
    if codes.dtype != torch.int8 or codes.dim() < 1 or not 1 <= codes.shape[-1] <= MAX_H:
        raise TypeError("codes must be int8 [..., H]")
    H = codes.shape[-1]
    _fits(codes.numel() // H)
    here, st = _on(dev, stream)
    with here:
        scale = _scales(a.scale, codes.shape[:-1], dev, "scale")
        r, ld = _rows(codes, H, "codes")
        y = torch.empty(codes.shape, dtype=dtype, device=dev)
        _check(_lib().sv_act8_unpack(r.shape[0], H, r.data_ptr(), ld, scale.data_ptr(), dt, y.data_ptr(), st))
    return y


def _hidden(hidden, H, what="hidden"):
    """(rows tensor, its scales or None, device) of hidden rows or an Act8."""
    import torch
    if isinstance(hidden, Act8):
        if hidden.codes.dtype != torch.int8:
            raise TypeError(f"{what} codes must be int8")
        return hidden.codes, hidden.scale, hidden.codes.device
    return hidden, None, hidden.device


def head_logits(hidden, weight: Act8, *, out_dtype=None, workspace=None, stream=None):
    """Logits [..., V] of hidden rows [..., H] under a head in 8-bit integers, as
    verify takes them: the int32 products of the codes times both scales.
    hidden: float32 or bfloat16 rows, put into 8 bits row by row on the way, or an
    Act8.  weight: Act8 with codes [V, H] (act8_pack of the head, once).
    out_dtype: bfloat16 unless given, or float32.  workspace: uint8 scratch of at
    least sv_head_logits_workspace_bytes, 256-byte aligned."""
    import torch
    if not isinstance(weight, Act8) or weight.codes.dim() != 2 or weight.codes.dtype != torch.int8:
        raise TypeError("weight must be an Act8 with int8 codes [V, H]")
    V, H = weight.codes.shape
    x, xs, dev = _hidden(hidden, H)
    odt = torch.bfloat16 if out_dtype is None else out_dtype
    oc = _code(odt, "out_dtype")
    hc = SV_I8 if xs is not None else _code(x.dtype, "hidden rows")
    if weight.codes.device != dev:
        raise ValueError("hidden and weight must be on one device")
    _fits(V | H | x.numel() // (H or 1))
    here, st = _on(dev, stream)
    with here:
        r, ld = _rows(x, H, "hidden")
        w, wld = _rows(weight.codes, H, "weight codes")
        ws = _scales(weight.scale, (V,), dev, "weight scale")
        if xs is not None:
            xs = _scales(xs, x.shape[:-1], dev, "hidden scale")
        out = torch.empty(*x.shape[:-1], V, dtype=odt, device=dev)
        shape = sv_logits_shape_t(r.shape[0], H, V, hc, oc, ld, wld, 0)
        n = _lib().sv_head_logits_workspace_bytes(ctypes.byref(shape))
        buf = _scratch(workspace, n, dev)
        _check(_lib().sv_head_logits(ctypes.byref(shape), r.data_ptr(), None if xs is None else xs.data_ptr(),
                                     w.data_ptr(), ws.data_ptr(), out.data_ptr(), buf.data_ptr(), buf.numel(), st))
    return out


def _int32(t, dev, what, shape, ignore=-1):
    """Integer indices as int32, values outside its range held at its ends, unless an
    end is the index to ignore: then they become another that is no entry."""
    import torch
    if t.dtype not in (torch.int32, torch.int64) or tuple(t.shape) != tuple(shape) or t.device != dev:
        raise ValueError(f"{what} must be int32 or int64 {list(shape)} on the rows' device")
    if t.dtype == torch.int64:
        low, high = -(1 << 31), (1 << 31) - 1
        if ignore in (low, high):
            t = torch.where((t < low) | (t > high), -1, t)
        t = t.clamp(low, high).to(torch.int32)
    return t.contiguous()


def _float(t, dev, what, shape):
    import torch
    if not t.is_floating_point() or tuple(t.shape) != tuple(shape) or t.device != dev:
        raise ValueError(f"{what} must be floating {list(shape)} on the rows' device")
    return t.to(dtype=torch.float32).contiguous()


def _loss(fn, result, hidden, weight, grad, two_terms, temperature, workspace, stream, inputs, **kw):
    import torch
    if weight.dim() != 2:
        raise ValueError("weight must be [V, H]")
    V, H = weight.shape
    dt = _code(weight.dtype, "weight")
    x, xs, dev = _hidden(hidden, H)
    if x.dim() != 2:
        raise ValueError("hidden must be [N, H]")
    if xs is None and x.dtype != weight.dtype:
        raise TypeError("hidden rows must have the weight's dtype, or be an Act8")
    if weight.device != dev:
        raise ValueError("hidden and weight must be on one device")
    grads = {True: GRAD_HIDDEN | GRAD_WEIGHT, False: 0, "hidden": GRAD_HIDDEN, "weight": GRAD_WEIGHT}.get(grad)
    if grads is None:
        raise ValueError('grad must be True, False, "hidden" or "weight"')
    if grads and two_terms:
        grads |= GRAD_TWO_TERMS
    N = x.shape[0]
    _fits(N | V | H | kw.get("S", 0))
    _fits(kw.get("group", 0))
    here, st = _on(dev, stream)
    with here:
        r, ld = _rows(x, H, "hidden")
        w, wld = _rows(weight, H, "weight")
        if xs is not None:
            xs = _scales(xs, (N,), dev, "hidden scale")
        ins = inputs(N, dev)
        shape = sv_head_shape_t(N, H, V, dt, SV_I8 if xs is not None else dt, grads, ld, wld, float(temperature),
                                kw.get("ignore_index", 0), kw.get("S", 0), kw.get("group", 0),
                                kw.get("w_max", float("inf")))
        fill = torch.empty if N else torch.zeros       # an empty batch: no launch, zero loss and gradients
        loss = fill(1, dtype=torch.float32, device=dev)
        rows, more = (torch.empty(N, dtype=torch.float32, device=dev) for _ in range(2))
        status = torch.empty(N, dtype=torch.int32, device=dev)
        gh = fill(N, H, dtype=weight.dtype, device=dev) if grads & GRAD_HIDDEN else None
        gw = fill(V, H, dtype=weight.dtype, device=dev) if grads & GRAD_WEIGHT else None
        lib = _lib()
        n = getattr(lib, fn + "_workspace_bytes")(ctypes.byref(shape))
        buf = _scratch(workspace, n, dev)
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        _check(getattr(lib, fn)(ctypes.byref(shape), p(r), p(xs), p(w), *[p(t) for t in ins], p(rows), p(more),
                                p(status), p(loss), p(gh), p(gw), p(buf), buf.numel(), st))
    return result(loss, rows, more, status, gh, gw)


def head_ce(hidden, weight, targets, row_weight=None, *, temperature: float = 1.0, ignore_index: int = -1,
            grad=True, two_terms: bool = False, workspace=None, stream=None) -> HeadCEResult:
    """Softmax cross entropy of hidden rows under a vocabulary head, from pieces
    of the vocabulary: no logits are kept.

    hidden [N, H] in the weight's dtype, or an Act8 (rows held in 8 bits; the
    gradients are then those at the rows it stands for); weight [V, H] float32 or
    bfloat16; targets [N] int32 or int64; row_weight [N] float32, any finite
    factors (1 / N, advantages), or None for ones.  Logits are divided by
    temperature.  Rows whose target is ignore_index are left out.

    grad: True for the gradients of hidden rows and weight, "hidden" or "weight"
    for one of them, False for none.  Returns loss [1] float32 = sum of row_weight
    * nll, nll and lse [N] float32, status [N] (HEAD_* bits; such a row has NaN
    results and adds nothing), and the gradients in the weight's dtype.

    two_terms: for bfloat16 the logits' gradient, an operand of both gradients'
    products, in two bfloat16 terms instead of one: the gradients are then off by
    their own rounding alone (0.0017 of the norm, else up to 0.0028), for a second
    product of each.  Up to 32 rows, and in float32, that is so anyway."""
    if not -(1 << 31) <= int(ignore_index) < (1 << 31):
        raise ValueError("ignore_index must fit in 32 bits")

    def inputs(N, dev):
        return (_int32(targets, dev, "targets", (N,), int(ignore_index)),
                None if row_weight is None else _float(row_weight, dev, "row_weight", (N,)))
    return _loss("sv_head_ce", HeadCEResult, hidden, weight, grad, two_terms, temperature, workspace, stream, inputs,
                 ignore_index=int(ignore_index))


def head_kd(hidden, weight, topk_val, topk_idx, row_sample, rewards, group: int, *, w_max: float = float("inf"),
            grad=True, two_terms: bool = False, workspace=None, stream=None) -> HeadKDResult:
    """kd's reward-weighted distillation loss over the stored top-32, from hidden
    rows and head instead of drafter logits: no logits are kept.  hidden, weight,
    grad, two_terms as in head_ce; topk_val, topk_idx [N, 32], row_sample [N], rewards [S],
    group and w_max as in kd.  Returns loss [1] float32, kl and weight [N] float32,
    status [N] (KD_* bits) and the gradients in the weight's dtype."""
    def inputs(N, dev):
        return (_float(topk_val, dev, "topk_val", (N, 32)), _int32(topk_idx, dev, "topk_idx", (N, 32)),
                _int32(row_sample, dev, "row_sample", (N,)), _float(rewards, dev, "rewards", (rewards.numel(),)))
    return _loss("sv_head_kd", HeadKDResult, hidden, weight, grad, two_terms, 1.0, workspace, stream, inputs,
                 S=rewards.numel(), group=int(group), w_max=float(w_max))
