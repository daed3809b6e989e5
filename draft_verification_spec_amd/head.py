"""Vocabulary-head operators (include/sv_head.h, include/sv_mx4.h) on torch tensors: rows
in 8 bits and in microscaled 4 bits, logits of a head held in either, and the
cross-entropy and distillation losses from hidden rows.

Argument marshalling only, as in the package's front end: every step runs in the
HIP library.  Scratch memory comes from torch's allocator, one piece per call on
the stream of the call, so calls on several streams, and captured ones, never
share it; `workspace` replaces it with the caller's own.
"""
from __future__ import annotations

import contextlib
import ctypes
from collections import namedtuple

SV_I8, SV_MX4 = 2, 3
MX4_BLOCK = 32
GRAD_HIDDEN, GRAD_WEIGHT, GRAD_TWO_TERMS = 1, 2, 4
HEAD_BAD_TARGET, HEAD_NAN, HEAD_POSINF, HEAD_EMPTY, HEAD_BAD_WEIGHT = 1, 2, 4, 8, 16
MAX_H, MAX_N, MAX_V = 131072, 1048576, 16777216


class sv_logits_shape_t(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("H", ctypes.c_int32), ("V", ctypes.c_int32), ("hidden_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("hidden_stride", ctypes.c_int64), ("weight_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64)]


class sv_logits4_shape_t(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("H", ctypes.c_int32), ("V", ctypes.c_int32), ("hidden_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("hidden_stride", ctypes.c_int64), ("hidden_scale_stride", ctypes.c_int64),
                ("weight_stride", ctypes.c_int64), ("weight_scale_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)]


class sv_head_shape_t(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("H", ctypes.c_int32), ("V", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("hidden_dtype", ctypes.c_int32), ("grads", ctypes.c_int32), ("hidden_stride", ctypes.c_int64),
                ("weight_stride", ctypes.c_int64), ("temperature", ctypes.c_float), ("ignore_index", ctypes.c_int32),
                ("S", ctypes.c_int32), ("group", ctypes.c_int32), ("w_max", ctypes.c_float)]


#: hidden rows (or a head's rows) in 8 bits: codes int8 [..., H], scale float32 [...]
Act8 = namedtuple("Act8", "codes scale")
#: rows [..., width] in 4 bits, 32 elements to a power-of-two scale (the OCP microscaling format
#: MXFP4): codes uint8 [..., (width + 1) // 2], the even element in the low half of a byte;
#: scale uint8 [..., (width + 31) // 32], e for 2 ** (e - 127), 255 for NaN
Mx4 = namedtuple("Mx4", "codes scale width")
HeadCEResult = namedtuple("HeadCEResult", "loss nll lse status grad_hidden grad_weight")
HeadKDResult = namedtuple("HeadKDResult", "loss kl weight status grad_hidden grad_weight")


def bind(lib):
    """Declare the operators' C entry points on a loaded library."""
    P, i32, i64, size = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L, H = ctypes.POINTER(sv_logits_shape_t), ctypes.POINTER(sv_head_shape_t)
    L4 = ctypes.POINTER(sv_logits4_shape_t)
    for name, args, res in (
            ("sv_act8_pack", [i32, i32, i32, P, i64, P, i64, P, P], ctypes.c_int),
            ("sv_act8_unpack", [i32, i32, P, i64, P, i32, P, P], ctypes.c_int),
            ("sv_head_logits_workspace_bytes", [L], size),
            ("sv_head_logits", [L, P, P, P, P, P, P, size, P], ctypes.c_int),
            ("sv_mx4_pack", [i32, i32, i32, P, i64, P, i64, P, i64, P], ctypes.c_int),
            ("sv_mx4_unpack", [i32, i32, P, i64, P, i64, i32, P, P], ctypes.c_int),
            ("sv_head_logits4_workspace_bytes", [L4], size),
            ("sv_head_logits4", [L4, P, P, P, P, P, P, size, P], ctypes.c_int),
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


_current = None


def _find_current():
    """(raw stream of a device, current device): torch's own functions behind current_stream and
    current_device, at a tenth of their time, where it has them."""
    global _current
    import torch
    _current = (getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream),
                getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device)
    return _current


def _on(dev, stream):
    """(context, stream handle): in the context the tensors' device and the call's
    stream are the current ones (conversions and allocations of the call belong to
    that stream)."""
    import torch
    if dev.type != "cuda":
        raise ValueError("tensors must live on the GPU")
    raw, now = _current or _find_current()
    index = dev.index
    cur = raw(index)
    if stream is None or stream == cur:
        return (_HERE if index == now() else torch.cuda.device(dev)), cur
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


def _padded(lead, n, unit, dtype, dev):
    """Memory for rows [..., n] that lie a multiple of `unit` elements apart."""
    import torch
    np = -(-n // unit) * unit
    if len(lead) == 1:
        return torch.empty_strided((lead[0], n), (np, 1), dtype=dtype, device=dev), np
    steps, k = [1], np
    for d in reversed(lead):
        steps.append(k)
        k *= max(d, 1)
    return torch.empty_strided((*lead, n), steps[::-1], dtype=dtype, device=dev), np


def mx4_pack(x, *, stream=None) -> Mx4:
    """Rows [..., H] (float32 or bfloat16) in microscaled 4 bits: to each 32 elements the scale
    2 ** (floor(log2(max|x|)) - 2), and x / scale rounded to the nearest of 0, 0.5, 1, 1.5, 2,
    3, 4, 6 and their negatives, ties to even, the largest magnitudes to 6.  A block with a
    NaN or an infinity stands for NaN.  Rows of codes lie 128 bytes apart or a multiple, rows
    of scales 16, so that head_logits reads a head in place."""
    import torch
    dt = _code(x.dtype, "rows")
    if x.dim() < 1 or not 1 <= x.shape[-1] <= MAX_H:
        raise ValueError(f"rows must be [..., H] with H of 1 .. {MAX_H}")
    lead, H, dev = x.shape[:-1], x.shape[-1], x.device
    _fits(x.numel() // H)
    here, st = _on(dev, stream)
    with here:
        r, ld = _rows(x, H, "rows")
        codes, cld = _padded(lead, (H + 1) // 2, 128, torch.uint8, dev)
        scale, sld = _padded(lead, -(-H // MX4_BLOCK), 16, torch.uint8, dev)
        _check(_lib().sv_mx4_pack(r.shape[0], H, dt, r.data_ptr(), ld, codes.data_ptr(), cld, scale.data_ptr(), sld, st))
    return Mx4(codes, scale, H)


def _mx4(a, what):
    """(width, leading shape, device) of an Mx4 whose parts belong together."""
    import torch
    codes, scale, H = a
    if codes.dtype is not torch.uint8 or scale.dtype is not torch.uint8:
        raise TypeError(f"{what} codes and scales must be uint8")
    H = int(H)
    if codes.dim() < 1 or not 1 <= H <= MAX_H or codes.shape[-1] != (H + 1) // 2:
        raise ValueError(f"{what} codes must be [..., (width + 1) // 2] with a width of 1 .. {MAX_H}")
    lead = codes.shape[:-1]
    if scale.shape != (*lead, -(-H // MX4_BLOCK)) or scale.device != codes.device:
        raise ValueError(f"{what} scales must be one byte per {MX4_BLOCK} elements of a row on the codes' device")
    return H, lead, codes.device


def mx4_unpack(a: Mx4, dtype=None, *, stream=None):
    """The rows [..., width] that 4-bit codes and their scales stand for, in dtype (bfloat16
    unless given)."""
    import torch
    if not isinstance(a, Mx4):
        raise TypeError("rows must be an Mx4")
    dtype = torch.bfloat16 if dtype is None else dtype
    dt = _code(dtype, "dtype")
    H, lead, dev = _mx4(a, "rows'")
    _fits(a.codes.numel() // ((H + 1) // 2))
    here, st = _on(dev, stream)
    with here:
        c, cld = _rows(a.codes, (H + 1) // 2, "codes")
        s, sld = _rows(a.scale, -(-H // MX4_BLOCK), "scales")
        y = torch.empty((*lead, H), dtype=dtype, device=dev)
        _check(_lib().sv_mx4_unpack(c.shape[0], H, c.data_ptr(), cld, s.data_ptr(), sld, dt, y.data_ptr(), st))
    return y


def _logits4(hidden, weight, out_dtype, workspace, stream):
    import torch
    H, lead, dev = _mx4(weight, "weight")
    if len(lead) != 1:
        raise TypeError("weight must be an Mx4 with codes [V, (H + 1) // 2]")
    V = lead[0]
    if isinstance(hidden, Act8):
        raise TypeError("hidden rows in 8 bits need a weight in 8 bits")
    if isinstance(hidden, Mx4):
        h, rows, hdev = _mx4(hidden, "hidden")
        if h != H:
            raise ValueError(f"hidden must be [..., {H}]")
        hc = SV_MX4
    else:
        rows, hdev, hc = hidden.shape[:-1], hidden.device, _code(hidden.dtype, "hidden rows")
    odt = torch.bfloat16 if out_dtype is None else out_dtype
    oc = _code(odt, "out_dtype")
    if hdev != dev:
        raise ValueError("hidden and weight must be on one device")
    _fits(V | (hidden.codes.numel() // ((H + 1) // 2) if hc == SV_MX4 else hidden.numel() // H))
    here, st = _on(dev, stream)
    with here:
        xs, xsld = None, 0
        if hc == SV_MX4:
            x, ld = _rows(hidden.codes, (H + 1) // 2, "hidden codes")
            xs, xsld = _rows(hidden.scale, -(-H // MX4_BLOCK), "hidden scales")
        else:
            x, ld = _rows(hidden, H, "hidden")
        w, wld = _rows(weight.codes, (H + 1) // 2, "weight codes")
        ws, wsld = _rows(weight.scale, -(-H // MX4_BLOCK), "weight scales")
        out = torch.empty((*rows, V), dtype=odt, device=dev)
        shape = sv_logits4_shape_t(x.shape[0], H, V, hc, oc, ld, xsld, wld, wsld, 0)
        lib = _lib()
        n = lib.sv_head_logits4_workspace_bytes(ctypes.byref(shape))
        buf = _scratch(workspace, n, dev) if n or workspace is not None else None
        _check(lib.sv_head_logits4(ctypes.byref(shape), x.data_ptr(), None if xs is None else xs.data_ptr(), w.data_ptr(),
                                   ws.data_ptr(), out.data_ptr(), None if buf is None else buf.data_ptr(),
                                   0 if buf is None else buf.numel(), st))
    return out


def _hidden(hidden, H, what="hidden"):
    """(rows tensor, its scales or None, device) of hidden rows or an Act8."""
    import torch
    if isinstance(hidden, Act8):
        if hidden.codes.dtype != torch.int8:
            raise TypeError(f"{what} codes must be int8")
        return hidden.codes, hidden.scale, hidden.codes.device
    if isinstance(hidden, Mx4):
        raise TypeError(f"{what} must be a tensor or an Act8")
    return hidden, None, hidden.device


def head_logits(hidden, weight, *, out_dtype=None, workspace=None, stream=None):
    """Logits [..., V] of hidden rows [..., H] under a head in 8-bit integers, as
    verify takes them: the int32 products of the codes times both scales.
    hidden: float32 or bfloat16 rows, put into 8 bits row by row on the way, or an
    Act8.  weight: Act8 with codes [V, H] (act8_pack of the head, once).
    Or, for a drafter, under a head in microscaled 4 bits: weight is the Mx4 of rows [V, H]
    (mx4_pack of the head, once), hidden rows are put into 4 bits on the way or given as an
    Mx4, and the products of what the codes stand for are summed in fp32 (for rows of normal
    values the logits are off by 0.115 of their norm for that, beside the head's own 0.117).
    out_dtype: bfloat16 unless given, or float32.  workspace: uint8 scratch of at
    least sv_head_logits_workspace_bytes (4 bits: sv_head_logits4_workspace_bytes),
    256-byte aligned."""
    import torch
    if isinstance(weight, Mx4):
        return _logits4(hidden, weight, out_dtype, workspace, stream)
    if isinstance(hidden, Mx4):
        raise TypeError("hidden rows in 4 bits need a weight in 4 bits")
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
    if t.dtype not in (torch.int32, torch.int64) or t.shape != shape or t.device != dev:
        raise ValueError(f"{what} must be int32 or int64 {list(shape)} on the rows' device")
    if t.dtype == torch.int64:
        low, high = -(1 << 31), (1 << 31) - 1
        if ignore in (low, high):
            t = torch.where((t < low) | (t > high), -1, t)
        t = t.clamp(low, high).to(torch.int32)
    return t.contiguous()


def _float(t, dev, what, shape):
    import torch
    if t.dtype is torch.float32 and t.shape == shape and t.device == dev:
        return t.contiguous()
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
