"""Binding of the products grouped by expert and of the microscaled 4-bit values.

As in the package itself, argument checks and marshalling only; the work runs
in the HIP kernels of ``libmoeffn.so`` and PyTorch supplies memory and streams.
Everything is enqueued on ``stream`` (default: the current stream of the
tensors' device); outputs that the caller does not give are allocated for that
stream.

Autograd does not see these calls.  Where it is on, an input that waits for a gradient
is refused: a training step calls them under torch.no_grad() or inside a
torch.autograd.Function, with grouped_matmul(dy, w, transpose=True) and grouped_matmul_dw
as the backward of grouped_matmul.
"""

from __future__ import annotations

import ctypes

from . import layer as _layer
from .layer import MOE_T_BF16, MOE_T_FP32, _call, _device, _output, _on, _rows, _type

__all__ = ["MoeGrouped", "MoeGroupedGrad", "MoeMx", "grouped_matmul", "grouped_matmul_dw", "grouped_dw_workspace_bytes",
           "mx_quantize", "mx_dequantize", "MOE_T_MXFP4", "MOE_G_W_KN", "MOE_Q_GELU", "MOE_Q_SILU"]

MOE_T_MXFP4 = 2
MOE_G_W_KN = 1
MOE_Q_GELU, MOE_Q_SILU = 1, 2


class MoeGrouped(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("A", "E", "N", "K", "x_type", "w_type", "out_type")] + \
               [("flags", ctypes.c_uint32)] + \
               [(n, ctypes.c_void_p) for n in ("offsets", "x", "w", "x_scales", "w_scales", "out")] + \
               [(n, ctypes.c_int64) for n in ("x_stride", "w_stride", "w_expert_stride", "out_stride")]


class MoeGroupedGrad(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("A", "E", "N", "K", "out_type")] + \
               [(n, ctypes.c_void_p) for n in ("offsets", "dy", "x", "dw")] + \
               [(n, ctypes.c_int64) for n in ("dy_stride", "x_stride")]


class MoeMx(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int64), ("K", ctypes.c_int32), ("type", ctypes.c_int32), ("flags", ctypes.c_uint32)] + \
               [(n, ctypes.c_void_p) for n in ("values", "codes", "scales")] + [("stride", ctypes.c_int64)]


def _no_autograd(*tensors):
    for t, name in tensors:
        if t.requires_grad and _layer.torch.is_grad_enabled():
            raise ValueError(f"{name} waits for a gradient, which this call would not pass on: use torch.no_grad(), detach() or a "
                             "torch.autograd.Function")


def _bytes(t, name, dev, shape, other):
    """Data pointer of contiguous codes or scales: uint8, or the type `other` of torch that holds the same bytes."""
    _on(t, name, dev)
    dtype = t.dtype
    if dtype is not _layer.torch.uint8 and dtype is not getattr(_layer.torch, other, None):
        raise ValueError(f"{name} must be uint8 or {other}, got {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _codes(t, name, dev, shape):
    return _bytes(t, name, dev, shape, "float4_e2m1fn_x2")


def _scales(t, name, dev, shape):
    return _bytes(t, name, dev, shape, "float8_e8m0fnu")


def _bf16(t, name):
    if t.dtype is not _layer.torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")


def _offsets(t, dev, E):
    _on(t, "offsets", dev)
    if t.dtype is not _layer.torch.int32 or t.shape != (E + 1,) or not t.is_contiguous():
        raise ValueError(f"offsets must be a contiguous int32 tensor of shape {(E + 1,)}, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _rows_count(n, name):
    if n >= 2**30:
        raise ValueError(f"{name} has {n} rows, more than a call takes (2^30 - 1)")


def _out_type(out, out_dtype):
    if out is None:
        dtype = _layer.torch.bfloat16 if out_dtype is None else out_dtype
    else:
        dtype = out.dtype
        if out_dtype is not None and out_dtype is not dtype:
            raise ValueError(f"out is {dtype}, out_dtype {out_dtype}")
    if dtype is not _layer.torch.bfloat16 and dtype is not _layer.torch.float32:
        raise ValueError(f"the output must be bfloat16 or float32, got {dtype}")
    return dtype, MOE_T_FP32 if dtype is _layer.torch.float32 else MOE_T_BF16


def grouped_matmul(x, w, offsets=None, *, x_scales=None, w_scales=None, transpose=False, out=None, out_dtype=None,
                   stream=None):
    """Products grouped by expert: the rows of x are sorted by expert, expert e has the
    rows offsets[e] .. offsets[e + 1] - 1 (int32 [E + 1], as sort_build_tiles makes them).

        out[r, n] = sum_k x[r, k] w[e, n, k]       w [E, N, K]
                  = sum_k x[r, k] w[e, k, n]       w [E, K, N], with transpose=True

    transpose=True gives the gradient of the rows: with the forward's w [E, N, K] and
    dy [A, N], dx = grouped_matmul(dy, w, offsets, transpose=True).  Without offsets w is
    one matrix for all rows ([N, K] or [1, N, K]).  N and K are multiples of 8.

    x [A, K] and w are bf16; rows of both may be strided.  Or w is microscaled: codes
    [E, N, K / 2] with w_scales [E, N, K / 32] (mx_quantize of the weights, K a multiple of
    32), and x bf16, or microscaled too with x_scales.  Products are exact, sums fp32.

    out [A, N] is bf16 or fp32 (`out`, whose rows share no memory with an input, else allocated
    in out_dtype, bf16 by default).  Rows that belong to no expert are not written.  Returns
    out."""
    bgq = _layer._api()
    if x.requires_grad or w.requires_grad:
        _no_autograd((x, "x"), (w, "w"))
    dev = _device(x, "x")
    xshape, shape = tuple(x.shape), tuple(w.shape)
    if len(xshape) != 2:
        raise ValueError(f"x has shape {xshape}, expected [A, K]")
    if len(shape) != 3 and (len(shape) != 2 or offsets is not None):
        raise ValueError(f"w has shape {shape}, expected {'[E, N, K]' if offsets is not None else '[N, K]'}")
    if len(shape) == 2:
        w, shape = w.unsqueeze(0), (1,) + shape
        w_scales = None if w_scales is None else w_scales.unsqueeze(0)
    (E, N, K), A = shape, xshape[0]
    if offsets is None and E != 1:
        raise ValueError(f"w holds {E} experts: offsets are needed")
    _rows_count(A, "x")
    dtype, out_type = _out_type(out, out_dtype)
    w_type = x_type = MOE_T_BF16
    flags = w_stride = w_expert = x_stride = 0
    ws = xs = None
    if w_scales is not None:
        if transpose:
            raise ValueError("microscaled weights cannot be transposed: their scales lie along K")
        K, w_type = 2 * K, MOE_T_MXFP4
        wp, ws = _codes(w, "w", dev, shape), _scales(w_scales, "w_scales", dev, (E, N, K // 32))
    else:
        _on(w, "w", dev)
        _bf16(w, "w")
        w_expert, w_stride, one = w.stride()
        if one != 1 and K > 1:
            raise ValueError("w must be contiguous along its rows")
        if N == 1:
            w_stride = K
        if E == 1:
            w_expert = 0
        if transpose:
            N, K, flags = K, N, MOE_G_W_KN
        wp = w.data_ptr()
    if x_scales is not None:
        if w_scales is None:
            raise ValueError("x_scales are given without w_scales")
        x_type = MOE_T_MXFP4
        xp, xs = _codes(x, "x", dev, (A, K // 2)), _scales(x_scales, "x_scales", dev, (A, K // 32))
    else:
        _bf16(x, "x")
        x_stride, xp = _rows(x, "x", dev, A, K), x.data_ptr()
    op = None if offsets is None else _offsets(offsets, dev, E)

    def go(raw):
        if out is None:
            o, stride = _layer.torch.empty(A, N, dtype=dtype, device=dev), N
        else:
            o, stride = out, _rows(out, "out", dev, A, N)
        g = MoeGrouped(A, E, N, K, x_type, w_type, out_type, flags, op, xp, wp, xs, ws, o.data_ptr(), x_stride, w_stride, w_expert, stride)
        st = bgq.lib().moe_grouped_matmul(ctypes.byref(g), raw)
        if st != 0:
            raise bgq.MoeError(st, "moe_grouped_matmul")
        return o

    return _call(dev, stream, go)


def grouped_dw_workspace_bytes(A, E, N, K):
    """Bytes of device workspace that grouped_matmul_dw needs for A rows (0: none)."""
    g = MoeGroupedGrad(A=A, E=E, N=N, K=K)
    return int(_layer._api().lib().moe_grouped_dw_workspace_bytes(ctypes.byref(g)))


def grouped_matmul_dw(dy, x, offsets=None, *, out=None, out_dtype=None, workspace=None, stream=None):
    """Gradient of the weights of grouped_matmul: out[e, n, k] = sum over the rows r of
    expert e of dy[r, n] x[r, k], zeros for an expert without rows.

    dy [A, N] and x [A, K] bf16 (rows may be strided), offsets int32 [E + 1]; without
    offsets all rows are one expert's.  N and K are multiples of 8.  Products are exact,
    sums fp32.  out [E, N, K] is bf16 or fp32 (`out`, contiguous and on memory of its own,
    else allocated in out_dtype, bf16 by default).  workspace: a uint8 tensor of grouped_dw_workspace_bytes(A,
    E, N, K) bytes, one per call at a time (allocated if None).  Returns out."""
    bgq = _layer._api()
    if dy.requires_grad or x.requires_grad:
        _no_autograd((dy, "dy"), (x, "x"))
    dev = _device(dy, "dy")
    shape, xshape = tuple(dy.shape), tuple(x.shape)
    if len(shape) != 2 or len(xshape) != 2:
        raise ValueError(f"dy and x must be [A, N] and [A, K], got {shape} and {xshape}")
    (A, N), K = shape, xshape[1]
    _rows_count(A, "dy")
    E = 1 if offsets is None else offsets.numel() - 1
    dtype, out_type = _out_type(out, out_dtype)
    _bf16(dy, "dy")
    _bf16(x, "x")
    dy_stride, x_stride = _rows(dy, "dy", dev, A, N), _rows(x, "x", dev, A, K)
    op = None if offsets is None else _offsets(offsets, dev, E)
    g = MoeGroupedGrad(A, E, N, K, out_type, op, dy.data_ptr(), x.data_ptr(), None, dy_stride, x_stride)

    def go(raw):
        if out is None:
            o = _layer.torch.empty(E, N, K, dtype=dtype, device=dev)
            g.dw = o.data_ptr()
        else:
            o, g.dw = out, _output(out, "out", dev, (E, N, K), dtype)
        ws = workspace
        if ws is None:
            need = bgq.lib().moe_grouped_dw_workspace_bytes(ctypes.byref(g))
            if need:
                ws = _layer.torch.empty(need, dtype=_layer.torch.uint8, device=dev)
        else:
            _on(ws, "workspace", dev)
            if ws.dtype is not _layer.torch.uint8 or not ws.is_contiguous():
                raise ValueError("workspace must be a contiguous uint8 tensor")
        st = bgq.lib().moe_grouped_matmul_dw(ctypes.byref(g), None if ws is None else ws.data_ptr(),
                                             0 if ws is None else ws.numel(), raw)
        if st != 0:
            raise bgq.MoeError(st, "moe_grouped_matmul_dw")
        return o

    return _call(dev, stream, go)


def _flat_rows(t, name, shape, width):
    """(rows, row stride) of a tensor of that shape whose last dimension is `width`: strided in two dimensions,
    contiguous in more."""
    rows = shape[0]
    if len(shape) == 2:
        row, one = t.stride()
        if one != 1 and width > 1:
            raise ValueError(f"{name} must be contiguous along its rows")
        return rows, row if rows > 1 else max(width, 1)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (or two-dimensional with contiguous rows)")
    for n in shape[1:-1]:
        rows *= n
    return rows, width


_GLU = {None: 0, "gelu": MOE_Q_GELU, "silu": MOE_Q_SILU}


def mx_quantize(x, *, glu=None, codes=None, scales=None, stream=None):
    """Microscaled 4-bit values of x [..., K], bf16 or fp32, in blocks of 32 along K (a
    multiple of 32):

        s    = floor(log2(max |v|)) - 2, at least -127, held as the byte s + 127
        code = v / 2^s as 1 sign, 2 exponent and 1 mantissa bit (0, 0.5, 1, 1.5, 2, 3, 4, 6),
               to nearest, ties to the even code, larger ones as 6; the first of two in the
               low half of a byte

    A block with a NaN or an infinity gets the byte 255 (all of it stands for NaN).  With
    glu="gelu" or "silu" a row of x holds 2 K values [g | u] and v = act(g) u, the product
    between an expert FFN's two matmuls; else v = x.  x may have strided rows in two
    dimensions.  Returns (codes uint8 [..., K / 2], scales uint8 [..., K / 32]), as
    grouped_matmul takes them (`codes` and `scales` if given, on none of x's memory)."""
    bgq = _layer._api()
    if x.requires_grad:
        _no_autograd((x, "x"))
    dev = _device(x, "x")
    shape = tuple(x.shape)
    if len(shape) < 2:
        raise ValueError(f"x has shape {shape}, expected [..., K]")
    if glu not in _GLU:
        raise ValueError(f"glu must be None, 'gelu' or 'silu', got {glu!r}")
    width = shape[-1]
    if width % (32 if glu is None else 64):
        raise ValueError(f"x has {width} values a row, expected a multiple of {32 if glu is None else 64}")
    K = width if glu is None else width // 2
    rows, stride = _flat_rows(x, "x", shape, width)
    q = MoeMx(rows, K, _type(x, "x"), _GLU[glu], x.data_ptr(), None, None, stride)
    lead = shape[:-1]
    uint8 = _layer.torch.uint8

    def go(raw):
        c, s = codes, scales
        if c is None:
            c = _layer.torch.empty(*lead, K // 2, dtype=uint8, device=dev)
            q.codes = c.data_ptr()
        else:
            q.codes = _codes(c, "codes", dev, lead + (K // 2,))
        if s is None:
            s = _layer.torch.empty(*lead, K // 32, dtype=uint8, device=dev)
            q.scales = s.data_ptr()
        else:
            q.scales = _scales(s, "scales", dev, lead + (K // 32,))
        st = bgq.lib().moe_mx_quantize(ctypes.byref(q), raw)
        if st != 0:
            raise bgq.MoeError(st, "moe_mx_quantize")
        return c, s

    return _call(dev, stream, go)


def mx_dequantize(codes, scales, *, out=None, out_dtype=None, stream=None):
    """The values [..., K] that microscaled codes [..., K / 2] and scales [..., K / 32] stand
    for, bf16 or fp32 (`out`, on memory of its own, else allocated in out_dtype, bf16 by default;
    both hold them exactly)."""
    bgq = _layer._api()
    dev = _device(codes, "codes")
    shape = tuple(codes.shape)
    if len(shape) < 2:
        raise ValueError(f"codes have shape {shape}, expected [..., K / 2]")
    lead, K = shape[:-1], 2 * shape[-1]
    dtype, kind = _out_type(out, out_dtype)
    q = MoeMx(0, K, kind, 0, None, _codes(codes, "codes", dev, shape), _scales(scales, "scales", dev, lead + (K // 32,)), 0)

    def go(raw):
        o = out
        if o is None:
            o = _layer.torch.empty(*lead, K, dtype=dtype, device=dev)
            q.R, q.stride = o.numel() // max(K, 1), K
        else:
            _on(o, "out", dev)
            if o.shape != lead + (K,):
                raise ValueError(f"out has shape {tuple(o.shape)}, expected {lead + (K,)}")
            q.R, q.stride = _flat_rows(o, "out", lead + (K,), K)
        q.values = o.data_ptr()
        st = bgq.lib().moe_mx_dequantize(ctypes.byref(q), raw)
        if st != 0:
            raise bgq.MoeError(st, "moe_mx_dequantize")
        return o

    return _call(dev, stream, go)
