"""Binding of the operators around the expert FFN: the block norms, the router
and the whole layer.

As in the package itself, argument checks and marshalling only; the work runs
in the HIP kernels of ``libmoeffn.so`` and PyTorch supplies memory and streams.
Everything is enqueued on ``stream`` (default: the current stream of the
tensors' device); outputs that the caller does not give are allocated for that
stream.
"""

from __future__ import annotations

import contextlib
import ctypes

__all__ = ["MoeNorm", "MoeRouter", "MoeLayerDesc", "MoeLayer", "block_norm", "router_forward", "MOE_R_NORM", "MOE_T_BF16", "MOE_T_FP32", "MOE_N_POST", "NORM_MAX_H"]

MOE_T_BF16, MOE_T_FP32 = 0, 1
MOE_N_POST = 1
MOE_R_NORM = 1
NORM_MAX_H = 16384


class MoeNorm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "H", "y_type", "stream_type", "normed_type", "weight_type", "gate_type")] + \
               [("flags", ctypes.c_uint32)] + \
               [(n, ctypes.c_float) for n in ("eps", "residual_scale", "gate_scale", "weight_offset")] + \
               [(n, ctypes.c_void_p) for n in
                ("residual", "post_weight", "gate", "pre_weight", "out", "normed")] + \
               [(n, ctypes.c_int64) for n in
                ("y_stride", "residual_stride", "out_stride", "normed_stride", "gate_stride_t", "gate_stride_h")]


class MoeRouter(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "E", "k", "weight_type")] + \
               [("flags", ctypes.c_uint32), ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("expert_scale", ctypes.c_void_p)]


# The package, which imports this module, and torch, which it does without until a
# tensor is there: imported by the first call (_api).  Import statements in the
# functions cost a call 0.3 us.
_package = torch = None


def _api():
    global _package, torch
    if _package is None:
        import torch as t
        import bit_gathered_quantized_amd as bgq
        torch, _package = t, bgq
    return _package


def _type(t, name):
    if t.dtype is torch.bfloat16:
        return MOE_T_BF16
    if t.dtype is torch.float32:
        return MOE_T_FP32
    raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _on(t, name, dev):
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    return t.device


def _rows(t, name, dev, T, H):
    """Row stride of a [T, H] tensor whose rows are contiguous."""
    _on(t, name, dev)
    if t.shape != (T, H):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(T, H)}")
    st, sh = t.stride()
    if sh != 1 and H > 1:
        raise ValueError(f"{name} must be contiguous along its rows")
    return st if T > 1 else max(H, 1)


def _vector(t, name, dev, n):
    _on(t, name, dev)
    if t.shape != (n,):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(n,)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _like(t):
    """A new contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


@contextlib.contextmanager
def _ambient(dev, stream):
    """Makes the tensors' device, and the stream if one is given, current."""
    with contextlib.ExitStack() as stack:
        if dev.index != torch.cuda.current_device():
            stack.enter_context(torch.cuda.device(dev))
        if stream is not None:
            if stream.device != dev:
                raise ValueError(f"stream belongs to {stream.device}, the tensors are on {dev}")
            stack.enter_context(torch.cuda.stream(stream))
        yield


def _call(dev, stream, f):
    """f(raw stream) with the device and stream current; no context in the usual case."""
    if stream is None and dev.index == torch._C._cuda_getDevice():  # current_device() without its check: a tensor is there
        return f(torch._C._cuda_getCurrentRawStream(dev.index))  # current_stream() without its object
    with _ambient(dev, stream):
        return f(torch.cuda.current_stream(dev).cuda_stream)


def _gate(n, gate, dev, T, H):
    """Fills a MoeNorm's gate from a number or a tensor that broadcasts to [T, H]."""
    if not hasattr(gate, "data_ptr"):  # a number of any type
        n.gate_scale = float(gate)
        return
    _on(gate, "gate", dev)
    n.gate_type = _type(gate, "gate")
    if gate.shape == (H,):
        st, (sh,) = 0, gate.stride()
    else:
        try:
            st, sh = gate.expand(T, H).stride()
        except RuntimeError:
            raise ValueError(f"gate has shape {tuple(gate.shape)}, which does not broadcast to {(T, H)}") from None
    if H == 1:
        sh = 0
    if sh not in (0, 1):
        raise ValueError("gate must be contiguous or broadcast along H")
    n.gate, n.gate_stride_t, n.gate_stride_h = gate.data_ptr(), st if T > 1 else 0, sh


def _norm_tail(n, T, H, dev, residual, post_norm, post_weight, gate, residual_scale, pre_norm, pre_weight,
               weight_offset, eps):
    """Fills everything of a MoeNorm but its outputs and y; returns the normed flag."""
    n.T, n.H, n.eps, n.residual_scale, n.weight_offset = T, H, eps, residual_scale, weight_offset
    n.gate_scale = 1.0
    if residual is not None:
        n.stream_type = _type(residual, "residual")
        n.residual_stride, n.residual = _rows(residual, "residual", dev, T, H), residual.data_ptr()
    if post_norm or post_weight is not None:
        n.flags = MOE_N_POST
    for name, w in (("post_weight", post_weight), ("pre_weight", pre_weight)):
        if w is not None:
            n.weight_type = _type(w, name)
            setattr(n, name, _vector(w, name, dev, H))
    if post_weight is not None and pre_weight is not None and post_weight.dtype != pre_weight.dtype:
        raise ValueError("post_weight and pre_weight must have the same type")
    if gate is not None:
        _gate(n, gate, dev, T, H)
    return pre_norm or pre_weight is not None


def block_norm(y, residual=None, *, post_norm=False, post_weight=None, gate=None, residual_scale=1.0,
               pre_norm=False, pre_weight=None, weight_offset=0.0, eps=1e-6, out=None, normed=None, want_out=True,
               stream=None):
    """Norms around a block, fused with its gate and the residual scale, in one pass:

        z      = gate * (rms(y) * (weight_offset + post_weight))     (post_norm or post_weight given)
               = gate * y                                            (neither)
        out    = residual_scale * residual + z
        normed = rms(out) * (weight_offset + pre_weight)             (pre_norm or pre_weight given)

    y [T, H] is the block's output, `out` the next residual stream, `normed` the
    next block's input; rms(v) = v / sqrt(mean(v^2) + eps).  y, residual, out,
    normed, gate and the weights are bf16 or fp32 (residual and out alike, both
    weights alike); rows may be strided.  gate is a number or a tensor that
    broadcasts to [T, H] ([H], [T, 1], ...); weights are [H], None for ones.
    `out` and `normed` are allocated in the residual's type (y's without one)
    unless given, and may be y or residual themselves (but not the same one).
    want_out=False skips `out`: a plain norm of y.

    Returns out, (out, normed) with a norm after the block, or normed alone
    with want_out=False."""
    bgq = _api()
    dev = _device(y, "y")
    if y.dim() != 2:
        raise ValueError(f"y has shape {tuple(y.shape)}, expected [T, H]")
    T, H = y.shape
    if T > 2**31 - 1:
        raise ValueError(f"y has {T} rows, more than a call takes (2^31 - 1)")
    n = MoeNorm()
    n.y_type = _type(y, "y")
    n.y_stride = _rows(y, "y", dev, T, H)
    n.stream_type = n.y_type
    with_normed = _norm_tail(n, T, H, dev, residual, post_norm, post_weight, gate, residual_scale, pre_norm,
                             pre_weight, weight_offset, eps)
    if not with_normed and normed is not None:
        raise ValueError("normed is given without pre_norm or pre_weight")
    if not want_out and (not with_normed or out is not None):
        raise ValueError("want_out=False takes no out and needs pre_norm or pre_weight")
    dtype = y.dtype if residual is None else residual.dtype
    if out is not None and residual is None:
        n.stream_type = _type(out, "out")
    elif out is not None and out.dtype != dtype:
        raise ValueError(f"out must have the residual's type {dtype}, got {out.dtype}")

    def go(raw):
        o, m = out, normed
        if want_out:
            if o is None:
                o = _like(y if residual is None else residual)
                n.out_stride = H
            else:
                n.out_stride = _rows(o, "out", dev, T, H)
            n.out = o.data_ptr()
        if with_normed:
            if m is None:
                m = _like(y if residual is None else residual)
                n.normed_type, n.normed_stride = _type(m, "normed"), H
            else:
                n.normed_type, n.normed_stride = _type(m, "normed"), _rows(m, "normed", dev, T, H)
            n.normed = m.data_ptr()
        st = bgq.lib().moe_block_norm(ctypes.byref(n), y.data_ptr(), raw)
        if st != 0:
            raise bgq.MoeError(st, "moe_block_norm")
        return (o, m) if want_out and with_normed else o if want_out else m

    return _call(dev, stream, go)


def _output(t, name, dev, shape, dtype):
    """Data pointer of a given contiguous output."""
    _on(t, name, dev)
    if tuple(t.shape) != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")
    return t.data_ptr()


def _new_or_given(t, name, dev, shape, dtype):
    """The output, allocated unless given, and its data pointer."""
    if t is not None:
        return t, _output(t, name, dev, shape, dtype)
    t = torch.empty(shape, dtype=dtype, device=dev)
    return t, t.data_ptr()


def router_forward(x, weight, k, *, norm=True, eps=1e-6, expert_scale=None, logits=None, ids=None, weights=None,
                   stream=None):
    """The whole router: norm, product and top-k.

        logits[t, e] = rstd_t * sum_c x[t, c] weight[e, c],   rstd_t = 1 / sqrt(mean(x_t^2) + eps)  (1 without norm)

    x bf16 [T, H] (rows may be strided), weight [E, H] bf16 or fp32 with a norm's
    weight or a router's scale already multiplied into its columns; H a multiple
    of 64.  ids int32 [T, k] are the k largest logits in descending order (the
    lower id first on ties), weights fp32 [T, k] their softmax, times
    expert_scale[id] if given (fp32 [E]).  Products of x are exact and sums fp32
    whichever type the weight has.  Returns (logits fp32 [T, E], ids, weights)."""
    bgq = _api()
    dev = _device(x, "x")
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError(f"x and weight must be [T, H] and [E, H], got {tuple(x.shape)} and {tuple(weight.shape)}")
    T, H = x.shape
    E = weight.shape[0]
    if x.dtype is not torch.bfloat16:
        raise ValueError(f"x must be bfloat16, got {x.dtype}")
    r = MoeRouter()
    r.T, r.H, r.E, r.k, r.eps, r.flags = T, H, E, k, eps, MOE_R_NORM if norm else 0
    r.x_stride = _rows(x, "x", dev, T, H)
    r.weight_type = _type(weight, "weight")
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    _rows(weight, "weight", dev, E, H)
    r.weight = weight.data_ptr()
    if expert_scale is not None:
        if expert_scale.dtype is not torch.float32:
            raise ValueError(f"expert_scale must be float32, got {expert_scale.dtype}")
        r.expert_scale = _vector(expert_scale, "expert_scale", dev, E)
    if not 1 <= k <= E:
        raise ValueError(f"k must be between 1 and the number of experts {E}, got {k}")

    def go(raw):
        lo, plo = _new_or_given(logits, "logits", dev, (T, E), torch.float32)
        i, pi = _new_or_given(ids, "ids", dev, (T, k), torch.int32)
        w, pw = _new_or_given(weights, "weights", dev, (T, k), torch.float32)
        st = bgq.lib().moe_router_forward(ctypes.byref(r), x.data_ptr(), plo, pi, pw, raw)
        if st != 0:
            raise bgq.MoeError(st, "moe_router_forward")
        return lo, i, w

    return _call(dev, stream, go)


class MoeLayerDesc(ctypes.Structure):
    _fields_ = [("flags", ctypes.c_uint32), ("router_flags", ctypes.c_uint32), ("norm_type", ctypes.c_int32),
                ("router_type", ctypes.c_int32), ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float)] + \
               [(n, ctypes.c_void_p) for n in
                ("norm_weight", "router_weight", "expert_scale", "w_gateup", "s_gateup", "b_gateup", "w_down",
                 "s_down", "b_down", "topk_ids", "topk_weights")]


class MoeLayer:
    """A whole mixture-of-experts layer over fixed weights:

        n   = rms(x) * (weight_offset + norm_weight)             (norm=False: n = x)
        ids, w = router_forward(x, router_weight, k, norm=router_norm, expert_scale=...)
        y   = sum_j w_j FFN of expert ids_j on n                 (expert_ffn_forward)
        out, normed = block_norm(y, residual, post_weight=..., gate=..., pre_weight=..., ...)

    Weights as for router_forward and expert_ffn_forward; norm_weight, post_weight
    and pre_weight are [H] in bf16 or fp32 (post and pre alike; pre_norm=True or
    post_norm=True without a weight norms by ones).  The handle checks them once and
    keeps their memory alive, so a parameter that is moved or converted later needs a
    new handle; it holds no other state, so calls on several streams are
    independent as long as each has a workspace of its own.

    Calls of up to 16 tokens take two launches and keep n and h to 16 significant
    bits.  Larger ones run the operators in turn, with n in bf16 and h in bf16, or in
    fp32 with fp32_intermediate.  So a token's output differs within these roundings
    with the size of its batch."""

    def __init__(self, router_weight, k, w_gateup, s_gateup, b_gateup, w_down, s_down, b_down, *, norm=True,
                 norm_weight=None, router_norm=True, expert_scale=None, post_norm=False, post_weight=None,
                 pre_norm=False, pre_weight=None, weight_offset=0.0, swiglu=False, fp32_intermediate=False, eps=1e-6):
        bgq = _api()
        dev = self.device = _device(router_weight, "router_weight")
        if router_weight.dim() != 2 or not router_weight.is_contiguous():
            raise ValueError("router_weight must be a contiguous [E, H] tensor")
        E, H = router_weight.shape
        if w_gateup.dim() != 3 or w_gateup.shape[0] != E or w_gateup.shape[1] % 2:
            raise ValueError(f"w_gateup has shape {tuple(w_gateup.shape)}, expected ({E}, 2 I, words)")
        I = w_gateup.shape[1] // 2
        bits = w_gateup.shape[2] * 32 // H
        if bits not in (4, 8) or w_gateup.shape[2] * 32 != bits * H:
            raise ValueError(f"w_gateup has {w_gateup.shape[2]} words per row: neither 4-bit nor 8-bit codes of H={H}")
        ng = s_gateup.shape[-1]
        if ng < 1 or H % ng:
            raise ValueError(f"s_gateup has {ng} groups per row, which does not divide H={H}")
        gs = H // ng
        if not 1 <= k <= min(E, 64):
            raise ValueError(f"k must be between 1 and min(E, 64) = {min(E, 64)}, got {k}")
        d = self._desc = MoeLayerDesc()
        for name, t, size, shape in (("w_gateup", w_gateup, 4, (E, 2 * I, H * bits // 32)),
                                     ("s_gateup", s_gateup, 2, (E, 2 * I, ng)), ("b_gateup", b_gateup, 2, (E, 2 * I, ng)),
                                     ("w_down", w_down, 4, (E, H, I * bits // 32)),
                                     ("s_down", s_down, 2, (E, H, I // gs)), ("b_down", b_down, 2, (E, H, I // gs))):
            _on(t, name, dev)
            if t.dtype is torch.float16:
                raise ValueError(f"{name} must hold bfloat16 values (or their bits in 2-byte integers), got {t.dtype}")
            setattr(d, name, bgq._dev_ptr(t, name, size, shape).value)
        d.flags = 1 if norm else 0
        d.router_flags = MOE_R_NORM if router_norm else 0
        d.eps, d.weight_offset = eps, weight_offset
        d.router_weight, d.router_type = router_weight.data_ptr(), _type(router_weight, "router_weight")
        if norm_weight is not None:
            if not norm:
                raise ValueError("norm_weight is given with norm=False")
            d.norm_weight, d.norm_type = _vector(norm_weight, "norm_weight", dev, H), _type(norm_weight, "norm_weight")
        if expert_scale is not None:
            if expert_scale.dtype is not torch.float32:
                raise ValueError(f"expert_scale must be float32, got {expert_scale.dtype}")
            d.expert_scale = _vector(expert_scale, "expert_scale", dev, E)
        self.E, self.H, self.I, self.k, self.group_size, self.bits = E, H, I, k, gs, bits
        self.eps, self.weight_offset = eps, weight_offset
        self._tail = MoeNorm()
        self._pre = _norm_tail(self._tail, 0, H, dev, None, post_norm, post_weight, None, 1.0, pre_norm, pre_weight,
                               weight_offset, eps)
        self._flags = (bgq.MOE_F_SWIGLU if swiglu else 0) | (bgq.MOE_F_FP32_INTERMEDIATE if fp32_intermediate else 0)
        for desc, names in ((d, ("router_weight", "norm_weight", "w_gateup", "s_gateup", "b_gateup", "w_down", "s_down",
                                 "b_down")), (self._tail, ("post_weight", "pre_weight"))):
            for name in names:
                if (getattr(desc, name) or 0) % 16:
                    raise ValueError(f"{name} must start on 16 bytes")
        # detached: tensors of their own on the same memory.  A module's .to() or an
        # assignment to .data gives a parameter other memory under the same object.
        self._keep = tuple(None if t is None else t.detach() for t in (
            router_weight, w_gateup, s_gateup, b_gateup, w_down, s_down, b_down, norm_weight, expert_scale, post_weight,
            pre_weight))
        if self.workspace_bytes(1) == 0:
            raise ValueError(f"unsupported layer: E={E}, H={H}, I={I}, k={k}, group size {gs}, {bits} bits")

    def _problem(self, T):
        return _api().problem(T, self.k, self.E, self.H, self.I, self._flags, group_size=self.group_size, bits=self.bits)

    def workspace_bytes(self, T):
        """Bytes of device workspace a call on T tokens, or fewer, needs (0: unsupported)."""
        return int(_api().lib().moe_layer_workspace_bytes(ctypes.byref(self._problem(T))))

    def __call__(self, x, *, residual=None, gate=None, residual_scale=1.0, out=None, normed=None, ids=None, weights=None,
                 workspace=None, stream=None):
        """The layer on x bf16 [T, H].  residual, gate and residual_scale as for
        block_norm (rows of residual, out, normed and a [T, H] gate start on 16
        bytes); out and normed default to the residual's type (x's without one), and one
        of them may be x or the residual itself.  ids (int32) and weights (fp32),
        [T, k], receive the routing if given.  workspace: a uint8 tensor of
        workspace_bytes(T) bytes, one per call at a time (allocated if None).  Returns
        out, or (out, normed) if the layer norms its output."""
        bgq = _api()
        dev, H, k = self.device, self.H, self.k
        if x.dim() != 2 or x.shape[1] != H or x.dtype is not torch.bfloat16 or not x.is_contiguous():
            raise ValueError(f"x must be a contiguous bfloat16 [T, {H}] tensor")
        _on(x, "x", dev)
        T = x.shape[0]
        p = self._problem(T)
        n = MoeNorm.from_buffer_copy(self._tail)
        n.T = T
        dtype = x.dtype if residual is None else residual.dtype
        n.residual_scale = residual_scale
        if residual is not None:
            n.stream_type = _type(residual, "residual")
            n.residual_stride, n.residual = _rows(residual, "residual", dev, T, H), residual.data_ptr()
        elif out is not None:
            n.stream_type, dtype = _type(out, "out"), out.dtype
        if out is not None and out.dtype is not dtype:
            raise ValueError(f"out must have the residual's type {dtype}, got {out.dtype}")
        if gate is not None:
            _gate(n, gate, dev, T, H)
        if normed is not None and not self._pre:
            raise ValueError("normed is given, but the layer has no norm after it")
        desc = self._desc
        if ids is not None or weights is not None:
            desc = MoeLayerDesc.from_buffer_copy(desc)
            if ids is not None:
                desc.topk_ids = _output(ids, "ids", dev, (T, k), torch.int32)
            if weights is not None:
                desc.topk_weights = _output(weights, "weights", dev, (T, k), torch.float32)

        def go(raw):
            o, m, ws = out, normed, workspace
            if o is None:
                o = _like(x if residual is None else residual)
                n.out_stride = H
            else:
                n.out_stride = _rows(o, "out", dev, T, H)
            n.out = o.data_ptr()
            if self._pre:
                if m is None:
                    m = _like(out if out is not None else x if residual is None else residual)
                    n.normed_type, n.normed_stride = _type(m, "normed"), H
                else:
                    n.normed_type, n.normed_stride = _type(m, "normed"), _rows(m, "normed", dev, T, H)
                n.normed = m.data_ptr()
            if ws is None:
                need = bgq.lib().moe_layer_workspace_bytes(ctypes.byref(p))
                ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
            else:
                _on(ws, "workspace", dev)
                if ws.dtype is not torch.uint8 or not ws.is_contiguous():
                    raise ValueError("workspace must be a contiguous uint8 tensor")
            st = bgq.lib().moe_layer_forward(ctypes.byref(p), ctypes.byref(desc), x.data_ptr(), ctypes.byref(n),
                                             ws.data_ptr(), ws.numel(), raw)
            if st != 0:
                raise bgq.MoeError(st, "moe_layer_forward")
            return (o, m) if self._pre else o

        return _call(dev, stream, go)
