"""The operators around and beside the KDA recurrence (``include/kda_layer.h``):
RMS normalisation with the residual's addition (bf16 or e4m3 output), the short
causal convolution and the selective state-space scan, each with its gradient,
and with a single-token step where generation has one.

As for the recurrence, the functions only marshal arguments: they check types,
devices and shapes, allocate outputs and workspaces that the caller does not
pass, and call libkda on torch's current HIP stream of the inputs' device.
Activations are bf16; they may be slices of wider tensors (only their last
dimensions have to be contiguous; the scan's x, B, C and d_out also have to begin
at multiples of 16 bytes, with strides that are multiples of 8 elements).  Tensors
that a call writes are contiguous.

``rms_norm``, ``short_conv`` and ``ssm_scan`` differentiate once.  To capture
their backward into a HIP graph, let no autograd graph of the same leaves from
before the capture live (delete the outputs and losses of the warm-up first):
torch ends such a capture with an error, or ends the process.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

_P = ctypes.c_void_p
_I = ctypes.c_int64
_BF16, _FP32 = 1, 2
_STATE_DTYPES = {torch.bfloat16: _BF16, torch.float32: _FP32}
_FP32_ONLY = {torch.float32: _FP32}
_INT64_ONLY = {torch.int64: 0}


class KdaRmsnormDesc(ctypes.Structure):
    _fields_ = [("rows", _I), ("D", _I), ("x_stride", _I), ("residual_stride", _I),
                ("residual_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("group", _I), ("d_out_stride", _I), ("d_residual_stride", _I), ("workspace", _P),
                ("workspace_bytes", ctypes.c_size_t)]


class KdaConvDesc(ctypes.Structure):
    _fields_ = [("B", _I), ("T", _I), ("D", _I), ("W", _I), ("num_seqs", _I), ("x_stride_b", _I), ("x_stride_t", _I),
                ("d_out_stride_b", _I), ("d_out_stride_t", _I), ("silu", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("initial_state_dtype", ctypes.c_int32),
                ("final_state_dtype", ctypes.c_int32), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class KdaSsmDesc(ctypes.Structure):
    _fields_ = [("B", _I), ("T", _I), ("H", _I), ("P", _I), ("G", _I), ("N", _I), ("num_seqs", _I),
                ("x_stride_b", _I), ("x_stride_t", _I), ("dt_stride_b", _I), ("dt_stride_t", _I),
                ("b_stride_b", _I), ("b_stride_t", _I), ("c_stride_b", _I), ("c_stride_t", _I),
                ("d_out_stride_b", _I), ("d_out_stride_t", _I), ("initial_state_dtype", ctypes.c_int32),
                ("final_state_dtype", ctypes.c_int32), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t),
                ("piece_chunks", _I), ("launch_piece", _I)]


def _declare(lib) -> None:
    """Argument types of the layer operators (called once, when the library is loaded)."""
    global _lib
    N, C, S = (ctypes.POINTER(t) for t in (KdaRmsnormDesc, KdaConvDesc, KdaSsmDesc))
    for name, n, desc in (("kda_rmsnorm_fwd", 5, N), ("kda_rmsnorm_quant", 6, N), ("kda_rmsnorm_bwd", 7, N),
                          ("kda_conv_fwd", 7, C), ("kda_conv_decode", 6, C), ("kda_conv_bwd", 11, C),
                          ("kda_ssm_fwd", 11, S), ("kda_ssm_decode", 10, S),
                          ("kda_ssm_bwd", 19, S)):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_int, [_P] * n + [desc, _P]
    for name, desc, kind in (("kda_rmsnorm_bwd_workspace_size", N, ctypes.c_size_t),
                             ("kda_conv_bwd_workspace_size", C, ctypes.c_size_t),
                             ("kda_ssm_fwd_workspace_size", S, ctypes.c_size_t), ("kda_ssm_piece_chunks", S, _I),
                             ("kda_ssm_bwd_workspace_size", S, ctypes.c_size_t)):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = kind, [desc]
    _lib = lib  # last: other threads call what they find here


_lib = None


def _library():
    if _lib is None:
        from . import library

        return library()
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _bf16(t: torch.Tensor, name: str, dev: int) -> None:
    if t.dtype != torch.bfloat16:
        raise ValueError("%s must be bfloat16, got %s" % (name, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s is on %s, expected cuda:%d" % (name, t.device, dev))


def _device_of(t: torch.Tensor) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError("inputs must be on a HIP device")
    return dev


def _whole(t: Optional[torch.Tensor], name: str, shape: tuple, dev: int, dtypes=_STATE_DTYPES) -> int:
    """Checks a contiguous parameter, state or index tensor; its type's code (0 for None)."""
    if t is None:
        return 0
    code = dtypes.get(t.dtype)
    if code is None:
        raise ValueError("%s must be %s, got %s" % (name, " or ".join(str(k) for k in dtypes), t.dtype))
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous tensor of shape %s" % (name, list(shape)))
    if t.get_device() != dev:
        raise ValueError("%s is on %s, expected cuda:%d" % (name, t.device, dev))
    return code


def _output(t: Optional[torch.Tensor], name: str, shape: tuple, dtype: torch.dtype, dev: int) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _whole(t, name, shape, dev, {dtype: 1})
    return t


def _workspace(t: Optional[torch.Tensor], need: int, dev: int, d) -> Optional[torch.Tensor]:
    if t is None:
        t = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    elif t.get_device() != dev or not t.is_contiguous() or t.numel() * t.element_size() < need:
        raise ValueError("workspace must be a contiguous tensor of %d bytes on cuda:%d" % (need, dev))
    d.workspace = t.data_ptr()
    d.workspace_bytes = t.numel() * t.element_size()
    return t


def _call(fn, dev: int, *args) -> None:
    """``fn(*args, stream)`` on the current stream of device ``dev``."""
    stream = torch.cuda.current_stream(dev).cuda_stream
    if torch.cuda.current_device() == dev:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != 0:
        from . import _raise_status

        _raise_status(_library(), st)


# ---- RMS normalisation ---------------------------------------------------------

def _rows(t: torch.Tensor, name: str, D: int) -> Tuple[int, int]:
    """(number of rows, elements between them) of [..., D] with even row strides."""
    if t.is_contiguous():
        return t.numel() // D, D
    shape, strides = t.shape, t.stride()
    if strides[-1] != 1 and D > 1:
        raise ValueError("%s must be contiguous along its last dimension" % name)
    rows, stride, span = 1, D, None
    for n, s in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if n == 1:
            continue
        if span is None:
            stride = s
        elif s != span:
            raise ValueError("%s must have rows at one stride (call .contiguous())" % name)
        rows, span = rows * n, s * n
    return rows, stride


def _rmsnorm_args(x, weight, eps, residual, residual_out, group=0):
    """(descriptor, device, residual_out)"""
    dev = _device_of(x)
    _bf16(x, "x", dev)
    shape = x.shape
    D = shape[-1] if shape else 0
    if D < 1:
        raise ValueError("x must be [..., D] with D >= 1")
    rows, xs = _rows(x, "x", D)
    wcode = _whole(weight, "weight", (D,), dev)
    rs = rcode = 0
    if residual is not None:
        rcode = _STATE_DTYPES.get(residual.dtype, 0)
        if residual.shape != shape or not rcode or residual.get_device() != dev:
            raise ValueError("residual must be bf16 or fp32, of x's shape and on its device")
        rs = _rows(residual, "residual", D)[1]
        residual_out = _output(residual_out, "residual_out", shape, residual.dtype, dev)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    return KdaRmsnormDesc(rows, D, xs, rs, rcode, wcode, eps, group), dev, residual_out


def rmsnorm_fwd(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None
                ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """RMS normalisation of ``h = x + residual`` over the last dimension:
    ``h / sqrt(mean(h^2) + eps) * weight``.  Returns ``(out, residual_out)``.

    x: bf16 [..., D]; weight: bf16 or fp32 [D]; residual: bf16 or fp32 of x's
    shape, or None; out: bf16, allocated if None (it may be x); residual_out: h
    in the residual's type, allocated if None (it may be the residual); None
    without a residual."""
    d, dev, residual_out = _rmsnorm_args(x, weight, eps, residual, residual_out)
    out = _output(out, "out", x.shape, torch.bfloat16, dev)
    _call(_library().kda_rmsnorm_fwd, dev, x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(residual_out),
          out.data_ptr(), d)
    return out, residual_out


def rmsnorm_quant(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                  group: int = 0, out: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                  residual_out: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """``rmsnorm_fwd`` with an 8-bit output: returns ``(q, scales, residual_out)``
    with q in ``torch.float8_e4m3fn`` and fp32 scales, the value of an entry
    being ``q * scale``.  group 0: one scale per row, [..., 1]; group 128: one
    per 128 columns, [..., ceil(D / 128)].  A scale is the group's largest
    magnitude / 448 (at least 2^-126)."""
    if group not in (0, 128):
        raise ValueError("group must be 0 (one scale per row) or 128")
    d, dev, residual_out = _rmsnorm_args(x, weight, eps, residual, residual_out, group)
    shape = x.shape
    out = _output(out, "out", shape, torch.float8_e4m3fn, dev)
    scales = _output(scales, "scales", shape[:-1] + (-(-shape[-1] // group) if group else 1,), torch.float32, dev)
    _call(_library().kda_rmsnorm_quant, dev, x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(residual_out),
          out.data_ptr(), scales.data_ptr(), d)
    return out, scales, residual_out


def rmsnorm_bwd_workspace_size(rows: int, D: int) -> int:
    """Workspace bytes ``rmsnorm_bwd`` needs."""
    return int(_library().kda_rmsnorm_bwd_workspace_size(KdaRmsnormDesc(rows, D)))


def rmsnorm_bwd(h: torch.Tensor, weight: torch.Tensor, eps: float, d_out: torch.Tensor,
                d_residual_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                outputs: Optional[dict] = None) -> dict:
    """Gradient of ``rmsnorm_fwd`` for the loss gradients d_out (bf16) and
    d_residual_out (of h's type, or None for zeros).  h: what the forward
    returned as residual_out, or x where it had no residual (bf16 or fp32).
    Returns a dict: dx (bf16; the gradient of x), dresidual (that of the
    residual: the fp32 gradient when h is fp32, dx itself when it is bf16, None
    without d_residual_out and a bf16 h) and dweight (fp32 [D]).  outputs: None,
    or a dict of tensors of those names to write into."""
    dev = _device_of(h)
    hcode = _STATE_DTYPES.get(h.dtype, 0)
    if not hcode:
        raise ValueError("h must be bf16 or fp32, got %s" % h.dtype)
    _bf16(d_out, "d_out", dev)
    shape = h.shape
    D = shape[-1] if shape else 0
    if D < 1 or d_out.shape != shape:
        raise ValueError("h must be [..., D] and d_out of its shape")
    rows, hs = _rows(h, "h", D)
    ds = _rows(d_out, "d_out", D)[1]
    rs = 0
    if d_residual_out is not None:
        if d_residual_out.shape != shape or d_residual_out.dtype != h.dtype or d_residual_out.get_device() != dev:
            raise ValueError("d_residual_out must be of h's shape and type and on its device")
        rs = _rows(d_residual_out, "d_residual_out", D)[1]
    d = KdaRmsnormDesc(rows, D, hs, 0, hcode, _whole(weight, "weight", (D,), dev), eps, 0, ds, rs)
    given = outputs or {}
    dx = _output(given.get("dx"), "dx", shape, torch.bfloat16, dev)
    dres = _output(given.get("dresidual"), "dresidual", shape, torch.float32, dev) if hcode == _FP32 else None
    dw = _output(given.get("dweight"), "dweight", (D,), torch.float32, dev)
    lib = _library()
    ws = _workspace(workspace, lib.kda_rmsnorm_bwd_workspace_size(d), dev, d)  # noqa: F841 (held until the call)
    _call(lib.kda_rmsnorm_bwd, dev, h.data_ptr(), weight.data_ptr(), d_out.data_ptr(), _ptr(d_residual_out),
          dx.data_ptr(), _ptr(dres), dw.data_ptr(), d)
    return {"dx": dx, "dresidual": dres if dres is not None else dx if d_residual_out is not None else None,
            "dweight": dw}


class RmsnormFunction(torch.autograd.Function):
    """``rmsnorm_fwd`` with ``rmsnorm_bwd`` as its gradient."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        out, res = rmsnorm_fwd(x, weight, eps, residual=residual)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x if res is None else res, weight)
        ctx.eps, ctx.with_residual = float(eps), res is not None
        return out, res

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out, d_res):
        h, weight = ctx.saved_tensors
        if d_res is not None:
            d_res = d_res.to(h.dtype).contiguous()
        if d_out is None:
            d_out = torch.zeros(h.shape, dtype=torch.bfloat16, device=h.device)
        g = rmsnorm_bwd(h, weight, ctx.eps, d_out.to(torch.bfloat16).contiguous(), d_residual_out=d_res)
        dres = None
        if ctx.with_residual:
            dres = g["dresidual"] if g["dresidual"] is not None else g["dx"]
        return g["dx"], g["dweight"].to(weight.dtype), dres, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, residual: Optional[torch.Tensor] = None
             ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``rmsnorm_fwd`` as an autograd operation: returns ``(out, residual_out)``
    and backpropagates into x, weight and the residual."""
    return RmsnormFunction.apply(x, weight, residual, eps)


# ---- short causal convolution ----------------------------------------------------

def _tokens(t: torch.Tensor, name: str) -> Tuple[int, int]:
    """Batch and token strides of [B, T, ...] with contiguous further dimensions."""
    shape, strides = t.shape, t.stride()
    n = 1
    for i in range(len(shape) - 1, 1, -1):
        if shape[i] > 1 and strides[i] != n:
            raise ValueError("%s must be contiguous in its dimensions behind [B, T]" % name)
        n *= shape[i]
    return (strides[0] if shape[0] > 1 else 0), (strides[1] if shape[1] > 1 else 0)


def _num_seqs(cu_seqlens: Optional[torch.Tensor], B: int, dev: Optional[int] = None) -> int:
    if cu_seqlens is None:
        return B
    n = cu_seqlens.numel()
    if cu_seqlens.dim() != 1 or n < 2:
        raise ValueError("cu_seqlens must be a 1-D int64 tensor of at least 2 entries")
    if B != 1:
        raise ValueError("with cu_seqlens the batch size must be 1")
    if dev is not None:
        _whole(cu_seqlens, "cu_seqlens", (n,), dev, _INT64_ONLY)
    return n - 1


_ACTIVATIONS = {None: 0, "silu": 1}


def _conv_args(x, weight, bias, activation, initial_state, final_state, cu_seqlens, final_name="final_state"):
    """(descriptor, device)"""
    dev = _device_of(x)
    _bf16(x, "x", dev)
    if x.dim() != 3 or x.shape[0] < 1 or x.shape[2] < 1:
        raise ValueError("x must be [B, T, D]")
    B, T, D = x.shape
    if weight.dim() != 2 or weight.shape[1] not in (2, 3, 4):
        raise ValueError("weight must be [D, W] with W = 2, 3 or 4")
    W = weight.shape[1]
    wcode = _whole(weight, "weight", (D, W), dev)
    if bias is not None and _whole(bias, "bias", (D,), dev) != wcode:
        raise ValueError("bias must have weight's dtype")
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be None or 'silu'")
    N = _num_seqs(cu_seqlens, B, dev)
    sb, st = _tokens(x, "x")
    return KdaConvDesc(B, T, D, W, N, sb, st, 0, 0, _ACTIVATIONS[activation], wcode,
                       _whole(initial_state, "initial_state", (N, W - 1, D), dev),
                       _whole(final_state, final_name, (N, W - 1, D), dev)), dev


def conv_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
             activation: Optional[str] = "silu", initial_state: Optional[torch.Tensor] = None,
             final_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The short causal depthwise convolution over the tokens of every sequence
    (``kda_conv_fwd``).  Returns ``(out, final_state)``.

    x: bf16 [B, T, D]; weight: bf16 or fp32 [D, W], W = 2, 3 or 4, the last tap
    on the current token; bias: [D] of the weight's type, or None; activation:
    None or "silu"; initial_state, final_state: bf16 or fp32 [N, W - 1, D], the
    inputs before and behind the tokens, oldest first, or None (zeros / not
    wanted; final_state may be initial_state); cu_seqlens: int64 [N + 1] on the
    device (then B == 1) or None; out: bf16 [B, T, D], allocated if None."""
    d, dev = _conv_args(x, weight, bias, activation, initial_state, final_state, cu_seqlens)
    out = _output(out, "out", x.shape, torch.bfloat16, dev)
    _call(_library().kda_conv_fwd, dev, x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(initial_state),
          _ptr(final_state), _ptr(cu_seqlens), out.data_ptr(), d)
    return out, final_state


def conv_decode(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                activation: Optional[str] = "silu", initial_state: Optional[torch.Tensor] = None,
                final_state: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None
                ) -> Tuple[torch.Tensor, torch.Tensor]:
    """One token per sequence of ``conv_fwd`` (``kda_conv_decode``): x is
    [N, 1, D].  final_state is required; passing the initial state updates it in
    place.  Returns ``(out, final_state)``."""
    if final_state is None:
        raise ValueError("final_state must be given (it may be initial_state)")
    if x.dim() != 3 or x.shape[1] != 1:
        raise ValueError("x must be [N, 1, D]")
    d, dev = _conv_args(x, weight, bias, activation, initial_state, final_state, None)
    out = _output(out, "out", x.shape, torch.bfloat16, dev)
    _call(_library().kda_conv_decode, dev, x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(initial_state),
          final_state.data_ptr(), out.data_ptr(), d)
    return out, final_state


def conv_bwd_workspace_size(B: int, T: int, D: int, W: int) -> int:
    """Workspace bytes ``conv_bwd`` needs."""
    return int(_library().kda_conv_bwd_workspace_size(KdaConvDesc(B, T, D, W, B, 0, 0, 0, 0, 0, _FP32)))


def conv_bwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor], activation: Optional[str],
             d_out: torch.Tensor, d_final_state: Optional[torch.Tensor] = None,
             initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
             with_d_initial: Optional[bool] = None, workspace: Optional[torch.Tensor] = None,
             outputs: Optional[dict] = None) -> dict:
    """Gradient of ``conv_fwd`` for the loss gradients d_out (bf16 [B, T, D]) and
    d_final_state (bf16 or fp32 [N, W - 1, D], or None).  Returns a dict: dx
    (bf16), dweight (fp32 [D, W]), dbias (fp32 [D], None without a bias),
    d_initial_state (fp32 [N, W - 1, D]; None unless wanted, by default where an
    initial_state is given).  Rows of dx behind a packed batch's last sequence
    are left as they were.  outputs: None, or a dict of tensors of those names
    to write into."""
    d, dev = _conv_args(x, weight, bias, activation, initial_state, d_final_state, cu_seqlens, "d_final_state")
    _bf16(d_out, "d_out", dev)
    if d_out.shape != x.shape:
        raise ValueError("d_out must be of x's shape")
    d.d_out_stride_b, d.d_out_stride_t = _tokens(d_out, "d_out")
    given = outputs or {}
    f32 = torch.float32
    if with_d_initial is None:
        with_d_initial = initial_state is not None
    res = {"dx": _output(given.get("dx"), "dx", x.shape, torch.bfloat16, dev),
           "dweight": _output(given.get("dweight"), "dweight", (d.D, d.W), f32, dev),
           "dbias": None if bias is None else _output(given.get("dbias"), "dbias", (d.D,), f32, dev),
           "d_initial_state": _output(given.get("d_initial_state"), "d_initial_state", (d.num_seqs, d.W - 1, d.D), f32, dev)
           if with_d_initial else None}
    lib = _library()
    ws = _workspace(workspace, lib.kda_conv_bwd_workspace_size(d), dev, d)  # noqa: F841 (held until the call)
    _call(lib.kda_conv_bwd, dev, x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(initial_state), _ptr(cu_seqlens),
          d_out.data_ptr(), _ptr(d_final_state), res["dx"].data_ptr(), res["dweight"].data_ptr(), _ptr(res["dbias"]),
          _ptr(res["d_initial_state"]), d)
    return res


def _packed_zeros(cu_seqlens: Optional[torch.Tensor], like: torch.Tensor) -> Optional[torch.Tensor]:
    """Zeros for a packed batch (rows behind its last sequence are not written), else None."""
    return None if cu_seqlens is None else torch.zeros(like.shape, dtype=torch.bfloat16, device=like.device)


class ConvFunction(torch.autograd.Function):
    """``conv_fwd`` with ``conv_bwd`` as its gradient."""

    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, activation, cu_seqlens, final_dtype):
        N, W = _num_seqs(cu_seqlens, x.shape[0]), weight.shape[1]
        final = None if final_dtype is None else torch.empty((N, W - 1, x.shape[2]), dtype=final_dtype, device=x.device)
        out, final = conv_fwd(x, weight, bias, activation, initial_state, final, cu_seqlens,
                              out=_packed_zeros(cu_seqlens, x))
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.activation = activation
        ctx.set_materialize_grads(False)
        return out, final

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out, d_final):
        x, weight, bias, initial_state, cu_seqlens = ctx.saved_tensors
        if d_out is None:
            d_out = torch.zeros(x.shape, dtype=torch.bfloat16, device=x.device)
        want = initial_state is not None and ctx.needs_input_grad[3]
        g = conv_bwd(x, weight, bias, ctx.activation, d_out.to(torch.bfloat16).contiguous(),
                     d_final_state=None if d_final is None else d_final.contiguous(), initial_state=initial_state,
                     cu_seqlens=cu_seqlens, with_d_initial=want,
                     outputs={"dx": _packed_zeros(cu_seqlens, x)})
        return (g["dx"], g["dweight"].to(weight.dtype), None if bias is None else g["dbias"].to(bias.dtype),
                g["d_initial_state"].to(initial_state.dtype) if want else None, None, None, None)


def short_conv(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               activation: Optional[str] = "silu", initial_state: Optional[torch.Tensor] = None,
               final_state_dtype: Optional[torch.dtype] = None, cu_seqlens: Optional[torch.Tensor] = None
               ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``conv_fwd`` as an autograd operation: returns ``(out, final_state)``, the
    final state in ``final_state_dtype`` or None, and backpropagates into x,
    weight, bias and the initial state.  Rows behind a packed batch's last
    sequence are zero, in the output and in x's gradient."""
    return ConvFunction.apply(x, weight, bias, initial_state, activation, cu_seqlens, final_state_dtype)


# ---- selective state-space scan ----------------------------------------------------

def _ssm_args(x, dt, B, C, A_log, dt_bias, D, initial_state, final_state, cu_seqlens, piece_chunks=0,
              launch_piece=0, final_name="final_state"):
    """(descriptor, device)"""
    dev = _device_of(x)
    _bf16(x, "x", dev), _bf16(dt, "dt", dev), _bf16(B, "B", dev), _bf16(C, "C", dev)
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [B, T, H, P] and B [B, T, G, N]")
    nb, T, H, P = x.shape
    nb2, T2, G, S = shape = B.shape
    if nb < 1 or H < 1 or G < 1 or H % G or nb2 != nb or T2 != T or C.shape != shape or dt.shape != (nb, T, H):
        raise ValueError("shape mismatch among x, dt, B and C (H must be a multiple of G)")
    _whole(A_log, "A_log", (H,), dev, _FP32_ONLY)
    _whole(dt_bias, "dt_bias", (H,), dev, _FP32_ONLY)
    _whole(D, "D", (H,), dev, _FP32_ONLY)
    N = _num_seqs(cu_seqlens, nb, dev)
    return KdaSsmDesc(nb, T, H, P, G, S, N, *_tokens(x, "x"), *_tokens(dt, "dt"), *_tokens(B, "B"), *_tokens(C, "C"), 0, 0,
                      _whole(initial_state, "initial_state", (N, H, P, S), dev),
                      _whole(final_state, final_name, (N, H, P, S), dev), None, 0, piece_chunks, launch_piece), dev


def _ssm_shape(B, T, H, P, G, N, num_seqs, piece_chunks) -> KdaSsmDesc:
    d = KdaSsmDesc(B, T, H, P, G, N, B if num_seqs is None else num_seqs)
    d.piece_chunks = piece_chunks
    return d


def ssm_workspace_size(B: int, T: int, H: int, P: int, G: int, N: int, num_seqs: Optional[int] = None,
                       piece_chunks: int = 0) -> int:
    """Workspace bytes ``ssm_fwd`` needs for these shapes."""
    return int(_library().kda_ssm_fwd_workspace_size(_ssm_shape(B, T, H, P, G, N, num_seqs, piece_chunks)))


def ssm_piece_chunks(B: int, T: int, H: int, P: int, G: int, N: int, num_seqs: Optional[int] = None,
                     piece_chunks: int = 0) -> int:
    """64-token chunks per piece of a state chain for these shapes (at most, in a packed
    batch of several sequences)."""
    n = int(_library().kda_ssm_piece_chunks(_ssm_shape(B, T, H, P, G, N, num_seqs, piece_chunks)))
    if n < 0:
        raise ValueError("invalid shapes")
    return n


def ssm_fwd(x: torch.Tensor, dt: torch.Tensor, B: torch.Tensor, C: torch.Tensor, A_log: torch.Tensor,
            dt_bias: Optional[torch.Tensor] = None, D: Optional[torch.Tensor] = None,
            initial_state: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
            cu_seqlens: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, piece_chunks: int = 0, launch_piece: int = 0
            ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The selective state-space scan (``kda_ssm_fwd``).  Returns ``(out, final_state)``.

    x: bf16 [B, T, H, P], P = 64 or 128; dt: bf16 [B, T, H], before the bias and
    the softplus; B, C: bf16 [B, T, G, N], N = 64 or 128, each group shared by
    H / G consecutive heads; A_log: fp32 [H]; dt_bias, D: fp32 [H] or None (zero);
    initial_state, final_state: bf16 or fp32 [num_seqs, H, P, N] or None (zeros /
    not wanted; final_state may be initial_state); cu_seqlens: int64
    [num_seqs + 1] on the device (then the batch size is 1) or None; out: bf16
    [B, T, H, P], allocated if None; workspace: uint8 of at least
    ``ssm_workspace_size`` bytes, allocated if None; piece_chunks: 0 or the
    chunks per piece (``kda_ssm_desc_t::piece_chunks``); launch_piece:
    kda_ssm_desc_t::launch_piece (0: the library's launch size).

    A NaN or infinity in a token reaches its sequence's outputs from that token on,
    and no other sequence."""
    d, dev = _ssm_args(x, dt, B, C, A_log, dt_bias, D, initial_state, final_state, cu_seqlens, piece_chunks,
                       launch_piece)
    out = _output(out, "out", x.shape, torch.bfloat16, dev)
    lib = _library()
    ws = _workspace(workspace, lib.kda_ssm_fwd_workspace_size(d), dev, d)  # noqa: F841 (held until the call)
    _call(lib.kda_ssm_fwd, dev, x.data_ptr(), dt.data_ptr(), B.data_ptr(), C.data_ptr(), A_log.data_ptr(),
          _ptr(dt_bias), _ptr(D), _ptr(initial_state), _ptr(final_state), _ptr(cu_seqlens), out.data_ptr(), d)
    return out, final_state


def ssm_decode(x: torch.Tensor, dt: torch.Tensor, B: torch.Tensor, C: torch.Tensor, A_log: torch.Tensor,
               dt_bias: Optional[torch.Tensor] = None, D: Optional[torch.Tensor] = None,
               initial_state: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, launch_piece: int = 0) -> Tuple[torch.Tensor, torch.Tensor]:
    """One step of ``ssm_fwd`` per sequence (``kda_ssm_decode``): T = 1.
    final_state is required; passing the initial state updates it in place.
    launch_piece: kda_ssm_desc_t::launch_piece (0: the library's launch size).
    Returns ``(out, final_state)``."""
    if final_state is None:
        raise ValueError("final_state must be given (it may be initial_state)")
    if x.dim() != 4 or x.shape[1] != 1:
        raise ValueError("x must be [N, 1, H, P]")
    d, dev = _ssm_args(x, dt, B, C, A_log, dt_bias, D, initial_state, final_state, None, 0, launch_piece)
    out = _output(out, "out", x.shape, torch.bfloat16, dev)
    _call(_library().kda_ssm_decode, dev, x.data_ptr(), dt.data_ptr(), B.data_ptr(), C.data_ptr(), A_log.data_ptr(),
          _ptr(dt_bias), _ptr(D), _ptr(initial_state), final_state.data_ptr(), out.data_ptr(), d)
    return out, final_state


def ssm_bwd_workspace_size(B: int, T: int, H: int, P: int, G: int, N: int, num_seqs: Optional[int] = None,
                           piece_chunks: int = 0) -> int:
    """Workspace bytes ``ssm_bwd`` needs for these shapes."""
    return int(_library().kda_ssm_bwd_workspace_size(_ssm_shape(B, T, H, P, G, N, num_seqs, piece_chunks)))


def ssm_bwd(x: torch.Tensor, dt: torch.Tensor, B: torch.Tensor, C: torch.Tensor, A_log: torch.Tensor,
            dt_bias: Optional[torch.Tensor], D: Optional[torch.Tensor], d_out: torch.Tensor,
            d_final_state: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
            cu_seqlens: Optional[torch.Tensor] = None, with_d_initial: Optional[bool] = None,
            workspace: Optional[torch.Tensor] = None, outputs: Optional[dict] = None, piece_chunks: int = 0,
            launch_piece: int = 0) -> dict:
    """Gradient of ``ssm_fwd`` (``kda_ssm_bwd``) for the loss gradients d_out (bf16
    [B, T, H, P]) and d_final_state (bf16 or fp32 [num_seqs, H, P, N], or None).
    Returns a dict: dx, ddt, dB and dC (bf16, of their inputs' shapes), dA_log,
    ddt_bias and dD (fp32 [H]; the latter two None where the input is) and
    d_initial_state (fp32 [num_seqs, H, P, N]; None unless wanted, by default
    where an initial_state is given).  Rows behind a packed batch's last sequence
    are left as they were.  outputs: None, or a dict of tensors of those names to
    write into; launch_piece: kda_ssm_desc_t::launch_piece (0: the library's launch
    size).  The workspace holds 8 P N bytes per 64-token chunk and head.

    A NaN or infinity in a token reaches all gradients of its 64-token chunk, those
    of its sequence that depend on the chunk's and the parameters'."""
    d, dev = _ssm_args(x, dt, B, C, A_log, dt_bias, D, initial_state, d_final_state, cu_seqlens, piece_chunks,
                       launch_piece, "d_final_state")
    _bf16(d_out, "d_out", dev)
    if d_out.shape != x.shape:
        raise ValueError("d_out must be of x's shape")
    d.d_out_stride_b, d.d_out_stride_t = _tokens(d_out, "d_out")
    given = outputs or {}
    bf16, f32, H = torch.bfloat16, torch.float32, (d.H,)
    if with_d_initial is None:
        with_d_initial = initial_state is not None
    res = {"dx": _output(given.get("dx"), "dx", x.shape, bf16, dev),
           "ddt": _output(given.get("ddt"), "ddt", dt.shape, bf16, dev),
           "dB": _output(given.get("dB"), "dB", B.shape, bf16, dev),
           "dC": _output(given.get("dC"), "dC", B.shape, bf16, dev),
           "dA_log": _output(given.get("dA_log"), "dA_log", H, f32, dev),
           "ddt_bias": None if dt_bias is None else _output(given.get("ddt_bias"), "ddt_bias", H, f32, dev),
           "dD": None if D is None else _output(given.get("dD"), "dD", H, f32, dev),
           "d_initial_state": _output(given.get("d_initial_state"), "d_initial_state", (d.num_seqs, d.H, d.P, d.N), f32, dev)
           if with_d_initial else None}
    lib = _library()
    ws = _workspace(workspace, lib.kda_ssm_bwd_workspace_size(d), dev, d)  # noqa: F841 (held until the call)
    _call(lib.kda_ssm_bwd, dev, x.data_ptr(), dt.data_ptr(), B.data_ptr(), C.data_ptr(), A_log.data_ptr(), _ptr(dt_bias),
          _ptr(D), _ptr(initial_state), _ptr(cu_seqlens), d_out.data_ptr(), _ptr(d_final_state), res["dx"].data_ptr(),
          res["ddt"].data_ptr(), res["dB"].data_ptr(), res["dC"].data_ptr(), res["dA_log"].data_ptr(),
          _ptr(res["ddt_bias"]), _ptr(res["dD"]), _ptr(res["d_initial_state"]), d)
    return res


class SsmFunction(torch.autograd.Function):
    """``ssm_fwd`` with ``ssm_bwd`` as its gradient."""

    @staticmethod
    def forward(ctx, x, dt, B, C, A_log, dt_bias, D, initial_state, cu_seqlens, final_dtype):
        N = _num_seqs(cu_seqlens, x.shape[0])
        final = None
        if final_dtype is not None:
            final = torch.empty((N, *x.shape[2:], B.shape[-1]), dtype=final_dtype, device=x.device)
        out, final = ssm_fwd(x, dt, B, C, A_log, dt_bias, D, initial_state, final, cu_seqlens,
                             out=_packed_zeros(cu_seqlens, x))
        ctx.save_for_backward(x, dt, B, C, A_log, dt_bias, D, initial_state, cu_seqlens)
        ctx.set_materialize_grads(False)
        return out, final

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out, d_final):
        x, dt, B, C, A_log, dt_bias, D, initial_state, cu_seqlens = ctx.saved_tensors
        if d_out is None:
            d_out = torch.zeros(x.shape, dtype=torch.bfloat16, device=x.device)
        want = initial_state is not None and ctx.needs_input_grad[7]
        g = ssm_bwd(x, dt, B, C, A_log, dt_bias, D, d_out.to(torch.bfloat16).contiguous(),
                    d_final_state=None if d_final is None else d_final.contiguous(), initial_state=initial_state,
                    cu_seqlens=cu_seqlens, with_d_initial=want,
                    outputs={"dx": _packed_zeros(cu_seqlens, x), "ddt": _packed_zeros(cu_seqlens, dt),
                             "dB": _packed_zeros(cu_seqlens, B), "dC": _packed_zeros(cu_seqlens, C)})
        return (g["dx"], g["ddt"], g["dB"], g["dC"], g["dA_log"], g["ddt_bias"], g["dD"],
                g["d_initial_state"].to(initial_state.dtype) if want else None, None, None)


def ssm_scan(x: torch.Tensor, dt: torch.Tensor, B: torch.Tensor, C: torch.Tensor, A_log: torch.Tensor,
             dt_bias: Optional[torch.Tensor] = None, D: Optional[torch.Tensor] = None,
             initial_state: Optional[torch.Tensor] = None, final_state_dtype: Optional[torch.dtype] = None,
             cu_seqlens: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``ssm_fwd`` as an autograd operation: returns ``(out, final_state)``, the
    final state in ``final_state_dtype`` or None, and backpropagates into x, dt,
    B, C, A_log, dt_bias, D and the initial state.  Rows behind a packed batch's
    last sequence are zero, in the output and in the gradients."""
    return SsmFunction.apply(x, dt, B, C, A_log, dt_bias, D, initial_state, cu_seqlens, final_state_dtype)
