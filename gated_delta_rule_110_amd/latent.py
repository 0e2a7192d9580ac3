"""Latent attention (``include/kda_latent.h``): keys and values that come from one
shared vector a token, in the expanded form for prompts and training and in the
absorbed form for generation from a paged cache of those vectors; the store into
that cache; and the pages, slots and offsets of a serving step.

The functions marshal arguments as those of ``layer`` do.  Activations are bf16 and
may be slices of wider tensors: q and kv have to be contiguous behind their token
dimension, all of them begin at multiples of 16 bytes and have strides that are
multiples of 8 elements.  Tensors that a call writes are contiguous.

``latent_attention`` differentiates once.  To capture its backward into a HIP
graph, let no autograd graph of the same leaves from before the capture live
(delete the outputs and losses of the warm-up first): torch ends such a capture
with an error, or ends the process.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from .layer import (_FP32_ONLY, _I, _INT64_ONLY, _P, _bf16, _call, _device_of, _library, _num_seqs, _output, _ptr,
                    _rows, _tokens, _whole, _workspace)

_INT32_ONLY = {torch.int32: 0}
_BOOL_ONLY = {torch.bool: 0}
NOPE, PE, VALUE, LATENT = 128, 64, 128, 512  # a head's own key values, the shared ones, its values, the latent


class KdaLatentDesc(ctypes.Structure):
    _fields_ = [("B", _I), ("T", _I), ("Tk", _I), ("H", _I), ("num_seqs", _I), ("q_stride_b", _I), ("q_stride_t", _I),
                ("kv_stride_b", _I), ("kv_stride_t", _I), ("pe_stride_b", _I), ("pe_stride_t", _I), ("out_stride_b", _I),
                ("out_stride_t", _I), ("d_out_stride_b", _I), ("d_out_stride_t", _I), ("scale", ctypes.c_float),
                ("causal", ctypes.c_int32), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t), ("launch_piece", _I)]


def _declare(lib) -> None:
    """Argument types of these functions (called once, when the library is loaded)."""
    A, D, S, G = (ctypes.POINTER(t) for t in (KdaLatentDesc, KdaLatentDecodeDesc, KdaLatentStoreDesc, KdaPageDesc))
    for name, n, desc in (("kda_latent_fwd", 7, A), ("kda_latent_bwd", 11, A), ("kda_latent_decode", 7, D),
                          ("kda_latent_store", 6, S), ("kda_page_assign", 11, G)):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_int, [_P] * n + [desc, _P]
    for name, desc in (("kda_latent_fwd_workspace_size", A), ("kda_latent_bwd_workspace_size", A),
                       ("kda_latent_decode_workspace_size", D), ("kda_page_workspace_size", G)):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_size_t, [desc]


# ---- the expanded form -----------------------------------------------------------

def _latent_args(q, kv, k_pe, scale, causal, cu, cu_k, launch_piece=0):
    """(descriptor, device) of a call's inputs."""
    dev = _device_of(q)
    for t, name in ((q, "q"), (kv, "kv"), (k_pe, "k_pe")):
        _bf16(t, name, dev)
    if q.dim() != 4 or q.shape[3] != NOPE + PE:
        raise ValueError("q must be [B, T, H, %d]" % (NOPE + PE))
    B, T, H = q.shape[:3]
    if kv.dim() != 4 or kv.shape[0] != B or kv.shape[2:] != (H, NOPE + VALUE):
        raise ValueError("kv must be [B, Tk, H, %d] with q's B and H" % (NOPE + VALUE))
    Tk = kv.shape[1]
    if k_pe.shape != (B, Tk, PE):
        raise ValueError("k_pe must be [B, Tk, %d] with kv's B and Tk" % PE)
    n = _num_seqs(cu, B, dev)
    if cu_k is not None:
        if cu is None:
            raise ValueError("cu_seqlens_k without cu_seqlens")
        _whole(cu_k, "cu_seqlens_k", (n + 1,), dev, _INT64_ONLY)
    elif cu is not None and T != Tk:
        raise ValueError("packed queries and keys of different number need cu_seqlens_k")
    return KdaLatentDesc(B, T, Tk, H, n, *_tokens(q, "q"), *_tokens(kv, "kv"), *_tokens(k_pe, "k_pe"), 0, 0, 0, 0, scale,
                         int(bool(causal)), None, 0, launch_piece), dev


def latent_workspace_size(B: int, T: int, Tk: int, H: int, num_seqs: Optional[int] = None) -> int:
    """Workspace bytes ``latent_fwd`` needs for these sizes (num_seqs: of a packed batch)."""
    return int(_library().kda_latent_fwd_workspace_size(_sizes(B, T, Tk, H, B if num_seqs is None else num_seqs)))


def _sizes(B, T, Tk, H, n):
    return KdaLatentDesc(B, T, Tk, H, n, scale=1.0)


def latent_fwd(q: torch.Tensor, kv: torch.Tensor, k_pe: torch.Tensor, scale: float, causal: bool = True,
               cu_seqlens: Optional[torch.Tensor] = None, cu_seqlens_k: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, launch_piece: int = 0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of every head with the keys ``(kv[..., :128], k_pe)``, of which the second part is shared by all
    heads, and the values ``kv[..., 128:]``.  Returns ``(out, lse)``: bf16 [B, T, H, 128] and the scores' log-sum-exp,
    fp32 [B, T, H].

    q: bf16 [B, T, H, 192]; kv: bf16 [B, Tk, H, 256]; k_pe: bf16 [B, Tk, 64]; scale: of the scores, above zero;
    causal: the last query of a sequence sees all its keys, each one before it one less; cu_seqlens, cu_seqlens_k:
    int64 offsets of a packed batch's queries and keys (B = 1; the keys' are the queries' if None).  A query that
    sees no key has out 0 and lse -inf.  launch_piece: kda_latent_desc_t::launch_piece (0: the library's launch
    size)."""
    d, dev = _latent_args(q, kv, k_pe, scale, causal, cu_seqlens, cu_seqlens_k, launch_piece)
    out = _output(out, "out", (d.B, d.T, d.H, VALUE), torch.bfloat16, dev)
    lse = _output(lse, "lse", (d.B, d.T, d.H), torch.float32, dev)
    need = _library().kda_latent_fwd_workspace_size(d)
    if need:
        ws = _workspace(workspace, need, dev, d)  # noqa: F841 (held until the call)
    _call(_library().kda_latent_fwd, dev, q.data_ptr(), kv.data_ptr(), k_pe.data_ptr(), _ptr(cu_seqlens), _ptr(cu_seqlens_k),
          out.data_ptr(), lse.data_ptr(), d)
    return out, lse


def latent_bwd_workspace_size(B: int, T: int, Tk: int, H: int, num_seqs: Optional[int] = None) -> int:
    """Workspace bytes ``latent_bwd`` needs for these sizes (num_seqs: of a packed batch)."""
    return int(_library().kda_latent_bwd_workspace_size(_sizes(B, T, Tk, H, B if num_seqs is None else num_seqs)))


def latent_bwd(q: torch.Tensor, kv: torch.Tensor, k_pe: torch.Tensor, scale: float, out: torch.Tensor, lse: torch.Tensor,
               d_out: torch.Tensor, causal: bool = True, cu_seqlens: Optional[torch.Tensor] = None,
               cu_seqlens_k: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               outputs: Optional[dict] = None, launch_piece: int = 0) -> dict:
    """Gradient of ``latent_fwd`` for the loss's gradient d_out (bf16 [B, T, H, 128]), from its inputs and what it
    returned (out, lse).  Returns a dict of bf16 tensors: dq [B, T, H, 192], dkv [B, Tk, H, 256] and dk_pe [B, Tk, 64],
    summed over the heads.  outputs: None, or a dict of tensors of those names to write into."""
    d, dev = _latent_args(q, kv, k_pe, scale, causal, cu_seqlens, cu_seqlens_k, launch_piece)
    for t, name in ((out, "out"), (d_out, "d_out")):
        _bf16(t, name, dev)
        if t.shape != (d.B, d.T, d.H, VALUE):
            raise ValueError("%s must be [B, T, H, %d]" % (name, VALUE))
    _whole(lse, "lse", (d.B, d.T, d.H), dev, _FP32_ONLY)
    d.out_stride_b, d.out_stride_t = _tokens(out, "out")
    d.d_out_stride_b, d.d_out_stride_t = _tokens(d_out, "d_out")
    given = outputs or {}
    dq = _output(given.get("dq"), "dq", (d.B, d.T, d.H, NOPE + PE), torch.bfloat16, dev)
    dkv = _output(given.get("dkv"), "dkv", (d.B, d.Tk, d.H, NOPE + VALUE), torch.bfloat16, dev)
    dpe = _output(given.get("dk_pe"), "dk_pe", (d.B, d.Tk, PE), torch.bfloat16, dev)
    lib = _library()
    ws = _workspace(workspace, lib.kda_latent_bwd_workspace_size(d), dev, d)  # noqa: F841 (held until the call)
    _call(lib.kda_latent_bwd, dev, q.data_ptr(), kv.data_ptr(), k_pe.data_ptr(), _ptr(cu_seqlens), _ptr(cu_seqlens_k),
          out.data_ptr(), lse.data_ptr(), d_out.data_ptr(), dq.data_ptr(), dkv.data_ptr(), dpe.data_ptr(), d)
    return {"dq": dq, "dkv": dkv, "dk_pe": dpe}


class LatentFunction(torch.autograd.Function):
    """``latent_fwd`` with ``latent_bwd`` as its gradient."""

    @staticmethod
    def forward(ctx, q, kv, k_pe, scale, causal, cu_seqlens, cu_seqlens_k):
        out, lse = latent_fwd(q, kv, k_pe, scale, causal, cu_seqlens, cu_seqlens_k)
        if cu_seqlens is not None:  # rows behind the last sequence, which the kernels leave as they were
            row = torch.arange(out.shape[1], device=out.device)[None, :, None, None]
            out.masked_fill_(row >= cu_seqlens[-1], 0)
        ctx.save_for_backward(q, kv, k_pe, out, lse, cu_seqlens, cu_seqlens_k)
        ctx.scale, ctx.causal = float(scale), bool(causal)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        q, kv, k_pe, out, lse, cu, cu_k = ctx.saved_tensors
        given = None
        if cu is not None:
            given = {"dq": torch.zeros(q.shape, dtype=q.dtype, device=q.device),
                     "dkv": torch.zeros(kv.shape, dtype=kv.dtype, device=kv.device),
                     "dk_pe": torch.zeros(k_pe.shape, dtype=k_pe.dtype, device=k_pe.device)}
        g = latent_bwd(q, kv, k_pe, ctx.scale, out, lse, d_out.to(torch.bfloat16).contiguous(), ctx.causal, cu, cu_k,
                       outputs=given)
        return g["dq"], g["dkv"], g["dk_pe"], None, None, None, None


def latent_attention(q: torch.Tensor, kv: torch.Tensor, k_pe: torch.Tensor, scale: float, causal: bool = True,
                     cu_seqlens: Optional[torch.Tensor] = None, cu_seqlens_k: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``latent_fwd`` as an autograd operation: returns out and backpropagates into q, kv and k_pe.  In a packed
    batch, rows behind the last sequence are zeros, as are their gradients."""
    return LatentFunction.apply(q, kv, k_pe, scale, causal, cu_seqlens, cu_seqlens_k)


# ---- the absorbed form -----------------------------------------------------------

class KdaLatentDecodeDesc(ctypes.Structure):
    _fields_ = [("N", _I), ("T", _I), ("H", _I), ("pages", _I), ("page_size", _I), ("max_pages", _I), ("ql_stride_n", _I),
                ("ql_stride_t", _I), ("ql_stride_h", _I), ("qp_stride_n", _I), ("qp_stride_t", _I), ("qp_stride_h", _I),
                ("scale", ctypes.c_float), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


def _row_strides(t, name):
    """Strides of [N, T, H, values] with contiguous values (0 for dimensions of one entry)."""
    shape, strides = t.shape, t.stride()
    if strides[3] != 1:
        raise ValueError("%s must be contiguous along its last dimension" % name)
    return tuple(st if n > 1 else 0 for n, st in zip(shape[:3], strides[:3]))


def _cache_args(cache, dev):
    _bf16(cache, "cache", dev)
    if cache.dim() != 3 or cache.shape[2] != LATENT + PE or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous tensor [pages, page_size, %d]" % (LATENT + PE))
    return cache.shape[0], cache.shape[1]


def latent_decode_workspace_size(N: int, T: int, H: int) -> int:
    """Workspace bytes ``latent_decode`` needs."""
    return int(_library().kda_latent_decode_workspace_size(KdaLatentDecodeDesc(N, T, H, 0, 1, scale=1.0)))


def latent_decode(q_latent: torch.Tensor, q_pe: torch.Tensor, cache: torch.Tensor, lengths: torch.Tensor,
                  block_table: torch.Tensor, scale: float, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of the last T tokens of N sequences over their rows in the cache, which are keys (576 values) and
    values (the first 512) of all heads.  Returns ``(out, lse)``: bf16 [N, T, H, 512], the mean latent of every head
    (which the head's values' projection expands), and the scores' log-sum-exp, fp32 [N, T, H].

    q_latent: bf16 [N, T, H, 512] (the head's query through its keys' projection) and q_pe: bf16 [N, T, H, 64], with
    any strides ahead of their last dimension; cache: bf16 [pages, page_size, 576], page_size a power of two; lengths:
    int64 [N], the sequences' rows, those of the T tokens among them; block_table: int32 [N, max_pages].  Token t sees
    the rows before lengths - T + t + 1; one that sees none has out 0 and lse -inf."""
    dev = _device_of(q_latent)
    _bf16(q_latent, "q_latent", dev)
    _bf16(q_pe, "q_pe", dev)
    if q_latent.dim() != 4 or q_latent.shape[3] != LATENT:
        raise ValueError("q_latent must be [N, T, H, %d]" % LATENT)
    N, T, H = q_latent.shape[:3]
    if q_pe.shape != (N, T, H, PE):
        raise ValueError("q_pe must be [N, T, H, %d] like q_latent" % PE)
    pages, size = _cache_args(cache, dev)
    _whole(lengths, "lengths", (N,), dev, _INT64_ONLY)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [N, max_pages]")
    _whole(block_table, "block_table", (N, block_table.shape[1]), dev, _INT32_ONLY)
    d = KdaLatentDecodeDesc(N, T, H, pages, size, block_table.shape[1], *_row_strides(q_latent, "q_latent"),
                            *_row_strides(q_pe, "q_pe"), scale)
    out = _output(out, "out", (N, T, H, LATENT), torch.bfloat16, dev)
    lse = _output(lse, "lse", (N, T, H), torch.float32, dev)
    lib = _library()
    ws = _workspace(workspace, lib.kda_latent_decode_workspace_size(d), dev, d)  # noqa: F841 (held until the call)
    _call(lib.kda_latent_decode, dev, q_latent.data_ptr(), q_pe.data_ptr(), cache.data_ptr(), lengths.data_ptr(),
          block_table.data_ptr(), out.data_ptr(), lse.data_ptr(), d)
    return out, lse


# ---- the cache ---------------------------------------------------------------------

class KdaLatentStoreDesc(ctypes.Structure):
    _fields_ = [("tokens", _I), ("num_slots", _I), ("latent_stride", _I), ("pe_stride", _I),
                ("weight_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


def latent_store(latent: torch.Tensor, k_pe: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor,
                 weight: Optional[torch.Tensor] = None, eps: float = 1e-6, keep_normed: bool = False,
                 normed: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Writes every token's row ``(n, k_pe)`` into the cache, n being the latent's RMS normalisation (with a weight) or
    the latent itself.  Returns ``(cache, normed)``: the cache, and n of all tokens, bf16 of latent's shape, where
    keep_normed asks for it or `normed` is given (what the expansion to keys and values reads), else None.

    latent: bf16 [..., 512]; k_pe: bf16 [..., 64]; slots: int64, one a token, page * page_size + offset; tokens with
    slots outside the cache (-1) are not stored, the others have to differ; cache: bf16 [pages, page_size, 576],
    written in place; weight: bf16 or fp32 [512]."""
    dev = _device_of(latent)
    _bf16(latent, "latent", dev)
    _bf16(k_pe, "k_pe", dev)
    if latent.dim() < 1 or latent.shape[-1] != LATENT or k_pe.shape != latent.shape[:-1] + (PE,):
        raise ValueError("latent must be [..., %d] and k_pe [..., %d] with the same tokens" % (LATENT, PE))
    tokens, ls = _rows(latent, "latent", LATENT)
    _whole(slots, "slots", latent.shape[:-1], dev, _INT64_ONLY)
    pages, size = _cache_args(cache, dev)
    d = KdaLatentStoreDesc(tokens, pages * size, ls, _rows(k_pe, "k_pe", PE)[1], _whole(weight, "weight", (LATENT,), dev), eps)
    if normed is not None or keep_normed:
        normed = _output(normed, "normed", latent.shape, torch.bfloat16, dev)
    _call(_library().kda_latent_store, dev, latent.data_ptr(), k_pe.data_ptr(), _ptr(weight), slots.data_ptr(),
          cache.data_ptr(), _ptr(normed), d)
    return cache, normed


class KdaPageDesc(ctypes.Structure):
    _fields_ = [("N", _I), ("max_pages", _I), ("page_size", _I), ("stack", _I), ("tokens", _I), ("workspace", _P),
                ("workspace_bytes", ctypes.c_size_t)]


def page_assign(lengths: torch.Tensor, new_tokens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                free_count: torch.Tensor, page_size: int, tokens: int, ended: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, outputs: Optional[dict] = None) -> dict:
    """The pages, slots and offsets of one serving step, from the requests' lengths, without the host.

    lengths, new_tokens: int64 [N], tokens that each request holds and gets; block_table: int32 [N, max_pages], the
    requests' pages, updated in place; free_pages: int32, a stack of the free ones of which the first free_count
    (int64 [1]) are in use, updated in place; page_size: a power of two; tokens: rows of the step's packed batch (at
    least the sum of new_tokens); ended: bool [N], requests that end: their pages go back to the stack and new_tokens
    begin the row's next request.

    Returns a dict: slots (int64 [tokens], a cache slot for every new token, request after request; -1 for those that
    were refused and for the rows behind the last), cu_seqlens (int64 [N + 1], the packed batch's offsets), lengths
    (int64 [N], the new ones), granted (int64 [N]: new_tokens, or 0 where the pages, the table's row or the rows of the
    batch do not suffice) and free_count (int64 [1], the new one).  outputs: None, or a dict of tensors of those names
    to write into; lengths and free_count may be the inputs."""
    dev = _device_of(lengths)
    N = lengths.shape[0] if lengths.dim() == 1 else -1
    _whole(lengths, "lengths", (max(N, 0),), dev, _INT64_ONLY)
    _whole(new_tokens, "new_tokens", (N,), dev, _INT64_ONLY)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [N, max_pages]")
    _whole(block_table, "block_table", (N, block_table.shape[1]), dev, _INT32_ONLY)
    _whole(free_pages, "free_pages", (free_pages.numel(),), dev, _INT32_ONLY)
    _whole(free_count, "free_count", (1,), dev, _INT64_ONLY)
    if ended is not None:
        _whole(ended, "ended", (N,), dev, _BOOL_ONLY)
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    d = KdaPageDesc(N, block_table.shape[1], page_size, free_pages.numel(), tokens)
    sizes = {"slots": tokens, "cu_seqlens": N + 1, "lengths": N, "granted": N, "free_count": 1}
    given = outputs or {}
    res = {k: _output(given[k], k, (n,), torch.int64, dev) for k, n in sizes.items() if given.get(k) is not None}
    lib = _library()
    need = [k for k in sizes if k not in res]
    if workspace is None:  # one allocation for it and all outputs that are not given
        words = lib.kda_page_workspace_size(d) // 8
        buf = torch.empty(words + sum(sizes[k] for k in need), dtype=torch.int64, device=dev)
        d.workspace, d.workspace_bytes = buf.data_ptr(), 8 * words
        res.update(zip(need, buf.split_with_sizes([words] + [sizes[k] for k in need])[1:]))
    else:
        _workspace(workspace, lib.kda_page_workspace_size(d), dev, d)
        res.update((k, torch.empty(sizes[k], dtype=torch.int64, device=dev)) for k in need)
    _call(lib.kda_page_assign, dev, lengths.data_ptr(), new_tokens.data_ptr(), _ptr(ended), block_table.data_ptr(),
          free_pages.data_ptr(), free_count.data_ptr(), *[res[k].data_ptr() for k in sizes], d)
    return {k: res[k] for k in sizes}
