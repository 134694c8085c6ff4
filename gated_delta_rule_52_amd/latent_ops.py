"""Torch-facing wrappers of latent attention in include/kda.h: rotary positions, the paged cache of latent vectors, attention
over expanded keys and values with its gradients, and attention of single tokens over the cache.

As in layer_ops.py, torch supplies device memory and the current HIP stream and every step runs in libkda.so.  Tensors
with heads may be slices of wider ones or have their heads in front of their rows in memory: the last dimension must be
dense, the rows equally spaced.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import _lib
from .layer_ops import (F32, _at, _call, _call_with_workspace, _fields, _first, _grad_dtype, _kind, _refuse, _size,
                        _step, _stream)

_ROTARY, _APPEND = _lib.packer(_lib.RotaryArgs), _lib.packer(_lib.LatentAppendArgs)
_STEP = _lib.packer(_lib.LatentStepArgs)
_FWD, _BWD = _lib.packer(_lib.LatentAttentionArgs), _lib.packer(_lib.LatentAttentionBwdArgs)
I32 = torch.int32


def _heads(t, name, shape, dtype, device):
    """Checks a tensor [..., H, D] and returns the distances between its rows and between its heads in elements."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        _refuse(t, name, shape, dtype, device)
    H, D = shape[-2:]
    if t.is_contiguous():
        return H * D, D
    strides = t.stride()
    if D != 1 and strides[-1] != 1:
        raise ValueError(f"{name} must be dense along its last dimension")
    row, span = None, 1
    for size, stride in zip(reversed(shape[:-2]), reversed(strides[:-2])):
        if size == 1:
            continue
        if row is None:
            row = stride
        elif stride != span * row:
            raise ValueError(f"the rows of {name} must be equally spaced")
        span *= size
    return H * D if row is None else row, strides[-2] if H != 1 else D


def rotary_frequencies(rot: int, base: float = 10000.0, factor: float = 1.0, original_length: Optional[int] = None,
                       slow: float = 1.0, fast: float = 32.0, device=None):
    """(inv_freq [rot/2] fp32, scale) of rotary positions: pair j turns by base^(-2j/rot) per position.

    A context stretched by ``factor``: without ``original_length`` every frequency is divided by it (positions
    interpolated evenly).  With it, frequencies that make fewer than ``slow`` turns over the original length are, those
    with more than ``fast`` are kept, and those between are mixed in proportion to their turns; scale is then
    0.1 ln(factor) + 1, for queries and keys both."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot={rot} must be even and positive")
    if not (base > 0 and factor >= 1 and fast > slow):
        raise ValueError("base must be positive, factor at least 1 and fast above slow")
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    scale = 1.0
    if factor != 1.0:
        keep = torch.zeros_like(f)
        if original_length is not None:
            keep = ((original_length * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
            scale = 0.1 * math.log(factor) + 1.0
        f = f * keep + f / factor * (1 - keep)
    return f.to(F32).to(device or "cuda"), scale


def _rotary(name, x, xname, positions, inv_freq, interleaved, offset, scale, y, yname):
    if x.dim() < 3:
        raise ValueError(f"{xname} must be [..., H, D]")
    device = _first(x, xname, (x.dim(),))
    shape, kind = x.shape, _kind(x, xname)
    xs = _heads(x, xname, shape, x.dtype, device)
    if y is None:
        y = torch.empty(shape, dtype=x.dtype, device=device)
    ys = _heads(y, yname, shape, x.dtype, device)
    half = inv_freq.numel()
    rows = positions.numel()
    _call(name, _ROTARY.pack(
        _ROTARY.size, x.data_ptr(), y.data_ptr(), _at(positions, "positions", tuple(shape[:-2]), I32, device),
        _at(inv_freq, "inv_freq", (half,), F32, device), *xs, *ys, rows, shape[-2], shape[-1], 2 * half, offset, scale,
        kind, _stream(device), _lib.KDA_ROTARY_INTERLEAVED if interleaved else 0), device)
    return y


def rotary_fwd(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, interleaved: bool = False, offset: int = 0,
               scale: float = 1.0, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotary positions: of each head of x [..., H, D] (bf16 or fp32) the 2 len(inv_freq) elements from ``offset`` on are
    turned in pairs (a, b), pair j by the angle position * inv_freq[j],

        (a, b) -> scale (a cos - b sin, b cos + a sin);

    pairs are adjacent elements where ``interleaved``, the halves' elements otherwise.  The others are copied.
    positions: int32 of x's shape without H and D; inv_freq: fp32 (``rotary_frequencies``).  ``y`` may be ``x``, whose
    other elements are then not touched.  Returns y."""
    return _rotary("kda_rotary_fwd", x, "x", positions, inv_freq, interleaved, offset, scale, y, "y")


def rotary_bwd(grad_y: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, interleaved: bool = False,
               offset: int = 0, scale: float = 1.0, grad_x: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of ``rotary_fwd``'s x for grad_y [..., H, D], in grad_y's type: turned the other way.  ``grad_x``
    may be ``grad_y``."""
    return _rotary("kda_rotary_bwd", grad_y, "grad_y", positions, inv_freq, interleaved, offset, scale, grad_x, "grad_x")


def latent_cache_append(latent: torch.Tensor, rope: torch.Tensor, cache: torch.Tensor, slots: torch.Tensor,
                        positions: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None,
                        interleaved: bool = False, scale: float = 1.0) -> torch.Tensor:
    """Rows into the paged cache, in place: row slots[i] of cache [blocks, page, dl + dr] (counted over all pages) becomes
    [latent_i | rope_i], with rope_i turned by its position as in ``rotary_fwd`` where positions and inv_freq
    [dr / 2] are given.

    latent [T, dl], rope [T, dr] (rows may be slices of wider ones) and cache are of one type; slots, positions: int32
    [T].  Rows with a slot below zero or behind the cache are skipped; the slots of a call must differ otherwise.
    Returns cache."""
    device = _first(latent, "latent", (2,))
    kind = _kind(latent, "latent")
    if rope.dim() != 2 or cache.dim() != 3:
        raise ValueError("rope must be [T,dr] and cache [blocks,page,dl+dr]")
    T, dl = latent.shape
    dr = rope.shape[1]
    blocks, page = cache.shape[:2]
    if blocks >> 31 or page >> 31:
        raise ValueError(f"cache has shape {tuple(cache.shape)}, expected sizes below 2^31")
    _call("kda_latent_cache_append", _APPEND.pack(
        _APPEND.size, latent.data_ptr(), rope.data_ptr(),
        _at(cache, "cache", (blocks, page, dl + dr), latent.dtype, device), _at(slots, "slots", (T,), I32, device),
        _at(positions, "positions", (T,), I32, device), _at(inv_freq, "inv_freq", (dr // 2,), F32, device),
        _step(latent, "latent", latent.shape, latent.dtype, device), _step(rope, "rope", (T, dr), latent.dtype, device),
        T, blocks, page, dl, dr, scale, kind, _stream(device), _lib.KDA_ROTARY_INTERLEAVED if interleaved else 0), device)
    return cache


def latent_attention_step_workspace_bytes(q_latent: torch.Tensor, dr: int, page: int, max_blocks: int) -> int:
    """Bytes that ``latent_attention_step`` needs for q_latent [N,H,dl] and block tables of max_blocks pages."""
    N, H, dl = q_latent.shape
    return _size("kda_latent_attention_step_workspace_bytes", _fields(
        _lib.LatentStepArgs, N=N, H=H, dl=dl, dr=dr, page=page, max_blocks=max_blocks, scale=1.0,
        in_dtype=_kind(q_latent, "q_latent")))


def latent_attention_step(q_latent: torch.Tensor, q_rope: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                          lengths: torch.Tensor, scale: float, out_dtype: Optional[torch.dtype] = None,
                          o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None):
    """Latent attention of one token per sequence over the paged cache, in the absorbed form: every head's key is the
    cached row [c | r], its value c,

        s_hj = scale (q_latent_h . c_j + q_rope_h . r_j),  lse_h = log sum_j exp(s_hj),  o_h = sum_j exp(s_hj - lse_h) c_j

    over the first lengths[n] rows of sequence n, row j at place j % page of block block_table[n, j // page].

    q_latent [N,H,dl], q_rope [N,H,dr], cache [blocks,page,dl+dr]: one type, bf16 or fp32; block_table [N,max_blocks],
    lengths [N]: int32.  Lengths are held to 0 .. max_blocks * page; rows on blocks that do not exist are left out.  A
    sequence without rows gets o = 0 and lse = -inf.  Where all sequences are much shorter than the table,
    block_table[:, :k] with the k columns in use may be faster.  Returns (o [N,H,dl], lse [N,H] fp32)."""
    device = _first(q_latent, "q_latent", (3,))
    kind, dtype = _kind(q_latent, "q_latent"), q_latent.dtype
    if q_rope.dim() != 3 or cache.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q_rope must be [N,H,dr], cache [blocks,page,dl+dr] and block_table [N,max_blocks]")
    shape = q_latent.shape
    N, H, dl = shape
    dr = q_rope.shape[2]
    blocks, page = cache.shape[:2]
    if blocks >> 31 or page >> 31:
        raise ValueError(f"cache has shape {tuple(cache.shape)}, expected sizes below 2^31")
    if o is None:
        o = torch.empty(shape, dtype=out_dtype or dtype, device=device)
    if lse is None:
        lse = torch.empty((N, H), dtype=F32, device=device)
    front = (
        _STEP.size, q_latent.data_ptr(), q_rope.data_ptr(), _at(cache, "cache", (blocks, page, dl + dr), dtype, device),
        block_table.data_ptr(), _at(lengths, "lengths", (N,), I32, device), o.data_ptr(),
        _at(lse, "lse", (N, H), F32, device), *_heads(q_latent, "q_latent", shape, dtype, device),
        *_heads(q_rope, "q_rope", (N, H, dr), dtype, device), *_heads(o, "o", shape, out_dtype or o.dtype, device),
        _step(block_table, "block_table", (N, block_table.shape[1]), I32, device), N, H, dl, dr, page, blocks,
        block_table.shape[1], scale, kind, _kind(o, "o"))
    _call_with_workspace("kda_latent_attention_step", _STEP.pack, front, (_stream(device),), workspace, device)
    return o, lse


def _attend(q, k, k_rope, v, scale, cu_seqlens_q, cu_seqlens_k):
    """Checks the inputs of an attention over prompts; returns what its calls share."""
    device = _first(q, "q", (4,))
    dtype = q.dtype
    kind = _kind(q, "q")
    if k.dim() != 4 or k_rope.dim() != 3 or v.dim() != 4:
        raise ValueError("k must be [B,Tk,H,dn], k_rope [B,Tk,dr] and v [B,Tk,H,dv]")
    B, Tq, H, dq = q.shape
    Tk, dn, dr, dv = k.shape[1], k.shape[3], k_rope.shape[2], v.shape[3]
    if max(B, Tq, Tk, H) >> 31:
        raise ValueError("sizes have to be below 2^31")
    if (cu_seqlens_q is None) != (cu_seqlens_k is None):
        raise ValueError("cu_seqlens_q and cu_seqlens_k are given together")
    N, cu_q, cu_k = B, 0, 0
    if cu_seqlens_q is not None:
        N = cu_seqlens_q.numel() - 1
        cu_q = _at(cu_seqlens_q, "cu_seqlens_q", (N + 1,), I32, device)
        cu_k = _at(cu_seqlens_k, "cu_seqlens_k", (N + 1,), I32, device)
    if scale is None:
        scale = dq ** -0.5
    strides = (*_heads(q, "q", (B, Tq, H, dn + dr), dtype, device), *_heads(k, "k", (B, Tk, H, dn), dtype, device),
               _step(k_rope, "k_rope", (B, Tk, dr), dtype, device), *_heads(v, "v", (B, Tk, H, dv), dtype, device))
    return device, dtype, kind, (B, Tq, Tk, H, dn, dr, dv, N, scale), strides, cu_q, cu_k


def latent_attention_fwd(q: torch.Tensor, k: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor,
                         scale: Optional[float] = None, causal: bool = True, cu_seqlens_q: Optional[torch.Tensor] = None,
                         cu_seqlens_k: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                         o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None):
    """Latent attention over expanded keys and values, per sequence and head,

        s_ij = scale (q_i[:dn] . k_j + q_i[dn:] . k_rope_j),  lse_i = log sum_j exp(s_ij),  o_i = sum_j exp(s_ij - lse_i) v_j.

    q [B,Tq,H,dn+dr], k [B,Tk,H,dn], k_rope [B,Tk,dr] (one for all heads), v [B,Tk,H,dv]: one type, bf16 or fp32; k and v
    may be slices of one [B,Tk,H,dn+dv] tensor.  ``causal``: query i of nq sees keys 0 .. i + nk - nq.  Packed input:
    B == 1 and int32 [N+1] offsets of the queries and of the keys; rows at and behind the last are left as they were.
    scale defaults to (dn + dr)^-0.5.  A query that sees no key gets o = 0 and lse = -inf.  Infinite or NaN values of a key
    that is hidden from a query of its sequence may reach that query's result.
    Returns (o [B,Tq,H,dv], lse [B,Tq,H] fp32); the gradients take both, o in q's type (``out_dtype`` left out)."""
    device, dtype, kind, sizes, strides, cu_q, cu_k = _attend(q, k, k_rope, v, scale, cu_seqlens_q, cu_seqlens_k)
    B, Tq, H, dv = sizes[0], sizes[1], sizes[3], sizes[6]
    if o is None:
        o = torch.empty((B, Tq, H, dv), dtype=out_dtype or dtype, device=device)
    if lse is None:
        lse = torch.empty((B, Tq, H), dtype=F32, device=device)
    _call("kda_latent_attention_fwd", _FWD.pack(
        _FWD.size, q.data_ptr(), k.data_ptr(), k_rope.data_ptr(), v.data_ptr(), o.data_ptr(),
        _at(lse, "lse", (B, Tq, H), F32, device), cu_q, cu_k, *strides,
        *_heads(o, "o", (B, Tq, H, dv), out_dtype or o.dtype, device), *sizes, kind, _kind(o, "o"), _stream(device),
        _lib.KDA_ATTENTION_CAUSAL if causal else 0), device)
    return o, lse


def latent_attention_bwd_workspace_bytes(q: torch.Tensor, k: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor) -> int:
    """Bytes that ``latent_attention_bwd`` needs for these inputs."""
    B, Tq, H, _ = q.shape
    return _size("kda_latent_attention_bwd_workspace_bytes", _fields(
        _lib.LatentAttentionBwdArgs, batch=B, Tq=Tq, Tk=k.shape[1], H=H, dn=k.shape[3], dr=k_rope.shape[2], dv=v.shape[3],
        num_seqs=B, scale=1.0, in_dtype=_kind(q, "q")))


def latent_attention_bwd(q: torch.Tensor, k: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                         lse: torch.Tensor, grad_o: torch.Tensor, scale: Optional[float] = None, causal: bool = True,
                         cu_seqlens_q: Optional[torch.Tensor] = None, cu_seqlens_k: Optional[torch.Tensor] = None,
                         grad_dtype: torch.dtype = F32, workspace: Optional[torch.Tensor] = None,
                         out: Optional[dict] = None) -> dict:
    """Gradients of ``latent_attention_fwd`` for grad_o [B,Tq,H,dv] (dtype of q), given its inputs, its o (dtype of q) and its
    lse.  Returns a dict dq, dk, dk_rope, dv of the inputs' shapes in ``grad_dtype``; ``out`` may supply them (dk and dv
    may be slices of one [B,Tk,H,dn+dv] tensor).  Rows outside the sequences of packed input are left as they were."""
    device, dtype, kind, sizes, strides, cu_q, cu_k = _attend(q, k, k_rope, v, scale, cu_seqlens_q, cu_seqlens_k)
    B, Tq, Tk, H, dn, dr, dv = sizes[:7]
    grad_kind = _grad_dtype(grad_dtype)
    shapes = dict(dq=(B, Tq, H, dn + dr), dk=(B, Tk, H, dn), dk_rope=(B, Tk, dr), dv=(B, Tk, H, dv))
    if out is None:
        out = {n: torch.empty(s, dtype=grad_dtype, device=device) for n, s in shapes.items()}
    got = {n: out[n] for n in shapes}
    rows = (B, Tq, H, dv)
    front = (
        _BWD.size, q.data_ptr(), k.data_ptr(), k_rope.data_ptr(), v.data_ptr(), o.data_ptr(),
        _at(lse, "lse", (B, Tq, H), F32, device), grad_o.data_ptr(), got["dq"].data_ptr(), got["dk"].data_ptr(),
        got["dk_rope"].data_ptr(), got["dv"].data_ptr(), cu_q, cu_k, *strides, *_heads(o, "o", rows, dtype, device),
        *_heads(grad_o, "grad_o", rows, dtype, device), *_heads(got["dq"], "dq", shapes["dq"], grad_dtype, device),
        *_heads(got["dk"], "dk", shapes["dk"], grad_dtype, device),
        _step(got["dk_rope"], "dk_rope", shapes["dk_rope"], grad_dtype, device),
        *_heads(got["dv"], "dv", shapes["dv"], grad_dtype, device), *sizes, kind, grad_kind)
    back = _stream(device), _lib.KDA_ATTENTION_CAUSAL if causal else 0
    _call_with_workspace("kda_latent_attention_bwd", _BWD.pack, front, back, workspace, device)
    return got
