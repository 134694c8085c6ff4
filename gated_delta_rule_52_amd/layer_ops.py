"""Torch-facing wrappers of the layer operators in include/kda.h: selective
state space scan, short causal convolution and layer norm.

As in ops.py, torch supplies device memory and the current HIP stream and every
step runs in libkda.so.  Token tensors may be column slices of wider ones: the
last dimension must be dense and the rows equally spaced.
"""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import _lib
from .ops import _DT, _need, _ptr, _stream

F32 = torch.float32


def _dtype(t: torch.Tensor, name: str) -> torch.dtype:
    if t.dtype not in _DT:
        raise ValueError(f"unsupported {name} dtype {t.dtype}")
    return t.dtype


def _rows(t: torch.Tensor, name: str, shape, dtype=None, device=None) -> int:
    """Checks a token tensor and returns the distance between its rows in elements."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    width, strides = shape[-1], t.stride()
    if width != 1 and strides[-1] != 1:
        raise ValueError(f"{name} must be dense along its last dimension")
    if t.numel() == 0:
        return width
    step, span = 0, 1  # of the innermost leading dimension with more than one entry, and the rows inside
    for size, stride in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if size == 1:
            continue
        if step == 0:
            step = stride
        elif stride != span * step:
            raise ValueError(f"the rows of {name} must be equally spaced")
        span *= size
    return step if span > 1 else width


def _opt(t, name, shape, dtype, device) -> int:
    return 0 if t is None else _rows(t, name, shape, dtype, device)


def _param(t: Optional[torch.Tensor], name, shape, dtype, device):
    if t is not None:
        _need(t, name, shape, dtype)
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _on(device):
    """Makes `device` current for a launch where it is not."""
    return contextlib.nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _sequences(x, cu_seqlens, device) -> int:
    if cu_seqlens is None:
        return x.shape[0]
    _need(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), torch.int32)
    if cu_seqlens.device != device:
        raise ValueError(f"cu_seqlens is on {cu_seqlens.device}, expected {device}")
    return cu_seqlens.numel() - 1


def _workspace(given, need: int, device):
    if need > 0 and (given is None or given.numel() * given.element_size() < need):
        return torch.empty(need, dtype=torch.uint8, device=device)
    return given


def _call(name: str, args, device):
    args.stream = _stream(device)
    with _on(device):
        _lib.check(_lib.layer_raw(name, args))


# ---- selective scan ------------------------------------------------------------------------------------

def _scan_shapes(u, A, B):
    if u.dim() not in (2, 3) or A.dim() != 2:
        raise ValueError("u must be [B,T,D] (or [N,D] for a step) and A [D,ds]")
    return tuple(u.shape), (*u.shape[:-1], A.shape[1]), u.shape[-1], A.shape[1]


def _scan_args(a, u, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens, dt_softplus):
    """Checks and fills what the scan's three entry points share; returns (device, N, dim, ds)."""
    wide, narrow, dim, ds = _scan_shapes(u, A, B)
    dtype, device = _dtype(u, "u"), u.device
    a.u_stride = _rows(u, "u", wide)
    a.dt_stride = _rows(dt, "dt", wide, dtype, device)
    a.B_stride = _rows(B, "B", narrow, dtype, device)
    a.C_stride = _rows(C, "C", narrow, dtype, device)
    a.z_stride = _opt(z, "z", wide, dtype, device)
    _param(A, "A", (dim, ds), F32, device)
    _param(D, "D", (dim,), F32, device)
    _param(dt_bias, "dt_bias", (dim,), F32, device)
    N = _sequences(u, cu_seqlens, device)
    _param(initial_state, "initial_state", (N, dim, ds), F32, device)
    a.u, a.dt, a.A, a.B, a.C = _ptr(u), _ptr(dt), _ptr(A), _ptr(B), _ptr(C)
    a.D, a.z, a.dt_bias = _ptr(D), _ptr(z), _ptr(dt_bias)
    a.initial_state, a.cu_seqlens = _ptr(initial_state), _ptr(cu_seqlens)
    a.batch, a.T = wide[0], wide[1] if len(wide) == 3 else 1
    a.dim, a.ds, a.num_seqs = dim, ds, N
    a.in_dtype = _DT[dtype]
    a.flags = _lib.KDA_SCAN_DT_SOFTPLUS if dt_softplus else 0
    return device, N, dim, ds


def _scan_sizes(a, u, ds, cu_seqlens):
    a.batch, a.T, a.dim, a.ds = u.shape[0], u.shape[1], u.shape[2], ds
    a.num_seqs = u.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
    a.cu_seqlens = _ptr(cu_seqlens)
    a.in_dtype = _DT[_dtype(u, "u")]
    return a


def selective_scan_fwd_workspace_bytes(u: torch.Tensor, ds: int, cu_seqlens: Optional[torch.Tensor] = None) -> int:
    """Bytes that ``selective_scan_fwd`` needs for u [B,T,D] and ds states per channel."""
    return _lib.layer_workspace("kda_selective_scan_fwd_workspace_bytes",
                                _scan_sizes(_lib.SelectiveScanArgs(), u, ds, cu_seqlens))


def selective_scan_bwd_workspace_bytes(u: torch.Tensor, ds: int, cu_seqlens: Optional[torch.Tensor] = None) -> int:
    """Bytes that ``selective_scan_bwd`` needs for u [B,T,D] and ds states per channel."""
    return _lib.layer_workspace("kda_selective_scan_bwd_workspace_bytes",
                                _scan_sizes(_lib.SelectiveScanBwdArgs(), u, ds, cu_seqlens))


def selective_scan_fwd(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                       D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                       dt_bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                       cu_seqlens: Optional[torch.Tensor] = None, dt_softplus: bool = False,
                       out_dtype: Optional[torch.dtype] = None, output_final_state: bool = True,
                       final_state: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None):
    """Selective state space scan over whole sequences.  Per channel,

        delta = softplus?(dt + dt_bias),  h_t = exp(delta A) h_{t-1} + delta u B_t,
        y_t = (C_t . h_t + D u_t) * silu?(z_t).

    u, dt, z: [B,T,D] (bf16 or fp32); B, C: [B,T,ds]; A: [D,ds], D, dt_bias: [D]
    fp32; initial_state: [N,D,ds] fp32 or None.  cu_seqlens: int32 [N+1] device
    tensor for packed input (B == 1); rows at and behind its last offset are
    left as they were.  ``final_state`` may be ``initial_state``.  Returns
    (y [B,T,D], final_state or None)."""
    a = _lib.SelectiveScanArgs()
    if u.dim() != 3:
        raise ValueError("u must be [B,T,D]")
    device, N, dim, ds = _scan_args(a, u, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens, dt_softplus)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, dim, ds), dtype=F32, device=device)
    _param(final_state, "final_state", (N, dim, ds), F32, device)
    if y is None:
        y = torch.empty(u.shape, dtype=out_dtype or u.dtype, device=device)
    a.y_stride = _rows(y, "y", u.shape, out_dtype, device)
    a.y, a.final_state, a.out_dtype = _ptr(y), _ptr(final_state), _DT[_dtype(y, "y")]
    need = _lib.layer_workspace("kda_selective_scan_fwd_workspace_bytes", a)
    workspace = _workspace(workspace, need, device)
    a.workspace, a.workspace_bytes = (_ptr(workspace), need) if need else (None, 0)
    _call("kda_selective_scan_fwd", a, device)
    return y, final_state


def selective_scan_step(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                        state: Optional[torch.Tensor], D: Optional[torch.Tensor] = None,
                        z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                        dt_softplus: bool = False, final_state: Optional[torch.Tensor] = None,
                        out_dtype: Optional[torch.dtype] = None, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of ``selective_scan_fwd`` for N sequences: u, dt, z [N,D], B, C
    [N,ds], state [N,D,ds] fp32 (or None for zeros).  The new state is written
    to ``final_state`` (default: ``state`` itself, in place).  Returns y [N,D]."""
    a = _lib.SelectiveScanArgs()
    if u.dim() != 2:
        raise ValueError("u must be [N,D]")
    device, N, dim, ds = _scan_args(a, u, dt, A, B, C, D, z, dt_bias, state, None, dt_softplus)
    if final_state is None:
        if state is None:
            raise ValueError("final_state is required when state is None")
        final_state = state
    _param(final_state, "final_state", (N, dim, ds), F32, device)
    if y is None:
        y = torch.empty(u.shape, dtype=out_dtype or u.dtype, device=device)
    a.y_stride = _rows(y, "y", u.shape, out_dtype, device)
    a.y, a.final_state, a.out_dtype = _ptr(y), _ptr(final_state), _DT[_dtype(y, "y")]
    _call("kda_selective_scan_step", a, device)
    return y


def selective_scan_bwd(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                       grad_y: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                       dt_bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                       grad_final_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                       dt_softplus: bool = False, grad_dtype: torch.dtype = F32,
                       output_grad_initial_state: bool = True, grad_initial_state: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None) -> dict:
    """Gradients of ``selective_scan_fwd`` for grad_y [B,T,D] (dtype of u) and the
    optional final-state gradient [N,D,ds] fp32.  Returns a dict: du, ddt, dz
    [B,T,D] and dB, dC [B,T,ds] in ``grad_dtype``; dA [D,ds], dD, ddt_bias [D]
    and dh0 [N,D,ds] in fp32; None for what has no input.  ``out`` may supply
    du, ddt, dB, dC, dz (their rows may be strided, as column slices of one
    buffer); ``grad_initial_state`` may be ``initial_state`` or
    ``grad_final_state``."""
    a = _lib.SelectiveScanBwdArgs()
    if u.dim() != 3:
        raise ValueError("u must be [B,T,D]")
    device, N, dim, ds = _scan_args(a, u, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens, dt_softplus)
    a.grad_y_stride = _rows(grad_y, "grad_y", u.shape, u.dtype, device)
    _param(grad_final_state, "grad_final_state", (N, dim, ds), F32, device)
    if grad_initial_state is None and output_grad_initial_state:
        grad_initial_state = torch.empty((N, dim, ds), dtype=F32, device=device)
    _param(grad_initial_state, "grad_initial_state", (N, dim, ds), F32, device)
    if grad_dtype not in _DT:
        raise ValueError(f"unsupported grad_dtype {grad_dtype}")
    got = {}
    for name, like in (("du", u), ("ddt", u), ("dB", B), ("dC", B), ("dz", z)):
        if like is None:
            got[name] = None
            continue
        t = out[name] if out is not None else torch.empty(like.shape, dtype=grad_dtype, device=device)
        got[name] = t
        stride = _rows(t, name, like.shape, grad_dtype, device)
        field = "grad_" + name[1:]
        setattr(a, field, t.data_ptr())
        setattr(a, field + "_stride", stride)
    got["dA"] = torch.empty((dim, ds), dtype=F32, device=device)
    got["dD"] = None if D is None else torch.empty((dim,), dtype=F32, device=device)
    got["ddt_bias"] = None if dt_bias is None else torch.empty((dim,), dtype=F32, device=device)
    got["dh0"] = grad_initial_state
    a.grad_y, a.grad_final_state, a.grad_initial_state = _ptr(grad_y), _ptr(grad_final_state), _ptr(grad_initial_state)
    a.grad_A, a.grad_D, a.grad_dt_bias = _ptr(got["dA"]), _ptr(got["dD"]), _ptr(got["ddt_bias"])
    a.grad_dtype = _DT[grad_dtype]
    need = _lib.layer_workspace("kda_selective_scan_bwd_workspace_bytes", a)
    workspace = _workspace(workspace, need, device)
    a.workspace, a.workspace_bytes = _ptr(workspace), need
    _call("kda_selective_scan_bwd", a, device)
    return got


# ---- short convolution ---------------------------------------------------------------------------------

def _conv_args(a, x, weight, bias, initial_state, cu_seqlens, silu):
    if x.dim() not in (2, 3) or weight.dim() != 2:
        raise ValueError("x must be [B,T,D] (or [N,D] for a step) and weight [D,W]")
    dtype, device, dim, width = _dtype(x, "x"), x.device, x.shape[-1], weight.shape[1]
    a.x_stride = _rows(x, "x", x.shape)
    _param(weight, "weight", (dim, width), _dtype(weight, "weight"), device)
    _param(bias, "bias", (dim,), weight.dtype, device)
    N = _sequences(x, cu_seqlens, device)
    _param(initial_state, "initial_state", (N, width - 1, dim), dtype, device)
    a.x, a.weight, a.bias = _ptr(x), _ptr(weight), _ptr(bias)
    a.initial_state, a.cu_seqlens = _ptr(initial_state), _ptr(cu_seqlens)
    a.batch, a.T = x.shape[0], x.shape[1] if x.dim() == 3 else 1
    a.dim, a.width, a.num_seqs = dim, width, N
    a.in_dtype, a.w_dtype = _DT[dtype], _DT[weight.dtype]
    a.flags = _lib.KDA_CONV_SILU if silu else 0
    return device, N, dim, width


def short_conv_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                   silu: bool = False, out_dtype: Optional[torch.dtype] = None, output_final_state: bool = True,
                   final_state: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """Short causal depthwise convolution: y_t = act(bias + sum_j weight[:, j] x_{t-W+1+j}).

    x: [B,T,D] (bf16 or fp32); weight: [D,W], W 2 to 4, and bias: [D] in one of
    the two dtypes; initial_state: [N,W-1,D] of x's dtype, each sequence's last
    inputs, oldest first (None: zeros).  cu_seqlens as in
    ``selective_scan_fwd``.  ``final_state`` may be ``initial_state``.  Returns
    (y, final_state or None)."""
    a = _lib.ShortConvArgs()
    if x.dim() != 3:
        raise ValueError("x must be [B,T,D]")
    device, N, dim, width = _conv_args(a, x, weight, bias, initial_state, cu_seqlens, silu)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, width - 1, dim), dtype=x.dtype, device=device)
    _param(final_state, "final_state", (N, width - 1, dim), x.dtype, device)
    if y is None:
        y = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=device)
    a.y_stride = _rows(y, "y", x.shape, out_dtype, device)
    a.y, a.final_state, a.out_dtype = _ptr(y), _ptr(final_state), _DT[_dtype(y, "y")]
    _call("kda_short_conv_fwd", a, device)
    return y, final_state


def short_conv_step(x: torch.Tensor, weight: torch.Tensor, state: Optional[torch.Tensor],
                    bias: Optional[torch.Tensor] = None, silu: bool = False,
                    final_state: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                    y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of ``short_conv_fwd`` for N sequences: x [N,D], state [N,W-1,D]
    (or None for zeros).  The shifted state is written to ``final_state``
    (default: ``state`` itself, in place).  Returns y [N,D]."""
    a = _lib.ShortConvArgs()
    if x.dim() != 2:
        raise ValueError("x must be [N,D]")
    device, N, dim, width = _conv_args(a, x, weight, bias, state, None, silu)
    if final_state is None:
        if state is None:
            raise ValueError("final_state is required when state is None")
        final_state = state
    _param(final_state, "final_state", (N, width - 1, dim), x.dtype, device)
    if y is None:
        y = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=device)
    a.y_stride = _rows(y, "y", x.shape, out_dtype, device)
    a.y, a.final_state, a.out_dtype = _ptr(y), _ptr(final_state), _DT[_dtype(y, "y")]
    _call("kda_short_conv_step", a, device)
    return y


def short_conv_bwd_workspace_bytes(x: torch.Tensor, width: int, cu_seqlens: Optional[torch.Tensor] = None) -> int:
    """Bytes that ``short_conv_bwd`` needs for x [B,T,D] and `width` taps."""
    a = _lib.ShortConvBwdArgs()
    a.batch, a.T, a.dim, a.width = x.shape[0], x.shape[1], x.shape[2], width
    a.num_seqs = x.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
    a.cu_seqlens = _ptr(cu_seqlens)
    a.in_dtype = _DT[_dtype(x, "x")]
    return _lib.layer_workspace("kda_short_conv_bwd_workspace_bytes", a)


def short_conv_bwd(x: torch.Tensor, weight: torch.Tensor, grad_y: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   initial_state: Optional[torch.Tensor] = None, grad_final_state: Optional[torch.Tensor] = None,
                   cu_seqlens: Optional[torch.Tensor] = None, silu: bool = False, grad_dtype: torch.dtype = F32,
                   output_grad_initial_state: bool = True, grad_initial_state: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None) -> dict:
    """Gradients of ``short_conv_fwd`` for grad_y [B,T,D] (dtype of x) and the
    optional final-state gradient [N,W-1,D] fp32.  Returns a dict: dx in
    ``grad_dtype`` (``out`` may supply it), dweight, dbias (None without a bias)
    and dh0 [N,W-1,D] in fp32 (``grad_initial_state`` may be
    ``grad_final_state``)."""
    a = _lib.ShortConvBwdArgs()
    if x.dim() != 3:
        raise ValueError("x must be [B,T,D]")
    device, N, dim, width = _conv_args(a, x, weight, bias, initial_state, cu_seqlens, silu)
    a.grad_y_stride = _rows(grad_y, "grad_y", x.shape, x.dtype, device)
    _param(grad_final_state, "grad_final_state", (N, width - 1, dim), F32, device)
    if grad_initial_state is None and output_grad_initial_state:
        grad_initial_state = torch.empty((N, width - 1, dim), dtype=F32, device=device)
    _param(grad_initial_state, "grad_initial_state", (N, width - 1, dim), F32, device)
    if grad_dtype not in _DT:
        raise ValueError(f"unsupported grad_dtype {grad_dtype}")
    dx = out["dx"] if out is not None else torch.empty(x.shape, dtype=grad_dtype, device=device)
    a.grad_x_stride = _rows(dx, "dx", x.shape, grad_dtype, device)
    got = dict(dx=dx, dweight=torch.empty((dim, width), dtype=F32, device=device),
               dbias=None if bias is None else torch.empty((dim,), dtype=F32, device=device), dh0=grad_initial_state)
    a.grad_y, a.grad_final_state, a.grad_initial_state = _ptr(grad_y), _ptr(grad_final_state), _ptr(grad_initial_state)
    a.grad_x, a.grad_weight, a.grad_bias = _ptr(dx), _ptr(got["dweight"]), _ptr(got["dbias"])
    a.grad_dtype = _DT[grad_dtype]
    need = _lib.layer_workspace("kda_short_conv_bwd_workspace_bytes", a)
    workspace = _workspace(workspace, need, device)
    a.workspace, a.workspace_bytes = _ptr(workspace), need
    _call("kda_short_conv_bwd", a, device)
    return got


# ---- layer norm ----------------------------------------------------------------------------------------

def layer_norm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                   residual: Optional[torch.Tensor] = None, eps: float = 1e-5,
                   out_dtype: Optional[torch.dtype] = None, y: Optional[torch.Tensor] = None,
                   residual_out: Optional[torch.Tensor] = None):
    """Layer norm over the last dimension (1 to 16384) of x [..., D]; weight and
    bias [D] share a dtype.  With ``residual`` [..., D] (bf16 or fp32) x +
    residual is normalised and also returned, in the residual's dtype
    (``residual_out`` may be ``residual``).  Returns y, or (y, residual_out)."""
    a = _lib.LayerNormArgs()
    dtype, device, dim = _dtype(x, "x"), x.device, x.shape[-1]
    a.x_stride = _rows(x, "x", x.shape)
    w = weight if weight is not None else bias
    wd = F32 if w is None else _dtype(w, "weight")
    _param(weight, "weight", (dim,), wd, device)
    _param(bias, "bias", (dim,), wd, device)
    if y is None:
        y = torch.empty(x.shape, dtype=out_dtype or dtype, device=device)
    a.y_stride = _rows(y, "y", x.shape, out_dtype, device)
    if residual is not None:
        rd = _dtype(residual, "residual")
        a.residual_stride = _rows(residual, "residual", x.shape, rd, device)
        if residual_out is None:
            residual_out = torch.empty(x.shape, dtype=rd, device=device)
        a.residual_out_stride = _rows(residual_out, "residual_out", x.shape, rd, device)
        a.residual, a.residual_out, a.res_dtype = _ptr(residual), _ptr(residual_out), _DT[rd]
    a.x, a.weight, a.bias, a.y = _ptr(x), _ptr(weight), _ptr(bias), _ptr(y)
    a.rows, a.dim, a.eps = x.numel() // dim if dim else 0, dim, eps
    a.x_dtype, a.w_dtype, a.out_dtype = _DT[dtype], _DT[wd], _DT[_dtype(y, "y")]
    _call("kda_layer_norm_fwd", a, device)
    return y if residual is None else (y, residual_out)


def layer_norm_bwd_workspace_bytes(x: torch.Tensor) -> int:
    """Bytes that ``layer_norm_bwd`` needs for x [..., D] with a weight or bias gradient."""
    a = _lib.LayerNormBwdArgs()
    a.dim = x.shape[-1]
    a.rows = x.numel() // a.dim if a.dim else 0
    a.grad_weight = 1
    return _lib.layer_workspace("kda_layer_norm_bwd_workspace_bytes", a)


def layer_norm_bwd(x: torch.Tensor, grad_y: torch.Tensor, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, grad_residual: Optional[torch.Tensor] = None,
                   eps: float = 1e-5, grad_dtype: torch.dtype = F32, workspace: Optional[torch.Tensor] = None,
                   out: Optional[dict] = None) -> dict:
    """Gradients of ``layer_norm_fwd`` for grad_y [..., D].  x is what was
    normalised (the returned residual where one was added); its mean and
    variance are computed again.  ``grad_residual`` [..., D] is the gradient that
    reaches the residual stream from behind; it is added to dx.  Returns a dict:
    dx in ``grad_dtype`` (``out`` may supply it; with a residual it is the
    gradient of both summands), dweight and dbias [D] fp32 (None where the
    parameter is None)."""
    a = _lib.LayerNormBwdArgs()
    dtype, device, dim = _dtype(x, "x"), x.device, x.shape[-1]
    a.x_stride = _rows(x, "x", x.shape)
    a.grad_y_stride = _rows(grad_y, "grad_y", x.shape, _dtype(grad_y, "grad_y"), device)
    w = weight if weight is not None else bias
    wd = F32 if w is None else _dtype(w, "weight")
    _param(weight, "weight", (dim,), wd, device)
    _param(bias, "bias", (dim,), wd, device)
    if grad_residual is not None:
        a.grad_residual_stride = _rows(grad_residual, "grad_residual", x.shape, _dtype(grad_residual, "grad_residual"), device)
        a.grad_residual, a.res_dtype = _ptr(grad_residual), _DT[grad_residual.dtype]
    if grad_dtype not in _DT:
        raise ValueError(f"unsupported grad_dtype {grad_dtype}")
    dx = out["dx"] if out is not None else torch.empty(x.shape, dtype=grad_dtype, device=device)
    a.grad_x_stride = _rows(dx, "dx", x.shape, grad_dtype, device)
    got = dict(dx=dx, dweight=None if weight is None else torch.empty((dim,), dtype=F32, device=device),
               dbias=None if bias is None else torch.empty((dim,), dtype=F32, device=device))
    a.x, a.grad_y, a.weight = _ptr(x), _ptr(grad_y), _ptr(weight)
    a.grad_x, a.grad_weight, a.grad_bias = _ptr(dx), _ptr(got["dweight"]), _ptr(got["dbias"])
    a.rows, a.dim, a.eps = x.numel() // dim if dim else 0, dim, eps
    a.x_dtype, a.gy_dtype, a.w_dtype, a.grad_dtype = _DT[dtype], _DT[grad_y.dtype], _DT[wd], _DT[grad_dtype]
    need = _lib.layer_workspace("kda_layer_norm_bwd_workspace_bytes", a)
    workspace = _workspace(workspace, need, device)
    a.workspace, a.workspace_bytes = (_ptr(workspace), need) if need else (None, 0)
    _call("kda_layer_norm_bwd", a, device)
    return got
