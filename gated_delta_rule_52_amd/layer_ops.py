"""Torch-facing wrappers of the layer operators in include/kda.h: selective
state space scan, short causal convolution and layer norm.

As in ops.py, torch supplies device memory and the current HIP stream and every
step runs in libkda.so.  Token tensors may be column slices of wider ones: the
last dimension must be dense and the rows equally spaced.

A decode step's kernels take a few microseconds, so the checks here look at a
tensor once, in one condition, and work out what was wrong only where it fails;
argument structs are packed by position, in the order of their fields.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .ops import _DT

F32 = torch.float32
_TOO_BIG = 2 ** 64 - 1
_SCAN, _SCAN_BWD = _lib.packer(_lib.SelectiveScanArgs), _lib.packer(_lib.SelectiveScanBwdArgs)
_CONV, _CONV_BWD = _lib.packer(_lib.ShortConvArgs), _lib.packer(_lib.ShortConvBwdArgs)
_NORM, _NORM_BWD = _lib.packer(_lib.LayerNormArgs), _lib.packer(_lib.LayerNormBwdArgs)


def _refuse(t, name, shape, dtype, device):
    """The reason why a tensor failed its check."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} must be contiguous")


def _kind(t, name: str) -> int:
    """The C dtype of a tensor, or of None as fp32."""
    if t is None:
        return _lib.KDA_DTYPE_FP32
    kind = _DT.get(t.dtype)
    if kind is None:
        raise ValueError(f"unsupported {name} dtype {t.dtype}")
    return kind


def _first(t, name: str, dims) -> torch.device:
    """Checks the tensor that sets a call's device."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() not in dims:
        raise ValueError(f"{name} has {t.dim()} dimensions, expected {' or '.join(map(str, dims))}")
    if t.shape[-1] >> 31:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected sizes below 2^31")
    return t.device


def _step(t, name, shape, dtype, device) -> int:
    """Checks a token tensor (None: 0) and returns the distance between its rows in elements."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        _refuse(t, name, shape, dtype, device)
    width = shape[-1]
    if t.is_contiguous():
        return width
    strides = t.stride()
    if width != 1 and strides[-1] != 1:
        raise ValueError(f"{name} must be dense along its last dimension")
    step, span = None, 1  # of the innermost leading dimension with more than one entry, and the rows inside
    for size, stride in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if size == 1:
            continue
        if step is None:
            step = stride
        elif stride != span * step:
            raise ValueError(f"the rows of {name} must be equally spaced")
        span *= size
    return width if step is None else step


def _at(t, name, shape, dtype, device):
    """Checks a contiguous tensor (or None) and returns its address."""
    if t is None:
        return 0
    if t.dtype is not dtype or tuple(t.shape) != shape or t.device != device or not t.is_contiguous():
        _refuse(t, name, shape, dtype, device)
    return t.data_ptr()


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _new(like, shape, dtype):
    """An output of `like`'s device, and its type where dtype is None."""
    if dtype is None and like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(shape, dtype=dtype or like.dtype, device=like.device)


def _sequences(x, cu_seqlens, device):
    """(number of sequences, address of the offsets) of tokens [B,T,D] or [N,D]"""
    if x.numel() >> 31 and max(x.shape) >> 31:  # the structs' sizes are int32
        raise ValueError(f"the tokens have shape {tuple(x.shape)}, expected sizes below 2^31")
    if cu_seqlens is None:
        return x.shape[0], 0
    return cu_seqlens.numel() - 1, _at(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), torch.int32, device)


def _stream(device) -> int:
    # the address alone, without a Stream object around it (1.8 us less per call)
    return torch._C._cuda_getCurrentRawStream(device.index)


def _call(name: str, args: bytes, device):
    if torch.cuda.current_device() == device.index:
        status = _lib.layer_function(name)(args)
    else:  # a launch goes to the current device
        with torch.cuda.device(device):
            status = _lib.layer_function(name)(args)
    if status:
        _lib.check(status)


def _size(name: str, args: bytes) -> int:
    """A workspace query; invalid sizes raise."""
    need = _lib.layer_function(name)(args)
    if need == _TOO_BIG:
        raise _lib.KdaError(_lib.STATUS_CODE["KDA_ERR_BAD_SHAPE"], _lib.load().kda_last_error().decode())
    return need


def _call_with_workspace(name: str, pack, front, back, workspace, device):
    """Calls an entry point whose struct has workspace and workspace_bytes between `front` and `back`, with a
    workspace of the size that it asks for."""
    need = _size(name + "_workspace_bytes", pack(*front, 0, 0, *back))
    at = 0
    if need:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        elif workspace.device != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the call's device")
        elif workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        at = workspace.data_ptr()
    _call(name, pack(*front, at, need, *back), device)


def _grad_dtype(dtype) -> int:
    kind = _DT.get(dtype)
    if kind is None:
        raise ValueError(f"unsupported grad_dtype {dtype}")
    return kind


# ---- selective scan ------------------------------------------------------------------------------------

def _fields(struct, **values) -> bytes:
    """A packed struct from its fields by name, the others zero."""
    values["struct_size"] = _lib.packer(struct).size
    return _lib.packer(struct).pack(*(values.get(name, 0) for name, _ in struct._fields_))


def _batch(x, name, cu_seqlens):
    device = _first(x, name, (3,))
    N, cu = _sequences(x, cu_seqlens, device)
    return dict(cu_seqlens=cu, batch=x.shape[0], T=x.shape[1], dim=x.shape[2], num_seqs=N, in_dtype=_kind(x, name))


def selective_scan_fwd_workspace_bytes(u: torch.Tensor, ds: int, cu_seqlens: Optional[torch.Tensor] = None) -> int:
    """Bytes that ``selective_scan_fwd`` needs for u [B,T,D] and ds states per channel."""
    return _size("kda_selective_scan_fwd_workspace_bytes",
                 _fields(_lib.SelectiveScanArgs, ds=ds, **_batch(u, "u", cu_seqlens)))


def selective_scan_bwd_workspace_bytes(u: torch.Tensor, ds: int, cu_seqlens: Optional[torch.Tensor] = None) -> int:
    """Bytes that ``selective_scan_bwd`` needs for u [B,T,D] and ds states per channel."""
    return _size("kda_selective_scan_bwd_workspace_bytes",
                 _fields(_lib.SelectiveScanBwdArgs, ds=ds, **_batch(u, "u", cu_seqlens)))


def _scan(u, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens, dt_softplus, out_dtype, final_state,
          output_final_state, y):
    """Checks the arguments of the scan's forward and step; returns (the struct's fields before the workspace, behind
    it, y, final state, device)."""
    device = _first(u, "u", (2, 3))
    shape, dtype = u.shape, u.dtype
    kind = _kind(u, "u")
    if A.dim() != 2:
        raise ValueError("A must be [D,ds]")
    dim, ds = shape[-1], A.shape[1]
    narrow = shape[:-1] + (ds,)
    N, cu = _sequences(u, cu_seqlens, device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, dim, ds), dtype=F32, device=device)
    if y is None:
        y = _new(u, shape, out_dtype)
    front = (
        _SCAN.size, u.data_ptr(), dt.data_ptr(), _at(A, "A", (dim, ds), F32, device),
        B.data_ptr(), C.data_ptr(), _at(D, "D", (dim,), F32, device), _ptr(z),
        _at(dt_bias, "dt_bias", (dim,), F32, device), _at(initial_state, "initial_state", (N, dim, ds), F32, device),
        _at(final_state, "final_state", (N, dim, ds), F32, device), y.data_ptr(), cu,
        _step(u, "u", shape, dtype, device), _step(dt, "dt", shape, dtype, device),
        _step(B, "B", narrow, dtype, device), _step(C, "C", narrow, dtype, device),
        _step(z, "z", shape, dtype, device), _step(y, "y", shape, out_dtype or y.dtype, device),
        shape[0], shape[1] if len(shape) == 3 else 1, dim, ds, N, kind, _kind(y, "y"))
    return front, (_stream(device), _lib.KDA_SCAN_DT_SOFTPLUS if dt_softplus else 0), y, final_state, device


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
    if u.dim() != 3:
        raise ValueError("u must be [B,T,D]")
    front, back, y, final_state, device = _scan(u, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens, dt_softplus,
                                                out_dtype, final_state, output_final_state, y)
    _call_with_workspace("kda_selective_scan_fwd", _SCAN.pack, front, back, workspace, device)
    return y, final_state


def selective_scan_step(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                        state: Optional[torch.Tensor], D: Optional[torch.Tensor] = None,
                        z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                        dt_softplus: bool = False, final_state: Optional[torch.Tensor] = None,
                        out_dtype: Optional[torch.dtype] = None, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of ``selective_scan_fwd`` for N sequences: u, dt, z [N,D], B, C
    [N,ds], state [N,D,ds] fp32 (or None for zeros).  The new state is written
    to ``final_state`` (default: ``state`` itself, in place).  Returns y [N,D]."""
    if u.dim() != 2:
        raise ValueError("u must be [N,D]")
    if final_state is None:
        if state is None:
            raise ValueError("final_state is required when state is None")
        final_state = state
    front, back, y, _, device = _scan(u, dt, A, B, C, D, z, dt_bias, state, None, dt_softplus, out_dtype, final_state,
                                      False, y)
    _call("kda_selective_scan_step", _SCAN.pack(*front, 0, 0, *back), device)
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
    device = _first(u, "u", (3,))
    shape, dtype = u.shape, u.dtype
    kind, grad_kind = _kind(u, "u"), _grad_dtype(grad_dtype)
    if A.dim() != 2:
        raise ValueError("A must be [D,ds]")
    dim, ds = shape[-1], A.shape[1]
    narrow = shape[:-1] + (ds,)
    N, cu = _sequences(u, cu_seqlens, device)
    states = (N, dim, ds)
    if grad_initial_state is None and output_grad_initial_state:
        grad_initial_state = torch.empty(states, dtype=F32, device=device)
    if out is None:
        new = lambda s: torch.empty(s, dtype=grad_dtype, device=device)  # noqa: E731
        out = dict(du=new(shape), ddt=new(shape), dB=new(narrow), dC=new(narrow), dz=None if z is None else new(shape))
    got = dict(du=out["du"], ddt=out["ddt"], dB=out["dB"], dC=out["dC"], dz=None if z is None else out["dz"],
               dA=torch.empty((dim, ds), dtype=F32, device=device),
               dD=None if D is None else torch.empty((dim,), dtype=F32, device=device),
               ddt_bias=None if dt_bias is None else torch.empty((dim,), dtype=F32, device=device),
               dh0=grad_initial_state)
    grads = (got["du"], got["ddt"], got["dB"], got["dC"], got["dz"])
    steps = [_step(t, n, s, grad_dtype, device) for t, n, s in
             zip(grads, ("du", "ddt", "dB", "dC", "dz"), (shape, shape, narrow, narrow, shape))]
    front = (
        _SCAN_BWD.size, u.data_ptr(), dt.data_ptr(), _at(A, "A", (dim, ds), F32, device),
        B.data_ptr(), C.data_ptr(), _at(D, "D", (dim,), F32, device), _ptr(z),
        _at(dt_bias, "dt_bias", (dim,), F32, device), _at(initial_state, "initial_state", states, F32, device),
        grad_y.data_ptr(), _at(grad_final_state, "grad_final_state", states, F32, device),
        got["du"].data_ptr(), got["ddt"].data_ptr(), got["dA"].data_ptr(), got["dB"].data_ptr(), got["dC"].data_ptr(),
        _ptr(got["dD"]), _ptr(got["dz"]), _ptr(got["ddt_bias"]),
        _at(grad_initial_state, "grad_initial_state", states, F32, device), cu,
        _step(u, "u", shape, dtype, device), _step(dt, "dt", shape, dtype, device),
        _step(B, "B", narrow, dtype, device), _step(C, "C", narrow, dtype, device),
        _step(z, "z", shape, dtype, device), _step(grad_y, "grad_y", shape, dtype, device), *steps,
        shape[0], shape[1], dim, ds, N, kind, grad_kind)
    back = _stream(device), _lib.KDA_SCAN_DT_SOFTPLUS if dt_softplus else 0
    _call_with_workspace("kda_selective_scan_bwd", _SCAN_BWD.pack, front, back, workspace, device)
    return got


# ---- short convolution ---------------------------------------------------------------------------------

def _conv(x, weight, bias, initial_state, cu_seqlens, silu, out_dtype, final_state, output_final_state, y):
    """Checks and packs the arguments of the convolution's forward and step; returns (args, y, final state, device)."""
    device = _first(x, "x", (2, 3))
    shape, dtype = x.shape, x.dtype
    kind = _kind(x, "x")
    if weight.dim() != 2:
        raise ValueError("weight must be [D,W]")
    dim, width = shape[-1], weight.shape[1]
    N, cu = _sequences(x, cu_seqlens, device)
    states = (N, width - 1, dim)
    if final_state is None and output_final_state:
        final_state = torch.empty(states, dtype=dtype, device=device)
    if y is None:
        y = _new(x, shape, out_dtype)
    a = _CONV.pack(
        _CONV.size, x.data_ptr(), _at(weight, "weight", (dim, width), weight.dtype, device),
        _at(bias, "bias", (dim,), weight.dtype, device), _at(initial_state, "initial_state", states, dtype, device),
        _at(final_state, "final_state", states, dtype, device), y.data_ptr(), cu, _step(x, "x", shape, dtype, device),
        _step(y, "y", shape, out_dtype or y.dtype, device), shape[0], shape[1] if len(shape) == 3 else 1, dim, width, N,
        kind, _kind(y, "y"), _kind(weight, "weight"), _stream(device), _lib.KDA_CONV_SILU if silu else 0)
    return a, y, final_state, device


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
    if x.dim() != 3:
        raise ValueError("x must be [B,T,D]")
    a, y, final_state, device = _conv(x, weight, bias, initial_state, cu_seqlens, silu, out_dtype, final_state,
                                      output_final_state, y)
    _call("kda_short_conv_fwd", a, device)
    return y, final_state


def short_conv_step(x: torch.Tensor, weight: torch.Tensor, state: Optional[torch.Tensor],
                    bias: Optional[torch.Tensor] = None, silu: bool = False,
                    final_state: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                    y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of ``short_conv_fwd`` for N sequences: x [N,D], state [N,W-1,D]
    (or None for zeros).  The shifted state is written to ``final_state``
    (default: ``state`` itself, in place).  Returns y [N,D]."""
    if x.dim() != 2:
        raise ValueError("x must be [N,D]")
    if final_state is None:
        if state is None:
            raise ValueError("final_state is required when state is None")
        final_state = state
    a, y, _, device = _conv(x, weight, bias, state, None, silu, out_dtype, final_state, False, y)
    _call("kda_short_conv_step", a, device)
    return y


def short_conv_bwd_workspace_bytes(x: torch.Tensor, width: int, cu_seqlens: Optional[torch.Tensor] = None) -> int:
    """Bytes that ``short_conv_bwd`` needs for x [B,T,D] and `width` taps."""
    return _size("kda_short_conv_bwd_workspace_bytes",
                 _fields(_lib.ShortConvBwdArgs, width=width, **_batch(x, "x", cu_seqlens)))


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
    device = _first(x, "x", (3,))
    shape, dtype = x.shape, x.dtype
    kind, grad_kind = _kind(x, "x"), _grad_dtype(grad_dtype)
    if weight.dim() != 2:
        raise ValueError("weight must be [D,W]")
    dim, width = shape[-1], weight.shape[1]
    N, cu = _sequences(x, cu_seqlens, device)
    states = (N, width - 1, dim)
    if grad_initial_state is None and output_grad_initial_state:
        grad_initial_state = torch.empty(states, dtype=F32, device=device)
    dx = out["dx"] if out is not None else torch.empty(shape, dtype=grad_dtype, device=device)
    got = dict(dx=dx, dweight=torch.empty((dim, width), dtype=F32, device=device),
               dbias=None if bias is None else torch.empty((dim,), dtype=F32, device=device), dh0=grad_initial_state)
    front = (
        _CONV_BWD.size, x.data_ptr(), _at(weight, "weight", (dim, width), weight.dtype, device),
        _at(bias, "bias", (dim,), weight.dtype, device), _at(initial_state, "initial_state", states, dtype, device),
        grad_y.data_ptr(), _at(grad_final_state, "grad_final_state", states, F32, device), dx.data_ptr(),
        got["dweight"].data_ptr(), _ptr(got["dbias"]),
        _at(grad_initial_state, "grad_initial_state", states, F32, device), cu, _step(x, "x", shape, dtype, device),
        _step(grad_y, "grad_y", shape, dtype, device), _step(dx, "dx", shape, grad_dtype, device), shape[0], shape[1],
        dim, width, N, kind, grad_kind, _kind(weight, "weight"))
    back = _stream(device), _lib.KDA_CONV_SILU if silu else 0
    _call_with_workspace("kda_short_conv_bwd", _CONV_BWD.pack, front, back, workspace, device)
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
    device = _first(x, "x", range(1, 9))
    shape, dtype, dim = x.shape, x.dtype, x.shape[-1]
    kind = _kind(x, "x")
    w = weight if weight is not None else bias
    wd = F32 if w is None else w.dtype
    if y is None:
        y = _new(x, shape, out_dtype)
    if residual is not None and residual_out is None:
        residual_out = _new(residual, shape, None)
    rd = F32 if residual is None else residual.dtype
    a = _NORM.pack(
        _NORM.size, x.data_ptr(), _ptr(residual), _at(weight, "weight", (dim,), wd, device),
        _at(bias, "bias", (dim,), wd, device), y.data_ptr(), _ptr(residual_out), _step(x, "x", shape, dtype, device),
        _step(residual, "residual", shape, rd, device), _step(y, "y", shape, out_dtype or y.dtype, device),
        _step(residual_out, "residual_out", shape, rd, device), x.numel() // dim if dim else 0, dim, eps, kind,
        _kind(residual, "residual"), _kind(w, "weight"), _kind(y, "y"), _stream(device))
    _call("kda_layer_norm_fwd", a, device)
    return y if residual is None else (y, residual_out)


def layer_norm_bwd_workspace_bytes(x: torch.Tensor) -> int:
    """Bytes that ``layer_norm_bwd`` needs for x [..., D] with a weight or bias gradient."""
    dim = x.shape[-1]
    return _size("kda_layer_norm_bwd_workspace_bytes",
                 _fields(_lib.LayerNormBwdArgs, dim=dim, rows=x.numel() // dim if dim else 0, grad_weight=1))


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
    device = _first(x, "x", range(1, 9))
    shape, dtype, dim = x.shape, x.dtype, x.shape[-1]
    kind, grad_kind = _kind(x, "x"), _grad_dtype(grad_dtype)
    w = weight if weight is not None else bias
    wd = F32 if w is None else w.dtype
    gd = grad_y.dtype
    rd = F32 if grad_residual is None else grad_residual.dtype
    dx = out["dx"] if out is not None else torch.empty(shape, dtype=grad_dtype, device=device)
    got = dict(dx=dx, dweight=None if weight is None else torch.empty((dim,), dtype=F32, device=device),
               dbias=None if bias is None else torch.empty((dim,), dtype=F32, device=device))
    _at(bias, "bias", (dim,), wd, device)
    front = (
        _NORM_BWD.size, x.data_ptr(), grad_y.data_ptr(), _at(weight, "weight", (dim,), wd, device),
        _ptr(grad_residual), dx.data_ptr(), _ptr(got["dweight"]), _ptr(got["dbias"]), _step(x, "x", shape, dtype, device),
        _step(grad_y, "grad_y", shape, gd, device), _step(grad_residual, "grad_residual", shape, rd, device),
        _step(dx, "dx", shape, grad_dtype, device), x.numel() // dim if dim else 0, dim, eps, kind,
        _kind(grad_y, "grad_y"), _kind(grad_residual, "grad_residual"), _kind(w, "weight"), grad_kind)
    _call_with_workspace("kda_layer_norm_bwd", _NORM_BWD.pack, front, (_stream(device),), workspace, device)
    return got
