"""Latent attention's C entry points where a tensor has one row, or one head: its stride is not looked at, whatever it holds."""
import ctypes

import pytest

from test_gpu_latent import kda, make, tdtype  # noqa: F401

pytestmark = pytest.mark.gpu

STRIDES = [0, 8, 64, -8, 1 << 31, (1 << 40) - 8]


def call(name, struct, **kw):
    import torch
    from gated_delta_rule_52_amd import _lib
    a = struct()
    a.struct_size = ctypes.sizeof(a)
    a.stream = torch.cuda.current_stream().cuda_stream
    for k, v in kw.items():
        setattr(a, k, v.data_ptr() if isinstance(v, torch.Tensor) else v)
    return _lib.layer_raw(name, a)


def both_directions(kda, x, dtype, causal, odd):
    """Outputs and gradients of contiguous tensors; odd: stride fields that replace the tensors' own."""
    import torch
    from gated_delta_rule_52_amd import _lib
    (B, Tq, H, _), Tk = x["q"].shape, x["k"].shape[1]
    dn, dr, dv = x["k"].shape[-1], x["k_rope"].shape[-1], x["v"].shape[-1]
    kind = _lib.KDA_DTYPE_BF16 if dtype == "bf16" else _lib.KDA_DTYPE_FP32
    new = lambda *s: torch.full(s, 7.0, dtype=tdtype(dtype), device="cuda")  # noqa: E731
    o, lse = new(B, Tq, H, dv), torch.full((B, Tq, H), 7.0, device="cuda")
    grads = dict(grad_q=new(B, Tq, H, dn + dr), grad_k=new(B, Tk, H, dn), grad_k_rope=new(B, Tk, dr), grad_v=new(B, Tk, H, dv))

    def strides(**tensors):
        got = {}
        for n, t in tensors.items():
            got[n + "_stride"] = t[0, 0].numel()
            if t.dim() == 4:
                got[n + "_head_stride"] = t.shape[-1]
        return {k: odd.get(k, v) for k, v in got.items()}

    sizes = dict(batch=B, Tq=Tq, Tk=Tk, H=H, dn=dn, dr=dr, dv=dv, num_seqs=B, scale=0.1, in_dtype=kind, flags=1 if causal else 0)
    assert call("kda_latent_attention_fwd", _lib.LatentAttentionArgs, **{n: x[n] for n in ("q", "k", "k_rope", "v")}, o=o, lse=lse,
                **strides(**{n: x[n] for n in ("q", "k", "k_rope", "v")}, o=o), **sizes, out_dtype=kind) == 0
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    assert call("kda_latent_attention_bwd", _lib.LatentAttentionBwdArgs, **x, o=o, lse=lse, **grads, **strides(**x, o=o, **grads), **sizes,
                grad_dtype=kind, workspace=ws, workspace_bytes=ws.numel()) == 0
    return [o, lse, *grads.values()]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Tq,Tk,H,dims", [(1, 200, 2, (128, 64, 128)), (130, 1, 2, (128, 64, 128)), (1, 1, 3, (64, 32, 64)), (1, 90, 1, (64, 32, 64)),
                                          (70, 40, 1, (72, 24, 104))])
def test_strides_of_single_rows_and_heads(kda, dtype, causal, Tq, Tk, H, dims):  # noqa: F811
    import torch
    dn, dr, dv = dims
    x = dict(q=make(1, (1, Tq, H, dn + dr), dtype), k=make(2, (1, Tk, H, dn), dtype), k_rope=make(3, (1, Tk, dr), dtype),
             v=make(4, (1, Tk, H, dv), dtype), grad_o=make(5, (1, Tq, H, dv), dtype))
    want = both_directions(kda, x, dtype, causal, {})
    of_q, of_k = ("q", "o", "grad_o", "grad_q"), ("k", "k_rope", "v", "grad_k", "grad_k_rope", "grad_v")
    for s in STRIDES:
        odd = {n + "_stride": s for n in (of_q if Tq == 1 else ()) + (of_k if Tk == 1 else ())}
        if H == 1:
            odd.update({n + "_head_stride": s for n in of_q + of_k})
        got = both_directions(kda, x, dtype, causal, odd)
        assert [torch.equal(a, b) for a, b in zip(want, got)] == [True] * len(want), s
