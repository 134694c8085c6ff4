"""Outputs of latent attention as slices of one buffer, in every layout that the strides can say: the bits of separate outputs,
and nothing written beside them."""
import pytest

from test_gpu_latent import ints, kda, make, tdtype  # noqa: F401

pytestmark = pytest.mark.gpu


def buffers(T, H, width, dtype):
    """[1, T, H, width] views of buffers of sevens: dense, in rows that are padded, heads in front of rows."""
    import torch
    new = lambda *s: torch.full(s, 7.0, dtype=tdtype(dtype), device="cuda")  # noqa: E731
    dense, padded, heads = new(T, H, width), new(T, H * width + 24), new(H, T, width)
    return dict(dense=(dense, dense[None]), padded=(padded, padded[:, :H * width].view(T, H, width)[None]), heads=(heads, heads.transpose(0, 1)[None]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_of_keys_and_values(kda, dtype):  # noqa: F811
    import torch
    T, H, dn, dr, dv = 90, 3, 64, 32, 56
    q, k, kr, v, go = (make(i, (1, T, *s), dtype) for i, s in enumerate(((H, dn + dr), (H, dn), (dr,), (H, dv), (H, dv))))
    o, lse = kda.latent_attention_fwd(q, k, kr, v)
    want = kda.latent_attention_bwd(q, k, kr, v, o, lse, go, grad_dtype=tdtype(dtype))
    for name, (buffer, view) in buffers(T, H, dn + dv + 8, dtype).items():
        out = dict(dq=torch.empty_like(q), dk_rope=torch.empty_like(kr), dk=view[..., :dn], dv=view[..., dn:dn + dv])
        got = kda.latent_attention_bwd(q, k, kr, v, o, lse, go, grad_dtype=tdtype(dtype), out=out)
        assert all(torch.equal(got[n], want[n]) for n in want), name
        assert (view[..., dn + dv:] == 7).all() and int((buffer == 7).sum()) >= buffer.numel() - T * H * (dn + dv), name


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rotation_beside_its_input(kda, dtype):  # noqa: F811
    import torch
    T, H, D = 37, 3, 96
    x, f = make(9, (1, T, H, D), dtype), kda.rotary_frequencies(32)[0]
    pos = ints(range(T)).view(1, T)
    want = kda.rotary_fwd(x, pos, f, offset=8)
    for name, (_, view) in buffers(T, H, 2 * D + 8, dtype).items():
        view[..., :D] = x
        y = view[..., D:2 * D]
        assert kda.rotary_fwd(view[..., :D], pos, f, offset=8, y=y) is y
        assert torch.equal(y, want) and torch.equal(view[..., :D], x) and (view[..., 2 * D:] == 7).all(), name
