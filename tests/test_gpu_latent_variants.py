"""Attention over prompts where its other compiled forms run: fp32 with four waves to a tile (above 512 workgroups) at both head
sizes, bf16 over more than 1,000 keys at both, against 64 bits."""
import pytest

from test_gpu_latent import check_bwd, check_fwd, kda  # noqa: F401

pytestmark = pytest.mark.gpu

LARGE, SMALL = (128, 64, 128), (64, 32, 64)
PACKED = ([513, 0, 200, 1, 700], [513, 4, 300, 1, 650])


@pytest.mark.parametrize("dims", [LARGE, SMALL, (72, 24, 104), (40, 24, 56)], ids=str)
def test_fp32_with_many_workgroups(kda, dims):  # noqa: F811
    """16 heads of 1,100 rows: 560 tiles of 32 queries and as many of keys."""
    check_bwd(kda, 300, (1, 1100, 1100), 16, dims, "fp32", True)


@pytest.mark.parametrize("dims", [LARGE, SMALL], ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_fp32_with_many_workgroups_packed(kda, dims, causal):  # noqa: F811
    """1,414 queries of 14 heads in sequences with lengths of their own."""
    check_bwd(kda, 310, PACKED, 14, dims, "fp32", causal, layout="sliced", extra=9)


@pytest.mark.parametrize("dims", [LARGE, SMALL, (128, 8, 16)], ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_bf16_over_many_keys(kda, dims, causal):  # noqa: F811
    check_bwd(kda, 320, (1, 900, 1300), 2, dims, "bf16", causal)
    check_bwd(kda, 330, PACKED, 3, dims, "bf16", causal, layout="sliced", extra=9)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_long_prompts(kda, dtype):  # noqa: F811
    check_fwd(kda, 340, (1, 130, 4100), 2, LARGE, dtype, True)
    check_bwd(kda, 350, (1, 2100, 2100), 1, SMALL, dtype, True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_in_front_of_the_first_sequence(kda, dtype):  # noqa: F811
    """NaN there enters nothing, and outputs keep what they hold there: the bits of a call without those rows elsewhere."""
    import torch
    from test_gpu_latent import ints, make, tdtype
    H, (dn, dr, dv), front = 3, LARGE, 141
    off_q, off_k = [0, 150, 150, 331], [0, 130, 140, 333]
    x = {n: make(360 + i, (1, T, *s), dtype) for i, (n, T, s) in enumerate((
        ("q", 331, (H, dn + dr)), ("k", 333, (H, dn)), ("kr", 333, (dr,)), ("v", 333, (H, dv)), ("go", 331, (H, dv))))}
    moved = {n: torch.cat([torch.full_like(t[:, :front], float("nan")), t], 1) for n, t in x.items()}

    def both(t, shift):
        new = lambda *s: torch.full((1, *s), 7.0, dtype=tdtype(dtype), device="cuda")  # noqa: E731
        Tq, Tk = t["q"].shape[1], t["k"].shape[1]
        kw = dict(cu_seqlens_q=ints(off_q) + shift, cu_seqlens_k=ints(off_k) + shift)
        args = (t["q"], t["k"], t["kr"], t["v"])
        o, lse = kda.latent_attention_fwd(*args, o=new(Tq, H, dv), lse=torch.full((1, Tq, H), 7.0, device="cuda"), **kw)
        out = dict(dq=new(Tq, H, dn + dr), dk=new(Tk, H, dn), dk_rope=new(Tk, dr), dv=new(Tk, H, dv))
        return [o, lse, *kda.latent_attention_bwd(*args, o, lse, t["go"], grad_dtype=tdtype(dtype), out=out, **kw).values()]
    a, b = both(x, 0), both(moved, front)
    for m, n in zip(a, b):
        assert (n[:, :front] == 7).all()
        assert torch.isfinite(n[:, front:]).sum() == torch.isfinite(m).sum() and torch.equal(m, n[:, front:])
