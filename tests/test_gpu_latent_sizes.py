"""Rotation of more heads than a workgroup each would leave room for in one launch."""
import pytest

from test_gpu_latent import ints, kda, make  # noqa: F401

pytestmark = pytest.mark.gpu


def test_rotation_of_many_heads(kda):  # noqa: F811
    """131,073 rows of 128 heads of 1,024 elements (34 GB), in place: sampled rows have the bits of a call on them alone, and elements
    beside the rotated part are not touched."""
    import torch
    T, H, D, rot, offset = (1 << 17) + 1, 128, 1024, 64, 904
    x = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 77, 65535, 65536, T - 2, T - 1]
    part = make(1, (len(rows), H, D), "bf16")
    x[rows] = part
    f, _ = kda.rotary_frequencies(rot)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    want = kda.rotary_fwd(part, ints(rows), f, offset=offset)
    assert kda.rotary_fwd(x, pos, f, offset=offset, y=x) is x
    assert torch.equal(x[rows], want)
    assert torch.equal(want[..., :offset], part[..., :offset]) and torch.equal(want[..., offset + rot:], part[..., offset + rot:])
