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
