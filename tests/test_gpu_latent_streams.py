"""The step at every compiled width with many tiles to a workgroup: both buffers in turn, a tile's rows loaded in two parts, the
move to the next sequence within a run, rescaled sums, and joins of up to 512 parts, against 64 bits.

Tiles are of 32 rows in bf16 (64 with more than 32 heads) and of 16 in fp32; 512 workgroups share them out with up to 32 heads, 256
with up to 64, 128 for each of two groups of heads with up to 128 in bf16."""
import pytest

from test_gpu_latent import check_step, kda  # noqa: F401

pytestmark = pytest.mark.gpu

# more than 512 tiles of 32 rows, or 256 of 64: four and more to a workgroup; sequences that end within a run, of a row, of none
RAGGED = [30011, 0, 5, 14000, 33, 9000, 1, 700]
SHORT = [9007, 0, 5, 4100, 17, 1, 700]  # the same for fp32's tiles


@pytest.mark.parametrize("dl,dr", [(512, 64), (504, 40), (256, 64), (200, 8), (128, 64)])
@pytest.mark.parametrize("H", [10, 20, 40])
def test_bf16(kda, dl, dr, H):  # noqa: F811
    check_step(kda, 200, RAGGED, H, dl, dr, 64, "bf16")


@pytest.mark.parametrize("dl,dr", [(512, 64), (504, 40), (256, 64), (200, 8), (128, 64)])
@pytest.mark.parametrize("H", [5, 20, 40])
def test_fp32(kda, dl, dr, H):  # noqa: F811
    check_step(kda, 210, SHORT if H > 32 else [2 * n for n in SHORT], H, dl, dr, 7, "fp32")


@pytest.mark.parametrize("H", [70, 128])
def test_two_groups_of_heads(kda, H):  # noqa: F811
    """128 workgroups to a group."""
    check_step(kda, 220, RAGGED, H, 512, 64, 16, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H", [16, 32, 64])
def test_scores_that_move_the_reference_point(kda, dtype, H):  # noqa: F811
    """Scores of about 50 in size: the sums are rescaled at many tiles, and parts differ by many powers of two."""
    check_step(kda, 230, [17000, 0, 6001], H, 512, 64, 16, dtype, std=4.0, scale=0.5)


@pytest.mark.parametrize("dtype,length", [("bf16", 16384), ("bf16", 16383), ("bf16", 16385), ("fp32", 8192), ("fp32", 8177), ("fp32", 8193)])
@pytest.mark.parametrize("H", [1, 16])
def test_as_many_parts_as_are_joined(kda, dtype, length, H):  # noqa: F811
    """One sequence in 512 tiles and so 512 parts, or in one tile more and so 257."""
    check_step(kda, 240, [length], H, 512, 64, 64, dtype)


def test_parts_of_many_heads(kda):  # noqa: F811
    """The join with all columns at once, from 512 pairs of sequence and head on: 257 parts, or sequences of fewer."""
    check_step(kda, 250, [16385] + [40] * 39, 16, 512, 64, 64, "bf16")
    check_step(kda, 251, [30000, 20000, 0, 8000, 90] + [1] * 13, 30, 256, 64, 64, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_pages_that_do_not_exist_within_a_run(kda, dtype):  # noqa: F811
    def edit(table):
        table[0, 5:40], table[0, 100:300:3], table[2, ::2] = -1, 2 ** 31 - 1, -5
    check_step(kda, 260, [20000, 5, 9000], 20, 512, 64, 16, dtype, table_edit=edit)
