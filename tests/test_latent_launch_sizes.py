"""CPU test of how large a rotation one launch holds: counted in the workgroups that it makes, and refused beyond.  The addresses are
made up; a call that is not refused for its size is refused for the output that lies on its positions."""
import pytest

from gated_delta_rule_52_amd import _lib
from test_latent_abi import ALIAS, F, FP32, S, UNSUP, rotary


def call(rows, heads, dim, rot, offset, dtype=0, **kw):
    a = rotary(rows=rows, heads=heads, dim=dim, rot=rot, offset=offset, dtype=dtype, x=F, y=1 << 50, positions=1 << 50,
               inv_freq=1 << 60, x_stride=heads * dim, x_head_stride=dim, y_stride=heads * dim, y_head_stride=dim, **kw)
    return _lib.layer_raw("kda_rotary_fwd", a)


@pytest.mark.parametrize("rows,heads,dim,rot,offset,dtype", [
    (1 << 20, 128, 192, 64, 128, 0),      # 51 heads of 20 units to a workgroup, three groups: 2^20 rows of 48 KiB
    ((1 << 24) - 1, 32, 192, 64, 128, 0),
    (5 << 20, 128, 192, 64, 128, 0),
    (1 << 22, 8, 128, 128, 0, FP32),
    ((1 << 24) - 1, 1, 150, 64, 80, 0)])  # single elements
def test_held(rows, heads, dim, rot, offset, dtype):
    assert call(rows, heads, dim, rot, offset, dtype) == S[ALIAS], _lib.load().kda_last_error()
    assert _lib.load().kda_last_error().decode() == "y overlaps positions"


@pytest.mark.parametrize("rows,heads,dim,rot,offset,dtype", [
    ((1 << 24) // 3 + 1, 128, 192, 64, 128, 0), (1 << 24, 1, 64, 64, 0, 0), (1 << 20, 128, 190, 64, 126, 0), (1 << 14, 1 << 20, 64, 64, 0, FP32)])
def test_refused(rows, heads, dim, rot, offset, dtype):
    assert call(rows, heads, dim, rot, offset, dtype) == S[UNSUP]
    assert _lib.load().kda_last_error().decode() == "problem too large for one launch"
