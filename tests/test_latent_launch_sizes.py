"""CPU tests of how large a rotation and how large gradients one launch holds: counted in the workgroups that it makes, and refused
beyond.  The addresses are made up; a call that is not refused for its size is refused for an output that lies on an input."""
import pytest

from gated_delta_rule_52_amd import _lib
from test_latent_abi import ALIAS, BF16, F, FP32, S, UNSUP, attend_bwd, rotary


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


def gradients(T, H, dtype):
    """Heads of 8 + 8 and 8, causal."""
    G = 1 << 48
    names = ("q", "k", "k_rope", "v", "o", "grad_o", "grad_q", "grad_k", "grad_k_rope", "grad_v")
    width = dict(q=16, grad_q=16)
    kw = {n: (i + 1) * G for i, n in enumerate(names)}
    kw.update({n + "_stride": 8 if "rope" in n else H * width.get(n, 8) for n in names})
    kw.update({n + "_head_stride": width.get(n, 8) for n in names if "rope" not in n})
    kw.update(lse=20 * G, workspace=30 * G, workspace_bytes=1 << 46, grad_q=G, batch=1, num_seqs=1, Tq=T, Tk=T, H=H, dn=8, dr=8, dv=8,
              in_dtype=dtype, grad_dtype=dtype)
    return _lib.layer_raw("kda_latent_attention_bwd", attend_bwd(**kw))


@pytest.mark.parametrize("T,H,dtype,status", [
    (1 << 26, 4, BF16, ALIAS), ((1 << 30) - 128, 1, BF16, ALIAS), (1 << 30, 2, BF16, UNSUP), ((1 << 27) - 32, 1, FP32, ALIAS), (1 << 27, 1, FP32, UNSUP)])
def test_gradients(T, H, dtype, status):
    assert gradients(T, H, dtype) == S[status], _lib.load().kda_last_error()
