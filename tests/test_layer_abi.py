"""CPU tests of the layer operators' C entry points: bad arguments are rejected with the documented status before
anything is launched (no GPU is touched: the addresses are made up and only compared)."""
import ctypes

import pytest

from gated_delta_rule_52_amd import _lib

F = 1 << 32
S = _lib.STATUS_CODE
BF16, FP32 = _lib.KDA_DTYPE_BF16, _lib.KDA_DTYPE_FP32


def fill(struct, base, kw):
    a = struct()
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


def scan(**kw):
    return fill(_lib.SelectiveScanArgs, dict(
        u=F, dt=2 * F, A=3 * F, B=4 * F, C=5 * F, D=6 * F, z=7 * F, dt_bias=8 * F, initial_state=9 * F,
        final_state=9 * F, y=10 * F, u_stride=100, dt_stride=100, B_stride=16, C_stride=16, z_stride=100, y_stride=100,
        batch=2, T=50, dim=100, ds=16, num_seqs=2, in_dtype=BF16, out_dtype=FP32, workspace=20 * F,
        workspace_bytes=1 << 30), kw)


def scan_bwd(**kw):
    return fill(_lib.SelectiveScanBwdArgs, dict(
        u=F, dt=2 * F, A=3 * F, B=4 * F, C=5 * F, D=6 * F, z=7 * F, dt_bias=8 * F, initial_state=9 * F, grad_y=10 * F,
        grad_final_state=11 * F, grad_u=12 * F, grad_dt=13 * F, grad_A=14 * F, grad_B=15 * F, grad_C=16 * F,
        grad_D=17 * F, grad_z=18 * F, grad_dt_bias=19 * F, grad_initial_state=9 * F, u_stride=100, dt_stride=100,
        B_stride=16, C_stride=16, z_stride=100, grad_y_stride=100, grad_u_stride=100, grad_dt_stride=100,
        grad_B_stride=16, grad_C_stride=16, grad_z_stride=100, batch=2, T=50, dim=100, ds=16, num_seqs=2,
        in_dtype=BF16, grad_dtype=FP32, workspace=20 * F, workspace_bytes=1 << 30), kw)


def conv(**kw):
    return fill(_lib.ShortConvArgs, dict(
        x=F, weight=2 * F, bias=3 * F, initial_state=4 * F, final_state=4 * F, y=5 * F, x_stride=100, y_stride=100,
        batch=2, T=50, dim=100, width=4, num_seqs=2, in_dtype=BF16, out_dtype=FP32, w_dtype=FP32), kw)


def conv_bwd(**kw):
    return fill(_lib.ShortConvBwdArgs, dict(
        x=F, weight=2 * F, bias=3 * F, initial_state=4 * F, grad_y=5 * F, grad_final_state=6 * F, grad_x=7 * F,
        grad_weight=8 * F, grad_bias=9 * F, grad_initial_state=6 * F, x_stride=100, grad_y_stride=100,
        grad_x_stride=100, batch=2, T=50, dim=100, width=4, num_seqs=2, in_dtype=BF16, grad_dtype=FP32, w_dtype=FP32,
        workspace=20 * F, workspace_bytes=1 << 30), kw)


def norm(**kw):
    return fill(_lib.LayerNormArgs, dict(
        x=F, residual=2 * F, weight=3 * F, bias=4 * F, y=5 * F, residual_out=2 * F, x_stride=100, residual_stride=100,
        y_stride=100, residual_out_stride=100, rows=70, dim=100, eps=1e-5, x_dtype=BF16, res_dtype=FP32, w_dtype=FP32,
        out_dtype=BF16), kw)


def norm_bwd(**kw):
    return fill(_lib.LayerNormBwdArgs, dict(
        x=F, grad_y=2 * F, weight=3 * F, grad_residual=4 * F, grad_x=5 * F, grad_weight=6 * F, grad_bias=7 * F,
        x_stride=100, grad_y_stride=100, grad_residual_stride=100, grad_x_stride=100, rows=70, dim=100, eps=1e-5,
        x_dtype=BF16, gy_dtype=BF16, res_dtype=FP32, w_dtype=FP32, grad_dtype=BF16, workspace=20 * F,
        workspace_bytes=1 << 30), kw)


NULL, SHAPE, UNSUP = "KDA_ERR_NULL_POINTER", "KDA_ERR_BAD_SHAPE", "KDA_ERR_UNSUPPORTED"
SMALL, ALIAS = "KDA_ERR_WORKSPACE_TOO_SMALL", "KDA_ERR_ALIAS"
BATCH = [(dict(batch=-1), SHAPE), (dict(T=-1), SHAPE), (dict(dim=0), SHAPE), (dict(num_seqs=3), SHAPE),
         (dict(cu_seqlens=30 * F), SHAPE), (dict(T=1 << 30, dim=1, ds=1), SHAPE), (dict(flags=2), UNSUP),
         (dict(in_dtype=5), UNSUP)]
CASES = [
    ("kda_selective_scan_fwd", scan, [b for b in BATCH] + [
        (dict(ds=0), UNSUP), (dict(ds=65), UNSUP), (dict(out_dtype=9), UNSUP), (dict(u=None), NULL),
        (dict(A=None), NULL), (dict(y=None), NULL), (dict(u_stride=99), SHAPE), (dict(C_stride=15), SHAPE),
        (dict(y_stride=0), SHAPE), (dict(z_stride=-100), SHAPE), (dict(y=F + 64), ALIAS),
        (dict(final_state=9 * F + 64), ALIAS), (dict(y=9 * F), ALIAS), (dict(final_state=8 * F), ALIAS),
        (dict(workspace=10 * F), ALIAS)]),
    ("kda_selective_scan_step", scan, [(dict(), SHAPE), (dict(T=1, batch=1, num_seqs=1, cu_seqlens=30 * F), SHAPE),
                                       (dict(T=1, final_state=None), NULL), (dict(T=1, y=7 * F), ALIAS)]),
    ("kda_selective_scan_bwd", scan_bwd, [b for b in BATCH] + [
        (dict(ds=65), UNSUP), (dict(grad_dtype=4), UNSUP), (dict(grad_y=None), NULL), (dict(grad_A=None), NULL),
        (dict(grad_B=None), NULL), (dict(grad_z=None), NULL), (dict(z=None), NULL), (dict(dt_bias=None), NULL),
        (dict(D=None), NULL), (dict(grad_u_stride=99), SHAPE), (dict(workspace_bytes=100), SMALL),
        (dict(workspace=None), SMALL), (dict(grad_u=F), ALIAS), (dict(grad_dt=12 * F + 4), ALIAS),
        (dict(grad_initial_state=9 * F + 16), ALIAS), (dict(grad_initial_state=14 * F), ALIAS),
        (dict(workspace=11 * F), ALIAS)]),
    ("kda_short_conv_fwd", conv, [b for b in BATCH] + [
        (dict(width=1), UNSUP), (dict(width=5), UNSUP), (dict(w_dtype=3), UNSUP), (dict(out_dtype=3), UNSUP),
        (dict(x=None), NULL), (dict(weight=None), NULL), (dict(x_stride=99), SHAPE), (dict(y=F), ALIAS),
        (dict(final_state=4 * F + 2), ALIAS), (dict(final_state=F), ALIAS)]),
    ("kda_short_conv_step", conv, [(dict(), SHAPE), (dict(T=1, final_state=None), NULL)]),
    ("kda_short_conv_bwd", conv_bwd, [b for b in BATCH] + [
        (dict(width=5), UNSUP), (dict(grad_dtype=3), UNSUP), (dict(grad_y=None), NULL), (dict(grad_weight=None), NULL),
        (dict(workspace_bytes=10), SMALL), (dict(grad_x=5 * F), ALIAS), (dict(grad_initial_state=4 * F), ALIAS),
        (dict(grad_initial_state=6 * F + 4), ALIAS)]),
    ("kda_layer_norm_fwd", norm, [
        (dict(rows=-1), SHAPE), (dict(dim=0), SHAPE), (dict(dim=16385), UNSUP), (dict(eps=float("nan")), SHAPE),
        (dict(eps=-1.0), SHAPE), (dict(x_dtype=2), UNSUP), (dict(res_dtype=2), UNSUP), (dict(x=None), NULL),
        (dict(y=None), NULL), (dict(residual_out=None), NULL), (dict(residual=None), NULL), (dict(y_stride=99), SHAPE),
        (dict(y=F), ALIAS), (dict(residual_out=2 * F + 4), ALIAS), (dict(residual_out_stride=101), ALIAS),
        (dict(y=4 * F), ALIAS)]),
    ("kda_layer_norm_bwd", norm_bwd, [
        (dict(rows=-1), SHAPE), (dict(dim=16385), UNSUP), (dict(gy_dtype=2), UNSUP), (dict(grad_dtype=2), UNSUP),
        (dict(grad_y=None), NULL), (dict(workspace_bytes=10), SMALL), (dict(workspace=None), SMALL),
        (dict(grad_x=F), ALIAS), (dict(grad_bias=6 * F), ALIAS), (dict(grad_x_stride=10), SHAPE)]),
]


@pytest.mark.parametrize("name,make,kw,status", [(n, m, kw, s) for n, m, rows in CASES for kw, s in rows])
def test_rejects(name, make, kw, status):
    rc = _lib.layer_raw(name, make(**kw))
    assert rc == S[status], (_lib.STATUS.get(rc), _lib.load().kda_last_error())
    assert _lib.load().kda_last_error().decode() != ""


@pytest.mark.parametrize("name,make", [(n, m) for n, m, _ in CASES])
def test_struct_size_and_null(name, make):
    fn = getattr(_lib.load(), name)
    a = make()
    a.struct_size = ctypes.sizeof(a) - 8
    assert fn(ctypes.byref(a)) == S["KDA_ERR_BAD_STRUCT"]
    assert fn(None) == S[NULL]


@pytest.mark.parametrize("struct", sorted({s for s, _ in _lib.LAYER_FUNCTIONS.values()}, key=lambda s: s.__name__))
def test_packed_structs_have_the_layout_of_the_c_ones(struct):
    """Every field packed with a value of its own comes back from the same bytes read as the C struct."""
    pack = _lib.packer(struct)
    assert pack.size == ctypes.sizeof(struct)
    values = [float(i + 1) if kind is ctypes.c_float else i + 1 for i, (_, kind) in enumerate(struct._fields_)]
    read = struct.from_buffer_copy(pack.pack(*values))
    assert [getattr(read, name) for name, _ in struct._fields_] == values


def test_empty_calls_are_no_ops():
    for name, make in (("kda_selective_scan_fwd", scan), ("kda_short_conv_fwd", conv)):
        assert _lib.layer_raw(name, make(batch=0, num_seqs=0)) == 0
    for name, make in (("kda_selective_scan_step", scan), ("kda_short_conv_step", conv)):
        assert _lib.layer_raw(name, make(T=1, batch=0, num_seqs=0)) == 0
    assert _lib.layer_raw("kda_layer_norm_fwd", norm(rows=0, x=None, y=None)) == 0


def test_slices_of_one_buffer_may_interleave():
    """u and z gradients as the halves of one projection's gradient: rows interleave, elements do not.  The call gets
    past the overlap check, to the next thing that is wrong with it."""
    pair = dict(grad_u=12 * F, grad_z=12 * F + 400, grad_u_stride=200, grad_z_stride=200)
    assert _lib.layer_raw("kda_selective_scan_bwd", scan_bwd(workspace=11 * F, **pair)) == S[ALIAS]
    assert b"workspace" in _lib.load().kda_last_error()
    pair["grad_z"] -= 4
    assert _lib.layer_raw("kda_selective_scan_bwd", scan_bwd(**pair)) == S[ALIAS]
    assert b"grad_u" in _lib.load().kda_last_error()


def test_workspace_queries():
    for name, make, wrong in (("kda_selective_scan_bwd_workspace_bytes", scan_bwd, dict(ds=0)),
                              ("kda_short_conv_bwd_workspace_bytes", conv_bwd, dict(width=9)),
                              ("kda_layer_norm_bwd_workspace_bytes", norm_bwd, dict(dim=0))):
        n = _lib.layer_raw(name, make())
        assert 0 < n < 1 << 30
        assert _lib.layer_raw(name, make(**wrong)) == 2 ** 64 - 1
    assert _lib.layer_raw("kda_layer_norm_bwd_workspace_bytes", norm_bwd(grad_weight=None, grad_bias=None)) == 0
    assert _lib.layer_raw("kda_selective_scan_fwd_workspace_bytes", scan(ds=0)) == 2 ** 64 - 1
    # packed input with many short sequences and one long: bounded by rows and sequences
    n = _lib.layer_raw("kda_selective_scan_bwd_workspace_bytes",
                       scan_bwd(batch=1, T=1 << 20, num_seqs=1 << 10, cu_seqlens=30 * F, dim=64))
    assert n < 1 << 36
