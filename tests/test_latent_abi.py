"""CPU tests of latent attention's C entry points: bad arguments are rejected with the documented status before anything is
launched (no GPU is touched: the addresses are made up and only compared)."""
import ctypes

import pytest

from gated_delta_rule_52_amd import _lib
from test_layer_abi import ALIAS, BF16, F, FP32, NULL, SHAPE, SMALL, UNSUP, S, fill


def rotary(**kw):
    return fill(_lib.RotaryArgs, dict(
        x=F, y=2 * F, positions=3 * F, inv_freq=4 * F, x_stride=600, x_head_stride=150, y_stride=600, y_head_stride=150,
        rows=70, heads=4, dim=150, rot=64, offset=80, scale=1.0, dtype=BF16), kw)


def append(**kw):
    return fill(_lib.LatentAppendArgs, dict(
        latent=F, rope=F + 512 * 2, cache=2 * F, slots=3 * F, positions=4 * F, inv_freq=5 * F, latent_stride=576,
        rope_stride=576, rows=70, num_blocks=9, page=16, dl=512, dr=64, scale=1.0, dtype=BF16), kw)


def step(**kw):
    return fill(_lib.LatentStepArgs, dict(
        q_latent=F, q_rope=2 * F, cache=3 * F, block_table=4 * F, lengths=5 * F, o=6 * F, lse=7 * F,
        q_latent_stride=16 * 512, q_latent_head_stride=512, q_rope_stride=16 * 64, q_rope_head_stride=64,
        o_stride=16 * 512, o_head_stride=512, block_table_stride=40, N=3, H=16, dl=512, dr=64, page=16, num_blocks=100,
        max_blocks=40, scale=0.1, in_dtype=BF16, out_dtype=FP32, workspace=20 * F, workspace_bytes=1 << 30), kw)


def attend(**kw):
    return fill(_lib.LatentAttentionArgs, dict(
        q=F, k=2 * F, k_rope=3 * F, v=2 * F + 256, o=5 * F, lse=6 * F, q_stride=768, q_head_stride=192, k_stride=1024,
        k_head_stride=256, k_rope_stride=64, v_stride=1024, v_head_stride=256, o_stride=512, o_head_stride=128, batch=2,
        Tq=50, Tk=60, H=4, dn=128, dr=64, dv=128, num_seqs=2, scale=0.1, in_dtype=BF16, out_dtype=BF16, flags=1), kw)


def attend_bwd(**kw):
    return fill(_lib.LatentAttentionBwdArgs, dict(
        q=F, k=2 * F, k_rope=3 * F, v=2 * F + 256, o=5 * F, lse=6 * F, grad_o=7 * F, grad_q=8 * F, grad_k=9 * F,
        grad_k_rope=10 * F, grad_v=9 * F + 512, q_stride=768, q_head_stride=192, k_stride=1024, k_head_stride=256,
        k_rope_stride=64, v_stride=1024, v_head_stride=256, o_stride=512, o_head_stride=128, grad_o_stride=512,
        grad_o_head_stride=128, grad_q_stride=768, grad_q_head_stride=192, grad_k_stride=1024, grad_k_head_stride=256,
        grad_k_rope_stride=64, grad_v_stride=1024, grad_v_head_stride=256, batch=2, Tq=50, Tk=60, H=4, dn=128, dr=64,
        dv=128, num_seqs=2, scale=0.1, in_dtype=BF16, grad_dtype=FP32, workspace=20 * F, workspace_bytes=1 << 30, flags=1), kw)


NAN, INF = float("nan"), float("inf")
ATTEND = [(dict(batch=-1), SHAPE), (dict(Tq=-1), SHAPE), (dict(Tk=-1), SHAPE), (dict(H=0), SHAPE), (dict(num_seqs=3), SHAPE),
          (dict(cu_seqlens_q=30 * F), NULL), (dict(cu_seqlens_k=30 * F), NULL),
          (dict(cu_seqlens_q=30 * F, cu_seqlens_k=31 * F), SHAPE), (dict(dn=0), SHAPE), (dict(dn=136), UNSUP),
          (dict(dn=12), UNSUP), (dict(dr=0), SHAPE), (dict(dr=72), UNSUP), (dict(dv=-8), SHAPE), (dict(dv=130), UNSUP),
          (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=NAN), SHAPE), (dict(scale=INF), SHAPE),
          (dict(in_dtype=2), UNSUP), (dict(flags=2), UNSUP), (dict(q=None), NULL), (dict(k=None), NULL),
          (dict(k_rope=None), NULL), (dict(v=None), NULL), (dict(q_stride=700), SHAPE), (dict(q_head_stride=184), SHAPE),
          (dict(k_stride=1 << 22), SHAPE), (dict(k_rope_stride=56), SHAPE), (dict(q=F + 8), UNSUP),
          (dict(v_stride=1028), UNSUP), (dict(k_head_stride=250), UNSUP),
          (dict(batch=1, num_seqs=1, Tq=(1 << 30) + 1), UNSUP), (dict(batch=70000, num_seqs=70000), UNSUP)]
CASES = [
    ("kda_rotary_fwd", rotary, [
        (dict(rows=-1), SHAPE), (dict(heads=-1), SHAPE), (dict(dim=0), SHAPE), (dict(rot=0), SHAPE), (dict(rot=63), SHAPE),
        (dict(offset=-2), SHAPE), (dict(offset=88), SHAPE), (dict(rot=152, offset=0), SHAPE), (dict(dtype=2), UNSUP),
        (dict(flags=2), UNSUP), (dict(scale=NAN), SHAPE), (dict(x=None), NULL), (dict(y=None), NULL),
        (dict(positions=None), NULL), (dict(inv_freq=None), NULL), (dict(x_stride=599), SHAPE),
        (dict(x_head_stride=149), SHAPE), (dict(y_head_stride=600), SHAPE), (dict(rows=1 << 31), UNSUP),
        (dict(rot=4098, dim=5000, x_stride=20000, x_head_stride=5000), UNSUP), (dict(heads=1 << 21), UNSUP),
        (dict(dim=(1 << 15) + 2, x_stride=300000, x_head_stride=40000, y_stride=300000, y_head_stride=40000), UNSUP),
        (dict(rows=1 << 24, heads=1, x_stride=150, y_stride=150), UNSUP), (dict(y=F, y_stride=900), ALIAS),
        (dict(y=F + 2), ALIAS), (dict(y=3 * F), ALIAS), (dict(y=4 * F + 64), ALIAS)]),
    ("kda_rotary_bwd", rotary, [(dict(x=None), NULL), (dict(y=F + 64), ALIAS)]),
    ("kda_latent_cache_append", append, [
        (dict(rows=-1), SHAPE), (dict(num_blocks=-1), SHAPE), (dict(page=0), SHAPE), (dict(dl=0), SHAPE), (dict(dr=0), SHAPE),
        (dict(dr=63), SHAPE), (dict(dl=1 << 17), UNSUP), (dict(num_blocks=1 << 30), UNSUP), (dict(rows=(1 << 30) + 1), UNSUP),
        (dict(dtype=2), UNSUP), (dict(flags=2), UNSUP), (dict(scale=INF), SHAPE), (dict(positions=None), NULL),
        (dict(inv_freq=None), NULL), (dict(latent=None), NULL), (dict(rope=None), NULL), (dict(cache=None), NULL),
        (dict(slots=None), NULL), (dict(latent_stride=511), SHAPE), (dict(rope_stride=63), SHAPE), (dict(cache=F), ALIAS),
        (dict(cache=3 * F), ALIAS), (dict(cache=F - 1024), ALIAS), (dict(rows=1 << 27), UNSUP)]),
    ("kda_latent_attention_step", step, [
        (dict(N=-1), SHAPE), (dict(H=0), SHAPE), (dict(page=0), SHAPE), (dict(num_blocks=-1), SHAPE), (dict(max_blocks=-1), SHAPE),
        (dict(dl=0), SHAPE), (dict(dl=520), UNSUP), (dict(dl=100), UNSUP), (dict(dr=72), UNSUP), (dict(dr=4), UNSUP),
        (dict(scale=0.0), SHAPE), (dict(scale=NAN), SHAPE), (dict(in_dtype=2), UNSUP), (dict(out_dtype=2), UNSUP),
        (dict(N=70000), UNSUP), (dict(H=70000), UNSUP), (dict(page=1 << 20, max_blocks=1 << 12), UNSUP),
        (dict(N=2000, page=1 << 10, max_blocks=1 << 20, block_table_stride=1 << 20), UNSUP),
        (dict(q_latent=None), NULL), (dict(q_rope=None), NULL), (dict(cache=None), NULL), (dict(block_table=None), NULL),
        (dict(lengths=None), NULL), (dict(o=None), NULL), (dict(q_latent_stride=100), SHAPE),
        (dict(q_rope_head_stride=56), SHAPE), (dict(block_table_stride=39), SHAPE), (dict(q_latent=F + 2), UNSUP),
        (dict(cache=3 * F + 8), UNSUP), (dict(o_head_stride=514), SHAPE), (dict(o_stride=16 * 516, o_head_stride=514), UNSUP), (dict(workspace_bytes=100), SMALL),
        (dict(workspace=None), SMALL), (dict(workspace=20 * F + 4), UNSUP), (dict(o=F), ALIAS), (dict(o=3 * F + 1024), ALIAS),
        (dict(lse=6 * F + 64), ALIAS), (dict(workspace=6 * F), ALIAS), (dict(o=4 * F), ALIAS), (dict(lse=5 * F), ALIAS)]),
    ("kda_latent_attention_fwd", attend, ATTEND + [
        (dict(out_dtype=2), UNSUP), (dict(o=None), NULL), (dict(o=F), ALIAS), (dict(o=2 * F + 512), ALIAS), (dict(lse=5 * F), ALIAS),
        (dict(o_stride=500), SHAPE), (dict(o=5 * F + 2), UNSUP)]),
    ("kda_latent_attention_bwd", attend_bwd, ATTEND + [
        (dict(grad_dtype=2), UNSUP), (dict(o=None), NULL), (dict(lse=None), NULL), (dict(grad_o=None), NULL),
        (dict(grad_q=None), NULL), (dict(grad_k=None), NULL), (dict(grad_k_rope=None), NULL), (dict(grad_v=None), NULL),
        (dict(workspace_bytes=100), SMALL), (dict(workspace=None), SMALL), (dict(workspace=20 * F + 8), UNSUP),
        (dict(grad_q=F), ALIAS), (dict(grad_v=9 * F), ALIAS), (dict(grad_v=9 * F + 256), ALIAS), (dict(grad_k_rope=8 * F), ALIAS),
        (dict(workspace=9 * F), ALIAS), (dict(grad_o_stride=300), SHAPE), (dict(grad_k_head_stride=124), SHAPE)]),
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


def test_empty_calls_are_no_ops():
    for name, a in (("kda_rotary_fwd", rotary(rows=0, x=None)), ("kda_rotary_bwd", rotary(heads=0, y=None)),
                    ("kda_latent_cache_append", append(rows=0, latent=None)), ("kda_latent_cache_append", append(num_blocks=0, cache=None)),
                    ("kda_latent_attention_step", step(N=0, o=None)), ("kda_latent_attention_fwd", attend(batch=0, num_seqs=0)),
                    ("kda_latent_attention_fwd", attend(Tq=0, q=None, o=None)),
                    ("kda_latent_attention_bwd", attend_bwd(batch=0, num_seqs=0))):
        assert _lib.layer_raw(name, a) == 0, _lib.load().kda_last_error()


def test_workspace_queries():
    for name, make in (("kda_latent_attention_step_workspace_bytes", step), ("kda_latent_attention_bwd_workspace_bytes", attend_bwd)):
        assert 0 < _lib.layer_raw(name, make()) < 1 << 30
        assert _lib.layer_raw(name, make(H=0)) == 2 ** 64 - 1
    # many sequences and heads: a workgroup per sequence, no parts
    assert _lib.layer_raw("kda_latent_attention_step_workspace_bytes", step(N=65535, H=128, page=16, max_blocks=4)) == 0
    # the rows' statistics and the heads' parts of the shared key's gradient
    for dtype, stats in ((BF16, 2), (FP32, 1)):
        assert _lib.layer_raw("kda_latent_attention_bwd_workspace_bytes", attend_bwd(in_dtype=dtype)) == stats * 2 * 50 * 4 * 4 + 2 * 60 * 4 * 64 * 4


def test_slices_of_one_buffer_may_interleave():
    """Gradients of k and v as the parts of one projection's gradient get past the overlap check, to the next output that
    lies wrong."""
    assert _lib.layer_raw("kda_latent_attention_bwd", attend_bwd(workspace=8 * F)) == S[ALIAS]
    assert b"workspace" in _lib.load().kda_last_error()
    # heads in front of rows
    q = dict(q_stride=192, q_head_stride=192 * 100)
    assert _lib.layer_raw("kda_latent_attention_fwd", attend(o=F, **q)) == S[ALIAS]
    assert _lib.layer_raw("kda_latent_attention_fwd", attend(q_stride=192, q_head_stride=192 * 99)) == S[SHAPE]
