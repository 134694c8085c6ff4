"""CPU tests of the layer operators' limits on a launch's threads, which have to stay below 2^32: calls just inside a
limit get past it, to the overlap that they also have, and calls outside are refused.  No call here can launch anything."""
import pytest

from gated_delta_rule_52_amd import _lib
from test_layer_abi import ALIAS, F, UNSUP, S, conv, conv_bwd, norm, scan_bwd

LONGEST = 2 ** 31 - 1


@pytest.mark.parametrize("dim,rows,fits", [
    (128, 2 ** 28 - 16, True), (128, 2 ** 28 - 15, False), (8, 2 ** 26, True), (256, 2 ** 27 - 8, True), (256, 2 ** 27 - 7, False),
    (1000, 2 ** 26 - 4, True), (1000, 2 ** 26 - 3, False), (4096, 2 ** 24 - 1, True), (4096, 2 ** 24, False),
    (8192, 2 ** 23 - 1, True), (8192, 2 ** 23, False), (16384, 2 ** 22 - 1, True), (16384, 2 ** 22, False)])
def test_norm(dim, rows, fits):
    s = dict(x_stride=dim, residual_stride=dim, y_stride=dim, residual_out_stride=dim)
    rc = _lib.layer_raw("kda_layer_norm_fwd", norm(dim=dim, rows=rows, y=F, **s))
    assert rc == S[ALIAS if fits else UNSUP], _lib.load().kda_last_error()


@pytest.mark.parametrize("dim,T,fits", [(4, 2 ** 28, True), (4, 2 ** 30 - 64, True), (4, 2 ** 30, False), (4096, 2 ** 25, True),
                                        (4096, 2 ** 26, False)])
def test_conv(dim, T, fits):
    a = conv(dim=dim, batch=1, num_seqs=1, T=T, x_stride=dim, y_stride=dim, y=F)
    assert _lib.layer_raw("kda_short_conv_fwd", a) == S[ALIAS if fits else UNSUP], _lib.load().kda_last_error()


@pytest.mark.parametrize("dim,T,fits", [(8, 2 ** 28, True), (8, LONGEST, True), (4096, 2 ** 25, True), (4096, 2 ** 28, True),
                                        (4096, 2 ** 28 + 1, False)])
def test_conv_gradients(dim, T, fits):
    a = conv_bwd(dim=dim, batch=1, num_seqs=1, T=T, x_stride=dim, grad_y_stride=dim, grad_x_stride=dim)
    n = _lib.layer_raw("kda_short_conv_bwd_workspace_bytes", a)
    assert (n < 1 << 50) == fits, n


@pytest.mark.parametrize("dim,ds,T,fits", [
    (1, 1, LONGEST - 256, True), (1, 1, LONGEST, False),  # the channel groups' sums: 2 ds threads per row, in whole workgroups
    (2 ** 20 - 1, 64, 16, False), (2 ** 26 // 66 - 16, 64, 16, True)])  # the parameters' sums: 64 threads per column
def test_scan_gradients(dim, ds, T, fits):
    s = dict(u_stride=dim, dt_stride=dim, z_stride=dim, grad_y_stride=dim, grad_u_stride=dim, grad_dt_stride=dim, grad_z_stride=dim,
             B_stride=ds, C_stride=ds, grad_B_stride=ds, grad_C_stride=ds)
    a = scan_bwd(dim=dim, ds=ds, batch=1, num_seqs=1, T=T, workspace_bytes=1 << 50, grad_u=F, **s)
    n = _lib.layer_raw("kda_selective_scan_bwd_workspace_bytes", a)
    assert (n < 1 << 50) == fits, n
    rc = _lib.layer_raw("kda_selective_scan_bwd", a)
    assert rc == S[ALIAS if fits else UNSUP], _lib.load().kda_last_error()
