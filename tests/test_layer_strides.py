"""CPU tests of the row strides that the layer operators take: those inside the limits get past their check, to the
overlap that every call here also has, and those outside are refused.  No call here can launch anything."""
import pytest

from gated_delta_rule_52_amd import _lib
from test_layer_abi import ALIAS, F, SHAPE, S, conv, conv_bwd, norm, norm_bwd, scan, scan_bwd

ONE = dict(batch=3, num_seqs=3, T=1)
PACKED = dict(batch=1, num_seqs=1, T=3, cu_seqlens=30 * F)
FAR = 1 << 38  # three rows of it stay within 2^40


@pytest.mark.parametrize("name,make,kw,stride,fits", [
    ("kda_selective_scan_step", scan, dict(ONE, y=7 * F), 1 << 22, True),
    ("kda_selective_scan_step", scan, dict(ONE, y=7 * F), FAR, True),
    ("kda_selective_scan_step", scan, dict(ONE, y=7 * F), FAR * 2, False),
    ("kda_selective_scan_fwd", scan, dict(ONE, y=7 * F), FAR, True),
    ("kda_selective_scan_fwd", scan, dict(ONE, T=2, y=7 * F), (1 << 22) - 1, True),
    ("kda_selective_scan_fwd", scan, dict(ONE, T=2, y=7 * F), 1 << 22, False),
    ("kda_selective_scan_fwd", scan, dict(PACKED, y=7 * F), 1 << 22, False),
    ("kda_selective_scan_bwd", scan_bwd, dict(ONE, grad_u=7 * F), FAR, True),
    ("kda_selective_scan_bwd", scan_bwd, dict(ONE, T=2, grad_u=7 * F), 1 << 22, False),
    ("kda_selective_scan_bwd", scan_bwd, dict(PACKED, grad_u=7 * F), 1 << 22, False),
    ("kda_short_conv_step", conv, dict(ONE, y=2 * F), FAR, True),
    ("kda_short_conv_fwd", conv, dict(PACKED, y=2 * F), FAR, True),
    ("kda_short_conv_bwd", conv_bwd, dict(PACKED, grad_x=2 * F), FAR, True),
    ("kda_layer_norm_fwd", norm, dict(rows=3, dim=2048, y=3 * F), (1 << 26) - 1, True),
    ("kda_layer_norm_fwd", norm, dict(rows=3, dim=2048, y=3 * F), 1 << 26, False),
    ("kda_layer_norm_fwd", norm, dict(rows=3, dim=2049, y=3 * F), FAR, True),
    ("kda_layer_norm_bwd", norm_bwd, dict(rows=3, dim=2048, grad_x=3 * F), (1 << 26) - 1, True),
    ("kda_layer_norm_bwd", norm_bwd, dict(rows=3, dim=2048, grad_x=3 * F), 1 << 26, False),
    ("kda_layer_norm_bwd", norm_bwd, dict(rows=3, dim=2049, grad_x=3 * F), FAR, True)])
def test_strides(name, make, kw, stride, fits):
    a = make(workspace_bytes=1 << 40, **kw) if "workspace_bytes" in dict(make()._fields_) else make(**kw)
    for field, _ in a._fields_:
        if field.endswith("_stride"):
            setattr(a, field, stride)
    assert _lib.layer_raw(name, a) == S[ALIAS if fits else SHAPE], _lib.load().kda_last_error()
