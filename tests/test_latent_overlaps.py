"""CPU tests of which tensors are taken to share memory: csrc/kda_spans.h, compiled here by the host's compiler, against an
enumeration of the bytes, and gradients of k and v as slices of one buffer in every layout."""
import os
import random
import subprocess

import pytest

from gated_delta_rule_52_amd import _lib
from test_latent_abi import ALIAS, BF16, F, FP32, S, attend_bwd, rotary

CSRC = os.path.join(os.path.dirname(_lib.__file__), "csrc")

PROGRAM = r"""
#include "kda_spans.h"
#include <cstdio>
int main() {
    kda::Span a{"a"}, b{"b"};
    unsigned long p, q;
    while (scanf("%lu %ld %ld %ld %ld %ld %lu %ld %ld %ld %ld %ld", &p, &a.rows, &a.width, &a.stride, &a.parts, &a.part_stride,
                 &q, &b.rows, &b.width, &b.stride, &b.parts, &b.part_stride) == 12) {
        a.at = p;
        b.at = q;
        printf("%d\n", kda::overlap(a, b));
    }
}
"""


@pytest.fixture(scope="module")
def overlaps(tmp_path_factory):
    where = tmp_path_factory.mktemp("spans")
    (where / "spans.cpp").write_text(PROGRAM)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-ftrapv", "-I", CSRC, str(where / "spans.cpp"), "-o", str(where / "spans")])

    def run(pairs):
        lines = "".join(" ".join(map(str, a + b)) + "\n" for a, b in pairs)
        return [w == "1" for w in subprocess.check_output([str(where / "spans")], input=lines, text=True).split()]
    return run


def bytes_of(at, rows, width, stride, parts, part_stride):
    return {at + r * stride + p * part_stride + i for r in range(rows) for p in range(parts) for i in range(width)}


def test_no_shared_byte_is_missed(overlaps):
    """Random patterns with the same and with other strides; where the function says that nothing is shared, nothing is."""
    rng = random.Random(0)

    def one(stride):
        parts, width = rng.randint(1, 4), rng.randint(1, 6)
        step = width + rng.randint(0, 6)
        row = (parts - 1) * step + width
        return (rng.randint(1, 60), rng.randint(0, 4), width, max(stride or 0, row) + (0 if stride else rng.randint(0, 5)), parts, step)
    pairs = []
    for _ in range(20000):
        a = one(None)
        b = one(a[3]) if rng.random() < 0.8 else one(None)
        if rng.random() < 0.5 and b[4] > 1:  # parts of the same distance
            b = b[:2] + (min(b[2], a[5]), b[3], b[4], a[5]) if (b[4] - 1) * a[5] + min(b[2], a[5]) <= b[3] else b
        pairs.append((a, b))
    said = overlaps(pairs)
    truth = [bool(bytes_of(*a) & bytes_of(*b)) for a, b in pairs]
    assert all(s or not t for s, t in zip(said, truth))
    assert sum(truth) > 1000 and sum(not s and a[0] < b[0] + b[3] * b[1] and b[0] < a[0] + a[3] * a[1] for s, (a, b) in zip(said, pairs)) > 500


@pytest.mark.parametrize("pad", [0, 1, 5, 11, 12, 30])
@pytest.mark.parametrize("rows,parts", [(1, 1), (2, 1), (2, 3), (5, 4)])
def test_slices_of_one_buffer_share_nothing(overlaps, pad, rows, parts):
    """The parts' first 7 and last 5 bytes, in rows that are padded by any number."""
    stride = parts * 12 + pad
    a, b = (100, rows, 7, stride, parts, 12), (107, rows, 5, stride, parts, 12)
    # one row is given as rows of its parts
    if rows == 1:
        a, b = (100, parts, 7, 12, 1, 0), (107, parts, 5, 12, 1, 0)
    assert overlaps([(a, b), (b, a), (a, a)]) == [False, False, True]


@pytest.mark.parametrize("odd", [0, -5, 10 ** 9])
def test_a_single_row_between_the_parts_of_many(overlaps, odd):
    """Its own stride is not looked at, nor that of a single part."""
    many, one = (100, 5, 7, 40, 3, 12), (187, 1, 5, odd, 3, 12)
    part = (187, 1, 5, odd, 1, odd)
    assert overlaps([(many, one), (one, many), (many, part), (part, many), (one, (192, 1, 7, odd, 2, 12)), (one, (191, 1, 7, odd, 2, 12)),
                     (many, (186, 1, 5, odd, 3, 12)), (part, (180, 1, 8, odd, 1, odd)), (part, (180, 1, 7, odd, 1, odd))]) \
        == [False, False, False, False, False, True, True, True, False]


# [rows, heads] strides of one buffer [rows, heads, 256] in bf16 or fp32: dense, padded rows, padded by less than a head, heads in front
@pytest.mark.parametrize("stride,head_stride", [(1024, 256), (2048, 256), (1032, 256), (1024 + 64, 256), (256, 256 * 120), (264, 264 * 120)])
def test_gradients_as_slices_of_one_buffer(stride, head_stride):
    """They get past the check against each other: the next output that lies wrong is named."""
    both = {f"grad_{t}_{n}": v for t in "kv" for n, v in (("stride", stride), ("head_stride", head_stride))}
    for dtype, e in ((FP32, 4), (BF16, 2)):
        kw = dict(both, grad_dtype=dtype)
        assert _lib.layer_raw("kda_latent_attention_bwd", attend_bwd(grad_v=9 * F + 128 * e, workspace=9 * F, **kw)) == S[ALIAS]
        assert _lib.load().kda_last_error().decode() == "grad_k overlaps workspace"
        assert _lib.layer_raw("kda_latent_attention_bwd", attend_bwd(grad_v=9 * F + 120 * e, **kw)) == S[ALIAS]
        assert _lib.load().kda_last_error().decode() == "grad_k overlaps grad_v"


def test_rotation_beside_its_input():
    """y as other columns of x's rows, which are no multiple of the heads' distance."""
    kw = dict(x_stride=1310, x_head_stride=320, y_stride=1310, y_head_stride=320)
    assert _lib.layer_raw("kda_rotary_fwd", rotary(y=F + 150 * 2, positions=F + 150 * 2 + 64, **kw)) == S[ALIAS]
    assert _lib.load().kda_last_error().decode() == "y overlaps positions"
    assert _lib.layer_raw("kda_rotary_fwd", rotary(y=F + 148 * 2, **kw)) == S[ALIAS]
    assert _lib.load().kda_last_error().decode() == "y overlaps x"
