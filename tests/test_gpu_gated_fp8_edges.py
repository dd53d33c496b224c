"""blockwise_scaled_gated_mm at the edge of what it allows, and its kernels over many
slabs, ranges and rounds, against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle.e4m3 import decode
from oracle.gated import F32
from tests.gpu_util import DEV, codes, q8
from tests.test_gpu_gated import T, check, f64, make
from tests.test_gpu_gated_fp8 import expect, operands

pytestmark = pytest.mark.gpu


def to(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


@pytest.mark.parametrize("K", [128, 256])
@pytest.mark.parametrize("M,I", [(5, 64), (16, 800), (33, 208), (65, 64), (300, 400), (600, 3584)])
def test_one_weight_scale_per_k_block(M, K, I):
    """Weight blocks as tall as the matrix and contractions shorter than the slabs
    that are copied ahead: scale buffers of one or two floats."""
    bn = 2 * I + 64 - 2 * I % 64
    (a, sa, w, sw), xv, wv = operands(M, K, I, bn, 128)
    assert sw.numel() == K // 128
    h = q8().blockwise_scaled_gated_mm(*to(a, w, sa, sw), block=(bn, 128))
    for r in (slice(0, 140), slice(max(M - 140, 0), M)):
        want, err = expect(xv[r], wv, "silu")
        check(h[r], want, err, "bf16", "h")
