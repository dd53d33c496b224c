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


def ends(M, n=130):
    return (slice(0, min(n, M)), slice(max(M - n, 0), M))


# on 256 compute units, K blocks of 32: a split contraction in tiles of 64 and of 128
# rows; tiles of 256 columns whose ring of stages comes round more than once;
# tiles of 128 columns in more than one round
@pytest.mark.parametrize("M,K,I", [(20, 2048, 64), (100, 1536, 64), (130, 2048, 144), (2100, 640, 1104), (600, 1024, 3600),
                                   (1000, 384, 5504), (1000, 640, 5504)])
def test_blocks_of_32(M, K, I):
    (a, sa, w, sw), xv, wv = operands(M, K, I, 32, 32)
    delta = make((M, 2 * I), "bf16", 3)
    h = q8().blockwise_scaled_gated_mm(*to(a, w, sa, sw), activation="gelu", block=(32, 32), delta=delta.to(DEV))
    for r in ends(M):
        want, err = expect(xv[r], wv, "gelu", f64(delta)[r])
        check(h[r], want, err, "bf16", "h")


def check_quantized(q, s, want, err):
    """Codes and scales against float64 values and a bound of the float32 ones (as in
    test_gpu_gated_fp8.test_quantized_output)."""
    M = want.shape[0]
    top, etop = np.abs(want).reshape(M, -1, 128).max(2), err.reshape(M, -1, 128).max(2)
    sv = s.cpu().double().numpy()
    assert np.all(np.abs(sv - np.maximum(top, 1e-10) / 448) <= etop / 448 + 2 * F32 * (top + etop) / 448)
    back = decode(codes(q)) * np.repeat(sv, 128, axis=1)
    bound = (np.abs(want) + err) * (2.0 ** -4 + 2 * F32) + np.repeat(sv, 128, axis=1) * 2.0 ** -10 + err
    assert np.all(np.abs(back - want) <= bound)
    assert (np.abs(decode(codes(q))).reshape(M, -1, 128).max(2) == 448).all()


# K blocks of 128: a few rows, small tiles, a split contraction, large tiles whole, all in
# halves, and the last 32 of 288 in halves; K blocks of 32: few rows, tiles of 64 and of 128
# rows, a split contraction, tiles of 256 and of 128 columns
@pytest.mark.parametrize("M,K,I,bk", [(3, 256, 128, 128), (16, 384, 256, 128), (40, 384, 256, 128), (100, 256, 384, 128),
                                      (100, 4096, 128, 128), (1100, 256, 3584, 128), (600, 256, 3584, 128),
                                      (4400, 256, 2048, 128), (4481, 384, 2048, 128),
                                      (1, 128, 128, 32), (5, 256, 128, 32), (40, 384, 256, 32), (100, 256, 384, 32),
                                      (20, 2048, 128, 32), (100, 1536, 128, 32), (2100, 512, 1152, 32), (1000, 256, 5504, 32)])
@pytest.mark.parametrize("name,with_delta", [("silu", True), ("gelu", False), ("gelu_tanh", True)])
def test_quantized(M, K, I, bk, name, with_delta):
    (a, sa, w, sw), xv, wv = operands(M, K, I, bk, bk)
    delta = make((M, 2 * I), "f16", 3, 2.0) if with_delta else None
    q, s = q8().blockwise_scaled_gated_mm(*to(a, w, sa, sw), torch.float8_e4m3fn, name, (bk, bk),
                                          delta=None if delta is None else delta.to(DEV))
    for r in ends(M):
        want, err = expect(xv[r], wv, name, None if delta is None else f64(delta)[r])
        check_quantized(q[r], s[r], want, err)


# delta through LDS in whole tiles and in halves, in both types
@pytest.mark.parametrize("M,K,I", [(1100, 256, 3584), (600, 384, 3584), (4400, 256, 2048), (4481, 640, 2048)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_big_tiles_delta(M, K, I, dtype):
    (a, sa, w, sw), xv, wv = operands(M, K, I, 128, 128)
    delta = make((M, 2 * I), dtype, 3, 2.0)
    h = q8().blockwise_scaled_gated_mm(*to(a, w, sa, sw), T[dtype], delta=delta.to(DEV))
    for r in ends(M):
        want, err = expect(xv[r], wv, "silu", f64(delta)[r])
        check(h[r], want, err, dtype, "h")


@pytest.mark.parametrize("M,K,I,bk", [(3, 256, 128, 128), (40, 256, 128, 128), (100, 4096, 128, 128), (600, 256, 3584, 128),
                                      (1100, 256, 3584, 128), (40, 256, 128, 32), (100, 1536, 128, 32), (2100, 256, 1152, 32)])
def test_rows_that_are_not_aligned(M, K, I, bk):
    """h and delta two bytes past an aligned address; of a quantized result delta."""
    (a, sa, w, sw), _, _ = operands(M, K, I, bk, bk)
    args, delta = to(a, w, sa, sw), make((M, 2 * I), "bf16", 3).to(DEV)
    f = q8().blockwise_scaled_gated_mm
    off = lambda t: torch.cat([t.flatten()[:1], t.flatten(), t.flatten()[:1]])[1:-1].view(t.shape)  # noqa: E731
    ref = f(*args, block=(bk, bk), delta=delta)
    d, out = off(delta), off(torch.zeros_like(ref))
    assert d.data_ptr() % 4 == 2 and out.data_ptr() % 4 == 2
    assert torch.equal(f(*args, block=(bk, bk), delta=d, out=out), ref)
    assert torch.equal(f(*args, block=(bk, bk), delta=delta, out=out.zero_()), ref)
    q, s = f(*args, torch.float8_e4m3fn, block=(bk, bk), delta=delta)
    q1, s1 = f(*args, torch.float8_e4m3fn, block=(bk, bk), delta=d)
    assert torch.equal(q.view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s, s1)
