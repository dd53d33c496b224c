"""The gated and adapter calls where outputs, operands and workspaces pass the range of
32-bit offsets: rows at both ends and around the 2^31st and 2^32nd element against
the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import gated as og
from tests.gpu_util import DEV, q8
from tests.test_gpu_gated import T, check, f64
from tests.test_gpu_gated_fp8 import expect

pytestmark = pytest.mark.gpu


def rand(shape, dtype, seed, std=1.0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = torch.empty(shape, dtype=dtype, device=DEV)
    for r in t.split(max(1, (1 << 26) // shape[-1])):
        r.copy_(torch.randn(r.shape, generator=gen, device=DEV) * std)
    return t


def rows_of(M, width):
    """Both ends, and where the row's first element passes 2^31 and 2^32."""
    at = [0, 1, 2, M - 3, M - 2, M - 1]
    for e in (1 << 31, 1 << 32):
        at += [e // width + d for d in (-1, 0, 1)]
    return sorted({r for r in at if 0 <= r < M})


def test_outputs_past_four_gib():
    M, K, I, dtype = 150001, 64, 16384, "bf16"
    x, w = rand((M, K), T[dtype], 1), rand((2 * I, K), T[dtype], 2, K ** -0.5)
    gate_up = torch.empty((M, 2 * I), dtype=T[dtype], device=DEV)
    h = q8().gated_mm(x, w, gate_up=gate_up)
    for r in (rows_of(M, I), rows_of(M, 2 * I)):
        want, gu, eh, eg = og.forward(f64(x[r]), f64(w), "silu")
        check(h[r], want, eh, dtype, "h")
        check(gate_up[r], gu, eg, dtype, "gate_up")
    # and read again as delta
    h2 = q8().gated_mm(x, w, delta=gate_up)
    r = rows_of(M, 2 * I)
    want, _, eh, _ = og.forward(f64(x[r]), f64(w), "silu", f64(gate_up[r]))
    check(h2[r], want, eh, dtype, "h with delta")


@pytest.mark.parametrize("I", [40, 300])  # small tiles and large ones
def test_x_close_to_four_gib(I):
    M, K, dtype = 261800, 8192, "f16"
    assert (M + 256) * K < 1 << 31 <= (M + 400) * K
    x, w = rand((M, K), T[dtype], 1), rand((2 * I, K), T[dtype], 2, K ** -0.5)
    h = q8().gated_mm(x, w)
    r = rows_of(M, K) + [(1 << 30) // K, (1 << 30) // K + 1]
    want, _, eh, _ = og.forward(f64(x[r]), f64(w), "silu")
    check(h[r], want, eh, dtype, "h")


def test_backward_close_to_four_gib():
    """[dG | dU] and x just below four GiB; dW's sums of 2^18 rows against float64 sums."""
    M, K, I, dtype = 261000, 8064, 4032, "bf16"
    assert (M + 256) * (2 * I + 64) < 1 << 31
    x, w = rand((M, K), T[dtype], 1), rand((2 * I, K), T[dtype], 2, K ** -0.5)
    gu, dh = rand((M, 2 * I), T[dtype], 3), rand((M, I), T[dtype], 4)
    d = torch.empty_like(gu)
    dx, dw = q8().gated_mm_backward(dh, x, w, gu, grad_gate_up=d)
    r = rows_of(M, 2 * I) + [(1 << 30) // K, (1 << 30) // (2 * I)]
    # dx of these rows: the oracle on them alone
    (wx, _, wd), (ex, _, ed) = og.backward(f64(dh[r]), f64(x[r]), f64(w), f64(gu[r]), "silu", dtype)
    check(d[r], wd, ed, dtype, "d gate_up")
    check(dx[r], wx, ex, dtype, "dx")
    # dW of some hidden units and columns, from the rounded gradients that the products
    # take (exact products, float32 sums of M terms)
    n, k = [0, 1, I - 1, I, 2 * I - 1], [0, 7, 4000, K - 1]
    dd, xx = d[:, n].double(), x[:, k].double()
    want = (dd.t() @ xx).cpu().numpy()
    mag = (dd.abs().t() @ xx.abs()).cpu().numpy()
    # M terms of random sign: the partial sums are about sqrt(M) terms large, their M
    # roundings add up like sqrt(M) of half a step each, so M terms' half steps, the
    # sum of magnitudes, is the error's size; 64 of them
    check(dw[n][:, k], want, 64 * og.F32 * mag, dtype, "dW")


def test_fp8_outputs_past_four_gib():
    M, K, I = 300001, 128, 8192
    rng = np.random.default_rng(5)
    a = rand((M, K), torch.bfloat16, 1, 100.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
    w = rand((2 * I, K), torch.bfloat16, 2, 100.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
    sa = torch.rand((M, 1), device=DEV) * 0.01 + 0.005
    sw = torch.tensor(rng.uniform(0.5, 1.5, size=(2 * I // 128, 1)) / 100 * K ** -0.5).float().to(DEV)
    h = q8().blockwise_scaled_gated_mm(a, w, sa, sw)
    q, s = q8().blockwise_scaled_gated_mm(a, w, sa, sw, torch.float8_e4m3fn)
    r = rows_of(M, I)
    xv = f64(a[r].float()) * f64(sa[r])
    wv = f64(w.float()) * np.repeat(f64(sw), 128, axis=0)
    want, err = expect(xv, wv, "silu")
    check(h[r], want, err, "bf16", "h")
    sv = np.repeat(f64(s[r]), 128, axis=1)
    back = f64(q[r].float()) * sv
    bound = (np.abs(want) + err) * (2.0 ** -4 + 2 * og.F32) + sv * 2.0 ** -10 + err
    assert np.all(np.abs(back - want) <= bound)


def test_adapters_past_four_gib():
    M, K, N, R, L = 100003, 64, 45056, 16, 3
    x, a, b = rand((M, K), torch.bfloat16, 1), rand((L, R, K), torch.bfloat16, 2, K ** -0.5), \
        rand((L, N, R), torch.bfloat16, 3, R ** -0.5)
    ids = (torch.arange(M, device=DEV) // 1000 % (L + 1) - 1).int()
    base = rand((M, N), torch.bfloat16, 4)
    r = rows_of(M, N)
    want, err = og.lora(f64(x[r]), f64(a), f64(b), ids[r].cpu().numpy(), None, f64(base[r]), "bf16")
    got = q8().lora_mm(x, a, b, ids, base=base, out=base)
    check(got[r], want, err, "bf16", "out")
