"""gated_mm and gated_mm_backward at the edge of what they allow, and their
kernels over many slabs, ranges and rounds, against the float64 oracle."""
import math

import numpy as np
import pytest
import torch

from oracle import gated as og
from tests.gpu_util import DEV, q8
from tests.test_gpu_gated import T, back, check, f64, make

pytestmark = pytest.mark.gpu


def gradients(M, K, I, name, dh_std, u_std, w_std, x_std, seed=0):
    """f16 operands of a backward pass, the gradients and their bounds: float32
    sums, and [dG | dU] rounded once to f16 with its largest value brought to
    [2^14, 2^15), so that the smallest values are off by 2^-25 of 2^(e - 15), with
    2^e the power of two above the largest (one more where the kernel's float32
    value lies across a power of two)."""
    x, w = make((M, K), "f16", [seed, 1], x_std), make((2 * I, K), "f16", [seed, 2], w_std)
    gu, dh = make((M, 2 * I), "f16", [seed, 3], 1.5), make((M, I), "f16", [seed, 4], dh_std)
    gu[:, I:] *= u_std
    d = og.backward(f64(dh), np.zeros((M, 1)), np.zeros((2 * I, 1)), f64(gu), name, "f16")[0][2]
    e = math.frexp(np.abs(d).max())[1] + 1
    ref = og.backward(f64(dh), f64(x), f64(w), f64(gu), name, "f16", 2.0 ** (e - 15 - 25))
    return (dh, x, w, gu), ref


# one launch for both products; ranges of the contraction; large tiles; few rows
SHAPES = [(200, 264, 130), (700, 136, 40), (140, 136, 1500), (2100, 2056, 131), (300, 2056, 1100), (20, 72, 45)]


# the activations differ in the first kernels only
@pytest.mark.parametrize("M,K,I,name", [(*s, "silu") for s in SHAPES] +
                         [(*s, n) for s in SHAPES[:1] + SHAPES[5:] for n in ("gelu", "gelu_tanh")])
def test_f16_gradients_of_small_values(M, K, I, name):
    """Gradients of 1e-6, among f16's subnormals, whose sums with large operands are
    ordinary numbers."""
    args, ((wx, ww, _), (ex, ew, _)) = gradients(M, K, I, name, 1e-6, 1.0, 30 * K ** -0.5, 30.0)
    dx, dw = q8().gated_mm_backward(*[t.to(DEV) for t in args], name)
    check(dx, wx, ex, "f16", "dx")
    check(dw, ww, ew, "f16", "dW")


@pytest.mark.parametrize("M,K,I", SHAPES)
def test_f16_gradients_above_the_largest_f16(M, K, I):
    """Gradients of the pre-activations of up to 1e6 between small operands."""
    args, ((wx, ww, wd), (ex, ew, ed)) = gradients(M, K, I, "silu", 300.0, 300.0, 2.0 ** -10, 2.0 ** -10)
    assert np.abs(wd).max() > 2 * 65504
    grad_gate_up = torch.empty((M, 2 * I), dtype=torch.float16, device=DEV)
    dx, dw = q8().gated_mm_backward(*[t.to(DEV) for t in args], grad_gate_up=grad_gate_up)
    check(dx, wx, ex, "f16", "dx")
    check(dw, ww, ew, "f16", "dW")
    # the gradient of the pre-activations itself is an f16 output
    got, fits = f64(grad_gate_up), np.abs(wd) < 65000
    assert not og.within(got[fits], wd[fits], ed[fits], "f16").any()
    assert np.isinf(got[np.abs(wd) > 66000]).all()


def test_f16_gradients_beside_a_row_that_is_not_finite():
    M, K, I = 200, 264, 130
    args, ((wx, _, _), (ex, _, _)) = gradients(M, K, I, "silu", 1e-6, 1.0, 30 * K ** -0.5, 30.0)
    dh = args[0].clone()
    dh[7, 3], dh[9, 5] = float("inf"), float("nan")
    dx, _ = q8().gated_mm_backward(*[t.to(DEV) for t in (dh, *args[1:])])
    keep = [i for i in range(M) if i not in (7, 9)]
    check(dx[keep], wx[keep], ex[keep], "f16", "dx")
    assert not torch.isfinite(dx[[7, 9]]).any()


def test_f16_gradients_that_are_all_zero():
    M, K, I = 70, 72, 40
    args, _ = gradients(M, K, I, "silu", 1.0, 1.0, 1.0, 1.0)
    dx, dw = q8().gated_mm_backward(*[t.to(DEV) for t in (torch.zeros_like(args[0]), *args[1:])])
    assert (dx == 0).all() and (dw == 0).all()


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradients_at_pre_activations_of_any_size(name, dtype):
    """act and act' from the smallest to the largest finite pre-activations."""
    top = float(torch.finfo(T[dtype]).max)
    g = [10.0 ** e for e in range(-7, 39) if 10.0 ** e < top] + [0.0, 0.5, 2.0, 3.0, 5.5, 20.0, 85.0, top]
    g = torch.tensor(sorted(g + [-v for v in g])).to(T[dtype])[None]
    I, K = g.shape[1], 8
    u, dh = torch.full_like(g, 0.75), torch.full_like(g, 0.5)
    gu = torch.cat([g, u], 1)
    d = torch.empty((1, 2 * I), dtype=T[dtype], device=DEV)
    q8().gated_mm_backward(dh.to(DEV), torch.zeros((1, K), dtype=T[dtype], device=DEV),
                           torch.zeros((2 * I, K), dtype=T[dtype], device=DEV), gu.to(DEV), name, need_x=False, need_w=False,
                           grad_gate_up=d)
    (_, _, want), (_, _, err) = og.backward(f64(dh), np.zeros((1, K)), np.zeros((2 * I, K)), f64(gu), name, dtype)
    # the derivative's own error (oracle/gated.py: 32 half steps of 1 + |g|) is that of
    # values near the bend; past it act' is 0 or 1 to float32
    far = np.abs(np.concatenate([f64(g), f64(g)], 1)) > 200
    err = np.where(far, 4 * og.F32 * np.abs(want), err)
    check(d, want, err, dtype, name)


# on 256 compute units: large tiles, whole (3 and 8 slabs) and all in halves (5), with
# the last 32 of 288 in halves (7); a split contraction in tiles of 128 and of 64 rows
@pytest.mark.parametrize("M,K,I", [(3850, 136, 1701), (3850, 456, 1700), (2100, 264, 1031), (4400, 392, 1930),
                                   (100, 2568, 63), (300, 2568, 259), (20, 2568, 64)])
@pytest.mark.parametrize("name,dtype", [("silu", "bf16"), ("gelu", "f16")])
def test_forward_delta(M, K, I, name, dtype):
    x, w = make((M, K), dtype, 1), make((2 * I, K), dtype, 2, K ** -0.5)
    delta = make((M, 2 * I), dtype, 3, 2.0)
    gate_up = torch.empty((M, 2 * I), dtype=T[dtype], device=DEV)
    h = q8().gated_mm(x.to(DEV), w.to(DEV), name, delta=delta.to(DEV), gate_up=gate_up)
    want, gu, eh, eg = og.forward(f64(x), f64(w), name, f64(delta))
    check(h, want, eh, dtype, "h")
    check(gate_up, gu, eg, dtype, "gate_up")


def test_forward_rows_that_are_not_aligned():
    """Outputs and delta two bytes past an aligned address, in every kernel."""
    for M, K, I in ((3, 136, 66), (40, 136, 66), (100, 136, 66), (100, 2568, 66), (2100, 136, 1030)):
        x, w, delta = make((M, K), "bf16", 1), make((2 * I, K), "bf16", 2, K ** -0.5), make((M, 2 * I), "bf16", 3)
        gate_up = torch.empty((M, 2 * I), dtype=torch.bfloat16, device=DEV)
        ref = q8().gated_mm(x.to(DEV), w.to(DEV), delta=delta.to(DEV), gate_up=gate_up)
        off = lambda t: torch.cat([t.flatten()[:1], t.flatten(), t.flatten()[:1]])[1:-1].view(t.shape)  # noqa: E731
        d, gu, out = off(delta.to(DEV)), off(torch.zeros_like(gate_up)), off(torch.zeros_like(ref))
        assert d.data_ptr() % 4 == 2 and out.data_ptr() % 4 == 2
        assert torch.equal(q8().gated_mm(x.to(DEV), w.to(DEV), delta=d, gate_up=gu, out=out), ref)
        assert torch.equal(gu, gate_up)


# dx, then dW, in large tiles over four slabs and more: whole, in halves, and the last
# of 306 in halves; either in ranges of its contraction
@pytest.mark.parametrize("M,K,I", [(3600, 3208, 131), (3600, 3208, 128), (4400, 4104, 100), (2100, 2056, 131),
                                   (333, 3208, 1900), (300, 3208, 1901), (257, 4104, 2200), (300, 2056, 1100),
                                   (100, 200, 1400), (300, 136, 1300), (2600, 200, 50), (2600, 264, 131)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_backward_long_contractions(M, K, I, dtype):
    back(M, K, I, dtype, "silu")


class GatedMM(torch.autograd.Function):
    """gated_mm in a graph, as its documentation says a caller writes it."""

    @staticmethod
    def forward(ctx, x, w, activation):
        gate_up = torch.empty((x.shape[0], w.shape[0]), dtype=x.dtype, device=x.device)
        h = q8().gated_mm(x, w, activation, gate_up=gate_up)
        ctx.save_for_backward(x, w, gate_up)
        ctx.activation = activation
        return h

    @staticmethod
    def backward(ctx, grad_out):
        x, w, gate_up = ctx.saved_tensors
        gx, gw = q8().gated_mm_backward(grad_out.contiguous(), x, w, gate_up, ctx.activation,
                                        need_x=ctx.needs_input_grad[0], need_w=ctx.needs_input_grad[1])
        return gx, gw, None


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_autograd_function(dtype):
    """Eager, with one gradient only, and captured while no eager graph of the leaves
    lives; replayed with the program's own steps between."""
    M, K, I = 150, 200, 90
    x, w, c = make((M, K), dtype, 1).to(DEV), make((2 * I, K), dtype, 2, K ** -0.5).to(DEV), make((M, I), dtype, 3).to(DEV)
    gate_up = torch.empty((M, 2 * I), dtype=T[dtype], device=DEV)
    h = q8().gated_mm(x, w, "gelu_tanh", gate_up=gate_up)
    ref = q8().gated_mm_backward(c, x, w, gate_up, "gelu_tanh")
    xl, wl = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    # the call itself leaves no graph
    assert q8().gated_mm(xl, wl).requires_grad is False

    def step():
        y = GatedMM.apply(xl, wl, "gelu_tanh")
        return y.detach(), *torch.autograd.grad(y, (xl, wl), c)

    assert all(torch.equal(a, b) for a, b in zip(step(), (h, *ref)))
    y = GatedMM.apply(xl, w, "gelu_tanh")
    assert torch.equal(torch.autograd.grad(y, xl, c)[0], ref[0])
    # a gradient without strides of its own
    y = GatedMM.apply(xl, wl, "gelu_tanh")
    one = torch.autograd.grad(y.float().sum(), wl)[0]
    assert torch.equal(one, q8().gated_mm_backward(torch.ones_like(c), x, w, gate_up, "gelu_tanh")[1])
    del y
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for k in range(3):
        with torch.no_grad():
            xl.copy_(x.roll(k, 0))
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """Backward passes of different sizes side by side: each call has its workspace."""
    m = q8()
    sets = []
    for M, K, I, dtype in ((700, 136, 40, "f16"), (100, 200, 1400, "f16"), (300, 264, 130, "bf16")):
        t = [make((M, I), dtype, 4), make((M, K), dtype, 1), make((2 * I, K), dtype, 2, K ** -0.5), make((M, 2 * I), dtype, 3)]
        sets.append([v.to(DEV) for v in t])
    ref = [m.gated_mm_backward(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                outs.append(m.gated_mm_backward(*s))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert all(torch.equal(a, b) for a, b in zip(o, ref[i % 3]))
