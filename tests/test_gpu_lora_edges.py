"""lora_mm at the edge of what it allows, and its kernels of many rows over many
slabs, ranges and row blocks, against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import gated as og
from tests.gpu_util import DEV, q8
from tests.test_gpu_gated import check, f64, make
from tests.test_gpu_lora import inputs, pattern

pytestmark = pytest.mark.gpu


def test_no_rows():
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    x, a, b, base = e(0, 64), e(2, 16, 64), e(2, 48, 16), e(0, 48)
    it = torch.empty(0, dtype=torch.int32, device=DEV)
    assert q8().lora_mm(x, a, b, it).shape == (0, 48)
    assert q8().lora_mm(x, a, b, it, torch.ones(2, device=DEV), base=base).shape == (0, 48)
    assert q8().lora_mm(x, a, b, it, base=base, out=base) is base


@pytest.mark.parametrize("M", [3, 600, 1100])  # the last through lora_join
def test_an_infinite_rank_beside_values_above_f16(M):
    """One infinite term of x A^T leaves the others what they are: they lie above
    f16's largest value and must not become infinities of the other sign."""
    K, N, R = 64, 1700, 16
    x = torch.full((M, K), 40.0, dtype=torch.float16)
    a = torch.full((1, R, K), 40.0, dtype=torch.float16)
    a[0, 5, 3] = float("inf")
    b = torch.full((1, N, R), -1.0, dtype=torch.float16)
    b[0, :, 5] = 1.0
    ids = torch.zeros(M, dtype=torch.int32)
    got = q8().lora_mm(*[t.to(DEV) for t in (x, a, b, ids)])
    assert (got == float("inf")).all()


# lora_shrink_tile with several slabs per range and several ranges (whose partials
# lora_join adds), lora_expand_tile with one to four blocks of rows per workgroup,
# the last one ragged: on 256 compute units
MANY = [(1100, 1032, 2052, 24, 9), (2100, 2056, 2052, 64, 5), (1100, 2056, 7168, 64, 4), (600, 520, 4100, 24, 20),
        (1500, 520, 5001, 128, 3), (4099, 2056, 2052, 40, 6)]


def some(M):
    """Rows to compare: the first and the last ones, and some of the rest."""
    return np.unique(np.concatenate([np.arange(70), np.arange(70, M - 70, 13), np.arange(M - 70, M)]))


@pytest.mark.parametrize("M,K,N,R,L", MANY)
@pytest.mark.parametrize("kind,dtype", [("runs", "bf16"), ("mixed", "f16"), ("one", "f16")])
def test_many_rows(M, K, N, R, L, kind, dtype):
    ids = pattern(kind, M, L)
    x, a, b, it = inputs(M, K, N, R, L, dtype, ids)
    s = torch.tensor(np.random.default_rng(7).uniform(0.25, 2, size=L)).float()
    base = make((M, N), dtype, 8)
    got = q8().lora_mm(x.to(DEV), a.to(DEV), b.to(DEV), it.to(DEV), s.to(DEV), base=base.to(DEV))
    r = some(M)
    want, err = og.lora(f64(x)[r], f64(a), f64(b), ids[r], s.double().numpy(), f64(base)[r], dtype)
    check(got[torch.tensor(r, device=DEV)], want, err, dtype, "out")


@pytest.mark.parametrize("M,K,N,R,L", [(1500, 520, 2100, 24, 3), (2101, 264, 2052, 64, 4)])
def test_many_rows_in_place_and_column_views(M, K, N, R, L):
    ids = pattern("mixed", M, L)
    x, a, b, it = inputs(M, K, N, R, L, "bf16", ids)
    wide = make((M, 2 * N + 4), "bf16", 8)
    buf = wide.to(DEV)
    part = buf[:, 4:4 + N]
    alone = q8().lora_mm(x.to(DEV), a.to(DEV), b.to(DEV), it.to(DEV), base=part.clone())
    assert q8().lora_mm(x.to(DEV), a.to(DEV), b.to(DEV), it.to(DEV), base=part, out=part) is part
    assert torch.equal(part, alone)
    assert torch.equal(buf[:, :4].cpu(), wide[:, :4]) and torch.equal(buf[:, 4 + N:].cpu(), wide[:, 4 + N:])
    xs = torch.zeros((M, K + 24), dtype=torch.bfloat16)
    xs[:, 8:8 + K] = x
    # an odd first column: rows that are not 8-byte aligned
    out = torch.zeros((M, N + 3), dtype=torch.bfloat16, device=DEV)
    q8().lora_mm(xs.to(DEV)[:, 8:8 + K], a.to(DEV), b.to(DEV), it.to(DEV), base=wide.to(DEV)[:, 4:4 + N], out=out[:, 1:1 + N])
    assert torch.equal(out[:, 1:1 + N], alone) and (out[:, 0] == 0).all() and (out[:, 1 + N:] == 0).all()
    r = some(M)
    want, err = og.lora(f64(x)[r], f64(a), f64(b), ids[r], None, f64(wide)[r][:, 4:4 + N], "bf16")
    check(alone[torch.tensor(r, device=DEV)], want, err, "bf16", "out")


def test_many_rows_without_an_adapter():
    M, K, N, R, L = 1300, 136, 2052, 24, 2
    x, a, b, it = inputs(M, K, N, R, L, "bf16", pattern("none", M, L))
    base = make((M, N), "bf16", 8).to(DEV)
    assert torch.equal(q8().lora_mm(x.to(DEV), a.to(DEV), b.to(DEV), it.to(DEV), base=base), base)
    assert (q8().lora_mm(x.to(DEV), a.to(DEV), b.to(DEV), it.to(DEV)) == 0).all()


def test_many_rows_do_not_meet():
    """NaN and infinities in one adapter or row stay with its rows, also where rows
    without an adapter lie between them."""
    M, K, N, R, L = 1300, 584, 2052, 24, 4
    ids = np.arange(M) % (L + 1) - 1
    x, a, b, it = inputs(M, K, N, R, L, "f16", ids)
    ref = q8().lora_mm(x.to(DEV), a.to(DEV), b.to(DEV), it.to(DEV))
    a[2], b[3] = float("nan"), float("inf")
    x[(ids == 1) & (np.arange(M) % 7 == 0)] = float("nan")
    x[ids < 0] = float("inf")
    got = q8().lora_mm(x.to(DEV), a.to(DEV), b.to(DEV), it.to(DEV))
    clean = torch.tensor((ids < 2) & ~((ids == 1) & (np.arange(M) % 7 == 0)), device=DEV)
    assert torch.equal(got[clean], ref[clean])
    assert not torch.isfinite(got[~clean]).any()
    assert (got[torch.tensor(ids < 0, device=DEV)] == 0).all()
