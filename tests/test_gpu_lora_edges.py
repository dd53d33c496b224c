"""lora_mm at the edge of what it allows, and its kernels of many rows over many
slabs, ranges and row blocks, against the float64 oracle."""
import pytest
import torch

from tests.gpu_util import DEV, q8

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
