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
