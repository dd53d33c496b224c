"""Calls at the edge of what the gated and adapter entry points allow, as far as
they can be seen without a GPU."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "int8_quantized_gemm_amd", "libq8gemm.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libq8gemm.so not built")


def test_size_queries_without_rows():
    """An empty batch needs no workspace (asked for in a process of its own: a
    division by the number of row tiles ended it)."""
    code = ("import int8_quantized_gemm_amd as q\n"
            "print(q._lora_ws(0, 64, 16), q._lora_ws(0, 8, 8), q._lora_ws(0, 1 << 20, 128), q._gated_ws(0, 64, 64),\n"
            "      q._gatedb_ws(0, 64, 64), q._bgated_ws(0, 128, 128, 128, 128, 0), q._bgated_ws(0, 128, 128, 32, 32, 1))")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["0"] * 7


@pytest.fixture(scope="module")
def q8():
    import int8_quantized_gemm_amd as m
    return m


def test_empty_batches_of_any_strides(q8):
    """torch calls a tensor without elements contiguous whatever its strides."""
    w, a, b = torch.zeros(12, 16).bfloat16(), torch.zeros(3, 8, 16).bfloat16(), torch.zeros(3, 20, 8).bfloat16()
    ids = torch.zeros(0, dtype=torch.int32)
    for x in (torch.empty_strided((0, 16), (0, 0), dtype=torch.bfloat16), torch.zeros(16, 4).bfloat16().t()[:0]):
        assert x.is_contiguous()
        for call in (lambda: q8.gated_mm(x, w), lambda: q8.lora_mm(x, a, b, ids),
                     lambda: q8.lora_mm(x, a, b, ids, base=torch.empty_strided((0, 20), (1, 7), dtype=torch.bfloat16))):
            with pytest.raises(ValueError, match="on the GPU"):
                call()


def test_sizes_are_asked_for_on_the_tensors_device(q8, monkeypatch):
    """The workspace of a call depends on its device's compute units, whichever device
    is current, and is remembered for each."""
    now, asked = [0], []

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.before, now[0] = now[0], self.d

        def __exit__(self, *exc):
            now[0] = self.before

    def sizes(M, I):
        asked.append(now[0])
        return 100 * (now[0] + 1) + M + I

    monkeypatch.setattr(q8.torch.cuda, "device", Device)
    monkeypatch.setattr(q8.torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(q8, "_ws_sizes", {})
    assert [q8._scratch_size(d, sizes, 3, 4) for d in (0, 1, 0, 1)] == [107, 207, 107, 207]
    assert asked == [0, 1] and now == [0]


def test_a_missing_library_names_a_command_that_builds_it(tmp_path):
    """The package cannot be imported before it is built, so not `python -m` of it."""
    pkg = tmp_path / "int8_quantized_gemm_amd"
    pkg.mkdir()
    (pkg / "__init__.py").write_text(open(os.path.join(ROOT, "int8_quantized_gemm_amd", "__init__.py")).read())
    r = subprocess.run([sys.executable, "-c", "import int8_quantized_gemm_amd"], cwd=tmp_path, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode and "ImportError" in r.stderr and "`python int8_quantized_gemm_amd/build.py`" in r.stderr
    assert os.path.exists(os.path.join(ROOT, "int8_quantized_gemm_amd", "build.py"))
