"""Calls at the edge of what the gated and adapter entry points allow, as far as
they can be seen without a GPU."""
import os
import subprocess
import sys

import pytest

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
