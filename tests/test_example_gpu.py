"""The decoding example runs and agrees with its plain form on a GB300."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens", ["1", "20"])
def test_moe_decode(tokens):
    from dense_fp16_gemm_f16_gb300 import build as gbuild
    gbuild.build()
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "moe_decode.py"), "--tokens", tokens, "--layers", "2",
                          "--hidden", "512", "--inner", "384", "--experts", "8", "--top", "2", "--steps", "3"],
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr
    assert "us per step" in out.stdout
