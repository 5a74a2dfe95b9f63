"""The binding and torch share one HIP runtime, whichever is imported first."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("imports", ["from fp64_gemm_emulation_amd import binding; import torch",
                                     "import torch; from fp64_gemm_emulation_amd import binding"])
def test_one_hip_runtime(imports):
    code = imports + "\nprint(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))"
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    assert out.stdout.split() == ["1"]
