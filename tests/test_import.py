"""The package imports with a torch that was built without CUDA (CPU)."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_imports_without_the_cuda_bindings():
    code = ("import torch\n"
            "for name in [n for n in dir(torch._C) if n.startswith('_cuda')]:\n"
            "    delattr(torch._C, name)\n"
            "import gemm_cq_gemv_gb300 as cq\n"
            "print(cq.f8_row_bytes(129))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "256"
