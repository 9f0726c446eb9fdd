"""Calls of the operators whose checks and launches are followed on the host: nothing here
reaches a GPU."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_cuda_in_torch():
    """A torch built for the CPU alone has no stream handles; importing needs none."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
            "    del torch._C._cuda_getCurrentRawStream\n"
            "from grammar_constrained_logit_gb300 import ops\n"
            "assert ops.get_bitmask_shape(2, 33) == (2, 2)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
