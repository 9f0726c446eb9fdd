"""Calls of the operators around their kernels: what a launch needs, what a failed one leaves
behind, whose scratch it uses."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from grammar_constrained_logit_gb300 import _lib  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.load()


EVERY_COUNT = """
import sys
import torch
from grammar_constrained_logit_gb300 import ops
for beams in map(int, sys.argv[1:]):
    t = torch.arange(2 * beams * 40, device="cuda", dtype=torch.int32).view(2 * beams, 40)
    p = torch.stack([(torch.arange(beams) * 7 + 1) % beams, torch.arange(beams) // 2])
    want = t.view(2, beams, 40).cpu().gather(1, p[..., None].expand(2, beams, 40))
    ops.reorder_states([t], p.int().cuda())
    assert torch.equal(t.view(2, beams, 40).cpu(), want), beams
"""


@pytest.mark.parametrize("counts", [[12], range(1, 257)])
def test_every_number_of_beams(counts):
    """In a process of its own, fewest beams first: how much shared memory a launch may
    take is set for the whole process by the first call that asks for more."""
    r = subprocess.run([sys.executable, "-c", EVERY_COUNT, *map(str, counts)], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
