"""A bounded wait inside the kernel of many rows made to run out, on the GPU.

The product build cannot reach this path on demand, so the test compiles its own copy of the
library with LP_TEST_CHUNK_TIMEOUT set: the loaders of the first two blocks poll a barrier on
which nothing ever arrives, 50 times, at the block's first tile and at its second, and give up.
All roles of those blocks stop.  The call must return normally, the blocks' queries must be NaN
and add NaN to the weights of what they see, whether they have been through a tile or not, and
all others must be as the product library has them.
"""
import ctypes

import numpy as np
import pytest

from grammar_constrained_logit_gb300 import _lib
from grammar_constrained_logit_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_queries_of_blocks_that_gave_up_are_nan(dtype, monkeypatch):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from grammar_constrained_logit_gb300 import ops
    from test_gpu_attend import TYPES, filled

    path = build.build_variant("chunk_timeout_test", {"LP_TEST_CHUNK_TIMEOUT": 50},
                               sources=("attend_chunk.cu",), rest=True)
    lib = ctypes.CDLL(path)
    _lib.declare(lib)
    _lib.declare_beam(lib)
    _lib.declare_attend(lib)

    # a head's 1200 queries are 5 blocks of 256, the last ones first; 600 tokens are 5 tiles
    rows, heads, shared, batch, n = 600, 8, 2, 2, 640
    cache = filled(batch * n, heads, 128, 8, 128, page=16)
    g = torch.Generator("cuda").manual_seed(3)
    q = torch.randn(batch, rows, heads * shared, 128, device="cuda", generator=g).to(TYPES[dtype])
    blocks = torch.arange(batch * n // 16, dtype=torch.int32, device="cuda").view(batch, -1)
    lengths = torch.full((batch,), n, dtype=torch.int32, device="cuda")

    def call():
        weights = torch.zeros(batch, heads, n, device="cuda")
        out = ops.cache_attend(cache, q, blocks, lengths, weights=weights)
        torch.cuda.synchronize()
        return out.float().cpu().numpy(), weights.cpu().numpy()

    want, weighed = call()
    assert np.isfinite(want).all() and np.isfinite(weighed).all()
    monkeypatch.setattr(_lib, "load", lambda: lib)
    lost = np.zeros(want.shape, bool)
    for r in range(rows):
        for j in range(shared):
            lost[0, r, j] = r * shared + j >= 3 * 256  # of head 0: rows of the last two blocks
    for _ in range(2):
        got, w = call()
        assert np.isnan(got[lost]).all() and np.array_equal(got[~lost], want[~lost])
        # the last row of all sees every token
        assert np.isnan(w[0, 0]).all()
        assert np.array_equal(w[0, 1:], weighed[0, 1:]) and np.array_equal(w[1], weighed[1])
    monkeypatch.undo()
    got, w = call()
    assert np.array_equal(got, want) and np.array_equal(w, weighed)
