"""The step that checks drafted tokens, where its kernels and calls could go wrong in
ways that random inputs do not show.  GPU, against the 64-bit oracle or exact values.

Tolerances are those of test_gpu_draft_step.py, or exact; the others are derived where
they stand.
"""
import numpy as np
import pytest

from gpu_util import need_gpu, torch
from test_gpu_draft_step import Tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.fixture(autouse=True)
def _clean():
    import dsa_sparse_mla_prefill_gb300 as dsa
    dsa.dsa_last_device_error()
    yield
    st, counts = dsa.dsa_last_device_error()
    assert st == 0 and counts[1] == 0, counts


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("n,H", [(3, 16), (7, 16), (8, 32)])
@pytest.mark.parametrize("per_range", [2, 3, 5])
def test_tree_requests_that_end_behind_one_another(fmt, n, H, per_range):
    """Ranges whose last tile is a whole request right behind another request's end, with sums that differ by orders
    of magnitude: each request is divided by its own sum, in every call."""
    rng = np.random.default_rng(per_range)
    blocks = -(-n * H // 128)
    B = 76 // blocks * per_range                        # one tile each
    lens = np.where(np.arange(B) % 2, rng.integers(n, n + 4, B), rng.integers(230, 257, B)).astype(np.int32)
    t = Tree(per_range, lens, n, H, fmt=fmt, bs=64)
    out, lse = t.run()
    t.check((out, lse))
    for _ in range(20):
        again = t.run()
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
