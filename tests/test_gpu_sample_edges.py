"""Filtered sampling where the filters' passes hand borders on to one another, and
for rows and numbers at the ends of what the calls accept.  Tolerances are those of
test_gpu_sample.py."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_best_gb300 import binding
from tests import indep_serving as ref
from tests.test_gpu_sample import NEAR, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_best_gb300 import build
    build.build()
    binding.load()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("R,V", [(1, 60000), (1, 151936), (30, 30000), (200, 20000)])
@pytest.mark.parametrize("low", [-2.0 ** -11, -2.0 ** -9])
def test_a_border_near_zero_after_ties(io, R, V, low):
    """top_k's border splits equal logits, top_p's then lies among logits within 2^-12
    of 0, too many for a list.  With the maximum -2^-13 the keys of the maximum and of
    the ties differ by powers of two (2^24 and 2^25): a selection whose range went by
    each CTA's own part of the ties had ranges of different widths."""
    x = np.where(np.arange(V) % 2 == 0, -2.0 ** -13, low) * np.ones((R, 1))
    k = 3 * V // 4
    assert ref.sample(x[0], 1.0, k, float(np.float32(0.3)))[2] >= NEAR
    n = check(x, io, k=[k] * R, p=[0.3] * R)
    assert len(n) == R and abs(n[0] - 0.3 * k) < 0.01 * k
