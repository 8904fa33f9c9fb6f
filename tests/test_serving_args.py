"""Host-side checks of the serving operators at the ends of their ranges (no
kernel is launched)."""
import ctypes

import pytest

from speculative_decoding_tree_best_gb300 import binding
from tests.test_chain_args import draft, lib  # noqa: F401


@pytest.mark.parametrize("V", [(1 << 30) + 1, (1 << 31) - 4096, (1 << 31) - 1])
def test_vocabularies_beyond_the_kernels_indices_are_refused(lib, V):  # noqa: F811
    cfg = binding.draft_cfg(B=1, N=1, V=V)
    assert draft(lib, cfg) == binding.ST_EINVAL
    assert lib.spec_draft_workspace_bytes(ctypes.byref(cfg), 152) == 0
    assert lib.spec_draft_workspace_bytes(ctypes.byref(binding.draft_cfg(B=1, N=1, V=1 << 30)), 152) > 0


def test_every_finite_temperature_is_accepted(lib):  # noqa: F811
    for t in (3.4028234663852886e38, 3.1e38, 1e-45):
        cfg = binding.draft_cfg(B=1, N=1, V=10, temperature=t)
        assert lib.spec_draft_workspace_bytes(ctypes.byref(cfg), 152) > 0
