"""Host-side checks of the rows that token_sample leaves out."""
import ctypes

import pytest

from speculative_decoding_tree_best_gb300 import binding
from tests.test_chain_args import P, lib  # noqa: F401


def test_idle_rows_are_checked(lib):  # noqa: F811
    cfg = binding.sample_cfg(2, 1000)
    out = binding.SpecSampleOut(16, 16, 16, 16)
    for last, idle in ((8, 0), (16, 2), (16, -1), (0, 2)):
        p = binding.SpecSampleParams(16, 16, 16, 16, last, idle)
        assert lib.token_sample(ctypes.byref(cfg), P, ctypes.byref(p), P, ctypes.byref(out), P,
                                None) == binding.ST_EINVAL


def test_layout_of_the_parameters():
    """The structure as the header has it: five pointers, then the rule."""
    assert binding.SpecSampleParams.last_row.offset == 32
    assert binding.SpecSampleParams.idle.offset == 40
    assert ctypes.sizeof(binding.SpecSampleParams) == 48
    with pytest.raises(KeyError):
        binding._IDLE["other"]
