"""Tables of a caller's own frequencies: the ramp over the pair's index, against the
rotation in 64 bits."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_tree_best_gb300 import binding
from tests.test_gpu_rope import near, randn

pytestmark = pytest.mark.gpu


def ramp_over_the_index(rot, base, factor, orig_len, beta_fast=32.0, beta_slow=1.0):
    def dim(turns):
        return rot * math.log(orig_len / (turns * 2 * math.pi)) / (2 * math.log(base))
    low, high = max(math.floor(dim(beta_fast)), 0), min(math.ceil(dim(beta_slow)), rot - 1)
    j = np.arange(rot // 2)
    f = base ** (-2.0 * j / rot)
    keep = 1 - np.clip((j - low) / max(high - low, 0.001), 0, 1)
    return f / factor * (1 - keep) + f * keep


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rot,factor", [(128, 4.0), (64, 40.0), (16, 1.0)])
def test_rotation_by_given_frequencies(io, rot, factor):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_best_gb300 import build
    build.build()
    rows, Hq, Hkv = 77, 3, 1
    f, amp = ramp_over_the_index(rot, 1e6, factor, 32768), 0.1 * math.log(factor) + 1
    table = binding.RopeTable.from_frequencies(f, amp)
    assert table.rot == rot and table.amp == amp
    pos = np.random.default_rng(rot).integers(0, 1 << 17, rows).astype(np.int32)
    q, k = randn((rows, Hq, 128), io, 1), randn((rows, Hkv, 128), io, 2)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    binding.rope_apply(binding.rope_cfg(rows, Hq, Hkv, 128, rot, io=io), table,
                       torch.from_numpy(pos).cuda(), q, k, qo, ko)
    near(qo, q, pos, f, amp, "half", io)
    near(ko, k, pos, f, amp, "half", io)
