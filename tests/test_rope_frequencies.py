"""Tables of a caller's own frequencies: the ramp over the pair's index, against the
rotation in 64 bits."""
import math
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

from speculative_decoding_tree_best_gb300 import binding
from tests.test_gpu_rope import near, randn
from tests.test_rope_turns import exact

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


@pytest.mark.parametrize("base", [1e4, 1e6])
def test_far_positions_against_exact_angles(base):
    """Positions up to the ends of 32 bits, their angles reduced to a turn in 60 digits:
    the same tolerance as near ones, (|a| + |b|) 2^-22."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_best_gb300 import build
    build.build()
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -(2 ** 29) - 7, 98765432, 2 ** 24 + 1, -3]
    with localcontext() as ctx:
        ctx.prec = 60
        turns = [t / 2 ** 64 for t in exact(128, base)]
        angle = 2 * math.pi * np.array([[float(p * t % 1) for t in turns] for p in map(Decimal, pos)])
    x = randn((len(pos), 3, 128), "f32", 8)
    out = torch.empty_like(x)
    binding.rope_apply(binding.rope_cfg(len(pos), 3, 0, 128, io="f32"),
                       binding.rope_table(128, base=base),
                       torch.tensor(pos, dtype=torch.int32, device="cuda"), x, None, out, None)
    y, got = x.double().cpu().numpy(), out.double().cpu().numpy()
    a, b, t = y[..., :64], y[..., 64:], angle[:, None]
    want = np.concatenate([a * np.cos(t) - b * np.sin(t), a * np.sin(t) + b * np.cos(t)], 2)
    tol = (np.abs(a) + np.abs(b)) * 2.0 ** -22
    assert (np.abs(got - want) <= np.concatenate([tol, tol], 2) + 1e-38).all()
