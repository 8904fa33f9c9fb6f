"""Filtered sampling where the filters' passes hand borders on to one another, and
for rows and numbers at the ends of what the calls accept.  Tolerances are those of
test_gpu_sample.py."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_tree_best_gb300 import binding
from tests import indep_serving as ref
from tests.test_gpu_sample import DT, NEAR, check, rows

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


# how a border is found, with the I/O type, rows, vocabulary, spread, top_k and top_p
# (cluster sizes from 1 to 16 CTAs)
BORDERS = {
    "masses and a list": ("f32", 30, 60013, 3.0, 0, 1),
    "masses, 16 CTAs": ("f32", 1, 151936, 3.0, 0, 1),
    "masses, few CTAs": ("f32", 150, 20011, 3.0, 0, 1),
    "counts of values": ("bf16", 30, 60013, 3.0, 0, 1),
    "counts of values, many rows": ("bf16", 256, 60013, 3.0, 0, 1),
    "counts, ties by value": ("bf16", 30, 60013, 3.0, 3000, 0),
    "counts and a list": ("f32", 30, 60013, 3.0, 3000, 0),
    "both in the histogram": ("bf16", 9, 120011, 3.0, 5000, 1),
    "both in the histogram, fp32": ("f32", 9, 120011, 3.0, 5000, 1),
    "radix": ("f32", 6, 60013, 1e-5, 30000, 1),
    "radix after ties": ("bf16", 6, 60013, 1e-5, 30000, 1),
    "short list": ("bf16", 30, 60013, 3.0, 40, 1),
    "short list by the threads' maxima": ("f32", 30, 60013, 3.0, 900, 1),
    "short list, 16 CTAs": ("bf16", 1, 151936, 3.0, 200, 1),
}


def test_cold_caches_of_all_borders():
    """Each way to a border in turn with the others, L2 overwritten before each call,
    so that instructions and inputs come from memory: the same borders each time."""
    jobs = []
    for i, (name, (io, R, V, spread, k, p)) in enumerate(BORDERS.items()):
        x = torch.from_numpy(rows(R, V, 40 + i, spread).astype(np.float32)).cuda().to(DT[io])
        p = np.random.default_rng(i).uniform(0.3, 0.999, R).astype(np.float32) if p else None
        some = range(0, R, max(1, R // 30))
        want = [ref.sample(x[r].float().cpu().numpy(), 1.0, k, 1.0 if p is None else float(p[r]))[1:]
                for r in some]
        sure = [m >= NEAR for _, m in want]
        assert sum(sure) >= len(want) - 2
        cfg = binding.sample_cfg(R, V, io=io)
        kw = dict(top_k=torch.full((R,), k, dtype=torch.int32, device="cuda") if k else None,
                  top_p=None if p is None else torch.from_numpy(p).cuda())
        jobs.append((name, cfg, x, binding.alloc_sample_workspace(cfg), kw,
                     binding.SampleBuffers(cfg, draw=False, logits=True),
                     [(r, n) for r, (n, _), ok in zip(some, want, sure) if ok]))
    flush = torch.empty(400 << 20, dtype=torch.uint8, device="cuda")         # more than L2
    for i in range(50):
        for name, cfg, x, ws, kw, out, want in jobs:
            flush.fill_(i % 100)
            binding.token_sample(cfg, x, None, out, ws, **kw)
            n = (out.logits > -np.inf).sum(1).cpu()
            assert [int(n[r]) for r, _ in want] == [w for _, w in want], name


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1000, 60013])
@pytest.mark.parametrize("k", [0, 100])
def test_races_between_small_weights(io, V, k):
    """Tokens whose weights and random numbers are both far below 1: scores 2^20, 2^10
    and 1, while weight times random number is below fp32's range.  (bf16 rounds the
    exponents 60 and 100 by at most 2^-9: the scores stay 2^9 apart.)"""
    x = torch.full((4, V), -150.0)
    e = torch.ones((4, V))
    order = [(7, 300, 500), (500, 300, 7), (V - 1, 8, V - 9), (400, V - 2, 3)]
    for r, (top, low, best) in enumerate(order):
        x[r, top] = 0.0
        x[r, best], e[r, best] = -60 * math.log(2.0), 2.0 ** -80
        x[r, low], e[r, low] = -100 * math.log(2.0), 2.0 ** -110
    cfg = binding.sample_cfg(4, V, io=io)
    out, ws = binding.SampleBuffers(cfg), binding.alloc_sample_workspace(cfg)
    top_k = torch.full((4,), k, dtype=torch.int32, device="cuda")
    binding.token_sample(cfg, x.cuda().to(DT[io]), e.cuda(), out, ws, top_k=top_k)
    assert out.tok.tolist() == [best for _, _, best in order]
    # and at the ends of the range that random numbers have: the largest score wins
    e = torch.full((4, V), 2.0 ** 126)
    e[0, 5], e[1, V // 2], e[2, V - 1] = 2.0 ** -126, 2.0 ** -126, float(2.0 ** 125)
    e[3, :] = float("inf")
    e[3, 4] = 2.0 ** 127
    x = torch.zeros((4, V))
    binding.token_sample(cfg, x.cuda().to(DT[io]), e.cuda(), out, ws, top_k=None)
    assert out.tok.tolist() == [5, V // 2, V - 1, 4]


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_logits_far_below_the_largest_in_magnitude(io):
    """Differences from the largest that round even between bf16 values (22 and
    numbers of 2^-8 to 2^-20), at temperatures where the exponent is up to 120: a
    rounding of the difference alone would be 2^-25 of that."""
    rng = np.random.default_rng(50)
    V = 5003
    x = np.exp2(rng.uniform(-20, -8, (5, V))) * rng.choice([-1, 1], (5, V))
    x[:, 77] = [22.0, 5.5, 21.75, 30.0, 17.0]
    t = [0.3, 0.1, 0.27, 0.5, 9.0]
    check(x, io, t=t)
    check(x, io, t=t, k=[0, 40, 3000, 0, 0], p=[0.9999, 1.0, 1.0, 1.0, 0.7])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_logits_as_far_apart_as_numbers_go(io):
    """The largest and the least logit further apart than fp32's largest number, at
    temperatures of their size: no probability is lost, negative or not a number."""
    rng = np.random.default_rng(51)
    V = 1003
    x = rng.uniform(-3.3e38, 3.3e38, (6, V))
    x[:, 5], x[:, 700] = 3.38e38, -3.38e38
    t = [1e37, 5e36, 3.3e38, float("inf"), 1e38, 2e37]
    check(x, io, t=t)
    check(x, io, t=t, k=[0, 300, 0, 900, 1000, 2], p=[0.9, 0.97, 0.6, 0.371, 1.0, 0.5])
