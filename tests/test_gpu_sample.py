"""Filtered sampling against the definition in 64 bits.

What stays compares exactly where the nearest border of top_p is further than
2^-26 of the mass from top_p: weights are integers of 2^-43 of the largest (for
V <= 2^18) from an exponential within 2^-29, so a sum of n of them is within
2^-29 + n 2^-44 of itself.  Probabilities: the exponent is taken in two parts, 2^-22
of the exponential, a division and a few roundings of 2^-24: within 2^-20.  Tokens
compare exactly where no other score comes within 2^-16 of the best."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_tree_best_gb300 import binding
from tests import indep_serving as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NEAR = 2.0 ** -26


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_best_gb300 import build
    build.build()
    binding.load()


def run(x, io="f32", per=1, t=None, k=None, p=None, m=None, seed=0, inplace=False, stream=None):
    """x: logits [R][V], of which the I/O type's values count.  Returns the
    outputs as numpy arrays, the logits as they were read, and e."""
    x = torch.as_tensor(np.asarray(x, np.float32)).cuda().to(DT[io]).contiguous()
    R, V = x.shape
    cfg = binding.sample_cfg(R, V, per, io)
    e = torch.from_numpy(np.random.default_rng(seed).exponential(size=(R, V)).astype(np.float32)
                         + np.float32(1e-30)).cuda()
    ws = binding.alloc_sample_workspace(cfg)
    par = {n: None if v is None else torch.tensor(v, dtype=d, device="cuda")
           for n, v, d in (("temperature", t, torch.float32), ("top_k", k, torch.int32),
                           ("top_p", p, torch.float32), ("min_p", m, torch.float32))}
    read = x.clone()
    out = binding.SampleBuffers(cfg, prob=True, logits=x if inplace else True)
    binding.token_sample(cfg, x, e, out, ws, stream=stream, **par)
    if stream is not None:
        stream.synchronize()
    got = dict(tok=out.tok, tok_prob=out.tok_prob, prob=out.prob, logits=out.logits.float())
    return ({n: y.cpu().numpy() for n, y in got.items()}, read.float().cpu().numpy(),
            e.cpu().numpy(), binding.spec_status_read(ws))


def check(x, io="f32", per=1, t=None, k=None, p=None, m=None, status=0, **kw):
    got, x, e, bits = run(x, io, per, t, k, p, m, **kw)
    assert bits == status
    R, V = x.shape
    at = lambda v, r, d: d if v is None else float(np.float32(v[r // per]))  # noqa: E731
    unsure, kept = 0, []
    for r in range(R):
        T = at(t, r, 1.0)
        prob, n, margin = ref.sample(x[r], T, 0 if k is None else int(k[r // per]), at(p, r, 1.0),
                                     at(m, r, 0.0))
        if margin < NEAR:
            unsure += 1
            continue
        kept.append(n)
        stays = got["logits"][r] > -np.inf
        np.testing.assert_array_equal(got["logits"][r][stays], x[r][stays])
        # weights below fp32's range are 0 on both sides
        np.testing.assert_array_equal(stays & (prob > 1e-37), prob > 1e-37)
        assert int(stays.sum()) == n
        np.testing.assert_allclose(got["prob"][r], prob, rtol=2.0 ** -20, atol=1e-37)
        score = prob / e[r]
        best = int(score.argmax())
        rival = np.where(np.arange(V) == best, -1, score).max()
        if rival < score[best] * (1 - 2.0 ** -16):
            assert got["tok"][r] == best
        assert stays[got["tok"][r]]
        np.testing.assert_allclose(got["tok_prob"][r], prob[got["tok"][r]], rtol=2.0 ** -20)
    assert unsure <= max(1, R // 8)
    return kept


def rows(R, V, seed=0, spread=3.0):
    return spread * np.random.default_rng(seed).standard_normal((R, V))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("R,V", [(1, 1), (1, 2), (3, 7), (2, 1000), (5, 4099), (1, 151936),
                                 (24, 10007), (3, 32768), (200, 515), (2, 131071)])
@pytest.mark.parametrize("f", ["none", "k", "p", "m", "kp", "all"])
def test_filters(io, R, V, f):
    rng = np.random.default_rng(V)
    k = rng.integers(1, min(V, 300) + 1, R) if f in ("k", "kp", "all") else None
    p = rng.uniform(0.3, 0.999, R) if f in ("p", "kp", "all") else None
    m = rng.uniform(0.001, 0.2, R) if f in ("m", "all") else None
    t = rng.uniform(0.3, 1.7, R) if f != "none" else None
    check(rows(R, V, seed=R), io, t=t, k=k, p=p, m=m)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_large_vocabularies(io):
    V = (1 << 20) - 3
    check(rows(2, V, 1), io, t=[1.0, 0.8], p=[0.9, 0.99], k=[0, 5000])
    check(rows(1, 1 << 20, 2), io, p=[0.5])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("k", [1, 2, 63, 500, 4000, 99999, 100001])
def test_top_k_sizes(io, k):
    x = rows(2, 100001, 3)
    assert check(x, io, k=[k, k]) == [min(k, 100001)] * 2


def test_rows_share_parameters():
    check(rows(10, 777, 4), "bf16", per=4, t=[0.5, 1.0, 1.5], k=[5, 0, 20], p=[1.0, 0.8, 0.9],
          m=[0.0, 0.05, 0.0])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_ties_go_to_the_lowest_index(io):
    V = 20001
    flat = np.zeros((3, V))
    flat[1, 5000:] = -0.0
    flat[2, ::2] = 1.0
    got, x, _, _ = run(flat, io, k=[7, 9, 11])
    for r, (n, step) in enumerate(((7, 1), (9, 1), (11, 2))):
        np.testing.assert_array_equal(np.nonzero(got["logits"][r] > -np.inf)[0],
                                      np.arange(n) * step)
    # equal masses: half of 20000 ones is 10000 of them, and a little more is one more
    # (2^-12 of 20000 is 4.9: a border between two, not on one)
    got, _, _, _ = run(np.zeros((1, 20000)), io, p=[0.5 - 2.0 ** -12])
    assert (got["logits"][0] > -np.inf).sum() == math.ceil((0.5 - 2.0 ** -12) * 20000)
    assert (got["logits"][0][:9996] == 0).all()
    # exactly half: what is before token 10000 is not less than half
    got, _, _, _ = run(np.zeros((1, 20000)), io, p=[0.5])
    assert (got["logits"][0] > -np.inf).sum() == 10000


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_ties_that_both_borders_meet(io):
    """top_k leaves 2000 of 3000 equal logits, and top_p's border is among them or at
    their end: those that top_k removed stay removed.  (In the last row one weighs
    e^2 times the others: the sum is 1 + 1999 e^-2 = 271.5, 0.6 of it 162.9, and before
    the token j there is 1 + (j - 1) e^-2, which is less up to j = 1197: 1198 tokens.
    0.75 of 2000 equal ones is on a border, and not compared.)"""
    x = np.full((4, 60000), -5.0)
    x[:, 7::20] = 2.0
    x[2:, 11] = 4.0
    p = [0.9999, 0.75, 0.9999, 0.6]
    assert check(x, io, k=[2000] * 4, p=p) == [2000, 2000, 1198]


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_masks_and_extremes(io):
    V = 5003
    low = float(torch.finfo(DT[io]).min)
    x = rows(8, V, 5)
    x[0, 10:] = -np.inf                                   # ten left
    x[1, :] = -np.inf
    x[1, 4711] = -1e30                                    # one left, far down
    x[2, 1:] = low                                        # masks of the lowest value
    x[3, :] = low                                         # nothing but masks
    x[4] = x[4] + 1e6                                     # far from zero
    x[5] = x[5] * 1e-6                                    # flat
    x[6] = x[6] * 1e30                                    # steep
    x[7, 100:] = -np.inf
    check(x, io, t=[1.0] * 8, k=[20, 20, 5, 9, 30, 0, 3, 100], p=[0.9, 0.5, 0.9, 0.7, 1.0, 0.37, 1.0, 1.0])
    check(x, io, m=[0.01, 0.5, 0.1, 1.0, 0.3, 0.5, 0.5, 2.0])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("R", [1, 30])
def test_sorted_rows(io, R):
    """All of a row's largest logits in one part of it: the bounds that each part
    gives are far below, and the short list overflows."""
    V = 60013
    x = np.sort(rows(R, V, 12), 1)
    x[::2] = x[::2, ::-1]
    for k in (40, 300, 900):
        check(x, io, k=[k] * R, p=[0.97] * R)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_borders_below_the_bins(io):
    """A few logits far above the others: the bins, which go down from the largest,
    do not reach the border."""
    V = 9001
    x = rows(6, V, 13) - 2000.0
    x[:, 5000:5003] = [[3.0, 1.0, 2.0]]
    check(x, io, k=[3000, 2, 1500, 4, 3, 8999], t=[1.0, 1.0, 900.0, 1e4, 2.0, 50.0])
    check(x, io, p=[0.9, 0.99, 0.8, 0.5, 0.3, 0.97], t=[900.0, 1.0, 2000.0, 1e4, 500.0, 3000.0])
    x = -(10.0 ** np.random.default_rng(14).uniform(33, 37, (3, V)))      # nothing near 0
    check(x, io, k=[2000, 7, 100], t=[1e33, 1e35, 1e36])
    check(x, io, p=[0.6, 0.9, 0.8], t=[1e35, 1e36, 1e37])


def test_small_magnitudes():
    """Most logits within 2^-12 of 0, many of them 0: one bin holds them."""
    x = rows(4, 20011, 15, 1e-5)
    x[1, ::3] = 0.0
    x[2, ::2] *= 1e5
    x[3, 100:] = -0.0
    for io in ("bf16", "f32"):
        check(x, io, p=[0.5, 0.7, 0.9, 0.3], t=[1e-5, 0.7, 1.0, 2.0])
        check(x, io, k=[5000, 12000, 1500, 60], p=[0.5, 0.7, 0.9, 0.35], t=[1e-5, 2e-5, 1.0, 2.0])


def test_temperatures_at_the_ends():
    x = rows(7, 999, 6)
    x[1, 500] = x[1, 300] = x[1].max() + 1                # greedy with a tie
    t = [0.0, 0.0, 1e-30, 1e-45, 3e38, float("inf"), 0.05]
    got, x32, _, bits = run(x, "f32", t=t, k=[0, 0, 0, 0, 0, 9, 0])
    assert bits == 0
    for r in (0, 1):
        assert got["tok"][r] == x32[r].argmax() and got["tok_prob"][r] == 1.0
        assert (got["prob"][r] > 0).sum() == 1
    for r in (2, 3):
        assert got["tok"][r] == x32[r].argmax() and got["tok_prob"][r] == 1.0
    np.testing.assert_allclose(got["prob"][4], 1 / 999, rtol=2.0 ** -20)
    assert (got["prob"][5] > 0).sum() == 9
    np.testing.assert_allclose(got["prob"][5].max(), 1 / 9, rtol=2.0 ** -20)


def test_parameters_at_the_ends():
    x = rows(8, 300, 7)
    nan = float("nan")
    got, _, _, bits = run(x, "f32", k=[0, -5, 300, 2 ** 31 - 1, 0, 0, 0, 0],
                          p=[1.0, 2.0, 1.5, 1.0, 0.0, -1.0, 1e-30, 1.0 - 2.0 ** -24],
                          m=[0.0, -1.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0])
    assert bits == 0
    n = (got["logits"] > -np.inf).sum(1)
    assert n[:4].tolist() == [300] * 4 and n[4:7].tolist() == [1, 1, 1]
    got, x32, _, bits = run(x[:4], "f32", t=[nan, -1.0, 1.0, 1.0], p=[1.0, 1.0, nan, 1.0],
                            m=[0.0, 0.0, 0.0, nan])
    assert bits == binding.SPEC_DEV_BADREQ
    assert (got["logits"] > -np.inf).sum(1).tolist() == [1, 1, 300, 300]


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows_that_are_not_finite(io):
    x = rows(5, 1203, 8)
    x[0, 700] = np.nan
    x[1, 3] = np.inf
    x[2, :] = -np.inf
    x[3, 1202] = np.nan
    got, x32, _, bits = run(x, io, k=[5] * 5, p=[0.9] * 5)
    assert bits == binding.SPEC_DEV_BADLOGIT
    assert got["tok"][:4].tolist() == [0] * 4 and (got["tok_prob"][:4] == 0).all()
    assert (got["prob"][:4] == 0).all()
    np.testing.assert_array_equal(got["logits"][:4], x32[:4])
    assert (got["prob"][4] > 0).sum() <= 5 and abs(got["prob"][4].sum() - 1) < 1e-5


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_in_place_and_one_output_at_a_time(io):
    R, V = 9, 3001
    x = rows(R, V, 9)
    kw = dict(t=[0.8] * R, k=[40] * R, p=[0.95] * R, m=[0.01] * R)
    a, read, e, _ = run(x, io, **kw)
    b, _, _, _ = run(x, io, inplace=True, **kw)
    for n in a:
        np.testing.assert_array_equal(a[n], b[n])
    cfg = binding.sample_cfg(R, V, io=io)
    ws = binding.alloc_sample_workspace(cfg)
    d = torch.from_numpy(read).cuda().to(DT[io])
    e = torch.from_numpy(e).cuda()
    par = dict(temperature=torch.full((R,), 0.8, device="cuda"),
               top_k=torch.full((R,), 40, dtype=torch.int32, device="cuda"),
               top_p=torch.full((R,), 0.95, device="cuda"),
               min_p=torch.full((R,), 0.01, device="cuda"))
    for draw, prob, logits in ((True, False, False), (False, True, False), (False, False, True)):
        out = binding.SampleBuffers(cfg, draw=draw, prob=prob, logits=logits)
        binding.token_sample(cfg, d, e if draw else None, out, ws, **par)
        for n, y in (("tok", out.tok), ("tok_prob", out.tok_prob), ("prob", out.prob),
                     ("logits", out.logits)):
            if y is not None:
                np.testing.assert_array_equal(y.float().cpu().numpy(), a[n].astype(np.float32))
    with pytest.raises(ValueError):
        binding.token_sample(cfg, d, None, binding.SampleBuffers(cfg), ws)


def test_law_of_the_draw():
    """Half a million draws follow the filtered probabilities (chi-square, 12
    tokens stay: 11 degrees of freedom, 60 is beyond 1e-8)."""
    V, n = 50, 1 << 19
    x = np.repeat(rows(1, V, 10, 1.0), n // 64, 0)
    prob, kept, _ = ref.sample(np.float32(x[0]), 0.9, 12, 1.0, 0.0)
    count = np.zeros(V)
    for seed in range(64):
        got, _, _, _ = run(x, "f32", per=n // 64, t=[0.9], k=[12], seed=seed)
        count += np.bincount(got["tok"], minlength=V)
    assert (count[prob == 0] == 0).all()
    want = prob[prob > 0] * n
    assert ((count[prob > 0] - want) ** 2 / want).sum() < 60


def test_results_do_not_depend_on_the_batch():
    """A row's outputs are the same alone and among others (another split)."""
    x = rows(40, 30011, 11)
    a, _, _, _ = run(x, "bf16", p=[0.9] * 40, k=[0, 50] * 20)
    for r in (0, 1, 39):
        b, _, _, _ = run(x[r:r + 1], "bf16", p=[0.9], k=[[0, 50][r % 2]])
        for n in ("prob", "logits"):
            np.testing.assert_array_equal(a[n][r], b[n][0])


def test_captured_on_another_stream():
    R, V = 6, 40000
    cfg = binding.sample_cfg(R, V)
    ws = binding.alloc_sample_workspace(cfg)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (3 * torch.randn((R, V), generator=g, device="cuda")).bfloat16()
    e = torch.rand((R, V), generator=g, device="cuda") + 1e-6
    p = torch.full((R,), 0.9, device="cuda")
    out, now = binding.SampleBuffers(cfg, prob=True), binding.SampleBuffers(cfg, prob=True)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            binding.token_sample(cfg, x, e, out, ws, top_p=p)
    for i in range(3):
        x.copy_((3 * torch.randn((R, V), generator=g, device="cuda")).bfloat16())
        p.fill_(0.3 + 0.2 * i)
        graph.replay()
        binding.token_sample(cfg, x, e, now, ws, top_p=p)
        assert torch.equal(out.tok, now.tok) and torch.equal(out.prob, now.prob)


def test_two_streams_at_once():
    """Calls of two streams, with outputs and workspaces of their own, beside one
    another: the same results as one after the other."""
    g = torch.Generator(device="cuda").manual_seed(3)
    jobs = []
    for R, V, io in ((40, 30000, "bf16"), (7, 60000, "f32")):
        cfg = binding.sample_cfg(R, V, io=io)
        x = (3 * torch.randn((R, V), generator=g, device="cuda")).to(DT[io])
        e = torch.rand((R, V), generator=g, device="cuda") + 1e-6
        p = 0.3 + 0.69 * torch.rand((R,), generator=g, device="cuda")
        k = torch.randint(0, 2000, (R,), generator=g, device="cuda", dtype=torch.int32)
        for kw in (dict(top_p=p), dict(top_k=k), dict(top_k=k, top_p=p)):
            want = binding.SampleBuffers(cfg, prob=True)
            binding.token_sample(cfg, x, e, want, binding.alloc_sample_workspace(cfg), **kw)
            jobs.append((cfg, x, e, kw, want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for i, (cfg, x, e, kw, want) in enumerate(jobs):
            out, ws = binding.SampleBuffers(cfg, prob=True), binding.alloc_sample_workspace(cfg)
            got.append((out, ws))
        torch.cuda.synchronize()
        for i, (cfg, x, e, kw, want) in enumerate(jobs):
            binding.token_sample(cfg, x, e, *got[i], stream=streams[i % 2], **kw)
        torch.cuda.synchronize()
        for (out, _), (_, _, _, _, want) in zip(got, jobs):
            assert torch.equal(out.tok, want.tok) and torch.equal(out.prob, want.prob)


def test_cold_caches():
    """Calls whose instructions and inputs come from memory, so that the warps of the
    CTAs that share a row are far apart: the same borders each time."""
    R, V = 30, 60013
    x = torch.from_numpy(rows(R, V, 24).astype(np.float32)).cuda()
    p = np.random.default_rng(1).uniform(0.3, 0.999, R).astype(np.float32)
    want = [ref.sample(y, 1.0, 0, float(q), 0.0)[1:] for y, q in zip(x.cpu().numpy(), p)]
    sure = torch.tensor([m >= NEAR for _, m in want])
    n = torch.tensor([n for n, _ in want])
    assert int(sure.sum()) >= R - 2
    cfg = binding.sample_cfg(R, V, io="f32")
    ws, e, top_p = binding.alloc_sample_workspace(cfg), torch.ones_like(x), torch.from_numpy(p).cuda()
    out = binding.SampleBuffers(cfg, logits=True)
    flush = torch.empty(400 << 20, dtype=torch.uint8, device="cuda")         # more than L2
    for i in range(200):
        flush.fill_(i)
        binding.token_sample(cfg, x, e, out, ws, top_p=top_p)
        got = (out.logits > -math.inf).sum(1).cpu()
        assert got[sure].tolist() == n[sure].tolist()
