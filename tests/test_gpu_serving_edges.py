"""The serving operators at the edges of what their calls accept: one workspace
for many shapes in turn, and inputs far from the ordinary ones."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_best_gb300 import binding
from tests import test_gpu_chain as chain
from tests.test_gpu_paged import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_best_gb300 import build
    build.build()
    binding.load()


# ------------------------------------------------- one workspace for many shapes

def one_workspace(needs):
    return torch.zeros(max(needs), dtype=torch.uint8, device="cuda")


def test_attention_of_many_shapes_on_one_workspace():
    """Shapes whose parts, row groups and tickets differ, in turn and back again:
    each call finds the counters at zero wherever the one before had its data."""
    rng = np.random.default_rng(1)
    shapes = [dict(lens=[9000], Hq=32, Hkv=8, D=128, page=64),
              dict(lens=rng.integers(3000, 6000, 24).tolist(), Hq=32, Hkv=8, D=128, page=64),
              dict(lens=[4000, 3100], T=33, Hq=8, Hkv=2, D=64, page=16),
              dict(lens=rng.integers(0, 900, 40).tolist(), T=2, Hq=8, Hkv=8, D=64, page=32)]
    xs = [Case(io="bf16", kv="e4m3", seed=i, **s) for i, s in enumerate(shapes)]
    want = [x.attend() for x in xs]                        # each on its own workspace
    for x, w in zip(xs, want):
        x.check(w)
    ws = one_workspace([binding.spec_paged_workspace_bytes(x.cfg) for x in xs])
    for i in (0, 1, 2, 3, 1, 0, 3, 2, 0, 1):
        xs[i].ws = ws
        assert torch.equal(xs[i].attend(), want[i]), i
    assert binding.spec_status_read(ws) == 0


def test_verifications_of_many_shapes_on_one_workspace():
    """Also beyond the number of requests whose races are cut into slices."""
    xs = [chain.make(B, N, V, seed=B + N) for B, N, V in
          ((24, 8, 30000), (24, 4, 30000), (8, 8, 30000), (1, 2, 100003), (700, 1, 50))]
    cfgs = [binding.draft_cfg(B=x["logits"].shape[0], N=x["toks"].shape[1], V=x["logits"].shape[2],
                              temperature=x["t"]) for x in xs]
    want = [chain.run(x)[0] for x in xs]
    for x, w in zip(xs, want):
        chain.check(x, w)
    ws = one_workspace([binding.spec_draft_workspace_bytes(c) for c in cfgs])
    for i in (0, 1, 0, 2, 0, 3, 4, 2, 1, 3, 0):
        out = binding.DraftBuffers(cfgs[i])
        for t in (out.accept_len, out.out_tok):
            t.fill_(-7)
        chain.run(xs[i], ws=ws, out=out)
        for name in ("accept_len", "out_tok", "target_prob"):
            assert torch.equal(getattr(out, name), getattr(want[i], name)), (i, name)
    assert binding.spec_status_read(ws) == 0


def test_attention_and_verification_share_a_workspace():
    x = Case([9000, 70], T=3, Hq=16, Hkv=4, D=128, page=64, kv="e4m3", seed=5)
    y = chain.make(6, 2, 40000, seed=6)
    want_o, want_t = x.attend(), chain.run(y)[0]
    cfg = binding.draft_cfg(B=6, N=2, V=40000)
    ws = one_workspace([binding.spec_paged_workspace_bytes(x.cfg),
                        binding.spec_draft_workspace_bytes(cfg)])
    x.ws = ws
    for _ in range(3):
        assert torch.equal(x.attend(), want_o)
        out = binding.DraftBuffers(cfg)
        out.out_tok.fill_(-7)
        chain.run(y, ws=ws, out=out)
        assert torch.equal(out.out_tok, want_t.out_tok)


# ---------------------------------------------------------- verification: row masses

@pytest.mark.parametrize("io,V", [("bf16", 4099), ("f32", 4099), ("bf16", 32768), ("f32", 1000)])
@pytest.mark.parametrize("t,at", [(1e-6, 15.0), (3e-9, 15.0), (1e-10, 1000.0), (1e-30, 20.0), (1e-44, 20.0)])
def test_small_temperatures(io, V, t, at):
    """Logits over the temperature far beyond 2^31: the largest logit, or the
    largest few that are equal, have all of the mass."""
    x = chain.make(24, 3, V, io, seed=V, spread=0.05 * at)
    x["t"] = float(np.float32(t))
    x["toks"][::2, :2] = x["logits"][::2, :2].argmax(-1)
    out, ws = chain.run(x)
    kepts = chain.check(x, out)
    assert binding.spec_status_read(ws) == 0
    assert max(kepts) >= 2


def test_logits_that_differ_by_a_small_temperature():
    """fp32 logits a few roundings apart at a temperature of that size."""
    x = chain.make(12, 2, 5000, "f32", seed=2)
    x["logits"] = (np.float32(15) + np.float32(2.0 ** -20) * np.random.default_rng(3).integers(
        -20, 20, x["logits"].shape)).astype(np.float32)
    x["t"] = float(np.float32(1e-6))
    out, ws = chain.run(x)
    chain.check(x, out)
    assert binding.spec_status_read(ws) == 0


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("t", [0.5, 1.0])
def test_masks_of_the_lowest_value(io, t):
    """All but a few tokens at the type's lowest value, in one row all of them."""
    lowest = np.float32(torch.finfo(chain.DT[io]).min)
    x = chain.make(8, 2, 5003, io, t=t, seed=4)
    x["logits"][:, :, 20:] = lowest
    x["q"][:, :, 20:] = 0
    x["q"] /= x["q"].sum(-1, keepdims=True)
    x["toks"] %= 20
    x["logits"][3] = lowest
    out, ws = chain.run(x)
    chain.check(x, out)
    assert binding.spec_status_read(ws) == 0


# ------------------------------------------------ verification: ends of the scores' range

@pytest.mark.parametrize("V", [4000, 4003])
@pytest.mark.parametrize("small", [2.0 ** -128, 2.0 ** -140, 2.0 ** -149])
def test_an_exponential_below_the_normal_range_beside_a_larger_score(V, small):
    """A token of little weight and a subnormal exponential, before and behind one
    whose score is larger, the same thread's or another's; and the other way round."""
    x = chain.make(8, 0, V, io="f32", seed=20, spread=0.1)
    x["e"][:] = 1.0
    pairs = [(8, 9), (9, 8), (8, 8 + 256), (264, 8), (100, 3000), (3000, 100), (16, 17), (17, 16)]
    for b, (i, j) in enumerate(pairs):                     # i has the small exponential
        x["e"][b, i] = small
        x["logits"][b, 0, i] = -14.0                       # weight about 2^-32
        x["e"][b, j] = small * (2.0 ** 20 if b < 6 else 2.0 ** 40)
        x["logits"][b, 0, j] = 0.5                         # 21 log2 units more
    out, ws = chain.run(x)
    chain.check(x, out)
    assert out.out_tok[:, 0].tolist() == [j for _, j in pairs[:6]] + [i for i, _ in pairs[6:]]


@pytest.mark.parametrize("V", [40, 43, 2600])
@pytest.mark.parametrize("N", [0, 2])
def test_exponentials_whose_reciprocal_vanishes(V, N):
    """All of them from 2^126 on: scores below the normal range, told apart."""
    x = chain.make(12, N, V, io="f32", seed=V + N, spread=4.0)
    x["e"] = (2.0 ** 126 * (1 + 0.99 * np.random.default_rng(V).random(x["e"].shape))).astype(np.float32)
    out, ws = chain.run(x)
    chain.check(x, out)
    assert binding.spec_status_read(ws) == 0


def test_drafts_of_point_masses_whose_reciprocals_vanish():
    """A refused draft is not drawn again there either."""
    x = chain.make(6, 1, 24, io="f32", seed=9, point=True, spread=4.0)
    x["toks"] = x["logits"][:, :1].argmax(-1).astype(np.int32)
    x["u"][:] = np.float32(1 - 2 ** -24)
    x["e"] = (2.0 ** 126 * (1 + 0.99 * np.random.default_rng(9).random(x["e"].shape))).astype(np.float32)
    out, _ = chain.run(x)
    assert chain.check(x, out) and (out.out_tok[:, 0].cpu().numpy() != x["toks"][:, 0]).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_large_temperatures(io):
    """Probabilities that are all but equal, up to the largest finite temperature."""
    for t in (1e6, 3.4028234663852886e38):
        x = chain.make(6, 2, 999, io, seed=21)
        x["t"] = float(np.float32(t))
        out, ws = chain.run(x)
        chain.check(x, out)
        assert binding.spec_status_read(ws) == 0
