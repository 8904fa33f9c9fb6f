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


# --------------------------------------------- attention: a few keys against very many

def long_request(L, T, sink, tail, first, io="bf16", kv="e4m3", Hq=4, D=128, page=256, seed=0):
    """One request whose first key has a score of log(L) + sink over the others'
    (equal ones, or normal ones of standard deviation 2 nats), and a first value of
    zeros, of one large element, or like the others; page table in order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = L + T
    cols = -(-n // page)
    cfg = binding.paged_cfg(B=1, T=T, Hq=Hq, Hkv=1, D=D, page=page, n_pages=cols, max_pages=cols,
                            io=io, kv=kv)
    rows = cols * page
    k = torch.zeros(rows, D, device="cuda")
    a = float(torch.tensor(2.0 * D ** 0.5).bfloat16())     # q = a on the first element: 2 nats a unit
    if tail == "normal":
        k[:, 0] = torch.randn(rows, generator=g, device="cuda").to(torch.float8_e4m3fn).float()
    k[0, 0] = float(torch.tensor((np.log(L) + sink) / 2).to(torch.float8_e4m3fn))
    v = torch.randn(rows, D, generator=g, device="cuda")
    v[0] *= {"zeros": 0, "one": 0, "like": 1}[first]
    if first == "one":
        v[0, 3] = 2000.0
    c = dict(cfg=cfg)
    if kv == "e4m3":
        scale = torch.where(v.abs().amax(-1) == 0, 1.0, v.abs().amax(-1) / 448)
        vc = (v / scale[:, None]).to(torch.float8_e4m3fn)
        pools, scales = [k.to(torch.float8_e4m3fn), vc], [torch.ones(rows, device="cuda"), scale]
        c["k"], c["v"] = k.double(), vc.double() * scale.double()[:, None]
        scales = [s.view(cols, 1, page).contiguous() for s in scales]
    else:
        pools, scales = [x.to(chain.DT[io]) for x in (k, v)], [None, None]
        c["k"], c["v"] = (p.double() for p in pools)
    q = torch.zeros(1, T, Hq, D, device="cuda")
    q[..., 0] = a
    c["q"] = q.to(chain.DT[io])
    c["kv"] = binding.PagedKV(cfg, *(p.view(cols, 1, page, D).contiguous() for p in pools),
                              torch.arange(cols, dtype=torch.int32, device="cuda").view(1, cols),
                              torch.full((1,), L, dtype=torch.int32, device="cuda"), *scales)
    c["L"] = L
    return c


def attend_and_bound(c, sums):
    """The library's output, the 64-bit one, and the bound of their difference:
    the terms of tests/test_gpu_paged.py, but for `sums` roundings of 2^-23 on the
    way of a weight or product through the fp32 sums."""
    cfg = c["cfg"]
    o = torch.full_like(c["q"], 7.0)
    ws = binding.alloc_paged_workspace(cfg)
    binding.attn_decode_paged(cfg, c["kv"], c["q"], o, ws)
    assert binding.spec_status_read(ws) == 0
    want, A = torch.zeros_like(o, dtype=torch.float64), torch.zeros_like(o, dtype=torch.float64)
    z = 0.0
    for i in range(cfg.T):
        n = c["L"] + i + 1
        k, v, q = c["k"][:n], c["v"][:n], c["q"][0, i].double()
        w = torch.softmax(q @ k.T / cfg.D ** 0.5, -1)
        want[0, i], A[0, i] = w @ v, w @ v.abs()
        z = max(z, float((q.abs() @ k.abs().T).max()) / cfg.D ** 0.5)
    d = (32 * 2.0 ** -23 + 2 * 2.0 ** -21) * z + 2.0 ** -20
    q8, bf = cfg.kv_dtype == binding.SPEC_KV_E4M3, cfg.io_dtype == binding.SPEC_IO_BF16
    cw = (2.0 ** -11 if q8 else 2.0 ** -16) if bf else 2.0 ** -20
    tol = (2.0 ** -8 if bf else 2.0 ** -24) * want.abs() + (cw + 2 * d + sums * 2.0 ** -23) * A + 1e-37
    return o.double(), want, tol


@pytest.mark.parametrize("io,kv", [("bf16", "e4m3"), ("f32", "e4m3"), ("bf16", "io")])
@pytest.mark.parametrize("L,T", [(8192, 1), (8191, 4), (32768, 1), (131071, 1), (131070, 5)])
@pytest.mark.parametrize("sink,tail,first", [(0.0, "equal", "zeros"), (5.0, "equal", "zeros"),
                                             (0.0, "equal", "one"), (0.0, "equal", "like"),
                                             (2.0, "normal", "zeros"), (2.0, "normal", "one")])
def test_one_key_against_all_others(L, T, sink, tail, first, io, kv):
    """Weights far below the largest one count by their sum.  (A weight goes into
    a sum with each 16 keys of its warp, one key warp of seven or more having at
    most every 8th part of a CTA's, and is joined over at most 200 parts.)"""
    got, want, tol = attend_and_bound(long_request(L, T, sink, tail, first, io, kv), L / 16 + 200)
    bad = (got - want).abs() > tol
    assert not bad.any(), float(((got - want).abs() / tol).max())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("least", [0.0, 2.0 ** -120])
def test_values_of_zeros_by_their_scale(io, T, least):
    """A scale of 0 (or next to it) stands for a row of zeros: it counts in the
    softmax's sum, before and behind values of ordinary size, and alone."""
    lens = [700, 700, 700, 9000, 60]
    x = Case(lens, T=T, Hq=8, Hkv=2, D=128, page=32, io=io, kv="e4m3", seed=41)
    for b, zero in enumerate((slice(0, 690), slice(10, 700 + T), slice(0, 700 + T, 2), slice(0, 8000),
                              slice(0, 60 + T))):
        x.scale["v"][b, zero] = least
    x.upload()
    o = x.attend()
    x.check(o)
    assert (o[4] == 0).all() or least > 0
    assert x.status() == 0


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -60, 2.0 ** 60, 2.0 ** 100])
def test_values_all_very_small_or_very_large(io, T, scale):
    x = Case([300, 5000], T=T, Hq=8, Hkv=2, D=64, page=16, io=io, kv="e4m3", seed=42)
    x.scale["v"] = (x.scale["v"] / x.scale["v"].max() * np.float32(scale)).astype(np.float32)
    x.upload()
    x.check(x.attend())
    assert x.status() == 0


@pytest.mark.parametrize("kv", ["io", "e4m3"])
@pytest.mark.parametrize("T,D", [(1, 64), (1, 128), (4, 64), (4, 128)])
def test_nothing_systematic_is_lost_in_fp32(kv, T, D):
    """The part of the error that goes with the output itself: sum of error x output
    over sum of output squared.  Roundings to nearest have no such part.  What has:
    an accumulator cut off by 2^-23 at most once per chunk of products, and products
    of third parts left out, on average below 2^-23 of a product: together 2^-22 of
    the output, and as much of each score, which moves weights by 2^-22 times the
    largest score."""
    B, L, Hkv, G, page = 6, 9000, 8, 4, 64
    g = torch.Generator(device="cuda").manual_seed(D + T)
    cols = -(-(L + T) // page)
    cfg = binding.paged_cfg(B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, n_pages=B * cols,
                            max_pages=cols, io="f32", kv=kv)
    pools = [torch.randn(B * cols, Hkv, page, D, generator=g, device="cuda") for _ in range(2)]
    scales = [None, None]
    if kv == "e4m3":
        scales = [p.abs().amax(-1) / 448 for p in pools]
        pools = [(p / s[..., None]).to(torch.float8_e4m3fn) for p, s in zip(pools, scales)]
    cache = binding.PagedKV(cfg, *pools, torch.arange(B * cols, dtype=torch.int32, device="cuda").view(B, cols),
                            torch.full((B,), L, dtype=torch.int32, device="cuda"), *scales)
    q = 2 * torch.randn(B, T, Hkv * G, D, generator=g, device="cuda")
    o = torch.empty_like(q)
    binding.attn_decode_paged(cfg, cache, q, o, binding.alloc_paged_workspace(cfg))
    along, square, z = 0.0, 0.0, 0.0
    for b in range(B):
        for h in range(Hkv):
            k, v = (p[b * cols:(b + 1) * cols, h].double() * (1 if s is None else
                    s[b * cols:(b + 1) * cols, h].double()[..., None]) for p, s in zip(pools, scales))
            k, v = k.reshape(-1, D), v.reshape(-1, D)
            for i in range(T):
                s = q[b, i, h * G:(h + 1) * G].double() @ k[:L + i + 1].T / D ** 0.5
                want = torch.softmax(s, -1) @ v[:L + i + 1]
                along += float(((o[b, i, h * G:(h + 1) * G].double() - want) * want).sum())
                square += float((want * want).sum())
                z = max(z, float(s.abs().max()))
    assert abs(along / square) <= (1 + z) * 2.0 ** -22, (along / square, z)


# ------------------------------------------------------------ slots without a request

@pytest.mark.parametrize("V", [997, 40000])
@pytest.mark.parametrize("N", [0, 3])
def test_verification_leaves_slots_without_a_request_out(N, V):
    x = chain.make(6, N, V, seed=30)
    x["n"] = np.array([N, -1, 0, -1, N, -1], np.int32)
    x["logits"][1::2] = np.nan
    kv = torch.arange(6, dtype=torch.int32, device="cuda")
    root = torch.full((6,), 77, dtype=torch.int32, device="cuda")
    ws = None
    for _ in range(2):                                     # counters are at zero again
        out, ws = chain.run(x, kv_len=kv, root=root, ws=ws)
    assert binding.spec_status_read(ws) == 0
    assert out.accept_len[1::2].tolist() == [0, 0, 0]
    assert (out.out_tok[1::2] == -1).all() and (out.target_prob[1::2] == 0).all()
    assert kv[1::2].tolist() == [1, 3, 5] and root[1::2].tolist() == [77] * 3
    live = dict(x, logits=x["logits"][::2], q=x["q"][::2], toks=x["toks"][::2], u=x["u"][::2],
                e=x["e"][::2], n=x["n"][::2])
    got = binding.DraftBuffers(binding.draft_cfg(B=3, N=N, V=V))
    for name in ("accept_len", "out_tok", "target_prob"):
        getattr(got, name).copy_(getattr(out, name)[::2])
    chain.check(live, got)
    assert kv[::2].tolist() == [2 * i + 2 * int(a) for i, a in enumerate(got.accept_len)]


@pytest.mark.parametrize("captured", [False, True])
def test_steps_with_slots_without_a_request(captured):
    """A request joins a batch whose other slots are empty and own no page; whole
    steps run eagerly or as one replayed graph."""
    from speculative_decoding_tree_best_gb300 import step
    B, N, V, Hq, Hkv, D, layers = 4, 2, 3001, 8, 2, 64, 2
    pc = binding.paged_cfg(B=B, T=N + 1, Hq=Hq, Hkv=Hkv, D=D, page=16, n_pages=8, max_pages=4, kv="e4m3")
    st = step.ChainStep(pc, binding.draft_cfg(B=B, N=N, V=V), layers)
    st.n_draft.fill_(-1)
    g = torch.Generator(device="cuda").manual_seed(3)
    f = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    rows = [[f(B, N + 1, h, D) for h in (Hq, Hkv, Hkv)] for _ in range(layers)]
    x = chain.make(B, N, V, seed=31)
    logits = torch.from_numpy(x["logits"]).bfloat16().cuda()
    d = [torch.from_numpy(x[c]).cuda() for c in ("toks", "q", "u", "e")]

    def run():
        o = [st.attend(i, *r) for i, r in enumerate(rows)]
        st.verify(logits, *d)
        return o
    run()
    assert st.kv_len.tolist() == [0] * B and st.status() == 0
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = run()
        go = graph.replay
    else:
        go = run
    at = 0
    for s in range(5):
        if s == 2:                                         # slot 1 gets a request and two pages
            st.page_table[1, :2] = torch.tensor([5, 2], dtype=torch.int32)
            st.n_draft[1] = N
        before = [c.k_pages.view(torch.uint8).clone() for c in st.caches]
        r = go()
        o = r if r is not None else o
        torch.cuda.synchronize()
        assert st.status() == 0
        lens = st.out.accept_len.tolist()
        at += lens[1]
        assert [lens[i] for i in (0, 2, 3)] == [0, 0, 0] and (lens[1] > 0) == (s >= 2)
        assert st.kv_len.tolist() == [0, at, 0, 0]
        for i in range(layers):
            assert (o[i][[0, 2, 3]] == 0).all() and bool((o[i][1] != 0).any()) == (s >= 2)
            changed = (st.caches[i].k_pages.view(torch.uint8) != before[i]).flatten(1).any(1)
            assert set(changed.nonzero().flatten().tolist()) <= ({5, 2} if s >= 2 else set())


@pytest.mark.parametrize("T", [1, 4])
def test_outputs_that_round_to_infinity_are_reported(T):
    """448 x 7.59e35 is finite in fp32 and beyond bf16's largest number."""
    x = Case([40], T=T, Hq=4, Hkv=1, D=64, page=16, kv="e4m3", seed=50)
    x.vals["v"][:] = 448.0
    x.scale["v"][:] = np.float32(7.59e35)
    x.upload()
    assert torch.isinf(x.attend()).all()
    assert x.status() == binding.SPEC_DEV_RANGE
    x.scale["v"][:] = np.float32(7.56e35)
    x.upload()
    assert torch.isfinite(x.attend()).all() and x.status() == 0


@pytest.mark.parametrize("io,kv", [("bf16", "e4m3"), ("f32", "e4m3"), ("f32", "io")])
@pytest.mark.parametrize("L", [20, 31, 8190])
@pytest.mark.parametrize("sink,first", [(5.0, "zeros"), (9.0, "one")])
def test_small_weights_beside_a_later_row_that_is_not_finite(io, kv, L, sink, first):
    """The fourth new row is NaN: the three before it keep their values, small
    weights and all, those from it on have none."""
    T = 6
    c = long_request(L, T, sink, "equal", first, io, kv)
    for pool in (c["kv"].k_pages, c["kv"].v_pages):
        raw = pool.view(torch.uint8) if kv == "e4m3" else pool
        raw[(L + 3) // 256, 0, (L + 3) % 256] = 0x7f if kv == "e4m3" else float("nan")
    cfg, o = c["cfg"], torch.full_like(c["q"], 7.0)
    ws = binding.alloc_paged_workspace(cfg)
    binding.attn_decode_paged(cfg, c["kv"], c["q"], o, ws)
    assert binding.spec_status_read(ws) == binding.SPEC_DEV_RANGE
    assert not torch.isfinite(o[0, 3:]).any()
    clean = long_request(L, T, sink, "equal", first, io, kv)
    got, want, tol = attend_and_bound(clean, L / 16 + 200)
    assert ((got - want).abs() <= tol).all()
    assert ((o.double() - want).abs() <= tol)[0, :3].all()
