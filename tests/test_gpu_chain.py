"""The drafted chain's verification against a plain 64-bit implementation, and
whole steps (append, attend, verify) as a serving loop makes them.

Tokens and lengths compare exactly where every decision of the chain is
further than MARGIN (relative) from its border: an fp32 probability is within
about 2^-24 times its exponent's size (at most 60) plus a few roundings, under
2^-17, of the 64-bit one.  A target probability compares at the same 2^-17."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_best_gb300 import binding, step
from tests import indep_chain as ref

pytestmark = pytest.mark.gpu

MARGIN = 2.0 ** -16
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_best_gb300 import build
    build.build()
    binding.load()


def make(B, N, V, io="bf16", t=1.0, seed=0, point=False, noise=0.7, spread=3.0):
    rng = np.random.default_rng(seed)
    z = (spread * rng.standard_normal((B, N + 1, V))).astype(np.float32)
    logits = ref.bf16(z) if io == "bf16" else z
    d = (z[:, :N] + noise * rng.standard_normal((B, N, V))) / t
    q = ref.softmax(d).astype(np.float32) if N else np.zeros((B, 0, V), np.float32)
    toks = (d + rng.gumbel(size=d.shape)).argmax(-1).astype(np.int32) if N else np.zeros((B, 0), np.int32)
    return dict(logits=logits, q=None if point else q, toks=toks,
                u=rng.random((B, N)).astype(np.float32),
                e=rng.exponential(size=(B, V)).astype(np.float32) + np.float32(1e-30), t=t, io=io,
                n=None)


def run(x, cfg=None, ws=None, kv_len=None, root=None, stream=None, out=None):
    B, N1, V = x["logits"].shape
    cfg = cfg or binding.draft_cfg(B=B, N=N1 - 1, V=V, io=x["io"], temperature=x["t"])
    out = out or binding.DraftBuffers(cfg)
    ws = binding.alloc_draft_workspace(cfg) if ws is None else ws
    d = {k: None if x[k] is None else torch.from_numpy(np.ascontiguousarray(x[k])).cuda()
         for k in ("logits", "q", "toks", "u", "e", "n")}
    binding.draft_verify_sampled(cfg, d["toks"], d["q"], d["logits"].to(DT[x["io"]]), d["u"], d["e"],
                                 out, ws, n_draft=d["n"], kv_len=kv_len, root_tok=root,
                                 stream=stream)
    return out, ws


def check(x, out):
    B, N1, V = x["logits"].shape
    lens, toks = out.accept_len.cpu().numpy(), out.out_tok.cpu().numpy()
    prob = out.target_prob.cpu().numpy()
    close, kepts = 0, []
    for b in range(B):
        n = N1 - 1 if x["n"] is None else int(x["n"][b])
        kept, tok, p, margin = ref.chain(x["logits"][b], None if x["q"] is None else x["q"][b],
                                         x["toks"][b, :n], x["u"][b], x["e"][b], x["t"])
        np.testing.assert_allclose(prob[b, :n], p, rtol=2.0 ** -17, atol=1e-37)
        assert (prob[b, n:] == 0).all()
        if margin < MARGIN:
            close += 1
            continue
        kepts.append(kept)
        assert lens[b] == kept + 1
        np.testing.assert_array_equal(toks[b], list(x["toks"][b, :kept]) + [tok] + [-1] * (N1 - 1 - kept))
    assert close <= max(1, B // 10)
    return kepts


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,V", [(1, 1, 1), (3, 1, 7), (2, 4, 1000), (5, 8, 4099), (1, 8, 151936),
                                   (24, 3, 10007), (2, 127, 513), (3, 2, 32768)])
def test_chain(io, B, N, V):
    x = make(B, N, V, io, seed=V)
    out, ws = run(x)
    check(x, out)
    assert binding.spec_status_read(ws) == 0


@pytest.mark.parametrize("t", [0.3, 1.7])
def test_temperatures_and_ragged_chains(t):
    x = make(16, 6, 5000, t=t, seed=3)
    x["n"] = np.array([0, 1, 2, 3, 4, 5, 6, 6] * 2, np.int32)
    x["logits"][3, 5:] = np.nan                            # rows beyond n_draft are not read
    out, ws = run(x)
    kepts = check(x, out)
    assert binding.spec_status_read(ws) == 0 and max(kepts) >= 3


def test_point_mass_drafts():
    x = make(12, 4, 300, point=True, seed=4, spread=5.0)
    x["toks"] = x["logits"][:, :4].argmax(-1).astype(np.int32)
    kepts = check(x, run(x)[0])
    assert len(set(kepts)) > 2


def test_plain_sampling_without_drafts():
    x = make(7, 0, 9001, seed=5)
    out, _ = run(x)
    check(x, out)
    assert (out.accept_len == 1).all()


def test_every_draft_kept_and_every_draft_refused():
    x = make(4, 5, 2000, seed=6, noise=0.0, io="f32")
    x["u"][:] = 0.0
    assert check(x, run(x)[0]) == [5] * 4
    x["q"][:] = 0
    x["q"][np.arange(4)[:, None], np.arange(5), x["toks"]] = 1.0
    x["u"][:] = np.float32(1 - 2 ** -24)
    assert check(x, run(x)[0]) == [0] * 4


def test_kv_len_and_root_token_advance():
    x = make(6, 3, 500, seed=7)
    kv = torch.arange(6, dtype=torch.int32, device="cuda") * 10
    root = torch.zeros(6, dtype=torch.int32, device="cuda")
    out, _ = run(x, kv_len=kv, root=root)
    lens = out.accept_len.cpu()
    assert torch.equal(kv.cpu(), torch.arange(6, dtype=torch.int32) * 10 + lens)
    assert torch.equal(root.cpu(), out.out_tok.cpu()[torch.arange(6), lens.long() - 1])


def test_masked_logits():
    """-inf logits (tokens ruled out) have probability 0 and are never drawn."""
    x = make(4, 3, 1000, seed=8, io="f32")
    x["logits"][:, :, 1::2] = -np.inf
    out, ws = run(x)
    check(x, out)
    assert binding.spec_status_read(ws) == 0
    lens = out.accept_len.cpu().numpy()
    assert (out.out_tok.cpu().numpy()[np.arange(4), lens - 1] % 2 == 0).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf, "all"])
def test_rows_without_probabilities(bad):
    x = make(3, 2, 700, seed=9, io="f32")
    if bad == "all":
        x["logits"][1, 0] = -np.inf
    else:
        x["logits"][1, 0, 5] = bad
    out, ws = run(x)
    assert binding.spec_status_read(ws) == binding.SPEC_DEV_BADLOGIT
    assert out.out_tok[1].tolist() == [0, -1, -1] and out.accept_len[1] == 1
    x["n"] = np.array([2, 0, 2], np.int32)
    assert out.target_prob[1, 0] == 0


def test_drafts_outside_the_vocabulary_and_counts_outside_the_range():
    x = make(3, 3, 400, seed=10)
    x["toks"][0, 0] = 400
    x["toks"][1, 1] = -1
    x["u"][:] = 0
    out, ws = run(x)
    assert binding.spec_status_read(ws) == binding.SPEC_DEV_BADTOK
    assert out.accept_len.tolist() == [1, 2, 4]
    assert out.target_prob[0, 0] == 0 and out.target_prob[1, 1] == 0
    x = make(3, 3, 400, seed=11)
    x["n"] = np.array([-2, 9, 3], np.int32)
    out, ws = run(x)
    assert binding.spec_status_read(ws) == binding.SPEC_DEV_BADREQ
    x["n"] = np.array([0, 3, 3], np.int32)
    check(x, out)


def test_ties_go_to_the_lowest_token():
    x = make(1, 0, 5000, seed=12, io="f32")
    x["logits"][:] = 0
    x["e"][:] = 1
    x["e"][0, [77, 1234, 4999]] = 0.5
    assert run(x)[0].out_tok.item() == 77


def test_exponentials_below_the_normal_range():
    """Scores of 2^110 and more, whose exponentials have no finite approximate
    reciprocal, are told apart; equal ones go to the lowest token."""
    x = make(3, 1, 4000, seed=14, spread=0.5)
    x["e"][:] = 1.0
    x["u"][:] = 1.0                                        # the draft is refused
    x["q"][:] = 0.0
    x["q"][:, 0, 0] = 1.0
    x["toks"][:] = 0
    pairs = [(8, 9), (100, 3000), (17, 2049)]
    for b, at in enumerate(pairs):
        x["e"][b, list(at)] = 2.0 ** -128
        x["logits"][b, 0, list(at)] = (0.25, 1.5 if b < 2 else 0.25)
    out, _ = run(x)
    assert out.accept_len.tolist() == [1, 1, 1]
    assert out.out_tok[:, 0].tolist() == [9, 3000, 17]


def test_drafters_that_equal_the_target_at_the_draft():
    """Residuals that vanish: a refusal by u q = p exactly, with q = p
    everywhere but for the roundings, falls back to a token of p."""
    V = 64
    x = make(1, 1, V, seed=13, io="f32")
    x["logits"][:] = 0
    x["q"][:] = 1.0 / V
    x["u"][:] = 1.0
    out, _ = run(x)
    assert out.accept_len.item() == 1
    assert out.out_tok[0, 0].item() == int((1 / x["e"][0].astype(np.float64)).argmax())


def test_graph_and_stream():
    x = make(4, 5, 20011, seed=14)
    want, ws = run(x)
    cfg = binding.draft_cfg(B=4, N=5, V=20011)
    d = {k: torch.from_numpy(x[k]).cuda() for k in ("q", "toks", "u", "e")}
    logits = torch.from_numpy(x["logits"]).bfloat16().cuda()
    out = binding.DraftBuffers(cfg)
    kv = torch.zeros(4, dtype=torch.int32, device="cuda")

    def call(stream=None):
        binding.draft_verify_sampled(cfg, d["toks"], d["q"], logits, d["u"], d["e"], out, ws,
                                     kv_len=kv, stream=stream)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    call(st)
    st.synchronize()
    assert torch.equal(out.out_tok, want.out_tok) and torch.equal(kv, want.accept_len)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    out.out_tok.zero_()
    for _ in range(4):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.out_tok, want.out_tok) and torch.equal(kv, 5 * want.accept_len)
    assert torch.equal(out.target_prob, want.target_prob)


def test_outputs_and_workspaces_of_another_shape_are_refused():
    x = make(3, 2, 100, seed=15)
    cfg = binding.draft_cfg(B=3, N=2, V=100)
    for B, N in ((2, 2), (3, 1)):
        with pytest.raises(ValueError):
            run(x, out=binding.DraftBuffers(binding.draft_cfg(B=B, N=N, V=100)))
    with pytest.raises((TypeError, ValueError)):
        run(x, out=binding.DraftBuffers(cfg, device="cpu"))
    for ws in (binding.alloc_draft_workspace(cfg)[:256], [0]):
        with pytest.raises((TypeError, ValueError)):
            run(x, ws=ws)
    with pytest.raises(TypeError):
        run(x, ws=torch.zeros(1 << 20, dtype=torch.uint8))
    check(x, run(x)[0])


def test_frequencies_follow_the_target():
    """4000 independent requests at once: the first emitted token of a chain of
    one draft follows p (chi-square over 6 tokens, 5 degrees: 99.9% is 20.5)."""
    B, V = 4000, 6
    rng = np.random.default_rng(15)
    z, d = rng.standard_normal(V).astype(np.float32), rng.standard_normal(V)
    q = ref.softmax(d).astype(np.float32)
    x = make(B, 1, V, io="f32", seed=16)
    x["logits"][:] = z
    x["q"][:] = q
    x["toks"] = rng.choice(V, size=(B, 1), p=q.astype(np.float64) / q.sum(dtype=np.float64)).astype(np.int32)
    out, _ = run(x)
    seen = np.bincount(out.out_tok[:, 0].cpu().numpy(), minlength=V)
    want = B * ref.softmax(z.astype(np.float64))
    assert ((seen - want) ** 2 / want).sum() < 20.5


# -------------------------------------------------------------- whole serving steps

@pytest.mark.parametrize("kv", ["e4m3", "io"])
def test_serving_steps(kv):
    """Four steps of three requests, two attention layers: rows appended,
    attended and verified by step.ChainStep, against the same steps in 64 bits
    with the rows kept by a plain list per request (rows of refused drafts are
    written over by the next step)."""
    rng = np.random.default_rng(20)
    B, N, V, Hq, Hkv, D, page, layers = 3, 4, 997, 8, 2, 64, 16, 2
    T = N + 1
    pc = binding.paged_cfg(B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, page=page, n_pages=12, max_pages=4, kv=kv)
    dc = binding.draft_cfg(B=B, N=N, V=V)
    table = rng.permutation(12).reshape(B, 4).astype(np.int32)
    st = step.ChainStep(pc, dc, layers)
    st.page_table.copy_(torch.from_numpy(table))
    hist = [[{"k": [], "v": []} for _ in range(B)] for _ in range(layers)]
    lens = np.zeros(B, int)
    f = lambda x: torch.from_numpy(np.ascontiguousarray(x)).bfloat16().cuda()  # noqa: E731
    for s in range(4):
        n = rng.integers(0, N + 1, B).astype(np.int32)
        st.n_draft.copy_(torch.from_numpy(n))
        for l in range(layers):
            new = {c: ref.bf16(rng.standard_normal((B, T, Hkv, D)).astype(np.float32)) for c in "kv"}
            q = ref.bf16(rng.standard_normal((B, T, Hq, D)).astype(np.float32))
            o = st.attend(l, f(q), f(new["k"]), f(new["v"])).double().cpu().numpy()
            for b in range(B):
                for c in "kv":
                    x = new[c][b, :n[b] + 1]
                    if kv == "e4m3":
                        y, sc = ref.quantise(x)
                        x = y * sc[..., None].astype(np.float64)
                    hist[l][b][c][lens[b]:] = list(x.astype(np.float64))
                k, v = (np.stack(hist[l][b][c]) for c in "kv")
                for i in range(T):
                    for h in range(Hq):
                        if i > n[b]:
                            assert (o[b, i, h] == 0).all()
                            continue
                        hk = h // (Hq // Hkv)
                        seen = (np.arange(len(k)) <= lens[b] + i)[None]
                        w, A, z = ref.attention(q[b, i, h:h + 1].astype(np.float64), k[:, hk], v[:, hk], seen)
                        tol = 2.0 ** -8 * np.abs(w) + (2.0 ** -11 + 2.0 ** -16 * (1 + z[:, None])) * A
                        assert (np.abs(o[b, i, h] - w[0]) <= tol[0]).all()
        x = make(B, N, V, seed=100 + s)
        x["n"] = n
        out = st.verify(f(x["logits"]), *(torch.from_numpy(x[c]).cuda() for c in ("toks", "q", "u", "e")))
        check(x, out)
        lens += out.accept_len.cpu().numpy()
        np.testing.assert_array_equal(st.kv_len.cpu().numpy(), lens)
        for l in range(layers):
            for b in range(B):
                for c in "kv":
                    del hist[l][b][c][lens[b]:]
    assert st.status() == 0


def test_paged_rows_read_back_feed_the_tree_attention():
    """kv_page_read's output is attn_tree_verify's cache: a chain of T rows as a
    tree over it equals attn_decode_paged over the pages, within their bounds."""
    import oracle  # noqa: F401  (the tree's layout is the library's own)
    from speculative_decoding_tree_best_gb300 import synth
    sc = synth.config(1).replace(B=2, m=4, K=2, N=4, L=200, headroom=24)
    cfg = binding.make_cfg(sc)
    T = sc.N + 1
    rng = np.random.default_rng(21)
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).bfloat16().cuda()  # noqa: E731
    pc = binding.paged_cfg(B=2, T=200, Hq=sc.Hq, Hkv=sc.Hkv, D=sc.D, page=32, n_pages=20, max_pages=8)
    kv = binding.PagedKV.empty(pc)
    kv.page_table.copy_(torch.from_numpy(rng.permutation(20)[:16].reshape(2, 8).astype(np.int32)))
    ws = binding.alloc_paged_workspace(pc)
    n = torch.tensor([200, 77], dtype=torch.int32, device="cuda")
    binding.kv_page_append(pc, kv, f(2, 200, sc.Hkv, sc.D), f(2, 200, sc.Hkv, sc.D), ws, n_new=n)
    kv.kv_len.copy_(n)
    cache = [torch.zeros((2, sc.Lmax, sc.Hkv, sc.D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    binding.kv_page_read(pc, kv, *cache, ws)
    # a chain as a tree
    tree = binding.TreeBuffers(cfg)
    i = torch.arange(T, dtype=torch.int32, device="cuda")
    for name, v in (("node_tok", i), ("node_parent", i - 1), ("node_depth", i), ("node_rank", i * 0)):
        getattr(tree, name).copy_(v.expand(2, T))
    tree.node_score.zero_()
    tree.n_nodes.fill_(T)
    tree.node_anc.zero_()
    tree.node_anc[:, :, 0] = (2 ** (i.long() + 1) - 1)
    q, k, v = f(2, T, sc.Hq, sc.D), f(2, T, sc.Hkv, sc.D), f(2, T, sc.Hkv, sc.D)
    want = torch.empty_like(q)
    binding.attn_tree_verify(cfg, tree, q, k, v, *cache, kv.kv_len, want, binding.alloc_workspace(cfg))
    step_cfg = binding.paged_cfg(B=2, T=T, Hq=sc.Hq, Hkv=sc.Hkv, D=sc.D, page=32, n_pages=20, max_pages=8)
    binding.kv_page_append(step_cfg, kv, k, v, ws)
    got = torch.empty_like(q)
    ws2 = binding.alloc_paged_workspace(step_cfg)
    binding.attn_decode_paged(step_cfg, kv, q, got, ws2)
    d = (got.double() - want.double())
    # each is within its own bound (rel-L2 2e-3 of the 64-bit result)
    assert float(d.norm() / want.double().norm()) < 4e-3
    assert binding.spec_status_read(ws) == 0 and binding.spec_status_read(ws2) == 0
