"""Filters in a serving step: rows and slots that do not count, temperatures that
change, steps captured before anything ran."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_best_gb300 import binding, step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_best_gb300 import build
    build.build()
    binding.load()


B, N, V = 6, 3, 2003


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def chain_step(temperature=0.8):
    pc = binding.paged_cfg(B=B, T=N + 1, Hq=2, Hkv=1, D=64, page=16, n_pages=24, max_pages=4)
    return step.ChainStep(pc, binding.draft_cfg(B=B, N=N, V=V, temperature=temperature), 1)


def inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    prob = r(B, N, V) + 1e-3
    return dict(logits=(3 * torch.randn((B, N + 1, V), generator=g, device="cuda")).bfloat16(),
                draft_tok=torch.randint(0, V, (B, N), generator=g, device="cuda", dtype=torch.int32),
                draft_prob=prob / prob.sum(2, keepdim=True), u=r(B, N) * 0.2,
                e=-torch.log(r(B, V) * 0.999 + 5e-4))


FILTERS = dict(top_k=[40, 0, 7, 300, 1, 60], top_p=[0.9, 0.8, 1.0, 0.95, 0.5, 0.7])


def filters():
    return dict(top_k=i32(*FILTERS["top_k"]), top_p=torch.tensor(FILTERS["top_p"], device="cuda"))


def result(out):
    return out.accept_len.tolist(), out.out_tok.tolist()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("R,V,per", [(24, 1009, 4), (10, 60013, 4), (7, 30011, 1), (9, 515, 20)])
def test_rows_that_do_not_count(io, R, V, per):
    """Skipped rows: outputs as they were, though their logits are NaN.  Quiet rows:
    outputs as without last_row.  Neither raises anything."""
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[io]
    g = torch.Generator(device="cuda").manual_seed(R)
    x = (3 * torch.randn((R, V), generator=g, device="cuda")).to(dt)
    e = torch.rand((R, V), generator=g, device="cuda") + 1e-3
    n = -(-R // per)
    last = torch.randint(-1, per + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    last[0], last[n // 2] = -1, -7                                      # held to 0: its first row counts
    counts = torch.tensor([int(last[r // per]) != -1 and r % per <= max(int(last[r // per]), 0)
                           for r in range(R)], device="cuda")
    assert 0 < int(counts.sum()) < R
    par = dict(top_k=torch.randint(0, 2000, (n,), generator=g, device="cuda", dtype=torch.int32),
               top_p=0.5 + 0.5 * torch.rand((n,), generator=g, device="cuda"))
    cfg = binding.sample_cfg(R, V, per, io)
    ws = binding.alloc_sample_workspace(cfg)
    bad = x.clone()
    bad[~counts, V // 2] = float("nan")

    def run(x, **kw):
        out = binding.SampleBuffers(cfg, prob=True, logits=True)
        for t in (out.tok, out.tok_prob, out.prob, out.logits):
            t.fill_(7)
        binding.token_sample(cfg, x, e, out, ws, **par, **kw)
        return out.tok, out.tok_prob, out.prob, out.logits
    want = run(x)
    for got, w in zip(run(bad, last_row=last), want):
        assert torch.equal(got[counts], w[counts]) and (got[~counts] == 7).all()
    for got, w in zip(run(x, last_row=last, idle="quiet"), want):
        assert torch.equal(got, w)
    got = run(bad, last_row=last, idle="quiet")
    assert (got[0][~counts] == 0).all() and (got[2][~counts] == 0).all()
    assert binding.spec_status_read(ws) == 0
    run(bad)
    assert binding.spec_status_read(ws) == binding.SPEC_DEV_BADLOGIT


def test_verify_with_filters_reads_what_counts():
    """Rows beyond n_draft and slots without a request hold NaN: results and status as
    with numbers there, and as without filters that remove nothing."""
    x = inputs(1)
    n = i32(N, 1, -1, 0, 2, -1)
    idle = torch.arange(N + 1, device="cuda") > n.view(-1, 1)
    nan = x["logits"].clone()
    nan[idle] = float("nan")
    got = []
    for logits, kw in ((x["logits"], filters()), (nan, filters()),
                       (x["logits"], {}), (nan, dict(top_k=i32(*[0] * B)))):
        st = chain_step()
        st.n_draft.copy_(n)
        got.append(result(st.verify(**dict(x, logits=logits), **kw)))
        assert st.status() == 0
    assert got[0] == got[1] and got[2] == got[3]
    assert got[0][0][2] == 0 and got[0][1][5] == [-1] * (N + 1)


def test_slots_without_a_request_draft_quietly():
    x = inputs(2)
    st = chain_step()
    st.n_draft.copy_(i32(N, 1, -1, 0, 2, -1))
    logits = x["logits"][:, 0].contiguous()
    logits[2, 5] = logits[5, 0] = float("nan")
    st.draft(1, logits, x["e"], x["draft_tok"], x["draft_prob"], **filters())
    assert st.status() == 0
    assert (x["draft_prob"][2, 1] == 0).all() and int(x["draft_tok"][2, 1]) == 0
    assert abs(float(x["draft_prob"][3, 1].sum()) - 1) < 1e-5
    logits[4, 9] = float("nan")
    st.draft(1, logits, x["e"], x["draft_tok"], x["draft_prob"], **filters())
    assert st.status() == binding.SPEC_DEV_BADLOGIT


def kept_at(x, temperature):
    st = chain_step(temperature)
    out = result(st.verify(**x, **filters()))
    return out, (st._filtered.logits > -np.inf).sum(1).tolist()


def test_the_temperature_changes_between_steps():
    x = inputs(3)
    st = chain_step(0.4)
    for t in (0.4, 1.7, 0.4):
        st.dcfg.temperature = t
        got = result(st.verify(**x, **filters()))
        assert (got, (st._filtered.logits > -np.inf).sum(1).tolist()) == kept_at(x, t)
    assert kept_at(x, 0.4)[1] != kept_at(x, 1.7)[1]


def test_steps_captured_before_anything_ran():
    """draft and verify captured as the step's first calls; calls outside the graph,
    at another temperature, before and between its replays."""
    x = inputs(4)
    z = x["logits"][:, 1].contiguous()
    toks, probs = x["draft_tok"].clone(), x["draft_prob"].clone()
    fresh = chain_step(0.5)
    fresh.draft(2, z, x["e"], toks, probs, temperature=torch.full((B,), 0.6, device="cuda"))
    want = result(fresh.verify(**dict(x, draft_tok=toks, draft_prob=probs), **filters()))
    st, f, t = chain_step(0.5), filters(), torch.full((B,), 0.6, device="cuda")
    toks2, probs2 = x["draft_tok"].clone(), x["draft_prob"].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.draft(2, z, x["e"], toks2, probs2, temperature=t)
        st.verify(**dict(x, draft_tok=toks2, draft_prob=probs2), **f)
    assert st.status() == 0
    for _ in range(2):
        st.dcfg.temperature = 1.7
        assert result(st.verify(**x, **f)) == kept_at(x, 1.7)[0]
        graph.replay()
        assert result(st.out) == want
        assert torch.equal(toks2, toks) and torch.equal(probs2, probs)
    assert st.status() == 0
