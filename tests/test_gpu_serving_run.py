"""A serving loop of step.ChainStep with everything a step has: pages from the
pool, rotated rows into the cache, attention, drafts drawn with filters, the
target's logits filtered and verified, pages given back.  Each part is held to
its 64-bit form on the inputs that the part before it left."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_best_gb300 import binding, step
from tests import indep_chain as chain, indep_serving as ref
from tests.test_gpu_chain import MARGIN
from tests.test_gpu_rope import near
from tests.test_gpu_sample import NEAR

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_best_gb300 import build
    build.build()
    binding.load()


@pytest.mark.parametrize("kv", ["io", "e4m3"])
def test_serving_loop(kv):
    rng = np.random.default_rng(31)
    B, N, V, Hq, Hkv, D, page, layers, n_pages = 4, 3, 1009, 4, 2, 64, 16, 2, 11
    T = N + 1
    pc = binding.paged_cfg(B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, page=page, n_pages=n_pages, max_pages=6,
                           kv=kv)
    st = step.ChainStep(pc, binding.draft_cfg(B=B, N=N, V=V, temperature=0.8), layers)
    scaling = dict(scaling="yarn", factor=4.0, orig_len=64)
    table = binding.rope_table(48, base=1e4, **scaling)
    f, amp = ref.frequencies(48, 1e4, **scaling)
    wide = (Hq + 2 * Hkv) * D
    rc = binding.rope_cfg(B * T, Hq, Hkv, D, 48, q_stride=wide, k_stride=wide, v_stride=wide)
    state = {n: getattr(st.pool, n).cpu().numpy() for n in ("page_table", "kv_len", "free_list",
                                                             "n_free", "n_held")}
    lens, refused, k, p = np.zeros(B, int), 0, np.array([40, 5, 0, 200], np.int32), np.array(
        [0.9, 1.0, 0.8, 0.95], np.float32)
    filters = dict(top_k=torch.from_numpy(k).cuda(), top_p=torch.from_numpy(p).cuda())
    temp = np.array([0.7, 1.0, 1.3, 0.9], np.float32)
    for s in range(14):
        n = rng.integers(0, N + 1, B).astype(np.int32)
        if s == 5:
            n[2] = -1                                     # no request in this slot
        st.n_draft.copy_(torch.from_numpy(n))
        st.begin()
        slots, ok = ref.extend(state, page, n + 1, T)
        np.testing.assert_array_equal(st.slots.cpu().numpy(), slots)
        np.testing.assert_array_equal(st.n_draft.cpu().numpy(), ok - 1)
        refused += int((ok < n + 1).sum())
        n = ok - 1
        for l in range(layers):
            rows = torch.from_numpy(rng.standard_normal((B, T, wide)).astype(np.float32)).cuda().bfloat16()
            q, kn, vn = (x.unflatten(2, (-1, D)) for x in rows.split([Hq * D, Hkv * D, Hkv * D], 2))
            o = st.attend_rope(l, rc, table, q, kn, vn).double().cpu().numpy()
            real = slots >= 0
            pos = (lens[:, None] + np.arange(T))[real]
            mask = torch.from_numpy(real).cuda()
            if real.any():
                near(st._q[mask], q[mask], pos, f, amp, "half", "bf16")
            # what the rows stand for in the cache, and attention over it
            total = lens + n + 1
            look = binding.PagedKV(pc, st.caches[l].k_pages, st.caches[l].v_pages, st.page_table,
                                   torch.from_numpy(total.astype(np.int32)).cuda(),
                                   st.caches[l].k_scale, st.caches[l].v_scale)
            got = [torch.zeros((B, 6 * page, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
            binding.kv_page_read(pc, look, *got, st.paged_ws)
            if kv == "io" and real.any():
                b, i = np.nonzero(real)
                near(got[0][b, lens[b] + i], kn[mask], pos, f, amp, "half", "bf16")
                assert torch.equal(got[1][b, lens[b] + i], vn[mask])
            if kv == "e4m3":                               # codes are exact in bf16, their products not
                got = [((c.view(torch.uint8).view(torch.float8_e4m3fn).double()
                         * sc.double().unsqueeze(-1))[st.page_table.long().clamp_min(0)]
                        .transpose(2, 3).reshape(B, -1, Hkv, D))
                       for c, sc in ((st.caches[l].k_pages, st.caches[l].k_scale),
                                     (st.caches[l].v_pages, st.caches[l].v_scale))]
            kk, vv = (x.double().cpu().numpy() for x in got)
            qr = st._q.double().cpu().numpy()
            for b in range(B):
                for i in range(T):
                    for h in range(Hq):
                        if i > n[b]:
                            assert (o[b, i, h] == 0).all()
                            continue
                        L = total[b]
                        seen = (np.arange(L) <= lens[b] + i)[None]
                        w, A, z = chain.attention(qr[b, i, h:h + 1], kk[b, :L, h // 2], vv[b, :L, h // 2], seen)
                        tol = 2.0 ** -8 * np.abs(w) + (2.0 ** -11 + 2.0 ** -16 * (1 + z[:, None])) * A
                        assert (np.abs(o[b, i, h] - w[0]) <= tol[0]).all()
        # drafts, with the distributions that they were drawn from
        toks = torch.zeros((B, N), dtype=torch.int32, device="cuda")
        probs = torch.zeros((B, N, V), device="cuda")
        for i in range(N):
            z = torch.from_numpy((2.5 * rng.standard_normal((B, V))).astype(np.float32)).cuda().bfloat16()
            e = torch.from_numpy(rng.exponential(size=(B, V)).astype(np.float32) + np.float32(1e-30)).cuda()
            st.draft(i, z, e, toks, probs, temperature=torch.from_numpy(temp).cuda(), **filters)
            for b in range(B):
                want, _, margin = ref.sample(z[b].float().cpu().numpy(), float(temp[b]), int(k[b]), float(p[b]))
                if margin < NEAR:
                    continue
                np.testing.assert_allclose(probs[b, i].cpu().numpy(), want, rtol=2.0 ** -20, atol=1e-37)
                assert want[int(toks[b, i])] > 0
        logits = torch.from_numpy((2.5 * rng.standard_normal((B, T, V))).astype(np.float32)).cuda().bfloat16()
        u = torch.from_numpy(rng.random((B, N)).astype(np.float32)).cuda()
        e = torch.from_numpy(rng.exponential(size=(B, V)).astype(np.float32) + np.float32(1e-30)).cuda()
        out = st.verify(logits, toks, probs, u, e, **filters)
        tau, got = out.accept_len.cpu().numpy(), out.out_tok.cpu().numpy()
        for b in range(B):
            if n[b] < 0:
                assert tau[b] == 0 and (got[b] == -1).all()
                continue
            x, sure = logits[b].float().cpu().numpy().astype(np.float64), True
            for i in range(n[b] + 1):
                want, _, margin = ref.sample(x[i], float(np.float32(0.8)), int(k[b]), float(p[b]))
                sure &= margin >= NEAR
                x[i][want == 0] = -np.inf
            with np.errstate(divide="ignore", invalid="ignore"):
                kept, tok, _, margin = chain.chain(x, probs[b].cpu().numpy(), toks[b, :n[b]].cpu().numpy(),
                                                   u[b].cpu().numpy(), e[b].cpu().numpy(), float(np.float32(0.8)))
            if sure and margin >= MARGIN:
                assert tau[b] == kept + 1 and got[b, kept] == tok
            assert np.isfinite(x[tau[b] - 1][got[b, tau[b] - 1]])      # filtered tokens never come out
        lens = lens + tau
        np.testing.assert_array_equal(st.kv_len.cpu().numpy(), lens)
        state["kv_len"][:] = lens
        ended = lens > 3 * page
        st.release(torch.from_numpy(ended).cuda())
        ref.trim(state, page, np.where(ended, 0, lens))
        lens = np.where(ended, 0, lens)
        for name, y in state.items():
            np.testing.assert_array_equal(getattr(st.pool, name).cpu().numpy(), y, err_msg=name)
    assert st.status() == (binding.SPEC_DEV_NOPAGE if refused else 0)


def test_requests_without_pages_wait():
    """Four requests and three pages: the last one has no request in its slot until
    another one's pages come back."""
    B, N, V, Hq, Hkv, D = 4, 2, 100, 2, 1, 64
    pc = binding.paged_cfg(B=B, T=N + 1, Hq=Hq, Hkv=Hkv, D=D, page=16, n_pages=3, max_pages=2)
    st = step.ChainStep(pc, binding.draft_cfg(B=B, N=N, V=V), 1)
    rc, table = binding.rope_cfg(B * (N + 1), Hq, Hkv, D), binding.rope_table(D)
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731

    def one_step():
        st.n_draft.fill_(0)
        st.begin()
        got = st.n_draft.tolist()
        o = st.attend_rope(0, rc, table, r(B, N + 1, Hq, D), r(B, N + 1, Hkv, D), r(B, N + 1, Hkv, D))
        for b in range(B):
            assert (o[b, 0].abs().sum() > 0) == (got[b] >= 0) and (o[b, 1:] == 0).all()
        out = st.verify(r(B, N + 1, V), torch.zeros((B, N), dtype=torch.int32, device="cuda"), None,
                        torch.zeros((B, N), device="cuda"), torch.ones((B, V), device="cuda"))
        return got, out.accept_len.tolist()

    assert one_step() == ([0, 0, 0, -1], [1, 1, 1, 0])
    assert st.status() == binding.SPEC_DEV_NOPAGE and st.kv_len.tolist() == [1, 1, 1, 0]
    st.release(torch.tensor([False, True, False, False], device="cuda"))
    assert st.kv_len.tolist() == [1, 0, 1, 0] and int(st.pool.n_free) == 1
    # request 1 comes first again; given back at once, its page goes to request 3
    assert one_step() == ([0, 0, 0, -1], [1, 1, 1, 0])
    st.release(torch.tensor([True, True, False, False], device="cuda"))
    assert one_step() == ([0, 0, 0, -1], [1, 1, 1, 0])
    st.release(torch.tensor([True, True, True, True], device="cuda"))
    assert int(st.pool.n_free) == 3 and (st.page_table == -1).all()
