"""The paged cache and the attention over it against plain 64-bit
implementations: rows of every type written and read back to the bit, and
attention from one key to long caches, odd sizes, ragged batches, masked and
poisoned rows, shared pages, other streams and captured graphs.

Tolerances.  The cache's codes, scales and values are single fp32 operations
and compare exactly.  An attention output differs from the 64-bit one by
  u |o|               its one rounding: u = 2^-8 (bf16), 2^-24 (fp32);
  c A, A = sum w |v|  with c = 2^-11 where the weights are rounded to fp16
                      (8-bit cache, bf16 I/O), 2^-16 where they are the sum of
                      two bf16 parts, 2^-20 in the fp32 paths (two tf32 or fp16
                      parts, 2^-21 or better each, on both sides of a product);
  2 d A               the weights' own error: a score is a sum of D products
                      in at most 32 fp32 additions, each within 2^-23 of the
                      sum of magnitudes z, and its operands are split to
                      2^-21 at worst: d = (32 2^-23 + 2 2^-21) z + 2^-20;
  L 2^-23 A           fp32 sums over L keys.
"""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_best_gb300 import binding
from tests import indep_chain as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_best_gb300 import build
    build.build()
    binding.load()


class Case:
    """A pool whose every slot is poisoned (NaN) but for the rows in use."""

    def __init__(self, lens, T=1, Hq=4, Hkv=2, D=64, page=16, io="bf16", kv="io", n_new=None,
                 max_pages=None, extra=3, seed=0, spread=1.0):
        rng = self.rng = np.random.default_rng(seed)
        B = len(lens)
        self.io, self.kvt, self.lens = io, kv, list(lens)
        self.n = [T] * B if n_new is None else list(n_new)
        need = max(max(lens) + T, 1)
        cols = max_pages or -(-need // page)
        n_pages = B * cols + extra
        self.cfg = binding.paged_cfg(B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, page=page, n_pages=n_pages,
                                     max_pages=cols, io=io, kv=kv)
        self.table = rng.permutation(n_pages)[:B * cols].reshape(B, cols).astype(np.int32)
        self.vals, self.scale, self.raw = {}, {}, {}
        for n in ("k", "v"):
            x = rng.standard_normal((B, cols * page, Hkv, D)).astype(np.float32)
            x *= np.exp(spread * rng.standard_normal(x.shape[:-1])).astype(np.float32)[..., None]
            x = ref.bf16(x) if io == "bf16" else x
            self.raw[n] = x
            if kv == "e4m3":
                self.vals[n], self.scale[n] = ref.quantise(x)
            else:
                self.vals[n] = x.astype(np.float64)
        self.q = rng.standard_normal((B, T, Hq, D)).astype(np.float32) * 1.5
        self.q = ref.bf16(self.q) if io == "bf16" else self.q
        self.upload()

    def row(self, n, b, r):
        """[Hkv][D] in 64 bits."""
        x = self.vals[n][b, r]
        return x * self.scale[n][b, r].astype(np.float64)[:, None] if self.kvt == "e4m3" else x

    def upload(self, filled=None):
        """Rows [0, kv_len + n_new) of each request in a pool of NaN."""
        c = self.cfg
        shape = (c.n_pages, c.Hkv, c.page, c.D)
        pools, scales = [], []
        for n in ("k", "v"):
            pool = np.full(shape, np.nan, np.float64)
            sc = np.full(shape[:3], np.nan, np.float32)
            for b, L in enumerate(self.lens):
                end = L + self.n[b] if filled is None else filled[b]
                for r in range(max(0, min(end, c.page * c.max_pages))):
                    p = self.table[b][r // c.page]
                    if 0 <= p < c.n_pages:
                        pool[p, :, r % c.page] = self.vals[n][b, r]
                        if self.kvt == "e4m3":
                            sc[p, :, r % c.page] = self.scale[n][b, r]
            dt = torch.float8_e4m3fn if self.kvt == "e4m3" else DT[self.io]
            pools.append(torch.from_numpy(pool.astype(np.float32)).to(dt).cuda())
            scales.append(torch.from_numpy(sc).cuda() if self.kvt == "e4m3" else None)
        self.pools, self.scales = pools, scales
        self.kv = binding.PagedKV(c, *pools, torch.from_numpy(self.table).cuda(),
                                  torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                                  *scales)
        self.ws = binding.alloc_paged_workspace(c)

    def dev(self, x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(DT[self.io]).cuda()

    def n_dev(self):
        return torch.tensor(self.n, dtype=torch.int32, device="cuda")

    def attend(self, o=None, **kw):
        c = self.cfg
        o = torch.full((c.B, c.T, c.Hq, c.D), 7.0, dtype=DT[self.io], device="cuda") if o is None else o
        binding.attn_decode_paged(c, self.kv, self.dev(self.q), o, self.ws, n_new=self.n_dev(), **kw)
        return o

    def check(self, o, hide=()):
        """o against the 64-bit attention; hide: {(b, page column)} not seen."""
        c = self.cfg
        got = o.double().cpu().numpy()
        G, cap = c.Hq // c.Hkv, c.page * c.max_pages
        u = 2.0 ** -8 if self.io == "bf16" else 2.0 ** -24
        cw = {("bf16", "e4m3"): 2.0 ** -11, ("bf16", "io"): 2.0 ** -16}.get((self.io, self.kvt), 2.0 ** -20)
        for b in range(c.B):
            end = min(self.lens[b] + self.n[b], cap)
            rows = {n: np.stack([self.row(n, b, r) for r in range(end)]) if end else
                    np.zeros((0, c.Hkv, c.D)) for n in ("k", "v")}
            ok = np.array([(b, r // c.page) not in hide for r in range(end)], bool)
            for h in range(c.Hkv):
                q = self.q[b, :, h * G:(h + 1) * G].reshape(c.T * G, c.D).astype(np.float64)
                lim = np.array([self.lens[b] + i + 1 if i < self.n[b] else 0 for i in range(c.T)
                                for _ in range(G)])
                seen = (np.arange(end) < lim[:, None]) & ok
                want, A, z = ref.attention(q, rows["k"][:, h], rows["v"][:, h], seen)
                g = got[b, :, h * G:(h + 1) * G].reshape(c.T * G, c.D)
                d = (32 * 2.0 ** -23 + 2 * 2.0 ** -21) * z[:, None] + 2.0 ** -20
                tol = u * np.abs(want) + (cw + 2 * d + end * 2.0 ** -23) * A + 1e-37
                assert np.isfinite(g[np.isfinite(want)]).all(), (b, h)
                bad = np.abs(g - want) > tol
                assert not bad.any(), (b, h, float((np.abs(g - want) / tol).max()))
                np.testing.assert_array_equal(g[lim == 0], 0.0)

    def status(self):
        return binding.spec_status_read(self.ws)


# --------------------------------------------------------------- write, read back

@pytest.mark.parametrize("io,kv", [("bf16", "e4m3"), ("f32", "e4m3"), ("bf16", "io"), ("f32", "io")])
@pytest.mark.parametrize("D,Hkv,page", [(64, 1, 16), (128, 3, 32), (128, 8, 64)])
def test_append_and_read(io, kv, D, Hkv, page):
    lens, n_new = [0, 1, 15, 16, 37, 64], [5, 1, 2, 0, 3, 5]
    x = Case(lens, T=5, Hq=Hkv, Hkv=Hkv, D=D, page=page, io=io, kv=kv, n_new=n_new, seed=D + Hkv)
    c = x.cfg
    x.upload(filled=lens)                                  # the new rows are not there yet
    before = [p.clone() for p in x.pools] + [s.clone() for s in x.scales if s is not None]
    new = {n: np.stack([x.raw[n][b, lens[b]:lens[b] + c.T] for b in range(c.B)]) for n in ("k", "v")}
    binding.kv_page_append(c, x.kv, x.dev(new["k"]), x.dev(new["v"]), x.ws, n_new=x.n_dev())
    done = ref.place(c, x.table, lens, n_new)
    assert len(done) == sum(n_new)
    for j, n in enumerate(("k", "v")):
        want = before[j].double().cpu().numpy()
        for b, i, p, s in done:
            want[p, :, s] = x.vals[n][b, lens[b] + i]
        np.testing.assert_array_equal(x.pools[j].double().cpu().numpy(), want)
        if kv == "e4m3":
            ws = before[2 + j].cpu().numpy()
            for b, i, p, s in done:
                ws[p, :, s] = x.scale[n][b, lens[b] + i]
            np.testing.assert_array_equal(x.scales[j].cpu().numpy(), ws)
    # read back everything, the new rows as well
    x.kv.kv_len.add_(x.n_dev())
    Lmax = 75
    out = [torch.full((c.B, Lmax, Hkv, D), 3.0, dtype=DT[io], device="cuda") for _ in range(2)]
    binding.kv_page_read(c, x.kv, *out, x.ws)
    for n, o in zip(("k", "v"), out):
        want = np.full((c.B, Lmax, Hkv, D), 3.0)
        for b in range(c.B):
            for r in range(lens[b] + n_new[b]):
                y = x.vals[n][b, r].astype(np.float32)
                if kv == "e4m3":
                    y = y * x.scale[n][b, r][:, None]      # one fp32 product
                want[b, r] = ref.bf16(y) if io == "bf16" else y
        np.testing.assert_array_equal(o.double().cpu().numpy(), want)
    assert x.status() == 0


def test_rows_of_zeros_extremes_and_non_finite_values():
    x = Case([0], T=8, Hq=1, Hkv=1, D=64, io="f32", kv="e4m3")
    k = np.ones((1, 8, 1, 64), np.float32)
    k[0, 0] = 0.0
    k[0, 1, 0, 5] = np.inf
    k[0, 2, 0, 6] = np.nan
    k[0, 3] = 3e38
    k[0, 4] = 1e-40                                        # below the scale's floor
    k[0, 5] = np.linspace(-1, 1, 64)
    k[0, 6] = 448.0 * 2.0 ** -120
    k[0, 7] = -np.float32(2) ** np.arange(-32, 32)
    binding.kv_page_append(x.cfg, x.kv, x.dev(k), x.dev(-k), x.ws)
    codes, scale = ref.quantise(k[0, :, 0])
    for pool, s, sign in zip(x.pools, x.scales, (1, -1)):
        p = x.table[0][0]
        np.testing.assert_array_equal(pool[p, 0, :8].double().cpu().numpy(), sign * codes)
        np.testing.assert_array_equal(s[p, 0, :8].cpu().numpy(), scale)
    assert np.isnan(scale[1]) and np.isnan(scale[2]) and scale[0] == 1


def test_append_refuses_what_does_not_fit():
    x = Case([30, 29, 5, 5], T=3, Hq=1, Hkv=1, D=64, page=16, kv="e4m3", max_pages=2)
    x.table[2, 0] = -1
    x.table[3, 0] = x.cfg.n_pages
    x.kv.page_table.copy_(torch.from_numpy(x.table))
    before = x.pools[0].view(torch.uint8).clone()
    k = x.dev(np.ones((4, 3, 1, 64), np.float32))
    binding.kv_page_append(x.cfg, x.kv, k, k, x.ws)
    got = x.pools[0].view(torch.uint8)
    changed = (got != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [int(x.table[1][1])]
    assert x.status() == binding.SPEC_DEV_OVERFLOW | binding.SPEC_DEV_BADPAGE
    binding.spec_status_clear(x.ws)
    n = torch.tensor([-1, 4, 0, 0], dtype=torch.int32, device="cuda")
    binding.kv_page_append(x.cfg, x.kv, k, k, x.ws, n_new=n)
    assert x.status() == binding.SPEC_DEV_BADREQ


def test_read_leaves_other_rows_and_reports_what_is_missing():
    x = Case([20, 33, 40], T=1, Hq=1, Hkv=1, D=64, page=16, kv="e4m3")
    x.table[0, 1] = 10 ** 6
    x.kv.page_table.copy_(torch.from_numpy(x.table))
    out = [torch.full((3, 34, 1, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    binding.kv_page_read(x.cfg, x.kv, *out, x.ws)          # request 2 has more than 34 rows
    assert x.status() == binding.SPEC_DEV_OVERFLOW | binding.SPEC_DEV_BADPAGE
    k = out[0].float().cpu().numpy()
    assert (k[0, 16:] == 9).all() and (k[1, 33:] == 9).all() and (k[2] != 9).all()
    assert np.isfinite(k).all()


# ---------------------------------------------------------------------- attention

LENS = [0, 1, 14, 15, 16, 17, 63, 64, 127, 300]


@pytest.mark.parametrize("io,kv", [("bf16", "e4m3"), ("f32", "e4m3"), ("bf16", "io"), ("f32", "io")])
@pytest.mark.parametrize("D,Hq,Hkv,page", [(64, 4, 4, 16), (128, 8, 2, 64), (128, 24, 3, 32),
                                           (64, 48, 3, 128), (128, 7, 1, 16)])
def test_one_token(io, kv, D, Hq, Hkv, page):
    x = Case(LENS, Hq=Hq, Hkv=Hkv, D=D, page=page, io=io, kv=kv, seed=Hq)
    x.check(x.attend())
    assert x.status() == 0


@pytest.mark.parametrize("io,kv", [("bf16", "e4m3"), ("f32", "e4m3"), ("bf16", "io"), ("f32", "io")])
@pytest.mark.parametrize("T,Hq,Hkv,D,page", [(2, 4, 2, 64, 16), (5, 8, 2, 128, 32), (8, 8, 2, 128, 64),
                                             (9, 8, 1, 64, 16), (33, 6, 2, 64, 16)])
def test_several_tokens(io, kv, T, Hq, Hkv, D, page):
    lens = [0, 3, 60, 129, 250]
    x = Case(lens, T=T, Hq=Hq, Hkv=Hkv, D=D, page=page, io=io, kv=kv, seed=T,
             n_new=[T, 1, 0, max(1, T - 1), T])
    x.check(x.attend())
    assert x.status() == 0


@pytest.mark.parametrize("io,kv", [("bf16", "e4m3"), ("bf16", "io"), ("f32", "io")])
def test_long_caches_are_split_and_joined(io, kv):
    x = Case([9000, 2, 4097], Hq=8, Hkv=2, D=128, page=64, io=io, kv=kv, seed=5)
    x.check(x.attend())
    again = x.attend()
    assert torch.equal(again, x.attend())                  # the same every time
    assert x.status() == 0


@pytest.mark.parametrize("kv", ["e4m3", "io"])
def test_one_long_request(kv):
    x = Case([20000], T=2, Hq=4, Hkv=1, D=128, page=256, kv=kv, seed=6)
    x.check(x.attend())


@pytest.mark.parametrize("B", [33, 300, 600])
@pytest.mark.parametrize("kv", ["e4m3", "io"])
def test_many_requests(B, kv):
    """Beyond 32 requests the block finds its share (several lengths per thread
    beyond its threads); some requests have no new row."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 90, B).tolist()
    lens[B // 2] = 700
    x = Case(lens, T=2, Hq=4, Hkv=2, D=64, page=16, kv=kv, seed=B, max_pages=45,
             n_new=rng.integers(0, 3, B).tolist())
    x.check(x.attend())
    assert x.status() == 0


@pytest.mark.parametrize("io,kv,T,Hq,Hkv,D", [("bf16", "e4m3", 12, 8, 2, 128), ("bf16", "io", 8, 16, 4, 64),
                                              ("f32", "io", 9, 8, 2, 64), ("bf16", "e4m3", 30, 8, 2, 64)])
@pytest.mark.parametrize("B", [2, 12, 40])
def test_requests_with_few_and_many_new_tokens(io, kv, T, Hq, Hkv, D, B):
    """Row tiles without rows leave their warps to the others; requests are
    dealt out by what they cost, in CTAs of their own, evenly cut, and beyond 32."""
    rng = np.random.default_rng(B + T)
    lens = rng.integers(0, 2500 if B < 40 else 500, B).tolist()
    n = [T, 1] + rng.integers(0, T + 1, B - 2).tolist()
    x = Case(lens, T=T, Hq=Hq, Hkv=Hkv, D=D, page=32, io=io, kv=kv, seed=B, n_new=n)
    x.check(x.attend())
    assert x.status() == 0


def test_the_most_new_tokens_and_the_largest_pages():
    x = Case([900, 3], T=128, Hq=6, Hkv=2, D=64, page=1024, kv="e4m3", seed=63, n_new=[128, 100])
    x.check(x.attend())
    x = Case([5, 1023, 1024, 2000], T=1, Hq=16, Hkv=1, D=128, page=1024, kv="io", seed=64)
    x.check(x.attend())


def test_two_calls_at_once_on_two_streams():
    """Each with its own workspace; the results are those of one after the other."""
    xs = [Case([3000, 50], T=1, Hq=8, Hkv=8, D=128, page=64, kv="e4m3", seed=70 + i) for i in range(2)]
    want = [x.attend() for x in xs]
    qs, ns = [x.dev(x.q) for x in xs], [x.n_dev() for x in xs]
    outs = [torch.zeros_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, q, n, o, st in zip(xs, qs, ns, outs, streams):
            binding.attn_decode_paged(x.cfg, x.kv, q, o, x.ws, n_new=n, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("io,kv,D", [("bf16", "e4m3", 128), ("bf16", "io", 64), ("bf16", "io", 128),
                                     ("f32", "io", 64)])
def test_many_granules_per_cta(io, kv, D):
    """Long enough that each CTA goes around its ring of copies many times."""
    x = Case([33000, 9001, 16000], T=1, Hq=8, Hkv=8, D=D, page=64, io=io, kv=kv, seed=61)
    x.check(x.attend())
    x = Case([9001, 6000], T=6, Hq=24, Hkv=8, D=D, page=16, io=io, kv=kv, seed=62)
    x.check(x.attend())
    assert x.status() == 0


def test_scales_of_very_different_rows():
    """Weights and scales far apart: a large key scale, tiny and huge values."""
    x = Case([500, 700], Hq=8, Hkv=2, D=128, page=32, kv="e4m3", seed=7, spread=4.0)
    x.check(x.attend())
    x = Case([500, 700], Hq=8, Hkv=2, D=128, page=32, kv="io", seed=7, spread=4.0)
    x.check(x.attend())


@pytest.mark.parametrize("io,kv", [("bf16", "e4m3"), ("bf16", "io"), ("f32", "e4m3"), ("f32", "io")])
def test_draft_rows_that_are_not_finite_stay_with_later_tokens(io, kv):
    """The third new token's key and value are not finite: the rows before it
    do not see it, the rows from it on are not finite."""
    x = Case([40, 130], T=4, Hq=4, Hkv=2, D=64, page=16, io=io, kv=kv, seed=8)
    for b, L in enumerate(x.lens):
        for n in ("k", "v"):
            x.vals[n][b, L + 2] = np.nan
            if kv == "e4m3":
                x.scale[n][b, L + 2] = np.nan
    x.upload()
    o = x.attend()
    got = o.float().cpu().numpy()
    assert np.isfinite(got[:, :2]).all() and not np.isfinite(got[:, 2:]).any()
    assert x.status() == binding.SPEC_DEV_RANGE
    x.n = [2, 2]
    x.check(x.attend())


@pytest.mark.parametrize("kv", ["e4m3", "io"])
def test_values_of_infinity_reach_only_rows_that_see_them(kv):
    x = Case([20], T=3, Hq=2, Hkv=1, D=64, page=16, kv=kv, io="f32", seed=9)
    if kv == "io":
        x.vals["v"][0, 21] = np.inf
    else:
        x.scale["v"][0, 21] = np.inf
    x.upload()
    got = x.attend().cpu().numpy()
    assert np.isfinite(got[0, 0]).all() and not np.isfinite(got[0, 1:]).any()


def test_pages_outside_the_pool_are_not_seen():
    x = Case([100, 5, 40], Hq=4, Hkv=2, D=128, page=16, kv="e4m3", seed=10)
    x.table[0, 2] = -1
    x.table[0, 6] = x.cfg.n_pages + 5
    x.table[1, 0] = -7                                     # everything of request 1
    x.upload()
    o = x.attend()
    x.check(o, hide={(0, 2), (0, 6), (1, 0)})
    assert (o[1] == 0).all()
    assert x.status() == binding.SPEC_DEV_BADPAGE


def test_lengths_outside_the_table_are_clamped():
    x = Case([31, 20], T=1, Hq=2, Hkv=2, D=64, page=16, kv="io", max_pages=2, seed=11)
    x.check(x.attend())                                    # up to the last row
    x.kv.kv_len.copy_(torch.tensor([10 ** 9, -3], dtype=torch.int32))
    x.lens = [31, 0]                                       # all 32 rows; the first row
    x.check(x.attend())
    assert x.status() == binding.SPEC_DEV_OVERFLOW


def test_shared_pages():
    """Two requests with the same prefix pages and one of their own."""
    x = Case([40, 40], Hq=4, Hkv=2, D=64, page=16, kv="e4m3", seed=12)
    x.table[1, :2] = x.table[0, :2]
    for n in ("k", "v"):
        x.vals[n][1, :32] = x.vals[n][0, :32]
        x.scale[n][1, :32] = x.scale[n][0, :32]
    x.upload()
    x.check(x.attend())


def test_another_stream_and_a_captured_graph():
    x = Case([700, 33], T=2, Hq=8, Hkv=2, D=128, page=64, kv="e4m3", seed=13)
    want = x.attend()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o = torch.zeros_like(want)
    q, n = x.dev(x.q), x.n_dev()
    torch.cuda.synchronize()
    binding.attn_decode_paged(x.cfg, x.kv, q, o, x.ws, n_new=n, stream=st)
    st.synchronize()
    assert torch.equal(o, want)
    g = torch.cuda.CUDAGraph()
    o.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        binding.attn_decode_paged(x.cfg, x.kv, q, o, x.ws, n_new=n)
        binding.attn_decode_paged(x.cfg, x.kv, q, o, x.ws, n_new=n)
    for _ in range(3):
        o.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    x.lens = [690, 20]                                     # a replay reads the lengths anew
    x.kv.kv_len.copy_(torch.tensor(x.lens, dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    x.check(o)


@pytest.mark.parametrize("before", ["nothing", "copy", "fill", "kernel", "join"])
def test_each_call_waits_for_what_comes_before(before):
    """The launches may start before the one ahead of them ends: a chain of append,
    attention and read-back follows copies, fills, kernels and other streams, in a
    graph and out of it, and sees their results."""
    x = Case([300, 70], T=2, Hq=8, Hkv=2, D=128, page=16, kv="e4m3", seed=31)
    want = x.attend()
    new = {n: torch.stack([torch.from_numpy(x.raw[n][b, L:L + 2]) for b, L in enumerate(x.lens)])
           .to(torch.bfloat16).cuda() for n in ("k", "v")}
    Lmax = 302
    q, ns = x.dev(x.q), x.n_dev()
    k, v, o = torch.zeros_like(new["k"]), torch.zeros_like(new["v"]), torch.zeros_like(want)
    out = [torch.zeros((2, Lmax, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kept = [torch.zeros_like(out[0]) for _ in range(2)]
    side = torch.cuda.Stream()

    def chain():
        cur = torch.cuda.current_stream()
        if before == "copy":
            k.copy_(new["k"]), v.copy_(new["v"])
        elif before == "fill":
            k.copy_(new["k"]), v.copy_(new["v"]), o.zero_()
        elif before == "kernel":
            torch.mul(new["k"], 1, out=k), torch.mul(new["v"], 1, out=v)
        elif before == "join":
            side.wait_stream(cur)
            with torch.cuda.stream(side):
                k.copy_(new["k"])
            v.copy_(new["v"])
            cur.wait_stream(side)
        src = (new["k"], new["v"]) if before == "nothing" else (k, v)
        binding.kv_page_append(x.cfg, x.kv, *src, x.ws, n_new=ns)
        binding.attn_decode_paged(x.cfg, x.kv, q, o, x.ws, n_new=ns)
        binding.kv_page_read(x.cfg, x.kv, *out, x.ws)
        kept[0].copy_(out[0]), kept[1].copy_(out[1])

    def spoil():
        for t in (k, v, o, *out, *kept):
            t.zero_()
        for b, L in enumerate(x.lens):                     # the rows that append writes
            for r in (L, L + 1):
                pg = int(x.table[b][r // 16])
                for pool in x.pools:
                    pool.view(torch.uint8)[pg, :, r % 16] = 0x7f
        torch.cuda.synchronize()

    chain()
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    read = [t.clone() for t in kept]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
        chain()
    for _ in range(5):
        spoil()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and all(torch.equal(a, b) for a, b in zip(kept, read))
        spoil()
        chain()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and all(torch.equal(a, b) for a, b in zip(kept, read))
    assert x.status() == 0


def test_a_pool_beyond_32_bit_offsets():
    page, Hkv, D = 64, 8, 128
    n_pages = (1 << 32) // (page * Hkv * D) + 8            # more than 2^32 codes a pool
    cfg = binding.paged_cfg(B=1, T=1, Hq=8, Hkv=Hkv, D=D, page=page, n_pages=n_pages, max_pages=2,
                            kv="e4m3")
    pools = [torch.empty((n_pages, Hkv, page, D), dtype=torch.float8_e4m3fn, device="cuda")
             for _ in range(2)]
    scales = [torch.empty((n_pages, Hkv, page), device="cuda") for _ in range(2)]
    table = torch.tensor([[n_pages - 1, n_pages - 3]], dtype=torch.int32, device="cuda")
    kv = binding.PagedKV(cfg, *pools, table, torch.zeros(1, dtype=torch.int32, device="cuda"), *scales)
    ws = binding.alloc_paged_workspace(cfg)
    rng = np.random.default_rng(3)
    new = ref.bf16(rng.standard_normal((2, 80, Hkv, D)).astype(np.float32))
    one = binding.paged_cfg(B=1, T=80, Hq=8, Hkv=Hkv, D=D, page=page, n_pages=n_pages, max_pages=2,
                            kv="e4m3")
    dev = [torch.from_numpy(x[None]).bfloat16().cuda() for x in new]
    binding.kv_page_append(one, kv, *dev, ws)
    kv.kv_len.fill_(80)
    out = [torch.zeros((1, 80, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    binding.kv_page_read(cfg, kv, *out, ws)
    for x, o in zip(new, out):
        v, s = ref.quantise(x)
        np.testing.assert_array_equal(o[0].float().cpu().numpy(),
                                      ref.bf16(v.astype(np.float32) * s[..., None]))
    kv.kv_len.fill_(79)
    q = ref.bf16(rng.standard_normal((8, D)).astype(np.float32))
    o = torch.zeros((1, 1, 8, D), dtype=torch.bfloat16, device="cuda")
    binding.attn_decode_paged(cfg, kv, torch.from_numpy(q[None, None]).bfloat16().cuda(), o, ws)
    got = o[0, 0].double().cpu().numpy()
    for h in range(8):
        k, v = (ref.quantise(x[:, h]) for x in new)
        want, A, z = ref.attention(q[h:h + 1].astype(np.float64), k[0] * k[1][:, None],
                                   v[0] * v[1][:, None], np.ones((1, 80), bool))
        d = (32 * 2.0 ** -23 + 2 * 2.0 ** -21) * z[0] + 2.0 ** -20
        assert (np.abs(got[h] - want[0]) <= 2.0 ** -8 * np.abs(want[0])
                + (2.0 ** -11 + 2 * d + 80 * 2.0 ** -23) * A[0]).all()
    assert binding.spec_status_read(ws) == 0


# ---------------------------------------------------------------------- refusals

def test_refusals():
    x = Case([5], T=1, Hq=4, Hkv=2, D=64, kv="e4m3")
    c, q = x.cfg, x.dev(x.q)
    o = torch.empty_like(q)
    for bad, exc in ((q.float(), TypeError), (q[:, :, :2], ValueError), (q.cpu(), TypeError),
                     (q.transpose(2, 3).contiguous().transpose(2, 3), ValueError)):
        with pytest.raises(exc):
            binding.attn_decode_paged(c, x.kv, bad, o, x.ws)
    with pytest.raises(ValueError):
        binding.attn_decode_paged(c, x.kv, q, o, x.ws[:128])
    other = binding.paged_cfg(B=1, T=1, Hq=4, Hkv=2, D=64, page=32, n_pages=c.n_pages,
                              max_pages=c.max_pages, kv="e4m3")
    with pytest.raises(ValueError):
        binding.attn_decode_paged(other, x.kv, q, o, x.ws)
    with pytest.raises(TypeError):
        binding.PagedKV(c, x.pools[0].float(), x.pools[1], x.kv.page_table, x.kv.kv_len, *x.scales)
    with pytest.raises(TypeError):
        binding.PagedKV(c, *x.pools, x.kv.page_table, x.kv.kv_len)
    with pytest.raises(binding.SpecError):                 # a 4-byte aligned view
        big = torch.zeros(q.numel() + 2, dtype=q.dtype, device="cuda")
        binding.attn_decode_paged(c, x.kv, big[2:].view(q.shape), o, x.ws)
    k = torch.zeros((1, 129, 4, 64), dtype=torch.bfloat16, device="cuda")
    long = binding.paged_cfg(B=1, T=129, Hq=4, Hkv=2, D=64, page=16, n_pages=c.n_pages,
                             max_pages=c.max_pages, kv="e4m3")
    with pytest.raises(binding.SpecError):
        binding.attn_decode_paged(long, x.kv, k, torch.empty_like(k), x.ws)
    assert x.status() == 0
