"""Page tables grown and trimmed on the device against a request-by-request
simulation: whole numbers, so everything compares exactly."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_best_gb300 import binding
from tests import indep_serving as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_best_gb300 import build
    build.build()
    binding.load()


def make(B, T, page, cols, n_pages, seed=0, full=0.5):
    """Requests that hold pages for lengths up to `full` of what a table or the pool can hold."""
    rng = np.random.default_rng(seed)
    most = max(0, int(min(cols, n_pages // B) * full) * page - 3)
    L = rng.integers(0, most + 1, B).astype(np.int32)
    held = -(-L // page).astype(np.int32)
    # some requests hold more than their rows need
    held = np.minimum(held + (rng.random(B) < 0.3), min(cols, n_pages // B)).astype(np.int32)
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((B, cols), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(n_pages, -7, np.int32)
    free[:n_pages - at] = ids[at:]
    return dict(page_table=table, kv_len=L, free_list=free,
                n_free=np.array([n_pages - at], np.int32), n_held=held)


def device(s, cfg):
    t = {n: torch.from_numpy(x.copy()).cuda() for n, x in s.items()}
    return binding.PagePool(cfg, t["page_table"], t["kv_len"], t["free_list"], t["n_free"],
                            t["n_held"])


def same(pool, s):
    for n, x in s.items():
        np.testing.assert_array_equal(getattr(pool, n).cpu().numpy(), x, err_msg=n)


def config(B, T, page, cols, n_pages):
    return binding.paged_cfg(B=B, T=T, Hq=1, Hkv=1, D=64, page=page, n_pages=n_pages,
                             max_pages=cols)


CASES = [(1, 1, 16, 1, 1), (1, 9, 64, 3, 7), (3, 5, 16, 4, 9), (256, 1, 64, 20, 4000),
         (700, 3, 16, 6, 3100), (4096, 1, 16, 3, 9000), (2, 20000, 16, 1300, 2700),
         (33, 1025, 32, 40, 700), (5, 4097, 1024, 6, 25)]


@pytest.mark.parametrize("B,T,page,cols,n_pages", CASES)
@pytest.mark.parametrize("ragged", [False, True])
def test_steps_of_growth_and_trim(B, T, page, cols, n_pages, ragged):
    cfg = config(B, T, page, cols, n_pages)
    s = make(B, T, page, cols, n_pages, seed=B + T)
    pool, ws = device(s, cfg), binding.alloc_paged_workspace(cfg)
    slots = torch.empty((B, T), dtype=torch.int64, device="cuda")
    n_ok = torch.empty((B,), dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(1)
    for step in range(3):
        n = rng.integers(0, T + 1, B).astype(np.int32) if ragged else np.full(B, T, np.int32)
        want, ok = ref.extend(s, page, n, T)
        binding.page_tables_extend(cfg, pool, slots, n_ok, ws,
                                   n_new=torch.from_numpy(n).cuda() if ragged else None)
        same(pool, s)
        np.testing.assert_array_equal(n_ok.cpu().numpy(), ok)
        np.testing.assert_array_equal(slots.cpu().numpy(), want)
        # some rows stay: the caller advances kv_len, as the verification does
        s["kv_len"] += rng.integers(0, ok + 1).astype(np.int32)
        pool.kv_len.copy_(torch.from_numpy(s["kv_len"]))
        keep = np.where(rng.random(B) < 0.2, 0, np.where(rng.random(B) < 0.2, -1, s["kv_len"]))
        keep = np.where(rng.random(B) < 0.2, s["kv_len"] // 2, keep).astype(np.int32)
        ref.trim(s, page, keep)
        binding.page_tables_trim(cfg, pool, torch.from_numpy(keep).cuda(), ws)
        same(pool, s)
    allowed = binding.SPEC_DEV_NOPAGE | binding.SPEC_DEV_OVERFLOW
    assert binding.spec_status_read(ws) & ~allowed == 0
    assert int(ws[256:].count_nonzero()) == 0          # tickets are back at zero


def test_every_page_is_held_once():
    B, T, page, cols, n_pages = 64, 40, 16, 30, 500
    cfg = config(B, T, page, cols, n_pages)
    pool, ws = binding.PagePool.empty(cfg), binding.alloc_paged_workspace(cfg)
    slots = torch.empty((B, T), dtype=torch.int64, device="cuda")
    n_ok = torch.empty((B,), dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    for _ in range(20):
        binding.page_tables_extend(cfg, pool, slots, n_ok, ws)
        used = slots[slots >= 0]
        assert used.unique().numel() == used.numel()
        pool.kv_len.add_(n_ok)
        held = pool.page_table[pool.page_table >= 0]
        free = pool.free_list[:int(pool.n_free)]
        every = torch.cat([held, free]).sort().values
        assert torch.equal(every, torch.arange(n_pages, dtype=torch.int32, device="cuda"))
        ends = torch.rand((B,), generator=g, device="cuda") < 0.3
        binding.page_tables_trim(cfg, pool, torch.where(ends, 0, -1).to(torch.int32), ws)
    torch.cuda.synchronize()


def test_first_requests_get_the_last_pages():
    """Five pages are free and four requests lack 2, 2, 2, 1: the third's total
    exceeds the list, and so does every later one that lacks any."""
    cfg = config(5, 32, 16, 4, 5)
    pool, ws = binding.PagePool.empty(cfg), binding.alloc_paged_workspace(cfg)
    slots = torch.empty((5, 32), dtype=torch.int64, device="cuda")
    n_ok = torch.empty((5,), dtype=torch.int32, device="cuda")
    n = torch.tensor([32, 17, 20, 1, 0], dtype=torch.int32, device="cuda")
    binding.page_tables_extend(cfg, pool, slots, n_ok, ws, n_new=n)
    assert n_ok.tolist() == [32, 17, 0, 0, 0] and int(pool.n_free) == 1
    assert pool.n_held.tolist() == [2, 2, 0, 0, 0]
    assert pool.page_table[:2, :2].tolist() == [[0, 1], [2, 3]]
    assert binding.spec_status_read(ws) == binding.SPEC_DEV_NOPAGE


def test_bad_requests_get_nothing():
    cfg = config(6, 8, 16, 4, 40)
    pool, ws = binding.PagePool.empty(cfg), binding.alloc_paged_workspace(cfg)
    pool.kv_len.copy_(torch.tensor([-1, 57, 0, 0, 0, 2 ** 31 - 1]))
    pool.n_held.copy_(torch.tensor([0, 4, -1, 5, 0, 0]))
    slots = torch.empty((6, 8), dtype=torch.int64, device="cuda")
    n_ok = torch.empty((6,), dtype=torch.int32, device="cuda")
    n = torch.tensor([8, 8, 8, 8, 9, 8], dtype=torch.int32, device="cuda")
    binding.page_tables_extend(cfg, pool, slots, n_ok, ws, n_new=n)
    assert n_ok.tolist() == [0, 0, 0, 0, 8, 0]
    assert (slots[[0, 1, 2, 3, 5]] == -1).all() and slots[4].tolist() == list(range(8))
    assert int(pool.n_free) == 39
    assert binding.spec_status_read(ws) == binding.SPEC_DEV_OVERFLOW | binding.SPEC_DEV_BADREQ
    binding.spec_status_clear(ws)
    before = pool.page_table.clone()
    binding.page_tables_trim(cfg, pool, torch.tensor([0, -1, 0, 0, -2, -1], dtype=torch.int32,
                                                     device="cuda"), ws)
    assert torch.equal(pool.page_table, before) and int(pool.n_free) == 39
    assert pool.kv_len.tolist()[:1] == [-1]             # below what is kept already
    assert binding.spec_status_read(ws) == binding.SPEC_DEV_BADREQ


def test_pages_outside_the_pool_and_lists_out_of_range():
    cfg = config(2, 20, 16, 4, 8)
    pool, ws = binding.PagePool.empty(cfg), binding.alloc_paged_workspace(cfg)
    pool.page_table[0, 0] = 8
    pool.n_held[0] = 1
    pool.free_list[7] = -3
    pool.n_free[0] = 9                                   # clamped to 8
    slots = torch.empty((2, 20), dtype=torch.int64, device="cuda")
    n_ok = torch.empty((2,), dtype=torch.int32, device="cuda")
    binding.page_tables_extend(cfg, pool, slots, n_ok, ws)
    assert n_ok.tolist() == [20, 20] and int(pool.n_free) == 5
    assert (slots[0] == -1).all()                        # page 8, then page -3
    assert slots[1].tolist() == list(range(16, 36))
    assert binding.spec_status_read(ws) == binding.SPEC_DEV_BADREQ | binding.SPEC_DEV_BADPAGE
    # a list that is full takes no more
    binding.spec_status_clear(ws)
    pool.n_free[0] = 8
    binding.page_tables_trim(cfg, pool, torch.zeros((2,), dtype=torch.int32, device="cuda"), ws)
    assert int(pool.n_free) == 8 and (pool.page_table == -1).all()
    assert binding.spec_status_read(ws) == binding.SPEC_DEV_BADREQ


def test_kv_len_itself_as_what_is_kept_and_captured():
    B, T, page, cols = 40, 9, 16, 8
    cfg = config(B, T, page, cols, B * cols)
    s = make(B, T, page, cols, B * cols, seed=3)
    pool, ws = device(s, cfg), binding.alloc_paged_workspace(cfg)
    slots = torch.empty((B, T), dtype=torch.int64, device="cuda")
    n_ok = torch.empty((B,), dtype=torch.int32, device="cuda")

    def step():
        binding.page_tables_extend(cfg, pool, slots, n_ok, ws)
        binding.page_tables_trim(cfg, pool, pool.kv_len, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    for _ in range(3):
        graph.replay()
        want, ok = ref.extend(s, page, np.full(B, T), T)
        ref.trim(s, page, s["kv_len"].copy())
        torch.cuda.synchronize()
        same(pool, s)
        np.testing.assert_array_equal(slots.cpu().numpy(), want)


def test_pools_and_arguments_of_another_shape_are_refused():
    cfg = config(3, 4, 16, 5, 20)
    pool, ws = binding.PagePool.empty(cfg), binding.alloc_paged_workspace(cfg)
    slots = torch.empty((3, 4), dtype=torch.int64, device="cuda")
    n_ok = torch.empty((3,), dtype=torch.int32, device="cuda")
    for other in (config(2, 4, 16, 5, 20), config(3, 4, 16, 6, 20), config(3, 4, 16, 5, 21),
                  config(3, 4, 32, 5, 20)):
        with pytest.raises(ValueError):
            binding.page_tables_extend(other, pool, slots, n_ok, ws)
        with pytest.raises(ValueError):
            binding.page_tables_trim(other, pool, n_ok, ws)
    for bad in (slots[:, :3], slots.int(), slots.cpu(), None):
        with pytest.raises((TypeError, ValueError)):
            binding.page_tables_extend(cfg, pool, bad, n_ok, ws)
    with pytest.raises(ValueError):
        binding.page_tables_trim(cfg, pool, n_ok, ws[:256])
    with pytest.raises(TypeError):
        binding.PagePool(cfg, pool.page_table.long(), pool.kv_len, pool.free_list, pool.n_free,
                         pool.n_held)
