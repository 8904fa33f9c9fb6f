"""Rotary positions against the rotation in 64 bits, and the pass that writes the
cache against the separate calls.

Tolerance.  The angle is off by at most 2^-32 turns (1.5e-9) and by the roundings of
its rest in [-pi/4, pi/4], half a step of a number below 1 each (2^-25); the Taylor
sums by 1.8e-9 and some roundings of 2^-25: sine and cosine are within 2^-23.  A value is two products and a sum of them in fp32: within
(|a| + |b|) amp (2^-23 + 2 * 2^-24) < (|a| + |b|) amp 2^-22, then half a step of the
I/O type.  Positions above 2^20 add the 64-bit product's own 2^-53 p."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_best_gb300 import binding
from tests import indep_serving as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_tree_best_gb300 import build
    build.build()
    binding.load()


def randn(shape, io, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(DT[io])


def near(got, x, pos, f, amp, layout, io, inverse=False):
    x64 = x.double().cpu().numpy()
    want = ref.rotate(x64, pos, f, amp, layout, inverse)
    size = ref.rotate(np.abs(x64), np.zeros(len(pos)), f, 1.0, layout)
    rot, half = 2 * len(f), len(f)
    both = size.copy()                                    # |a| + |b| of the pair
    if layout == "half":
        both[..., :half] = both[..., half:rot] = size[..., :half] + size[..., half:rot]
    else:
        both[..., 0:rot:2] = both[..., 1:rot:2] = size[..., 0:rot:2] + size[..., 1:rot:2]
    both[..., rot:] = 0
    far = np.maximum(np.abs(np.asarray(pos, np.float64)) * 2.0 ** -52, 0)[:, None, None]
    tol = both * amp * (2.0 ** -22 + far) + np.abs(want) * (torch.finfo(DT[io]).eps / 2) * (io == "bf16")
    off = np.abs(got.double().cpu().numpy() - want)
    assert (off <= tol + 1e-38).all(), float((off / (tol + 1e-30)).max())
    np.testing.assert_array_equal(got[..., rot:].double().cpu().numpy(), x64[..., rot:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rows,Hq,Hkv,D,rot,scaling", [
    (1, 1, 1, 64, 16, {}), (1, 32, 8, 128, 128, {}), (25, 32, 8, 128, 128, {}),
    (7, 3, 1, 64, 64, dict(scaling="linear", factor=4.0)),
    (257, 5, 5, 128, 48, dict(scaling="ntk", factor=8.0)),
    (1030, 8, 2, 64, 32, dict(scaling="yarn", factor=4.0, orig_len=4096)),
    (3001, 7, 1, 128, 112, dict(scaling="yarn", factor=16.0, orig_len=300, beta_fast=8.0,
                                beta_slow=0.5)),
    (9, 200, 100, 64, 64, {}), (33, 2, 0, 128, 128, {})])
def test_rows(io, layout, rows, Hq, Hkv, D, rot, scaling):
    table = binding.rope_table(rot, base=1e6, **scaling)
    f, amp = ref.frequencies(rot, 1e6, **scaling)
    g = np.random.default_rng(rows)
    pos = np.exp(g.uniform(0, np.log(1e6), rows)).astype(np.int32)
    pos[0] = 0
    q = randn((rows, Hq, D), io, 1)
    k = randn((rows, Hkv, D), io, 2) if Hkv else None
    for inverse in (False, True):
        cfg = binding.rope_cfg(rows, Hq, Hkv, D, rot, layout, io, inverse)
        qo, ko = torch.empty_like(q), None if k is None else torch.empty_like(k)
        binding.rope_apply(cfg, table, torch.from_numpy(pos).cuda(), q, k, qo, ko)
        near(qo, q, pos, f, amp, layout, io, inverse)
        if Hkv:
            near(ko, k, pos, f, amp, layout, io, inverse)


def test_far_and_negative_positions():
    pos = np.array([2 ** 31 - 1, -2 ** 31, -1, 1, 2 ** 30 + 1, -(2 ** 24) - 3, 0], np.int32)
    q = randn((7, 2, 128), "f32", 3)
    cfg = binding.rope_cfg(7, 2, 0, 128, io="f32")
    out = torch.empty_like(q)
    binding.rope_apply(cfg, binding.rope_table(128, base=1e4), torch.from_numpy(pos).cuda(), q,
                       None, out, None)
    f, amp = ref.frequencies(128, 1e4)
    near(out, q, pos, f, amp, "half", "f32")


def test_in_place_slices_and_streams():
    rows, Hq, Hkv, D = 300, 6, 2, 64
    wide = randn((rows, (Hq + 2 * Hkv) * D + 16), "bf16", 4)
    q = wide[:, :Hq * D].unflatten(1, (Hq, D))
    k = wide[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") * 7
    table = binding.rope_table(D)
    a, b = q.contiguous(), k.contiguous()
    binding.rope_apply(binding.rope_cfg(rows, Hq, Hkv, D), table, pos, a, b, a, b)     # in place
    st = wide.stride(0)
    cfg = binding.rope_cfg(rows, Hq, Hkv, D, q_stride=st, k_stride=st)
    qo, ko = torch.empty_like(a), torch.empty_like(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    binding.rope_apply(cfg, table, pos, q, k, qo, ko, stream=side)
    side.synchronize()
    assert torch.equal(a, qo) and torch.equal(b, ko)
    near(qo, q, pos.cpu().numpy(), *ref.frequencies(D, 1e4), "half", "bf16")
    with pytest.raises(ValueError, match="strides"):
        binding.rope_apply(cfg, table, pos, a, k, qo, ko)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_the_inverse_is_the_gradient(layout):
    """sum(rope(x) g) has the gradient inverse(g): compared with differences in 64
    bits, and there and back gives x."""
    rows, H, D, rot = 11, 3, 64, 48
    table = binding.rope_table(rot, scaling="yarn", factor=4.0, orig_len=64)
    f, amp = ref.frequencies(rot, 1e4, "yarn", 4.0, 64)
    pos = np.arange(rows, dtype=np.int32) * 31
    x, g = randn((rows, H, D), "f32", 5), randn((rows, H, D), "f32", 6)
    grad = torch.empty_like(x)
    cfg = binding.rope_cfg(rows, H, 0, D, rot, layout, "f32", inverse=True)
    binding.rope_apply(cfg, table, torch.from_numpy(pos).cuda(), g, None, grad, None)
    x64, g64, rng = x.double().cpu().numpy(), g.double().cpu().numpy(), np.random.default_rng(0)
    for _ in range(20):
        d = rng.standard_normal(x64.shape)
        up, down = (float((ref.rotate(x64 + s * d, pos, f, amp, layout) * g64).sum())
                    for s in (0.5, -0.5))                  # linear: any step is exact
        assert abs(float((grad.double().cpu().numpy() * d).sum()) - (up - down)) < 1e-3
    y, back = torch.empty_like(x), torch.empty_like(x)
    binding.rope_apply(binding.rope_cfg(rows, H, 0, D, rot, layout, "f32"), table,
                       torch.from_numpy(pos).cuda(), x, None, y, None)
    binding.rope_apply(cfg, table, torch.from_numpy(pos).cuda(), y, None, back, None)
    # amp on the way there and back; two rotations, each within 2^-22 of |a| + |b|
    want = x.clone()
    want[..., :rot] *= amp * amp
    assert float((back - want).abs().max()) < 8 * 2 ** -22 * float(x.abs().max()) * amp * amp


def cache(cfg, seed=0):
    kv = binding.PagedKV.empty(cfg)
    for t in (kv.k_pages, kv.v_pages):
        t.view(torch.uint8).fill_(0x2b)                    # rows that nobody writes stay so
    return kv


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("io,kv", [("bf16", "io"), ("bf16", "e4m3"), ("f32", "io"), ("f32", "e4m3")])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot,page", [
    (1, 1, 4, 4, 64, 64, 16), (24, 1, 32, 8, 128, 128, 64), (3, 37, 6, 2, 128, 64, 16),
    (2, 700, 5, 5, 64, 48, 128), (5, 9, 8, 1, 128, 112, 1024)])
@pytest.mark.parametrize("fused", [False, True])
def test_append(io, kv, layout, B, T, Hq, Hkv, D, rot, page, fused):
    cols = (T + 130) // page + 2
    pcfg = binding.paged_cfg(B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, page=page, n_pages=B * cols + 3,
                             max_pages=cols, io=io, kv=kv)
    c = cache(pcfg)
    pool, ws = (binding.PagePool.empty(pcfg, c.page_table, c.kv_len),
                binding.alloc_paged_workspace(pcfg))
    g = np.random.default_rng(B * T)
    slots = torch.empty((B, T), dtype=torch.int64, device="cuda")
    n_ok = torch.empty((B,), dtype=torch.int32, device="cuda")
    L = g.integers(0, 100, B).astype(np.int32)
    c.kv_len.copy_(torch.from_numpy(L))
    n = g.integers(0, T + 1, B).astype(np.int32)
    n[0] = T
    binding.page_tables_extend(pcfg, pool, slots, n_ok, ws, n_new=torch.from_numpy(n).cuda())
    wide = randn((B, T, (Hq + 2 * Hkv) * D), io, 7)
    q, k, v = (x.unflatten(2, (-1, D)) for x in wide.split([Hq * D, Hkv * D, Hkv * D], 2))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    st = (Hq + 2 * Hkv) * D if fused else 0
    cfg = binding.rope_cfg(B * T, Hq, Hkv, D, rot, layout, io, q_stride=st, k_stride=st, v_stride=st)
    table = binding.rope_table(rot, base=1e6)
    q_out = torch.full((B, T, Hq, D), 3.0, dtype=DT[io], device="cuda")
    binding.rope_page_append(cfg, pcfg, c, table, slots, q, k, v, q_out, ws)
    assert binding.spec_status_read(ws) == 0
    # the separate calls
    pos = (c.kv_len.view(B, 1) + torch.arange(T, device="cuda", dtype=torch.int32)).to(torch.int32)
    one = binding.rope_cfg(B * T, Hq, Hkv, D, rot, layout, io)
    qr, kr = torch.empty((B * T, Hq, D), dtype=DT[io], device="cuda"), torch.empty(
        (B * T, Hkv, D), dtype=DT[io], device="cuda")
    binding.rope_apply(one, table, pos.reshape(-1), q.reshape(B * T, Hq, D).contiguous(),
                       k.reshape(B * T, Hkv, D).contiguous(), qr, kr)
    real = (slots >= 0).view(B, T, 1, 1)
    assert int(real.sum()) == int(n.sum())
    assert torch.equal(q_out, torch.where(real, qr.view(B, T, Hq, D), torch.full_like(q_out, 3.0)))
    d = cache(pcfg)
    d.page_table.copy_(c.page_table)
    d.kv_len.copy_(c.kv_len)
    binding.kv_page_append(pcfg, d, kr.view(B, T, Hkv, D), v.contiguous(), ws,
                           n_new=torch.from_numpy(n).cuda())
    assert torch.equal(c.v_pages.view(torch.uint8), d.v_pages.view(torch.uint8))
    if kv == "io" or io == "f32":
        assert torch.equal(c.k_pages.view(torch.uint8), d.k_pages.view(torch.uint8))
    if kv == "e4m3":
        assert torch.equal(c.v_scale, d.v_scale)
    if kv == "e4m3" and io == "bf16":
        # from the rotated fp32 values: half a step of e4m3 (2^-4, 2^-10 scale below its
        # normal range), the scale's rounding, the rotation's own
        f, amp = ref.frequencies(rot, 1e6)
        x = k.reshape(B * T, Hkv, D).double().cpu().numpy()
        want = ref.rotate(x, pos.reshape(-1).cpu().numpy(), f, amp, layout)
        flat = real.view(-1).cpu().numpy()
        s = slots.view(-1)[real.view(-1)]
        p, at = s // page, s % page
        scale = c.k_scale[p, :, at].double().cpu().numpy()
        most = np.abs(want[flat]).max(-1) / 448
        np.testing.assert_allclose(scale, most, rtol=2.0 ** -20)
        got = c.k_pages[p, :, at].double().cpu().numpy() * scale[..., None]
        off = np.abs(got - want[flat])
        assert (off <= np.abs(want[flat]) * 2.0 ** -4 * (1 + 2.0 ** -10)
                + scale[..., None] * (2.0 ** -10 + 2.0 ** -10)).all()


def test_append_rows_that_are_not_finite_zeros_and_bad_slots():
    pcfg = binding.paged_cfg(B=1, T=5, Hq=1, Hkv=1, D=64, page=16, n_pages=2, max_pages=2,
                             kv="e4m3")
    c, ws = cache(pcfg), binding.alloc_paged_workspace(pcfg)
    q, k, v = (randn((1, 5, 1, 64), "bf16", s) for s in (1, 2, 3))
    k[0, 0] = 0.0
    k[0, 1, 0, 3] = float("inf")
    v[0, 2, 0, 63] = float("nan")
    slots = torch.tensor([[0, 1, 2, 32, 2 ** 40]], device="cuda")     # a pool of 32 slots
    q_out = torch.zeros_like(q)
    binding.rope_page_append(binding.rope_cfg(5, 1, 1, 64), pcfg, c, binding.rope_table(64), slots,
                             q, k, v, q_out, ws)
    assert binding.spec_status_read(ws) == binding.SPEC_DEV_BADPAGE
    sk, sv = c.k_scale[0, 0].cpu(), c.v_scale[0, 0].cpu()
    assert sk[0] == 1.0 and sk[1].isnan() and not sk[2].isnan() and sv[2].isnan()
    assert (c.k_pages[0, 0, 0].float() == 0).all() and c.v_pages[0, 0, 2].float().isnan().all()
    assert (c.k_pages.view(torch.uint8)[0, 0, 3:] == 0x2b).all()
    assert (c.k_pages.view(torch.uint8)[1] == 0x2b).all() and (q_out[0, 3:] != 0).any()


def test_captured_steps_follow_their_inputs():
    """rope_page_append in a graph: replays read the lengths, slots and rows of their time."""
    B, T, Hq, Hkv, D = 3, 2, 4, 2, 64
    pcfg = binding.paged_cfg(B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, page=16, n_pages=12, max_pages=4)
    c, d, ws = cache(pcfg), cache(pcfg), binding.alloc_paged_workspace(pcfg)
    rc, table = binding.rope_cfg(B * T, Hq, Hkv, D), binding.rope_table(D)
    q, k, v = (randn((B, T, h, D), "bf16", s) for s, h in ((1, Hq), (2, Hkv), (3, Hkv)))
    slots = torch.arange(B * T, device="cuda").view(B, T) * 17
    q_out, now = torch.zeros_like(q), torch.zeros_like(q)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            binding.rope_page_append(rc, pcfg, c, table, slots, q, k, v, q_out, ws)
    for step in range(3):
        for kv in (c, d):
            kv.kv_len.copy_(torch.tensor([5, 0, 40], dtype=torch.int32) + step)
        slots.add_(1)
        k.copy_(randn((B, T, Hkv, D), "bf16", 10 + step))
        graph.replay()
        binding.rope_page_append(rc, pcfg, d, table, slots, q, k, v, now, ws)
        assert torch.equal(q_out, now)
        for a, b in ((c.k_pages, d.k_pages), (c.v_pages, d.v_pages)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
