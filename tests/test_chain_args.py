"""Host-side checks of the paged-cache calls and the chain verification (no
kernel is launched), and the law of the plain verification they are held to."""
import ctypes
import os
import shutil

import numpy as np
import pytest

from speculative_decoding_tree_best_gb300 import binding
from tests import indep_chain as ref

P = ctypes.c_void_p(16)
GOOD = dict(B=2, T=3, Hq=8, Hkv=2, D=128, page=64, n_pages=10, max_pages=4)


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from speculative_decoding_tree_best_gb300 import build
    build.build()
    return binding.load()


def calls(lib, cfg, kv=None, n_new=None, x=P, ws=P, Lmax=8):
    kv = binding.SpecPagedKV(*([16] * 6)) if kv is None else kv
    c, k = ctypes.byref(cfg), ctypes.byref(kv)
    return (lib.kv_page_append(c, k, x, P, n_new, ws, None),
            lib.kv_page_read(c, k, Lmax, x, P, ws, None),
            lib.attn_decode_paged(c, k, x, n_new, P, ws, None))


@pytest.mark.parametrize("field,value", [
    ("B", 0), ("B", 4097), ("Hkv", 2048), ("T", 0), ("T", 1 << 21), ("Hq", 7), ("Hkv", 0), ("D", 96), ("D", 256),
    ("page", 8), ("page", 48), ("page", 2048), ("n_pages", 0), ("max_pages", 0),
    ("max_pages", 1 << 26), ("io_dtype", 5), ("kv_dtype", 2)])
def test_paged_shapes_are_refused(lib, field, value):
    cfg = binding.paged_cfg(**GOOD)
    setattr(cfg, field, value)
    want = binding.ST_EUNSUPPORTED if field.endswith("dtype") else binding.ST_EINVAL
    assert calls(lib, cfg) == (want,) * 3
    assert lib.spec_paged_workspace_bytes(ctypes.byref(cfg), 152) == 0


def test_paged_pointers_are_refused(lib):
    cfg = binding.paged_cfg(**GOOD, kv="e4m3")
    E = (binding.ST_EINVAL,) * 3
    assert calls(lib, cfg, x=None) == E and calls(lib, cfg, x=ctypes.c_void_p(24)) == E
    assert calls(lib, cfg, ws=None) == E
    for i in range(6):
        for bad in (0, 8):
            kv = binding.SpecPagedKV(*[bad if j == i else 16 for j in range(6)])
            assert calls(lib, cfg, kv=kv) == E
    assert calls(lib, cfg, Lmax=0)[1] == binding.ST_EINVAL
    n = calls(lib, cfg, n_new=ctypes.c_void_p(4))
    assert n[0] == n[2] == binding.ST_EINVAL
    kv = ctypes.byref(binding.SpecPagedKV(*([16] * 6)))
    for bad in (dict(T=129), dict(T=128, Hq=2048, Hkv=2),         # rows of a kv-head
                dict(B=4096, Hq=1024, Hkv=1024, max_pages=1 << 20)):   # granules in 32 bits
        long = binding.paged_cfg(**dict(GOOD, **bad))
        assert lib.attn_decode_paged(ctypes.byref(long), kv, P, None, P, P, None) == binding.ST_EINVAL


def test_workspace_sizes_are_host_only(lib):
    n = binding.spec_paged_workspace_bytes(binding.paged_cfg(**GOOD), 152)
    assert n >= 256 and n % 256 == 0
    m = binding.spec_draft_workspace_bytes(binding.draft_cfg(B=3, N=4, V=1000), 152)
    assert m >= 256 and m % 256 == 0
    assert lib.spec_paged_workspace_bytes(ctypes.byref(binding.paged_cfg(**GOOD)), -1) == 0
    assert lib.spec_draft_workspace_bytes(ctypes.byref(binding.draft_cfg(B=3, N=4, V=0)), 152) == 0


def draft(lib, cfg, toks=P, q=P, logits=P, u=P, e=P, out=(16, 16, 16), n=None, kv=None, ws=P):
    o = binding.SpecDraftOut(*out)
    return lib.draft_verify_sampled(ctypes.byref(cfg), toks, n, q, logits, u, e, ctypes.byref(o), kv,
                                    None, ws, None)


@pytest.mark.parametrize("field,value", [
    ("B", 0), ("B", 65536), ("N", -1), ("N", 128), ("V", 0), ("temperature", 0.0),
    ("temperature", -1.0), ("temperature", float("nan")), ("temperature", float("inf")),
    ("reserved", 1), ("io_dtype", 3)])
def test_chain_shapes_are_refused(lib, field, value):
    cfg = binding.draft_cfg(B=2, N=3, V=100)
    setattr(cfg, field, value)
    want = binding.ST_EUNSUPPORTED if field == "io_dtype" else binding.ST_EINVAL
    assert draft(lib, cfg) == want


def test_chain_pointers_are_refused(lib):
    cfg = binding.draft_cfg(B=2, N=3, V=100)
    odd = ctypes.c_void_p(20)
    for kw in (dict(toks=None), dict(logits=None), dict(u=None), dict(e=None), dict(ws=None),
               dict(q=odd), dict(n=odd), dict(kv=odd), dict(out=(0, 16, 16)), dict(out=(16, 4, 16)),
               dict(out=(16, 16, 0))):
        assert draft(lib, cfg, **kw) == binding.ST_EINVAL, kw


def test_cpu_tensors_are_refused():
    import torch
    with pytest.raises(TypeError):
        binding._arg(torch.zeros(2), torch.float32, (2,), "x", 0)
    with pytest.raises(TypeError):
        binding._arg([1.0, 2.0], torch.float32, (2,), "x", 0)
    with pytest.raises(TypeError):
        binding._required(None, "x")


# ---------------------------------------------------- the plain implementations

def test_rounding_to_e4m3():
    import torch
    x = np.concatenate([np.linspace(-448, 448, 20001), np.exp2(np.linspace(-12, 8.7, 3001)),
                        (np.arange(256) + 0.5) * 2.0 ** -10]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.e4m3(x), want)


def test_rounding_to_bf16():
    import torch
    x = np.random.default_rng(0).standard_normal(10000).astype(np.float32)
    np.testing.assert_array_equal(ref.bf16(x), torch.from_numpy(x).bfloat16().float().numpy())


def test_the_plain_chain_follows_the_target():
    """First and second tokens of 20000 chains of two drafts against p0 and
    p1 (chi-square over 5 tokens, 4 degrees: 99.9% is 18.5)."""
    rng = np.random.default_rng(1)
    V, n = 5, 20000
    z = rng.standard_normal((3, V))
    q = ref.softmax(rng.standard_normal((2, V)))
    p = ref.softmax(z)
    first, second = np.zeros(V), np.zeros(V)
    for _ in range(n):
        toks = [rng.choice(V, p=q[0]), rng.choice(V, p=q[1])]
        kept, tok, _, _ = ref.chain(z, q, toks, rng.random(2), rng.exponential(size=V), 1.0)
        out = toks[:kept] + [tok]
        first[out[0]] += 1
        if len(out) > 1:
            second[out[1]] += 1
    for seen, w in ((first, p[0]), (second, p[1])):
        want = seen.sum() * w
        assert ((seen - want) ** 2 / want).sum() < 18.5
