"""Host-side checks of the page-table, rotation and sampling calls (no kernel is
launched), and the rotation's table against 64-bit arithmetic."""
import ctypes

import numpy as np
import pytest

from speculative_decoding_tree_best_gb300 import binding
from tests import indep_serving as ref
from tests.test_chain_args import GOOD, P, lib  # noqa: F401

EINVAL, EUNSUP = binding.ST_EINVAL, binding.ST_EUNSUPPORTED
BAD = ctypes.c_void_p(24)


def pages(lib, cfg, pool=None, slots=P, ok=P, keep=P, n_new=None, ws=P):  # noqa: F811
    pool = binding.SpecPagePool(*([16] * 5)) if pool is None else pool
    c, p = ctypes.byref(cfg), ctypes.byref(pool)
    return (lib.page_tables_extend(c, p, n_new, slots, ok, ws, None),
            lib.page_tables_trim(c, p, keep, ws, None))


def test_page_table_arguments_are_refused(lib):  # noqa: F811
    for field, value in (("B", 0), ("B", 4097), ("T", 0), ("page", 48), ("n_pages", 0),
                         ("max_pages", 0), ("max_pages", 1 << 26)):
        cfg = binding.paged_cfg(**GOOD)
        setattr(cfg, field, value)
        assert pages(lib, cfg) == (EINVAL,) * 2
    cfg = binding.paged_cfg(**GOOD)
    for i in range(5):
        for bad in (0, 8):
            pool = binding.SpecPagePool(*[bad if j == i else 16 for j in range(5)])
            assert pages(lib, cfg, pool) == (EINVAL,) * 2
    for bad in (None, BAD):
        assert pages(lib, cfg, ws=bad) == (EINVAL,) * 2
        assert pages(lib, cfg, slots=bad)[0] == pages(lib, cfg, ok=bad)[0] == EINVAL
        assert pages(lib, cfg, keep=bad)[1] == EINVAL
    assert pages(lib, cfg, n_new=BAD)[0] == EINVAL
    assert lib.page_tables_extend(ctypes.byref(cfg), None, None, P, P, P, None) == EINVAL


def rope(lib, cfg, turns=P, amp=1.0, pos=P, q=P, k=P, qo=P, ko=P):  # noqa: F811
    return lib.rope_apply(ctypes.byref(cfg), turns, amp, pos, q, k, qo, ko, None)


def append(lib, cfg, pcfg, kv=None, turns=P, amp=1.0, slots=P, q=P, k=P, v=P, qo=P, ws=P):  # noqa: F811
    kv = binding.SpecPagedKV(*([16] * 6)) if kv is None else kv
    return lib.rope_page_append(ctypes.byref(cfg), ctypes.byref(pcfg), ctypes.byref(kv), turns, amp,
                                slots, q, k, v, qo, ws, None)


@pytest.mark.parametrize("field,value", [
    ("rows", 0), ("rows", -1), ("Hq", 0), ("Hq", 1 << 17), ("Hkv", -1), ("D", 96), ("rot", 0), ("rot", 24),
    ("rot", 144), ("layout", 2), ("layout", -1), ("inverse", 2), ("io_dtype", 3), ("q_stride", 8),
    ("q_stride", 1028), ("q_stride", -1024), ("k_stride", 100), ("v_stride", 255)])
def test_rotation_shapes_are_refused(lib, field, value):  # noqa: F811
    want = EUNSUP if field == "io_dtype" else EINVAL
    cfg = binding.rope_cfg(6, 8, 2, 128)
    setattr(cfg, field, value)
    assert rope(lib, cfg) == want
    pcfg = binding.paged_cfg(**GOOD)
    assert append(lib, cfg, pcfg) == want


def test_rotation_arguments_are_refused(lib):  # noqa: F811
    cfg, pcfg = binding.rope_cfg(6, 8, 2, 128), binding.paged_cfg(**GOOD, kv="e4m3")
    for bad in (None, BAD):
        for n in ("turns", "pos", "q", "k", "qo", "ko"):
            assert rope(lib, cfg, **{n: bad}) == EINVAL
        for n in ("turns", "slots", "q", "k", "v", "qo", "ws"):
            assert append(lib, cfg, pcfg, **{n: bad}) == EINVAL
    for amp in (float("nan"), float("inf")):
        assert rope(lib, cfg, amp=amp) == EINVAL and append(lib, cfg, pcfg, amp=amp) == EINVAL
    for i in range(6):
        kv = binding.SpecPagedKV(*[8 if j == i else 16 for j in range(6)])
        assert append(lib, cfg, pcfg, kv=kv) == EINVAL
    for other in (dict(rows=5), dict(Hq=6), dict(Hkv=4), dict(D=64), dict(io="f32")):
        c = binding.rope_cfg(**{**dict(rows=6, Hq=8, Hkv=2, D=128), **other})
        c.rot = 64
        assert append(lib, c, pcfg) == EINVAL
    assert append(lib, binding.rope_cfg(6, 8, 0, 128), pcfg) == EINVAL
    assert rope(lib, binding.rope_cfg(1 << 30, 128, 64, 128)) == EINVAL      # heads in all


@pytest.mark.parametrize("rot", [16, 48, 128])
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=8.0),
                                dict(scaling="ntk", factor=4.0),
                                dict(scaling="yarn", factor=32.0, orig_len=8192),
                                dict(scaling="yarn", factor=1.0, orig_len=1, beta_fast=2.5, beta_slow=0.0)])
@pytest.mark.parametrize("base", [1.0, 1e4, 5e6])
def test_table(lib, rot, kw, base):  # noqa: F811
    turns, amp = binding.spec_rope_turns(rot, base, **kw)
    f, a = ref.frequencies(rot, base, **{k: v for k, v in kw.items()})
    # a few roundings of 64-bit arithmetic, and half a unit
    np.testing.assert_allclose(np.array(turns, np.float64), f / (2 * np.pi) * 2.0 ** 64,
                               rtol=2.0 ** -47, atol=1.0)
    assert amp == np.float32(a)


def test_tables_are_refused(lib):  # noqa: F811
    nan, inf = float("nan"), float("inf")
    for rot in (0, 8, 20, 144, -16):
        with pytest.raises(binding.SpecError):
            binding.spec_rope_turns(rot)
    for kw in (dict(base=0.5), dict(base=nan), dict(base=inf), dict(scaling="linear", factor=0.5),
               dict(scaling="ntk", factor=nan), dict(scaling="ntk", factor=1e300, base=1e300),
               dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, orig_len=10, beta_fast=1.0),
               dict(scaling="yarn", factor=2.0, orig_len=10, beta_slow=-1.0),
               dict(scaling="yarn", factor=inf, orig_len=10)):
        with pytest.raises(binding.SpecError):
            binding.spec_rope_turns(64, **kw)
    with pytest.raises(KeyError):
        binding.spec_rope_turns(64, scaling="other")
    s = binding.SpecRopeScaling(1e4, 1.0, 32.0, 1.0, 0, 4)
    assert lib.spec_rope_turns(64, ctypes.byref(s), P, ctypes.byref(ctypes.c_float())) == EINVAL
    assert lib.spec_rope_turns(64, None, P, ctypes.byref(ctypes.c_float())) == EINVAL


def sample(lib, cfg, logits=P, params=(16,) * 4, e=P, out=(16,) * 4, ws=P):  # noqa: F811
    p, o = binding.SpecSampleParams(*params), binding.SpecSampleOut(*out)
    return lib.token_sample(ctypes.byref(cfg), logits, ctypes.byref(p), e, ctypes.byref(o), ws, None)


def test_sampling_arguments_are_refused(lib):  # noqa: F811
    for field, value in (("R", 0), ("R", (1 << 20) + 1), ("V", 0), ("V", (1 << 20) + 1),
                         ("per", 0), ("io_dtype", 2)):
        cfg = binding.sample_cfg(2, 1000)
        setattr(cfg, field, value)
        assert sample(lib, cfg) == (EUNSUP if field == "io_dtype" else EINVAL)
        assert lib.spec_sample_workspace_bytes(ctypes.byref(cfg), 152) == 0
    cfg = binding.sample_cfg(2, 1000)
    assert lib.spec_sample_workspace_bytes(ctypes.byref(cfg), -1) == 0
    assert binding.spec_sample_workspace_bytes(cfg, 152) % 256 == 0
    for bad in (None, BAD):
        assert sample(lib, cfg, logits=bad) == EINVAL and sample(lib, cfg, ws=bad) == EINVAL
        assert sample(lib, cfg, e=bad) == EINVAL                 # a token without random numbers
    for i in range(4):
        assert sample(lib, cfg, params=[8 if j == i else 16 for j in range(4)]) == EINVAL
        assert sample(lib, cfg, out=[8 if j == i else 16 for j in range(4)]) == EINVAL
    assert sample(lib, cfg, e=None, out=(0, 0, 0, 0)) == EINVAL      # nothing to do
    assert sample(lib, cfg, e=None, out=(0, 16, 16, 0)) == EINVAL    # a probability without a token
    assert sample(lib, cfg, out=(0, 0, 16, 16)) == EINVAL            # random numbers without a token
    assert lib.token_sample(ctypes.byref(cfg), P, None, P, ctypes.byref(binding.SpecSampleOut(
        *([16] * 4))), P, None) == EINVAL
