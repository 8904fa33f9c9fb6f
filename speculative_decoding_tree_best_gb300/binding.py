"""Thin ctypes binding of libspectree (include/spec_tree.h).

The functions below carry the C entry points' names and do argument
marshalling only: they check that tensors are CUDA, contiguous and of the
expected dtype, then pass raw device pointers and the current CUDA stream.
Every step of the computation runs in the library's kernels; there is no
fallback, and loading fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspectree.so")

ST_OK, ST_EINVAL, ST_EUNSUPPORTED, ST_ECUDA, ST_EOVERFLOW, ST_TIMEOUT, ST_ESCRATCH = range(7)
NOALLOC_SCRATCH_BYTES = 8 << 20
SPEC_DEV_OVERFLOW, SPEC_DEV_BADLAT, SPEC_DEV_TIMEOUT, SPEC_DEV_BADREQ = 0x1, 0x2, 0x4, 0x8
SPEC_DEV_BADLOGIT, SPEC_DEV_RANGE = 0x10, 0x20
SPEC_DEV_BADPAGE, SPEC_DEV_BADTOK = 0x40, 0x80
SPEC_IO_F32, SPEC_IO_BF16 = 0, 1
SPEC_KV_IO, SPEC_KV_E4M3 = 0, 1
EXPORTS = ("spec_workspace_bytes", "spec_workspace_bytes_for_sms", "spec_tree_build", "gdn_tree_verify", "attn_tree_verify",
           "accept_and_commit", "spec_verify_step", "spec_status_read", "spec_status_clear",
           "spec_status_string", "spec_abi_version", "attn_tree_verify_noalloc",
           "spec_wait_probe", "spec_step_launches", "spec_tree_build_ragged",
           "spec_verify_step_ragged", "spec_tree_build_markov", "spec_verify_step_markov",
           "accept_and_commit_sampled", "spec_verify_step_sampled",
           "spec_verify_step_persistent", "spec_step_launches_persistent",
           "spec_paged_workspace_bytes", "kv_page_append", "kv_page_read", "attn_decode_paged",
           "spec_draft_workspace_bytes", "draft_verify_sampled")
SAMPLE_CHUNK = 4096
_STATUS_BYTES = 256          # the status word and its reserve, at the head of a workspace

_lock = threading.Lock()
_lib = None


class SpecError(RuntimeError):
    def __init__(self, fn, code, msg):
        super().__init__(f"{fn} returned {code}: {msg}")
        self.code = code


class SpecCfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "B", "m", "K", "N", "Hk", "Hv", "dk", "dv", "Hq", "Hkv", "D", "Lmax", "V",
        "n_gdn_layers", "n_attn_layers", "io_dtype")]


class SpecTree(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "node_tok", "node_parent", "node_depth", "node_rank", "node_score", "node_anc", "n_nodes")]


class SpecCommitIO(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "h0", "gdn_k", "gdn_v", "alpha", "beta", "k_tree", "v_tree", "k_cache", "v_cache",
        "kv_len", "root_tok")]


class SpecStepIO(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("gdn_q", "gdn_o", "gdn_c", "attn_q", "attn_o")]


class SpecAccept(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("argmax", "accept_len", "accept_nodes", "out_tok")]


class SpecSampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("reserved", ctypes.c_uint32),
                ("seed", ctypes.c_uint64)]


class SpecPagedCfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "B", "T", "Hq", "Hkv", "D", "page", "n_pages", "max_pages", "io_dtype", "kv_dtype")]


class SpecPagedKV(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "k_pages", "v_pages", "k_scale", "v_scale", "page_table", "kv_len")]


class SpecDraftCfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "N", "V", "io_dtype")] + [
        ("temperature", ctypes.c_float), ("reserved", ctypes.c_uint32)]


class SpecDraftOut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("accept_len", "out_tok", "target_prob")]


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libspectree.so (raises if it is missing: build it first)."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"libspectree not built ({p} missing): run "
                                   "`python -c 'import __graft_entry__ as g; g.build()'`")
            lib = ctypes.CDLL(p)
            vp, cfgp = ctypes.c_void_p, ctypes.POINTER(SpecCfg)
            lib.spec_workspace_bytes.argtypes = [cfgp]
            lib.spec_workspace_bytes.restype = ctypes.c_size_t
            lib.spec_workspace_bytes_for_sms.argtypes = [cfgp, ctypes.c_int]
            lib.spec_workspace_bytes_for_sms.restype = ctypes.c_size_t
            lib.spec_tree_build.argtypes = [cfgp, vp, vp, vp, ctypes.POINTER(SpecTree), vp, vp]
            lib.gdn_tree_verify.argtypes = [cfgp, ctypes.POINTER(SpecTree)] + [vp] * 10
            lib.attn_tree_verify.argtypes = [cfgp, ctypes.POINTER(SpecTree)] + [vp] * 9
            lib.accept_and_commit.argtypes = [cfgp, ctypes.POINTER(SpecTree), vp,
                                              ctypes.POINTER(SpecCommitIO),
                                              ctypes.POINTER(SpecAccept), vp, vp]
            lib.spec_verify_step.argtypes = [cfgp, vp, vp, ctypes.POINTER(SpecTree),
                                             ctypes.POINTER(SpecStepIO), vp,
                                             ctypes.POINTER(SpecCommitIO),
                                             ctypes.POINTER(SpecAccept), vp, vp]
            lib.spec_tree_build_ragged.argtypes = [cfgp, vp, vp, vp, vp, ctypes.c_int,
                                                   ctypes.POINTER(SpecTree), vp, vp]
            lib.spec_verify_step_ragged.argtypes = [cfgp, vp, vp, vp, ctypes.c_int,
                                                    ctypes.POINTER(SpecTree),
                                                    ctypes.POINTER(SpecStepIO), vp,
                                                    ctypes.POINTER(SpecCommitIO),
                                                    ctypes.POINTER(SpecAccept), vp, vp]
            lib.spec_tree_build_markov.argtypes = [cfgp, vp, vp, vp, vp, ctypes.c_int, vp,
                                                   ctypes.POINTER(SpecTree), vp, vp]
            lib.spec_verify_step_markov.argtypes = [cfgp, vp, vp, vp, vp, ctypes.c_int,
                                                    ctypes.POINTER(SpecTree),
                                                    ctypes.POINTER(SpecStepIO), vp,
                                                    ctypes.POINTER(SpecCommitIO),
                                                    ctypes.POINTER(SpecAccept), vp, vp]
            smpp = ctypes.POINTER(SpecSampling)
            lib.accept_and_commit_sampled.argtypes = [cfgp, ctypes.POINTER(SpecTree), vp, smpp,
                                                      ctypes.POINTER(SpecCommitIO),
                                                      ctypes.POINTER(SpecAccept), vp, vp]
            lib.spec_verify_step_sampled.argtypes = [cfgp, vp, vp, smpp, ctypes.POINTER(SpecTree),
                                                     ctypes.POINTER(SpecStepIO), vp,
                                                     ctypes.POINTER(SpecCommitIO),
                                                     ctypes.POINTER(SpecAccept), vp, vp]
            lib.spec_verify_step_persistent.argtypes = lib.spec_verify_step.argtypes
            lib.spec_step_launches_persistent.argtypes = [cfgp]
            lib.spec_status_read.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
            lib.spec_status_clear.argtypes = [vp, vp]
            lib.spec_status_string.argtypes = [ctypes.c_int]
            lib.spec_status_string.restype = ctypes.c_char_p
            lib.attn_tree_verify_noalloc.argtypes = [cfgp, ctypes.POINTER(SpecTree)] + [vp] * 9
            lib.spec_wait_probe.argtypes = [ctypes.c_uint32, ctypes.c_int, vp, vp]
            lib.spec_step_launches.argtypes = [cfgp]
            pcfgp, pkvp = ctypes.POINTER(SpecPagedCfg), ctypes.POINTER(SpecPagedKV)
            dcfgp = ctypes.POINTER(SpecDraftCfg)
            lib.spec_paged_workspace_bytes.argtypes = [pcfgp, ctypes.c_int]
            lib.spec_paged_workspace_bytes.restype = ctypes.c_size_t
            lib.spec_draft_workspace_bytes.argtypes = [dcfgp, ctypes.c_int]
            lib.spec_draft_workspace_bytes.restype = ctypes.c_size_t
            lib.kv_page_append.argtypes = [pcfgp, pkvp] + [vp] * 5
            lib.kv_page_read.argtypes = [pcfgp, pkvp, ctypes.c_int] + [vp] * 4
            lib.attn_decode_paged.argtypes = [pcfgp, pkvp] + [vp] * 5
            lib.draft_verify_sampled.argtypes = [dcfgp] + [vp] * 6 + [
                ctypes.POINTER(SpecDraftOut)] + [vp] * 4
            for n in ("kv_page_append", "kv_page_read", "attn_decode_paged",
                      "draft_verify_sampled"):
                getattr(lib, n).restype = ctypes.c_int
            for n in ("spec_tree_build", "gdn_tree_verify", "attn_tree_verify",
                      "attn_tree_verify_noalloc", "spec_wait_probe", "spec_step_launches",
                      "spec_tree_build_ragged", "spec_verify_step_ragged", "spec_tree_build_markov",
                      "spec_verify_step_markov", "accept_and_commit_sampled",
                      "spec_verify_step_sampled", "spec_verify_step_persistent",
                      "spec_step_launches_persistent", "accept_and_commit", "spec_verify_step", "spec_status_read",
                      "spec_status_clear", "spec_abi_version"):
                getattr(lib, n).restype = ctypes.c_int
            _lib = lib
    return _lib


# ------------------------------------------------------------------ helpers

def make_cfg(sc, **over) -> SpecCfg:
    """SpecCfg from a synth.SpecConfig (or any object with the same fields)."""
    d = dict(B=sc.B, m=sc.m, K=sc.K, N=sc.N, Hk=sc.Hk, Hv=sc.Hv, dk=sc.dk, dv=sc.dv, Hq=sc.Hq,
             Hkv=sc.Hkv, D=sc.D, Lmax=sc.Lmax, V=sc.V, n_gdn_layers=sc.n_gdn,
             n_attn_layers=sc.n_attn, io_dtype=SPEC_IO_BF16 if sc.io == "bf16" else SPEC_IO_F32)
    d.update(over)
    return SpecCfg(**d)


def _io_dtype(cfg: SpecCfg):
    return torch.bfloat16 if cfg.io_dtype == SPEC_IO_BF16 else torch.float32


def _ptr(t: Optional[torch.Tensor], dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(fn, rc):
    if rc != ST_OK:
        raise SpecError(fn, rc, load().spec_status_string(rc).decode())


class TreeBuffers:
    """Device buffers of a spec_tree for B requests and T = N + 1 rows."""

    def __init__(self, cfg: SpecCfg, device="cuda"):
        B, T = cfg.B, cfg.N + 1
        i32 = dict(dtype=torch.int32, device=device)
        self.node_tok = torch.empty((B, T), **i32)
        self.node_parent = torch.empty((B, T), **i32)
        self.node_depth = torch.empty((B, T), **i32)
        self.node_rank = torch.empty((B, T), **i32)
        self.node_score = torch.empty((B, T), dtype=torch.float32, device=device)
        self.node_anc = torch.empty((B, T, 2), dtype=torch.int64, device=device)
        self.n_nodes = torch.empty((B,), **i32)

    def c(self) -> SpecTree:
        return SpecTree(*(t.data_ptr() for t in (
            self.node_tok, self.node_parent, self.node_depth, self.node_rank, self.node_score,
            self.node_anc, self.n_nodes)))

    def to_numpy(self) -> dict:
        import numpy as np
        d = {k: getattr(self, k).cpu().numpy() for k in (
            "node_tok", "node_parent", "node_depth", "node_rank", "node_score", "n_nodes")}
        d["node_anc"] = self.node_anc.cpu().numpy().view(np.uint64)
        return d


class AcceptBuffers:
    def __init__(self, cfg: SpecCfg, device="cuda"):
        B, T, m = cfg.B, cfg.N + 1, cfg.m
        i32 = dict(dtype=torch.int32, device=device)
        self.argmax = torch.empty((B, T), **i32)
        self.accept_len = torch.empty((B,), **i32)
        self.accept_nodes = torch.empty((B, m + 1), **i32)
        self.out_tok = torch.empty((B, m + 1), **i32)

    def c(self) -> SpecAccept:
        return SpecAccept(self.argmax.data_ptr(), self.accept_len.data_ptr(),
                          self.accept_nodes.data_ptr(), self.out_tok.data_ptr())


# ------------------------------------------------------------- entry points

def spec_workspace_bytes(cfg: SpecCfg) -> int:
    """Workspace bytes for the current device."""
    n = load().spec_workspace_bytes(ctypes.byref(cfg))
    if n == 0:
        raise SpecError("spec_workspace_bytes", ST_EINVAL,
                        "invalid configuration (or no CUDA device visible)")
    return int(n)


def spec_workspace_bytes_for_sms(cfg: SpecCfg, num_sms: int) -> int:
    """Workspace bytes for a device with num_sms SMs (host only)."""
    n = load().spec_workspace_bytes_for_sms(ctypes.byref(cfg), int(num_sms))
    if n == 0:
        raise SpecError("spec_workspace_bytes_for_sms", ST_EINVAL, "invalid configuration")
    return int(n)


def alloc_workspace(cfg: SpecCfg, device="cuda") -> torch.Tensor:
    """Zero-filled workspace of spec_workspace_bytes(cfg) bytes."""
    return torch.zeros((spec_workspace_bytes(cfg),), dtype=torch.uint8, device=device)


def spec_tree_build(cfg, lat_tok, lat_score, root_tok, tree: TreeBuffers, ws, stream=None):
    _check("spec_tree_build", load().spec_tree_build(
        ctypes.byref(cfg), _ptr(lat_tok, torch.int32, "lat_tok"),
        _ptr(lat_score, torch.float32, "lat_score"), _ptr(root_tok, torch.int32, "root_tok"),
        ctypes.byref(tree.c()), _ptr(ws, name="ws"), _stream(stream)))


def gdn_tree_verify(cfg, tree: TreeBuffers, h0, q, k, v, alpha, beta, o, c=None, ws=None,
                    stream=None):
    dt = _io_dtype(cfg)
    _check("gdn_tree_verify", load().gdn_tree_verify(
        ctypes.byref(cfg), ctypes.byref(tree.c()), _ptr(h0, torch.float32, "h0"),
        _ptr(q, dt, "q"), _ptr(k, dt, "k"), _ptr(v, dt, "v"), _ptr(alpha, torch.float32, "alpha"),
        _ptr(beta, torch.float32, "beta"), _ptr(o, dt, "o"), _ptr(c, torch.float32, "c"),
        _ptr(ws, name="ws"), _stream(stream)))


def attn_tree_verify(cfg, tree: TreeBuffers, q, k_tree, v_tree, k_cache, v_cache, kv_len, o, ws,
                     stream=None):
    dt = _io_dtype(cfg)
    _check("attn_tree_verify", load().attn_tree_verify(
        ctypes.byref(cfg), ctypes.byref(tree.c()), _ptr(q, dt, "q"), _ptr(k_tree, dt, "k_tree"),
        _ptr(v_tree, dt, "v_tree"), _ptr(k_cache, dt, "k_cache"), _ptr(v_cache, dt, "v_cache"),
        _ptr(kv_len, torch.int32, "kv_len"), _ptr(o, dt, "o"), _ptr(ws, name="ws"),
        _stream(stream)))


def attn_tree_verify_noalloc(cfg, tree: TreeBuffers, q, k_tree, v_tree, k_cache, v_cache, kv_len,
                             o, dev_status=None, stream=None):
    """attn_tree_verify with the library's static scratch (no workspace);
    dev_status: None or a CUDA uint32/int32 word that receives SPEC_DEV_* bits."""
    dt = _io_dtype(cfg)
    if dev_status is not None and dev_status.dtype not in (torch.int32, torch.uint32):
        raise TypeError("dev_status: expected an int32 or uint32 CUDA tensor")
    _check("attn_tree_verify_noalloc", load().attn_tree_verify_noalloc(
        ctypes.byref(cfg), ctypes.byref(tree.c()), _ptr(q, dt, "q"), _ptr(k_tree, dt, "k_tree"),
        _ptr(v_tree, dt, "v_tree"), _ptr(k_cache, dt, "k_cache"), _ptr(v_cache, dt, "v_cache"),
        _ptr(kv_len, torch.int32, "kv_len"), _ptr(o, dt, "o"),
        _ptr(dev_status, name="dev_status"), _stream(stream)))


def _commit_io(cfg, io: dict) -> SpecCommitIO:
    dt = _io_dtype(cfg)
    f32, i32 = torch.float32, torch.int32
    types = dict(h0=f32, gdn_k=dt, gdn_v=dt, alpha=f32, beta=f32, k_tree=dt, v_tree=dt,
                 k_cache=dt, v_cache=dt, kv_len=i32, root_tok=i32)
    return SpecCommitIO(*(_ptr(io.get(n), types[n], n) for n in types))


def accept_and_commit(cfg, tree: TreeBuffers, logits, io: dict, out: AcceptBuffers, ws,
                      stream=None):
    """io: dict with stacked h0, gdn_k, gdn_v, alpha, beta, k_tree, v_tree,
    k_cache, v_cache (None allowed where the layer count is 0), kv_len, root_tok."""
    dt = _io_dtype(cfg)
    cio = _commit_io(cfg, io)
    _check("accept_and_commit", load().accept_and_commit(
        ctypes.byref(cfg), ctypes.byref(tree.c()), _ptr(logits, dt, "logits"), ctypes.byref(cio),
        ctypes.byref(out.c()), _ptr(ws, name="ws"), _stream(stream)))


def sampling(temperature: float, seed: int) -> SpecSampling:
    return SpecSampling(float(temperature), 0, int(seed) & 0xFFFFFFFFFFFFFFFF)


def accept_and_commit_sampled(cfg, tree: TreeBuffers, logits, smp: SpecSampling, io: dict,
                              out: AcceptBuffers, ws, stream=None):
    """accept_and_commit at temperature > 0: out.argmax receives each row's draw."""
    dt = _io_dtype(cfg)
    cio = _commit_io(cfg, io)
    _check("accept_and_commit_sampled", load().accept_and_commit_sampled(
        ctypes.byref(cfg), ctypes.byref(tree.c()), _ptr(logits, dt, "logits"), ctypes.byref(smp),
        ctypes.byref(cio), ctypes.byref(out.c()), _ptr(ws, name="ws"), _stream(stream)))


def spec_tree_build_ragged(cfg, lat_tok, lat_score, root_tok, m_req, node_budget: int,
                           tree: TreeBuffers, ws, stream=None):
    """Trees with per-request draft positions (m_req: CUDA int32 [B] or None) and
    a node budget shared by the batch (node_budget < 0: none)."""
    _check("spec_tree_build_ragged", load().spec_tree_build_ragged(
        ctypes.byref(cfg), _ptr(lat_tok, torch.int32, "lat_tok"),
        _ptr(lat_score, torch.float32, "lat_score"), _ptr(root_tok, torch.int32, "root_tok"),
        _ptr(m_req, torch.int32, "m_req"), int(node_budget), ctypes.byref(tree.c()),
        _ptr(ws, name="ws"), _stream(stream)))


def spec_tree_build_markov(cfg, lat_tok, lat_base, W1, W2, root_tok, tree: TreeBuffers, ws,
                           stream=None):
    """Best-first tree with Markov-head edge scores (W1, W2: CUDA f32 [V][R])."""
    _check("spec_tree_build_markov", load().spec_tree_build_markov(
        ctypes.byref(cfg), _ptr(lat_tok, torch.int32, "lat_tok"),
        _ptr(lat_base, torch.float32, "lat_base"), _ptr(W1, torch.float32, "W1"),
        _ptr(W2, torch.float32, "W2"), int(W1.shape[1]), _ptr(root_tok, torch.int32, "root_tok"),
        ctypes.byref(tree.c()), _ptr(ws, name="ws"), _stream(stream)))


def _step_io(cfg, step: dict) -> SpecStepIO:
    dt = _io_dtype(cfg)
    return SpecStepIO(_ptr(step.get("gdn_q"), dt, "gdn_q"), _ptr(step.get("gdn_o"), dt, "gdn_o"),
                      _ptr(step.get("gdn_c"), torch.float32, "gdn_c"),
                      _ptr(step.get("attn_q"), dt, "attn_q"), _ptr(step.get("attn_o"), dt, "attn_o"))


def spec_verify_step(cfg, lat_tok, lat_score, tree: TreeBuffers, step: dict, logits, io: dict,
                     out: AcceptBuffers, ws, stream=None):
    """Whole verify step (tree, every GDN and attention layer, accept+commit).
    step: dict with stacked gdn_q, gdn_o, gdn_c (or None), attn_q, attn_o."""
    dt = _io_dtype(cfg)
    sio = _step_io(cfg, step)
    _check("spec_verify_step", load().spec_verify_step(
        ctypes.byref(cfg), _ptr(lat_tok, torch.int32, "lat_tok"),
        _ptr(lat_score, torch.float32, "lat_score"), ctypes.byref(tree.c()), ctypes.byref(sio),
        _ptr(logits, dt, "logits"), ctypes.byref(_commit_io(cfg, io)), ctypes.byref(out.c()),
        _ptr(ws, name="ws"), _stream(stream)))


def spec_verify_step_persistent(cfg, lat_tok, lat_score, tree: TreeBuffers, step: dict, logits,
                                io: dict, out: AcceptBuffers, ws, stream=None):
    """spec_verify_step with the argmax, acceptance and every GDN layer's
    verify + commit in one persistent launch."""
    dt = _io_dtype(cfg)
    sio = _step_io(cfg, step)
    _check("spec_verify_step_persistent", load().spec_verify_step_persistent(
        ctypes.byref(cfg), _ptr(lat_tok, torch.int32, "lat_tok"),
        _ptr(lat_score, torch.float32, "lat_score"), ctypes.byref(tree.c()), ctypes.byref(sio),
        _ptr(logits, dt, "logits"), ctypes.byref(_commit_io(cfg, io)), ctypes.byref(out.c()),
        _ptr(ws, name="ws"), _stream(stream)))


def spec_step_launches_persistent(cfg) -> int:
    return int(load().spec_step_launches_persistent(ctypes.byref(cfg)))


def spec_verify_step_sampled(cfg, lat_tok, lat_score, smp: SpecSampling, tree: TreeBuffers,
                             step: dict, logits, io: dict, out: AcceptBuffers, ws, stream=None):
    """spec_verify_step with the sampled acceptance."""
    dt = _io_dtype(cfg)
    sio = _step_io(cfg, step)
    _check("spec_verify_step_sampled", load().spec_verify_step_sampled(
        ctypes.byref(cfg), _ptr(lat_tok, torch.int32, "lat_tok"),
        _ptr(lat_score, torch.float32, "lat_score"), ctypes.byref(smp), ctypes.byref(tree.c()),
        ctypes.byref(sio), _ptr(logits, dt, "logits"), ctypes.byref(_commit_io(cfg, io)),
        ctypes.byref(out.c()), _ptr(ws, name="ws"), _stream(stream)))


def spec_verify_step_ragged(cfg, lat_tok, lat_score, m_req, node_budget: int, tree: TreeBuffers,
                            step: dict, logits, io: dict, out: AcceptBuffers, ws, stream=None):
    """spec_verify_step over the trees of spec_tree_build_ragged."""
    dt = _io_dtype(cfg)
    sio = _step_io(cfg, step)
    _check("spec_verify_step_ragged", load().spec_verify_step_ragged(
        ctypes.byref(cfg), _ptr(lat_tok, torch.int32, "lat_tok"),
        _ptr(lat_score, torch.float32, "lat_score"), _ptr(m_req, torch.int32, "m_req"),
        int(node_budget), ctypes.byref(tree.c()), ctypes.byref(sio), _ptr(logits, dt, "logits"),
        ctypes.byref(_commit_io(cfg, io)), ctypes.byref(out.c()), _ptr(ws, name="ws"),
        _stream(stream)))


def spec_verify_step_markov(cfg, lat_tok, lat_base, W1, W2, tree: TreeBuffers, step: dict, logits,
                            io: dict, out: AcceptBuffers, ws, stream=None):
    """spec_verify_step over the tree of spec_tree_build_markov."""
    dt = _io_dtype(cfg)
    sio = _step_io(cfg, step)
    _check("spec_verify_step_markov", load().spec_verify_step_markov(
        ctypes.byref(cfg), _ptr(lat_tok, torch.int32, "lat_tok"),
        _ptr(lat_base, torch.float32, "lat_base"), _ptr(W1, torch.float32, "W1"),
        _ptr(W2, torch.float32, "W2"), int(W1.shape[1]), ctypes.byref(tree.c()),
        ctypes.byref(sio), _ptr(logits, dt, "logits"), ctypes.byref(_commit_io(cfg, io)),
        ctypes.byref(out.c()), _ptr(ws, name="ws"), _stream(stream)))


def spec_status_read(ws, stream=None) -> int:
    v = ctypes.c_uint32(0)
    _check("spec_status_read", load().spec_status_read(_ptr(ws, name="ws"), ctypes.byref(v),
                                                       _stream(stream)))
    return int(v.value)


def spec_step_launches(cfg) -> int:
    """Kernel launches one spec_verify_step call makes (host only)."""
    n = load().spec_step_launches(ctypes.byref(cfg))
    if n < 0:
        raise SpecError("spec_step_launches", ST_EINVAL, "invalid cfg")
    return n


def spec_wait_probe(limit_us: int, satisfy: bool, ws, stream=None):
    """One bounded device wait (diagnostic): SPEC_DEV_TIMEOUT when unsatisfied."""
    _check("spec_wait_probe", load().spec_wait_probe(int(limit_us), int(bool(satisfy)),
                                                     _ptr(ws, name="ws"), _stream(stream)))


def spec_status_clear(ws, stream=None):
    _check("spec_status_clear", load().spec_status_clear(_ptr(ws, name="ws"), _stream(stream)))


# ------------------------------------------- paged cache, decode, drafted chain

_IO = {"bf16": (SPEC_IO_BF16, torch.bfloat16), "f32": (SPEC_IO_F32, torch.float32)}
_KV = {"io": SPEC_KV_IO, "e4m3": SPEC_KV_E4M3}


def paged_cfg(B, T, Hq, Hkv, D, page, n_pages, max_pages, io="bf16", kv="io") -> SpecPagedCfg:
    """Shape of the paged calls; io "bf16" or "f32", kv "io" or "e4m3"."""
    return SpecPagedCfg(B, T, Hq, Hkv, D, page, n_pages, max_pages, _IO[io][0], _KV[kv])


def draft_cfg(B, N, V, io="bf16", temperature=1.0) -> SpecDraftCfg:
    """Shape of draft_verify_sampled; io is the logits' type."""
    return SpecDraftCfg(B, N, V, _IO[io][0], float(temperature), 0)


def _arg(t, dtype, shape, name, device):
    """Data pointer of a contiguous CUDA tensor of that type and shape on the
    current device (None passes: an argument that may be absent)."""
    if t is None:
        return None
    try:
        if (t.dtype is dtype and t.get_device() == device and t.shape == shape
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{device}")
    raise ValueError(f"{name} must be contiguous")


def _workspace(ws, need, device):
    try:
        if ws.get_device() == device and ws.nbytes >= need and ws.is_contiguous():
            return ws.data_ptr()
    except AttributeError:
        pass
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or not ws.is_contiguous():
        raise TypeError("ws must be a contiguous CUDA tensor")
    if ws.get_device() != device:
        raise ValueError(f"ws is on cuda:{ws.get_device()}, the current device is cuda:{device}")
    raise ValueError(f"ws holds {ws.nbytes} bytes, {need} are needed")


class _Plan:
    """What the calls of one configuration on one device need to know: the
    shapes and types of their arguments and the workspace's size."""
    __slots__ = ("new", "q", "b", "dt", "need", "rows", "probs", "e")

    def __init__(self, cfg):
        if isinstance(cfg, SpecPagedCfg):
            self.new = (cfg.B, cfg.T, cfg.Hkv, cfg.D)
            self.q = (cfg.B, cfg.T, cfg.Hq, cfg.D)
            self.need = int(load().spec_paged_workspace_bytes(ctypes.byref(cfg), 0))
        else:
            self.new = (cfg.B, cfg.N)
            self.q = (cfg.B, cfg.N + 1, cfg.V)
            self.rows = self.q[:2]
            self.probs = self.new + (cfg.V,)
            self.e = (cfg.B, cfg.V)
            self.need = int(load().spec_draft_workspace_bytes(ctypes.byref(cfg), 0))
        self.b = (cfg.B,)
        self.dt = _io_dtype(cfg)


_plans = {}
# what a call asks of torch, looked up once
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_get_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _plan(cfg, raw, device) -> _Plan:
    """raw: bytes(cfg) (the two configurations differ in length)."""
    p = _plans.get((raw, device))
    if p is None:
        if len(_plans) >= 1024:
            _plans.clear()
        p = _plans[raw, device] = _Plan(cfg)
    return p


def _raw_stream(stream, device):
    """_stream as an integer; the current stream without making an object."""
    if stream is None:
        return _get_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _required(t, name):
    if t is None:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t


def spec_paged_workspace_bytes(cfg: SpecPagedCfg, num_sms: int = 0) -> int:
    """Workspace bytes of the paged calls (num_sms 0: the current device's)."""
    n = load().spec_paged_workspace_bytes(ctypes.byref(cfg), int(num_sms))
    if n == 0:
        raise SpecError("spec_paged_workspace_bytes", ST_EINVAL,
                        "invalid configuration (or no CUDA device visible)")
    return int(n)


def spec_draft_workspace_bytes(cfg: SpecDraftCfg, num_sms: int = 0) -> int:
    """Workspace bytes of draft_verify_sampled (num_sms 0: the current device's)."""
    n = load().spec_draft_workspace_bytes(ctypes.byref(cfg), int(num_sms))
    if n == 0:
        raise SpecError("spec_draft_workspace_bytes", ST_EINVAL,
                        "invalid configuration (or no CUDA device visible)")
    return int(n)


def alloc_paged_workspace(cfg: SpecPagedCfg, device="cuda") -> torch.Tensor:
    """Zero-filled workspace of spec_paged_workspace_bytes(cfg) bytes."""
    return torch.zeros((spec_paged_workspace_bytes(cfg),), dtype=torch.uint8, device=device)


def alloc_draft_workspace(cfg: SpecDraftCfg, device="cuda") -> torch.Tensor:
    """Zero-filled workspace of spec_draft_workspace_bytes(cfg) bytes."""
    return torch.zeros((spec_draft_workspace_bytes(cfg),), dtype=torch.uint8, device=device)


class PagedKV:
    """A paged cache's tensors, checked once against a SpecPagedCfg.

    k_pages, v_pages [n_pages][Hkv][page][D] (io type; float8_e4m3fn with
    kv="e4m3"), k_scale, v_scale [n_pages][Hkv][page] fp32 (e4m3 only),
    page_table [B][max_pages] and kv_len [B] int32.  The tensors are fixed for
    the object's life; their contents are the caller's.
    """

    def __init__(self, cfg: SpecPagedCfg, k_pages, v_pages, page_table, kv_len, k_scale=None,
                 v_scale=None):
        q8 = cfg.kv_dtype == SPEC_KV_E4M3
        dt = torch.float8_e4m3fn if q8 else _io_dtype(cfg)
        dev = torch.cuda.current_device()
        pool = (cfg.n_pages, cfg.Hkv, cfg.page, cfg.D)
        i32, f32 = torch.int32, torch.float32
        if not q8 and (k_scale is not None or v_scale is not None):
            raise ValueError("k_scale and v_scale belong to a cache in 8 bits")
        sc = [_arg(_required(t, n), f32, pool[:3], n, dev) if q8 else None
              for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale"))]
        self._c = SpecPagedKV(
            _arg(_required(k_pages, "k_pages"), dt, pool, "k_pages", dev),
            _arg(_required(v_pages, "v_pages"), dt, pool, "v_pages", dev), *sc,
            _arg(_required(page_table, "page_table"), i32, (cfg.B, cfg.max_pages), "page_table",
                 dev),
            _arg(_required(kv_len, "kv_len"), i32, (cfg.B,), "kv_len", dev))
        self._ref = ctypes.byref(self._c)
        self._t = (k_pages, v_pages, k_scale, v_scale, page_table, kv_len)
        self.key = (pool, cfg.B, cfg.max_pages, cfg.kv_dtype, dt, dev)
        self._fits = set()

    k_pages, v_pages, k_scale, v_scale, page_table, kv_len = (
        property(lambda self, i=i: self._t[i]) for i in range(6))

    @classmethod
    def empty(cls, cfg: SpecPagedCfg, device="cuda") -> "PagedKV":
        """Zero-filled pool, a page table that owns no page (-1) and kv_len 0."""
        q8 = cfg.kv_dtype == SPEC_KV_E4M3
        dt = torch.float8_e4m3fn if q8 else _io_dtype(cfg)
        pool = (cfg.n_pages, cfg.Hkv, cfg.page, cfg.D)
        sc = [torch.ones(pool[:3], dtype=torch.float32, device=device) if q8 else None
              for _ in range(2)]
        return cls(cfg, torch.zeros(pool, dtype=dt, device=device),
                   torch.zeros(pool, dtype=dt, device=device),
                   torch.full((cfg.B, cfg.max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros((cfg.B,), dtype=torch.int32, device=device), *sc)

    def ref(self, cfg: SpecPagedCfg, raw: bytes, device: int):
        """The cache as an argument of a call with that configuration (raw: its bytes)."""
        if device != self.key[5]:
            raise ValueError(f"the cache is on cuda:{self.key[5]}, the current device is "
                             f"cuda:{device}")
        if raw not in self._fits:                  # T and Hq may differ from call to call
            pool = (cfg.n_pages, cfg.Hkv, cfg.page, cfg.D)
            if self.key[:4] != (pool, cfg.B, cfg.max_pages, cfg.kv_dtype) or (
                    cfg.kv_dtype == SPEC_KV_IO and self.key[4] != _io_dtype(cfg)):
                raise ValueError("the cache was made for another configuration")
            if len(self._fits) >= 64:
                self._fits.clear()
            self._fits.add(raw)
        return self._ref


def kv_page_append(cfg: SpecPagedCfg, kv: PagedKV, k_new, v_new, ws, n_new=None, stream=None):
    """Write the new tokens' rows (k_new, v_new [B][T][Hkv][D] io) behind the
    committed ones; n_new: None or CUDA int32 [B]."""
    dev, raw = _get_device(), bytes(cfg)
    p = _plan(cfg, raw, dev)
    rc = (_lib or load()).kv_page_append(
        ctypes.byref(cfg), kv.ref(cfg, raw, dev), _arg(k_new, p.dt, p.new, "k_new", dev),
        _arg(v_new, p.dt, p.new, "v_new", dev), _arg(n_new, torch.int32, p.b, "n_new", dev),
        _workspace(ws, _STATUS_BYTES, dev), _raw_stream(stream, dev))
    if rc:
        _check("kv_page_append", rc)


def kv_page_read(cfg: SpecPagedCfg, kv: PagedKV, k_out, v_out, ws, stream=None):
    """The committed rows as a contiguous cache [B][Lmax][Hkv][D] io (rows at
    or past kv_len are left as they were)."""
    dev, raw = _get_device(), bytes(cfg)
    p = _plan(cfg, raw, dev)
    Lmax = k_out.shape[1] if isinstance(k_out, torch.Tensor) and k_out.dim() == 4 else 0
    shape = (cfg.B, Lmax, cfg.Hkv, cfg.D)
    rc = (_lib or load()).kv_page_read(
        ctypes.byref(cfg), kv.ref(cfg, raw, dev), Lmax, _arg(k_out, p.dt, shape, "k_out", dev),
        _arg(v_out, p.dt, shape, "v_out", dev), _workspace(ws, _STATUS_BYTES, dev),
        _raw_stream(stream, dev))
    if rc:
        _check("kv_page_read", rc)


def attn_decode_paged(cfg: SpecPagedCfg, kv: PagedKV, q, o, ws, n_new=None, stream=None):
    """Attention of the new tokens (q, o [B][T][Hq][D] io) over the paged cache."""
    dev, raw = _get_device(), bytes(cfg)
    p = _plan(cfg, raw, dev)
    rc = (_lib or load()).attn_decode_paged(
        ctypes.byref(cfg), kv.ref(cfg, raw, dev), _arg(q, p.dt, p.q, "q", dev),
        _arg(n_new, torch.int32, p.b, "n_new", dev), _arg(o, p.dt, p.q, "o", dev),
        _workspace(ws, p.need, dev), _raw_stream(stream, dev))
    if rc:
        _check("attn_decode_paged", rc)


class DraftBuffers:
    """Outputs of draft_verify_sampled: accept_len [B], out_tok [B][N+1] int32 and
    target_prob [B][N] fp32.  The tensors are fixed for the object's life."""

    def __init__(self, cfg: SpecDraftCfg, device="cuda"):
        B, N = cfg.B, cfg.N
        self._t = (torch.empty((B,), dtype=torch.int32, device=device),
                   torch.empty((B, N + 1), dtype=torch.int32, device=device),
                   torch.empty((B, N), dtype=torch.float32, device=device))
        self.key = ((B, N + 1), self._t[0].get_device())
        self._c = SpecDraftOut(*(t.data_ptr() if t.numel() else None for t in self._t))
        self._ref = ctypes.byref(self._c)

    accept_len, out_tok, target_prob = (property(lambda self, i=i: self._t[i]) for i in range(3))

    def ref(self, rows, device: int):
        """The outputs as an argument of a call with (B, N + 1) rows."""
        if self.key != (rows, device):
            _arg(self.accept_len, torch.int32, rows[:1], "accept_len", device)
            _arg(self.out_tok, torch.int32, rows, "out_tok", device)
        return self._ref


def draft_verify_sampled(cfg: SpecDraftCfg, draft_tok, draft_prob, logits, u, e,
                         out: DraftBuffers, ws, n_draft=None, kv_len=None, root_tok=None,
                         stream=None):
    """Verify drafted chains from given random numbers: draft_tok int32 [B][N],
    draft_prob f32 [B][N][V] or None (point masses), logits io [B][N+1][V], u
    f32 [B][N], e f32 [B][V]; kv_len / root_tok are advanced when given.  n_draft
    int32 [B], -1 where a slot has no request, or None (N each).  With N = 0
    (plain sampling) draft_tok, draft_prob and u are not read."""
    dev, f32, i32 = _get_device(), torch.float32, torch.int32
    p = _plan(cfg, bytes(cfg), dev)
    if cfg.N == 0:
        draft_tok = draft_prob = u = None
    rc = (_lib or load()).draft_verify_sampled(
        ctypes.byref(cfg), _arg(draft_tok, i32, p.new, "draft_tok", dev),
        _arg(n_draft, i32, p.b, "n_draft", dev),
        _arg(draft_prob, f32, p.probs, "draft_prob", dev),
        _arg(logits, p.dt, p.q, "logits", dev), _arg(u, f32, p.new, "u", dev),
        _arg(e, f32, p.e, "e", dev), out.ref(p.rows, dev), _arg(kv_len, i32, p.b, "kv_len", dev),
        _arg(root_tok, i32, p.b, "root_tok", dev), _workspace(ws, p.need, dev),
        _raw_stream(stream, dev))
    if rc:
        _check("draft_verify_sampled", rc)
