"""One whole verify step on device buffers: tree build, every GDN layer, every
attention layer, then acceptance and commit -- each a call through the C ABI.

The driver owns the device buffers (stacked per layer, layer outermost, so
the commit sees every layer through one pointer per tensor) and issues the
calls on one stream.  It does no arithmetic of its own.
"""
from __future__ import annotations

import torch

from . import binding
from .synth import SpecConfig


def stack_inputs(inp: dict, device="cuda") -> dict:
    """Device copies of synth.make_step_inputs' output with layers stacked."""
    d = {}
    for k in ("lat_tok", "lat_score", "root_tok", "kv_len", "logits", "m_req", "lat_base", "W1",
              "W2"):
        if k in inp:
            d[k] = inp[k].to(device).contiguous()
    g, a = inp["gdn"], inp["attn"]
    for src, dst in (("h0", "gdn_h0"), ("q", "gdn_q"), ("k", "gdn_k"), ("v", "gdn_v"),
                     ("alpha", "gdn_alpha"), ("beta", "gdn_beta")):
        d[dst] = torch.stack([lay[src] for lay in g]).to(device).contiguous() if g else None
    for src, dst in (("q", "attn_q"), ("k_tree", "k_tree"), ("v_tree", "v_tree"),
                     ("k_cache", "k_cache"), ("v_cache", "v_cache")):
        d[dst] = torch.stack([lay[src] for lay in a]).to(device).contiguous() if a else None
    return d


class VerifyStep:
    """Buffers and calls of one verify step for a synthetic workload."""

    def __init__(self, scfg: SpecConfig, x: dict, device="cuda", persistent: bool = False):
        self.scfg = scfg
        self.persistent = persistent
        self.cfg = binding.make_cfg(scfg)
        self.x = x
        self.device = device
        c = self.cfg
        T = c.N + 1
        dt = torch.bfloat16 if scfg.io == "bf16" else torch.float32
        self.tree = binding.TreeBuffers(c, device)
        self.acc = binding.AcceptBuffers(c, device)
        self.ws = binding.alloc_workspace(c, device)
        self.gdn_o = torch.empty((c.n_gdn_layers, c.B, T, c.Hv, c.dv), dtype=dt, device=device)
        self.attn_o = torch.empty((c.n_attn_layers, c.B, T, c.Hq, c.D), dtype=dt, device=device)

    # the three phases ----------------------------------------------------------
    def build_tree(self, stream=None):
        x = self.x
        if self.scfg.markov_R > 0:
            binding.spec_tree_build_markov(self.cfg, x["lat_tok"], x["lat_base"], x["W1"], x["W2"],
                                           x["root_tok"], self.tree, self.ws, stream)
        elif self.scfg.ragged:
            binding.spec_tree_build_ragged(self.cfg, x["lat_tok"], x["lat_score"], x["root_tok"],
                                           x.get("m_req"), self.scfg.budget, self.tree, self.ws,
                                           stream)
        else:
            binding.spec_tree_build(self.cfg, x["lat_tok"], x["lat_score"], x["root_tok"],
                                    self.tree, self.ws, stream)

    def verify_gdn(self, stream=None):
        x, c = self.x, self.cfg
        for l in range(c.n_gdn_layers):
            binding.gdn_tree_verify(c, self.tree, x["gdn_h0"][l], x["gdn_q"][l], x["gdn_k"][l],
                                    x["gdn_v"][l], x["gdn_alpha"][l], x["gdn_beta"][l],
                                    self.gdn_o[l], None, self.ws, stream)

    def verify_attention(self, stream=None):
        x, c = self.x, self.cfg
        for l in range(c.n_attn_layers):
            binding.attn_tree_verify(c, self.tree, x["attn_q"][l], x["k_tree"][l], x["v_tree"][l],
                                     x["k_cache"][l], x["v_cache"][l], x["kv_len"],
                                     self.attn_o[l], self.ws, stream)

    def verify(self, stream=None):
        self.verify_gdn(stream)
        self.verify_attention(stream)

    def commit_io(self) -> dict:
        x = self.x
        return dict(h0=x["gdn_h0"], gdn_k=x["gdn_k"], gdn_v=x["gdn_v"], alpha=x["gdn_alpha"],
                    beta=x["gdn_beta"], k_tree=x["k_tree"], v_tree=x["v_tree"],
                    k_cache=x["k_cache"], v_cache=x["v_cache"], kv_len=x["kv_len"],
                    root_tok=x["root_tok"])

    def accept_commit(self, stream=None):
        if self.scfg.temperature > 0:
            binding.accept_and_commit_sampled(self.cfg, self.tree, self.x["logits"],
                                              self.sampling(), self.commit_io(), self.acc,
                                              self.ws, stream)
        else:
            binding.accept_and_commit(self.cfg, self.tree, self.x["logits"], self.commit_io(),
                                      self.acc, self.ws, stream)

    def sampling(self):
        return binding.sampling(self.scfg.temperature, self.scfg.sample_seed)

    def run_calls(self, stream=None):
        """The step as the four single-operation calls."""
        self.build_tree(stream)
        self.verify(stream)
        self.accept_commit(stream)

    def run(self, stream=None):
        """The step as one spec_verify_step call (programmatic dependent launch)."""
        x = self.x
        step = dict(gdn_q=x["gdn_q"], gdn_o=self.gdn_o if self.cfg.n_gdn_layers else None,
                    gdn_c=None, attn_q=x["attn_q"],
                    attn_o=self.attn_o if self.cfg.n_attn_layers else None)
        if self.persistent:
            if self.scfg.markov_R > 0 or self.scfg.ragged or self.scfg.temperature > 0:
                raise ValueError("the persistent step takes the plain lattice and the argmax")
            binding.spec_verify_step_persistent(self.cfg, x["lat_tok"], x["lat_score"], self.tree,
                                                step, x["logits"], self.commit_io(), self.acc,
                                                self.ws, stream)
        elif self.scfg.temperature > 0:
            if self.scfg.markov_R > 0 or self.scfg.ragged:
                raise ValueError("the fused sampled step takes the plain lattice")
            binding.spec_verify_step_sampled(self.cfg, x["lat_tok"], x["lat_score"],
                                             self.sampling(), self.tree, step, x["logits"],
                                             self.commit_io(), self.acc, self.ws, stream)
        elif self.scfg.markov_R > 0:
            binding.spec_verify_step_markov(self.cfg, x["lat_tok"], x["lat_base"], x["W1"], x["W2"],
                                            self.tree, step, x["logits"], self.commit_io(), self.acc,
                                            self.ws, stream)
        elif self.scfg.ragged:
            binding.spec_verify_step_ragged(self.cfg, x["lat_tok"], x["lat_score"], x.get("m_req"),
                                            self.scfg.budget, self.tree, step, x["logits"],
                                            self.commit_io(), self.acc, self.ws, stream)
        else:
            binding.spec_verify_step(self.cfg, x["lat_tok"], x["lat_score"], self.tree, step,
                                     x["logits"], self.commit_io(), self.acc, self.ws, stream)

    @property
    def launches_per_step(self) -> int:
        if self.persistent:
            return binding.spec_step_launches_persistent(self.cfg)
        # the shared budget adds one launch (the selection) to the step; the
        # sampled acceptance is a launch of its own (the argmax shares the last
        # attention merge's)
        extra = (1 if self.scfg.budget >= 0 else 0)
        merged = self.cfg.n_attn_layers > 0 and self.cfg.B * (self.cfg.N + 1) <= 64
        extra += 1 if (self.scfg.temperature > 0 and merged) else 0
        return binding.spec_step_launches(self.cfg) + extra


# The step's per-step inputs in three pieces, in the order the copies are
# issued: the lattice with the attention rows (the tree build and the
# attention layers), the GDN rows, then the logits, read only by the
# acceptance.  Each copy costs a few microseconds of its own, so small pieces
# go together; the GDN rows stay apart because with many GDN layers they are
# most of the non-logits bytes and the attention need not wait for them.
HOST_PIECES = (("rows", ("lat_tok", "lat_score", "m_req", "lat_base", "attn_q", "k_tree",
                         "v_tree")),
               ("gdn", ("gdn_q", "gdn_k", "gdn_v", "gdn_alpha", "gdn_beta")),
               ("logits", ("logits",)))


class HostStep:
    """A verify step whose per-step inputs come from pinned host memory.

    The inputs are copied in three pieces on a copy stream (the lattice with
    the attention rows, the GDN rows, the logits), in the order the step reads
    them, and each phase on the compute stream waits only for its own piece:
    the logits -- most of the bytes -- are copied while the tree, attention
    and GDN layers run, and only the acceptance and commit wait for them.  The accepted lengths and tokens come back to pinned host
    memory at the end.  The whole sequence is captured once as a CUDA graph
    and replayed per step.

    st: a VerifyStep whose per-step input tensors this object re-points at
    its device pieces (their current values are copied into the pinned host
    buffers, which the caller then refills per step through `views`).
    """

    def __init__(self, st: "VerifyStep"):
        self.st = st
        x = st.x
        self.host, self.dev, self.views = {}, {}, {}
        self.h2d_bytes = 0
        for piece, keys in HOST_PIECES:
            keys = [k for k in keys if x.get(k) is not None]
            if not keys:
                continue
            offs, total = {}, 0
            for k in keys:
                offs[k] = total
                total += (x[k].numel() * x[k].element_size() + 255) // 256 * 256
            dev = torch.empty(total, dtype=torch.uint8, device=st.device)
            host = torch.empty(total, dtype=torch.uint8).pin_memory()
            for k in keys:
                n = x[k].numel() * x[k].element_size()
                view = dev[offs[k]:offs[k] + n].view(x[k].dtype).view(x[k].shape)
                view.copy_(x[k])
                host[offs[k]:offs[k] + n].copy_(x[k].cpu().contiguous().view(-1).view(torch.uint8))
                x[k] = view
                self.views[k] = host[offs[k]:offs[k] + n].view(view.dtype).view(view.shape)
            self.host[piece], self.dev[piece] = host, dev
            self.h2d_bytes += sum(x[k].numel() * x[k].element_size() for k in keys)
        self.out = {k: torch.empty_like(getattr(st.acc, k), device="cpu").pin_memory()
                    for k in ("accept_len", "out_tok")}
        self.d2h_bytes = sum(t.numel() * t.element_size() for t in self.out.values())
        self.copy_stream = torch.cuda.Stream(device=st.device)
        self.graph = None

    def _sequence(self):
        st = self.st
        comp = torch.cuda.current_stream()
        cs = self.copy_stream
        cs.wait_stream(comp)                 # the previous step's readers are done
        ev = {}
        with torch.cuda.stream(cs):
            for piece, _ in HOST_PIECES:
                if piece in self.dev:
                    self.dev[piece].copy_(self.host[piece], non_blocking=True)
                    ev[piece] = torch.cuda.Event()
                    ev[piece].record(cs)
        for piece, run in (("rows", st.build_tree), (None, st.verify_attention),
                           ("gdn", st.verify_gdn), ("logits", st.accept_commit)):
            if piece in ev:
                comp.wait_event(ev[piece])
            run()
        comp.wait_stream(cs)
        for k, t in self.out.items():
            t.copy_(getattr(st.acc, k), non_blocking=True)

    def capture(self):
        """Run the copies, the four phases and the result read-back once,
        then capture them as a CUDA graph."""
        self._sequence()
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, capture_error_mode="thread_local"):
            self._sequence()
        torch.cuda.synchronize()

    def run(self):
        """One step: copies in, the step, results out (asynchronous on the
        current stream; synchronize before reading self.out)."""
        if self.graph is None:
            self.capture()
        self.graph.replay()


class ChainStep:
    """Buffers and calls of a serving step over a paged cache with a chain of
    drafts: per attention layer the new tokens' rows are appended and attended
    from (attend), then the drafts are verified (verify), which advances kv_len
    over what was kept.  A step of request b has n_draft[b] + 1 new tokens: the
    pending token and its drafts; with n_draft 0 it is a plain decode step, and
    with n_draft -1 the slot has no request: it is neither written nor advanced.

    The layers share one page table, kv_len and root_tok, which the caller
    owns the contents of (page_table names the pages of each request; a page
    id is good for every layer's pool).  Rows of refused drafts are written
    over by the next step.

    The page table can be left to the step: begin() takes the pages that the new
    tokens' rows need from `pool`, attend_rope() rotates and appends by the slots
    that it found, and release() gives pages back.  A request that got no pages
    has no request in its slot (n_draft -1) for that step.  draft() draws a
    drafter's tokens, and verify() can filter the target's logits.
    """

    def __init__(self, pcfg: binding.SpecPagedCfg, dcfg: binding.SpecDraftCfg, n_layers: int,
                 device="cuda"):
        if pcfg.T != dcfg.N + 1 or pcfg.B != dcfg.B or pcfg.io_dtype != dcfg.io_dtype:
            raise ValueError("a step needs T = N + 1 and the same B and I/O type on both sides")
        self.pcfg, self.dcfg = pcfg, dcfg
        first = binding.PagedKV.empty(pcfg, device)
        self.page_table, self.kv_len = first.page_table, first.kv_len
        self.caches = [first]
        for _ in range(n_layers - 1):
            e = binding.PagedKV.empty(pcfg, device)
            self.caches.append(binding.PagedKV(pcfg, e.k_pages, e.v_pages, self.page_table,
                                               self.kv_len, e.k_scale, e.v_scale))
        i32 = dict(dtype=torch.int32, device=device)
        self.root_tok = torch.zeros((pcfg.B,), **i32)
        self.n_draft = torch.full((pcfg.B,), dcfg.N, **i32)
        self._n_new = torch.empty((pcfg.B,), **i32)
        dt = torch.bfloat16 if pcfg.io_dtype == binding.SPEC_IO_BF16 else torch.float32
        self.attn_o = torch.empty((n_layers, pcfg.B, pcfg.T, pcfg.Hq, pcfg.D), dtype=dt,
                                  device=device)
        self.out = binding.DraftBuffers(dcfg, device)
        self.paged_ws = binding.alloc_paged_workspace(pcfg, device)
        self.draft_ws = binding.alloc_draft_workspace(dcfg, device)
        self.pool = binding.PagePool.empty(pcfg, self.page_table, self.kv_len, device)
        self.slots = torch.full((pcfg.B, pcfg.T), -1, dtype=torch.int64, device=device)
        self._keep = torch.empty((pcfg.B,), **i32)
        self._q = torch.empty((pcfg.B, pcfg.T, pcfg.Hq, pcfg.D), dtype=dt, device=device)
        self._temperature = torch.empty((pcfg.B,), dtype=torch.float32, device=device)
        # outputs of token_sample, made by the first call that needs them
        self._drafter = self._filtered = None

    def begin(self):
        """Pages for this step's new tokens (n_draft + 1 each); requests that get
        none have n_draft -1 afterwards."""
        torch.add(self.n_draft, 1, out=self._n_new)
        binding.page_tables_extend(self.pcfg, self.pool, self.slots, self._keep, self.paged_ws,
                                   n_new=self._n_new)
        torch.sub(self._keep, 1, out=self.n_draft)

    def attend_rope(self, layer: int, rcfg: binding.SpecRopeCfg, table: binding.RopeTable, q,
                    k_new, v_new):
        """attend() of queries and keys that are not rotated yet, after begin()."""
        torch.add(self.n_draft, 1, out=self._n_new)
        o, kv = self.attn_o[layer], self.caches[layer]
        binding.rope_page_append(rcfg, self.pcfg, kv, table, self.slots, q, k_new, v_new, self._q,
                                 self.paged_ws)
        binding.attn_decode_paged(self.pcfg, kv, self._q, o, self.paged_ws, n_new=self._n_new)
        return o

    def release(self, ended=None):
        """Pages past the committed rows go back to the pool, and all pages of the
        requests where `ended` (bool [B]) is set."""
        if ended is None:
            self._keep.copy_(self.kv_len)
        else:
            torch.where(ended, torch.zeros_like(self.kv_len), self.kv_len, out=self._keep)
        binding.page_tables_trim(self.pcfg, self.pool, self._keep, self.paged_ws)

    def attend(self, layer: int, q, k_new, v_new):
        """Append layer `layer`'s rows and attend from them: [B][T][Hq][D]."""
        torch.add(self.n_draft, 1, out=self._n_new)
        o = self.attn_o[layer]
        kv = self.caches[layer]
        binding.kv_page_append(self.pcfg, kv, k_new, v_new, self.paged_ws, n_new=self._n_new)
        binding.attn_decode_paged(self.pcfg, kv, q, o, self.paged_ws, n_new=self._n_new)
        return o

    def draft(self, i: int, logits, e, draft_tok, draft_prob, **filters):
        """Draft i of every request from a drafter's logits io [B][V] and e f32
        [B][V]: draft_tok [B][N] and draft_prob [B][N][V], as verify() takes them,
        receive the token and the distribution that it was drawn from.  filters:
        temperature, top_k, top_p, min_p [B] as token_sample's.  A slot with n_draft
        -1 is sampled too, since n_draft may be set later, but raises nothing."""
        d = self.dcfg
        cfg = binding.sample_cfg(d.B, d.V, io="bf16" if d.io_dtype else "f32")
        if self._drafter is None:
            self._drafter = binding.SampleBuffers(cfg, prob=True, device=self.kv_len.device)
        out = self._drafter
        binding.token_sample(cfg, logits, e, out, self.draft_ws, last_row=self.n_draft,
                             idle="quiet", **filters)
        draft_tok[:, i].copy_(out.tok)
        draft_prob[:, i].copy_(out.prob)

    def verify(self, logits, draft_tok, draft_prob, u, e, **filters) -> binding.DraftBuffers:
        """Verify the drafts, advance kv_len and root_tok.  filters: top_k, top_p,
        min_p [B] as token_sample's, applied to those of a request's rows that count
        (the first n_draft + 1) at dcfg's temperature."""
        if filters:
            d = self.dcfg
            cfg = binding.sample_cfg(d.B * (d.N + 1), d.V, per=d.N + 1,
                                     io="bf16" if d.io_dtype else "f32")
            if self._filtered is None:
                self._filtered = binding.SampleBuffers(cfg, draw=False, logits=True,
                                                       device=self.kv_len.device)
            out = self._filtered
            # by every call, so that a captured step and others each have their own
            self._temperature.fill_(d.temperature)
            binding.token_sample(cfg, logits.view(cfg.R, cfg.V), None, out, self.draft_ws,
                                 temperature=self._temperature, last_row=self.n_draft, **filters)
            logits = out.logits.view(logits.shape)
        binding.draft_verify_sampled(self.dcfg, draft_tok, draft_prob, logits, u, e, self.out,
                                     self.draft_ws, n_draft=self.n_draft, kv_len=self.kv_len,
                                     root_tok=self.root_tok)
        return self.out

    def status(self) -> int:
        """SPEC_DEV_* bits of the calls so far."""
        return (binding.spec_status_read(self.paged_ws)
                | binding.spec_status_read(self.draft_ws))
