"""What a serving step needs around the paged cache and the chain verification,
as cases to be measured: the page tables of growing and shrinking requests,
rotary positions (alone, and in one pass with the write into the cache's
pages), and sampling with filters from given random numbers.

Where `own` is false, `run` computes the operators from elementary torch
operations (angles, orders and masses in 64 bits, the rest in 32); where it is
true, it calls the library.

Formulas.
  pages     a request with kv_len rows, n_new to come and `held` pages needs
            ceil((kv_len + n_new) / page); what it lacks is taken from the end of
            the free list, in the order (request, column).  Requests that lack
            pages when the running total of what is lacking exceeds the list
            get none.  Row i then has the slot table[pos / page] page + pos % page,
            pos = kv_len + i; -1 where there is no row.  Given back: the columns
            past ceil(keep / page), in the order (request, column).
  rotation  a pair (a, b) of a head's first `rot` values (elements j and
            j + rot/2, or 2j and 2j + 1) becomes amp (a cos t - b sin t,
            a sin t + b cos t), t = pos f_j, f_j = base^(-2j/rot); linear: f_j /
            s; ntk: base s^(rot/(rot-2)) for base; yarn: (1 - g) f_j / s + g f_j
            with g = (orig f_j / 2 pi - 1) / 31 held to [0, 1], amp 0.1 ln s + 1.
            The inverse turns by -t.
  cache     key rows are rotated at kv_len + i; with 8 bits a row x has the scale
            max(amax|x| / 448, 2^-100) (1 for zeros) and codes e4m3(x / scale),
            else it is rounded to the I/O type.
  sampling  w = exp((x - max) / t).  Tokens with x < max + t ln(min_p) leave, of
            the rest all but the first top_k in the order (x descending, index),
            of those the ones with mass before them >= top_p of their sum; the
            first always stays.  p = w / sum over what stays; the token is
            argmax p / e, e exponential and given.
"""
import math

import torch

own = False

IO = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of 256 requests: a few of them need a new page, which is
        # given back as if the step were taken back
        dict(name="pages_decode", op="pages", B=256, T=1, page=64, lo=0, hi=8192, ragged=False,
             scarce=False),
        # prompts of up to 8192 tokens admitted, more of them than there are pages
        dict(name="pages_prompt", op="pages", B=32, T=8192, page=16, lo=0, hi=100, ragged=True,
             scarce=True),
        # the root and 24 drafts of one request at their tree positions
        dict(name="rope_tree_one", op="rope", rows=25, Hq=32, Hkv=8, D=128, rot=128,
             layout="half", io="bf16", inverse=False, far=4200, base=1e6, scaling="none",
             factor=1.0, orig=0),
        # a small fp32 target, part of the head, neighbours paired
        dict(name="rope_f32_part", op="rope", rows=5 * 257, Hq=4, Hkv=4, D=64, rot=32,
             layout="interleaved", io="f32", inverse=False, far=131072, base=1e4,
             scaling="linear", factor=4.0, orig=0),
        # a long prompt's rows turned back, positions beyond the trained length
        dict(name="rope_prompt_back", op="rope", rows=16383, Hq=32, Hkv=8, D=128, rot=128,
             layout="half", io="bf16", inverse=True, far=1000000, base=1e6, scaling="yarn",
             factor=8.0, orig=32768),
        # one new token of each of 24 requests into the 8-bit cache
        dict(name="append_token_e4m3", op="append", B=24, T=1, Hq=32, Hkv=8, D=128, rot=128,
             layout="half", io="bf16", kv="e4m3", page=64, lo=1024, hi=8192, ragged=False,
             fused=True, base=1e6, scaling="none", factor=1.0, orig=0),
        # prompts of up to 4096 tokens, slices of one projection's rows, 8-bit cache
        dict(name="append_prompt_e4m3", op="append", B=4, T=4096, Hq=32, Hkv=8, D=128, rot=64,
             layout="half", io="bf16", kv="e4m3", page=64, lo=1, hi=4000, ragged=True,
             fused=True, base=1e6, scaling="ntk", factor=4.0, orig=0),
        # prompts behind a long prefix, cache in the I/O type
        dict(name="append_prompt_bf16", op="append", B=8, T=2047, Hq=32, Hkv=8, D=128, rot=128,
             layout="interleaved", io="bf16", kv="io", page=128, lo=30000, hi=60000,
             ragged=False, fused=False, base=1e6, scaling="yarn", factor=4.0, orig=16384),
        # one request's next token: nucleus of the 50 best
        dict(name="sample_one", op="sample", R=1, per=1, V=151936, io="bf16", spread=3.0,
             filters="both", outs="tok"),
        # drafts of 24 requests with the distributions they were drawn from
        dict(name="sample_draft_f32", op="sample", R=24, per=1, V=151936, io="f32", spread=3.0,
             filters="mixed", outs="prob"),
        # the target's rows of 24 requests with 8 drafts each, filtered for verification
        dict(name="sample_filter_rows", op="sample", R=216, per=9, V=151936, io="bf16",
             spread=3.0, filters="mixed", outs="logits"),
        # a large batch's next tokens, nucleus of the whole vocabulary
        dict(name="sample_batch_nucleus", op="sample", R=256, per=1, V=151936, io="bf16",
             spread=2.5, filters="top_p", outs="tok"),
    ]


def _log_int(rng, lo, hi):
    """An integer in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "rope", "append", "sample", "sample"])
    if op == "pages":
        T = _log_int(rng, 1, 8192)
        return dict(op=op, B=_log_int(rng, 1, max(2, min(2048, 262144 // T))), T=T,
                    page=rng.choice([16, 32, 64, 128]), lo=0, hi=_log_int(rng, 16, 16384),
                    ragged=rng.random() < 0.7, scarce=rng.random() < 0.4)
    if op == "sample":
        V = _log_int(rng, 1000, 151936)
        R = _log_int(rng, 1, 256)
        outs = rng.choice(["tok", "prob", "logits"])
        return dict(op=op, R=R, per=rng.choice([1, 1, 3, 8]), V=V,
                    io=rng.choice(["bf16", "bf16", "f32"]) if R * V <= 6_000_000 else "bf16",
                    spread=round(rng.uniform(1.0, 4.0), 2),
                    filters=rng.choice(["none", "top_k", "top_p", "min_p", "both", "mixed"]),
                    outs=outs if outs != "prob" or R * V <= 6_000_000 else "tok")
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128, 128])
    scaling = rng.choice(["none", "none", "linear", "ntk", "yarn"])
    c = dict(op=op, Hq=Hkv * rng.choice([1, 2, 3, 4]), Hkv=Hkv, D=D,
             rot=rng.choice([D, D, rng.randrange(16, D + 1, 16)]),
             layout=rng.choice(["half", "interleaved"]), io=rng.choice(["bf16", "bf16", "f32"]),
             base=rng.choice([1e4, 1e6]), scaling=scaling,
             factor=1.0 if scaling == "none" else float(rng.choice([2, 4, 8])),
             orig=rng.choice([4096, 32768]) if scaling == "yarn" else 0)
    if op == "rope":
        c.update(rows=_log_int(rng, 1, 8192), inverse=rng.random() < 0.4,
                 far=_log_int(rng, 64, 1000000))
    else:
        c.update(B=_log_int(rng, 1, 32), page=rng.choice([16, 32, 64, 128]),
                 kv=rng.choice(["io", "e4m3", "e4m3"]), ragged=rng.random() < 0.5,
                 fused=rng.random() < 0.5, lo=0, hi=_log_int(rng, 16, 16384))
        c["T"] = _log_int(rng, 1, max(2, 8192 // c["B"]))
    return c


# ---------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _table(c, g, n_rows, spare):
    """Page tables that hold kv_len rows of each request, the rest on a free list."""
    B, page = c["B"], c["page"]
    kv_len = _ints(g, c["lo"], c["hi"], B)
    held = (kv_len + page - 1) // page
    cols = (c["hi"] + c["T"] + page - 1) // page + 1
    n_pages = B * ((c["hi"] + page - 1) // page) + spare
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    start = held.cumsum(0) - held
    col = torch.arange(cols, device="cuda")
    at = (start.view(B, 1) + col).clamp_max(n_pages - 1)
    table = torch.where(col < held.view(B, 1), ids[at], -1).to(torch.int32)
    used = held.sum()
    free = ids.roll(-int(used))                          # what no request has comes first
    n_new = _ints(g, 0, c["T"], B) if c["ragged"] else None
    return dict(kv_len=kv_len, n_held=held.to(torch.int32), page_table=table.contiguous(),
                free_list=free.contiguous(),
                n_free=(n_pages - used).to(torch.int32).view(1), n_new=n_new)


def _pages(c, seed):
    g = _generator(seed)
    need = c["B"] * (c["T"] // c["page"] + 2)
    s = _table(c, g, c["T"], max(1, need // 3) if c["scarce"] else need)
    s["keep"] = s["kv_len"].clone()
    s["slots"] = torch.empty((c["B"], c["T"]), dtype=torch.int64, device="cuda")
    s["n_ok"] = torch.empty((c["B"],), dtype=torch.int32, device="cuda")
    return s


def _randn(g, shape, io):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(IO[io])


def _rope(c, seed):
    g = _generator(seed)
    n = c["rows"]
    q, k = (_randn(g, (n, c[h], c["D"]), c["io"]) for h in ("Hq", "Hkv"))
    return dict(q=q, k=k, q_out=torch.empty_like(q), k_out=torch.empty_like(k),
                pos=_ints(g, 0, c["far"] - 1, n))


def _append(c, seed):
    g = _generator(seed)
    B, T, Hq, Hkv, D, page = (c[n] for n in ("B", "T", "Hq", "Hkv", "D", "page"))
    s = _table({**c, "T": 0}, g, 0, B * (T // page + 2))
    n_pages = s["free_list"].numel()
    i = torch.arange(T, device="cuda")
    n = s["n_new"] = _ints(g, 0, T, B) if c["ragged"] else torch.full_like(s["kv_len"], T)
    # the pages of the new rows, and the rows' slots
    pos = s["kv_len"].view(B, 1) + i
    col = pos // page - s["n_held"].view(B, 1)
    per = T // page + 2
    new = s["free_list"][torch.arange(B * per, device="cuda")].view(B, per)
    last = s["page_table"].gather(1, (s["n_held"].view(B, 1) - 1).clamp_min(0).long())
    p = torch.where(col < 0, last, new.gather(1, col.clamp_min(0).long()))
    s["slots"] = torch.where(i < n.view(B, 1), p.long() * page + pos % page, -1).contiguous()
    rows = _randn(g, (B, T, (Hq + 2 * Hkv) * D), c["io"])
    parts = [x.unflatten(2, (-1, D)) for x in rows.split([Hq * D, Hkv * D, Hkv * D], 2)]
    s["q"], s["k_new"], s["v_new"] = parts if c["fused"] else [x.contiguous() for x in parts]
    s["q_out"] = torch.zeros((B, T, Hq, D), dtype=IO[c["io"]], device="cuda")
    pool = (n_pages, Hkv, page, D)
    dt = torch.float8_e4m3fn if c["kv"] == "e4m3" else IO[c["io"]]
    s["k_pages"], s["v_pages"] = (torch.zeros(pool, dtype=dt, device="cuda") for _ in "kv")
    s["k_scale"], s["v_scale"] = ((torch.ones(pool[:3], device="cuda") for _ in "kv")
                                  if c["kv"] == "e4m3" else (None, None))
    return s


def _sample(c, seed):
    """Logits of a language model's spread, a likely token or two in each row,
    and the filters that requests ask for."""
    g = _generator(seed)
    R, V = c["R"], c["V"]
    rnd = dict(generator=g, device="cuda", dtype=torch.float32)
    x = c["spread"] * torch.randn((R, V), **rnd)
    top = torch.randint(0, V, (R, 2), generator=g, device="cuda")
    x.scatter_add_(1, top, 4.0 * c["spread"] * torch.rand((R, 2), **rnd))
    s = dict(logits=x.to(IO[c["io"]]))
    del x
    N = (R + c["per"] - 1) // c["per"]
    s["temperature"] = 0.5 + torch.rand((N,), **rnd)
    f = c["filters"]
    some = torch.rand((3, N), **rnd) < (0.6 if f == "mixed" else 1.0)
    k = torch.where(some[0], _ints(g, 10, min(200, V), N), 0)
    p = torch.where(some[1], 0.8 + 0.19 * torch.rand((N,), **rnd), 1.0)
    m = torch.where(some[2], 0.01 + 0.1 * torch.rand((N,), **rnd), 0.0)
    s["top_k"] = k if f in ("top_k", "both", "mixed") else None
    s["top_p"] = p if f in ("top_p", "both", "mixed") else None
    s["min_p"] = m if f in ("min_p", "mixed") else None
    s["e"] = (None if c["outs"] == "logits" else
              (-torch.log1p(-torch.rand((R, V), **rnd))).clamp_min(1e-30))
    return s


def _inputs(c, seed):
    s = {"pages": _pages, "rope": _rope, "append": _append, "sample": _sample}[c["op"]](c, seed)
    s["case"] = c
    return s


def prepare(case, seed):
    s, c = _inputs(case, seed), case
    if own:
        # what a serving program keeps: shapes, the cache's handle, the rotation's
        # table, workspaces
        from speculative_decoding_tree_best_gb300 import binding
        if c["op"] == "sample":
            s["cfg"] = binding.sample_cfg(R=c["R"], V=c["V"], per=c["per"], io=c["io"])
            s["out"] = binding.SampleBuffers(s["cfg"], draw=c["outs"] != "logits",
                                             prob=c["outs"] == "prob",
                                             logits=c["outs"] == "logits")
            s["ws"] = binding.alloc_sample_workspace(s["cfg"])
            return s
        if c["op"] != "pages":
            s["rope"] = binding.rope_table(c["rot"], base=c["base"], scaling=c["scaling"],
                                           factor=c["factor"], orig_len=c["orig"])
            wide = (c["Hq"] + 2 * c["Hkv"]) * c["D"] if c.get("fused") else 0
            strides = dict(q_stride=wide, k_stride=wide, v_stride=wide)
            s["rcfg"] = binding.rope_cfg(rows=c["rows"] if c["op"] == "rope" else c["B"] * c["T"],
                                         Hq=c["Hq"], Hkv=c["Hkv"], D=c["D"], rot=c["rot"],
                                         layout=c["layout"], io=c["io"],
                                         inverse=c.get("inverse", False), **strides)
        if c["op"] != "rope":
            n_pages, cols = s["free_list"].numel(), s["page_table"].shape[1]
            if c["op"] == "pages":
                # the tables are the same for every layer's pool: the smallest one here
                s["cfg"] = binding.paged_cfg(B=c["B"], T=c["T"], Hq=1, Hkv=1, D=64,
                                             page=c["page"], n_pages=n_pages, max_pages=cols)
                s["pool"] = binding.PagePool(s["cfg"], s["page_table"], s["kv_len"],
                                             s["free_list"], s["n_free"], s["n_held"])
            else:
                s["cfg"] = binding.paged_cfg(B=c["B"], T=c["T"], Hq=c["Hq"], Hkv=c["Hkv"],
                                             D=c["D"], page=c["page"], n_pages=n_pages,
                                             max_pages=cols, io=c["io"], kv=c["kv"])
                s["kv"] = binding.PagedKV(s["cfg"], s["k_pages"], s["v_pages"], s["page_table"],
                                          s["kv_len"], s["k_scale"], s["v_scale"])
            s["ws"] = binding.alloc_paged_workspace(s["cfg"])
    return s


# ---------------------------------------------------------------- plain forms

def _plain_pages(s):
    c = s["case"]
    B, T, page = c["B"], c["T"], c["page"]
    table, held, free, n_free = s["page_table"], s["n_held"], s["free_list"], s["n_free"]
    cols = table.shape[1]
    n = s["n_new"] if s["n_new"] is not None else torch.full_like(s["kv_len"], T)
    grow = ((s["kv_len"] + n + page - 1) // page - held).clamp_min(0)
    total = grow.cumsum(0)
    ok = (grow == 0) | (total <= n_free)
    grow = torch.where(ok, grow, 0)
    first = total - grow                          # pages that go to the requests before
    col = torch.arange(cols, device="cuda")
    new = (col >= held.view(B, 1)) & (col < (held + grow).view(B, 1))
    at = n_free - 1 - (first.view(B, 1) + col - held.view(B, 1))
    table.copy_(torch.where(new, free[at.clamp(0, free.numel() - 1)], table))
    held.add_(grow)
    n_free.sub_(grow.sum().view(1).to(torch.int32))
    s["n_ok"].copy_(torch.where(ok, n, 0))
    i = torch.arange(T, device="cuda")
    pos = s["kv_len"].view(B, 1) + i
    p = table.gather(1, (pos // page).clamp_max(cols - 1).long())
    s["slots"].copy_(torch.where(i < s["n_ok"].view(B, 1), p.long() * page + pos % page, -1))
    # given back
    left = torch.minimum(held, (s["keep"] + page - 1) // page)
    back = held - left
    first = back.cumsum(0) - back
    gone = (col >= left.view(B, 1)) & (col < held.view(B, 1))
    at = (n_free + first.view(B, 1) + col - left.view(B, 1)).long()
    free[at[gone]] = table[gone]
    table.masked_fill_(gone, -1)
    n_free.add_(back.sum().view(1).to(torch.int32))
    held.copy_(left)
    s["kv_len"].copy_(torch.minimum(s["kv_len"], s["keep"]))
    return _page_state(s)


def _page_state(s):
    return {n: s[n] for n in ("page_table", "n_held", "free_list", "n_free", "kv_len", "slots",
                              "n_ok")}


def _frequencies(c):
    """f_j and amp, in 64 bits."""
    rot, s = c["rot"], c["factor"]
    base = c["base"] * s ** (rot / (rot - 2)) if c["scaling"] == "ntk" else c["base"]
    j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    f = base ** (-2.0 * j / rot)
    if c["scaling"] == "linear":
        f = f / s
    if c["scaling"] != "yarn":
        return f, 1.0
    g = ((c["orig"] * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return (1 - g) * f / s + g * f, 0.1 * math.log(s) + 1.0


def _turned(x, pos, c):
    """Rows x [..., H, D] at positions pos [...], in fp32."""
    rot, half = c["rot"], c["rot"] // 2
    f, amp = _frequencies(c)
    t = (pos.double().unsqueeze(-1) * f).unsqueeze(-2)
    cos, sin = (amp * t.cos()).float(), (amp * t.sin()).float()
    if c.get("inverse", False):
        sin = -sin
    x = x.float()
    if c["layout"] == "half":
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(s):
    c = s["case"]
    s["q_out"].copy_(_turned(s["q"], s["pos"], c))
    s["k_out"].copy_(_turned(s["k"], s["pos"], c))
    return s["q_out"], s["k_out"]


def _quantise(x):
    """(codes, scales) of fp32 rows [..., D] by the formula above."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax == 0, torch.ones_like(amax), (amax / 448.0).clamp_min(2.0 ** -100))
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn), scale


def _plain_append(s):
    c = s["case"]
    pos = s["kv_len"].view(-1, 1) + torch.arange(c["T"], device="cuda")
    real = s["slots"] >= 0
    s["q_out"].copy_(torch.where(real.unsqueeze(-1).unsqueeze(-1),
                                 _turned(s["q"], pos, c).to(s["q_out"].dtype), s["q_out"]))
    slot = s["slots"][real]
    p, at = slot // c["page"], slot % c["page"]
    k = _turned(s["k_new"][real], pos[real], c)
    v = s["v_new"][real].float()
    if c["kv"] == "e4m3":
        codes, s["k_scale"][p, :, at] = _quantise(k)
        s["k_pages"].view(torch.uint8)[p, :, at] = codes.view(torch.uint8)
        codes, s["v_scale"][p, :, at] = _quantise(v)
        s["v_pages"].view(torch.uint8)[p, :, at] = codes.view(torch.uint8)
    else:
        s["k_pages"][p, :, at] = k.to(s["k_pages"].dtype)
        s["v_pages"][p, :, at] = v.to(s["v_pages"].dtype)
    return _written(s)


def _written(s):
    return {n: s[n] for n in ("q_out", "k_pages", "v_pages", "k_scale", "v_scale")
            if s[n] is not None}


def _per_row(c, x, default):
    """A request's parameter at each of its rows [R][1], in 64 bits."""
    if x is None:
        return torch.full((c["R"], 1), default, dtype=torch.float64, device="cuda")
    return x.double().repeat_interleave(c["per"])[:c["R"]].view(-1, 1)


def _plain_sample(s):
    c = s["case"]
    V = c["V"]
    t, k, p, m = (_per_row(c, s[n], d) for n, d in (("temperature", 1.0), ("top_k", 0.0),
                                                    ("top_p", 1.0), ("min_p", 0.0)))
    x, order = s["logits"].float().sort(dim=-1, descending=True, stable=True)
    x = x.double()
    rank = torch.arange(V, device="cuda")
    kept = ((x >= x[:, :1] + t * torch.log(m)) & ((rank < k) | (k <= 0))) | (rank == 0)
    w = torch.where(kept, torch.exp((x - x[:, :1]) / t), 0.0)
    mass = w.cumsum(-1)
    kept &= (mass - w < p * mass[:, -1:]) | (p >= 1) | (rank == 0)
    w = torch.where(kept, w, 0.0)
    w = w / w.sum(-1, keepdim=True)
    keep = torch.zeros_like(kept).scatter_(1, order, kept)
    if c["outs"] == "logits":
        return {"logits": torch.where(keep, s["logits"], -math.inf)}
    prob = torch.zeros_like(w).scatter_(1, order, w)
    tok = torch.where(keep, prob / s["e"], -1.0).argmax(-1, keepdim=True)
    prob = prob.float()
    out = {"tok": tok.view(-1).to(torch.int32), "tok_prob": prob.gather(1, tok).view(-1)}
    if c["outs"] == "prob":
        out["prob"] = prob
    return out


# ------------------------------------------------------------------------- run

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"pages": _plain_pages, "rope": _plain_rope, "append": _plain_append,
                "sample": _plain_sample}[op](s)
    from speculative_decoding_tree_best_gb300 import binding
    if op == "pages":
        binding.page_tables_extend(s["cfg"], s["pool"], s["slots"], s["n_ok"], s["ws"],
                                   n_new=s["n_new"])
        binding.page_tables_trim(s["cfg"], s["pool"], s["keep"], s["ws"])
        return _page_state(s)
    if op == "rope":
        binding.rope_apply(s["rcfg"], s["rope"], s["pos"], s["q"], s["k"], s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    if op == "append":
        binding.rope_page_append(s["rcfg"], s["cfg"], s["kv"], s["rope"], s["slots"], s["q"],
                                 s["k_new"], s["v_new"], s["q_out"], s["ws"])
        return _written(s)
    out = s["out"]
    binding.token_sample(s["cfg"], s["logits"], s["e"], out, s["ws"],
                         temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                         min_p=s["min_p"])
    if out.logits is not None:
        return {"logits": out.logits}
    got = {"tok": out.tok, "tok_prob": out.tok_prob}
    if out.prob is not None:
        got["prob"] = out.prob
    return got


def work(case):
    """Bytes: each input that is needed once, each output once; sizes that are
    drawn count with their mean."""
    c = case
    if c["op"] == "pages":
        rows = c["B"] * c["T"]
        new = rows / (2 if c["ragged"] else 1) / c["page"]
        return {"bytes": 8 * rows + 28 * c["B"] + 16 * new, "flops": 4.0 * rows}
    b = 2 if c["io"] == "bf16" else 4
    if c["op"] == "sample":
        n = c["R"] * c["V"]
        more = {"tok": 0, "prob": 4, "logits": b}[c["outs"]]
        # the exponentials of what stays are a part of a row where anything filters
        e = 4 if c["filters"] == "none" and c["outs"] != "logits" else 0
        return {"bytes": n * (b + e + more), "flops": 4.0 * n}
    if c["op"] == "rope":
        n = c["rows"] * (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": 2 * n * b + 4 * c["rows"], "flops": 3.0 * n * c["rot"] / c["D"]}
    rows = c["B"] * (c["T"] / 2 if c["ragged"] else c["T"])
    e = 1 + 4 / c["D"] if c["kv"] == "e4m3" else b
    per = c["D"] * (2 * c["Hq"] * b + 2 * c["Hkv"] * (b + e))
    return {"bytes": rows * per + 8 * c["B"] * c["T"],
            "flops": rows * (3.0 * (c["Hq"] + c["Hkv"]) * c["rot"] + 4.0 * c["Hkv"] * c["D"])}


# ----------------------------------------------------------------- in 64 bits

def _angles(c, pos):
    """amp cos t and amp sin t [rows][rot/2] of positions, by the definition."""
    rot, f, amp = c["rot"], [], 1.0
    for j in range(rot // 2):
        base = c["base"]
        if c["scaling"] == "ntk":
            base *= math.exp(math.log(c["factor"]) * rot / (rot - 2))
        x = math.exp(-math.log(base) * 2 * j / rot)
        if c["scaling"] == "linear":
            x /= c["factor"]
        if c["scaling"] == "yarn":
            turns = c["orig"] * x / (2 * math.pi)
            g = min(1.0, max(0.0, (turns - 1) / 31))
            x *= g + (1 - g) / c["factor"]
            amp = 1 + math.log(c["factor"]) / 10
        f.append(x)
    t = torch.outer(pos.double(), torch.tensor(f, dtype=torch.float64, device="cuda"))
    return amp * torch.cos(t), amp * torch.sin(t) * (-1 if c.get("inverse") else 1)


def _exact_turn(x, pos, c):
    """x [rows][H][D] turned, as products with complex numbers."""
    cos, sin = _angles(c, pos)
    z = torch.complex(cos, sin).unsqueeze(1)
    y, half = x.double().clone(), c["rot"] // 2
    a, b = ((y[..., :half], y[..., half:c["rot"]]) if c["layout"] == "half"
            else (y[..., :c["rot"]:2], y[..., 1:c["rot"]:2]))
    w = torch.complex(a, b) * z
    a.copy_(w.real)
    b.copy_(w.imag)
    return y


def _e4m3(x):
    """The nearest e4m3 value (ties to the even one) of |x| <= 448, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_append(s):
    c = s["case"]
    out = {n: x.double() for n, x in _written(s).items()}
    b, i = torch.nonzero(s["slots"] >= 0, as_tuple=True)
    pos, slot = s["kv_len"][b] + i, s["slots"][b, i]
    out["q_out"][b, i] = _exact_turn(s["q"][b, i], pos, c)
    for n, x in (("k", _exact_turn(s["k_new"][b, i], pos, c)), ("v", s["v_new"][b, i].double())):
        if c["kv"] == "e4m3":
            most = x.abs().amax(-1)
            scale = torch.where(most == 0, 1.0, (most / 448).clamp_min(2.0 ** -100))
            out[n + "_scale"][slot // c["page"], :, slot % c["page"]] = scale
            x = _e4m3(x / scale.unsqueeze(-1))
        out[n + "_pages"][slot // c["page"], :, slot % c["page"]] = x
    return out


def _exact_sample(s):
    c = s["case"]
    R, V = c["R"], c["V"]
    get = lambda n, r, d: d if s[n] is None else s[n][r // c["per"]].item()  # noqa: E731
    prob = torch.zeros((R, V), dtype=torch.float64, device="cuda")
    for r in range(R):
        x = s["logits"][r].double()
        t = get("temperature", r, 1.0)
        order = torch.argsort(-x, stable=True)
        y = x[order]
        n, m, p, k = V, get("min_p", r, 0.0), get("top_p", r, 1.0), get("top_k", r, 0)
        if m > 0:
            n = int((y >= y[0] + t * math.log(m)).sum())
        if k > 0:
            n = min(n, k)
        w = torch.exp((y[:max(n, 1)] - y[0]) / t)
        if p < 1:
            below = w.cumsum(0) < p * w.sum()         # the first that is not is the last to stay
            w = w[:min(int(below.sum()) + 1, w.numel())]
        prob[r, order[:w.numel()]] = w / w.sum()
    return prob


def exact(case, seed):
    s, c = _inputs(case, seed), case
    if c["op"] == "pages":
        return None                                        # whole numbers
    if c["op"] == "rope":
        return _exact_turn(s["q"], s["pos"], c), _exact_turn(s["k"], s["pos"], c)
    if c["op"] == "append":
        return _exact_append(s)
    prob = _exact_sample(s)
    if c["outs"] == "logits":
        return {"logits": torch.where(prob > 0, s["logits"].double(), -math.inf)}
    tok = (prob / s["e"].double()).argmax(-1)
    out = {"tok": tok.to(torch.int32), "tok_prob": prob.gather(1, tok.view(-1, 1)).view(-1)}
    if c["outs"] == "prob":
        out["prob"] = prob
    return out
