"""The serving operators beside the tree step, as cases to be measured: a paged
key/value cache that is written and read back in 8 bits (or in the I/O type),
attention of a step's new tokens over that cache, and the verification of a
drafted chain against the target's probabilities.

Where `own` is false, `run` computes the operators from elementary torch
operations in 32 bits; where it is true, it calls the library.

Formulas.  A cache row is one token's key or value of one head, x in R^D.
  8-bit rows      scale = max(amax|x| / 448, 2^-100), 1 for a row of zeros and
                  NaN for a row with a non-finite value; code = e4m3(x / scale)
                  (round to nearest even; NaN code in a NaN row); it stands for
                  code * scale.  Rows in the I/O type are stored as they are.
  attention       row i < n_new[b] of request b sees cache rows
                  [0, kv_len[b] + i]: o = softmax(q K^T / sqrt(D)) V; rows
                  i >= n_new[b] are 0.
  verification    p_i = softmax(logits[b][i] / temperature); draft i is kept
                  while u_i q_i(x_i) < p_i(x_i); at the first draft j that is
                  not kept the token is argmax_v max(0, p_j(v) - q_j(v)) / e(v),
                  with every draft kept it is argmax_v p_n(v) / e(v); u uniform,
                  e exponential, both given.
"""
import math

import torch

own = False

IO = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token of each of 24 requests enters the 8-bit cache
        dict(name="append_token_e4m3", op="append", B=24, T=1, Hq=32, Hkv=8, D=128, page=64,
             cap=1024, lo=100, hi=1000, io="bf16", kv="e4m3", ragged=False),
        # prompts of up to 4096 tokens enter it behind a prefix of odd length
        dict(name="append_prompt_e4m3", op="append", B=4, T=4096, Hq=32, Hkv=8, D=128, page=64,
             cap=8192, lo=1, hi=4000, io="bf16", kv="e4m3", ragged=True),
        # the pages of 8 requests as the contiguous cache of the tree attention
        dict(name="read_e4m3", op="read", B=8, T=1, Hq=32, Hkv=8, D=128, page=64, cap=8256,
             lo=1024, hi=8192, io="bf16", kv="e4m3", ragged=False),
        # one request's pages kept in the I/O type
        dict(name="read_bf16_one", op="read", B=1, T=1, Hq=32, Hkv=8, D=128, page=16, cap=4160,
             lo=4095, hi=4095, io="bf16", kv="io", ragged=False),
        # a small fp32 target, lengths from a single token on
        dict(name="decode_f32_small", op="decode", B=5, T=1, Hq=4, Hkv=4, D=64, page=16, cap=192,
             lo=0, hi=128, io="f32", kv="io", ragged=False),
        # one request at the single workload's length
        dict(name="decode_bf16_one", op="decode", B=1, T=1, Hq=32, Hkv=8, D=128, page=64,
             cap=4160, lo=4096, hi=4096, io="bf16", kv="io", ragged=False),
        # the batched workload's lengths, cache in the I/O type
        dict(name="decode_bf16_batch", op="decode", B=24, T=1, Hq=32, Hkv=8, D=128, page=64,
             cap=8256, lo=1024, hi=8192, io="bf16", kv="io", ragged=False),
        # the same in 8 bits
        dict(name="decode_e4m3_batch", op="decode", B=24, T=1, Hq=32, Hkv=8, D=128, page=64,
             cap=8256, lo=1024, hi=8192, io="bf16", kv="e4m3", ragged=False),
        # the root and up to 7 drafts of each of 8 requests at once
        dict(name="decode_e4m3_drafts", op="decode", B=8, T=8, Hq=32, Hkv=8, D=128, page=64,
             cap=8256, lo=4096, hi=8192, io="bf16", kv="e4m3", ragged=True),
        # long contexts
        dict(name="decode_e4m3_long", op="decode", B=8, T=1, Hq=32, Hkv=8, D=128, page=128,
             cap=131200, lo=131071, hi=131071, io="bf16", kv="e4m3", ragged=False),
        # a chain of 8 drafts of one request over the whole vocabulary
        dict(name="verify_bf16_one", op="verify", B=1, N=8, V=151936, io="bf16", ragged=False,
             temperature=1.0),
        # 24 requests with up to 8 drafts each
        dict(name="verify_bf16_batch", op="verify", B=24, N=8, V=151936, io="bf16", ragged=True,
             temperature=0.7),
    ]


def _log_int(rng, lo, hi):
    """An integer in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "decode", "verify"])
    if op == "verify":
        V = _log_int(rng, 1000, 151936)
        if rng.random() < 0.5:
            V = V // 8 * 8
        return dict(op=op, B=_log_int(rng, 1, 24), N=rng.randint(1, 8), V=V,
                    io=rng.choice(["bf16", "bf16", "f32"]), ragged=rng.random() < 0.5,
                    temperature=round(rng.uniform(0.5, 1.5), 2))
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    c = dict(op=op, B=_log_int(rng, 1, 24), T=1, Hq=Hkv * rng.choice([1, 2, 3, 4, 8]), Hkv=Hkv,
             D=rng.choice([64, 128, 128]), page=page, cap=0, lo=0, hi=0,
             io=rng.choice(["bf16", "bf16", "f32"]), kv=rng.choice(["io", "e4m3", "e4m3"]),
             ragged=rng.random() < 0.5)
    hi = _log_int(rng, 16, 65536 if op == "decode" and c["B"] <= 4 else 8192)
    if op == "append":
        c["T"] = _log_int(rng, 1, 2048)
    elif op == "decode":
        c["T"] = rng.choice([1, 1, 1, 2, 4, 5, 8])
    c["hi"] = hi
    c["lo"] = rng.choice([0, hi // 8, hi])
    c["cap"] = (hi + c["T"] + page - 1) // page * page
    return c


# ---------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _dequant(codes, scale):
    return codes.float() * scale.unsqueeze(-1)


def _quantise(x):
    """(codes, scales) of fp32 rows [..., D] by the formula above."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax == 0, torch.ones_like(amax), (amax / 448.0).clamp_min(2.0 ** -100))
    scale = torch.where(torch.isfinite(amax), scale, torch.full_like(scale, math.nan))
    return (x / scale.unsqueeze(-1)).to(torch.float8_e4m3fn), scale


def _lengths(c, g):
    n = torch.randint(c["lo"], c["hi"] + 1, (c["B"],), generator=g, device="cuda",
                      dtype=torch.int32)
    return n


def _paged(c, seed):
    g = _generator(seed)
    B, T, Hq, Hkv, D, page = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "page"))
    dt = IO[c["io"]]
    cols = c["cap"] // page
    n_pages = B * cols + 1
    s = {"case": c}
    s["page_table"] = torch.randperm(n_pages, generator=g, device="cuda")[:B * cols].to(
        torch.int32).view(B, cols)
    s["kv_len"] = _lengths(c, g)
    s["n_new"] = (torch.randint(1, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
                  if c["ragged"] else None)
    shape = (n_pages, Hkv, page, D)
    for n in ("k", "v"):
        rows = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        if c["kv"] == "e4m3":
            s[n + "_pages"], s[n + "_scale"] = _quantise(rows)
        else:
            s[n + "_pages"], s[n + "_scale"] = rows.to(dt), None
        del rows
    if c["op"] == "append":
        for n in ("k_new", "v_new"):
            s[n] = torch.randn((B, T, Hkv, D), generator=g, device="cuda").to(dt)
    elif c["op"] == "read":
        for n in ("k_out", "v_out"):
            s[n] = torch.zeros((B, c["cap"], Hkv, D), device="cuda", dtype=dt)
    else:
        s["q"] = (2.0 * torch.randn((B, T, Hq, D), generator=g, device="cuda")).to(dt)
        s["o"] = torch.empty((B, T, Hq, D), device="cuda", dtype=dt)
    return s


def _chain(c, seed):
    """Target logits of a language model's spread (a few likely tokens), a
    drafter that knows them up to noise, drafts drawn from the drafter."""
    g = _generator(seed)
    B, N, V, t = c["B"], c["N"], c["V"], c["temperature"]
    rnd = dict(generator=g, device="cuda", dtype=torch.float32)
    z = 3.0 * torch.randn((B, N + 1, V), **rnd)
    s = {"case": c, "logits": z.to(IO[c["io"]])}
    d = (z[:, :N] + 0.7 * torch.randn((B, N, V), **rnd)) / t
    s["draft_prob"] = torch.softmax(d, -1)
    noise = -torch.log(torch.rand((B, N, V), **rnd).clamp_min(1e-30))
    s["draft_tok"] = (d - torch.log(noise.clamp_min(1e-30))).argmax(-1).to(torch.int32)
    s["n_draft"] = (torch.randint(0, N + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
                    if c["ragged"] else None)
    s["u"] = torch.rand((B, N), **rnd)
    s["e"] = (-torch.log1p(-torch.rand((B, V), **rnd))).clamp_min(1e-30)
    return s


def _inputs(c, seed):
    return _chain(c, seed) if c["op"] == "verify" else _paged(c, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        # what a serving program keeps: the shape, the cache's handle, a workspace
        from speculative_decoding_tree_best_gb300 import binding
        c = case
        if c["op"] == "verify":
            s["cfg"] = binding.draft_cfg(B=c["B"], N=c["N"], V=c["V"], io=c["io"],
                                         temperature=c["temperature"])
            s["out"] = binding.DraftBuffers(s["cfg"])
            s["ws"] = binding.alloc_draft_workspace(s["cfg"])
        else:
            s["cfg"] = binding.paged_cfg(B=c["B"], T=c["T"], Hq=c["Hq"], Hkv=c["Hkv"], D=c["D"],
                                         page=c["page"], n_pages=s["k_pages"].shape[0],
                                         max_pages=s["page_table"].shape[1], io=c["io"],
                                         kv=c["kv"])
            s["kv"] = binding.PagedKV(s["cfg"], s["k_pages"], s["v_pages"], s["page_table"],
                                      s["kv_len"], s["k_scale"], s["v_scale"])
            s["ws"] = binding.alloc_paged_workspace(s["cfg"])
    return s


# ---------------------------------------------------------------- plain forms

def _new_rows(s):
    """Where the new tokens' rows go: (request, token, page, slot)."""
    c = s["case"]
    B, T, page = c["B"], c["T"], c["page"]
    i = torch.arange(T, device="cuda").expand(B, T)
    n = s["n_new"] if s["n_new"] is not None else torch.full_like(s["kv_len"], T)
    b, i = torch.nonzero(i < n.view(B, 1), as_tuple=True)
    pos = s["kv_len"][b].long() + i
    return b, i, s["page_table"][b, pos // page].long(), pos % page


def _plain_append(s):
    b, i, p, slot = _new_rows(s)
    for n in ("k", "v"):
        x = s[n + "_new"][b, i].float()
        if s[n + "_scale"] is not None:
            codes, scale = _quantise(x)
            s[n + "_pages"].view(torch.uint8)[p, :, slot] = codes.view(torch.uint8)
            s[n + "_scale"][p, :, slot] = scale
        else:
            s[n + "_pages"][p, :, slot] = x.to(s[n + "_pages"].dtype)
    return _cache(s)


def _cache(s):
    return {n: s[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale") if s[n] is not None}


def _rows(s, n):
    """The requests' rows [B][Hkv][cap][D] in fp32."""
    t = s["page_table"].long()
    x = s[n + "_pages"]
    if s[n + "_scale"] is not None:
        x = _dequant(x.view(torch.uint8)[t].view(torch.float8_e4m3fn), s[n + "_scale"][t])
    else:
        x = x[t].float()
    B, P, H, page, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, P * page, D)


def _plain_read(s):
    L = s["k_out"].shape[1]
    seen = (torch.arange(L, device="cuda") < s["kv_len"].view(-1, 1)).view(-1, L, 1, 1)
    for n in ("k", "v"):
        x = _rows(s, n).transpose(1, 2)[:, :L].to(s[n + "_out"].dtype)
        s[n + "_out"].copy_(torch.where(seen, x, s[n + "_out"]))
    return s["k_out"], s["v_out"]


def _plain_decode(s):
    c = s["case"]
    B, T, Hq, Hkv, D = (c[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    k, v = _rows(s, "k"), _rows(s, "v")
    L = k.shape[2]
    n = s["n_new"] if s["n_new"] is not None else torch.full_like(s["kv_len"], T)
    i = torch.arange(T, device="cuda")
    limit = torch.where(i < n.view(B, 1), s["kv_len"].view(B, 1) + i + 1, 0)        # [B][T]
    seen = torch.arange(L, device="cuda") < limit.view(B, T, 1)                       # [B][T][L]
    seen = seen.view(B, 1, T, 1, L).expand(B, 1, T, G, L).reshape(B, 1, T * G, L)
    q = s["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    x = (q @ k.transpose(2, 3)) / math.sqrt(D)
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    tot = w.sum(-1, keepdim=True)
    v = torch.where(seen.any(2).unsqueeze(-1), v, 0.0)
    o = torch.where(tot == 0, 0.0, (w @ v) / tot)
    o = o.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    s["o"].copy_(o)
    return s["o"]


def _verify(logits, draft_prob, draft_tok, n, u, e, t):
    """The rule in the precision of its arguments."""
    B, N1, V = logits.shape
    N = N1 - 1
    z = logits / t
    z = torch.exp(z - z.amax(-1, keepdim=True))
    p = z / z.sum(-1, keepdim=True)
    x = draft_tok.long().unsqueeze(-1)
    px = p[:, :N].gather(2, x).squeeze(-1)
    qx = draft_prob.gather(2, x).squeeze(-1)
    i = torch.arange(N, device=logits.device)
    real = i < n.view(B, 1)
    keep = (u * qx < px) & real
    kept = keep.long().cumprod(1).sum(1)                                             # [B]
    row = p.gather(1, kept.view(B, 1, 1).expand(B, 1, V)).squeeze(1)
    q = draft_prob.gather(1, kept.clamp_max(N - 1).view(B, 1, 1).expand(B, 1, V)).squeeze(1)
    rest = (row - q).clamp_min(0)
    rest = torch.where((kept < n).view(B, 1) & (rest.amax(-1, keepdim=True) > 0), rest, row)
    last = (rest / e).argmax(-1)
    j = torch.arange(N + 1, device=logits.device)
    pad = torch.cat([draft_tok.long(), draft_tok.new_zeros((B, 1)).long()], 1)
    tok = torch.where(j < kept.view(B, 1), pad, torch.where(j == kept.view(B, 1),
                                                            last.view(B, 1), -1))
    return {"accept_len": (kept + 1).to(torch.int32), "out_tok": tok.to(torch.int32),
            "target_prob": torch.where(real, px, 0.0)}


def _counts(s):
    c = s["case"]
    if s["n_draft"] is not None:
        return s["n_draft"]
    return torch.full((c["B"],), c["N"], device="cuda", dtype=torch.int32)


def _plain_verify(s):
    return _verify(s["logits"].float(), s["draft_prob"], s["draft_tok"], _counts(s), s["u"],
                   s["e"], s["case"]["temperature"])


# ------------------------------------------------------------------------- run

def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "decode": _plain_decode,
                "verify": _plain_verify}[op](s)
    from speculative_decoding_tree_best_gb300 import binding
    if op == "append":
        binding.kv_page_append(s["cfg"], s["kv"], s["k_new"], s["v_new"], s["ws"],
                               n_new=s["n_new"])
        return _cache(s)
    if op == "read":
        binding.kv_page_read(s["cfg"], s["kv"], s["k_out"], s["v_out"], s["ws"])
        return s["k_out"], s["v_out"]
    if op == "decode":
        binding.attn_decode_paged(s["cfg"], s["kv"], s["q"], s["o"], s["ws"], n_new=s["n_new"])
        return s["o"]
    out = s["out"]
    binding.draft_verify_sampled(s["cfg"], s["draft_tok"], s["draft_prob"], s["logits"], s["u"],
                                 s["e"], out, s["ws"], n_draft=s["n_draft"])
    return {"accept_len": out.accept_len, "out_tok": out.out_tok, "target_prob": out.target_prob}


def work(case):
    """Bytes: each cache row that a request has, each logits row, each input
    once; sizes that are drawn count with their mean."""
    c = case
    b = 2 if c["io"] == "bf16" else 4
    if c["op"] == "verify":
        rows = c["B"] * ((c["N"] / 2 if c["ragged"] else c["N"]) + 1)
        # every logits row; the exponentials, and a drafter row where one is refused
        return {"bytes": rows * c["V"] * b + c["B"] * c["V"] * 8, "flops": 4.0 * rows * c["V"]}
    e = 1 + 4 / c["D"] if c["kv"] == "e4m3" else b           # bytes of a cached value
    per = 2 * c["Hkv"] * c["D"]                               # key and value of a token
    new = (c["T"] + 1) / 2 if c["ragged"] else c["T"]
    held = c["B"] * (c["lo"] + c["hi"]) / 2
    if c["op"] == "append":
        n = c["B"] * new * per
        return {"bytes": n * (b + e), "flops": 2.0 * n}
    if c["op"] == "read":
        return {"bytes": held * per * (b + e), "flops": held * per}
    seen = held + c["B"] * new
    return {"bytes": seen * per * e + 2 * c["B"] * c["T"] * c["Hq"] * c["D"] * b,
            "flops": 4.0 * seen * new * c["Hq"] * c["D"]}


# ----------------------------------------------------------------- in 64 bits

def _e4m3(x):
    """The nearest e4m3 value (ties to the even one) of |x| <= 448, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s, c = _inputs(case, seed), case
    B, page = c["B"], c.get("page", 1)
    if c["op"] == "verify":
        return _exact_verify(s)
    n_new = (s["n_new"] if s["n_new"] is not None else torch.full_like(s["kv_len"], c["T"])).tolist()
    kv_len, table = s["kv_len"].tolist(), s["page_table"].long()
    if c["op"] == "append":
        out = {n: x.double() for n, x in _cache(s).items()}
        for b in range(B):
            pos = kv_len[b] + torch.arange(n_new[b], device="cuda")
            p, slot = table[b, pos // page], pos % page
            for n in ("k", "v"):
                x = s[n + "_new"][b, :n_new[b]].double()
                if c["kv"] == "e4m3":
                    scale = (x.abs().amax(-1) / 448).clamp_min(2.0 ** -100)
                    scale = torch.where(x.abs().amax(-1) == 0, 1.0, scale)
                    out[n + "_scale"][p, :, slot] = scale
                    x = _e4m3(x / scale.unsqueeze(-1))
                out[n + "_pages"][p, :, slot] = x
        return out

    def rows(n, b, count):
        pos = torch.arange(count, device="cuda")
        p, slot = table[b, pos // page], pos % page
        if c["kv"] == "e4m3":
            x = s[n + "_pages"].view(torch.uint8)[p, :, slot].view(torch.float8_e4m3fn).double()
            return x * s[n + "_scale"][p, :, slot].double().unsqueeze(-1)
        return s[n + "_pages"][p, :, slot].double()          # [count][Hkv][D]

    if c["op"] == "read":
        out = [s["k_out"].double(), s["v_out"].double()]
        for b in range(B):
            for o, n in zip(out, ("k", "v")):
                o[b, :kv_len[b]] = rows(n, b, kv_len[b])
        return tuple(out)
    G = c["Hq"] // c["Hkv"]
    o = torch.zeros(s["o"].shape, device="cuda", dtype=torch.float64)
    for b in range(B):
        k, v = (rows(n, b, kv_len[b] + n_new[b]).transpose(0, 1) for n in ("k", "v"))
        for i in range(n_new[b]):
            end = kv_len[b] + i + 1
            q = s["q"][b, i].double().view(c["Hkv"], G, c["D"])
            w = torch.softmax(torch.einsum("hgd,hld->hgl", q, k[:, :end]) / c["D"] ** 0.5, -1)
            o[b, i] = torch.einsum("hgl,hld->hgd", w, v[:, :end]).reshape(c["Hq"], c["D"])
        del k, v
    return o


def _exact_verify(s):
    c = s["case"]
    B, N, V = c["B"], c["N"], c["V"]
    n = _counts(s).tolist()
    drafts = s["draft_tok"].tolist()
    lens, toks = [], []
    prob = torch.zeros((B, N), device="cuda", dtype=torch.float64)
    for b in range(B):
        p = torch.softmax(s["logits"][b].double() / c["temperature"], -1)
        q = s["draft_prob"][b].double()
        kept, going = 0, True
        for i in range(n[b]):
            x = drafts[b][i]
            prob[b, i] = p[i, x]
            going = going and bool(s["u"][b, i].double() * q[i, x] < p[i, x])
            kept += going
        w = p[kept]
        if kept < n[b]:
            w = (p[kept] - q[kept]).clamp_min(0)
        last = int((w / s["e"][b].double()).argmax())
        lens.append(kept + 1)
        toks.append(drafts[b][:kept] + [last] + [-1] * (N - kept))
    return {"accept_len": torch.tensor(lens, dtype=torch.int32),
            "out_tok": torch.tensor(toks, dtype=torch.int32), "target_prob": prob}
