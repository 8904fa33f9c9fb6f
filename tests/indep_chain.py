"""Plain 64-bit implementations of the paged cache, the attention over it and
the drafted chain's verification, written from their definitions with numpy
(no code shared with the library or with the oracle)."""
from __future__ import annotations

import numpy as np

E4M3_MAX, FLOOR = 448.0, 2.0 ** -100


def bf16(x):
    """fp32 values rounded to bfloat16 (nearest even), as fp32; NaN stays NaN."""
    x = np.asarray(x, np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    return np.where(np.isnan(x), np.float32(np.nan), r.view(np.float32))


def e4m3(x):
    """The nearest e4m3 value of |x| <= 448 (ties to the even mantissa)."""
    x = np.asarray(x, np.float64)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.round(x / step) * step


def quantise(x):
    """(values of the codes, scales) of fp32 rows [..., D]: the scale and the
    quotient are fp32 divisions, the code the quotient's nearest e4m3 value."""
    x = np.asarray(x, np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        amax = np.abs(x).max(-1)
        scale = np.maximum(amax / np.float32(E4M3_MAX), np.float32(FLOOR)).astype(np.float32)
        scale = np.where(amax == 0, np.float32(1), scale)
        scale = np.where(np.isfinite(x).all(-1), scale, np.float32(np.nan)).astype(np.float32)
        y = (x / scale[..., None]).astype(np.float32)
        return e4m3(np.where(np.isnan(y), 0, y)) + np.where(np.isnan(y), np.nan, 0.0), scale


def place(cfg, table, kv_len, n_new):
    """[(b, i, page, slot)] of the new rows that are written."""
    out = []
    cap = cfg.page * cfg.max_pages
    for b in range(cfg.B):
        if kv_len[b] < 0 or kv_len[b] + n_new[b] > cap:
            continue
        for i in range(n_new[b]):
            pos = kv_len[b] + i
            p = table[b][pos // cfg.page]
            if 0 <= p < cfg.n_pages:
                out.append((b, i, int(p), int(pos % cfg.page)))
    return out


def attention(q, k, v, seen):
    """q [R][D], k, v [L][D], seen [R][L] bool -> (o [R][D], mean |v| [R][D],
    largest sum |q k| / sqrt(D) over the seen keys [R]); float64."""
    R, D = q.shape
    o, a, z = np.zeros((R, D)), np.zeros((R, D)), np.zeros(R)
    for r in range(R):
        j = np.flatnonzero(seen[r])
        if not len(j):
            continue
        with np.errstate(invalid="ignore"):
            s = (k[j] @ q[r]) / np.sqrt(D)
            w = np.exp(s - s.max())
            w = w / w.sum()
            o[r], a[r] = w @ v[j], w @ np.abs(v[j])
            z[r] = (np.abs(k[j]) @ np.abs(q[r])).max() / np.sqrt(D)
    return o, a, z


def softmax(x):
    with np.errstate(invalid="ignore"):
        e = np.exp(x - x.max(-1, keepdims=True))
        return e / e.sum(-1, keepdims=True)


def chain(logits, q, toks, u, e, t):
    """One request: (kept, token, target probabilities, margin): the margin is
    the smallest relative distance of a decision from its border."""
    p = softmax(np.asarray(logits, np.float64) / t)
    n, kept, margin = len(toks), 0, np.inf
    probs = np.array([p[i, x] for i, x in enumerate(toks)])
    for i, x in enumerate(toks):
        lhs = float(u[i]) * (1.0 if q is None else float(q[i, x]))
        margin = min(margin, abs(lhs - p[i, x]) / max(lhs, p[i, x]))
        if not lhs < p[i, x]:
            break
        kept += 1
    w = p[kept]
    slack = 0.0
    if kept < n:
        qr = np.zeros(len(w)) if q is None else np.asarray(q[kept], np.float64).copy()
        if q is None:
            qr[toks[kept]] = 1.0
        rest = np.maximum(w - qr, 0)
        slack = np.maximum(w, qr)                     # what a difference's rounding goes by
        w = rest if rest.max() > 0 else w
    score = w / np.asarray(e, np.float64)
    best = int(np.argmax(score))
    err = (slack if kept < n else w) / np.asarray(e, np.float64)
    gap = (score[best] - np.delete(score, best)) / np.maximum(err[best], np.delete(err, best))
    if len(gap):
        margin = min(margin, float(gap.min()))
    return kept, best, probs, margin
