"""Plain 64-bit (or whole-number) forms of the calls around a serving step, for
tests: page tables, rotary positions, filtered sampling."""
import math

import numpy as np


# ------------------------------------------------------------------- page tables

def extend(s, page, n_new, T):
    """One page_tables_extend on a dict of numpy arrays (page_table, kv_len,
    free_list, n_free, n_held), request by request.  Returns (slots, n_ok)."""
    B, cols = s["page_table"].shape
    slots = np.full((B, T), -1, np.int64)
    n_ok = np.zeros(B, np.int32)
    free = int(s["n_free"][0])
    lacking, taken = 0, 0
    for b in range(B):
        n, L, H = int(min(max(n_new[b], 0), T)), int(s["kv_len"][b]), int(s["n_held"][b])
        if L < 0 or L + n > cols * page or H < 0 or H > cols:
            continue
        grow = max(0, -(-(L + n) // page) - H) if n else 0
        lacking += grow
        if grow and lacking > free:
            continue
        for c in range(H, H + grow):
            taken += 1
            s["page_table"][b, c] = s["free_list"][free - taken]
        s["n_held"][b] = H + grow
        n_ok[b] = n
        for i in range(n):
            slots[b, i] = int(s["page_table"][b, (L + i) // page]) * page + (L + i) % page
    s["n_free"][0] = free - taken
    return slots, n_ok


def trim(s, page, keep):
    for b in range(len(keep)):
        k, H = int(keep[b]), int(s["n_held"][b])
        if k < 0:
            continue
        left = min(H, -(-k // page))
        for c in range(left, H):
            s["free_list"][s["n_free"][0]] = s["page_table"][b, c]
            s["n_free"][0] += 1
            s["page_table"][b, c] = -1
        s["n_held"][b] = left
        s["kv_len"][b] = min(int(s["kv_len"][b]), k)


# --------------------------------------------------------------- rotary positions

def frequencies(rot, base, scaling="none", factor=1.0, orig_len=0, beta_fast=32.0, beta_slow=1.0):
    """(f_j, amp)."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * j / rot) for j in range(rot // 2)])
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        turns = orig_len * f / (2 * math.pi)
        g = np.clip((turns - beta_slow) / (beta_fast - beta_slow), 0, 1)
        return (1 - g) * f / factor + g * f, 0.1 * math.log(factor) + 1
    return f, 1.0


def rotate(x, pos, f, amp, layout, inverse=False):
    """x [rows][H][D] in 64 bits at pos [rows]."""
    y, half, rot = np.array(x, np.float64), len(f), 2 * len(f)
    t = (np.asarray(pos, np.float64)[:, None] * f)[:, None, :] * (-1 if inverse else 1)
    cos, sin = amp * np.cos(t), amp * np.sin(t)
    a, b = ((slice(0, half), slice(half, rot)) if layout == "half"
            else (slice(0, rot, 2), slice(1, rot, 2)))
    p, q = y[..., a].copy(), y[..., b].copy()
    y[..., a] = p * cos - q * sin
    y[..., b] = p * sin + q * cos
    return y


# ---------------------------------------------------------------------- sampling

def sample(x, t=1.0, k=0, p=1.0, m=0.0):
    """What stays of a row of logits: (probabilities, the order's length kept, how
    near (relative) the nearest border of top_p is)."""
    x = np.asarray(x, np.float64)
    order = np.lexsort((np.arange(x.size), -x))
    y = x[order]
    n = int((y > -np.inf).sum())
    if m > 0:
        n = int((y[:n] >= (y[0] if m >= 1 else y[0] + t * math.log(m))).sum())
    if t == 0:
        n = 1
    if k > 0:
        n = min(n, k)
    n = max(n, 1)
    if t > 0:
        with np.errstate(over="ignore"):
            w = np.exp((y[:n] - y[0]) / t)
    else:
        w = np.ones(1)
    margin = math.inf
    if p < 1:
        mass = np.cumsum(w)
        before = np.concatenate([[0.0], mass[:-1]])
        inside = before < p * mass[-1]
        inside[0] = True
        margin = float(np.abs(before[1:] / mass[-1] - p).min()) if n > 1 else math.inf
        n = int(inside.sum())
        w = w[:n]
    out = np.zeros(x.size)
    out[order[:n]] = w / w.sum()
    return out, n, margin
