"""The serving operators in 64 bits, from their definitions, in numpy: RMSNorm with
an 8-bit result, attention of one token over a paged cache, and sampling. Shares no
code with the library."""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def rmsnorm(s: np.ndarray, w, eps: float) -> np.ndarray:
    s = s.astype(np.float64)
    y = s / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return y if w is None else y * w.astype(np.float64)


def quant_scales(y: np.ndarray, group: int) -> np.ndarray:
    """(M, groups) scales of y's rows, one for every `group` columns (0: one a row)."""
    M, N = y.shape
    group = group or N
    starts = np.arange(0, N, group)
    top = np.maximum.reduceat(np.abs(y), starts, axis=1)
    return np.maximum(top / E4M3_MAX, 2.0**-126)


def e4m3_half_step(v: np.ndarray) -> np.ndarray:
    """The most that rounding v (at most 448) to e4m3 moves it: 3 bits behind the
    leading one, exponents from -6 on."""
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0**-6)))
    return np.exp2(e - 4)


def paged_attention(q, k, v, table, lengths, scale, window=0):
    """(out, lse, size, steps): size is sum p |v|, and steps the largest |scale| sum
    |q k| of a head, which rounding errors are relative to. k, v: (pages, slots,
    kv_heads, D)."""
    B, H, D = q.shape
    pages, page, K, _ = k.shape
    out, size = np.zeros((B, H, D)), np.zeros((B, H, D))
    lse, steps = np.full((B, H), -np.inf), np.zeros((B, H))
    for b in range(B):
        n = int(lengths[b])
        if n > table.shape[1] * page:
            out[b], lse[b] = np.nan, np.nan
            continue
        first = max(0, n - window) if window else 0
        if n <= first:
            continue
        at = np.arange(first, n)
        where = table[b, at // page].astype(np.int64)
        if np.any((where < 0) | (where >= pages)):
            out[b], lse[b] = np.nan, np.nan
            continue
        for h in range(H):
            kk = k[where, at % page, h // (H // K)].astype(np.float64)
            vv = v[where, at % page, h // (H // K)].astype(np.float64)
            qq = q[b, h].astype(np.float64)
            s = kk @ qq * scale
            m = s.max()
            if m == -np.inf:
                continue
            p = np.exp(s - m)
            lse[b, h] = m + math.log(p.sum())
            out[b, h] = p @ vv / p.sum()
            size[b, h] = p @ np.abs(vv) / p.sum()
            steps[b, h] = (np.abs(kk) @ np.abs(qq)).max() * abs(scale)
    return out, lse, size, steps


def sample_row(x: np.ndarray, u: float, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, margin) of one row: margin is how near the nearest decision was
    to its border, as a relative error of the weights that could turn it (with 2^-17 of
    the largest for each column's absolute error)."""
    x = x.astype(np.float64)
    n = len(x)
    if np.isnan(x).any() or x.max() == -np.inf:
        return -1, np.nan, np.inf
    m = x.max()
    if not temperature > 0:
        return int(np.argmax(x == m)), 0.0, np.inf
    with np.errstate(invalid="ignore"):
        w = np.where(x == m, 1.0, np.exp((x - m) / temperature))
    order = np.lexsort((np.arange(n), -x))  # the largest first, equal ones by index
    keep = n
    margin = np.inf

    def distance(mass, part):
        """Of the running sums `mass` from the part `part` of the last of them."""
        total = mass[-1]
        weighed = abs(1 - part) * mass + part * (total - mass) + n * 2.0**-17
        return float((np.abs(mass - part * total) / weighed).min())

    if 0 < top_k < n:
        keep = top_k
    if top_p < 1:
        mass = np.cumsum(w[order[:keep]])
        goal = top_p * mass[-1]
        margin = min(margin, distance(mass, top_p))
        keep = min(keep, 1 + int((mass[:-1] < goal).sum()))
    if min_p > 0:
        keep = min(keep, int((w >= min_p).sum()))
    kept = np.sort(order[:keep])
    mass = np.cumsum(w[kept])
    goal = u * mass[-1]
    margin = min(margin, distance(mass, u) if keep > 1 else np.inf)
    j = min(int((mass <= goal).sum()), keep - 1)
    while w[kept[j]] == 0:
        j -= 1
    token = int(kept[j])
    return token, (0.0 if x[token] == m else (x[token] - m) / temperature) - math.log(mass[-1]), margin
