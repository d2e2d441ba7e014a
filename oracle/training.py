"""The training operators in 64 bits, from their definitions, in numpy: group
norm + activation, bias + dropout + residual, and the router's balance loss,
with their gradients. Shares no code with the library."""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])
K0, K1 = 0.79788456, 0.044715


def act(z: np.ndarray, name: str) -> np.ndarray:
    if name == "none":
        return z
    if name == "silu":
        return z * 0.5 * (1 + np.tanh(z / 2))
    if name == "gelu":
        return 0.5 * z * (1 + _erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(K0 * (z + K1 * z**3)))
    raise ValueError(name)


def act_grad(z: np.ndarray, name: str) -> np.ndarray:
    if name == "none":
        return np.ones_like(z)
    if name == "silu":
        q = 0.5 * (1 + np.tanh(z / 2))
        return q + z * q * (1 - q)
    if name == "gelu":
        return 0.5 * (1 + _erf(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = np.tanh(K0 * (z + K1 * z**3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * K0 * (1 + 3 * K1 * z * z)
    raise ValueError(name)


def groupnorm_stats(x: np.ndarray, groups: int, eps: float) -> np.ndarray:
    """(B, groups, 2): mean and 1 / sqrt(var + eps) of (B, S, C)."""
    B, S, C = x.shape
    v = x.astype(np.float64).reshape(B, S, groups, C // groups)
    mean = v.mean(axis=(1, 3))
    var = ((v - mean[:, None, :, None]) ** 2).mean(axis=(1, 3))
    return np.stack([mean, 1 / np.sqrt(var + eps)], axis=2)


def _per_channel(stats: np.ndarray, C: int) -> tuple:
    L = C // stats.shape[1]
    return tuple(np.repeat(stats[:, None, :, k], L, axis=2) for k in (0, 1))


def groupnorm_act(x, groups, w=None, b=None, eps=1e-5, name="silu", stats=None) -> np.ndarray:
    x = x.astype(np.float64)
    stats = groupnorm_stats(x, groups, eps) if stats is None else stats
    mean, rstd = _per_channel(stats, x.shape[2])
    z = (x - mean) * rstd
    if w is not None:
        z = z * w
    if b is not None:
        z = z + b
    return act(z, name)


def groupnorm_act_backward(x, dy, groups, w=None, b=None, eps=1e-5, name="silu"):
    """(dx, dw, db, size, (size_w, size_b)): the gradients, and the sums of the
    magnitudes that each adds up, which rounding errors are relative to (act' is
    at most 1.13, and taken as 1)."""
    B, S, C = x.shape
    x, dy = x.astype(np.float64), dy.astype(np.float64)
    w = np.ones(C) if w is None else w.astype(np.float64)
    b = np.zeros(C) if b is None else b.astype(np.float64)
    mean, rstd = _per_channel(groupnorm_stats(x, groups, eps), C)
    xh = (x - mean) * rstd
    dz = dy * act_grad(xh * w + b, name)
    dxh = dz * w

    def group_mean(v):
        m = v.reshape(B, S, groups, C // groups).mean(axis=(1, 3))
        return np.repeat(m[:, None, :], C // groups, axis=2)

    dx = rstd * (dxh - group_mean(dxh) - xh * group_mean(dxh * xh))
    size = rstd * (np.abs(dy * w) + group_mean(np.abs(dy * w)) + np.abs(xh) * group_mean(np.abs(dy * w * xh)))
    sums = (np.abs(dy * xh).sum(axis=(0, 1)), np.abs(dy).sum(axis=(0, 1)))
    return dx, (dz * xh).sum(axis=(0, 1)), dz.sum(axis=(0, 1)), size, sums


def philox4x32_10(counter, key) -> np.ndarray:
    """Philox4x32-10 (Salmon, Moraes, Dror and Shaw, SC 2011) of an (..., 4)
    array of counters and a key of two words."""
    c = np.asarray(counter, dtype=np.uint64)
    k = [int(v) for v in key]
    low = np.uint64(0xFFFFFFFF)
    c = [c[..., i] for i in range(4)]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=-1)


def dropout_steps(p: float) -> int:
    """round(65536 p) of the fp32 p, the probability's held form."""
    return int(np.rint(np.float64(np.float32(p)) * 65536))


def dropout_keep(rows, N: int, p: float, seed: int, offset: int) -> np.ndarray:
    """Where the mask keeps: (len(rows), N) of the given row numbers."""
    rows = np.asarray(rows, dtype=np.uint64)
    blocks = (N + 7) // 8
    offset %= 1 << 64
    seed %= 1 << 64
    c = np.zeros((len(rows), blocks, 4), dtype=np.uint64)
    c[..., 0] = np.arange(blocks, dtype=np.uint64)[None, :]
    c[..., 1] = rows[:, None]
    c[..., 2], c[..., 3] = offset & 0xFFFFFFFF, offset >> 32
    q = philox4x32_10(c, (seed & 0xFFFFFFFF, seed >> 32))
    half = np.stack([q & np.uint64(0xFFFF), q >> np.uint64(16)], axis=-1)  # low, high half of every word
    return half.reshape(len(rows), -1)[:, :N] >= np.uint64(dropout_steps(p))


def dropout_scale(p: float) -> float:
    q = dropout_steps(p)
    return 65536 / (65536 - q) if q < 65536 else 0.0


def bias_dropout_residual(x, residual, bias, keep, p) -> np.ndarray:
    v = x.astype(np.float64)
    if bias is not None:
        v = v + bias
    v = np.where(keep, v * dropout_scale(p), 0.0)
    return v if residual is None else v + residual


def _softmax(logits: np.ndarray) -> np.ndarray:
    v = logits.astype(np.float64)
    m = v.max(axis=1, keepdims=True)
    m = np.where(m == -np.inf, 0.0, m)
    e = np.exp(v - m)
    s = e.sum(axis=1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s != 0)


def router_balance_loss(logits, experts, coef, mask=None):
    """(loss, counts): counts (E + 1,), the last of them the rows that take part."""
    T, E = logits.shape
    mask = np.ones(T, dtype=bool) if mask is None else mask.astype(bool)
    chosen = experts[mask].reshape(-1)
    chosen = chosen[(chosen >= 0) & (chosen < E)]
    n = int(mask.sum())
    counts = np.append(np.bincount(chosen, minlength=E), n).astype(np.int64)
    if n == 0:
        return 0.0, counts
    P = _softmax(logits[mask]).sum(axis=0) / n
    return coef * E * float((counts[:E] / (n * experts.shape[1]) * P).sum()), counts


def router_balance_loss_backward(logits, counts, top_k, dloss, coef, mask=None):
    """(dlogits, scale): the gradient, and the magnitudes that it is the difference of."""
    T, E = logits.shape
    n = int(counts[E])
    mask = np.ones(T, dtype=bool) if mask is None else mask.astype(bool)
    if n == 0:
        return np.zeros((T, E)), np.zeros((T, E))
    p = np.zeros((T, E))
    p[mask] = _softmax(logits[mask])
    c = counts[:E] - counts[:E].mean()
    k = dloss * coef * E / (n * n * top_k)
    d = k * p * (c - (p * c).sum(axis=1, keepdims=True))
    return d, abs(k) * p * (np.abs(c) + (p * np.abs(c)).sum(axis=1, keepdims=True))
