"""The decode operators around the expert step in 64 bits with numpy: the
rotation and append, attention over pages with a shared prefix, the choice of
a token.  Written from the formulas in include/qexpert.h, one row at a time."""
import math

import numpy as np

U32 = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25}  # half the distance of the smallest values


def rotate(x, pos, inv_freq, axis, adjacent):
    """x [T, H, D], pos [axes, T] -> x turned, and the bound's scale |u| + |v| of each element."""
    x = x.astype(np.float64)
    y, size = x.copy(), np.zeros_like(x)
    half = len(inv_freq)
    for i in range(half):
        t = pos[axis[i]].astype(np.float64) * np.float64(inv_freq[i])
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
        size[:, :, a] = size[:, :, b] = np.abs(x[:, :, a]) + np.abs(x[:, :, b])
    return y, size


def gather(pages, page_size, list_, n, h):
    """Keys (or values) 0 .. n-1 of head h on the pages list_, [n, D]."""
    j = np.arange(n)
    return pages[np.asarray(list_, np.int64)[j // page_size], h, j % page_size] if n else np.zeros((0, pages.shape[3]))


def attend(q, k, v, scale, dtype):
    """One key head: q [G, D], k, v [n, D] (float64) -> out, lse and bounds on
    a kernel that keeps scores and sums in fp32 and rounds the softmax's
    numerators and the result to `dtype`.

    Score: products of 16-bit numbers are exact in fp32; D additions, each off
    by at most a unit in the last place (2 U32, the tensor cores may cut instead of
    round), one product with scale log2(e) (itself rounded) and one subtraction:
    ds = 2 (D + 2) U32 scale sum |q k| + 4 U32 |s|.  A numerator is off by ds, by
    2^-22 of exp2f, by half a step of dtype relative, or TINY absolute; sums of n
    terms, rescaled at most once a tile and joined over chunks, add (n + 64) 2 U32.
    The denominator is off alike, without dtype's rounding; one division and the
    rounding of the result follow.
    """
    g, n = q.shape[0], k.shape[0]
    if n == 0:
        return np.zeros((g, v.shape[1])), np.full(g, -np.inf), np.zeros((g, v.shape[1])), np.zeros(g)
    s = scale * (q @ k.T)
    size = abs(scale) * (np.abs(q) @ np.abs(k).T)
    ds = (2 * (q.shape[1] + 2) * U32 * size + 4 * U32 * np.abs(s)).max(axis=1)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(axis=1, keepdims=True)
    out = p @ v / total
    lse = (m + np.log(total))[:, 0]
    sums = (n + 64) * 2 * U32 + 4 * U32
    mag = p @ np.abs(v) / total
    num = (HALF_STEP[dtype] + 2.0 ** -22 + ds + sums)[:, None] * mag + TINY[dtype] * np.abs(v).sum(axis=0)[None, :] / total
    den = (2.0 ** -22 + ds + sums)[:, None] * np.abs(out)
    tol = (num + den) * 1.05 + HALF_STEP[dtype] * (np.abs(out) + num + den) + TINY[dtype]
    return out, lse, tol, 1.05 * (2.0 ** -22 + ds + sums) + 4 * U32 * np.abs(lse) + 4 * U32


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob) of one row of logits (float64)."""
    x = np.where(np.isnan(x), -np.inf, x)
    best = x.max()
    if best == -np.inf:
        return -1, -np.inf
    order = np.argsort(-x, kind="stable")
    if not temperature > 0:
        return int(order[0]), 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.where(x == best, 1.0, np.where(x == -np.inf, 0.0, np.exp((x - best) / temperature)))
    e = np.where(np.isnan(e), 0.0, e)
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        mass = np.cumsum(e[order])
        order = order[:1 + int(np.searchsorted(mass, max(top_p, 0.0) * mass[-1], side="left"))] if top_p > 0 else order[:1]
    if min_p > 0:
        order = order[e[order] >= min(min_p, 1.0)]
    order = np.sort(order)
    order = order[e[order] > 0]
    mass = np.cumsum(e[order])
    at = min(int(np.searchsorted(mass, (u if u > 0 else 0.0) * mass[-1], side="right")), len(order) - 1)
    return int(order[at]), math.log(e[order[at]] / mass[-1])
