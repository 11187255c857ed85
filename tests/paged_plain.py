"""The paged cache and sampling with filters by their definitions, in float64 numpy, and the error
bounds of the CUDA kernels; shared by the tests.

Bound of one attention output element, derived from the arithmetic (e = 2^-24 the f32 unit roundoff, p the
exact weights, W = sum_n p_n |v_n|):

- a score sums dim products in f32 (exact products of 16-bit or 8-bit factors) and is multiplied by the
  scales in f32: (dim + 2) e scale sum_d |q_d k_nd| + 12 e |s|, and the exponential adds 2^-21; where an 8-bit
  value's scale enters the weight as a power of two, its logarithm adds (1.5 |s| + 130) 2^-23 + 2^-21;
- the sums of weights and of weighted values: (n + 16) e each;
- 16-bit queries: the weights rounded to f16 (8-bit pages) or the pages' type, `wu` relatively, and in f16
  by 2^-32 of the largest weight where they are subnormal (the largest is kept between 2^7 and 2^15 and the
  smallest step is 2^-24); the result's own rounding `ou` |o|.

Bound of a sum of sampling weights: a weight is off by at most 2^-28 relatively (half a unit of 2^-29 each for the
table's entry and for the correction, of a value of 1/2 or more) plus 2^-30 (four f32 roundings of a correction
below 2^-7.5) plus 2^-32 (the argument's own rounding), and by one unit of 2^-44 of the largest where it is cut off.
"""
from __future__ import annotations

import numpy as np

UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
E = 2.0 ** -24


def e4m3_round(x):
    """float64 to the nearest e4m3 (ties to even), 448 at most."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.clip(np.round(x / step) * step, -448.0, 448.0)


def quantise(x, cache):
    """(codes, scale) of head vectors x [..., dim] (float64 values of f32 or fewer bits)."""
    a = np.abs(x).max(axis=-1)
    if cache == "e4m3":
        m, e = np.frexp(a)
        e = np.maximum(np.where(m <= 0.875, e - 9, e - 8), -126)
        s = np.ldexp(1.0, np.where(a == 0, -126, e))
        return e4m3_round(x / s[..., None]), s
    s = np.maximum((a.astype(np.float32) * np.float32(1 / 127)).astype(np.float64), 2.0 ** -126)
    return np.round(x / s[..., None]), s


def place(table, page_size, num_pages, r, n):
    """(page, place) of position n of row r, or None."""
    if n < 0 or n >= table.shape[1] * page_size:
        return None
    page = int(table[r, n // page_size])
    return (page, n % page_size) if 0 <= page < num_pages else None


def attend(q, keys, values, vscale, scale, dtype, cache):
    """(output, bound) of one query [dim] over keys / values [n, dim] (float64); vscale [n]."""
    n, dim = keys.shape
    if n == 0:
        return np.zeros(dim), np.zeros(dim)
    s = keys @ q * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    o = p @ values
    W = p @ np.abs(values)
    ds = (dim + 2) * E * abs(scale) * (np.abs(keys) @ np.abs(q)).max() + 12 * E * np.abs(s).max() + 2.0 ** -21
    rel = 2 * ds + 2 * (n + 16) * E
    coded = cache in ("e4m3", "i8")
    if coded:
        rel += (1.5 * np.abs(s).max() + 130) * 2.0 ** -23 + 2.0 ** -21
    bound = rel * W + UNIT[dtype] * np.abs(o)
    if dtype != "f32":
        bound = bound + UNIT["f16" if coded else dtype] * W
        if coded or dtype == "f16":
            top = (p * vscale).max() * (np.abs(values) / np.maximum(vscale, 1e-300)[:, None]).max() if coded else p.max() * np.abs(values).max()
            bound = bound + n * 2.0 ** -32 * top + (2.0 ** -25 if dtype == "f16" else 0.0)
    return o, 1.0001 * bound + 1e-30


def sample(x, temperature, top_k, top_p, min_p, u):
    """(token, logprob, sure) of one row x (float64, as the f32 sum of logit and bias): sure is False where the result hangs
    on less than the kernel's error bound."""
    x = np.where(np.isnan(x), -np.inf, x)
    V, M = len(x), x.max()
    if M == -np.inf:
        return -1, -np.inf, True
    if temperature == 0:
        return int(x.argmax()), 0.0, True
    w = np.exp((x - M) / temperature)
    order = np.lexsort((np.arange(V), -x))
    n = V if top_k == 0 else min(V, top_k)
    tol = lambda total: 2.0 ** -27 * total + V * 2.0 ** -44  # noqa: E731
    sure = True
    if top_p < 1:
        up = np.cumsum(w[order[:n]])
        limit = top_p * up[-1]
        # (equal values: every border between them is a whole number of the same weight, on both sides)
        cut = int(np.searchsorted(up, limit, side="left"))
        near = np.abs(up - limit) < tol(up[-1])
        if near.any() and x[order[0]] != x[order[n - 1]]:
            sure = False
        n = min(n, cut + 1)
    if min_p > 0:
        n = min(n, int((w[order] >= min_p).sum()))
        if (np.abs(w / min_p - 1) < 1e-12).any() and min_p != 1.0:
            sure = False
    kept = np.sort(order[:n])
    up = np.cumsum(w[kept])
    target = u * up[-1]
    if (np.abs(up[:-1] - target) < tol(up[-1])).any() and not (w[kept] == w[kept[0]]).all():
        sure = False
    j = min(int(np.searchsorted(up, target, side="right")), len(kept) - 1)
    while w[kept[j]] == 0:
        j -= 1
    return int(kept[j]), float(np.log(w[kept[j]] / up[-1])), sure
