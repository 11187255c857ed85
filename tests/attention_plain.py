"""Attention and the draft tree's commit by their definitions, in float64 numpy, one query at a
time, and the error bounds of the CUDA kernels; shared by the tests.

Error bound of one output element, derived from the arithmetic (u = the type's unit roundoff,
e = 2^-24 the f32 one, W = sum_n p_n |v_n| with the exact weights p, V = max_n |v_n|):

- a score is a sum of dim products in f32 (exact products for 16-bit types): its error is at
  most (dim + 2) e scale sum_d |q_d k_nd|, and the exponent's argument s * log2(e) - max adds
  three roundings of at most |s| log2(e) 2 e; a weight is off by that (in absolute terms of its
  exponent, times ln 2 <= 1) plus the exponential's 2^-21, relatively;
- the sums of weights and of weighted values add at most (n + 16) e relatively (n keys, a few
  rescalings), twice for numerator and denominator;
- 16-bit types: weights rounded to the type, u each (for f16 plus 2^-25 where a weight is
  subnormal, against a largest weight that may be as small as 2^-8 of the scale in use: 2^-17
  of the sum), and the result's own rounding u |o|.
"""
from __future__ import annotations

import numpy as np

UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
E = 2.0 ** -24


def branch(parents, i):
    """Node i and its ancestors, or [] for an empty place (or one under an empty place)."""
    out = []
    while True:
        p = int(parents[i])
        if p < -1 or p >= i:
            return []
        out.append(i)
        if p == -1:
            return out
        i = p


def one_query(q, keys, values, scale, dtype):
    """(output, bound) of one query [dim] over keys / values [n, dim] (float64)."""
    n, dim = keys.shape
    if n == 0:
        return np.zeros(dim), np.zeros(dim)
    s = keys @ q * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    o = p @ values
    W = p @ np.abs(values)
    ds = (dim + 2) * E * abs(scale) * (np.abs(keys) @ np.abs(q)).max() + 8 * E * np.abs(s).max() + 2.0 ** -21
    rel = 2 * ds + 2 * (n + 16) * E
    bound = rel * W
    if dtype != "f32":
        bound = bound + UNIT[dtype] * W + UNIT[dtype] * np.abs(o)
        if dtype == "f16":
            bound = bound + 2.0 ** -17 * np.abs(values).max() * min(1.0, n * p.max()) + 2.0 ** -25
    else:
        bound = bound + UNIT[dtype] * np.abs(o)
    return o, 1.0001 * bound + 1e-30


def cross(q, key, value, src_len, scale, dtype):
    """q [batch, k, q_len, heads, dim]; key, value [batch, kv_heads, max_src, dim] (float64)."""
    B, K, T, H, D = q.shape
    g = H // key.shape[1]
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        n = min(max(int(src_len[b]), 0), key.shape[2])
        for h in range(H):
            ks, vs = key[b, h // g, :n], value[b, h // g, :n]
            for j in range(K):
                for t in range(T):
                    out[b, j, t, h], bound[b, j, t, h] = one_query(q[b, j, t, h], ks, vs, scale, dtype)
    return out, bound


def tree(q, ck, cv, cache_len, dk, dv, parent, scale, dtype):
    """q [rows, nodes, heads, dim]; ck, cv [rows, kv_heads, max_len, dim]; dk, dv [rows, nodes, kv_heads, dim]."""
    R, N, H, D = q.shape
    g = H // ck.shape[1]
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for r in range(R):
        n = min(max(int(cache_len[r]), 0), ck.shape[2])
        for i in range(N):
            br = branch(parent[r], i)
            if not br:
                continue
            for h in range(H):
                ks = np.concatenate([ck[r, h // g, :n], dk[r, br, h // g]])
                vs = np.concatenate([cv[r, h // g, :n], dv[r, br, h // g]])
                out[r, i, h], bound[r, i, h] = one_query(q[r, i, h], ks, vs, scale, dtype)
    return out, bound


def commit(cache_len, parent, token, target, finished, eos, max_len):
    """Per row (path, next token, finished) by walking from the root."""
    R, N = parent.shape
    res = []
    for r in range(R):
        n = int(cache_len[r])
        if finished is not None and finished[r]:
            res.append(([], eos, 1))
            continue
        if parent[r, 0] != -1 or n < 0 or n >= max_len:
            res.append(([], int(token[r, 0]), 0))
            continue
        path = [0]
        while len(path) < max_len - n:
            want = int(target[r, path[-1]])
            if want == eos:
                break
            kids = [i for i in range(N) if parent[r, i] == path[-1] and i > path[-1] and token[r, i] == want]
            if not kids:
                break
            path.append(kids[0])
        nxt = int(target[r, path[-1]])
        res.append((path, nxt, int(nxt == eos)))
    return res
