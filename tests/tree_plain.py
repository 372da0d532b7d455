"""Speculative decoding over the paged cache, plainly: numpy, 64 bits, one step of each definition a line.

Shares nothing with the CUDA sources.
"""
import numpy as np


def bf16_values(bits):
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def masks(parent):
    """Node i's bits: itself and its ancestors."""
    parent = np.asarray(parent)
    bits = np.zeros(parent.shape, dtype=np.uint64)
    for b, row in enumerate(parent):
        for i in range(len(row)):
            at = i
            while True:
                bits[b, i] |= np.uint64(1 << at)
                if at == 0:
                    break
                at = int(row[at])
    return bits


def attend(q, k, v, shown, scale):
    """Rows q [R, D] over tokens k, v [N, D]; shown [R, N] bool.  Returns out, lse, and what their errors scale with:
    the sum of weight * |v| (over the weights' sum), and the largest sum of |q k| of a row's shown tokens, scaled."""
    z = np.where(shown, q @ k.T * scale, -np.inf)
    m = z.max(-1, initial=-np.inf, keepdims=True)
    e = np.exp(z - np.where(np.isfinite(m), m, 0.0))
    l = e.sum(-1, keepdims=True)
    some = l > 0
    w = e / np.where(some, l, 1.0)
    lse = np.where(some, np.where(np.isfinite(m), m, 0.0) + np.log(np.where(some, l, 1.0)), -np.inf)[:, 0]
    size = np.where(shown, np.abs(q) @ np.abs(k).T * scale, 0.0).max(-1, initial=0.0)
    return w @ v, lse, w @ np.abs(v), size


def out_bound(out, weighted, size, D, N):
    """How far a bf16 output may be off: its own rounding and each weight's to bf16 are half a step (2^-8 of the value);
    a score of D products summed in fp32 is off by at most (D + 2) 2^-23 of the products' sizes (an addition that
    truncates is off by 2^-23), which moves every weight by e^x, the sum of the weights likewise; N weights, and the
    products with their values, are summed in fp32."""
    z = size[:, None] * (D + 8) * 2.0 ** -23
    weight = 2.0 ** -8 + 2 * z + (2 * N + 16) * 2.0 ** -23
    return 1.01 * (2.0 ** -8 * np.abs(out) + weight * weighted) + 1e-30


def lse_bound(lse, size, D, N):
    return size * (D + 8) * 2.0 ** -23 + (N + 16) * 2.0 ** -23 + np.where(np.isfinite(lse), np.abs(lse), 0.0) * 2.0 ** -21


def weights(row):
    """floor(x * 2^53) of probabilities, as Python-sized whole numbers."""
    x = np.clip(np.nan_to_num(row.astype(np.float64)), 0.0, 512.0)
    return np.floor(np.ldexp(x, 53)).astype(np.int64)


def verify(target, draft, tokens, parent, u_accept, u_next, distinct, n=None):
    """One sequence: target, draft [n, V] float32 (draft None: certain candidates).  Returns path and out_tokens."""
    n = len(tokens) if n is None else n
    V = target.shape[1]
    if n == 0:
        return [], []
    walk, said = [0], []
    while True:
        at = walk[-1]
        full = weights(target[at])
        w, W, Q, took = full.copy(), 1 << 53, 1.0, None
        for i in range(1, n):
            x = int(tokens[i])
            if not (0 <= parent[i] < i) or parent[i] != at or not 0 <= x < V:
                continue
            if draft is None:
                c = W
            else:
                f = np.float32(float(W) / 2.0 ** 53 / Q) if W > 0 and Q > 0 else np.float32(0)
                cs = weights(draft[at] * f)
                c = int(cs[x])
            if float(u_accept[i]) * float(c) < float(int(w[x])):
                took = i
                break
            if draft is None:
                W = max(W - int(w[x]), 0)
                w[x] = 0
            else:
                w = np.maximum(w - cs, 0)
                W = int(w.sum())
                Q -= float(draft[at][x]) if distinct else 0.0
        if took is None:
            break
        walk.append(took)
        said.append(int(tokens[took]))
    if w.sum() == 0:
        w = full
    total = int(w.sum())
    goal = min(int(float(u_next) * float(total)), total - 1)
    c = 0
    for x in range(V):
        c += int(w[x])
        if c > goal:
            break
    return walk, said + [x]


def keep(k, v, seq, path):
    """Token rows k, v [tokens, ...] of one unit with the path's rows moved (token by token, from the old ones)."""
    k2, v2 = k.copy(), v.copy()
    for j, i in enumerate(path):
        k2[seq + j], v2[seq + j] = k[seq + i], v[seq + i]
    return k2, v2
