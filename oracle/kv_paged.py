"""fp64 definitions of the paged INT8 KV-cache operators (test infrastructure).

Plain numpy loops over sequences and heads, written from the formulas of
include/q4.h and sharing no code with the CUDA path.  A pool is a dict of
float64 arrays: "kc", "vc" [pages, heads, page_size, d] codes and "ks", "vs"
[pages, heads, page_size] scales.
"""
import numpy as np


def rows(codes, scales, table, length, page_size, head):
    """(codes, scales) of the first ``length`` tokens of a table row."""
    j = np.arange(length)
    page = np.asarray(table)[j // page_size]
    return codes[page, head, j % page_size], scales[page, head, j % page_size]


def rotate(x, weight, eps, pos, inv_freq, interleaved):
    """Norm (weight not None) and rotation of x [tokens, heads, d]."""
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    half = 0 if inv_freq is None else len(inv_freq)
    y = x.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        phi = np.asarray(pos, dtype=np.float64) * np.float64(inv_freq[i])
        c, s = np.cos(phi)[:, None], np.sin(phi)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def visible(length, n, i, window):
    """[lo, hi): the cached tokens that new token i of n sees."""
    at = length - n + i
    hi = max(at + 1, 0)
    lo = max(at - window + 1, 0) if window else 0
    return min(lo, hi), hi


def attention(pool, q, table, lens, cu, page_size, scale, window):
    """Per sequence; returns out, lse and, for error bounds, per output row the
    sums  sum_j p_j |v_j|,  max_j p_j sv_j * sum_j |vq_j|  and the largest
    scale * sum_k |q_k k_jk| and |S_j|."""
    T, hq, d = q.shape
    heads = pool["kc"].shape[1]
    group = hq // heads
    out = np.zeros((T, hq, d))
    lse = np.full((T, hq), -np.inf)
    spread, floor = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    reach = np.zeros((T, hq))
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        for h in range(heads):
            kc, ks = rows(pool["kc"], pool["ks"], table[b], length, page_size, h)
            vc, vs = rows(pool["vc"], pool["vs"], table[b], length, page_size, h)
            for i in range(n):
                lo, hi = visible(length, n, i, window)
                if hi <= lo:
                    continue
                k, v = kc[lo:hi] * ks[lo:hi, None], vc[lo:hi] * vs[lo:hi, None]
                for x in range(h * group, (h + 1) * group):
                    qr = q[cu[b] + i, x]
                    s = scale * (k @ qr)
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    p /= l
                    t = cu[b] + i
                    out[t, x] = p @ v
                    lse[t, x] = m + np.log(l)
                    spread[t, x] = p @ np.abs(v)
                    floor[t, x] = (p * vs[lo:hi]).max() * np.abs(vc[lo:hi]).sum(0)
                    reach[t, x] = abs(scale) * (np.abs(k) @ np.abs(qr)).max() + np.abs(s).max()
    return out, lse, spread, floor, reach


def mass(pool, q, lse, table, lens, cu, page_size, scale, window, start):
    """start + the weight every cached token received, and the same with the
    weights' bound on the relative error of their exponents as a factor."""
    hq = q.shape[1]
    heads = pool["kc"].shape[1]
    group = hq // heads
    got = np.array(start, dtype=np.float64)
    err = np.zeros_like(got)
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        for h in range(heads):
            kc, ks = rows(pool["kc"], pool["ks"], table[b], length, page_size, h)
            for i in range(n):
                lo, hi = visible(length, n, i, window)
                j = np.arange(lo, hi)
                k = kc[lo:hi] * ks[lo:hi, None]
                page = np.asarray(table[b])[j // page_size]
                for x in range(h * group, (h + 1) * group):
                    qr, ls = q[cu[b] + i, x], lse[cu[b] + i, x]
                    s = scale * (k @ qr)
                    w = np.exp(s - ls)
                    np.add.at(got, (page, h, j % page_size), w)
                    e = abs(scale) * (np.abs(k) @ np.abs(qr)) + np.abs(s) + abs(ls)
                    np.add.at(err, (page, h, j % page_size), w * e)
    return got, err


def evict(arrays, m, table, lens, page_size, budget, recent, sinks, dst):
    """The pools after eviction: every array of ``arrays`` and the mass m
    [pages, heads, page_size], and the new lengths."""
    new = [a.copy() for a in arrays] + [m.copy()]
    heads = m.shape[1]
    for b, length in enumerate(lens):
        j = np.arange(length)
        for h in range(heads):
            src = j
            if length > budget:
                w = m[np.asarray(table[b])[j // page_size], h, j % page_size].astype(np.float64)
                order = sorted(range(sinks, length - recent),
                               key=lambda t: (-np.inf if np.isnan(w[t]) else w[t], not np.isnan(w[t]), -t),
                               reverse=True)
                keep = set(range(sinks)) | set(range(length - recent, length))
                keep |= set(order[: budget - sinks - recent])
                src = np.array(sorted(keep), dtype=np.int64)
            i = np.arange(len(src))
            if len(src):
                sp, dp = np.asarray(table[b])[src // page_size], np.asarray(dst[b])[i // page_size]
                for a, z in zip(list(arrays) + [m], new):
                    z[dp, h, i % page_size] = a[sp, h, src % page_size]
    return new, np.minimum(lens, budget).astype(np.int32)
