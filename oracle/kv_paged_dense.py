"""fp64 definition of attention over a paged INT8 cache for long contexts (test
infrastructure): one matrix product per sequence and KV head, in torch, so that
hundreds of thousands of cached tokens take seconds.  Written from the formulas
of include/q4.h; shares no code with the CUDA path.
"""
import math

import torch


def attention(cache, q, table, lens, cu, page_size, scale, window=0):
    """As oracle.kv_paged.attention: (out, lse, spread, floor, reach) in fp64 on q's device."""
    T, hq, d = q.shape
    heads = cache.k_codes.shape[1]
    group = hq // heads
    f64 = dict(dtype=torch.float64, device=q.device)
    out, spread, floor = (torch.zeros(T, hq, d, **f64) for _ in range(3))
    lse, reach = torch.full((T, hq), -math.inf, **f64), torch.zeros(T, hq, **f64)
    for b, length in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        if hi == lo or length == 0:
            continue
        j = torch.arange(length, device=q.device)
        page = torch.as_tensor(table[b], device=q.device).long()[j // page_size]
        at = length - (hi - lo) + torch.arange(hi - lo, device=q.device)
        seen = j <= at[:, None]
        if window:
            seen &= j > at[:, None] - window
        seen = seen[:, None, :].expand(-1, group, -1)
        for h in range(heads):
            k = cache.k_codes[page, h, j % page_size].double() * cache.k_scales[page, h, j % page_size].double()[:, None]
            vq = cache.v_codes[page, h, j % page_size].double()
            sv = cache.v_scales[page, h, j % page_size].double()
            x = slice(h * group, (h + 1) * group)
            qr = q[lo:hi, x].double()
            s = (qr.reshape(-1, d) @ k.T).reshape(hi - lo, group, length) * scale
            size = (qr.abs().reshape(-1, d) @ k.abs().T).reshape(s.shape) * abs(scale)
            s = s.masked_fill(~seen, -math.inf)
            some = seen.any(-1)
            p = torch.softmax(s, -1).masked_fill(~some[..., None], 0.0)
            out[lo:hi, x] = (p * sv) @ vq
            lse[lo:hi, x] = torch.logsumexp(s, -1)
            spread[lo:hi, x] = (p * sv) @ vq.abs()
            floor[lo:hi, x] = (p * sv).amax(-1, keepdim=True) * (seen.double() @ vq.abs())
            reach[lo:hi, x] = torch.where(some, size.masked_fill(~seen, 0).amax(-1) +
                                          s.abs().masked_fill(~seen, 0).amax(-1), 0.0)
    return out, lse, spread, floor, reach
