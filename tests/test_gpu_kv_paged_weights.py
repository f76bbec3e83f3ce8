"""Attention over a paged INT8 cache where many small weights add up to much:
tokens far above all the others of a long context.

Bounds as in test_gpu_kv_paged.py, with two more terms and a third made tighter.
  Weights below fp16's normals.  A row's weights are rounded to fp16 on a scale where its
  largest (weight times V scale) lies at 2^7 or above, so a weight is off by 2^-11 of itself
  or by 2^-25 on that scale, 2^-32 of the largest.  In a tile of a chunk in which a row's maximum
  grows, the weights before it are rounded a second time, after a factor of 2^-8 or less: another 2^-11 of
  themselves, and 2^-25 of which the first one's is 2^-8.
  Accumulators.  An fp32 accumulator of the tensor cores that holds A adds a product aligned to
  A's exponent and cuts what lies below its last place: each is off by less than 2^-23 |A|,
  |A| <= sum p|v|.  It adds all n tokens of a row in the kernel of chunks, an eighth of them (one
  warp's) in that of single tokens.
  The weights' sum is rounded to nearest, 2^-24 of it at each addition: a thread makes n / 8 (chunks: 16
  packed pairs of a tile's 128) or n / 64 of them.
  out       e |ref| + sum p|v| (2^-11 + 4 dS + adds 2^-23) + 1.01 2^-32 max(p sv) sum |vq|; chunks: 2^-10
  lse       2 dS + 2^-22 |lse| + adds 2^-24
"""
import math

import pytest
import torch

import post_weight_quantization_group_b200 as q4
from oracle import kv_paged_dense as dense
from test_gpu_kv_paged import BF, HF, _d_s, _gen, _lib, _sync_ok  # noqa: F401 (_lib: the module's fixture)

pytestmark = pytest.mark.gpu


def _check(cache, q, table, lens, cu, ps, scale, got, chunk, what=""):
    out, lse = got
    o, l, spread, floor, reach = dense.attention(cache, q, table, lens, cu, ps, scale)
    ds, n = _d_s(reach), max(lens)
    fi = torch.finfo(q.dtype)
    bound = fi.eps / 2 * o.abs() + spread * ((2.0 ** -10 if chunk else 2.0 ** -11) + 4 * ds[..., None] +
                                             (n if chunk else n / 8) * 2.0 ** -23) \
        + 1.01 * 2.0 ** -32 * floor + fi.tiny * fi.eps
    err = (out.double() - o).abs()
    assert bool((err <= bound).all()), f"{what} out: worst {float((err / bound).max()):.3f}"
    lb = 2 * ds + 2.0 ** -22 * l.abs() + n / (8 if chunk else 64) * 2.0 ** -24
    assert bool(((lse.double() - l).abs() <= lb).all()), f"{what} lse"


@pytest.mark.parametrize("value", [2, 0])
@pytest.mark.parametrize("top", ["first", "middle", "late"])
@pytest.mark.parametrize("new,seqs", [(1, 400), (40, 100), (1, 1), (40, 1)])
@pytest.mark.parametrize("n,d,dtype", [(131071, 64, HF), (131071, 128, BF), (131071, 128, HF), (1 << 20, 16, HF),
                                       (140000, 256, HF)])
def test_tokens_far_above_the_others(n, d, dtype, new, seqs, top, value):
    """Scores of zero but eight tokens' of 17.5, one in each 16 tokens of a 128-token
    tile: e^17.5 is 4e7 of the others' weights, which are then 2^-25 of the largest and, with their larger
    values, 1% to 10% of the output, or all of it.  Many sequences over the same pages:
    a CTA then has a row's whole context, one sequence: a part of it."""
    ps, hk, hq = 64, 1, 8
    pages = -(-n // ps)
    g = _gen(n + new)
    cache = q4.kv_paged_int8(pages, hk, ps, d, dtype)
    cache.k_scales.fill_(2.0 ** -6)
    cache.v_scales.fill_(2.0 ** -6)
    cache.v_codes.fill_(60)
    page = torch.randperm(pages, generator=g, device="cuda")
    at = {"first": 0, "middle": n // 256 * 128, "late": n // 128 * 128 - 256}[top] + \
        16 * torch.arange(8, device="cuda") + 3
    cache.k_codes[page[at // ps], 0, at % ps, 0] = 112
    cache.v_codes[page[at // ps], 0, at % ps] = value
    q = torch.zeros(new, hq, d, dtype=dtype, device="cuda")
    q[:, :, 0] = 10.0  # the tokens' scores: 10 * 112 / 64 = 17.5
    table = page.int().expand(seqs, pages).contiguous()
    out, lse = q4.kv_attention_int8_paged(
        cache, q.repeat(seqs, 1, 1), table, torch.full((seqs,), n, dtype=torch.int32, device="cuda"),
        torch.arange(0, seqs * new + 1, new, dtype=torch.int32, device="cuda"), max_new=new, scale=1.0)
    _sync_ok()
    _check(cache, q, [page.tolist()], [n], [0, new], ps, 1.0, (out.view(seqs, new, hq, d), lse.view(seqs, new, hq)),
           d <= 128 and new > 1, top)


@pytest.mark.parametrize("new", [1, 40])
def test_values_of_zero_in_a_long_context(new):
    """2^21 tokens whose value rows are zero (scale 0): the output is zero and the
    log-sum-exp theirs, with scores that grow along the context."""
    n, ps, d, hq = 1 << 21, 128, 16, 8
    pages = n // ps
    cache = q4.kv_paged_int8(pages, 1, ps, d, BF)
    j = torch.arange(n, device="cuda").view(pages, ps)
    cache.k_codes[:, 0, :, 0] = (j * 100 // n).to(torch.int8)
    cache.k_scales.fill_(0.0625)
    q = torch.zeros(new, hq, d, dtype=BF, device="cuda")
    q[:, :, 0] = 1.0
    table, lens, cu = [list(range(pages))], [n], [0, new]
    out, lse = q4.kv_attention_int8_paged(cache, q, torch.tensor(table, dtype=torch.int32, device="cuda"),
                                          torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                          torch.tensor(cu, dtype=torch.int32, device="cuda"), max_new=new, scale=1.0)
    _sync_ok()
    assert bool((out == 0).all())
    s = (j.flatten() * 100 // n).double() * 0.0625
    for i in range(new):
        want = float(torch.logsumexp(s[:n - new + i + 1], 0))
        # x, the logarithm of the sum and its product are rounded at magnitudes below 128 (2^-18 each);
        # the sum's parts 2^-19 of it
        assert float((lse[i].double() - want).abs().max()) <= 3 * 2.0 ** -18 + 2.0 ** -19 + 2.0 ** -22 * abs(want)
    assert math.isfinite(float(lse.sum()))
