"""The paged INT8 cache's attention and mass where a CTA has much to do: many
tiles of a unit one after another, many units, against the fp64 definition.  What a
CTA gets is computed with a model of the division of work, so that the
cases keep reaching what they are for.

Bounds as in test_gpu_kv_paged.py, with the terms of test_gpu_kv_paged_weights.py for weights
that are far below a row's largest and, in chunks, are rounded twice; the accumulators' own term
is left out, which is stricter.
"""
import numpy as np
import pytest
import torch

import post_weight_quantization_group_b200 as q4
from oracle import kv_paged as ref
from oracle import kv_paged_dense as dense
from test_gpu_kv_paged import BF, HF, _Case, _d_s, _f64, _gen, _lib, _np_pool, _sync_ok  # noqa: F401
from test_kv_paged_abi import _tiles

pytestmark = pytest.mark.gpu


def _reached(c, R, lead, ctas, window=0):
    """(most tiles of a segment, most segments of a CTA), 128-token tiles and R rows."""
    group = c.hq // c.hk
    sizes = []
    for length, n in zip(c.lens, c.news):
        for rt in range(-(-n * group // R)):
            sizes += [_tiles(length, n, rt, R, 128, group, window)[1]] * c.hk
    T = sum(sizes) + lead * len(sizes)
    P = min(ctas, T)
    cuts = [T * p // P for p in range(P + 1)]
    most, count, at, segs = 0, 0, 0, np.zeros(P, dtype=int)
    for s in sizes:
        a, b = at + lead, at + lead + s
        for p in range(max(((a + 1) * P - 1) // T, 0), ((b * P - 1) // T) + 1):
            n = min(cuts[p + 1], b) - max(cuts[p], a)
            if n > 0:
                most = max(most, n)
                segs[p] += 1
        at = b
    return most, int(segs.max())


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _check(c, window=0, chunk=False):
    scale = c.d ** -0.5
    out, lse = c.attention(window=window)
    _sync_ok()
    o, l, spread, floor, reach = dense.attention(c.cache, c.q, c.rows, c.lens, c.cu, c.ps, scale, window)
    ds = _d_s(reach)
    bound = torch.finfo(c.dtype).eps / 2 * o.abs() + spread * ((2.0 ** -10 if chunk else 2.0 ** -11) + 4 * ds[..., None]) \
        + 1.01 * 2.0 ** -32 * floor + torch.finfo(c.dtype).tiny
    err = (out.double() - o).abs()
    assert bool((err <= bound).all()), f"out: worst {float((err / bound).max()):.3f}"
    assert bool(((lse.double() - l).abs() <= 2 * ds + 2.0 ** -22 * l.abs()).all()), "lse"


def _rising(c):
    """Scores that grow along every sequence: a row's maximum moves in late tiles too."""
    u = torch.randn(c.hk, c.d, generator=_gen(7), device="cuda")
    u /= u.norm(dim=1, keepdim=True)
    c.q = (c.q.float() + 30 * u.repeat_interleave(c.hq // c.hk, 0)).to(c.dtype)
    for b, n in enumerate(c.lens):
        j = torch.arange(n, device="cuda")
        page = torch.tensor(c.rows[b], device="cuda")[j // c.ps]
        grow = (30.0 * j / n)[:, None, None]  # scores up to 30 * 30 / sqrt(d): 80 to 110
        k = torch.randn(n, c.hk, c.d, generator=_gen(b), device="cuda") + grow * u
        s = (k.abs().amax(-1) / 127).to(c.dtype)
        c.cache.k_codes[page, :, j % c.ps] = torch.round(k / s.float()[..., None]).clamp(-127, 127).to(torch.int8)
        c.cache.k_scales[page, :, j % c.ps] = s
    return c


@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("hq,hk,d,ps,dtype,lens", [
    (64, 8, 128, 16, BF, [20000, 9001, 13, 15011, 8191]), (32, 4, 64, 64, HF, [60000, 30001, 1]),
    (30, 6, 96, 24, BF, [17, 33000, 24000]), (8, 4, 256, 32, HF, [25000, 20001]), (16, 1, 128, 48, HF, [160001])])
def test_decode_many_tiles(hq, hk, d, ps, dtype, lens, rising):
    c = _Case([(n, 1) for n in lens], hq, hk, d, ps, dtype, seed=d)
    nr = 1 if hq // hk <= 8 else 2
    dp = 64 if d <= 64 else 128 if d <= 128 else 256
    most, _ = _reached(c, 8 * nr, 3, _sms() * (1 if dp * nr > 128 else 2))
    assert most >= 8
    _check(_rising(c) if rising else c)


@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("hq,hk,d,ps,dtype,seqs,window", [
    (32, 4, 128, 16, BF, [(6100, 256)], 0), (16, 2, 96, 24, HF, [(9000, 300), (4000, 200)], 0),
    (32, 4, 64, 64, HF, [(7000, 257)], 6000), (10, 2, 128, 32, BF, [(7000, 900)], 0)])
def test_chunk_many_tiles(hq, hk, d, ps, dtype, seqs, window, rising):
    c = _Case(seqs, hq, hk, d, ps, dtype, seed=d)
    most, _ = _reached(c, 256, 1, _sms(), window)
    assert most >= 10
    _check(_rising(c) if rising else c, window, chunk=True)


@pytest.mark.parametrize("d,dtype", [(128, BF), (96, HF), (64, BF), (16, HF)])
def test_chunk_many_segments(d, dtype):
    """Hundreds of short chunks, a CTA's segments one after another."""
    seqs = [(3 + (b * 71) % 333, 3 + (b * 29) % 30) for b in range(500)]
    seqs = [(max(n, m), m) for n, m in seqs]
    c = _Case(seqs, 16, 2, d, 16, dtype, seed=d)
    most, segs = _reached(c, 256, 1, _sms())
    assert segs > 5
    _check(c, chunk=True)


@pytest.mark.parametrize("d,dtype", [(128, HF), (64, BF), (256, BF)])
def test_decode_many_segments(d, dtype):
    c = _Case([(1 + (b * 71) % 333, 1) for b in range(900)], 16, 4, d, 16, dtype, seed=d)
    _, segs = _reached(c, 8, 3, _sms() * (1 if d > 128 else 2))
    assert segs > 5
    _check(c)


@pytest.mark.parametrize("hq,hk,d,dtype,window", [(32, 8, 128, BF, 0), (32, 8, 64, HF, 700), (24, 8, 96, BF, 0),
                                                  (16, 8, 256, HF, 0)])
def test_mass_many_units(hq, hk, d, dtype, window):
    """A CTA of the chunks' kernel has more than eight units of 128 tokens."""
    seqs = [(900 + 37 * b, 6 + b % 5) for b in range(20)]
    c = _Case(seqs, hq, hk, d, 16, dtype, seed=d)
    units = sum(-(-n // 128) for n in c.lens) * hk
    assert window or units > 8 * _sms()
    _, lse = c.attention(window=window)
    start = torch.rand(c.cache.k_scales.shape, generator=_gen(2), device="cuda")
    got = q4.kv_attention_mass_int8_paged(c.cache, c.q, lse, start.clone(), c.table, c.len_t, c.cu_t,
                                          max_new=c.max_new, window=window)
    _sync_ok()
    want, err = ref.mass(_np_pool(c.cache), _f64(c.q), _f64(lse), c.rows, c.lens, c.cu, 16, d ** -0.5, window,
                         _f64(start))
    add = want - _f64(start)
    nrows = max(c.news) * (hq // hk)
    bound = (2.0 ** -19 + 2e-6) * err + 64e-6 * add + (nrows + 2) * 2.0 ** -24 * want
    assert np.all(np.abs(_f64(got) - want) <= bound)


@pytest.mark.parametrize("lens", [[20000, 9001, 15011], [160001]])
def test_mass_decode_many_tiles(lens):
    c = _Case([(n, 1) for n in lens], 64, 8, 64, 64, BF, seed=4) if len(lens) > 1 else \
        _Case([(n, 1) for n in lens], 16, 2, 128, 64, HF, seed=4)
    most, _ = _reached(c, 8, 3, _sms() * 2)
    assert most >= 6
    _, lse = c.attention()
    start = torch.zeros(c.cache.k_scales.shape, device="cuda")
    got = q4.kv_attention_mass_int8_paged(c.cache, c.q, lse, start.clone(), c.table, c.len_t)
    _sync_ok()
    want, err = ref.mass(_np_pool(c.cache), _f64(c.q), _f64(lse), c.rows, c.lens, c.cu, 64, c.d ** -0.5, 0,
                         _f64(start))
    bound = (2.0 ** -19 + 2e-6) * err + 64e-6 * want + (8 + 2) * 2.0 ** -24 * want
    assert np.all(np.abs(_f64(got) - want) <= bound)
