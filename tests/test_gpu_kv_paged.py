"""The paged INT8 KV-cache operators against their fp64 definitions
(oracle/kv_paged.py), at the sizes and masks where they can go wrong.

Error bounds, u = 2^-24 (fp32), e = the output type's half step
(torch.finfo(t).eps / 2):
  queries   the norm and the rotation are a dozen fp32 operations and an angle
            within 4e-7 of exact: |err| <= e |ref| + 2e-6 rowmax
  keys      quantized from a value within 2e-6 rowmax: the code differs from the
            definition's only where that is within 1e-3 of a tie, the scale's bits only where
            the unrounded scale is within 1e-5 of a tie
  S         an fp32 MMA chain over d / 16 steps: |err| <= 2^-19 reach, reach = scale sum |q||k| + |S|;
            x = S log2e + log2 sv adds a rounding of each at magnitude |S| + 150: 2e-6 (|S| + 32) (scales
            within 2^+-20 of one; their logarithm is within 2^-21 (|log2 sv| + 1))
  out       e |ref| + sum p|v| (2^-11 + 4 dS)  [p' rounded to fp16, half a step] + 2^-25 max(p sv) sum |vq|
            [p' below fp16's normals]
  lse       2 dS + 2^-22 |lse|
  mass      the weights' relative error is dS(1 + |lse|): sums of w (2^-19 reach + 2e-6 (reach + 32)) plus
            (rows + 2) u of the sum
"""
import numpy as np
import pytest
import torch

import oracle
import post_weight_quantization_group_b200 as q4
from oracle import kv_paged as ref

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from post_weight_quantization_group_b200 import build
    build.build()
    q4.load_library()


def _sync_ok():
    assert q4.q4_sync_status() == q4.Q4_OK


def _f64(t):
    return t.detach().cpu().double().numpy()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pool(pages, heads, ps, d, dtype, seed, layers=1, layer=0):
    """A filled pool (a slice of a pool of several layers, if asked) whose V
    magnitudes differ from row to row by up to 2^8."""
    g = _gen(seed)
    shape = (pages, layers, heads, ps)
    kc = torch.randint(-127, 128, shape + (d,), generator=g, device="cuda", dtype=torch.int8)
    vc = torch.randint(-127, 128, shape + (d,), generator=g, device="cuda", dtype=torch.int8)
    ks = (torch.rand(shape, generator=g, device="cuda") * 0.03 + 0.002).to(dtype)
    vs = torch.exp2(-8 * torch.rand(shape, generator=g, device="cuda")).mul(0.05).to(dtype)
    return q4.KVPagedInt8(kc[:, layer], ks[:, layer], vc[:, layer], vs[:, layer])


def _np_pool(c):
    return {"kc": _f64(c.k_codes), "ks": _f64(c.k_scales), "vc": _f64(c.v_codes), "vs": _f64(c.v_scales)}


def _tables(lens, ps, pages, seed, extra=0, garbage=-1):
    """Random distinct pages for every sequence; unused entries hold garbage."""
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    counts = [-(-n // ps) for n in lens]
    width = max(counts + [1]) + extra
    rows, at = [], 0
    for n in counts:
        rows.append(perm[at:at + n] + [garbage] * (width - n))
        at += n
    assert at <= pages
    return rows


def _cuda32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class _Case:
    """Sequences of (cached, new) tokens over a pool, with queries."""

    def __init__(self, seqs, hq, hk, d, ps, dtype, seed=0, spare_rows=0, q_scale=1.0, extra=0,
                 garbage=-1, layers=1):
        self.lens = [s[0] for s in seqs]
        self.news = [s[1] for s in seqs]
        self.cu = np.concatenate([[0], np.cumsum(self.news)]).astype(int).tolist()
        self.T = self.cu[-1]
        pages = sum(-(-n // ps) for n in self.lens) + 3
        self.ps, self.d, self.hq, self.hk, self.dtype = ps, d, hq, hk, dtype
        self.cache = _pool(pages, hk, ps, d, dtype, seed + 1, layers=layers, layer=layers - 1)
        self.rows = _tables(self.lens, ps, pages, seed + 2, extra, garbage)
        self.table, self.len_t, self.cu_t = _cuda32(self.rows), _cuda32(self.lens), _cuda32(self.cu)
        q = torch.randn(self.T + spare_rows, hq, d, generator=_gen(seed + 3), device="cuda") * q_scale
        self.q = q.to(dtype)
        self.max_new = max(self.news + [1])

    def attention(self, **kw):
        return q4.kv_attention_int8_paged(self.cache, self.q, self.table, self.len_t, self.cu_t,
                                          max_new=self.max_new, **kw)

    def expected(self, scale, window):
        return ref.attention(_np_pool(self.cache), _f64(self.q), self.rows, self.lens, self.cu,
                             self.ps, scale, window)


def _d_s(reach):
    return 2.0 ** -19 * reach + 2e-6 * (reach + 32)


def _check_attention(c, scale=None, window=0, got=None):
    scale = c.d ** -0.5 if scale is None else scale
    out, lse = got if got is not None else c.attention(scale=scale, window=window)
    _sync_ok()
    o, l, spread, floor, reach = c.expected(scale, window)
    T = c.T
    out, lse = _f64(out)[:T], _f64(lse)[:T]
    o, l, spread, floor, reach = o[:T], l[:T], spread[:T], floor[:T], reach[:T]
    ds = _d_s(reach)
    bound = torch.finfo(c.dtype).eps / 2 * np.abs(o) + spread * (2.0 ** -11 + 4 * ds[..., None]) \
        + 2.0 ** -25 * floor + torch.finfo(c.dtype).tiny
    err = np.abs(out - o)
    assert np.all(err <= bound), f"out: worst {np.nanmax(err / bound):.3f}"
    none = np.isinf(l)
    assert np.array_equal(none, np.isinf(lse) & (lse < 0))
    assert np.all(out[none] == 0)
    lb = 2 * ds + 2.0 ** -22 * np.abs(np.where(none, 0, l))
    assert np.all(np.abs(lse - l)[~none] <= lb[~none]), "lse"
    return out, lse


# --------------------------------------------------------------- attention

DECODE = [[(1, 1)], [(2, 1), (16, 1), (17, 1)], [(127, 1), (128, 1), (129, 1), (1000, 1), (5, 1)],
          [(4100, 1)]]


@pytest.mark.parametrize("seqs", DECODE)
@pytest.mark.parametrize("hq,hk,d,ps", [(8, 1, 128, 16), (6, 2, 64, 64), (16, 2, 128, 24),
                                        (2, 2, 16, 1), (32, 2, 96, 16), (4, 4, 256, 32),
                                        (40, 1, 80, 48), (3, 1, 192, 3)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_attention_decode(seqs, hq, hk, d, ps, dtype):
    if ps < 4 and seqs[0][0] > 2000:
        seqs = [(600, 1)]
    _check_attention(_Case(seqs, hq, hk, d, ps, dtype, seed=len(seqs) * 7 + d))


CHUNK = [
    [(300, 300)],                       # a prompt from its beginning
    [(517, 40), (9, 9), (260, 1)],      # a chunk beside a short prompt and a decode step
    [(0, 0), (130, 3), (0, 0), (64, 0), (33, 33), (0, 0)],  # sequences without tokens
    [(5, 9), (0, 4), (200, 130)],       # more new tokens than cached ones: rows that see nothing
]


@pytest.mark.parametrize("seqs", CHUNK)
@pytest.mark.parametrize("hq,hk,d,ps", [(8, 1, 128, 16), (4, 2, 64, 24), (6, 2, 128, 64), (2, 2, 256, 16),
                                        (5, 1, 48, 32)])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("window", [0, 1, 37, 129])
def test_attention_chunk(seqs, hq, hk, d, ps, dtype, window):
    _check_attention(_Case(seqs, hq, hk, d, ps, dtype, seed=d + len(seqs)), window=window)


@pytest.mark.parametrize("scale", [0.0, -0.11, 3.0])
@pytest.mark.parametrize("seqs", [[(700, 1)], [(400, 50)]])
def test_attention_scales(scale, seqs):
    """Any scale: zero (a mean), negative, and one that leaves one token."""
    _check_attention(_Case(seqs, 8, 2, 128, 16, BF, seed=5), scale=scale)


@pytest.mark.parametrize("new", [1, 70])
def test_attention_rows_behind_and_strides(new):
    """Rows behind the last sequence stay; q, out and the pool strided; unused
    table entries and everything behind a sequence's end are not read."""
    c = _Case([(130, new), (77, 1)], 8, 2, 128, 16, BF, seed=9, spare_rows=3, extra=2,
              garbage=2 ** 31 - 1, layers=3)
    wide = torch.zeros(c.q.shape[0], 12, 128, dtype=BF, device="cuda")
    wide[:, 2:10] = c.q
    c.q = wide[:, 2:10]
    buf = torch.full((c.q.shape[0], 10, 128), 7.0, dtype=BF, device="cuda")
    lse = torch.full((c.q.shape[0], 8), 5.0, device="cuda")
    used = torch.zeros(c.cache.k_scales.shape, dtype=torch.bool, device="cuda")
    for b, n in enumerate(c.lens):
        for j in range(n):
            used[c.rows[b][j // 16], :, j % 16] = True
    c.cache.k_scales[~used] = float("nan")
    c.cache.v_scales[~used] = float("inf")
    got = c.attention(out=buf[:, 1:9], lse=lse)
    clean = c.cache
    c.cache = q4.KVPagedInt8(clean.k_codes, torch.where(used, clean.k_scales, 0), clean.v_codes,
                             torch.where(used, clean.v_scales, 0))
    _check_attention(c, got=got)
    assert torch.all(buf[:, 0] == 7) and torch.all(buf[:, 9] == 7)
    assert torch.all(buf[c.T:] == 7) and torch.all(lse[c.T:] == 5)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("new", [1, 40, 150])
def test_attention_masked_nonfinite(bad, new):
    """Rows that a query may not see hold NaN or infinite scales: earlier new
    tokens do not notice the last one's, nor a window what lies before it."""
    c = _Case([(300, new + 1)], 8, 2, 128, 16, BF, seed=3)
    last, first = 299, 0
    for j in (last, first):
        page, off = c.rows[0][j // 16], j % 16
        c.cache.k_scales[page, :, off] = bad
        c.cache.v_scales[page, :, off] = bad
    out, lse = c.attention(window=100)
    _sync_ok()
    for j in (last, first):
        page, off = c.rows[0][j // 16], j % 16
        c.cache.k_scales[page, :, off] = 0.01
        c.cache.v_scales[page, :, off] = 0.01
    want, wl = c.attention(window=100)
    _sync_ok()
    seen_first = [i for i in range(new + 1) if 300 - (new + 1) + i - 100 < first]
    fine = [i for i in range(new) if i not in seen_first]
    assert torch.equal(out[fine], want[fine]) and torch.equal(lse[fine], wl[fine])
    if bad != bad:
        assert torch.isnan(out[new]).all()


def test_attention_zero_and_tiny_value_scales():
    c = _Case([(200, 1), (90, 30)], 4, 2, 64, 16, BF, seed=4)
    c.cache.v_scales[:, 0] = 0.0
    c.cache.v_codes[:, 0] = 0
    c.cache.v_scales[::2, 1] = 2.0 ** -60
    out, lse = c.attention()
    _sync_ok()
    o, l, *_ = c.expected(64 ** -0.5, 0)
    assert torch.all(out[:, :2] == 0)
    assert np.abs(_f64(lse) - l).max() < 1e-4
    assert np.abs(_f64(out) - o).max() <= 2 ** -7 * np.abs(o).max()


@pytest.mark.parametrize("new", [1, 33])
def test_attention_repeats_bit_for_bit(new):
    c = _Case([(5000, new), (300, 1), (2900, new)], 16, 2, 128, 16, BF, seed=6)
    a, la = c.attention()
    for _ in range(5):
        b, lb = c.attention()
        assert torch.equal(a, b) and torch.equal(la, lb)
    _sync_ok()


def test_attention_no_cu_is_one_token_each():
    c = _Case([(40, 1), (300, 1), (1, 1)], 8, 2, 128, 16, BF, seed=8)
    got = q4.kv_attention_int8_paged(c.cache, c.q, c.table, c.len_t)
    _check_attention(c, got=got)


def test_attention_many_sequences():
    """More sequences than a block has threads."""
    seqs = [((b * 37) % 61, 1 if (b * 37) % 61 else 0) for b in range(700)]
    _check_attention(_Case(seqs, 4, 2, 64, 16, BF, seed=11))


def test_attention_max_new_is_a_hint():
    """A max_new that does not hold changes the kernel, not the result's extent."""
    c = _Case([(200, 60), (90, 1)], 8, 2, 128, 16, BF, seed=12)
    c.max_new = 1
    _check_attention(c)
    c.max_new = 500
    _check_attention(c)


def test_attention_empty_calls():
    c = _Case([(20, 1)], 8, 2, 64, 16, BF)
    out, lse = q4.kv_attention_int8_paged(c.cache, c.q[:0], c.table, c.len_t, c.cu_t * 0)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    none = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    q4.kv_attention_int8_paged(c.cache, c.q, none, c.len_t[:0], c.cu_t[:1], out=c.q.clone())
    _sync_ok()


def test_attention_streams_and_graphs():
    """Two streams at once, each with its workspace; a captured call replayed
    with other lengths, beside another graph."""
    a = _Case([(3000, 1), (100, 1)], 16, 2, 128, 16, BF, seed=20)
    b = _Case([(2500, 1), (1700, 1)], 16, 2, 128, 16, BF, seed=21)
    want = [x.attention() for x in (a, b)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        for x, st in zip((a, b), s):
            got.append(x.attention(stream=st))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
    graphs, outs = [], []
    for x, st in zip((a, b), s):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            outs.append(x.attention())
        graphs.append(gr)
    for _ in range(5):
        for gr, st in zip(graphs, s):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for (o, l), w in zip(outs, want):
        assert torch.equal(o, w[0]) and torch.equal(l, w[1])
    a.lens = [700, 99]
    a.len_t.copy_(_cuda32(a.lens))
    graphs[0].replay()
    _check_attention(a, got=outs[0])


@pytest.mark.parametrize("new", [1, 20])
def test_attention_out_of_range_arrays(new):
    """Pages, lengths and row ranges out of range: told, nothing out of bounds."""
    for what in ("page", "neg", "len", "cu"):
        c = _Case([(200, new), (90, 1)], 8, 2, 128, 16, BF, seed=12)
        if what == "page":
            c.table[0, 3] = c.cache.k_codes.shape[0]
        elif what == "neg":
            c.table[1, 2] = -5
        elif what == "len":
            c.len_t[1] = 10 ** 6
            c.table[1] = 0
        else:
            c.cu_t[2] = 10 ** 6
        c.attention()
        assert q4.q4_sync_status() == q4.Q4_ERR_INVALID_ARG
        _sync_ok()


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("new", [1, 20])
def test_bad_pages_are_not_written(d, new):
    """A page that is none gets no mass and no evicted row; the rest is as without it."""
    c = _Case([(200, new), (90, 1)], 8, 2, d, 16, BF, seed=12)
    _, lse = c.attention()
    zero = torch.zeros(c.cache.k_scales.shape, device="cuda")
    args = (c.cache, c.q, lse)
    want = q4.kv_attention_mass_int8_paged(*args, zero.clone(), c.table, c.len_t, c.cu_t, max_new=c.max_new)
    _sync_ok()
    for bad in (-1, c.cache.k_codes.shape[0]):
        page = int(c.table[0, 4])
        table = c.table.clone()
        table[0, 4] = bad
        got = q4.kv_attention_mass_int8_paged(*args, zero.clone(), table, c.len_t, c.cu_t, max_new=c.max_new)
        assert q4.q4_sync_status() == q4.Q4_ERR_INVALID_ARG
        expect = want.clone()
        expect[page] = 0
        assert torch.equal(got, expect)
    big = _pool(40, 2, 16, d, BF, 5)
    mass = torch.rand(40, 2, 16, generator=_gen(1), device="cuda")
    before = [x.clone() for x in (big.k_codes, big.v_codes, big.k_scales, big.v_scales, mass)]
    src = _cuda32([list(range(13))])
    for bad in (-7, 40):
        q4.kv_evict_int8_paged(big, mass, src, _cuda32([200]), 48, recent=4,
                               dst_table=_cuda32([[20, bad, 22]]))
        assert q4.q4_sync_status() == q4.Q4_ERR_INVALID_ARG
        for x, y in zip((big.k_codes, big.v_codes, big.k_scales, big.v_scales, mass), before):
            keep = [p for p in range(40) if p not in (20, 22)]
            assert torch.equal(x[keep], y[keep])


def test_attention_far_pages():
    """Codes beyond 2^32 bytes of a pool."""
    ps, hk, d = 128, 8, 128
    pages = (2 ** 32 // (ps * hk * d)) + 40
    cache = q4.KVPagedInt8(torch.zeros(pages, hk, ps, d, dtype=torch.int8, device="cuda"),
                           torch.zeros(pages, hk, ps, dtype=BF, device="cuda"),
                           torch.zeros(pages, hk, ps, d, dtype=torch.int8, device="cuda"),
                           torch.zeros(pages, hk, ps, dtype=BF, device="cuda"))
    small = _Case([(500, 1), (300, 70)], 16, hk, d, ps, BF, seed=31)
    n = small.cache.k_codes.shape[0]
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        getattr(cache, name)[pages - n:] = getattr(small.cache, name)
    far = torch.where(small.table >= 0, small.table + (pages - n), small.table)
    want = small.attention()
    got = q4.kv_attention_int8_paged(cache, small.q, far, small.len_t, small.cu_t, max_new=70)
    _sync_ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    mass = torch.zeros(pages, hk, ps, device="cuda")
    m2 = torch.zeros(n, hk, ps, device="cuda")
    q4.kv_attention_mass_int8_paged(cache, small.q, got[1], mass, far, small.len_t, small.cu_t, max_new=70)
    q4.kv_attention_mass_int8_paged(small.cache, small.q, got[1], m2, small.table, small.len_t, small.cu_t,
                                    max_new=70)
    assert torch.equal(mass[pages - n:], m2) and not mass[:pages - n].any()
    _sync_ok()


# -------------------------------------------------------------------- mass

@pytest.mark.parametrize("seqs", [[(1, 1)], [(129, 1), (1000, 1), (16, 1)], [(300, 300)],
                                  [(517, 40), (0, 0), (9, 9), (260, 1)], [(5, 9), (0, 4), (200, 130)]])
@pytest.mark.parametrize("hq,hk,d,ps", [(8, 1, 128, 16), (6, 2, 64, 24), (32, 2, 96, 64), (2, 2, 256, 16),
                                        (5, 1, 48, 3)])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("window", [0, 50])
def test_mass(seqs, hq, hk, d, ps, dtype, window):
    c = _Case(seqs, hq, hk, d, ps, dtype, seed=d + 1)
    _, lse = c.attention(window=window)
    start = torch.rand(c.cache.k_scales.shape, generator=_gen(2), device="cuda")
    got = q4.kv_attention_mass_int8_paged(c.cache, c.q, lse, start.clone(), c.table, c.len_t, c.cu_t,
                                          max_new=c.max_new, window=window)
    _sync_ok()
    want, err = ref.mass(_np_pool(c.cache), _f64(c.q), _f64(lse), c.rows, c.lens, c.cu, ps, d ** -0.5,
                         window, _f64(start))
    add = want - _f64(start)
    nrows = max(c.news) * (hq // hk)
    bound = (2.0 ** -19 + 2e-6) * err + 64e-6 * add + (nrows + 2) * 2.0 ** -24 * want
    assert np.all(np.abs(_f64(got) - want) <= bound)
    # what a row's softmax hands out adds up to one
    seen = sum(1 for n, k in zip(c.lens, c.news) for i in range(k) if n - k + i >= 0) * hq
    assert abs(add.sum() - seen) <= 1e-4 * max(seen, 1)


def test_mass_shared_pages_and_masked_nan():
    """Two sequences that share a prefix's page both count; slots behind a
    sequence's end hold NaN."""
    c = _Case([(40, 1), (40, 1)], 8, 2, 128, 16, BF, seed=2)
    c.rows[1][0] = c.rows[0][0]
    c.table = _cuda32(c.rows)
    used = {(c.rows[b][j // 16], j % 16) for b in range(2) for j in range(40)}
    _, lse = c.attention()
    want, _ = ref.mass(_np_pool(c.cache), _f64(c.q), _f64(lse), c.rows, c.lens, c.cu, 16, 128 ** -0.5, 0,
                       np.zeros(c.cache.k_scales.shape))
    for p in range(c.cache.k_scales.shape[0]):
        for o in range(16):
            if (p, o) not in used:
                c.cache.k_scales[p, :, o] = float("nan")
    got = q4.kv_attention_mass_int8_paged(c.cache, c.q, lse, torch.zeros_like(c.cache.k_scales, dtype=torch.float32),
                                          c.table, c.len_t)
    _sync_ok()
    assert np.allclose(_f64(got), want, rtol=1e-4, atol=1e-9)


# ------------------------------------------------------------------ append

def _near_tie(x, width):
    f = np.abs(x - np.floor(x) - 0.5)
    return f < width


def _check_append(tokens, hq, hk, d, ps, dtype, rot, interleaved, norm, far=5000, seed=0, pad=()):
    g = _gen(seed)
    pages = tokens // ps + 5
    cache = _pool(pages, hk, ps, d, dtype, seed + 1, layers=2, layer=1)
    before = _np_pool(cache)
    qkv = (torch.randn(tokens, hq + 2 * hk + 1, d, generator=g, device="cuda") *
           torch.rand(tokens, hq + 2 * hk + 1, 1, generator=g, device="cuda") * 4).to(dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:hq + 2 * hk]
    if tokens > 3:
        k[2] = 0
        v[1] = 0
    slots = torch.randperm(pages * ps, generator=torch.Generator().manual_seed(seed))[:tokens]
    for p in pad:
        slots[p] = -1
    slots = slots.cuda()
    pos = torch.randint(0, far, (tokens,), generator=g, device="cuda").int()
    inv = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda").double() / max(rot, 1))).float() if rot else None
    w = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype) if norm else None for _ in range(2)]
    src = qkv.clone()
    got = q4.kv_append_int8_paged(cache, q, k, v, slots, pos, inv, q_norm=w[0], k_norm=w[1], eps=1e-5,
                                  interleaved=interleaved)
    _sync_ok()
    assert torch.equal(src, qkv)
    f = [None if inv is None else inv.cpu().numpy(), None if not norm else _f64(w[0]),
         None if not norm else _f64(w[1])]
    p = pos.cpu().numpy()
    qr = ref.rotate(_f64(q), f[1], 1e-5, p, f[0], interleaved)
    kr = ref.rotate(_f64(k), f[2], 1e-5, p, f[0], interleaved)
    tol = 2e-6 * np.abs(qr).max(-1, keepdims=True)
    assert np.all(np.abs(_f64(got) - qr) <= torch.finfo(dtype).eps / 2 * np.abs(qr) + tol + 1e-7)

    sl = slots.cpu().numpy()
    live = sl >= 0
    page, off = sl[live] // ps, sl[live] % ps
    after = _np_pool(cache)
    # V: bit for bit what kv_quantize_int8 gives
    vq, vsc = oracle.kv_quantize_int8(v[torch.from_numpy(live)].float().cpu().numpy(), dtype == BF)
    assert np.array_equal(after["vc"][page, :, off], vq.reshape(-1, hk, d))
    got_vs = cache.v_scales.cpu().view(torch.int16).numpy().view(np.uint16)[page, :, off]
    assert np.array_equal(got_vs, vsc.reshape(-1, hk))
    # K: scale and codes of a value within tol
    kr = kr[live]
    s_exact = np.abs(kr).max(-1) / 127
    s_got = after["ks"][page, :, off]
    s_ref = torch.from_numpy(s_exact).to(dtype).double().numpy()
    step = np.abs(torch.from_numpy(s_exact).to(dtype).double().numpy()) * torch.finfo(dtype).eps
    off_by = s_got != s_ref
    assert np.all(np.abs(s_got - s_exact)[off_by] <= (step / 2 + 1e-5 * s_exact + 1e-10)[off_by])
    with np.errstate(divide="ignore", invalid="ignore"):
        quot = np.where(s_got[..., None] > 0, kr / s_got[..., None], 0.0)
    want = np.clip(np.rint(quot), -128, 127)
    codes = after["kc"][page, :, off]
    differ = codes != want
    assert np.all(np.abs(codes - want) <= 1)
    assert np.all(_near_tie(np.abs(quot), 1e-3)[differ])
    # nothing else changed
    for name in before:
        a, b = before[name].copy(), after[name]
        a[page, :, off] = b[page, :, off]
        assert np.array_equal(a, b), name
    # the read-back
    kg, vg = q4.kv_gather_int8_paged(cache, slots[torch.from_numpy(live).cuda()])
    _sync_ok()
    for x, c_, s_ in ((kg, "kc", "ks"), (vg, "vc", "vs")):
        exact = after[c_][page, :, off] * after[s_][page, :, off][..., None]
        assert torch.equal(x.cpu(), torch.from_numpy(exact).to(torch.float32).to(dtype))


@pytest.mark.parametrize("tokens", [1, 2, 67, 1500])
@pytest.mark.parametrize("hq,hk,d,ps,rot", [(8, 2, 128, 16, 128), (4, 4, 64, 24, 32), (5, 1, 96, 1, 96),
                                            (3, 1, 256, 64, 64), (2, 1, 16, 16, 16), (6, 2, 80, 16, 0),
                                            (17, 3, 192, 7, 192)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_append(tokens, hq, hk, d, ps, rot, interleaved, dtype):
    _check_append(tokens, hq, hk, d, ps, dtype, rot, interleaved, norm=(tokens + d) % 3 != 0,
                  pad=(0, 5) if tokens == 67 else ())


def test_append_far_positions():
    """Angles of positions near 2^31 stay exact."""
    _check_append(40, 4, 1, 128, 16, BF, 128, False, True, far=2 ** 31 - 1, seed=3)


def test_append_interleaved_odd_rotation():
    _check_append(9, 4, 1, 64, 16, BF, 22, True, True, seed=3)


def test_append_in_place_without_queries_and_bad_slots():
    cache = q4.kv_paged_int8(3, 2, 16, 64)
    g = _gen(1)
    q = torch.randn(4, 8, 64, generator=g, device="cuda").to(BF)
    k, v = (torch.randn(4, 2, 64, generator=g, device="cuda").to(BF) for _ in range(2))
    pos = _cuda32([5, 6, 7, 8])
    inv = torch.rand(32, generator=g, device="cuda")
    slots = torch.tensor([0, 17, -1, 40], device="cuda")
    out = q4.kv_append_int8_paged(cache, q, k, v, slots, pos, inv)
    q2 = q.clone()
    same = q4.kv_append_int8_paged(cache, q2, k, v, slots, pos, inv, q_out=q2)
    assert same is q2 and torch.equal(q2, out)
    again = q4.kv_paged_int8(3, 2, 16, 64)
    assert q4.kv_append_int8_paged(again, None, k, v, slots, pos, inv) is None
    _sync_ok()
    assert torch.equal(again.k_codes, cache.k_codes) and torch.equal(again.v_scales, cache.v_scales)
    keep = [x.clone() for x in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    q4.kv_append_int8_paged(cache, None, k, v, slots * 0 + 48, pos, inv)
    assert q4.q4_sync_status() == q4.Q4_ERR_INVALID_ARG
    kg = torch.full((4, 2, 64), 3.0, dtype=BF, device="cuda")
    q4.kv_gather_int8_paged(cache, torch.tensor([48, -1, 1 << 40, -(1 << 40)], device="cuda"), k_out=kg,
                            v_out=kg.clone())
    assert q4.q4_sync_status() == q4.Q4_ERR_INVALID_ARG
    assert torch.all(kg == 3)
    for x, y in zip(keep, (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)):
        assert torch.equal(x, y)


# ---------------------------------------------------------------- eviction

def _check_evict(lens, hk, d, ps, dtype, budget, recent, sinks, in_place, seed=0, mass_of=None):
    cache = _pool(sum(-(-n // ps) for n in lens) + sum(-(-min(n, budget) // ps) for n in lens) + 2, hk, ps, d,
                  dtype, seed, layers=2)
    pages = cache.k_codes.shape[0]
    rows = _tables(lens, ps, pages, seed + 1)
    used = {p for r in rows for p in r if p >= 0}
    free = [p for p in range(pages) if p not in used]
    dst = rows
    if not in_place:
        dst, width = [], max([-(-min(n, budget) // ps) for n in lens] + [1])
        width = max(width, -(-min(budget, len(rows[0]) * ps) // ps))
        for n in lens:
            k = -(-min(n, budget) // ps)
            dst.append(free[:k] + [-1] * (width - k))
            free = free[k:]
    mass = torch.rand(pages, hk, ps, generator=_gen(seed + 5), device="cuda")
    if mass_of:
        mass = mass_of(mass)
    arrays = [cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales]
    before = [x.float().cpu().numpy() for x in arrays]
    m0 = mass.cpu().numpy()
    table, len_t = _cuda32(rows), _cuda32(lens)
    got = q4.kv_evict_int8_paged(cache, mass, table, len_t, budget, recent=recent, sinks=sinks,
                                 dst_table=None if in_place else _cuda32(dst))
    _sync_ok()
    want, new_lens = ref.evict(before, m0, rows, lens, ps, budget, recent, sinks, dst)
    assert np.array_equal(got.cpu().numpy(), new_lens)
    for x, w in zip(arrays + [mass], want):
        assert np.array_equal(x.float().cpu().numpy(), w, equal_nan=True)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,budget,recent,sinks", [
    ([100], 10, 3, 2), ([1, 0, 17, 64, 300], 40, 8, 4), ([5000, 1200], 1024, 100, 4),
    ([700], 1, 0, 0), ([700], 1, 1, 0), ([33, 500], 32, 20, 12), ([2300], 2299, 0, 1)])
@pytest.mark.parametrize("hk,d,ps", [(2, 128, 16), (1, 64, 24), (3, 48, 1), (2, 256, 64)])
def test_evict(in_place, lens, budget, recent, sinks, hk, d, ps):
    if ps == 1 and max(lens) > 1000:
        lens = [min(n, 900) for n in lens]
        budget, recent = min(budget, 300), min(recent, 100)
    _check_evict(lens, hk, d, ps, BF if d != 64 else HF, budget, recent, sinks, in_place, seed=budget)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_ties_and_odd_masses(in_place):
    """Equal masses keep the lower index; zeros of both signs are equal;
    infinities and NaN have their places."""
    def ties(m):
        return (m * 4).floor()

    def zeros(m):
        return torch.where(m > 0.5, torch.zeros_like(m), -torch.zeros_like(m))

    def odd(m):
        m = m - 0.5
        m[m > 0.45] = float("inf")
        m[m < -0.45] = -float("inf")
        m[(m > 0) & (m < 0.2)] = float("nan")
        return m
    for f in (ties, zeros, odd):
        _check_evict([400, 90], 2, 64, 16, BF, 61, 5, 3, in_place, seed=9, mass_of=f)


@pytest.mark.parametrize("n", [40000])
def test_evict_long(n):
    """More tokens than the selection holds in registers."""
    _check_evict([n, 100], 1, 16, 64, BF, 5001, 7, 3, False, seed=2, mass_of=lambda m: (m * 50).floor())
    _check_evict([n, 100], 1, 16, 64, BF, 5001, 7, 3, True, seed=2)


def test_evict_new_lens_may_be_seq_lens():
    for in_place in (True, False):
        c = _Case([(300, 1), (20, 1)], 2, 2, 64, 16, BF, seed=1)
        mass = torch.rand(c.cache.k_scales.shape, generator=_gen(4), device="cuda")
        pages = c.cache.k_scales.shape[0]
        big = _pool(pages + 8, 2, 16, 64, BF, 3)
        big_mass = torch.rand(pages + 8, 2, 16, generator=_gen(4), device="cuda")
        dst = None if in_place else _cuda32([[pages, pages + 1, pages + 2], [pages + 3, pages + 4, pages + 5]])
        other = q4.KVPagedInt8(big.k_codes.clone(), big.k_scales.clone(), big.v_codes.clone(), big.v_scales.clone())
        m2 = big_mass.clone()
        want = q4.kv_evict_int8_paged(other, m2, c.table, c.len_t, 48, recent=4, dst_table=dst)
        lens = c.len_t.clone()
        got = q4.kv_evict_int8_paged(big, big_mass, c.table, lens, 48, recent=4, dst_table=dst, new_lens=lens)
        _sync_ok()
        assert got is lens and torch.equal(got, want) and want.tolist() == [48, 20]
        for x, y in ((big.k_codes, other.k_codes), (big.v_scales, other.v_scales), (big_mass, m2)):
            assert torch.equal(x, y)


# ---------------------------------------------------- a run of all of them

def test_decode_loop():
    """A prompt in two chunks, decode steps, the mass of each step, a cut in
    place, and decode steps on the cut cache: against the definitions on the
    cache's own rows."""
    hq, hk, d, ps, dt = 8, 2, 64, 16, BF
    cache = q4.kv_paged_int8(24, hk, ps, d, dt)
    mass = torch.zeros(24, hk, ps, device="cuda")
    table = _cuda32([list(range(3, 15)), list(range(15, 24)) + [-1] * 3])
    rows = table.tolist()
    inv = (10000.0 ** (-torch.arange(0, d, 2, device="cuda").double() / d)).float()
    w = torch.ones(d, dtype=dt, device="cuda")
    g = _gen(0)
    lens, pos = [0, 0], [0, 0]

    def step(news):
        cu = [0, news[0], sum(news)]
        qkv = torch.randn(sum(news), hq + 2 * hk, d, generator=g, device="cuda").to(dt)
        slots, positions = [], []
        for b, n in enumerate(news):
            for i in range(n):
                j = lens[b] + i
                slots.append(rows[b][j // ps] * ps + j % ps)
                positions.append(pos[b] + i)
            lens[b] += n
            pos[b] += n
        q = q4.kv_append_int8_paged(cache, qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:],
                                    torch.tensor(slots, device="cuda"), _cuda32(positions), inv, q_norm=w, k_norm=w)
        len_t, cu_t = _cuda32(lens), _cuda32(cu)
        out, lse = q4.kv_attention_int8_paged(cache, q, table, len_t, cu_t, max_new=max(news))
        before = mass.clone()
        q4.kv_attention_mass_int8_paged(cache, q, lse, mass, table, len_t, cu_t, max_new=max(news))
        _sync_ok()
        o, l, spread, floor, reach = ref.attention(_np_pool(cache), _f64(q), rows, lens, cu, ps, d ** -0.5, 0)
        ds = _d_s(reach)
        assert np.all(np.abs(_f64(out) - o) <= 2.0 ** -8 * np.abs(o) + spread * (2.0 ** -11 + 4 * ds[..., None])
                      + 2.0 ** -25 * floor)
        m, _ = ref.mass(_np_pool(cache), _f64(q), _f64(lse), rows, lens, cu, ps, d ** -0.5, 0, _f64(before))
        assert np.allclose(_f64(mass), m, rtol=1e-4, atol=1e-7)

    step([100, 37])
    step([61, 1])
    for _ in range(3):
        step([1, 1])
    new = q4.kv_evict_int8_paged(cache, mass, table, _cuda32(lens), 64, recent=16, sinks=4)
    _sync_ok()
    assert new.tolist() == [64, 41]
    lens[:] = new.tolist()
    for _ in range(3):
        step([1, 1])
    step([5, 20])


class _Step:
    """A decode step's buffers: everything the operators read that changes."""

    def __init__(self, seed):
        g = _gen(seed)
        self.hq, self.hk, self.d, self.ps = 16, 2, 128, 16
        self.cache = _pool(30, self.hk, self.ps, self.d, BF, seed)
        self.mass = torch.rand(30, self.hk, self.ps, generator=g, device="cuda")
        self.table = _cuda32([list(range(10)), list(range(10, 20)), list(range(20, 30))])
        self.lens = _cuda32([0, 0, 0])
        self.slots = torch.zeros(3, dtype=torch.int64, device="cuda")
        self.pos = _cuda32([0, 0, 0])
        self.qkv = torch.zeros(3, self.hq + 2 * self.hk, self.d, dtype=BF, device="cuda")
        self.inv = (10000.0 ** (-torch.arange(0, self.d, 2, device="cuda").double() / self.d)).float()

    def set(self, i):
        lens = [41 + i, 0, 150 + i]  # the middle row is padding: no cached token, no slot
        self.lens.copy_(_cuda32(lens))
        self.slots.copy_(torch.tensor([(n - 1) // 16 * 16 + b * 160 + (n - 1) % 16 if n else -1
                                       for b, n in enumerate(lens)], device="cuda"))
        self.pos.copy_(_cuda32([max(n - 1, 0) for n in lens]))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=_gen(100 + i), device="cuda"))

    def run(self, **kw):
        q = q4.kv_append_int8_paged(self.cache, self.qkv[:, :self.hq], self.qkv[:, self.hq:self.hq + self.hk],
                                    self.qkv[:, self.hq + self.hk:], self.slots, self.pos, self.inv, **kw)
        out, lse = q4.kv_attention_int8_paged(self.cache, q, self.table, self.lens, **kw)
        q4.kv_attention_mass_int8_paged(self.cache, q, lse, self.mass, self.table, self.lens, **kw)
        return out, lse

    def state(self):
        c = self.cache
        return [c.k_codes, c.k_scales, c.v_codes, c.v_scales, self.mass]


def test_captured_decode_steps():
    """A step captured once and replayed with other lengths, slots and inputs, a
    padding row among them, against the same steps run one by one."""
    a, b = _Step(50), _Step(50)
    a.set(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = a.run()
    for i in range(4):
        a.set(i)
        b.set(i)
        graph.replay()
        want, wl = b.run()
        _sync_ok()
        assert torch.equal(out, want) and torch.equal(lse, wl)
        assert torch.all(out[1] == 0) and torch.all(lse[1] == -float("inf"))
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y)


@pytest.mark.parametrize("raw", [False, True])
def test_operators_on_a_given_stream(raw):
    """stream= as a torch stream and as a handle, another than the current one."""
    a, b = _Step(60), _Step(60)
    a.set(3)
    b.set(3)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    s = st.cuda_stream if raw else st
    out, lse = a.run(stream=s)
    lens = q4.kv_evict_int8_paged(a.cache, a.mass, a.table, a.lens, 32, recent=4, stream=s)
    k, v = q4.kv_gather_int8_paged(a.cache, a.slots, stream=s)
    torch.cuda.current_stream().wait_stream(st)
    want, wl = b.run()
    wlens = q4.kv_evict_int8_paged(b.cache, b.mass, b.table, b.lens, 32, recent=4)
    wk, wv = q4.kv_gather_int8_paged(b.cache, b.slots)
    _sync_ok()
    live = [0, 2]  # the padding row's keys and values are not written
    for x, y in ((out, want), (lse, wl), (lens, wlens), (k[live], wk[live]), (v[live], wv[live])):
        assert torch.equal(x, y)
    for x, y in zip(a.state(), b.state()):
        assert torch.equal(x, y)


def test_calls_right_behind_one_another():
    """Evictions, attention over the lengths that they return, mass and appends
    without a pause between them, in rounds over three caches,
    each call's data written by the one before it, against the same calls with
    a wait after each."""
    def steps(wait):
        out = []

        def ran(*x):
            if wait:
                torch.cuda.synchronize()
            out.extend(x)
        st = [_Step(70 + i) for i in range(3)]
        for i, s in enumerate(st):
            s.set(2 * i)
        torch.cuda.synchronize()
        for r in range(4):
            for s in st:
                s.lens = q4.kv_evict_int8_paged(s.cache, s.mass, s.table, s.lens, 120 - 20 * r, recent=4)
                ran(s.lens)
            for s in st:
                ran(*s.run())
        ran(*(x for s in st for x in s.state()))
        torch.cuda.synchronize()
        return out
    for x, y in zip(steps(False), steps(True)):
        assert torch.equal(x, y)
    _sync_ok()


def test_refused_workspaces():
    """A workspace that is not one run of bytes, is too small, or lies on the host."""
    s = _Step(80)
    s.set(1)
    q = s.qkv[:, :s.hq].contiguous()
    for ws, err in ((torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 26), ValueError),
                    (torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")[::2], ValueError),
                    (torch.zeros(64, dtype=torch.uint8, device="cuda"), q4.Q4Error),
                    (torch.zeros(1 << 26, dtype=torch.uint8), ValueError)):
        with pytest.raises(err):
            q4.kv_attention_int8_paged(s.cache, q, s.table, s.lens, workspace=ws)
        with pytest.raises(err):
            q4.kv_evict_int8_paged(s.cache, s.mass, s.table, s.lens, 32, workspace=ws)
    _sync_ok()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq", [1, 40])
def test_append_infinities_behind_the_rotation(hq, interleaved):
    """What is not rotated comes out as it went in, infinities among it, and
    they reach no other element."""
    tokens, d, rot, dt = 3, 64, 32, BF
    g = _gen(90)
    qkv = torch.randn(tokens, hq + 2, d, generator=g, device="cuda").to(dt)
    qkv[:, :hq, rot + 5] = float("inf")
    qkv[:, :hq, d - 1] = -float("inf")
    cache = _pool(2, 1, 16, d, dt, 91)
    pos = _cuda32([3, 1000, 77])
    inv = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda").double() / rot)).float()
    got = q4.kv_append_int8_paged(cache, qkv[:, :hq], qkv[:, hq:hq + 1], qkv[:, hq + 1:],
                                  torch.arange(tokens, device="cuda"), pos, inv, interleaved=interleaved)
    _sync_ok()
    assert torch.equal(got[..., rot:], qkv[:, :hq, rot:])
    assert torch.all(torch.isfinite(got[..., :rot]))
