"""Cases that measure the operators of the paged INT8 KV cache.

One layer's cache is a pool of pages, [pages, kv_heads, page_size, head_dim] INT8 codes of K
and of V with one scale per (page, head, slot) in the model's 16-bit type; a block table names
each sequence's pages.  Four operators work on it:

  append  a layer's new tokens: RMS norm of each query and key head, rotation by position,
          INT8 quantization of K and V into their cache slots; and the read-back of those rows
  attn    attention of each sequence's new tokens (one, or a chunk) over its cached tokens
  mass    the attention weight every cached token received, added up over queries and heads
  evict   per sequence and KV head, the tokens kept by that weight, compacted into other pages

`run` computes them with elementary torch operations in fp32 (own = False) or through the
package's entry points (own = True); `exact` is the definition in fp64.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of one user, a 32/8-head layer: latency is all there is
        dict(name="append_decode_b1", op="append", tokens=1, hq=32, hk=8, d=128, ps=16,
             dtype="bf16", norm=True, interleaved=False, rot=128, far=4000),
        # one decode step of a batch of 64, interleaved rotation of half the head, no norm
        dict(name="append_decode_b64", op="append", tokens=64, hq=64, hk=8, d=128, ps=32,
             dtype="fp16", norm=False, interleaved=True, rot=64, far=30000),
        # a long prompt's tokens at far positions
        dict(name="append_prompt", op="append", tokens=8191, hq=64, hk=8, d=128, ps=64,
             dtype="bf16", norm=True, interleaved=False, rot=128, far=900000),
        # one decode step of one user with a short context
        dict(name="attn_decode_b1", op="attn", seqs=1, length=1001, ragged=False, new=1,
             chunk_every=1, hq=32, hk=8, d=128, ps=16, dtype="bf16", window=0),
        # a decode step of a serving batch with contexts of very different length
        dict(name="attn_decode_b32", op="attn", seqs=32, length=8192, ragged=True, new=1,
             chunk_every=1, hq=64, hk=8, d=128, ps=16, dtype="bf16", window=0),
        # a decode step of one user with a very long context
        dict(name="attn_decode_long", op="attn", seqs=1, length=131071, ragged=False, new=1,
             chunk_every=1, hq=64, hk=8, d=128, ps=64, dtype="fp16", window=0),
        # a chunk of a long prompt over what is cached of it already
        dict(name="attn_chunk", op="attn", seqs=1, length=32768, ragged=False, new=1024,
             chunk_every=1, hq=64, hk=8, d=128, ps=64, dtype="bf16", window=0),
        # chunks of some prompts beside the decode steps of others, heads of 64, a window
        dict(name="attn_mixed", op="attn", seqs=16, length=8100, ragged=True, new=257,
             chunk_every=4, hq=32, hk=8, d=64, ps=32, dtype="fp16", window=4096),
        # the weight that one decode step of a batch gives the cached tokens
        dict(name="mass_decode", op="mass", seqs=16, length=8000, ragged=True, new=1,
             chunk_every=1, hq=64, hk=8, d=128, ps=16, dtype="bf16", window=0),
        # the weight that a prompt's last tokens give all of it, before a cut of the cache
        dict(name="mass_chunk", op="mass", seqs=1, length=32768, ragged=False, new=256,
             chunk_every=1, hq=64, hk=8, d=128, ps=64, dtype="bf16", window=0),
        # a long prompt's cache cut to an eighth
        dict(name="evict_prompt", op="evict", seqs=1, length=32768, ragged=False, budget=4096,
             recent=256, sinks=4, hk=8, d=128, ps=64, dtype="bf16"),
        # a decode batch's caches trimmed to a budget that some are still below
        dict(name="evict_batch", op="evict", seqs=16, length=4099, ragged=True, budget=1023,
             recent=65, sinks=4, hk=8, d=128, ps=16, dtype="fp16"),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "mass", "evict"])
    hq, hk = rng.choice([(32, 8), (64, 8), (8, 8), (16, 2), (12, 4), (16, 1), (28, 4)])
    d = rng.choice([64, 128, 128, 96])
    ps = rng.choice([16, 32, 64, 128, 24])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "append":
        tokens = _between(rng, 1, 8000)
        return dict(op=op, tokens=tokens, hq=hq, hk=hk, d=d, ps=ps, dtype=dtype,
                    norm=rng.random() < 0.7, interleaved=rng.random() < 0.3,
                    rot=rng.choice([d, d, d // 2]), far=_between(rng, 100, 900000))
    seqs = _between(rng, 1, 32)
    length = _between(rng, 1, 130000 // seqs)
    if op == "evict":
        budget = _between(rng, 1, length)
        sinks = min(budget, rng.choice([0, 1, 4]))
        return dict(op=op, seqs=seqs, length=length, ragged=rng.random() < 0.5, budget=budget,
                    recent=rng.randint(0, (budget - sinks) // 2), sinks=sinks, hk=hk, d=d, ps=ps,
                    dtype=dtype)
    most = max(2, min(1000, 2 * 10**9 // (seqs * hq * length)))
    new = 1 if rng.random() < 0.4 else _between(rng, 2, most)
    window = rng.choice([0, 0, 0, _between(rng, 1, 4096)]) if op == "attn" else 0
    return dict(op=op, seqs=seqs, length=length, ragged=rng.random() < 0.5, new=min(new, length),
                chunk_every=rng.choice([1, 1, 3]), hq=hq, hk=hk, d=d, ps=ps, dtype=dtype,
                window=window)


def _lens(case):
    """Cached tokens of each sequence, the new ones among them."""
    n, top = case["seqs"], case["length"]
    if not case["ragged"]:
        return [top] * n
    return [1 + (top - 1) * ((b * 619 + 407) % 1000) // 999 for b in range(n)]


def _news(case):
    """New tokens of each sequence: a chunk for every chunk_every-th, one for the others."""
    return [min(l, case["new"] if b % case["chunk_every"] == 0 else 1)
            for b, l in enumerate(_lens(case))]


# --------------------------------------------------------- bytes and flops

def work(case):
    hk, d = case["hk"], case["d"]
    row = d + 2  # a cached row: its codes and its scale
    if case["op"] == "append":
        t, hq = case["tokens"], case["hq"]
        read = t * (hq + 2 * hk) * d * 2 + t * 12
        write = t * hq * d * 2 + t * 2 * hk * row + t * 2 * hk * d * 2
        return {"bytes": read + write, "flops": t * (hq + 2 * hk) * d * 8}
    lens = _lens(case)
    if case["op"] == "evict":
        kept = sum(min(l, case["budget"]) for l in lens)
        return {"bytes": hk * (sum(lens) * 4 + kept * 2 * (2 * row + 4)), "flops": hk * sum(lens)}
    hq, news, window = case["hq"], _news(case), case["window"]
    pairs = seen = 0
    for l, n in zip(lens, news):
        first = l - n + 1  # keys of the first new token
        if window:
            pairs += sum(min(k, window) for k in range(first, l + 1))
            seen += min(l, window + n - 1)
        else:
            pairs += (first + l) * n // 2
            seen += l
    t = sum(news)
    if case["op"] == "attn":
        return {"bytes": seen * hk * 2 * row + t * hq * (4 * d + 4),
                "flops": pairs * hq * (4 * d + 4)}
    return {"bytes": seen * hk * (row + 8) + t * hq * (2 * d + 4),
            "flops": pairs * hq * (2 * d + 4)}


# ------------------------------------------------------------------ inputs

class _Cache:
    """The pool: codes [pages, heads, page_size, d], scales and mass [pages, heads, page_size]."""


def _quantized(x, dtype):
    s = (x.abs().amax(-1) / 127).to(dtype)
    sf = s.float().unsqueeze(-1)
    return torch.where(sf == 0, torch.zeros_like(x), torch.round(x / sf)).clamp(-128, 127).to(torch.int8), s


def _filled(case, pages, g, u):
    """A pool of rows as a model leaves them: a magnitude of each head, a few heavy rows."""
    hk, d, ps, dt = case["hk"], case["d"], case["ps"], DTYPES[case["dtype"]]
    c = _Cache()
    shape = (pages, hk, ps, d)
    k = torch.randn(shape, generator=g, device="cuda")
    k *= torch.empty(1, hk, 1, 1, device="cuda").uniform_(0.5, 1.5, generator=g)
    k += u * (torch.rand(pages, hk, ps, 1, generator=g, device="cuda") < 0.01)
    c.k_codes, c.k_scales = _quantized(k, dt)
    v = torch.randn(shape, generator=g, device="cuda", out=k)
    v *= torch.empty(1, hk, 1, 1, device="cuda").uniform_(-2.3, 2.3, generator=g).exp_()
    c.v_codes, c.v_scales = _quantized(v, dt)
    return c


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    hk, d, ps, dt = case["hk"], case["d"], case["ps"], DTYPES[case["dtype"]]
    st = _Cache()
    st.case, st.op = case, case["op"]
    if st.op == "append":
        return _prepare_append(st, case, g, dt)
    lens = _lens(case)
    st.longest = max(lens)
    counts = [-(-l // ps) for l in lens]
    width, source = max(counts), sum(counts)
    kept = [min(l, case.get("budget", 0)) for l in lens]
    dcounts = [-(-k // ps) for k in kept] if st.op == "evict" else [0] * len(lens)
    u = torch.randn(1, hk, 1, d, generator=g, device="cuda")
    c = _filled(case, source + sum(dcounts) + 1, g, 2 * u)
    st.cache = c
    order = torch.randperm(source, generator=g, device="cuda").tolist()
    table, owner_b, owner_j = [], [-1] * source, [0] * source
    at = 0
    for b, n in enumerate(counts):
        mine = order[at:at + n]
        at += n
        table.append(mine + [-1] * (width - n))
        for i, p in enumerate(mine):
            owner_b[p], owner_j[p] = b, i * ps
    st.table, st.lens, st.source = _ints(table), _ints(lens), source
    # for each slot of the pool's source pages: its sequence, its place, whether it holds a token
    st.owner_b = _ints(owner_b, torch.int64)[:, None].expand(source, ps)
    st.owner_j = _ints(owner_j, torch.int64)[:, None] + torch.arange(ps, device="cuda")
    st.owned = st.owner_j < st.lens.long()[st.owner_b]
    if st.op == "evict":
        mass = torch.rand(source + sum(dcounts) + 1, hk, ps, generator=g, device="cuda")
        mass = mass.pow_(8).mul_(50.0)
        mass[mass < 1e-4] = 0.0  # many tokens that no query looked at: ties
        st.mass = mass
        dwidth, at, dtable, db, dj = max(dcounts), source, [], [], []
        for b, n in enumerate(dcounts):
            dtable.append(list(range(at, at + n)) + [-1] * (dwidth - n))
            db += [b] * n
            dj += [i * ps for i in range(n)]
            at += n
        st.dst_table, st.dst_end = _ints(dtable), at
        st.dst_b = _ints(db, torch.int64)[:, None].expand(len(db), ps)
        st.dst_j = _ints(dj, torch.int64)[:, None] + torch.arange(ps, device="cuda")
        st.kept = _ints(kept)
        return st
    news, hq = _news(case), case["hq"]
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    t = starts[-1]
    st.cu, st.max_new = _ints(starts), max(news)
    st.tok_b = _ints([b for b, n in enumerate(news) for _ in range(n)], torch.int64)
    st.tok_i = _ints([i for n in news for i in range(n)], torch.int64)
    q = torch.randn(t, hq, d, generator=g, device="cuda")
    st.q = (q + 0.4 * u.reshape(1, hk, 1, d).expand(1, hk, hq // hk, d).reshape(1, hq, d)).to(dt)
    st.scale, st.window = d ** -0.5, case["window"]
    if st.op == "mass":
        st.mass = torch.rand(source + 1, hk, ps, generator=g, device="cuda")
        st.lse = _attention(st, values=False)[1]
    return st


def _prepare_append(st, case, g, dt):
    t, hq, hk, d, ps = case["tokens"], case["hq"], case["hk"], case["d"], case["ps"]
    # the three projections of a layer come as one product's output, side by side in a row
    qkv = torch.randn(t, (hq + 2 * hk) * d, generator=g, device="cuda")
    qkv *= torch.empty(1, (hq + 2 * hk) * d, device="cuda").uniform_(0.2, 3.0, generator=g)
    qkv = qkv.to(dt)
    st.q = qkv[:, :hq * d].unflatten(1, (hq, d))
    st.k = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    st.v = qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
    pages = -(-t // ps) * 2 + 3
    if t <= 256:  # decode steps: every token in a page of its own
        pages = 2 * t + 3
        at = torch.randperm(pages, generator=g, device="cuda")[:t] * ps
        st.slots = at + torch.randint(0, ps, (t,), generator=g, device="cuda")
        st.positions = torch.randint(0, case["far"], (t,), generator=g, device="cuda").int()
    else:  # a prompt: its pages filled one after another
        order = torch.randperm(pages, generator=g, device="cuda")
        i = torch.arange(t, device="cuda") + 5
        st.slots = order[i // ps] * ps + i % ps
        st.positions = (case["far"] + i).int()
    st.cache = _filled(case, pages, g, 0)
    st.rot = case["rot"]
    st.inv_freq = (500000.0 ** (-torch.arange(0, st.rot, 2, device="cuda").double() / st.rot)).float()
    st.interleaved, st.eps = case["interleaved"], 1e-6
    if case["norm"]:
        st.q_norm = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dt)
        st.k_norm = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dt)
    else:
        st.q_norm = st.k_norm = None
    return st


# ------------------------------------------------------------- plain forms

def _rotated(x, weight, st):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + st.eps) * weight.float()
    angle = st.positions.double()[:, None, None] * st.inv_freq.double()  # far positions: 64 bits
    c, s = angle.cos().float(), angle.sin().float()
    if st.interleaved:
        a, b = x[..., 0:st.rot:2], x[..., 1:st.rot:2]
        r = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :st.rot // 2], x[..., st.rot // 2:st.rot]
        r = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((r, x[..., st.rot:]), -1)


def _append(st):
    c, dt, ps = st.cache, st.q.dtype, st.case["ps"]
    q = _rotated(st.q, st.q_norm, st).to(dt)
    k_codes, k_scales = _quantized(_rotated(st.k, st.k_norm, st), dt)
    v_codes, v_scales = _quantized(st.v.float(), dt)
    page, off = st.slots // ps, st.slots % ps
    c.k_codes[page, :, off], c.k_scales[page, :, off] = k_codes, k_scales
    c.v_codes[page, :, off], c.v_scales[page, :, off] = v_codes, v_scales
    k = (c.k_codes[page, :, off].float() * c.k_scales[page, :, off].float().unsqueeze(-1)).to(dt)
    v = (c.v_codes[page, :, off].float() * c.v_scales[page, :, off].float().unsqueeze(-1)).to(dt)
    return q, k, v


def _rows(st, codes, scales):
    """The cached rows of every sequence side by side, [seqs, heads, longest, d], in fp32."""
    ps = st.case["ps"]
    j = torch.arange(st.longest, device="cuda")
    page, off = st.table.clamp(min=0).long()[:, j // ps], j % ps
    x = codes[page, :, off].float() * scales[page, :, off].float().unsqueeze(-1)
    return x.transpose(1, 2)


def _scores(st):
    """Scaled scores [seqs, heads, new tokens x group, longest], -inf where masked."""
    hk, d, n = st.case["hk"], st.case["d"], st.max_new
    i = torch.arange(n, device="cuda")
    count = st.cu[1:] - st.cu[:-1]
    tok = (st.cu[:-1, None] + i).clamp(max=st.q.shape[0] - 1).long()
    q = st.q[tok].float().unflatten(2, (hk, -1))  # [seqs, n, hk, group, d]
    q = q.permute(0, 2, 1, 3, 4)
    group = q.shape[3]
    s = q.reshape(q.shape[0], hk, n * group, d) @ _rows(st, st.cache.k_codes, st.cache.k_scales).transpose(2, 3)
    s *= st.scale
    j = torch.arange(st.longest, device="cuda")
    at = (st.lens - count)[:, None] + i  # the last key that each new token sees
    seen = (j <= at[..., None]) & (i < count[:, None])[..., None]
    if st.window:
        seen &= j > at[..., None] - st.window
    seen = seen[:, None, :, None].expand(-1, 1, n, group, -1).reshape(q.shape[0], 1, n * group, -1)
    return s.masked_fill_(~seen, -math.inf)


def _attention(st, values=True):
    hk, n = st.case["hk"], st.max_new
    s = _scores(st)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log()).reshape(s.shape[0], hk, n, -1)[st.tok_b, :, st.tok_i].flatten(1)
    if not values:
        return None, lse
    o = p @ _rows(st, st.cache.v_codes, st.cache.v_scales)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    o = o.reshape(s.shape[0], hk, n, -1, st.case["d"])[st.tok_b, :, st.tok_i].flatten(1, 2)
    return o.to(st.q.dtype), lse


def _mass(st):
    hk, n = st.case["hk"], st.max_new
    s = _scores(st)
    lse = torch.zeros(s.shape[0], hk, n, s.shape[2] // n, device="cuda")
    lse[st.tok_b, :, st.tok_i] = st.lse.unflatten(1, (hk, -1))
    got = s.sub_(lse.reshape(s.shape[0], hk, -1, 1)).exp_().sum(2)  # [seqs, heads, longest]
    add = got[st.owner_b, :, st.owner_j.clamp(max=st.longest - 1)]  # [source, ps, heads]
    st.mass[:st.source] += torch.where(st.owned[..., None], add, torch.zeros_like(add)).transpose(1, 2)
    return st.mass


def _evict(st):
    c, case, ps = st.cache, st.case, st.case["ps"]
    j = torch.arange(st.longest, device="cuda")
    page, off = st.table.clamp(min=0).long()[:, j // ps], j % ps
    mass = st.mass[page, :, off].transpose(1, 2)  # [seqs, heads, longest]
    n = st.lens[:, None, None]
    always = (j < case["sinks"]) | (j >= n - case["recent"])
    key = mass.masked_fill(always, math.inf).masked_fill(j >= n, -math.inf)
    keep = torch.sort(key, dim=-1, descending=True, stable=True)[1][..., :case["budget"]].sort(-1)[0]
    j2, b2 = st.dst_j.clamp(max=keep.shape[2] - 1), st.dst_b
    src = keep[b2, :, j2]  # [destination pages, ps, heads]: the token that each slot gets
    page = st.table.clamp(min=0).long()[b2[..., None].expand_as(src), src // ps]
    head = torch.arange(case["hk"], device="cuda")
    live = (st.dst_j < st.kept.long()[b2])[:, None]

    def moved(x, mask):
        old = x[st.source:st.dst_end]
        old.copy_(torch.where(mask, x[page, head, src % ps].transpose(1, 2), old))

    moved(c.k_codes, live[..., None])
    moved(c.v_codes, live[..., None])
    moved(c.k_scales, live)
    moved(c.v_scales, live)
    moved(st.mass, live)
    return torch.minimum(st.lens, torch.full_like(st.lens, case["budget"]))


def _evicted(st, lens):
    """What the destination pages hold now."""
    c, a, z = st.cache, st.source, st.dst_end
    return (lens, c.k_codes[a:z], c.v_codes[a:z], c.k_scales[a:z], c.v_scales[a:z], st.mass[a:z])


# --------------------------------------------------------------------- run

def run(st):
    if own:
        return _run_own(st)
    if st.op == "append":
        return _append(st)
    if st.op == "attn":
        return _attention(st)
    if st.op == "mass":
        return _mass(st)
    return _evicted(st, _evict(st))


def _run_own(st):
    import post_weight_quantization_group_b200 as q4

    c = st.cache
    cache = q4.KVPagedInt8(c.k_codes, c.k_scales, c.v_codes, c.v_scales)
    if st.op == "append":
        q = q4.kv_append_int8_paged(cache, st.q, st.k, st.v, st.slots, st.positions, st.inv_freq,
                                    q_norm=st.q_norm, k_norm=st.k_norm, eps=st.eps,
                                    interleaved=st.interleaved)
        return (q, *q4.kv_gather_int8_paged(cache, st.slots))
    if st.op == "attn":
        return q4.kv_attention_int8_paged(cache, st.q, st.table, st.lens, cu_new=st.cu,
                                          max_new=st.max_new, scale=st.scale, window=st.window)
    if st.op == "mass":
        return q4.kv_attention_mass_int8_paged(cache, st.q, st.lse, st.mass, st.table, st.lens,
                                               cu_new=st.cu, max_new=st.max_new, scale=st.scale,
                                               window=st.window)
    lens = q4.kv_evict_int8_paged(cache, st.mass, st.table, st.lens, st.case["budget"],
                                  recent=st.case["recent"], sinks=st.case["sinks"],
                                  dst_table=st.dst_table)
    return _evicted(st, lens)


# --------------------------------------------------------- the definitions

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attention, "mass": _exact_mass,
            "evict": _exact_evict}[case["op"]](st, case)


def _exact_append(st, case):
    def head(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / case["d"] + st.eps).sqrt() * w.double()
        y, half = x.clone(), st.rot // 2
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            phi = (st.positions.double() * st.inv_freq[i].double())[:, None]
            y[..., a] = x[..., a] * phi.cos() - x[..., b] * phi.sin()
            y[..., b] = x[..., a] * phi.sin() + x[..., b] * phi.cos()
        return y

    def stored(x):
        s = (x.abs().amax(-1, keepdim=True) / 127).to(st.q.dtype).double()
        return torch.where(s > 0, (x / s).round().clamp(-128, 127), 0 * x) * s

    return head(st.q, st.q_norm), stored(head(st.k, st.k_norm)), stored(st.v.double())


def _exact_sequences(st, case):
    """Per sequence and KV head: the scores of its new rows [n, group, len] with their places."""
    lens, cu, table, ps = st.lens.tolist(), st.cu.tolist(), st.table.long(), case["ps"]
    group = case["hq"] // case["hk"]
    for b, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        page, off = table[b, j // ps], j % ps
        at = torch.arange(n - (cu[b + 1] - cu[b]), n, device="cuda")
        hidden = j[None] > at[:, None]
        if st.window:
            hidden |= j[None] <= at[:, None] - st.window
        for h in range(case["hk"]):
            k = st.cache.k_codes[page, h, off].double() * st.cache.k_scales[page, h, off].double()[:, None]
            q = st.q[cu[b]:cu[b + 1], h * group:(h + 1) * group].double()
            s = torch.einsum("ngd,jd->ngj", q, k) * st.scale
            yield b, h, slice(cu[b], cu[b + 1]), slice(h * group, (h + 1) * group), page, off, \
                s.masked_fill(hidden[:, None], -math.inf)


def _exact_attention(st, case):
    out = torch.zeros(st.q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st.q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, h, tok, heads, page, off, s in _exact_sequences(st, case):
        v = st.cache.v_codes[page, h, off].double() * st.cache.v_scales[page, h, off].double()[:, None]
        lse[tok, heads] = torch.logsumexp(s, -1)
        out[tok, heads] = torch.softmax(s, -1) @ v
    return out, lse


def _exact_mass(st, case):
    mass = st.mass.double()
    for b, h, tok, heads, page, off, s in _exact_sequences(st, case):
        mass[page, h, off] += (s - st.lse[tok, heads].double()[..., None]).exp().sum((0, 1))
    return mass


def _exact_evict(st, case):
    c, ps = st.cache, case["ps"]
    table, dst, lens = st.table.cpu().numpy(), st.dst_table.cpu().numpy(), st.lens.tolist()
    arrays = [x.float().cpu().numpy() for x in (c.k_codes, c.v_codes, c.k_scales, c.v_scales, st.mass)]
    new = [x.copy() for x in arrays]
    for b, n in enumerate(lens):
        j = np.arange(n)
        for h in range(case["hk"]):
            mass = arrays[4][table[b, j // ps], h, j % ps].astype(np.float64)
            mass[: case["sinks"]] = np.inf
            mass[max(0, n - case["recent"]):] = np.inf
            src = np.sort(np.lexsort((j, -mass))[: case["budget"]])
            i = np.arange(len(src))
            for x, y in zip(arrays, new):
                y[dst[b, i // ps], h, i % ps] = x[table[b, src // ps], h, src % ps]
    a, z = st.source, st.dst_end
    return [np.minimum(lens, case["budget"])] + [x[a:z] for x in new]
