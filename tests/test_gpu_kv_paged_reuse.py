"""Slots of a paged INT8 cache that are written anew: a new token's attention
mass starts at zero, whatever the slot's last token had."""
import numpy as np
import pytest
import torch

import post_weight_quantization_group_b200 as q4
from oracle import kv_paged as ref
from test_gpu_kv_paged import BF, HF, _cuda32, _f64, _gen, _lib, _np_pool, _pool, _sync_ok  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 5, 1200])
@pytest.mark.parametrize("hq,hk,d,ps,dtype", [(8, 2, 128, 16, BF), (0, 3, 64, 24, HF), (5, 1, 256, 1, BF),
                                              (3, 2, 16, 64, HF), (17, 3, 192, 7, BF)])
def test_append_clears_the_mass_of_its_slots(tokens, hq, hk, d, ps, dtype):
    """Of the slots it writes and of no other; the cache and the queries as without it."""
    pages = tokens // ps + 3
    a, b = (_pool(pages, hk, ps, d, dtype, 3) for _ in range(2))
    g = _gen(tokens + d)
    wide = torch.rand(pages, 2, hk, ps, generator=g, device="cuda") + 1
    before = wide.clone()
    mass = wide[:, 1]  # pages lie apart
    qkv = torch.randn(tokens, hq + 2 * hk, d, generator=g, device="cuda").to(dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    slots = torch.randperm(pages * ps, generator=g, device="cuda")[:tokens]
    if tokens > 2:
        slots[1] = -1
    pos = torch.arange(tokens, device="cuda").int()
    inv = torch.rand(d // 2 // 16 * 16 or 8, generator=g, device="cuda")
    qa = q4.kv_append_int8_paged(a, q if hq else None, k, v, slots, pos, inv, mass=mass)
    qb = q4.kv_append_int8_paged(b, q if hq else None, k, v, slots, pos, inv)
    _sync_ok()
    assert qa is None and qb is None if hq == 0 else torch.equal(qa, qb)
    for x, y in ((a.k_codes, b.k_codes), (a.v_codes, b.v_codes), (a.k_scales, b.k_scales), (a.v_scales, b.v_scales)):
        assert torch.equal(x, y)
    live = slots[slots >= 0]
    before[live // ps, 1, :, live % ps] = 0
    assert torch.equal(wide, before)


def test_append_mass_of_a_bad_slot():
    cache = _pool(2, 1, 16, 64, BF, 3)
    mass = torch.ones(2, 1, 16, device="cuda")
    kv = torch.randn(2, 1, 64, generator=_gen(1), device="cuda").to(BF)
    q4.kv_append_int8_paged(cache, None, kv, kv, torch.tensor([32, 1 << 40], device="cuda"), mass=mass)
    assert q4.q4_sync_status() == q4.Q4_ERR_INVALID_ARG
    assert torch.all(mass == 1)


def test_two_cuts_with_new_tokens_between():
    """Prompt, cut in place, decode steps into the freed slots, a second cut: the
    mass of every token is what its own queries gave it, and the second cut keeps the
    heaviest by that."""
    hq, hk, d, ps = 8, 2, 64, 16
    cache = q4.kv_paged_int8(12, hk, ps, d, BF)
    mass = torch.zeros(12, hk, ps, device="cuda")
    rows = [list(range(1, 9)), [9, 10, 11, 0, -1, -1, -1, -1]]
    table = _cuda32(rows)
    inv = (10000.0 ** (-torch.arange(0, d, 2, device="cuda").double() / d)).float()
    g = _gen(5)
    lens, pos = [0, 0], [0, 0]
    want = [[np.zeros(0) for _ in range(hk)] for _ in lens]  # the mass of each logical token
    tol = [[np.zeros(0) for _ in range(hk)] for _ in lens]  # and how far off the device's may be (test_mass)

    def held(b, h):
        j = np.arange(lens[b])
        return _f64(mass)[np.asarray(rows[b])[j // ps], h, j % ps]

    def same():
        for b in range(2):
            for h in range(hk):
                assert np.all(np.abs(held(b, h) - want[b][h]) <= tol[b][h]), (b, h)

    def step(news):
        cu = [0, news[0], sum(news)]
        qkv = torch.randn(sum(news), hq + 2 * hk, d, generator=g, device="cuda").to(BF)
        slots, positions = [], []
        for b, n in enumerate(news):
            for i in range(n):
                j = lens[b] + i
                slots.append(rows[b][j // ps] * ps + j % ps)
                positions.append(pos[b] + i)
            lens[b] += n
            pos[b] += n
        q = q4.kv_append_int8_paged(cache, qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:],
                                    torch.tensor(slots, device="cuda"), _cuda32(positions), inv, mass=mass)
        len_t, cu_t = _cuda32(lens), _cuda32(cu)
        _, lse = q4.kv_attention_int8_paged(cache, q, table, len_t, cu_t, max_new=max(news))
        q4.kv_attention_mass_int8_paged(cache, q, lse, mass, table, len_t, cu_t, max_new=max(news))
        _sync_ok()
        add, err = ref.mass(_np_pool(cache), _f64(q), _f64(lse), rows, lens, cu, ps, d ** -0.5, 0,
                          np.zeros(mass.shape))
        for b in range(2):
            j = np.arange(lens[b])
            for h in range(hk):
                new = np.zeros(lens[b] - len(want[b][h]))
                at = np.asarray(rows[b])[j // ps], h, j % ps
                want[b][h] = np.concatenate([want[b][h], new]) + add[at]
                tol[b][h] = np.concatenate([tol[b][h], new]) + (2.0 ** -19 + 2e-6) * err[at] + 64e-6 * add[at] + \
                    (news[b] * hq // hk + 2) * 2.0 ** -24 * want[b][h]
        same()

    def cut(budget, recent, sinks):
        got = q4.kv_evict_int8_paged(cache, mass, table, _cuda32(lens), budget, recent=recent, sinks=sinks)
        _sync_ok()
        for b in range(2):
            n = lens[b]
            for h in range(hk):
                if n > budget:
                    m, e = want[b][h], tol[b][h]
                    mid = sorted(range(sinks, n - recent), key=lambda j: -m[j])
                    k = budget - recent - sinks
                    # the border is clear of the masses' rounding, so both sides cut alike
                    assert min(m[j] - e[j] for j in mid[:k]) > max(m[j] + e[j] for j in mid[k:])
                    keep = sorted(list(range(sinks)) + mid[:k] + list(range(n - recent, n)))
                    want[b][h], tol[b][h] = m[keep], e[keep]
            lens[b] = min(n, budget)
        assert got.tolist() == lens
        same()

    step([120, 50])
    cut(40, 8, 2)
    for _ in range(9):  # into the slots behind token 40, which evicted tokens had
        step([1, 1])
    step([30, 10])
    cut(33, 4, 2)
    step([1, 1])


def test_append_mass_is_checked():
    cache = _pool(2, 1, 16, 64, BF, 3)
    kv = torch.zeros(1, 1, 64, dtype=BF, device="cuda")
    slot = torch.zeros(1, dtype=torch.int64, device="cuda")
    for bad in (torch.zeros(2, 1, 16, dtype=BF, device="cuda"), torch.zeros(2, 16, device="cuda"),
                torch.zeros(2, 1, 16), torch.zeros(2, 1, 32, device="cuda")[:, :, ::2]):
        with pytest.raises(ValueError):
            q4.kv_append_int8_paged(cache, None, kv, kv, slot, mass=bad)
    _sync_ok()
