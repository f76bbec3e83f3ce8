"""The paged INT8 KV-cache calls refuse bad arguments on the host (before any
CUDA call), and a CPU model of their division of work.  No GPU needed."""
import ctypes
import random

import pytest
import torch

import post_weight_quantization_group_b200 as q4
from post_weight_quantization_group_b200 import build as q4build

A = 0x10000  # a fake device address: compared, never read


@pytest.fixture(scope="module")
def lib():
    q4build.build()
    return q4.load_library()


def _pool(**kw):
    d = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, k_codes_stride=2 * 16 * 64, k_scales_stride=32,
             v_codes_stride=2 * 16 * 64, v_scales_stride=32, pages=4, heads=2, page_size=16, head_dim=64,
             dtype=q4.Q4_BF16)
    d.update(kw)
    return q4._CKVPaged(**d)


def _batch(**kw):
    d = dict(block_table=A, seq_lens=A, cu_new=None, table_width=4, tokens=3, max_new=1, seqs=3)
    d.update(kw)
    return q4._CKVBatch(**d)


POOL_FAULTS = [
    (dict(dtype=9), "INVALID_ARG"), (dict(dtype=q4.Q4_F32), "UNSUPPORTED"), (dict(head_dim=24), "SHAPE"),
    (dict(head_dim=8), "SHAPE"), (dict(head_dim=272), "SHAPE"), (dict(heads=0), "SHAPE"),
    (dict(page_size=0), "SHAPE"), (dict(pages=0), "SHAPE"), (dict(pages=2 ** 31), "SHAPE"),
    (dict(k_codes_stride=2047), "SHAPE"), (dict(v_codes_stride=2056), "ALIGNMENT"),
    (dict(k_scales_stride=31), "SHAPE"), (dict(k_codes=None), "INVALID_ARG"), (dict(v_scales=None), "INVALID_ARG"),
    (dict(k_codes=A + 8), "ALIGNMENT"), (dict(v_scales=A + 1), "ALIGNMENT"),
]


def _status(name):
    return getattr(q4, "Q4_ERR_" + name)


@pytest.mark.parametrize("kw,status", POOL_FAULTS)
def test_pool_faults(lib, kw, status):
    p = ctypes.byref(_pool(**kw))
    b = ctypes.byref(_batch())
    want = _status(status)
    assert lib.kv_append_int8_paged(p, A, 128, 2, A, 128, A, 128, 3, A, A, A, 64, 0, None, None, 1e-6, A, 128,
                                    None) == want
    assert lib.kv_gather_int8_paged(p, A, 3, A, A, None) == want
    assert lib.kv_attention_int8_paged(p, A, 256, 4, b, 1.0, 0, A, 256, A, A, 1 << 30, None) == want
    assert lib.kv_attention_mass_int8_paged(p, A, 256, 4, A, b, 1.0, 0, A, 32, None) == want
    assert lib.kv_evict_int8_paged(p, A, 32, b, 8, 1, 1, None, 0, A, A, 1 << 20, None) == want


def test_append_faults(lib):
    ok = dict(q=A, qs=256, hq=4, k=A, ks=128, v=A, vs=128, n=3, slots=A, pos=A, inv=A, rot=64, il=0, qn=None,
              kn=None, eps=1e-6, qo=A, qos=256)

    def call(**kw):
        a = dict(ok)
        a.update(kw)
        p = ctypes.byref(_pool())
        return lib.kv_append_int8_paged(p, a["q"], a["qs"], a["hq"], a["k"], a["ks"], a["v"], a["vs"], a["n"],
                                        a["slots"], a["pos"], a["inv"], a["rot"], a["il"], a["qn"], a["kn"],
                                        a["eps"], a["qo"], a["qos"], None)

    assert call(n=0) == q4.Q4_OK
    assert call(n=-1) == q4.Q4_ERR_SHAPE
    assert call(hq=-1) == q4.Q4_ERR_SHAPE
    assert call(rot=80) == q4.Q4_ERR_SHAPE           # more than head_dim
    assert call(rot=24) == q4.Q4_ERR_SHAPE           # halves of 12
    assert call(rot=23, il=1) == q4.Q4_ERR_SHAPE
    assert call(il=2) == q4.Q4_ERR_INVALID_ARG
    assert call(eps=-1.0) == q4.Q4_ERR_INVALID_ARG
    assert call(eps=float("nan")) == q4.Q4_ERR_INVALID_ARG
    for name in ("slots", "pos", "inv", "k", "v", "q", "qo"):
        assert call(**{name: None}) == q4.Q4_ERR_INVALID_ARG, name
    assert call(ks=120) == q4.Q4_ERR_SHAPE and call(qs=255) == q4.Q4_ERR_SHAPE
    assert call(ks=132) == q4.Q4_ERR_ALIGNMENT and call(qos=260) == q4.Q4_ERR_ALIGNMENT
    assert call(k=A + 2) == q4.Q4_ERR_ALIGNMENT and call(qn=A + 8) == q4.Q4_ERR_ALIGNMENT
    assert call(slots=A + 4) == q4.Q4_ERR_ALIGNMENT and call(pos=A + 2) == q4.Q4_ERR_ALIGNMENT


def test_gather_faults(lib):
    p = ctypes.byref(_pool())
    assert lib.kv_gather_int8_paged(p, A, 0, A, A, None) == q4.Q4_OK
    assert lib.kv_gather_int8_paged(p, A, -1, A, A, None) == q4.Q4_ERR_SHAPE
    assert lib.kv_gather_int8_paged(p, None, 1, A, A, None) == q4.Q4_ERR_INVALID_ARG
    assert lib.kv_gather_int8_paged(p, A, 1, A, A + 8, None) == q4.Q4_ERR_ALIGNMENT


BATCH_FAULTS = [
    (dict(seqs=-1), "SHAPE"), (dict(table_width=-1), "SHAPE"), (dict(table_width=2 ** 27), "SHAPE"),
    (dict(tokens=-1), "SHAPE"), (dict(max_new=0), "SHAPE"), (dict(tokens=2 ** 29), "SHAPE"),
    (dict(seq_lens=None), "INVALID_ARG"), (dict(block_table=None), "INVALID_ARG"),
    (dict(seq_lens=A + 2), "ALIGNMENT"), (dict(cu_new=A + 1), "ALIGNMENT"),
]


@pytest.mark.parametrize("kw,status", BATCH_FAULTS)
def test_batch_faults(lib, kw, status):
    p, b = ctypes.byref(_pool()), ctypes.byref(_batch(**kw))
    want = _status(status)
    assert lib.kv_attention_int8_paged(p, A, 256, 4, b, 1.0, 0, A, 256, A, A, 1 << 30, None) == want
    assert lib.kv_attention_mass_int8_paged(p, A, 256, 4, A, b, 1.0, 0, A, 32, None) == want


def test_attention_faults(lib):
    ok = dict(q=A, qs=256, hq=4, scale=1.0, window=0, out=A, os=256, lse=A, ws=A, wsb=1 << 30, b={})

    def call(**kw):
        a = dict(ok)
        a.update(kw)
        return lib.kv_attention_int8_paged(ctypes.byref(_pool()), a["q"], a["qs"], a["hq"],
                                           ctypes.byref(_batch(**a["b"])), a["scale"], a["window"], a["out"],
                                           a["os"], a["lse"], a["ws"], a["wsb"], None)

    assert call(b=dict(tokens=0)) == q4.Q4_OK and call(b=dict(seqs=0)) == q4.Q4_OK
    assert call(hq=3) == q4.Q4_ERR_SHAPE and call(hq=0) == q4.Q4_ERR_SHAPE
    assert call(scale=float("inf")) == q4.Q4_ERR_INVALID_ARG
    assert call(window=-1) == q4.Q4_ERR_INVALID_ARG
    assert call(q=None) == q4.Q4_ERR_INVALID_ARG and call(out=None) == q4.Q4_ERR_INVALID_ARG
    assert call(qs=128) == q4.Q4_ERR_SHAPE and call(os=257) == q4.Q4_ERR_ALIGNMENT
    assert call(lse=A + 2) == q4.Q4_ERR_ALIGNMENT
    assert call(ws=None) == q4.Q4_ERR_WORKSPACE and call(wsb=1000) == q4.Q4_ERR_WORKSPACE
    assert call(ws=A + 16) == q4.Q4_ERR_ALIGNMENT
    w = lib.kv_attention_workspace_bytes
    assert w(64, 4, 2, 1) > 256 * 1024
    assert w(24, 4, 2, 1) == 0 and w(64, 3, 2, 1) == 0 and w(64, 4, 2, 0) == 0


def test_evict_faults(lib):
    ok = dict(mass=A, ms=32, budget=8, recent=2, sinks=2, dst=None, dw=0, nl=A, ws=A, wsb=1 << 20, b={})

    def call(**kw):
        a = dict(ok)
        a.update(kw)
        return lib.kv_evict_int8_paged(ctypes.byref(_pool()), a["mass"], a["ms"], ctypes.byref(_batch(**a["b"])),
                                       a["budget"], a["recent"], a["sinks"], a["dst"], a["dw"], a["nl"], a["ws"],
                                       a["wsb"], None)

    assert call(b=dict(seqs=0)) == q4.Q4_OK
    assert call(budget=0) == q4.Q4_ERR_INVALID_ARG and call(recent=-1) == q4.Q4_ERR_INVALID_ARG
    assert call(sinks=7) == q4.Q4_ERR_INVALID_ARG and call(recent=9) == q4.Q4_ERR_INVALID_ARG
    assert call(ms=31) == q4.Q4_ERR_SHAPE
    assert call(dst=A + 64, dw=0) == q4.Q4_ERR_SHAPE      # too narrow for the budget
    assert call(budget=17, dst=A + 64, dw=1) == q4.Q4_ERR_SHAPE
    assert call(mass=None) == q4.Q4_ERR_INVALID_ARG and call(nl=None) == q4.Q4_ERR_INVALID_ARG
    assert call(nl=A + 1) == q4.Q4_ERR_ALIGNMENT and call(dst=A + 2, dw=9) == q4.Q4_ERR_ALIGNMENT
    assert call(ws=None) == q4.Q4_ERR_WORKSPACE and call(wsb=10) == q4.Q4_ERR_WORKSPACE
    assert lib.kv_evict_workspace_bytes(3, 2, 8) == (3 * 2 * 8 + 3) * 4
    assert lib.kv_evict_workspace_bytes(0, 2, 8) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    cache = q4.KVPagedInt8(torch.zeros(2, 1, 16, 64, dtype=torch.int8), torch.zeros(2, 1, 16).half(),
                           torch.zeros(2, 1, 16, 64, dtype=torch.int8), torch.zeros(2, 1, 16).half())
    with pytest.raises(ValueError):
        cache.c_struct()  # on the host
    bad = q4.KVPagedInt8(cache.k_codes, torch.zeros(2, 16, 1).half(), cache.v_codes, cache.v_scales)
    with pytest.raises(ValueError):
        bad.c_struct()
    bad = q4.KVPagedInt8(cache.k_codes.transpose(1, 2), cache.k_scales, cache.v_codes, cache.v_scales)
    with pytest.raises(ValueError):
        bad.c_struct()


# The kernels' division of work (kv_paged.cuh): units in order, each as `lead`
# empty places and then its tiles, at least one, cut into P equal ranges.

def _tiles(length, n, rt, R, KT, group, window):
    r0 = rt * R
    r1 = min(r0 + R, n * group) - 1
    hi = max(length - n + r1 // group + 1, 0)
    first = max(length - n + r0 // group + 1 - window, 0) if window else 0
    lo = first // KT
    return lo, max((hi + KT - 1) // KT - lo, 1)


def test_division_of_work_model():
    rng = random.Random(1)
    for _ in range(80):
        group, heads, window = rng.choice([1, 3, 8, 40]), rng.choice([1, 2, 8]), rng.choice([0, 0, 1, 100, 700])
        R, KT = rng.choice([8, 16, 128, 256]), 128
        seqs = [(rng.choice([0, 1, 127, 128, 129, rng.randint(0, 3000)]), rng.choice([0, 1, 1, rng.randint(1, 90)]))
                for _ in range(rng.randint(1, 9))]
        units = []
        for b, (length, n) in enumerate(seqs):
            for rt in range(-(-n * group // R)):
                lo, count = _tiles(length, n, rt, R, KT, group, window)
                # every key that a row of the tile sees is in the unit's tiles
                for r in range(rt * R, min((rt + 1) * R, n * group)):
                    at = length - n + r // group
                    keys = range(max(at - window + 1, 0) if window else 0, at + 1)
                    if len(keys):
                        assert lo * KT <= keys[0] and keys[-1] < (lo + count) * KT
                assert (lo + count - 1) * KT < max(length, 1) + KT
                units += [(b, rt, h, count) for h in range(heads)]
        lead = rng.choice([0, 1, 3])
        T = sum(u[3] + lead for u in units)
        P = max(min(rng.choice([1, 7, 148, 296]), T), 1)
        cuts = [T * p // P for p in range(P + 1)]
        done, at = [], 0
        slots = {}
        for x, (b, rt, h, count) in enumerate(units):
            s = at + lead  # the unit's first tile
            e = s + count
            first, last = ((s + 1) * P - 1) // T, (e * P - 1) // T
            holders = [p for p in range(P) if cuts[p] < e and cuts[p + 1] > s]
            # the owners are exactly the CTAs whose ranges hold one of its tiles
            assert holders == list(range(first, last + 1))
            for p in holders:
                lo, hi = max(cuts[p], s), min(cuts[p + 1], e)
                done += [(x, t - s) for t in range(lo, hi)]
                if len(holders) > 1:
                    # the CTA's partial slot: 0 for the first unit it holds tiles of
                    mine = 0 if p not in slots else 1
                    assert mine == (0 if p > first or cuts[p] >= at else 1)
                slots[p] = True
            at = e
        assert done == [(x, t) for x, u in enumerate(units) for t in range(u[3])]
