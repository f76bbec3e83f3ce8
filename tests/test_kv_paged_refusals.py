"""Refusals of the paged INT8 KV-cache calls on the host, before any CUDA call, and
the binding's guess of the new tokens.  No GPU needed; every call here is refused or
has nothing to do."""
import ctypes

import pytest
import torch

import post_weight_quantization_group_b200 as q4
from post_weight_quantization_group_b200 import build as q4build
from test_kv_paged_abi import A, BATCH_FAULTS, POOL_FAULTS, _batch, _pool, _status


@pytest.fixture(scope="module")
def lib():
    q4build.build()
    return q4.load_library()


def _append_mass(lib, pool=None, **kw):
    a = dict(k=A, n=3, mass=A, ms=32)
    a.update(kw)
    return lib.kv_append_mass_int8_paged(ctypes.byref(pool or _pool()), A, 256, 4, a["k"], 128, A, 128, a["n"], A, A,
                                         A, 64, 0, None, None, 1e-6, A, 256, a["mass"], a["ms"], None)


@pytest.mark.parametrize("kw,status", POOL_FAULTS)
def test_append_mass_pool_faults(lib, kw, status):
    assert _append_mass(lib, _pool(**kw)) == _status(status)


def test_append_mass_faults(lib):
    assert _append_mass(lib, n=0) == q4.Q4_OK
    assert _append_mass(lib, n=0, mass=None, ms=0) == q4.Q4_OK
    assert _append_mass(lib, ms=31) == q4.Q4_ERR_SHAPE
    assert _append_mass(lib, mass=A + 2) == q4.Q4_ERR_ALIGNMENT
    assert _append_mass(lib, k=None) == q4.Q4_ERR_INVALID_ARG


def _fill(lib, fill, pool=None, batch=None, **kw):
    a = dict(out=A, ws=A, wsb=1 << 30)
    a.update(kw)
    return lib.kv_attention_fill_int8_paged(ctypes.byref(pool or _pool()), A, 256, 4, ctypes.byref(batch or _batch()),
                                            1.0, 0, a["out"], 256, A, a["ws"], a["wsb"], fill, None)


@pytest.mark.parametrize("kw,status", BATCH_FAULTS)
def test_attention_fill_batch_faults(lib, kw, status):
    assert _fill(lib, 3, batch=_batch(**kw)) == _status(status)


def test_attention_fill_faults(lib):
    for bad in (-1, 4, 1 << 20):
        assert _fill(lib, bad) == q4.Q4_ERR_INVALID_ARG
        assert _fill(lib, bad, batch=_batch(tokens=0)) == q4.Q4_ERR_INVALID_ARG
    assert _fill(lib, 3, batch=_batch(tokens=0)) == q4.Q4_OK
    assert _fill(lib, 0, batch=_batch(seqs=0)) == q4.Q4_OK
    # rows to fill are an output even where there is no sequence
    for seqs in (0, 3):
        assert _fill(lib, 1, batch=_batch(seqs=seqs), out=None) == q4.Q4_ERR_INVALID_ARG
        assert _fill(lib, 1, batch=_batch(seqs=seqs), ws=None) == q4.Q4_ERR_WORKSPACE


def test_evict_workspace(lib):
    """Enough for the selection, or for the lengths alone where the tables (4 pages of 16) name
    no more than the budget."""
    def call(budget, wsb):
        return lib.kv_evict_int8_paged(ctypes.byref(_pool()), A, 32, ctypes.byref(_batch()), budget, 1, 1, None, 0, A,
                                       A, wsb, None)

    assert call(63, lib.kv_evict_workspace_bytes(3, 2, 63) - 1) == q4.Q4_ERR_WORKSPACE
    for budget in (64, 65, 1 << 30):
        assert call(budget, 11) == q4.Q4_ERR_WORKSPACE


def test_a_stream_of_another_device(monkeypatch):
    class Stream:  # as much of a torch stream as is looked at
        def __init__(self, device):
            self.device, self.cuda_stream = torch.device(device), 0x1234

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    with pytest.raises(ValueError):
        q4._Call(torch.device("cuda", 0), Stream("cuda:1"))
    q4._same_stream_device(torch.device("cuda", 0), Stream("cuda:0"))
    q4._same_stream_device(torch.device("cuda", 0), None)
    q4._same_stream_device(torch.device("cuda", 0), 0x1234)


def test_likely_max_new():
    guess = q4._likely_max_new
    assert guess(300, 1) == 300 and guess(64, 64) == 1 and guess(64, 32) == 2  # a prompt, decode steps, drafts
    assert guess(363, 64) == 300  # a chunk of 300 beside 63 decode steps
    assert guess(0, 5) == 1 and guess(3, 5) == 1 and guess(7, 0) == 7
