"""What a call of the paged INT8 cache returns and allocates by default."""
import pytest
import torch

import post_weight_quantization_group_b200 as q4
from test_gpu_kv_paged import BF, HF, _Case, _cuda32, _gen, _lib, _pool, _sync_ok  # noqa: F401

pytestmark = pytest.mark.gpu


def _poison(*shapes):
    """Leaves what is neither zero nor finite in the blocks that the next tensors get."""
    keep = [torch.full(s, float("nan"), device="cuda") for s in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del keep


# sequences of (cached, new), rows of q behind the last one's
UNNAMED = [([(40, 1), (300, 1)], 3), ([(500, 200)], 70), ([(90, 30), (700, 1), (0, 0)], 5), ([(20, 0)], 4)]


@pytest.mark.parametrize("seqs,spare", UNNAMED)
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (6, 2, 64), (4, 2, 256)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_rows_that_no_sequence_names(seqs, spare, hq, hk, d, dtype):
    """A padded batch: zeros and -inf in what the call allocates, left as they
    are in what it is given; the named rows are the same either way."""
    c = _Case(seqs, hq, hk, d, 16, dtype, seed=3, spare_rows=spare)
    o, l = torch.full(c.q.shape, 7.0, dtype=dtype, device="cuda"), torch.full(c.q.shape[:2], 5.0, device="cuda")
    c.attention(out=o, lse=l)
    _sync_ok()
    assert torch.all(o[c.T:] == 7) and torch.all(l[c.T:] == 5)
    rows = c.q.shape[0]
    for kw in ({}, {"out": torch.full_like(o, 7.0)}, {"lse": torch.full_like(l, 5.0)}):
        _poison((rows, hq, d // 2), (rows, hq))
        got, lse = c.attention(**kw)
        _sync_ok()
        assert torch.equal(got[:c.T], o[:c.T]) and torch.equal(lse[:c.T], l[:c.T])
        assert torch.all(got[c.T:] == (7 if "out" in kw else 0))
        assert torch.all(lse[c.T:] == (5 if "lse" in kw else -float("inf")))


def test_more_rows_than_sequences_without_cu_new():
    c = _Case([(40, 1), (300, 1), (1, 1)], 8, 2, 128, 16, BF, seed=8, spare_rows=4)
    want, wl = q4.kv_attention_int8_paged(c.cache, c.q[:3], c.table, c.len_t)
    _poison((7, 8, 64), (7, 8))
    got, lse = q4.kv_attention_int8_paged(c.cache, c.q, c.table, c.len_t)
    _sync_ok()
    assert torch.equal(got[:3], want) and torch.equal(lse[:3], wl)
    assert torch.all(got[3:] == 0) and torch.all(lse[3:] == -float("inf"))


def test_rows_before_the_first_sequence_and_no_sequences():
    c = _Case([(60, 5), (70, 2)], 8, 2, 128, 16, BF, seed=8, spare_rows=4)
    want, wl = c.attention()
    moved = torch.cat([c.q[-4:], c.q[:7]])
    _poison((11, 8, 64), (11, 8))
    got, lse = q4.kv_attention_int8_paged(c.cache, moved, c.table, c.len_t, c.cu_t + 4, max_new=5)
    _sync_ok()
    assert torch.equal(got[4:], want[:7]) and torch.equal(lse[4:], wl[:7])
    assert torch.all(got[:4] == 0) and torch.all(lse[:4] == -float("inf"))
    none = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    _poison((11, 8, 64), (11, 8))
    got, lse = q4.kv_attention_int8_paged(c.cache, moved, none, c.len_t[:0], c.cu_t[:1] * 0)
    _sync_ok()
    assert torch.all(got == 0) and torch.all(lse == -float("inf"))


def test_unnamed_rows_of_a_captured_call():
    """Replayed with fewer rows named than at the capture."""
    c = _Case([(400, 60), (300, 1)], 8, 2, 128, 16, BF, seed=4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = c.attention()
    for n in (60, 20, 41):
        c.cu_t.copy_(_cuda32([0, n, n + 1]))
        want, wl = c.attention()
        out.fill_(9)
        lse.fill_(9)
        graph.replay()
        _sync_ok()
        assert torch.equal(out, want) and torch.equal(lse, wl)
        assert torch.all(out[n + 1:] == 0) and torch.all(lse[n + 1:] == -float("inf"))


@pytest.mark.parametrize("seqs,bound", [([(600, 300)], 300), ([(500, 90), (40, 40), (77, 1)], 129),
                                        ([(50, 1), (60, 1)], 1), ([(400, 2), (9, 2), (70, 2)], 2)])
def test_max_new_from_the_rows(seqs, bound):
    """Without max_new it is guessed from the rows of q, so a chunk gets the
    chunks' kernel: bit for bit what the same number gives when it is passed."""
    c = _Case(seqs, 16, 2, 128, 16, BF, seed=6)
    want = q4.kv_attention_int8_paged(c.cache, c.q, c.table, c.len_t, c.cu_t, max_new=bound)
    got = q4.kv_attention_int8_paged(c.cache, c.q, c.table, c.len_t, c.cu_t)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    m = [torch.zeros(c.cache.k_scales.shape, device="cuda") for _ in range(2)]
    q4.kv_attention_mass_int8_paged(c.cache, c.q, want[1], m[0], c.table, c.len_t, c.cu_t, max_new=bound)
    q4.kv_attention_mass_int8_paged(c.cache, c.q, want[1], m[1], c.table, c.len_t, c.cu_t)
    _sync_ok()
    assert torch.equal(*m)


def test_max_new_from_the_rows_and_a_small_workspace():
    """A workspace of the caller's that is enough for single tokens still serves."""
    c = _Case([(600, 300)], 16, 2, 128, 16, BF, seed=6)
    need = q4.load_library().kv_attention_workspace_bytes
    assert need(128, 16, 2, 1) < need(128, 16, 2, 300)
    want = q4.kv_attention_int8_paged(c.cache, c.q, c.table, c.len_t, c.cu_t, max_new=1)
    ws = torch.zeros(need(128, 16, 2, 1), dtype=torch.uint8, device="cuda")
    got = q4.kv_attention_int8_paged(c.cache, c.q, c.table, c.len_t, c.cu_t, workspace=ws)
    _sync_ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(q4.Q4Error):
        q4.kv_attention_int8_paged(c.cache, c.q, c.table, c.len_t, c.cu_t, max_new=300, workspace=ws)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("budget", [128, 1 << 20, 1 << 30])
def test_evict_to_more_than_the_tables_name(budget, in_place):
    """A budget that no sequence can pass moves nothing away, and asks for no
    workspace beyond the lengths."""
    lens = [100, 0, 33]
    cache = _pool(40, 2, 16, 64, BF, 5)
    mass = torch.rand(40, 2, 16, generator=_gen(1), device="cuda")
    table = _cuda32([list(range(8)), list(range(8, 16)), list(range(16, 24))])
    dst = None if in_place else _cuda32([list(range(24, 31)) + [-1], [-1] * 8, [31, 32, 33] + [-1] * 5])
    before = [x.clone() for x in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales, mass)]
    len_t = _cuda32(lens)
    torch.cuda.synchronize()
    base = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    got = q4.kv_evict_int8_paged(cache, mass, table, len_t, budget, recent=4, sinks=2, dst_table=dst)
    assert torch.cuda.max_memory_allocated() - base <= 8192
    assert q4.q4_sync_status() == q4.Q4_OK and got.tolist() == lens
    for x, y in zip((cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales, mass), before):
        if in_place:
            assert torch.equal(x, y)
        else:
            want = y.clone()
            for b, row in ((0, range(24, 31)), (2, range(31, 34))):
                for i in range(lens[b]):
                    want[row[i // 16], :, i % 16] = y[8 * b + i // 16, :, i % 16]
            assert torch.equal(x, want)
    ws = torch.zeros(12, dtype=torch.uint8, device="cuda")
    got = q4.kv_evict_int8_paged(cache, mass, table, len_t, budget, dst_table=dst, workspace=ws)
    assert q4.q4_sync_status() == q4.Q4_OK and got.tolist() == lens
    with pytest.raises(q4.Q4Error):
        q4.kv_evict_int8_paged(cache, mass, table, len_t, budget, dst_table=dst, workspace=ws[:8])


def test_the_default_stream_by_its_handle():
    """stream=0 inside another stream's block."""
    c = _Case([(400, 1), (300, 1)], 8, 2, 128, 16, BF, seed=4)
    want, wl = c.attention()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got, lse = c.attention(stream=0)
    torch.cuda.synchronize()
    _sync_ok()
    assert torch.equal(got, want) and torch.equal(lse, wl)
