"""Host-side bookkeeping of the hybrid cache (no GPU): the block free list, block-table growth
as entries complete, release, and the layout struct handed to the C calls."""
import copy
import ctypes
import pickle

import pytest
import torch

import long_context_compressed_04_b200 as L
from long_context_compressed_04_b200 import cache


def test_block_allocator_order_exhaustion_and_release():
    a = cache.BlockAllocator(3)
    assert [a.alloc(), a.alloc()] == [0, 1]
    a.release([0])
    assert a.alloc() == 0 and a.alloc() == 2
    with pytest.raises(RuntimeError, match="full"):
        a.alloc()


def test_blocks_follow_completed_entries():
    hc = cache.HybridCache(2, 128, L.CSA_KV_BF16, 128, n_blocks=8, max_blocks=4, device="cpu")
    # 32 entries fill one block of 128 tokens; the 33rd needs a second
    assert hc._ensure_blocks(0, 32) and int((hc.bt_host[0] >= 0).sum()) == 1
    assert not hc._ensure_blocks(0, 32)
    assert hc._ensure_blocks(0, 33) and int((hc.bt_host[0] >= 0).sum()) == 2
    assert hc._ensure_blocks(1, 1)
    used = sorted(int(x) for x in hc.bt_host.flatten() if int(x) >= 0)
    assert used == [0, 1, 2] and len(hc.alloc.free) == 5
    hc.release(0)
    assert int((hc.bt_host[0] >= 0).sum()) == 0 and len(hc.alloc.free) == 7
    assert torch.equal(hc.block_table, hc.bt_host)


def test_layout_struct_fields():
    assert L.cache_layout() is None
    bt = torch.zeros((3, 5), dtype=torch.int32)
    lay = L.cache_layout(bt, kv_ring=128)
    assert lay.block_table == bt.data_ptr() and lay.bt_stride == 5 and lay.kv_ring == 128
    assert ctypes.sizeof(L.CacheLayout) == 24
    ring_only = L.cache_layout(kv_ring=64)
    assert ring_only.block_table is None and ring_only.kv_ring == 64


def test_layout_validation_on_the_host():
    # a block table needs m = 4; the check runs before any launch
    lib = L._lib
    fake = ctypes.c_void_p(4096)
    bt = torch.zeros((1, 4), dtype=torch.int32)
    lay = L.cache_layout(bt)
    st = lib.hca_compress(fake, fake, fake, fake, fake, None, None, fake, fake, 1, 1, 128, 0,
                          10000.0, 1e-6, fake, ctypes.byref(lay), None, None)
    assert st == 1 and b"m = 4" in lib.csa_last_error()
    # without a block table, ent_off is required
    st = lib.csa_compress(fake, fake, fake, fake, fake, fake, None, fake, fake, 1, 1, 128, 0,
                          10000.0, 1e-6, fake, None, None, None)
    assert st == 1 and b"ent_off" in lib.csa_last_error()


@pytest.fixture
def calls(monkeypatch):
    """The library's calls that the cache makes, named in order instead of made."""
    seen = []
    for name in ("csa_cache_append", "csa_indexer_append", "lightning_indexer_topk", "lightning_indexer_topk_mxfp4"):
        monkeypatch.setattr(cache, name, lambda *a, _n=name, **kw: seen.append(_n))
    return seen


def _decode_cache(idx_fmt, B=2):
    hc = cache.HybridCache(B, 128, L.CSA_KV_BF16, 128, n_blocks=8, max_blocks=4, device="cpu", idx_fmt=idx_fmt)
    kv = torch.zeros((B, 128), dtype=torch.bfloat16)

    def select(q_pos=None, seqs=None):
        seqs = list(range(B)) if seqs is None else seqs
        q_pos = [hc.len_host[b] - 1 for b in seqs] if q_pos is None else q_pos
        hc.select(None, None, None, torch.tensor(seqs, dtype=torch.int32), torch.tensor(q_pos, dtype=torch.int32),
                  None, H_I=64, k=8)
    return hc, kv, select


@pytest.mark.parametrize("idx_fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
def test_select_refuses_entries_without_their_key(calls, idx_fmt):
    hc, kv, select = _decode_cache(idx_fmt)
    k = torch.zeros((2, 128), dtype=torch.bfloat16)
    for _ in range(3):
        assert hc.append(kv, kv)[0].numel() == 0
    select()                                       # no entry yet
    items = hc.append(kv, kv)                      # entry 0 of both sequences
    assert isinstance(items, tuple) and items[0].tolist() == [0, 1] and items[1].tolist() == [0, 0]
    with pytest.raises(RuntimeError, match="entry 0 of sequence 0 has no indexer key"):
        select()
    select([2, 2])                                 # queries that see no entry
    hc.append_keys((items[0][1:], items[1][1:]), k[1:])
    select(seqs=[1])
    with pytest.raises(RuntimeError, match="sequence 0"):
        select()
    hc.append_keys(items, k)                       # an entry twice counts once
    select()
    for _ in range(4):
        items2 = hc.append(kv, kv)
    hc.append_keys(items, k)                       # the wrong entries
    with pytest.raises(RuntimeError, match="entry 1 of sequence 0"):
        select()
    hc.note_keys(items2)                           # brought by other means
    select()
    n = len(calls)
    hc.append_keys((items2[0][:0], items2[1][:0]), k[:0])
    assert len(calls) == n and calls.count("csa_indexer_append") == 3


def test_select_refuses_a_prefix_and_a_reused_sequence_without_keys(calls):
    hc, kv, select = _decode_cache(L.CSA_IDX_FP8)
    row = L.csa_entry_row_bytes(L.CSA_KV_BF16, 128)
    ents, kI, ks = torch.zeros((50, row), dtype=torch.uint8), torch.zeros((50, 128), dtype=torch.uint8), torch.ones(50)
    tail = torch.zeros((128, 128), dtype=torch.bfloat16)
    hc.load_prefix(0, tail, tail, 201, ents, kI, ks)
    hc.load_prefix(1, tail, tail, 201, ents)
    select(seqs=[0])
    with pytest.raises(RuntimeError, match="entry 0 of sequence 1"):
        select()
    i = torch.arange(50, dtype=torch.int32)
    bad = torch.tensor([-1, 1, 1, 7], dtype=torch.int32), torch.tensor([0, 50, -1, 0], dtype=torch.int32)
    hc.append_keys(bad, torch.zeros((4, 128)))     # entries that are not there (flagged by the call itself)
    hc.append_keys((torch.ones_like(i[:49]), i[:49]), torch.zeros((49, 128)))
    select([196, 196])                             # sees 49 entries
    with pytest.raises(RuntimeError, match="entry 49 of sequence 1"):
        select([200, 199])
    hc.append_keys((torch.ones_like(i[49:]), i[49:]), torch.zeros((1, 128)))
    select()
    # the next user of a sequence has no keys of the last one's
    hc.release(1)
    select()
    hc.load_prefix(1, tail, tail, 100, ents[:25])
    with pytest.raises(RuntimeError, match="entry 0 of sequence 1"):
        select()
    hc.load_prefix(1, tail, tail, 100, ents[:25], kI[:25], ks[:25])
    select()
    # ready-made keys with the tokens
    for _ in range(5):
        hc.append(kv, kv, torch.zeros((2, 128), dtype=torch.uint8), torch.ones(2))
    select()
    assert hc._unkeyed == [0, 0]


def test_a_store_that_no_indexer_reads_is_refused():
    # the MXFP4 indexer takes 128 channels only: the cache says so when it is made, not in select
    with pytest.raises(ValueError, match="128 channels, not 64"):
        cache.HybridCache(1, 128, 0, 64, n_blocks=2, max_blocks=2, device="cpu", idx_fmt=L.CSA_IDX_MXFP4)
    for d, f in ((64, L.CSA_IDX_FP8), (128, L.CSA_IDX_FP8), (128, L.CSA_IDX_MXFP4)):
        cache.HybridCache(1, 128, 0, d, n_blocks=2, max_blocks=2, device="cpu", idx_fmt=f)


def test_item_lists_are_tuples_that_can_be_copied(calls):
    hc, kv, _ = _decode_cache(L.CSA_IDX_FP8)
    for _ in range(4):
        items = hc.append(kv, kv)
    seq, ent = items
    for c in (copy.copy(items), copy.deepcopy(items), pickle.loads(pickle.dumps(items))):
        assert torch.equal(c[0], seq) and torch.equal(c[1], ent) and c.host == ([0, 1], [0, 0])
