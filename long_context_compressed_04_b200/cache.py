"""The hybrid KV cache of one CSA layer for decode ("DeepSeek-V4 深度分析报告" 3.5, KV cache
management).

- State cache: a fixed-size ring of ``ring`` raw-token rows per sequence (the sliding
  window's KV and the tokens the next entry pools); token p of sequence b sits in row
  b * ring + p mod ring.
- Classical cache: compressed entries (and their indexer keys) in blocks of 128 tokens, i.e.
  32 CSA entries; a block table maps each sequence's blocks to physical blocks, which a
  free list hands out as entries complete.

A decode step appends one token per sequence (``csa_cache_append``: ring row, and the
indexer key of an entry the token completes), compresses the entries completed this step
from the ring into their blocks (``csa_compress``), selects (``lightning_indexer_topk``) and
attends (``sparse_mqa_attn``), every call with the same cache layout.  Indexer keys come
ready-made with the token, or as bf16 / fp32 rows that ``append_keys`` norms, rotates and
quantises on the way into their blocks (``csa_indexer_append``); the key store holds FP8 or
MXFP4 rows.  This module keeps the host-side bookkeeping (block allocation, the item lists of
completed entries, which entries have their key yet: ``select`` refuses queries that see one
without); every copy, compression, score, selection and attention runs in libcsa.
"""
from __future__ import annotations

import contextlib
from typing import List, Optional

import torch

from . import (CSA_IDX_FP8, CSA_IDX_MXFP4, CSA_KV_BF16, cache_layout, csa_cache_append,
               csa_compress, csa_entry_row_bytes, csa_indexer_append,
               csa_indexer_workspace_size, lightning_indexer_topk,
               lightning_indexer_topk_mxfp4, sparse_mqa_attn)

BLOCK_TOKENS = 128      # lcm(m, m') of the pages
M = 4                   # CSA compression ratio
BLOCK_ENTRIES = BLOCK_TOKENS // M


class BlockAllocator:
    """Free list of classical-cache blocks."""

    def __init__(self, n_blocks: int):
        self.free: List[int] = list(range(n_blocks - 1, -1, -1))

    def alloc(self) -> int:
        if not self.free:
            raise RuntimeError("classical cache full")
        return self.free.pop()

    def release(self, blocks):
        self.free.extend(int(x) for x in blocks)


class Items(tuple):
    """(item_seq, item_ent) of entries on the device, with the same as host lists."""

    def __new__(cls, tensors, host):
        self = super().__new__(cls, tensors)
        self.host = host
        return self

    def __getnewargs__(self):
        return tuple(self), self.host


class HybridCache:
    """Device buffers and bookkeeping of one CSA layer's cache for B decode sequences."""

    def __init__(self, B: int, D: int, fmt: int, d_I: int, n_blocks: int, max_blocks: int,
                 ring: int = 128, device="cuda", idx_fmt: int = CSA_IDX_FP8):
        """idx_fmt: the key store's rows, CSA_IDX_FP8 (kI e4m3, ks fp32) or CSA_IDX_MXFP4
        (kI packed e2m1, ks UE8M0 bytes; d_I = 128, as its indexer takes)."""
        if idx_fmt not in (CSA_IDX_FP8, CSA_IDX_MXFP4):
            raise ValueError(f"unknown indexer format {idx_fmt}")
        if idx_fmt == CSA_IDX_MXFP4 and d_I != 128:
            raise ValueError(f"the MXFP4 indexer reads keys of 128 channels, not {d_I}")
        self.B, self.D, self.fmt, self.d_I, self.ring = B, D, fmt, d_I, ring
        self.idx_fmt = idx_fmt
        dev = torch.device(device)
        self.device = dev
        rb = csa_entry_row_bytes(fmt, D)
        rows = n_blocks * BLOCK_ENTRIES
        self.kv = torch.zeros((B * ring, D), dtype=torch.bfloat16, device=dev)
        self.gate = torch.zeros((B * ring, D), dtype=torch.bfloat16, device=dev)
        self.kv_off = torch.arange(B, dtype=torch.int64, device=dev) * ring
        self.entries = torch.zeros((rows, rb), dtype=torch.uint8, device=dev)
        if idx_fmt == CSA_IDX_FP8:
            self.kI = torch.zeros((rows, d_I), dtype=torch.uint8, device=dev)
            self.ks = torch.zeros(rows, dtype=torch.float32, device=dev)
        else:
            self.kI = torch.zeros((rows, d_I // 2), dtype=torch.uint8, device=dev)
            self.ks = torch.zeros((rows, d_I // 32), dtype=torch.uint8, device=dev)
        self.block_table = torch.full((B, max_blocks), -1, dtype=torch.int32, device=dev)
        self.bt_host = torch.full((B, max_blocks), -1, dtype=torch.int32)
        self.seq_len = torch.zeros(B, dtype=torch.int64, device=dev)
        self.len_host = [0] * B
        # a byte per entry of a sequence: its key is in the store; and the complete entries without
        self._keyed = [bytearray(max_blocks * BLOCK_ENTRIES) for _ in range(B)]
        self._unkeyed = [0] * B
        self.alloc = BlockAllocator(n_blocks)
        self.layout = cache_layout(self.block_table, kv_ring=ring)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)

    # ---- bookkeeping ---------------------------------------------------------------
    def _ensure_blocks(self, b: int, n_entries: int):
        need = (n_entries + BLOCK_ENTRIES - 1) // BLOCK_ENTRIES
        changed = False
        for j in range(need):
            if int(self.bt_host[b, j]) < 0:
                self.bt_host[b, j] = self.alloc.alloc()
                changed = True
        return changed

    def _push_table(self):
        self.block_table.copy_(self.bt_host, non_blocking=False)

    def release(self, b: int):
        """Frees sequence b's blocks (the sequence ends)."""
        blocks = [int(x) for x in self.bt_host[b] if int(x) >= 0]
        self.alloc.release(blocks)
        self.bt_host[b] = -1
        self.len_host[b] = 0
        self._set_keyed(b, 0, False)
        self._push_table()
        self.seq_len[b] = 0

    # ---- which entries have their indexer key -----------------------------------------
    def _set_keyed(self, b: int, n: int, keyed: bool):
        """Sequence b anew, with n entries that all have their keys or all lack them."""
        size = len(self._keyed[b])
        self._keyed[b] = bytearray((b"\1" * n if keyed else b"").ljust(size, b"\0"))
        self._unkeyed[b] = 0 if keyed else n

    def note_keys(self, items, stream=None):
        """Entries items[1][j] of sequences items[0][j] have their indexer keys in the store:
        append_keys calls it, and so does one who writes to the store otherwise (a replayed
        graph, say).  Lists that append() returned cost nothing; others are read back from the
        device while entries lack keys, and count as all of those during a stream capture, when
        they cannot be."""
        if not any(self._unkeyed):
            return
        if isinstance(items, Items):
            seqs, ents = items.host
        elif self._capturing(stream):
            for b in range(self.B):
                self._set_keyed(b, self.len_host[b] // M, True)
            return
        else:
            seqs, ents = self._read(stream, *items)
        for b, i in zip(seqs, ents):
            if 0 <= b < self.B and 0 <= i < self.len_host[b] // M and not self._keyed[b][i]:
                self._keyed[b][i] = 1
                self._unkeyed[b] -= 1

    def _on(self, stream):
        return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)

    def _capturing(self, stream):
        with self._on(stream):
            return self.device.type == "cuda" and torch.cuda.is_current_stream_capturing()

    def _read(self, stream, *tensors):
        with self._on(stream):
            return [t.tolist() for t in tensors]

    def _check_keys(self, q_seq, q_pos, stream):
        """Refuses queries that see an entry without its key."""
        if self._capturing(stream):
            return
        for b, p in zip(*self._read(stream, q_seq, q_pos)):
            if 0 <= b < self.B and self._unkeyed[b]:
                i = self._keyed[b].find(0, 0, min((p + 1) // M, self.len_host[b] // M))
                if i >= 0:
                    raise RuntimeError(f"entry {i} of sequence {b} has no indexer key: append_keys "
                                       "brings it (note_keys where something else wrote it)")

    # ---- loading a prefix (set-up) -----------------------------------------------
    def load_prefix(self, b: int, kv_tail, gate_tail, T: int, entries, kI=None, ks=None):
        """Sequence b with T tokens: the last min(T, ring) raw rows (kv_tail, gate_tail, in
        position order), its T // 4 entry rows, indexer keys and scales (in entry order; None:
        append_keys brings them)."""
        n = T // M
        self._ensure_blocks(b, n)
        self._push_table()
        t0 = T - kv_tail.shape[0]
        slots = (torch.arange(t0, T) % self.ring) + b * self.ring
        self.kv[slots.to(self.device)] = kv_tail
        self.gate[slots.to(self.device)] = gate_tail
        i = torch.arange(n)
        rows = (self.bt_host[b, i // BLOCK_ENTRIES].to(torch.int64) * BLOCK_ENTRIES
                + i % BLOCK_ENTRIES).to(self.device)
        self.entries[rows] = entries
        if kI is not None:
            self.kI[rows] = kI
            self.ks[rows] = ks
        self.seq_len[b] = T
        self.len_host[b] = T
        self._set_keyed(b, n, kI is not None)

    # ---- one decode step -----------------------------------------------------------
    def append(self, kv_new, gate_new, kI_new=None, ks_new=None, stream=None):
        """One token per sequence (bf16 [B, D] raw KV and gate; with an FP8 key store, e4m3
        [B, d_I] indexer key and fp32 [B] scale, used by the sequences whose token completes
        an entry; None: append_keys brings the keys).  Returns the (item_seq, item_ent) lists
        of the entries completed, for compress() and append_keys()."""
        if kI_new is not None and self.idx_fmt != CSA_IDX_FP8:
            raise ValueError("ready-made keys are copied into an FP8 key store only: use append_keys")
        changed = False
        for b in range(self.B):
            changed |= self._ensure_blocks(b, (self.len_host[b] + 1) // M)
        if changed:
            self._push_table()
        csa_cache_append(kv_new, gate_new, self.seq_len, self.kv_off, None, self.kv, self.gate,
                         B=self.B, D=self.D, m=M, kI_new=kI_new, kI_scale_new=ks_new,
                         kI=None if kI_new is None else self.kI,
                         kI_scale=None if kI_new is None else self.ks, layout=self.layout,
                         dev_status=self.dev_status, stream=stream)
        seqs, ents = [], []
        for b in range(self.B):
            self.len_host[b] += 1
            if self.len_host[b] % M == 0:
                i = self.len_host[b] // M - 1
                seqs.append(b)
                ents.append(i)
                self._keyed[b][i] = kI_new is not None
                self._unkeyed[b] += kI_new is None
        return Items((torch.tensor(seqs, dtype=torch.int32, device=self.device),
                      torch.tensor(ents, dtype=torch.int32, device=self.device)), (seqs, ents))

    def append_keys(self, items, k, weight=None, norm: bool = True, rope_dims: int = 64,
                    rope_theta=10000.0, eps=1e-6, stream=None):
        """Indexer keys of entries already in the cache's sequences: k [n, d_I] (bf16, fp16 or
        fp32), row j for entry items[1][j] of sequence items[0][j]; normed, rotated at the
        entries' block ends, quantised and written to their blocks."""
        seq, ent = items
        if seq.numel() == 0:
            return
        csa_indexer_append(k, self.seq_len, None, seq, ent, self.kI, self.ks, B=self.B, m=M,
                           fmt=self.idx_fmt, weight=weight, norm=norm, rope_dims=rope_dims,
                           rope_theta=rope_theta, eps=eps, layout=self.layout,
                           dev_status=self.dev_status, stream=stream)
        self.note_keys(items, stream)

    def compress(self, items, bias, rope_theta=10000.0, eps=1e-6, stream=None):
        seq, ent = items
        if seq.numel() == 0:
            return
        csa_compress(self.kv, self.gate, bias, self.seq_len, self.kv_off, None, None, seq, ent,
                     self.entries, B=self.B, D=self.D, fmt=self.fmt, rope_theta=rope_theta,
                     eps=eps, layout=self.layout, dev_status=self.dev_status, stream=stream)

    def select(self, qI, qs, w, q_seq, q_pos, idx_out, *, H_I: int, k: int,
               workspace: Optional[torch.Tensor] = None, stream=None,
               select_bf16: bool = False):
        """Top-k of every query; qI, qs: e4m3 codes and fp32 scales, or with an MXFP4 key
        store packed codes and scale bytes (select_bf16 as in lightning_indexer_topk_mxfp4).
        Queries that see an entry whose key was never brought are refused (RuntimeError)."""
        if any(self._unkeyed):
            self._check_keys(q_seq, q_pos, stream)
        max_n = max(self.len_host) // M
        if workspace is None:
            workspace = torch.empty(max(csa_indexer_workspace_size(q_seq.numel(), max(max_n, 1), k), 256),
                                    dtype=torch.uint8, device=self.device)
        if self.idx_fmt == CSA_IDX_MXFP4:
            lightning_indexer_topk_mxfp4(qI, qs, w, self.kI, self.ks, self.seq_len, None, q_seq,
                                         q_pos, idx_out, workspace, B=self.B, H_I=H_I,
                                         d_I=self.d_I, m=M, k=k, max_n=max(max_n, 1),
                                         select_bf16=select_bf16, layout=self.layout,
                                         dev_status=self.dev_status, stream=stream)
            return
        lightning_indexer_topk(qI, qs, w, self.kI, self.ks, self.seq_len, None, q_seq, q_pos,
                               idx_out, workspace, B=self.B, H_I=H_I, d_I=self.d_I, m=M, k=k,
                               max_n=max(max_n, 1), layout=self.layout,
                               dev_status=self.dev_status, stream=stream)

    def attend(self, q, q_seq, q_pos, idx, sink, out, *, H: int, W: int, k: int,
               softmax_scale: float, rope_theta=10000.0, eps=1e-6, stream=None):
        sparse_mqa_attn(q, self.entries, self.seq_len, None, self.kv, self.kv_off, None, q_seq,
                        q_pos, idx, sink, out, fmt=self.fmt, B=self.B, H=H, D=self.D, W=W, m=M,
                        k=k, softmax_scale=softmax_scale, rope_theta=rope_theta, eps=eps,
                        layout=self.layout, dev_status=self.dev_status, stream=stream)


__all__ = ["BlockAllocator", "HybridCache", "Items", "BLOCK_TOKENS", "BLOCK_ENTRIES", "CSA_KV_BF16"]
