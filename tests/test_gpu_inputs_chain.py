"""The operators that make the indexer's inputs, run together as a layer runs them: hidden
states through the MXFP4 query projection, the heads' norm, rotation and quantisation; keys
appended to the hybrid cache's blocks; selection and attention on what they wrote.

Codes are compared bit for bit with the 64-bit forms, and the index sets with the same selection
from a contiguous store.  The
projection's inputs keep fp32 sums exact (K = 256 and block exponents within a few binades:
multiples of 2^-6 below 2^14), so nothing between the hidden states and the codes rounds twice."""
import numpy as np
import pytest
import torch

import _inputs_orc as io
import long_context_compressed_04_b200 as L
from long_context_compressed_04_b200 import cache, pipeline

pytestmark = pytest.mark.gpu
DEV = "cuda"
K, HI, DI, D, H, TOPK = 256, 64, 128, 128, 64, 64


def _hidden(g, n):
    return torch.randn((n, K), generator=g, device=DEV).to(torch.bfloat16)


def _f64(t):
    return t.detach().cpu().double().numpy()


def _heads_ref(x, w, pos, head_w, fmt):
    """The query heads' codes and scales in 64 bits."""
    a, b = (io.mxfp4_values(*io.mxfp4(_f64(t))) for t in (x, w))
    y = torch.from_numpy(a @ b.T).to(torch.bfloat16)
    y = io.norm_rope(_f64(y).reshape(len(a), HI, DI), pos.cpu().numpy(), _f64(head_w))
    return io.fp8(y) if fmt == L.CSA_IDX_FP8 else io.mxfp4(y)


def _keys_ref(k, ent, key_w, fmt):
    y = io.norm_rope(_f64(k)[:, None], (np.asarray(ent, np.int64) + 1) * 4 - 1, _f64(key_w))[:, 0]
    return io.fp8(y) if fmt == L.CSA_IDX_FP8 else io.mxfp4(y)


def _select(fmt, qI, qs, w, kI, ks, seq_len, off, q_seq, q_pos, idx, max_n):
    ws = torch.empty(L.csa_indexer_workspace_size(q_seq.numel(), max_n, TOPK), dtype=torch.uint8, device=DEV)
    fn = L.lightning_indexer_topk if fmt == L.CSA_IDX_FP8 else L.lightning_indexer_topk_mxfp4
    fn(qI, qs, w, kI, ks, seq_len, off, q_seq, q_pos, idx, ws, B=seq_len.numel(), H_I=HI, d_I=DI, m=4,
       k=TOPK, max_n=max_n)


def _same_scales(got, ref):
    """Scale bytes exactly, fp32 scales to their 30 roundings of 2^-24 (see test_gpu_inputs)."""
    got = got.cpu().numpy()
    assert np.array_equal(got, ref) if ref.dtype == np.uint8 else np.all(np.abs(got - ref) <= 30 * 2.0 ** -24 * ref)


def _up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


@pytest.mark.parametrize("fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
def test_decode_steps_match_the_64_bit_forms(fmt):
    g = torch.Generator(device=DEV).manual_seed(17)
    T0, S = [1001, 130, 515], 9
    B = len(T0)
    Tmax = [t + S for t in T0]
    n_max = [t // 4 for t in Tmax]
    off = np.concatenate([[0], np.cumsum(n_max)[:-1]]).astype(np.int64)
    head_w, key_w = (1 + 0.2 * torch.randn(DI, generator=g, device=DEV) for _ in range(2))
    proj_w = (torch.randn((HI * DI, K), generator=g, device=DEV) / 16).to(torch.bfloat16)
    keys = torch.randn((sum(n_max), DI), generator=g, device=DEV).to(torch.bfloat16)
    kv, gate = (torch.randn((sum(Tmax), D), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    kv_off = np.concatenate([[0], np.cumsum(Tmax)[:-1]]).astype(np.int64)
    bias = torch.randn((8, D), generator=g, device=DEV) * 0.1
    sink = torch.randn(H, generator=g, device=DEV)
    # a contiguous store of every key the run will use; the codes are the 64-bit forms'
    ient = np.concatenate([np.arange(n) for n in n_max]).astype(np.int32)
    kI_ref, ks_ref = _keys_ref(keys, ient, key_w, fmt)
    kI_lin, ks_lin = torch.zeros_like(_up(kI_ref)), torch.zeros_like(_up(ks_ref))
    L.csa_indexer_append(keys, torch.tensor(Tmax, device=DEV), _up(off),
                         _up(np.repeat(np.arange(B, dtype=np.int32), n_max)), _up(ient), kI_lin, ks_lin, B=B,
                         fmt=fmt, weight=key_w)
    assert np.array_equal(kI_lin.cpu().numpy(), kI_ref)
    _same_scales(ks_lin, ks_ref)

    proj = pipeline.QueryProjection(proj_w, HI, DI, max_q=8, fmt=fmt, head_weight=head_w)
    hc = cache.HybridCache(B, D, 0, DI, n_blocks=40, max_blocks=12, device=DEV, idx_fmt=fmt)
    hc.alloc.free = torch.randperm(40, generator=torch.Generator().manual_seed(5)).tolist()
    for b, T in enumerate(T0):          # the prefix: raw tail, entries from their tokens, keys
        r0, lo = int(kv_off[b]), max(T - 128, 0)
        n = T // 4
        ents = torch.zeros((n, 2 * D), dtype=torch.uint8, device=DEV)
        i32 = torch.arange(n, dtype=torch.int32, device=DEV)
        L.csa_compress(kv[r0:r0 + T], gate[r0:r0 + T], bias, torch.tensor([T], device=DEV),
                       torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV),
                       torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros_like(i32), i32, ents, B=1, D=D)
        hc.load_prefix(b, kv[r0 + lo:r0 + T], gate[r0 + lo:r0 + T], T, ents)
        hc.append_keys((torch.full((n,), b, dtype=torch.int32, device=DEV), i32), keys[off[b]:off[b] + n], key_w)

    q_seq = torch.arange(B, dtype=torch.int32, device=DEV)
    for s in range(S):
        p = [t + s for t in T0]
        rows = torch.tensor([int(kv_off[b]) + p[b] for b in range(B)], device=DEV)
        x = _hidden(g, B)
        w = torch.rand((B, HI), generator=g, device=DEV)
        q = torch.randn((B, H, D), generator=g, device=DEV).to(torch.bfloat16)
        q_pos = torch.tensor(p, dtype=torch.int32, device=DEV)
        # the step: append, compress and key the completed entries, project, select, attend
        items = hc.append(kv[rows], gate[rows])
        hc.compress(items, bias)
        done = list(zip(items[0].tolist(), items[1].tolist()))
        if done:
            hc.append_keys(items, keys[torch.tensor([int(off[b]) + i for b, i in done], device=DEV)], key_w)
        qI, qs = proj(x, q_pos)
        L.csa_qk_norm_rope(q, None, q_pos, q, None, rope_dims=0)
        idx = torch.full((B, TOPK), -1, dtype=torch.int32, device=DEV)
        hc.select(qI, qs, w, q_seq, q_pos, idx, H_I=HI, k=TOPK)
        out = torch.zeros((B, H, D), dtype=torch.bfloat16, device=DEV)
        hc.attend(q, q_seq, q_pos, idx, sink, out, H=H, W=128, k=TOPK, softmax_scale=D ** -0.5)
        torch.cuda.synchronize()
        assert int(hc.dev_status.item()) == 0 and int(proj.dev_status.item()) == 0, s
        ref = _heads_ref(x, proj_w, q_pos, head_w, fmt)
        assert np.array_equal(qI.cpu().numpy(), ref[0]), s
        _same_scales(qs, ref[1])
        # the same selection from the contiguous store
        idx_ref = torch.full_like(idx, -1)
        _select(fmt, _up(ref[0]), qs.clone(), w, kI_lin, ks_lin, torch.tensor([t + 1 for t in p], device=DEV),
                _up(off), q_seq, q_pos, idx_ref, max(t + 1 for t in p) // 4)
        assert torch.equal(idx, idx_ref), s
        assert bool(out.isfinite().all())
    # every key in its block
    for b in range(B):
        i = torch.arange(Tmax[b] // 4)
        at = (hc.bt_host[b, i // 32].to(torch.int64) * 32 + i % 32).to(DEV)
        e0 = int(off[b])
        assert torch.equal(hc.kI[at], kI_lin[e0:e0 + len(i)]) and torch.equal(hc.ks[at], ks_lin[e0:e0 + len(i)])


@pytest.mark.parametrize("fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
def test_captured_chain_replays_and_overlaps_exactly(fmt):
    """Append, projection and selection as one graph, replayed on new inputs without a wait
    in between, twice over the same buffers: each launch may start while its predecessor
    finishes, and every replay has to give what separate, synchronised calls give."""
    g = torch.Generator(device=DEV).manual_seed(23)
    B, n, Q = 3, 700, 3
    T = 4 * n
    proj_w = (torch.randn((HI * DI, K), generator=g, device=DEV) / 16).to(torch.bfloat16)
    proj = pipeline.QueryProjection(proj_w, HI, DI, max_q=Q, fmt=fmt)
    seq_len = torch.full((B,), T, dtype=torch.int64, device=DEV)
    off = torch.arange(B, dtype=torch.int64, device=DEV) * n
    iseq = torch.arange(B, dtype=torch.int32, device=DEV).repeat_interleave(n)
    ient = torch.arange(n, dtype=torch.int32, device=DEV).repeat(B)
    kI = torch.zeros((B * n, DI if fmt == L.CSA_IDX_FP8 else DI // 2), dtype=torch.uint8, device=DEV)
    ks = torch.zeros(B * n, device=DEV) if fmt == L.CSA_IDX_FP8 else \
        torch.zeros((B * n, DI // 32), dtype=torch.uint8, device=DEV)
    x, keys = _hidden(g, Q), torch.zeros((B * n, DI), dtype=torch.bfloat16, device=DEV)
    w = torch.rand((Q, HI), generator=g, device=DEV)
    q_seq = torch.arange(Q, dtype=torch.int32, device=DEV)
    q_pos = torch.full((Q,), T - 1, dtype=torch.int32, device=DEV)
    idx = torch.full((Q, TOPK), -1, dtype=torch.int32, device=DEV)
    ws = torch.empty(L.csa_indexer_workspace_size(Q, n, TOPK), dtype=torch.uint8, device=DEV)
    fn = L.lightning_indexer_topk if fmt == L.CSA_IDX_FP8 else L.lightning_indexer_topk_mxfp4

    def step():
        L.csa_indexer_append(keys, seq_len, off, iseq, ient, kI, ks, B=B, fmt=fmt)
        qI, qs = proj(x, q_pos)
        fn(qI, qs, w, kI, ks, seq_len, off, q_seq, q_pos, idx, ws, B=B, H_I=HI, d_I=DI, m=4, k=TOPK, max_n=n)

    data = [(_hidden(g, Q), torch.randn((B * n, DI), generator=g, device=DEV).to(torch.bfloat16))
            for _ in range(6)]
    want = []
    for a, b in data:
        x.copy_(a), keys.copy_(b)
        step()
        torch.cuda.synchronize()
        want.append((idx.clone(), proj.codes.clone(), kI.clone()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):                   # two graphs over the same workspaces
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            step()
            step()                       # overwrites in place what the first one read
        graphs.append(gr)
    got = []
    for r in range(12):
        x.copy_(data[r % 6][0]), keys.copy_(data[r % 6][1])
        graphs[r % 2].replay()
        got.append((idx.clone(), proj.codes.clone(), kI.clone()))
    torch.cuda.synchronize()
    for r in range(12):
        for a, b in zip(got[r], want[r % 6]):
            assert torch.equal(a, b), r
    # the same without a graph, calls back to back
    got = []
    for r in range(12):
        x.copy_(data[r % 6][0]), keys.copy_(data[r % 6][1])
        step()
        step()
        got.append((idx.clone(), proj.codes.clone(), kI.clone()))
    torch.cuda.synchronize()
    for r in range(12):
        for a, b in zip(got[r], want[r % 6]):
            assert torch.equal(a, b), r


def test_projection_and_cache_refuse_what_they_cannot_hold():
    w = torch.zeros((HI * DI, K), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="rows"):
        pipeline.QueryProjection(w[1:], HI, DI, max_q=4)
    proj = pipeline.QueryProjection(w, HI, DI, max_q=4)
    pos = torch.zeros(5, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="at most 4"):
        proj(torch.zeros((5, K), dtype=torch.bfloat16, device=DEV), pos)
    with pytest.raises(L.CSAError, match="q_pos"):
        proj(torch.zeros((3, K), dtype=torch.bfloat16, device=DEV), pos)
    with pytest.raises(ValueError, match="format"):
        cache.HybridCache(1, 128, 0, 128, n_blocks=2, max_blocks=2, device=DEV, idx_fmt=7)
    hc = cache.HybridCache(1, 128, 0, 128, n_blocks=2, max_blocks=2, device=DEV, idx_fmt=L.CSA_IDX_MXFP4)
    z = torch.zeros((1, 128), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="append_keys"):
        hc.append(z, z, z.to(torch.uint8), torch.zeros(1, device=DEV))


def test_normed_queries_go_straight_into_the_attention():
    """csa_qk_norm_rope directly before the attention that reads its rows ahead of its own wait:
    back to back on changing inputs, against synchronised calls."""
    g = torch.Generator(device=DEV).manual_seed(29)
    B, T, k = 4, 3000, 64
    kv = torch.randn((B * T, D), generator=g, device=DEV).to(torch.bfloat16)
    ents = torch.randn((B * T // 4, D), generator=g, device=DEV).to(torch.bfloat16).view(torch.uint8)
    i64 = lambda v: torch.tensor(v, dtype=torch.int64, device=DEV)  # noqa: E731
    seq_len, off, kvo, p0 = i64([T] * B), i64([b * (T // 4) for b in range(B)]), i64([b * T for b in range(B)]), i64([0] * B)
    q_seq = torch.arange(B, dtype=torch.int32, device=DEV)
    q_pos = torch.full((B,), T - 1, dtype=torch.int32, device=DEV)
    idx = torch.stack([torch.randperm(T // 4, generator=g, device=DEV)[:k].sort().values for _ in range(B)]).to(torch.int32)
    sink = torch.randn(H, generator=g, device=DEV)
    w = 1 + 0.2 * torch.randn(D, generator=g, device=DEV)
    data = [torch.randn((B, H, D), generator=g, device=DEV).to(torch.bfloat16) for _ in range(5)]
    q, qn = torch.empty_like(data[0]), torch.empty_like(data[0])
    out = torch.empty_like(q)

    def step(sync):
        L.csa_qk_norm_rope(q, None, q_pos, qn, None, q_weight=w, rope_dims=0)
        if sync:
            torch.cuda.synchronize()
        L.sparse_mqa_attn(qn, ents, seq_len, off, kv, kvo, p0, q_seq, q_pos, idx, sink, out, fmt=0, B=B, H=H, D=D,
                          W=128, m=4, k=k, softmax_scale=D ** -0.5)

    want, got = [], []
    for r in range(5):
        q.copy_(data[r])
        step(True)
        want.append(out.clone())
    for r in range(20):
        q.copy_(data[r % 5])
        step(False)
        got.append(out.clone())
    for r in range(20):              # and without a copy in between: the previous attention still runs
        step(False)
    torch.cuda.synchronize()
    for r in range(20):
        assert torch.equal(got[r], want[r % 5]), r
    assert torch.equal(out, want[19 % 5])


def test_projection_on_another_stream_than_it_was_built_on():
    # the building stream is busy; the first call goes to another one.  A weight with a NaN is
    # reported where the calls report
    g = torch.Generator(device=DEV).manual_seed(31)
    proj_w = (torch.randn((HI * DI, K), generator=g, device=DEV) / 16).to(torch.bfloat16)
    x, pos = _hidden(g, 4), torch.arange(4, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    proj = pipeline.QueryProjection(proj_w, HI, DI, max_q=4)
    qI, qs = proj(x, pos, stream=side)
    side.synchronize()
    ref = _heads_ref(x, proj_w, pos, torch.ones(DI), L.CSA_IDX_FP8)
    assert np.array_equal(qI.cpu().numpy(), ref[0])
    _same_scales(qs, ref[1])
    assert int(proj.dev_status.item()) == 0
    proj_w[77, 5] = float("nan")
    assert int(pipeline.QueryProjection(proj_w, HI, DI, max_q=4).dev_status.item()) == L.CSA_DEV_NAN


@pytest.mark.parametrize("fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
def test_select_refuses_missing_keys_on_any_stream_and_inside_a_capture(fmt):
    # lists on the device are read on the stream they are used on; a capture reads nothing
    g = torch.Generator(device=DEV).manual_seed(37)
    hc = cache.HybridCache(2, D, 0, DI, n_blocks=8, max_blocks=4, device=DEV, idx_fmt=fmt)
    tail = torch.randn((128, D), generator=g, device=DEV).to(torch.bfloat16)
    ents = torch.zeros((64, 2 * D), dtype=torch.uint8, device=DEV)
    keys = torch.randn((128, DI), generator=g, device=DEV).to(torch.bfloat16)
    for b in range(2):
        hc.load_prefix(b, tail, tail, 256, ents)
    i = torch.arange(64, dtype=torch.int32, device=DEV)
    proj = pipeline.QueryProjection((torch.randn((HI * DI, K), generator=g, device=DEV) / 16).to(torch.bfloat16), HI, DI,
                                    max_q=2, fmt=fmt)
    q_seq, q_pos = i[:2].clone(), torch.full((2,), 255, dtype=torch.int32, device=DEV)
    w = torch.rand((2, HI), generator=g, device=DEV)
    qI, qs = proj(_hidden(g, 2), q_pos)
    idx = torch.full((2, 16), -1, dtype=torch.int32, device=DEV)
    ws = torch.empty(L.csa_indexer_workspace_size(2, 64, 16), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    select = lambda s=None: hc.select(qI, qs, w, q_seq, q_pos, idx, H_I=HI, k=16, workspace=ws, stream=s)  # noqa: E731
    with torch.cuda.stream(side):
        torch.cuda._sleep(5_000_000)
        seq = torch.zeros_like(i) + 1
    hc.append_keys((seq, i), keys[64:], stream=side)
    with pytest.raises(RuntimeError, match="sequence 0"):
        select(side)
    hc.append_keys((torch.zeros_like(i), i), keys[:64])
    torch.cuda.synchronize()
    select()
    want = idx.clone()
    items = torch.cat([torch.zeros_like(i), seq]), torch.cat([i, i])
    for b in range(2):
        hc.load_prefix(b, tail, tail, 256, ents)
    hc.kI.zero_()
    idx.fill_(-1)
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        hc.append_keys(items, keys)
        select()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(idx, want) and int(hc.dev_status.item()) == 0
    select()
    assert torch.equal(idx, want)
