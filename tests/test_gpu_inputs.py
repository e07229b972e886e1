"""GPU parity of the operators that make the indexer's inputs with their 64-bit forms.

Codes, scale bytes, stored query heads and keys are compared bit for bit: the quantisers
are exact by construction.  Products of inputs whose sums fp32 holds exactly have to equal the
rounded 64-bit product; others are held to a bound from the accumulation order.  Norm and
rotation in fp32 are held to a bound counted in roundings."""
import numpy as np
import pytest
import torch

import _inputs_orc as io
import long_context_compressed_04_b200 as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _sync(st, want=0):
    torch.cuda.synchronize()
    assert int(st.item()) == want


def f64(t):
    return t.detach().cpu().double().numpy()


def _gpu(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV) if dtype is None else \
        torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def _sf_empty(rows, cols, lay):
    n = L.csa_mxfp4_sf_bytes(rows, cols, lay)
    return torch.full((n,) if lay == L.CSA_SF_TILED else (rows, cols // 32), 0xAA, dtype=torch.uint8,
                      device=DEV)


# ---- MXFP4 quantisation --------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (3, 96, 8), (127, 160, 0), (129, 128, 32),
                                           (1000, 2048, 0), (33, 4064, 16)])
def test_quantize_and_back_bit_exact(rows, cols, pad, tiled, dt):
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    x = torch.randn((rows, cols + pad), generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-8, 9, (rows, 1), generator=g, device=DEV).float())
    x = x.to(DT[dt])[:, :cols]
    lay = L.CSA_SF_TILED if tiled else L.CSA_SF_ROWS
    codes = torch.full((rows, cols // 2), 0x55, dtype=torch.uint8, device=DEV)
    sf, st = _sf_empty(rows, cols, lay), _status()
    L.csa_mxfp4_quantize(x, codes, sf, sf_layout=lay, dev_status=st)
    _sync(st)
    p, s = io.mxfp4(f64(x))
    assert np.array_equal(codes.cpu().numpy(), p)
    assert np.array_equal(sf.cpu().numpy(), io.tile_scales(s) if tiled else s)
    ref = io.mxfp4_values(p, s)
    for out_dt in DT.values():
        out = torch.full((rows, cols + pad), 7.0, dtype=out_dt, device=DEV)
        L.csa_mxfp4_dequantize(codes, sf, out[:, :cols], sf_layout=lay)
        torch.cuda.synchronize()
        want = torch.from_numpy(ref).to(out_dt)
        assert torch.equal(out[:, :cols].cpu(), want)
        assert bool((out[:, cols:] == 7.0).all())


def test_quantize_borders_and_extremes():
    # every midpoint (a tie) and its neighbours in fp32, at scales over the whole exponent
    # range (subnormals among them), zeros of both signs
    mids = (io.LEVELS[1:] + io.LEVELS[:-1]) / 2
    base = np.concatenate([mids, mids * (1 + 2.0 ** -22), mids * (1 - 2.0 ** -22), io.LEVELS[1:]])
    base = np.concatenate([base, [0.0, -0.0, 6.0, 4.0]])
    rows = [np.roll(base, r) * (-1) ** np.arange(32) * 2.0 ** e
            for r, e in enumerate([0, 1, -1, 60, -60, 125, -126, -128, -133, -149])]
    rows += [np.zeros(32), -np.zeros(32), np.full(32, 2.0 ** -149),
             np.full(32, np.finfo(np.float32).max)]
    x = np.stack(rows).astype(np.float32)
    codes = torch.empty((len(x), 16), dtype=torch.uint8, device=DEV)
    sf, st = _sf_empty(len(x), 32, 0), _status()
    L.csa_mxfp4_quantize(_gpu(x), codes, sf, dev_status=st)
    _sync(st)
    p, s = io.mxfp4(x.astype(np.float64))
    assert np.array_equal(sf.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), p)
    out = torch.empty((len(x), 32), device=DEV)
    L.csa_mxfp4_dequantize(codes, sf, out)
    torch.cuda.synchronize()
    assert np.array_equal(f64(out), io.mxfp4_values(p, s).astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_marks_non_finite_blocks(bad):
    x = torch.randn((40, 128), device=DEV).to(torch.bfloat16)
    x[17, 70] = bad
    codes, sf, st = torch.empty((40, 64), dtype=torch.uint8, device=DEV), _sf_empty(40, 128, 0), _status()
    L.csa_mxfp4_quantize(x, codes, sf, dev_status=st)
    _sync(st, L.CSA_DEV_NAN)
    p, s = io.mxfp4(f64(x))
    assert s[17, 2] == 255 and (s == 255).sum() == 1
    assert np.array_equal(codes.cpu().numpy(), p) and np.array_equal(sf.cpu().numpy(), s)
    out = torch.empty((40, 128), device=DEV)
    L.csa_mxfp4_dequantize(codes, sf, out)
    assert bool(out[17, 64:96].isnan().all()) and int(out.isnan().sum()) == 32


# ---- MXFP4 product ---------------------------------------------------------------------------
def _operands(rng, M, N, K, lo, hi):
    """Random codes and scale bytes, and their values."""
    out = []
    for r in (M, N):
        c = rng.integers(0, 16, (r, K)).astype(np.uint8)
        s = rng.integers(lo, hi + 1, (r, K // 32)).astype(np.uint8)
        out.append((io.pack(c), s, io.mxfp4_values(io.pack(c), s)))
    return out


def _matmul(a, b, dt, ld=None, st=None, fill=0):
    M, N = len(a[0]), len(b[0])
    out = torch.full((M, ld or N), 3.0, dtype=DT[dt], device=DEV)
    L.csa_mxfp4_matmul(_gpu(a[0]), _gpu(io.tile_scales(a[1], fill)), _gpu(b[0]),
                       _gpu(io.tile_scales(b[1], fill)), out[:, :N], dev_status=st)
    return out


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 128, 64), (3, 130, 96), (8, 8192, 256),
                                   (16, 96, 2048), (17, 333, 544), (33, 64, 1504), (65, 4104, 288),
                                   (128, 200, 1024), (129, 77, 160), (300, 515, 2048),
                                   (1000, 1111, 320), (513, 20000, 64)])
def test_matmul_exact_sums_bit_exact(M, N, K, dt):
    # block exponents -1 .. 0: every partial sum is a multiple of 1/16 below 2^20 (36 * K),
    # so fp32 holds it whatever the order; the one rounding left is that to the output type
    rng = np.random.default_rng(M * 7 + N + K)
    a, b = _operands(rng, M, N, K, 126, 127)
    st = _status()
    out = _matmul(a, b, dt, ld=N + 5, st=st)
    _sync(st)
    want = torch.from_numpy(a[2] @ b[2].T).to(DT[dt])
    got = out[:, :N].cpu()
    assert torch.equal(got, want), (got.float() - want.float()).abs().max()
    assert bool((out[:, N:] == 3.0).all())


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,pad", [(70, 64, 256, 0), (129, 200, 96, 8), (300, 264, 2048, 16), (1, 8, 32, 8),
                                       (257, 4104, 64, 0), (1000, 1112, 320, 24), (2000, 2560, 160, 0),
                                       (100, 8, 544, 8), (65, 24, 32, 0)])
def test_matmul_aligned_rows_bit_exact(M, N, K, pad, dt):
    # rows of whole 16-byte pieces (the tiles are then stored by the TMA unit): nothing outside
    # the N columns is written, rows past M neither
    rng = np.random.default_rng(M + N + K + pad)
    a, b = _operands(rng, M, N, K, 126, 127)
    out = torch.full((M + 3, N + pad), 3.0, dtype=DT[dt], device=DEV)
    st = _status()
    L.csa_mxfp4_matmul(_gpu(a[0]), _gpu(io.tile_scales(a[1])), _gpu(b[0]), _gpu(io.tile_scales(b[1])),
                       out[:M, :N], dev_status=st)
    _sync(st)
    assert torch.equal(out[:M, :N].cpu(), torch.from_numpy(a[2] @ b[2].T).to(DT[dt]))
    assert bool((out[:M, N:] == 3.0).all()) and bool((out[M:] == 3.0).all())


@pytest.mark.parametrize("M,N,K", [(5, 300, 4096), (200, 256, 1504), (40, 130, 32)])
def test_matmul_wide_scales(M, N, K):
    # block exponents spread over 2^-12 .. 2^12: sums round.  Accumulating K / 64 instructions'
    # sums of 64 products, each addition off by at most 2^-22 of the sum of magnitudes (a
    # truncated alignment among the products of an instruction included): (K / 64 + 2) 2^-22
    rng = np.random.default_rng(K)
    a, b = _operands(rng, M, N, K, 115, 139)
    out = _matmul(a, b, "f32")
    torch.cuda.synchronize()
    err = np.abs(f64(out) - a[2] @ b[2].T)
    bound = (K / 64 + 2) * 2.0 ** -22 * (np.abs(a[2]) @ np.abs(b[2]).T) + 1e-300
    assert np.all(err <= bound), (err / bound).max()


def test_matmul_rows_do_not_depend_on_the_batch():
    # the same rows at every batch size (every token tile width), wide scales so that the
    # order of the additions shows in the last bits
    rng = np.random.default_rng(5)
    a, b = _operands(rng, 700, 260, 1536, 115, 139)
    full = _matmul(a, b, "f32")
    for lo, n in [(0, 1), (3, 5), (100, 16), (40, 31), (10, 64), (200, 127), (300, 200), (444, 256)]:
        part = _matmul([x[lo:lo + n] for x in a], b, "f32")
        assert torch.equal(part.view(torch.int32), full[lo:lo + n].view(torch.int32)), (lo, n)
    # ... nor on the weight's other rows
    for lo, n in [(0, 100), (128, 32), (224, 36)]:
        part = _matmul(a, [x[lo:lo + n] for x in b], "f32")
        assert torch.equal(part.view(torch.int32), full[:, lo:lo + n].contiguous().view(torch.int32))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 32, 33, 47, 49, 63, 64, 65, 79, 95, 96, 97])
def test_matmul_every_token_tile_width(M, dt):
    # both sides of each width of the token tile: exact sums (K = 1504 keeps them below 2^20 / 16),
    # nothing written past the N columns or the M rows, and wide scales with the bits of a larger
    # batch
    rng = np.random.default_rng(M)
    N, K = 215, 1504
    a, b = _operands(rng, M, N, K, 126, 127)
    out = torch.full((M + 2, N + 3), 3.0, dtype=DT[dt], device=DEV)
    st = _status()
    L.csa_mxfp4_matmul(_gpu(a[0]), _gpu(io.tile_scales(a[1])), _gpu(b[0]), _gpu(io.tile_scales(b[1])),
                       out[:M, :N], dev_status=st)
    _sync(st)
    assert torch.equal(out[:M, :N].cpu(), torch.from_numpy(a[2] @ b[2].T).to(DT[dt]))
    assert bool((out[M:] == 3.0).all()) and bool((out[:, N:] == 3.0).all())
    a, b = _operands(rng, 130, N, K, 115, 139)
    full = _matmul(a, b, dt)
    assert torch.equal(_matmul([x[5:5 + M] for x in a], b, dt), full[5:5 + M])


def test_matmul_nan_scales_reach_their_results_only():
    rng = np.random.default_rng(6)
    M, N, K = 20, 140, 160
    a, b = _operands(rng, M, N, K, 126, 127)
    a[1][7, 4], b[1][131, 0] = 255, 255
    out = f64(_matmul(a, b, "f32"))
    want = a[2] @ b[2].T
    want[7, :] = np.nan
    want[:, 131] = np.nan
    assert np.array_equal(np.isnan(out), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(out[ok], want[ok])


# ---- norm and rotation ---------------------------------------------------------------------
def _qk_bound(x, w, rope, D, y, dt):
    """Of fp32 roundings of 2^-24: the sum of squares takes 8 ceil(D / 256) + 5 additions per
    lane chain and their halves reach y, rsqrtf 2 ulp (4), the division and eps sum 2, the
    product with the weight and with x 2, cos and sin 2 (the reduced angle and sincos), the
    rotation's products and sum 3; relative to |u| + |v| in rotated channels.  Plus half a
    step of the stored type."""
    n = (8 * -(-D // 256) + 6) / 2 + 13
    mag = np.abs(io.norm_rope(x, 0, w, rope=0))
    if rope:
        r = mag[..., D - rope:]
        pair = r[..., 0::2] + r[..., 1::2]
        mag[..., D - rope:] = np.repeat(pair, 2, -1)
    fi = torch.finfo(DT[dt])
    return n * 2.0 ** -24 * mag + np.abs(y) * fi.eps / 2 * (1 + 1e-3) + fi.tiny * fi.eps


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H,Hk,D,rope", [(1, 1, 0, 8, 8), (1, 64, 1, 128, 64), (3, 5, 2, 64, 64),
                                           (7, 128, 1, 576, 64), (50, 3, 3, 40, 22), (2, 16, 1, 128, 128),
                                           (33, 4, 0, 264, 32), (5, 2, 1, 520, 0), (4, 7, 1, 1024, 128),
                                           (300, 16, 1, 128, 64), (2000, 9, 1, 72, 64)])
def test_qk_norm_rope(T, H, Hk, D, rope, dt):
    g = torch.Generator(device=DEV).manual_seed(T + D)
    q = torch.randn((T, H, D), generator=g, device=DEV) * torch.rand((T, H, 1), generator=g, device=DEV) * 4
    k = torch.randn((T, Hk, D), generator=g, device=DEV) if Hk else None
    q, k = q.to(DT[dt]), None if k is None else k.to(DT[dt])
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
    qw = 1 + 0.2 * torch.randn(D, generator=g, device=DEV)
    kw = None if Hk == 2 else 1 + 0.2 * torch.randn(D, generator=g, device=DEV)
    qo, ko = torch.zeros_like(q), None if k is None else torch.zeros_like(k)
    L.csa_qk_norm_rope(q, k, pos, qo, ko, q_weight=qw, k_weight=kw, rope_dims=rope)
    torch.cuda.synchronize()
    for x, o, w in ((q, qo, qw), (k, ko, kw)):
        if x is None:
            continue
        w = None if w is None else f64(w)
        y = io.norm_rope(f64(x), pos.cpu().numpy(), w, rope=rope)
        err = np.abs(f64(o) - y)
        bound = _qk_bound(f64(x), w, rope, D, y, dt)
        assert np.all(err <= bound), (err / bound).max()


def test_qk_norm_rope_strides_in_place_and_one_side():
    g = torch.Generator(device=DEV).manual_seed(3)
    T, H, D = 37, 6, 128
    # one projection output [T, (H + 1) * D + 64]: q and k are slices of its rows
    x = torch.randn((T, (H + 1) * D + 64), generator=g, device=DEV).to(torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 1000
    q, k = x[:, :H * D].unflatten(1, (H, D)), x[:, H * D:(H + 1) * D].unflatten(1, (1, D))
    qo, ko = torch.empty((T, H, D), dtype=x.dtype, device=DEV), torch.empty((T, 1, D), dtype=x.dtype, device=DEV)
    L.csa_qk_norm_rope(q, k, pos, qo, ko)
    # head-major storage of both sides
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    qto = torch.empty((H, T, D), dtype=x.dtype, device=DEV).transpose(0, 1)
    L.csa_qk_norm_rope(qt, None, pos, qto, None)
    kto = torch.empty_like(ko)
    L.csa_qk_norm_rope(None, k, pos, None, kto)
    tail = x[:, (H + 1) * D:].clone()
    L.csa_qk_norm_rope(q, k, pos, q, k)           # in place
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qto, qo) and torch.equal(kto, ko)
    assert torch.equal(x[:, (H + 1) * D:], tail)


def test_qk_norm_rope_zero_rows_and_non_finite():
    x = torch.randn((4, 3, 128), device=DEV)
    x[1, 2] = 0
    x[2, 0, 5] = float("nan")
    pos = torch.full((4,), 9, dtype=torch.int32, device=DEV)
    y = torch.empty_like(x)
    L.csa_qk_norm_rope(x, None, pos, y, None)
    torch.cuda.synchronize()
    assert bool((y[1, 2] == 0).all())
    assert bool(y[2, 0].isnan().all()) and int(y.isnan().sum()) == 128
    # without the norm and the rotation the rows pass through
    L.csa_qk_norm_rope(x, None, pos, y, None, norm=False, rope_dims=0)
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(y, 5.0), torch.nan_to_num(x, 5.0))


# ---- the indexer's query heads and keys ---------------------------------------------------------
def _store(fmt, lead, D):
    if fmt == L.CSA_IDX_FP8:
        return (torch.full((*lead, D), 0x11, dtype=torch.uint8, device=DEV),
                torch.full(lead, 0.5, device=DEV))
    return (torch.full((*lead, D // 2), 0x11, dtype=torch.uint8, device=DEV),
            torch.full((*lead, D // 32), 100, dtype=torch.uint8, device=DEV))


def _quant_ref(y, fmt):
    return io.fp8(y) if fmt == L.CSA_IDX_FP8 else io.mxfp4(y)


def _same(codes, scale, ref):
    """Codes and UE8M0 scales bit for bit.  An fp32 scale is absmax / 448 in fp32: off by at
    most 28 roundings of 2^-24 (14 of y relative to |y1| + |y2| <= 2 absmax) and 2 of its own
    product."""
    assert np.array_equal(codes.cpu().numpy(), ref[0])
    s = scale.cpu().numpy()
    if scale.dtype == torch.uint8:
        assert np.array_equal(s, ref[1])
    else:
        nan = np.isnan(ref[1])
        assert np.array_equal(np.isnan(s), nan)
        assert np.all(np.abs(s - ref[1])[~nan] <= 30 * 2.0 ** -24 * ref[1][~nan])


@pytest.mark.parametrize("fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Q,H,D,norm,rope,weight", [(1, 1, 64, True, 64, False), (1, 64, 128, True, 64, True),
                                                    (5, 4, 64, True, 32, True), (33, 16, 128, True, 128, False),
                                                    (3, 7, 128, False, 0, False), (9, 5, 128, False, 64, True),
                                                    (700, 32, 128, True, 64, True)])
def test_indexer_queries_bit_exact(Q, H, D, norm, rope, weight, dt, fmt):
    g = torch.Generator(device=DEV).manual_seed(Q * H + D)
    x = torch.randn((Q, H, D + 32), generator=g, device=DEV)
    x = (x * torch.exp2(torch.randint(-6, 7, (Q, H, 1), generator=g, device=DEV).float())).to(DT[dt])[..., :D]
    pos = torch.randint(0, 1 << 20, (Q,), generator=g, device=DEV, dtype=torch.int32)
    w = 1 + 0.2 * torch.randn(D, generator=g, device=DEV) if weight else None
    codes, scale = _store(fmt, (Q, H), D)
    st = _status()
    L.csa_indexer_queries(x, pos, codes, scale, fmt=fmt, weight=w, norm=norm, rope_dims=rope, dev_status=st)
    _sync(st)
    y = io.norm_rope(f64(x), pos.cpu().numpy(), None if w is None else f64(w), norm=norm, rope=rope)
    _same(codes, scale, _quant_ref(y, fmt))


@pytest.mark.parametrize("fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
def test_indexer_queries_zero_and_non_finite_rows(fmt):
    x = torch.randn((6, 4, 128), device=DEV)
    x[0, 1] = 0
    x[1, 2, 77] = float("nan")
    x[2, 3, 3] = float("inf")
    x[3, 0] *= 1e-30
    x[4, 0] *= 1e30
    pos = torch.arange(6, dtype=torch.int32, device=DEV)
    for norm in (True, False):
        codes, scale = _store(fmt, (6, 4), 128)
        st = _status()
        L.csa_indexer_queries(x, pos, codes, scale, fmt=fmt, norm=norm, dev_status=st)
        _sync(st, L.CSA_DEV_NAN)
        _same(codes, scale, _quant_ref(io.norm_rope(f64(x), pos.cpu().numpy(), norm=norm), fmt))


@pytest.mark.parametrize("fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
@pytest.mark.parametrize("D,dt,m,paged", [(128, "bf16", 4, True), (64, "f32", 4, True), (128, "f16", 4, False),
                                          (64, "bf16", 128, False), (128, "f32", 128, False)])
def test_indexer_append_bit_exact(D, dt, m, paged, fmt):
    rng = np.random.default_rng(D + m)
    T = [m * 70 + 3, m * 33, m - 1, m * 5 + 1]           # entries 70, 33, 0, 5
    n_ent = [t // m for t in T]
    items = [(b, i) for b, n in enumerate(n_ent) for i in range(n) if (b, i) not in ((0, 3), (1, 0))]
    rng.shuffle(items)
    bad = [(0, 70), (2, 0), (3, 6), (4, 0), (-1, 0), (1, -1), (0, 2 ** 31 - 1)]
    items = items[:20] + bad + items[20:]
    seq, ent = (np.array([x[j] for x in items], np.int32) for j in (0, 1))
    k = _gpu(rng.standard_normal((len(items), D + 8)).astype(np.float32), DT[dt])[:, :D]
    w = _gpu((1 + 0.1 * rng.standard_normal(D)).astype(np.float32))
    if paged:
        table = rng.permutation(12).astype(np.int32).reshape(4, 3)
        row = lambda b, i: int(table[b, i // 32]) * 32 + i % 32  # noqa: E731
        rows, off, layout = 12 * 32, None, L.cache_layout(_gpu(table))
    else:
        o = np.concatenate([[5], 5 + np.cumsum(n_ent)[:-1] + 3]).astype(np.int64)
        row = lambda b, i: int(o[b]) + i  # noqa: E731
        rows, off, layout = sum(n_ent) + 20, _gpu(o), None
    codes, scale = _store(fmt, (rows,), D)
    want_c, want_s = codes.cpu().numpy(), scale.cpu().numpy()
    st = _status()
    L.csa_indexer_append(k, _gpu(np.array(T, np.int64)), off, _gpu(seq), _gpu(ent), codes, scale, B=4, m=m,
                         fmt=fmt, weight=w, layout=layout, dev_status=st)
    _sync(st, L.CSA_DEV_OOB)
    ok = np.array([0 <= b < 4 and 0 <= i < n_ent[b] for b, i in items])
    y = io.norm_rope(f64(k)[ok][:, None], (ent[ok].astype(np.int64) + 1) * m - 1, f64(w))[:, 0]
    at = [row(b, i) for (b, i), g in zip(items, ok) if g]
    want_c[at], want_s[at] = _quant_ref(y, fmt)
    _same(codes, scale, (want_c, want_s))


def test_indexer_append_bad_blocks_are_skipped():
    # block table entries that are unset, or whose rows lie past the store; a sequence longer
    # than its table
    table = torch.tensor([[0, -1, 5, 2]], dtype=torch.int32, device=DEV)
    codes, scale = _store(L.CSA_IDX_FP8, (3 * 32,), 128)
    k = torch.randn((5, 128), device=DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    st = _status()
    L.csa_indexer_append(k, torch.tensor([4000], device=DEV), None, i32(0, 0, 0, 0, 0), i32(3, 40, 70, 100, 130),
                         codes, scale, B=1, layout=L.cache_layout(table), dev_status=st)
    _sync(st, L.CSA_DEV_OOB)
    written = (scale != 0.5).nonzero().flatten().tolist()
    assert written == [3, 2 * 32 + 4]


def test_other_stream_and_current_device():
    s = torch.cuda.Stream()
    x = torch.randn((64, 256), device=DEV)
    codes, sf = torch.zeros((64, 128), dtype=torch.uint8, device=DEV), _sf_empty(64, 256, 0)
    s.wait_stream(torch.cuda.current_stream())
    L.csa_mxfp4_quantize(x, codes, sf, stream=s)
    with torch.cuda.stream(s):
        out = torch.empty_like(x)
        L.csa_mxfp4_dequantize(codes, sf, out)
    s.synchronize()
    p, b = io.mxfp4(f64(x))
    assert np.array_equal(f64(out), io.mxfp4_values(p, b))


def test_empty_calls_launch_nothing():
    n0 = L.csa_launch_count()
    u8 = lambda *n: torch.empty(n, dtype=torch.uint8, device=DEV)  # noqa: E731
    L.csa_mxfp4_quantize(torch.empty((0, 64), device=DEV), u8(0, 32), u8(0, 2))
    L.csa_mxfp4_matmul(u8(0, 32), u8(0), u8(8, 32), u8(512), torch.empty((0, 8), device=DEV))
    e32 = torch.empty(0, dtype=torch.int32, device=DEV)
    L.csa_qk_norm_rope(torch.empty((0, 4, 64), device=DEV), None, e32, torch.empty((0, 4, 64), device=DEV), None)
    L.csa_indexer_queries(torch.empty((0, 4, 64), device=DEV), e32, u8(0, 4, 64), torch.empty((0, 4), device=DEV))
    L.csa_indexer_append(torch.empty((0, 64), device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV),
                         torch.zeros(1, dtype=torch.int64, device=DEV), e32, e32, u8(4, 64),
                         torch.empty(4, device=DEV), B=1)
    torch.cuda.synchronize()
    assert L.csa_launch_count() == n0


@pytest.mark.parametrize("fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
@pytest.mark.parametrize("what", ["tiny", "huge", "weights", "zeros", "no eps", "spread", "nan weight"])
def test_indexer_queries_past_the_fp32_range(what, fmt):
    # inputs that the fp32 bracket does not cover: settled in fp64, same codes
    g = torch.Generator(device=DEV).manual_seed(77)
    x = torch.randn((40, 8, 128), generator=g, device=DEV)
    w = torch.ones(128, device=DEV)
    eps = 1e-6
    if what == "tiny":
        x *= 1e-25
    elif what == "huge":
        x *= 1e17
    elif what == "weights":
        w = torch.exp2(torch.randint(-60, 60, (128,), generator=g, device=DEV).float())
    elif what == "zeros":
        x[:, :, ::3] = 0
        x[:, ::2, 32:64] = 0
    elif what == "no eps":
        x *= torch.exp2(torch.randint(-45, 45, (40, 8, 1), generator=g, device=DEV).float())
        eps = 0.0
    elif what == "spread":
        x *= torch.exp2(torch.randint(-40, 20, (40, 8, 128), generator=g, device=DEV).float())
    else:
        w[5] = float("nan")
    pos = torch.randint(1, 1 << 20, (40,), generator=g, device=DEV, dtype=torch.int32)
    codes, scale = _store(fmt, (40, 8), 128)
    st = _status()
    L.csa_indexer_queries(x, pos, codes, scale, fmt=fmt, weight=w, eps=eps, dev_status=st)
    _sync(st, L.CSA_DEV_NAN if what == "nan weight" else 0)
    _same(codes, scale, _quant_ref(io.norm_rope(f64(x), pos.cpu().numpy(), f64(w), eps=eps), fmt))


@pytest.mark.parametrize("fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
def test_rows_do_not_depend_on_their_neighbours(fmt):
    # all heads at once, in other orders and one by one: codes and scales bit for bit
    g = torch.Generator(device=DEV).manual_seed(78)
    x = torch.randn((50, 64, 128), generator=g, device=DEV).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (50,), generator=g, device=DEV, dtype=torch.int32)
    codes, scale = _store(fmt, (50, 64), 128)
    L.csa_indexer_queries(x, pos, codes, scale, fmt=fmt)
    perm = torch.randperm(64, generator=g, device=DEV)
    c2, s2 = _store(fmt, (50, 64), 128)
    L.csa_indexer_queries(x[:, perm].contiguous(), pos, c2, s2, fmt=fmt)
    assert torch.equal(c2, codes[:, perm]) and torch.equal(s2, scale[:, perm])
    for h in range(0, 64, 7):
        c1, s1 = _store(fmt, (50, 1), 128)
        L.csa_indexer_queries(x[:, h:h + 1], pos, c1, s1, fmt=fmt)
        assert torch.equal(c1, codes[:, h:h + 1]) and torch.equal(s1, scale[:, h:h + 1])
    # the same rows as keys of entries at the same positions
    i = torch.arange(50, dtype=torch.int32, device=DEV)
    pos4 = i * 4 + 3
    L.csa_indexer_queries(x, pos4, codes, scale, fmt=fmt)
    k, ks = _store(fmt, (50,), 128)
    L.csa_indexer_append(x[:, 5], torch.tensor([1000], device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV),
                         torch.zeros_like(i), i, k, ks, B=1, fmt=fmt)
    assert torch.equal(k, codes[:, 5]) and torch.equal(ks, scale[:, 5])


@pytest.mark.parametrize("M,N,K", [(8, 4096, 4096), (300, 4096, 4096), (2000, 4096, 2048)])
def test_matmul_wait_timeout_is_reported_and_recovers(M, N, K):
    # the kernels' bounded waits with a limit far below a tile load's time (no kernel here runs
    # in a cluster): the call reports CSA_DEV_TIMEOUT and returns, the next one is exact again
    rng = np.random.default_rng(9)
    a, b = _operands(rng, M, N, K, 126, 126)
    st = _status()
    torch.cuda.synchronize()
    L.csa_debug_set_wait_limit(300)
    try:
        _matmul(a, b, "f32", st=st)
        torch.cuda.synchronize()
    finally:
        L.csa_debug_set_wait_limit(0)
    assert int(st.item()) == L.CSA_DEV_TIMEOUT
    st.zero_()
    out = _matmul(a, b, "f32", st=st)
    _sync(st)
    assert np.array_equal(f64(out), a[2] @ b[2].T)


def test_expanded_inputs_and_overlapping_outputs():
    # one row read for every head and token; an expanded output is refused
    x = torch.randn((1, 1, 128), device=DEV)
    pos = torch.arange(5, dtype=torch.int32, device=DEV)
    y = torch.empty((5, 3, 128), device=DEV)
    L.csa_qk_norm_rope(x.expand(5, 3, 128), None, pos, y, None)
    ref = io.norm_rope(f64(x.expand(5, 3, 128)), np.arange(5))
    torch.cuda.synchronize()
    assert np.abs(f64(y) - ref).max() < 1e-5
    with pytest.raises(L.CSAError, match="overlap"):
        L.csa_qk_norm_rope(y, None, pos, x.expand(5, 3, 128), None)
    codes, scale = _store(L.CSA_IDX_FP8, (5, 3), 128)
    L.csa_indexer_queries(x.expand(5, 3, 128), pos, codes, scale)
    torch.cuda.synchronize()
    _same(codes, scale, io.fp8(ref))


def test_offsets_past_32_bits():
    # quantised rows, a product's result and a key store whose last rows lie past 2^32 bytes (and
    # past 2^31 elements)
    g = torch.Generator(device=DEV).manual_seed(3)
    rows, cols = (1 << 26) + 40, 64
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    x[-70:] = torch.randn((70, cols), generator=g, device=DEV).to(torch.bfloat16)
    codes, sf = torch.full((rows, cols // 2), 9, dtype=torch.uint8, device=DEV), _sf_empty(rows, cols, 0)
    L.csa_mxfp4_quantize(x, codes, sf)
    p, s = io.mxfp4(f64(x[-70:]))
    assert np.array_equal(codes[-70:].cpu().numpy(), p) and np.array_equal(sf[-70:].cpu().numpy(), s)
    assert int(codes[:-70].max()) == 0 and int(sf[:-70].max()) == 0
    x.fill_(7.0)
    L.csa_mxfp4_dequantize(codes, sf, x)
    assert np.array_equal(f64(x[-70:]), io.mxfp4_values(p, s)) and float(x[:-70].abs().max()) == 0
    del x, codes, sf
    rng = np.random.default_rng(4)
    M, N, K = 70001, 32768, 32
    a, b = _operands(rng, M, N, K, 126, 127)
    out = _matmul(a, b, "bf16")
    for r in (0, 65536, 65537, M - 1):
        want = torch.from_numpy(a[2][r:r + 1] @ b[2].T).to(torch.bfloat16)
        assert torch.equal(out[r:r + 1].cpu(), want), r
    del out
    ent_rows = (1 << 25) + 64
    for fmt in (L.CSA_IDX_FP8, L.CSA_IDX_MXFP4):
        codes, scale = _store(fmt, (ent_rows,), 128)
        k = torch.randn((3, 128), generator=g, device=DEV)
        table = torch.tensor([[5, (1 << 20) + 1]], dtype=torch.int32, device=DEV)
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        st = _status()
        L.csa_indexer_append(k, torch.tensor([250], device=DEV), None, i32(0, 0, 0), i32(3, 40, 61), codes, scale,
                             B=1, fmt=fmt, layout=L.cache_layout(table), dev_status=st)
        _sync(st)
        at = torch.tensor([5 * 32 + 3, (1 << 25) + 32 + 8, (1 << 25) + 32 + 29], device=DEV)
        y = io.norm_rope(f64(k)[:, None], np.array([15, 163, 247]))[:, 0]
        _same(codes[at], scale[at], _quant_ref(y, fmt))
        del codes, scale


@pytest.mark.parametrize("M,N,K,fill", [(5, 70, 256, 255), (300, 70, 256, 255), (5, 70, 96, 254), (300, 515, 96, 254),
                                        (300, 1, 64, 255), (65, 2, 32, 254)])
def test_matmul_padding_scales_do_not_matter(M, N, K, fill):
    # scale tiles whose padding was never written: of rows anything (K fills its tiles), of
    # blocks past K anything finite
    rng = np.random.default_rng(K + fill)
    a, b = _operands(rng, M, N, K, 126, 127)
    if fill == 255 and K % 128:
        fill = 254
    out = _matmul(a, b, "f32", fill=fill)
    torch.cuda.synchronize()
    assert np.array_equal(f64(out), a[2] @ b[2].T)


def test_misaligned_views_are_refused():
    u8 = lambda *n: torch.zeros(n, dtype=torch.uint8, device=DEV)  # noqa: E731
    x = torch.zeros((8, 256), dtype=torch.bfloat16, device=DEV)
    L.csa_mxfp4_quantize(x[:, 8:136], u8(8, 64), u8(8, 4))
    with pytest.raises(L.CSAError, match="aligned"):
        L.csa_mxfp4_quantize(x[:, 4:132], u8(8, 64), u8(8, 4))
    with pytest.raises(L.CSAError, match="multiple of 16 bytes"):
        L.csa_mxfp4_quantize(torch.zeros((8, 132), dtype=torch.bfloat16, device=DEV)[:, :128], u8(8, 64), u8(8, 4))
    q = torch.zeros((2, 4, 132), dtype=torch.bfloat16, device=DEV)[..., :128]
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(L.CSAError, match="aligned"):
        L.csa_indexer_queries(q, pos, u8(2, 4, 128), torch.zeros((2, 4), device=DEV))
    with pytest.raises(L.CSAError, match="contiguous along|contiguous channels"):
        L.csa_qk_norm_rope(x.unflatten(1, (128, 2)).transpose(1, 2), None, torch.zeros(8, dtype=torch.int32, device=DEV),
                           torch.zeros((8, 2, 128), dtype=torch.bfloat16, device=DEV), None)


def test_two_threads_on_two_streams():
    import threading
    rng = np.random.default_rng(12)
    jobs = []
    for M, N, K in ((40, 1000, 512), (700, 520, 512)):
        a, b = _operands(rng, M, N, K, 126, 127)
        dev = [_gpu(v) for v in (a[0], io.tile_scales(a[1]), b[0], io.tile_scales(b[1]))]
        jobs.append((dev, torch.zeros((M, N), device=DEV), a[2] @ b[2].T, torch.cuda.Stream(), []))
    torch.cuda.synchronize()

    def work(dev, out, want, stream, errors):
        try:
            with torch.cuda.stream(stream):
                for _ in range(50):
                    L.csa_mxfp4_matmul(*dev, out)
                try:
                    L.csa_mxfp4_matmul(*dev[:3], dev[3][:16], out)
                    errors.append("not refused")
                except L.CSAError as e:
                    if "b's scales" not in str(e):
                        errors.append(str(e))
        except Exception as e:      # noqa: BLE001  (reported by the main thread)
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for _, out, want, _, errors in jobs:
        assert not errors and np.array_equal(f64(out), want)


def test_compiled_and_python_marshalling_agree(monkeypatch):
    # the same calls through csrc/marshal.cpp and through ctypes, bit for bit, with every optional
    # argument; and both refuse alike
    assert L._marshal is not None, "build the package: _csa_marshal.so is missing"
    g = torch.Generator(device=DEV).manual_seed(41)
    T, H, D = 6, 5, 128
    x = torch.randn((T, H * D + 64), generator=g, device=DEV).to(torch.bfloat16)
    q, k = x[:, :H * D].unflatten(1, (H, D)), torch.randn((T, 1, D), generator=g, device=DEV).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
    w, w2 = (1 + 0.2 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
    table = torch.randperm(8, generator=g, device=DEV).to(torch.int32).view(2, 4)
    seq = torch.tensor([0, 1, 1, 0, 1, 0], dtype=torch.int32, device=DEV)
    ent = torch.tensor([3, 100, 7, 64, 90, 0], dtype=torch.int32, device=DEV)
    seq_len, off = torch.tensor([500, 450], device=DEV), torch.tensor([0, 128], device=DEV)
    stream = torch.cuda.Stream()

    def run(s):
        out, st = [], _status()
        u8 = lambda *n: torch.zeros(n, dtype=torch.uint8, device=DEV)  # noqa: E731
        for lay in (L.CSA_SF_ROWS, L.CSA_SF_TILED):
            codes, sf = u8(T, H * D // 2), u8(L.csa_mxfp4_sf_bytes(T, H * D, lay))
            back = torch.zeros((T, H * D + 8), device=DEV)[:, :H * D]
            L.csa_mxfp4_quantize(x[:, :H * D], codes, sf, sf_layout=lay, dev_status=st, stream=s)
            L.csa_mxfp4_dequantize(codes, sf, back, sf_layout=lay, stream=s)
            out += [codes, sf, back]
        prod = torch.zeros((T, T + 3), dtype=torch.float16, device=DEV)
        L.csa_mxfp4_matmul(codes, sf, codes, sf, prod[:, :T], dev_status=st, stream=s)
        qo, ko = torch.zeros_like(q), torch.zeros_like(k)
        L.csa_qk_norm_rope(q, k, pos, qo, ko, q_weight=w, k_weight=w2, rope_dims=32, rope_theta=500.0, eps=1e-5, stream=s)
        k2 = torch.zeros_like(k)
        L.csa_qk_norm_rope(None, k, pos, None, k2, norm=False, stream=s)
        out += [prod, qo, ko, k2]
        for fmt in (L.CSA_IDX_FP8, L.CSA_IDX_MXFP4):
            codes, scale = _store(fmt, (T, H), D)
            L.csa_indexer_queries(q, pos, codes, scale, fmt=fmt, weight=w, norm=False, rope_dims=32, rope_theta=500.0,
                                  eps=1e-5, dev_status=st, stream=s)
            kc, ks = _store(fmt, (256,), D)
            for kw in (dict(layout=L.cache_layout(table)), dict(layout=None)):
                L.csa_indexer_append(k[:, 0], seq_len, off, seq, ent, kc, ks, B=2, m=4, fmt=fmt, weight=w2, rope_dims=32,
                                     rope_theta=500.0, eps=1e-5, dev_status=st, stream=s, **kw)
            out += [codes, scale, kc, ks]
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        errors = []
        for bad in (lambda: L.csa_mxfp4_quantize(x[:, :48], u8(T, 24), u8(T, 2)),
                    lambda: L.csa_mxfp4_quantize(x[:, :64], u8(T, 32), u8(T, 2), sf_layout=5),
                    lambda: L.csa_mxfp4_matmul(u8(4, 32), u8(8), u8(8, 32), u8(512), prod),
                    lambda: L.csa_qk_norm_rope(q, k, pos.long(), qo, ko),
                    lambda: L.csa_qk_norm_rope(q, None, pos, qo, None, rope_dims=63),
                    lambda: L.csa_indexer_queries(q, pos, kc, ks),
                    lambda: L.csa_indexer_append(k[:, 0], seq_len, None, seq, ent, u8(4, D), torch.zeros(4, device=DEV), B=2)):
            with pytest.raises(L.CSAError) as e:
                bad()
            errors.append(str(e.value))
        return out, errors

    for s in (None, stream):
        torch.cuda.synchronize()
        fast = run(s)
        with monkeypatch.context() as mp:
            mp.setattr(L, "_marshal", None)
            slow = run(s)
        assert fast[1] == slow[1]
        for a, b in zip(fast[0], slow[0]):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_no_weight_is_a_weight_of_ones(D, dt, fmt):
    # the unit weight that a call without one reads, on every kernel that reads it
    g = torch.Generator(device=DEV).manual_seed(D)
    x = torch.randn((19, 6, D), generator=g, device=DEV).to(DT[dt])
    pos = torch.randint(0, 1 << 20, (19,), generator=g, device=DEV, dtype=torch.int32)
    item = torch.arange(19, dtype=torch.int32, device=DEV)
    seq_len, off = torch.tensor([80], device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    for rope in (64, 32):
        got = []
        for w in (None, torch.ones(D, device=DEV)):
            qc, qs = _store(fmt, (19, 6), D)
            kc, ks = _store(fmt, (20,), D)
            L.csa_indexer_queries(x, pos, qc, qs, fmt=fmt, weight=w, rope_dims=rope)
            L.csa_indexer_append(x[:, 2], seq_len, off, torch.zeros_like(item), item, kc, ks, B=1, fmt=fmt, weight=w,
                                 rope_dims=rope)
            got.append((qc, qs, kc, ks))
        torch.cuda.synchronize()
        for a, b in zip(*got):
            assert torch.equal(a, b)
        y = io.norm_rope(f64(x), pos.cpu().numpy(), rope=rope)
        _same(got[0][0], got[0][1], _quant_ref(y, fmt))


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
def test_append_through_a_slice_of_a_block_table(fmt, compiled, monkeypatch):
    # a slice of columns: the same rows as through a table of its own; entries past the slice (whose
    # blocks a wider table has) are flagged and written nowhere, whatever the sequences' lengths
    if not compiled:
        monkeypatch.setattr(L, "_marshal", None)
    g = torch.Generator(device=DEV).manual_seed(31)
    big = torch.randperm(24, generator=g, device=DEV).to(torch.int32).view(3, 8)
    k = torch.randn((7, 128), generator=g, device=DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    seq, ent = i32(0, 1, 2, 2, 1, 0, 2), i32(0, 40, 95, 96, 100, 255, 200)
    seq_len = torch.full((3,), 4 * 256, dtype=torch.int64, device=DEV)
    side = torch.cuda.Stream()
    for view in (big[:, 2:5], big[:, 5:], big[:, :3]):
        want_c, want_s = _store(fmt, (24 * 32,), 128)
        st = _status()
        L.csa_indexer_append(k[:3], seq_len, None, seq[:3], ent[:3], want_c, want_s, B=3, fmt=fmt,
                             layout=L.cache_layout(view.contiguous()), dev_status=st)
        _sync(st)
        for stream in (None, side):
            codes, scale = _store(fmt, (24 * 32,), 128)
            torch.cuda.synchronize()
            L.csa_indexer_append(k, seq_len, None, seq, ent, codes, scale, B=3, fmt=fmt,
                                 layout=L.cache_layout(view), dev_status=st, stream=stream)
            _sync(st, L.CSA_DEV_OOB)
            st.zero_()
            assert torch.equal(codes, want_c) and torch.equal(scale, want_s)
    # one sequence: its row alone, in a table with a gap behind it
    codes, scale = _store(fmt, (24 * 32,), 128)
    st = _status()
    L.csa_indexer_append(k[:2], seq_len[:1], None, i32(0, 0), i32(64, 96), codes, scale, B=1, fmt=fmt,
                         layout=L.cache_layout(big[2:, 5:]), dev_status=st)
    _sync(st, L.CSA_DEV_OOB)
    row = int(big[2, 7]) * 32
    y = io.norm_rope(f64(k)[:1, None], np.array([65 * 4 - 1]))[:, 0]
    _same(codes[row:row + 1], scale[row:row + 1], _quant_ref(y, fmt))
    codes[row], scale[row] = 0x11, scale[(row + 1) % 768]
    blank = _store(fmt, (24 * 32,), 128)
    assert torch.equal(codes, blank[0]) and torch.equal(scale, blank[1])


@pytest.mark.parametrize("fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
@pytest.mark.parametrize("rope", [0, 64, 128])
def test_zeros_keep_their_sign(rope, fmt):
    # zeros of both signs (channels, and pairs of them, which a rotation turns into either) in enough
    # rows that many are settled in fp64
    g = torch.Generator(device=DEV).manual_seed(rope + 1)
    x = torch.randn((200, 16, 128), generator=g, device=DEV)
    drop = torch.rand((200, 16, 64, 1), generator=g, device=DEV) < 0.2
    x = torch.where(drop, torch.copysign(torch.zeros_like(x), x).unflatten(2, (64, 2)), x.unflatten(2, (64, 2))).flatten(2)
    x[:, :, 5] = -0.0
    pos = torch.randint(0, 1 << 20, (200,), generator=g, device=DEV, dtype=torch.int32)
    codes, scale = _store(fmt, (200, 16), 128)
    st = _status()
    L.csa_indexer_queries(x, pos, codes, scale, fmt=fmt, rope_dims=rope, dev_status=st)
    _sync(st)
    _same(codes, scale, _quant_ref(io.norm_rope(f64(x), pos.cpu().numpy(), rope=rope), fmt))


@pytest.mark.parametrize("fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,rope", [(64, 0), (64, 32), (64, 64), (128, 0), (128, 32), (128, 64), (128, 128)])
def test_ties_and_their_neighbours_on_every_kernel(D, rope, dt, fmt):
    # values on the borders between codes, and in fp32 one step to either side, which no bracket settles:
    # without the norm, at position 0 (no angle), in every kernel.  Zero blocks and rows among them
    rng = np.random.default_rng(D + rope + fmt)
    if fmt == L.CSA_IDX_MXFP4:
        v, top, one = (io.LEVELS[1:] + io.LEVELS[:-1]) / 2, 6.0, 32
    else:
        codes = np.arange(127, dtype=np.uint8).view(io.ml_dtypes.float8_e4m3fn).astype(np.float64)
        v, top, one = (codes[1:] + codes[:-1]) / 2, 448.0, D
    rows = rng.choice(v[v >= 2.0 ** -6], (300, 2, D)) * rng.choice([-1, 1], (300, 2, D))
    if dt == "f32":
        rows *= 1 + rng.integers(-1, 2, rows.shape) * 2.0 ** -23
    rows.reshape(-1, one)[:, 0] = top                    # the scale is the row's power of two
    rows.reshape(-1, one)[::7] = 0
    rows *= 2.0 ** rng.integers(-6, 7, (300, 2, 1))
    x = _gpu(rows.astype(np.float32), DT[dt])
    assert dt != "bf16" or np.array_equal(f64(x), rows)  # borders stay borders
    pos = torch.zeros(300, dtype=torch.int32, device=DEV)
    codes, scale = _store(fmt, (300, 2), D)
    st = _status()
    L.csa_indexer_queries(x, pos, codes, scale, fmt=fmt, norm=False, rope_dims=rope, dev_status=st)
    _sync(st)
    _same(codes, scale, _quant_ref(f64(x), fmt))
    # and as keys: entry 0 of its sequence, one token long, stands at position 0
    kc, ks = _store(fmt, (300,), D)
    b = torch.arange(300, dtype=torch.int32, device=DEV)
    L.csa_indexer_append(x[:, 1], torch.ones(300, dtype=torch.int64, device=DEV), b.long(), b, torch.zeros_like(b), kc, ks,
                         B=300, m=1, fmt=fmt, norm=False, rope_dims=rope, dev_status=st)
    _sync(st)
    _same(kc, ks, _quant_ref(f64(x[:, 1]), fmt))


def _unsigned_zeros(packed):
    """Packed e2m1 codes with -0 as 0."""
    packed = packed * (packed & 0x0f != 8) | packed * (packed & 0x0f == 8) & 0xf0
    return packed * (packed & 0xf0 != 0x80) | packed * (packed & 0xf0 == 0x80) & 0x0f


@pytest.mark.parametrize("fmt", [L.CSA_IDX_FP8, L.CSA_IDX_MXFP4])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("rope", [0, 64])
def test_rows_whose_products_underflow_are_not_zero_rows(rope, norm, fmt):
    # products x * weight below fp32's least, while the norm lifts the rows to 2^-121 and their
    # scales into range: whole rows (FP8's zero test) and blocks (MXFP4's), beside rows of true
    # zeros, and rows that only a weight of zero empties.  The sign of a zero code is the definition's
    # but where rotated products underflow in an MXFP4 block (which stays on the fp32 path)
    x = torch.zeros((8, 4, 128), device=DEV)
    sign = 1 - 2 * (torch.arange(128, device=DEV) % 3 == 1).float()
    small = sign * torch.linspace(1.0, 1.5, 128, device=DEV) * 2.0 ** -90
    x[1], x[1, :, 0] = small, 2.0 ** -26
    x[2, :, 32:64], x[2, :, 0] = small[32:64], 2.0 ** -26
    x[3, 1:3, 96:], x[3, 1:3, 0] = small[96:], 2.0 ** -26
    x[4] = small * 2.0 ** -50
    x[5, :, 0] = 3.0
    x[6, :, 1:] = torch.randn(127, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    x[7, 2] = small
    w = torch.full((128,), 2.0 ** -61, device=DEV)
    w[0] = 0
    pos = torch.arange(8, dtype=torch.int32, device=DEV) * 1001
    for eps in (0.0, 1e-30, 1e-6):
        # (a row of zeros has no norm without an eps)
        keep = [1, 2, 4, 5, 6] if norm and eps == 0.0 else list(range(8))
        q, p = x[keep].contiguous(), pos[keep].contiguous()
        codes, scale = _store(fmt, q.shape[:2], 128)
        st = _status()
        L.csa_indexer_queries(q, p, codes, scale, fmt=fmt, weight=w, norm=norm, rope_dims=rope, eps=eps, dev_status=st)
        _sync(st)
        ref = _quant_ref(io.norm_rope(f64(q), p.cpu().numpy(), f64(w), norm=norm, rope=rope, eps=eps), fmt)
        lax = _unsigned_zeros if rope and fmt == L.CSA_IDX_MXFP4 else (lambda c: c)  # noqa: E731
        _same(lax(codes), scale, (lax(ref[0]), ref[1]))
        kc, ks = _store(fmt, (8,), 128)
        item = torch.arange(len(keep), dtype=torch.int32, device=DEV)
        L.csa_indexer_append(q[:, 1], torch.tensor([400], device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV),
                             torch.zeros_like(item), item, kc, ks, B=1, fmt=fmt, weight=w, norm=norm, rope_dims=rope,
                             eps=eps, dev_status=st)
        _sync(st)
        y = io.norm_rope(f64(q[:, 1:2]), np.arange(len(keep)) * 4 + 3, f64(w), norm=norm, rope=rope, eps=eps)
        ref = _quant_ref(y[:, 0], fmt)
        _same(lax(kc[:len(keep)]), ks[:len(keep)], (lax(ref[0]), ref[1]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
@pytest.mark.parametrize("H,D,rope", [(9, 64, 64), (6, 128, 64), (5, 256, 32), (5, 512, 0), (4, 576, 64), (3, 1024, 128)])
def test_qk_norm_rope_past_the_range_of_fp32_squares(H, D, rope, eps, dt):
    # rows whose squares overflow or underflow fp32, whole or in their largest element only, beside
    # ordinary ones, whose results have the bits of a call without the others
    g = torch.Generator(device=DEV).manual_seed(D)
    x = torch.randn((12, H, D), generator=g, device=DEV)
    plain = x.to(DT[dt])
    for t, s in ((1, 1e25), (2, 1e-25), (3, 2.0 ** 120), (4, 2.0 ** -120), (6, 1e19), (7, 1e-19)):
        x[t, 1 - t % 2::2] *= s
    x[8, 0, 7] = 3e38
    x[9, 1] *= 1e-38
    x[9, 1, -1] = 1e-20
    x[10] *= 1e-40
    x = x.to(DT[dt])
    same = (x == plain).all(-1)
    pos = torch.randint(0, 1 << 20, (12,), generator=g, device=DEV, dtype=torch.int32)
    w = 1 + 0.2 * torch.randn(D, generator=g, device=DEV)
    out, ref, kout = (torch.empty_like(x) for _ in range(3))
    L.csa_qk_norm_rope(x, x, pos, out, kout, q_weight=w, k_weight=w, rope_dims=rope, eps=eps)
    L.csa_qk_norm_rope(plain, None, pos, ref, None, q_weight=w, rope_dims=rope, eps=eps)
    torch.cuda.synchronize()
    assert torch.equal(out[same], ref[same]) and torch.equal(out, kout)
    y = io.norm_rope(f64(x), pos.cpu().numpy(), f64(w), rope=rope, eps=eps)
    # the bound of the fp32 path, whose magnitudes are those of the normed row without a rotation
    n = (8 * -(-D // 256) + 6) / 2 + 13
    mag = np.abs(io.norm_rope(f64(x), 0, f64(w), rope=0, eps=eps))
    if rope:
        pair = mag[..., D - rope::2] + mag[..., D - rope + 1::2]
        mag[..., D - rope:] = np.repeat(pair, 2, -1)
    fi = torch.finfo(DT[dt])
    bound = n * 2.0 ** -24 * mag + np.abs(y) * fi.eps / 2 * (1 + 1e-3) + fi.tiny * fi.eps
    err = np.abs(f64(out) - y)
    assert np.all(err <= bound), (err / bound).max()


def _feature_tile(M, N, K):
    """The features per tile that the library takes for more than 96 tokens: the least cost of rounds
    over the SMs (the rule and its constants stand at launch_mxfp4_matmul)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    nk = -(-K // 256)
    cost = {ct: -(-(-(-M // 128) * -(-N // ct)) // sms) * (fixed + stage * nk)
            for ct, fixed, stage in ((256, 160, 41), (128, 70, 28), (64, 45, 27))}
    return min(cost, key=lambda ct: (cost[ct], -ct))


# (M, N, K) of every feature tile: N past a tile by less and by more than half of it, whole and ragged K
_TILES = [(700, 5000, 1504, 256), (1900, 2100, 1504, 256), (450, 5003, 736, 256), (2000, 2200, 1536, 256),
          (300, 5000, 1504, 128), (1300, 3330, 800, 128), (900, 4999, 1248, 128), (515, 1300, 2048, 64)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,ct", _TILES)
def test_matmul_every_feature_tile_bit_exact(M, N, K, ct, dt):
    # exact sums; rows of the output that the TMA unit stores (whole 16-byte pieces) and others
    if torch.cuda.get_device_properties(0).multi_processor_count == 148:
        assert _feature_tile(M, N, K) == ct
    rng = np.random.default_rng(M + N)
    a, b = _operands(rng, M, N, K, 126, 127)
    want = torch.from_numpy(a[2] @ b[2].T).to(DT[dt])
    for pad in (0, 3, 8 + -N % 8):
        out = torch.full((M + 2, N + pad), 3.0, dtype=DT[dt], device=DEV)
        st = _status()
        L.csa_mxfp4_matmul(_gpu(a[0]), _gpu(io.tile_scales(a[1])), _gpu(b[0]), _gpu(io.tile_scales(b[1])), out[:M, :N],
                           dev_status=st)
        _sync(st)
        assert torch.equal(out[:M, :N].cpu(), want), pad
        assert bool((out[:M, N:] == 3.0).all()) and bool((out[M:] == 3.0).all()), pad


@pytest.mark.parametrize("M,N,K,ct", [t for t in _TILES if t[3] > 64])
def test_matmul_rows_do_not_depend_on_the_feature_tile(M, N, K, ct):
    # wide block exponents, so that the order of the additions shows: the same rows in batches of the
    # few-token kernel's widths and of narrower tiles, and the same features of narrower weights
    rng = np.random.default_rng(M + N + 1)
    a, b = _operands(rng, M, N, K, 115, 139)
    full = _matmul(a, b, "f32")
    bits = lambda t: t.contiguous().view(torch.int32)  # noqa: E731
    for lo, n in [(0, 1), (M - 17, 17), (5, 65), (130, 97), (M - 128, 128)]:
        part = _matmul([x[lo:lo + n] for x in a], b, "f32")
        assert torch.equal(bits(part), bits(full[lo:lo + n])), (lo, n)
    for lo, n in [(0, 100), (128, 32), (N - 260, 260), (N - 7, 7), (256, 700)]:
        part = _matmul(a, [x[lo:lo + n] for x in b], "f32")
        assert torch.equal(bits(part), bits(full[:, lo:lo + n])), (lo, n)
    for dt in ("bf16", "f16"):
        assert torch.equal(_matmul(a, b, dt), full.to(DT[dt]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D", [(3, 70, 128), (2, 131, 64), (3, 37, 320), (2, 5, 1024), (2000, 9, 128)])
def test_qk_norm_rope_past_the_range_in_place(T, H, D, dt):
    # rows that are done again from their inputs, in place and strided, here and there among many heads
    g = torch.Generator(device=DEV).manual_seed(H)
    x = torch.randn((T, H * D + 64), generator=g, device=DEV)
    scale = torch.tensor([1.0, 1.0, 1.0, 1e24, 1e-24], device=DEV)
    pick = torch.randint(0, 5, (T, H), generator=g, device=DEV)
    x[:, :H * D] *= scale[pick].repeat_interleave(D, 1)
    x = x.to(DT[dt])
    q, tail = x[:, :H * D].unflatten(1, (H, D)), x[:, H * D:].clone()
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
    out, want = torch.empty((T, H, D), dtype=x.dtype, device=DEV), io.norm_rope(f64(q), pos.cpu().numpy(), rope=64, eps=0.0)
    L.csa_qk_norm_rope(q, None, pos, out, None, eps=0.0)
    L.csa_qk_norm_rope(q, None, pos, q, None, eps=0.0)
    torch.cuda.synchronize()
    assert torch.equal(q, out) and torch.equal(x[:, H * D:], tail)
    # pairs of normed magnitude below 64: 2^-24 of it some twenty times, and half a step of the type
    assert np.all(np.abs(f64(out) - want) <= 64 * 30 * 2.0 ** -24 + np.abs(want) * torch.finfo(x.dtype).eps / 2 * 1.001)
