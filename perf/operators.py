"""Timed cases of the operators that make the lightning indexer's inputs: MXFP4 quantisation and
its inverse, the MXFP4 product, the per-head norm with the position rotation, the indexer's
query heads in their stored format, and the append of indexer keys to the (paged) key store.

``run`` computes a case in its plain form (elementary torch operations) while ``own`` is
false, and through the package's calls when it is true.  ``exact`` gives the same outputs in
64 bits from the definitions, written apart from the plain form."""
import math

import torch

own = False

DEV = "cuda"
THETA, EPS = 10000.0, 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---- cases ---------------------------------------------------------------------------
def listed():
    return [
        # the query heads of 8 decode tokens (64 heads x 128), quantised and read back
        dict(name="quant_decode_heads", op="quant", rows=512, cols=128, pad=0, dtype="bf16",
             tiled=False),
        # an fp32 projection weight laid out once for the product, and read back
        dict(name="quant_weight_f32", op="quant", rows=8192, cols=2048, pad=0, dtype="f32",
             tiled=True),
        # decode: the indexer's query projection (64 heads x 128 outputs) of 8 tokens
        dict(name="product_decode", op="product", M=8, N=8192, K=2048, pad=0, dtype="bf16",
             out="bf16"),
        # a ragged batch of 197 tokens, sizes off every tile, fp32 result, strided rows
        dict(name="product_ragged_f32", op="product", M=197, N=4104, K=1504, pad=32,
             dtype="f32", out="f32"),
        # prefill chunk of 8192 tokens through the same projection
        dict(name="product_prefill", op="product", M=8192, N=8192, K=2048, pad=0, dtype="bf16",
             out="bf16"),
        # decode at 1M tokens: 8 tokens, 128 query heads of 576 channels and their shared key
        dict(name="qk_decode_576", op="qk", T=8, H=128, Hk=1, D=576, rope=64, far=1 << 20,
             pad=0, dtype="bf16"),
        # a ragged fp32 batch with strided tokens, every channel rotated
        dict(name="qk_ragged_f32", op="qk", T=333, H=16, Hk=2, D=128, rope=128, far=131072,
             pad=256, dtype="f32"),
        # prefill chunk: 8192 tokens, 64 query heads of 128 channels and their shared key
        dict(name="qk_prefill", op="qk", T=8192, H=64, Hk=1, D=128, rope=64, far=73728, pad=0,
             dtype="bf16"),
        # decode: the FP8 indexer's query heads of 8 sequences at 1M tokens
        dict(name="queries_decode_fp8", op="queries", Q=8, H=64, D=128, far=1 << 20,
             fmt="fp8", dtype="bf16"),
        # prefill chunk: the MXFP4 indexer's query heads of 8192 tokens
        dict(name="queries_prefill_mxfp4", op="queries", Q=8192, H=64, D=128, far=73728,
             fmt="mxfp4", dtype="bf16"),
        # decode: the newest entry of each of 32 sequences into a paged FP8 key store
        dict(name="append_decode_fp8", op="append", B=32, have=4096, add=1, D=128, m=4,
             paged=True, fmt="fp8", dtype="bf16"),
        # prefill chunks of 8192 tokens (2048 entries) of 4 sequences into a paged MXFP4 store
        dict(name="append_prefill_mxfp4", op="append", B=4, have=2048, add=2048, D=128, m=4,
             paged=True, fmt="mxfp4", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "product", "qk", "queries", "append"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quant":
        cols = 32 * _log(rng, 1, 256)
        rows = _log(rng, 1, max(1, (1 << 24) // cols))
        return dict(op=op, rows=rows, cols=cols, pad=rng.choice([0, 0, 8, 96]), dtype=dtype,
                    tiled=rng.random() < 0.5)
    if op == "product":
        K = 32 * _log(rng, 1, 128)
        N = _log(rng, 1, 8192)
        M = _log(rng, 1, max(1, min(8192, 8192 * 8192 * 2048 // (N * K))))
        return dict(op=op, M=M, N=N, K=K, pad=rng.choice([0, 0, 32]), dtype=dtype,
                    out=rng.choice(["bf16", "f16", "f32"]))
    if op == "qk":
        D = rng.choice([64, 128, 128, 576, 8 * rng.randint(2, 64)])
        H = rng.choice([1, 4, 16, 64, 128])
        T = _log(rng, 1, max(1, min(8192, 8192 * 64 * 128 * 2 // (H * D * BYTES[dtype]))))
        rope = rng.choice([64, 64, 32, 0])
        return dict(op=op, T=T, H=H, Hk=rng.choice([0, 1, 1, 4]), D=D, rope=min(rope, D // 2 * 2),
                    far=_log(rng, 8192, 1 << 20), pad=rng.choice([0, 0, 64]), dtype=dtype)
    if op == "queries":
        H = rng.choice([4, 16, 32, 64])
        return dict(op=op, Q=_log(rng, 1, 8192 * 2 * 64 // (H * BYTES[dtype])), H=H,
                    D=rng.choice([64, 128, 128]), far=_log(rng, 8192, 1 << 20),
                    fmt=rng.choice(["fp8", "mxfp4"]), dtype=dtype)
    B = _log(rng, 1, 32)
    add = _log(rng, 1, max(1, 65536 // B))
    m = rng.choice([4, 4, 128])
    return dict(op="append", B=B, have=_log(rng, 1, 4096), add=add, D=rng.choice([64, 128, 128]),
                m=m, paged=m == 4 and rng.random() < 0.6, fmt=rng.choice(["fp8", "mxfp4"]),
                dtype=dtype)


# ---- inputs --------------------------------------------------------------------------
def _rows(g, rows, cols, pad, dtype):
    """Normal rows whose magnitudes differ by row, as activations' do, with a row stride of
    cols + pad."""
    x = torch.randn((rows, cols + pad), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device=DEV))
    return x.to(TYPES[dtype])[:, :cols]


def _weight(g, D):
    return 1.0 + 0.1 * torch.randn((D,), generator=g, device=DEV)


def _mxfp4_of(x):
    """(packed codes, scale bytes) of fp32 rows: what a weight file holds."""
    mag, sf = _fp4_steps(x)
    code = torch.where(mag < 2, 2 * mag, torch.where(mag < 4, mag + 2, mag / 2 + 4))
    code = code.to(torch.int32) | ((x < 0).to(torch.int32) << 3)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8), sf


def _tile_scales(sf):
    """Scale bytes [rows, n] in tiles of 128 rows x 4 blocks: byte 16 (r mod 32) + 4 (r div 32)
    + j of a tile is block j of its row r; tiles go along the blocks first, zero padded."""
    r, n = sf.shape
    R, N = -(-r // 128) * 128, -(-n // 4) * 4
    p = torch.zeros((R, N), dtype=torch.uint8, device=sf.device)
    p[:r, :n] = sf
    return p.view(R // 128, 4, 32, N // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    c = dict(case)
    op = c["op"]
    s = {"case": c}
    u8 = lambda *n: torch.empty(n, dtype=torch.uint8, device=DEV)  # noqa: E731
    if op == "quant":
        s["x"] = _rows(g, c["rows"], c["cols"], c["pad"], c["dtype"])
        s["codes"] = u8(c["rows"], c["cols"] // 2)
        s["sf"] = u8(-(-c["rows"] // 128) * -(-c["cols"] // 128) * 512) if c["tiled"] else \
            u8(c["rows"], c["cols"] // 32)
        s["out"] = torch.empty((c["rows"], c["cols"]), dtype=torch.bfloat16, device=DEV)
    elif op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        s["x"] = _rows(g, M, K, c["pad"], c["dtype"])
        s["w"], s["w_sf"] = _mxfp4_of(torch.randn((N, K), generator=g, device=DEV) / math.sqrt(K))
        s["w_sf_tiled"] = _tile_scales(s["w_sf"])
        s["codes"] = u8(M, K // 2)
        s["sf"] = u8(-(-M // 128) * -(-K // 128) * 512)
        s["out"] = torch.empty((M, N), dtype=TYPES[c["out"]], device=DEV)
    elif op == "qk":
        T, H, Hk, D = c["T"], c["H"], c["Hk"], c["D"]
        s["q"] = _rows(g, T, H * D, c["pad"], c["dtype"]).unflatten(1, (H, D))
        s["k"] = _rows(g, T, Hk * D, 0, c["dtype"]).unflatten(1, (Hk, D)) if Hk else None
        s["pos"] = torch.randint(0, c["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
        s["qw"], s["kw"] = _weight(g, D), _weight(g, D)
        s["q_out"] = torch.empty((T, H, D), dtype=TYPES[c["dtype"]], device=DEV)
        s["k_out"] = torch.empty((T, Hk, D), dtype=TYPES[c["dtype"]], device=DEV) if Hk else None
    elif op == "queries":
        Q, H, D = c["Q"], c["H"], c["D"]
        s["q"] = _rows(g, Q * H, D, 0, c["dtype"]).view(Q, H, D)
        s["pos"] = torch.randint(0, c["far"], (Q,), generator=g, device=DEV, dtype=torch.int32)
        s["qw"] = _weight(g, D)
        if c["fmt"] == "fp8":
            s["codes"] = u8(Q, H, D)
            s["scale"] = torch.empty((Q, H), dtype=torch.float32, device=DEV)
        else:
            s["codes"], s["scale"] = u8(Q, H, D // 2), u8(Q, H, D // 32)
            s["out"] = torch.empty((Q * H, D), dtype=torch.bfloat16, device=DEV)
    else:
        B, D, m, have, add = c["B"], c["D"], c["m"], c["have"], c["add"]
        n = have + add                                       # entries of each sequence
        s["k"] = _rows(g, B * add, D, 0, c["dtype"])
        s["kw"] = _weight(g, D)
        s["seq"] = torch.arange(B, device=DEV, dtype=torch.int32).repeat_interleave(add)
        s["ent"] = torch.arange(have, n, device=DEV, dtype=torch.int32).repeat(B)
        s["seq_len"] = torch.full((B,), n * m + m // 2, dtype=torch.int64, device=DEV)
        if c["paged"]:
            nb = -(-n // 32)
            perm = torch.randperm(B * nb, generator=g, device=DEV).to(torch.int32)
            s["table"], s["ent_off"], rows = perm.view(B, nb), None, B * nb * 32
        else:
            s["table"], rows = None, B * n
            s["ent_off"] = torch.arange(B, device=DEV, dtype=torch.int64) * n
        # what the store holds before: finite codes
        if c["fmt"] == "fp8":
            s["codes"] = torch.randn((rows, D), generator=g, device=DEV).to(
                torch.float8_e4m3fn).view(torch.uint8)
            s["scale"] = torch.rand((rows,), generator=g, device=DEV) + 0.5
        else:
            s["codes"] = torch.randint(0, 256, (rows, D // 2), generator=g, device=DEV).to(
                torch.uint8)
            s["scale"] = torch.randint(120, 130, (rows, D // 32), generator=g, device=DEV).to(
                torch.uint8)
            s["out"] = torch.empty((rows, D), dtype=torch.bfloat16, device=DEV)
    return s


# ---- plain forms ---------------------------------------------------------------------
def _fp4_steps(x):
    """(magnitudes 0 .. 6 in units of each block's scale, scale bytes) of rows in blocks of 32:
    the scale is 2^(floor(log2(amax)) - 2), elements go to the nearest of 0, 0.5, 1, 1.5, 2,
    3, 4, 6 (ties to the even code), larger ones to 6."""
    b = x.unflatten(-1, (-1, 32))
    e = torch.frexp(b.abs().amax(-1)).exponent - 3
    y = torch.ldexp(b.abs(), -e.unsqueeze(-1))
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    mag = (torch.round(y / step) * step).clamp(max=6.0).flatten(-2)
    sf = torch.where(b.abs().amax(-1) > 0, (e + 127).clamp(0, 254), 0)
    return mag, sf.to(torch.uint8)


def _fp4_values(x):
    """The values that the rows of x are held as in MXFP4."""
    mag, sf = _fp4_steps(x)
    scale = torch.ldexp(torch.ones_like(mag), sf.to(torch.int32).repeat_interleave(32, -1) - 127)
    return torch.copysign(mag * scale, x)


def _fp4_read(codes, sf):
    """Packed codes and scale bytes (rows layout) as fp32 values."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int32)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    v = torch.where(c >= 8, -table[c & 7], table[c & 7])
    return torch.ldexp(v, sf.to(torch.int32).repeat_interleave(32, -1) - 127)


def _norm_rope(x, pos, weight, rope, work):
    """RMSNorm of each head and rotation of its last `rope` channels (interleaved pairs), in
    the type `work`; the angles in 64 bits."""
    x = x.to(work)
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.to(work)
    if not rope:
        return y
    f = THETA ** (-torch.arange(0, rope, 2, device=x.device, dtype=torch.float64) / rope)
    a = pos.to(torch.float64)[:, None, None] * f
    c, s = torch.cos(a).to(work), torch.sin(a).to(work)
    u, v = y[..., -rope::2], y[..., y.shape[-1] - rope + 1::2]
    r = torch.stack([u * c - v * s, u * s + v * c], -1).flatten(-2)
    return torch.cat([y[..., :y.shape[-1] - rope], r], -1)


def _fp8(y):
    """(codes, scale): one scale per row, absmax / 448."""
    amax = y.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, 1.0).to(torch.float32)
    return (y / scale.to(y.dtype).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float32).to(
        torch.float8_e4m3fn), scale


def _place(s):
    """Store rows of the appended entries."""
    e = s["ent"].to(torch.int64)
    b = s["seq"].to(torch.int64)
    if s["table"] is None:
        return s["ent_off"][b] + e
    return s["table"][b, e // 32].to(torch.int64) * 32 + e % 32


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "quant":
        return _fp4_values(s["x"].float()).to(torch.bfloat16)
    if op == "product":
        a = _fp4_values(s["x"].float())
        return (a @ _fp4_read(s["w"], s["w_sf"]).t()).to(TYPES[c["out"]])
    if op == "qk":
        t = TYPES[c["dtype"]]
        q = _norm_rope(s["q"], s["pos"], s["qw"], c["rope"], torch.float32).to(t)
        k = None if s["k"] is None else _norm_rope(s["k"], s["pos"], s["kw"], c["rope"],
                                                   torch.float32).to(t)
        return {"q": q, "k": k}
    if op == "queries":
        # in 64 bits: values next to a rounding border
        y = _norm_rope(s["q"], s["pos"], s["qw"], 64, torch.float64)
        if c["fmt"] == "fp8":
            codes, scale = _fp8(y)
            return {"codes": codes, "scale": scale}
        return _fp4_values(y).to(torch.bfloat16).flatten(0, 1)
    p = (s["ent"].to(torch.int64) + 1) * c["m"] - 1
    y = _norm_rope(s["k"].unsqueeze(1), p, s["kw"], 64, torch.float64).squeeze(1)
    at = _place(s)
    if c["fmt"] == "fp8":
        codes, scale = _fp8(y)
        s["codes"][at] = codes.view(torch.uint8)
        s["scale"][at] = scale
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scale": s["scale"]}
    out = _fp4_read(s["codes"], s["scale"]).to(torch.bfloat16)
    out[at] = _fp4_values(y).to(torch.bfloat16)
    return out


# ---- the framework's calls -----------------------------------------------------------
def _own(s):
    import long_context_compressed_04_b200 as L
    c = s["case"]
    op = c["op"]
    if op == "quant":
        lay = L.CSA_SF_TILED if c["tiled"] else L.CSA_SF_ROWS
        L.csa_mxfp4_quantize(s["x"], s["codes"], s["sf"], sf_layout=lay)
        L.csa_mxfp4_dequantize(s["codes"], s["sf"], s["out"], sf_layout=lay)
        return s["out"]
    if op == "product":
        L.csa_mxfp4_quantize(s["x"], s["codes"], s["sf"], sf_layout=L.CSA_SF_TILED)
        L.csa_mxfp4_matmul(s["codes"], s["sf"], s["w"], s["w_sf_tiled"], s["out"])
        return s["out"]
    if op == "qk":
        L.csa_qk_norm_rope(s["q"], s["k"], s["pos"], s["q_out"], s["k_out"], q_weight=s["qw"],
                           k_weight=s["kw"], rope_dims=c["rope"], rope_theta=THETA, eps=EPS)
        return {"q": s["q_out"], "k": s["k_out"]}
    fmt = L.CSA_IDX_FP8 if c["fmt"] == "fp8" else L.CSA_IDX_MXFP4
    if op == "queries":
        L.csa_indexer_queries(s["q"], s["pos"], s["codes"], s["scale"], fmt=fmt, weight=s["qw"],
                              rope_theta=THETA, eps=EPS)
        if c["fmt"] == "fp8":
            return {"codes": s["codes"].view(torch.float8_e4m3fn), "scale": s["scale"]}
        L.csa_mxfp4_dequantize(s["codes"].flatten(0, 1), s["scale"].flatten(0, 1), s["out"])
        return s["out"]
    layout = L.cache_layout(s["table"])
    L.csa_indexer_append(s["k"], s["seq_len"], s["ent_off"], s["seq"], s["ent"], s["codes"],
                         s["scale"], B=c["B"], m=c["m"], fmt=fmt, weight=s["kw"],
                         rope_theta=THETA, eps=EPS, layout=layout)
    if c["fmt"] == "fp8":
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scale": s["scale"]}
    L.csa_mxfp4_dequantize(s["codes"], s["scale"], s["out"])
    return s["out"]


def run(s):
    return _own(s) if own else _plain(s)


# ---- the least that a pass reads, writes and computes ------------------------------------
def work(case):
    c = case
    op = c["op"]
    if op == "quant":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (BYTES[c["dtype"]] + 2), "flops": 3 * n}
    if op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K * BYTES[c["dtype"]] + N * K * 17 / 32 + M * N * BYTES[c["out"]],
                "flops": 2 * M * N * K}
    if op == "qk":
        n = c["T"] * (c["H"] + c["Hk"]) * c["D"]
        return {"bytes": n * 2 * BYTES[c["dtype"]] + 4 * c["T"] + 8 * c["D"], "flops": 7 * n}
    held = 1 if c["fmt"] == "fp8" else 2                 # e4m3 codes, or the values as bf16
    if op == "queries":
        n = c["Q"] * c["H"] * c["D"]
        return {"bytes": n * (BYTES[c["dtype"]] + held) + (4 * n / c["D"] if held == 1 else 0),
                "flops": 10 * n}
    n = c["B"] * c["add"] * c["D"]
    old = c["B"] * c["have"] * c["D"]
    if held == 1:
        return {"bytes": n * (BYTES[c["dtype"]] + 1) + 12 * n / c["D"], "flops": 10 * n}
    return {"bytes": n * (BYTES[c["dtype"]] + 2) + 8 * n / c["D"] + old * (17 / 32 + 2),
            "flops": 10 * n + old}


# ---- from the definitions, in 64 bits --------------------------------------------------
def _nearest(y, levels):
    """Nearest of the ascending `levels` to each y >= 0, as a level number; a tie goes to the
    even number, y past the last level to it."""
    mid = (levels[1:] + levels[:-1]) / 2
    lo = torch.bucketize(y, mid, right=False)              # numbers of midpoints < y
    hi = torch.bucketize(y, mid, right=True)               # ... <= y
    return torch.where(lo % 2 == 0, lo, hi)


def _exact_fp4(y):
    """MXFP4 values of rows in 64 bits."""
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=y.device)
    b = y.to(torch.float64).reshape(y.shape[:-1] + (y.shape[-1] // 32, 32))
    top = b.abs().max(-1, keepdim=True).values
    lg = torch.floor(torch.log2(top))                      # mended where log2 rounded across
    lg = torch.where(torch.exp2(lg) > top, lg - 1, lg)
    lg = torch.where(torch.exp2(lg + 1) <= top, lg + 1, lg)
    scale = torch.exp2(lg.clamp(min=-125.0) - 2)
    return (torch.sign(b) * levels[_nearest(b.abs() / scale, levels)] * scale).reshape(y.shape)


def _exact_rows(x, pos, weight, rope):
    """The normed and rotated rows in 64 bits, as complex pairs."""
    x = x.to(torch.float64)
    D = x.shape[-1]
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * weight.to(torch.float64)
    if rope == 0:
        return y
    j = torch.arange(rope // 2, dtype=torch.float64, device=x.device)
    angle = pos.to(torch.float64).reshape(-1, 1, 1) / THETA ** (2 * j / rope)
    z = torch.view_as_complex(y[..., D - rope:].reshape(y.shape[:-1] + (rope // 2, 2)).contiguous())
    z = torch.view_as_real(z * torch.polar(torch.ones_like(angle), angle)).flatten(-2)
    y = y.clone()
    y[..., D - rope:] = z
    return y


def _exact_fp8(y):
    """(code values, scales) of rows: e4m3 by its spacing, 2^-3 of the binade (least binade
    -6), one scale per row, itself held in fp32."""
    amax = y.abs().max(-1).values
    scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax)).to(torch.float32)
    v = y / scale.to(torch.float64)[..., None]
    ulp = torch.exp2((torch.frexp(v).exponent.to(torch.float64) - 1).clamp(min=-6.0) - 3)
    return (torch.round(v / ulp) * ulp).clamp(-448, 448), scale.to(torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "quant":
        return _exact_fp4(s["x"])
    if op == "product":
        v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6],
                         dtype=torch.float64, device=DEV)
        w = torch.empty((c["N"], c["K"]), dtype=torch.float64, device=DEV)
        w[:, 0::2], w[:, 1::2] = v[(s["w"] % 16).long()], v[(s["w"] // 16).long()]
        w = (w.view(c["N"], -1, 32) * torch.exp2(s["w_sf"].double() - 127)[..., None]).flatten(1)
        return _exact_fp4(s["x"]) @ w.t()
    if op == "qk":
        return {"q": _exact_rows(s["q"], s["pos"], s["qw"], c["rope"]),
                "k": None if s["k"] is None else _exact_rows(s["k"], s["pos"], s["kw"],
                                                             c["rope"])}
    if op == "queries":
        y = _exact_rows(s["q"], s["pos"], s["qw"], 64)
        if c["fmt"] == "mxfp4":
            return _exact_fp4(y).flatten(0, 1)
        codes, scale = _exact_fp8(y)
        return {"codes": codes, "scale": scale}
    y = _exact_rows(s["k"][:, None], c["m"] * (s["ent"].double() + 1) - 1, s["kw"], 64)[:, 0]
    e, b = s["ent"].long(), s["seq"].long()
    at = s["ent_off"][b] + e if s["table"] is None else \
        32 * s["table"].long()[b, e.div(32, rounding_mode="floor")] + e.remainder(32)
    if c["fmt"] == "fp8":
        codes, scale = s["codes"].view(torch.float8_e4m3fn).double(), s["scale"].double()
        codes[at], scale[at] = _exact_fp8(y)
        return {"codes": codes, "scale": scale}
    v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6],
                     dtype=torch.float64, device=DEV)
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
    out[:, 0::2], out[:, 1::2] = v[(s["codes"] % 16).long()], v[(s["codes"] // 16).long()]
    out = (out.view(out.shape[0], -1, 32)
           * torch.exp2(s["scale"].double() - 127)[..., None]).flatten(1)
    out[at] = _exact_fp4(y)
    return out
