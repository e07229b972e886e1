"""Host side of the operators that make the indexer's inputs (CPU only): the 64-bit forms
against library casts, the scale sizes, and every refusal of bad arguments before a launch."""
import ctypes
import os
import subprocess
import sys

import ml_dtypes
import numpy as np
import pytest
import torch

import _inputs_orc as io
import long_context_compressed_04_b200 as L
from long_context_compressed_04_b200 import build, pipeline

P = ctypes.c_void_p
F = P(4096)          # never dereferenced: validation fails before any launch
ODD = P(4098)
lib = L._lib


def _err():
    return lib.csa_last_error().decode()


def test_e2m1_rounding_matches_library_cast():
    y = np.concatenate([np.linspace(-7, 7, 20001), io.LEVELS, -io.LEVELS,
                        (io.LEVELS[1:] + io.LEVELS[:-1]) / 2, [1e-30, -1e-30, 5.0, -5.0, 100.0]])
    ref = np.clip(y, -6, 6).astype(ml_dtypes.float4_e2m1fn).astype(np.float64)
    c = io.e2m1_codes(y)
    assert np.array_equal(np.where(c >= 8, -1, 1) * io.LEVELS[c & 7], ref)


def test_e4m3_rounding_matches_library_cast():
    # on fp32 values, where the library's cast rounds once; and between them
    y = np.linspace(-470, 470, 200001).astype(np.float32).astype(np.float64)
    y = np.concatenate([y, y / 500, y / 2.0 ** 16])
    ref = np.clip(y, -448, 448).astype(np.float32).astype(ml_dtypes.float8_e4m3fn)
    assert np.array_equal(io.e4m3_round(y), ref.astype(np.float64))
    assert io.e4m3_round(np.array([12.5 * (1 + 2.0 ** -30), 12.5, 13.5 * (1 - 2.0 ** -30)])).tolist() == [13, 12, 13]


def test_mxfp4_of_values_it_holds_is_lossless():
    # rows whose blocks each hold a 4 or a 6, so that the scale is the drawn one; powers of two
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, (20, 96)).astype(np.uint8)
    codes[:, ::32] = 7
    sf = rng.integers(1, 250, (20, 3)).astype(np.uint8)
    v = io.mxfp4_values(io.pack(codes), sf)
    p, s = io.mxfp4(v)
    assert np.array_equal(s, sf) and np.array_equal(p, io.pack(codes))
    assert np.array_equal(io.mxfp4_values(p, s), v)


def test_rotation_keeps_norms_and_relative_angles():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 2, 128))
    a = io.norm_rope(x, [5, 100, 1 << 20], rope=64)
    assert np.allclose((a * a).mean(-1), 1, atol=1e-5)
    q, k = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    d = [np.sum(io.norm_rope(q, [p], norm=False) * io.norm_rope(k, [p - 7], norm=False))
         for p in (7, 1000, 70000)]
    assert np.allclose(d, d[0], rtol=1e-9)


def test_scale_sizes():
    assert L.csa_mxfp4_sf_bytes(5, 96) == 15
    assert L.csa_mxfp4_sf_bytes(5, 96, L.CSA_SF_TILED) == 512
    assert L.csa_mxfp4_sf_bytes(129, 160, L.CSA_SF_TILED) == 4 * 512
    assert L.csa_mxfp4_sf_bytes(0, 96) == 0 and L.csa_mxfp4_sf_bytes(-1, 96) == 0
    # offsets past 32 bits
    assert L.csa_mxfp4_sf_bytes(1 << 31, 4096) == (1 << 31) * 128


def _quant(x=F, dt=0, rows=4, cols=64, ld=64, codes=F, sf=F, lay=0):
    return lib.csa_mxfp4_quantize(x, dt, rows, cols, ld, codes, sf, lay, None, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dt=3), 1, "element type"), (dict(lay=2), 1, "layout"), (dict(rows=-1), 1, ">= 0"),
    (dict(cols=48, ld=48), 1, "multiple of 32"), (dict(cols=0), 1, "multiple of 32"),
    (dict(cols=1 << 21, ld=1 << 21), 2, "not supported"),
    (dict(rows=1 << 31), 2, "not supported"), (dict(x=None), 1, "null"),
    (dict(codes=None), 1, "null"), (dict(sf=None), 1, "null"), (dict(x=ODD), 1, "aligned"),
    (dict(ld=63), 1, "stride"), (dict(ld=66), 1, "stride"), (dict(ld=32), 1, "stride")])
def test_quantize_refusals(kw, status, text):
    assert _quant(**kw) == status and text in _err()


def test_zero_sizes_are_no_ops():
    assert _quant(rows=0, x=None, codes=None, sf=None) == 0
    assert lib.csa_mxfp4_dequantize(None, None, 0, 0, 64, None, 0, 64, None) == 0
    assert lib.csa_mxfp4_matmul(None, None, None, None, 0, 8, 64, None, 0, 8, None, None) == 0
    assert lib.csa_mxfp4_matmul(None, None, None, None, 8, 0, 64, None, 0, 8, None, None) == 0
    assert _qk(T=0, q=None, qo=None) == 0 and _qk(H=0, Hk=0, pos=None) == 0
    assert _queries(Q=0, q=None) == 0 and _append(n=0, k=None) == 0


@pytest.mark.parametrize("args,status,text", [
    ((None, F, 0, 4, 64, F, 0, 64, None), 1, "null"),
    ((F, F, 0, 4, 64, ODD, 0, 64, None), 1, "aligned"),
    ((F, F, 0, 4, 64, F, 0, 60, None), 1, "stride"),
    ((F, F, 0, 4, 40, F, 0, 64, None), 1, "multiple of 32"),
    ((F, F, 7, 4, 64, F, 0, 64, None), 1, "layout"),
    ((F, F, 0, 4, 64, F, 9, 64, None), 1, "element type")])
def test_dequantize_refusals(args, status, text):
    assert lib.csa_mxfp4_dequantize(*args) == status and text in _err()


@pytest.mark.parametrize("args,status,text", [
    ((F, F, F, F, 4, 8, 48, F, 0, 8, None, None), 1, "multiple of 32"),
    ((F, F, F, F, -4, 8, 64, F, 0, 8, None, None), 1, ">= 0"),
    ((F, F, F, F, 4, -8, 64, F, 0, 8, None, None), 1, ">= 0"),
    ((F, F, F, F, 4, 8, 64, F, 0, 7, None, None), 1, "stride"),
    ((F, F, F, F, 4, 8, 64, P(4097), 0, 8, None, None), 1, "alignment"),
    ((F, ODD, F, F, 4, 8, 64, F, 0, 8, None, None), 1, "aligned"),
    ((F, F, F, None, 4, 8, 64, F, 0, 8, None, None), 1, "null"),
    ((F, F, F, F, (1 << 23) + 1, 8, 64, F, 0, 8, None, None), 2, "not supported"),
    ((F, F, F, F, 4, 8, 64, F, 5, 8, None, None), 1, "element type")])
def test_matmul_refusals(args, status, text):
    assert lib.csa_mxfp4_matmul(*args) == status and text in _err()


def _qk(q=F, st=256, sh=128, k=F, pos=F, qw=None, qo=F, ko=F, dt=0, T=2, H=2, Hk=1, D=128,
        rope=64, norm=1, theta=1e4, eps=1e-6, ost=256, osh=128, kst=128):
    return lib.csa_qk_norm_rope(q, st, sh, k, 128, 128, pos, qw, None, qo, ost, osh, ko, kst, 128,
                                dt, T, H, Hk, D, rope, norm, theta, eps, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(D=100), 2, "head dim"), (dict(D=1032), 2, "head dim"), (dict(D=0), 2, "head dim"),
    (dict(rope=63), 1, "rope_dims"), (dict(rope=130), 1, "rope_dims"), (dict(rope=-2), 1, "rope"),
    (dict(D=256, rope=130), 2, "rope_dims"), (dict(norm=2), 1, "norm"), (dict(theta=1.0), 1, "theta"),
    (dict(eps=-1.0), 1, "eps"), (dict(qw=P(4100)), 1, "aligned"), (dict(q=None), 1, "null"),
    (dict(ko=None), 1, "null"), (dict(pos=None), 1, "null"), (dict(q=ODD), 1, "aligned"),
    (dict(sh=130), 1, "aligned"), (dict(st=100), 1, "aligned"), (dict(T=-1), 1, ">= 0"),
    (dict(Hk=-1), 1, ">= 0"), (dict(dt=4), 1, "element type"),
    (dict(theta=float("nan")), 1, "theta"), (dict(H=(1 << 20) + 1), 2, "heads"),
    (dict(osh=0), 1, "overlap"), (dict(ost=128), 1, "overlap"), (dict(ost=0), 1, "overlap"),
    (dict(osh=64), 1, "overlap"), (dict(kst=64), 1, "overlap"), (dict(ost=-256), 1, "overlap")])
def test_qk_norm_rope_refusals(kw, status, text):
    assert _qk(**kw) == status and text in _err()


def _queries(q=F, dt=0, st=256, sh=128, pos=F, w=None, norm=1, rope=64, theta=1e4, eps=1e-6, Q=2,
             H=2, D=128, fmt=0, codes=F, scale=F):
    return lib.csa_indexer_queries(q, dt, st, sh, pos, w, norm, rope, theta, eps, Q, H, D, fmt,
                                   codes, scale, None, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(D=96), 2, "indexer dim"), (dict(fmt=2), 1, "format"), (dict(rope=60), 1, "rope_dims"),
    (dict(D=64, rope=72), 1, "rope_dims"), (dict(q=None), 1, "null"), (dict(scale=None), 1, "null"),
    (dict(codes=P(4104)), 1, "aligned"), (dict(scale=P(4097)), 1, "aligned"),
    (dict(st=100), 1, "aligned"), (dict(Q=-1), 1, ">= 0"), (dict(norm=-1), 1, "norm"),
    (dict(dt=-1), 1, "element type"), (dict(w=P(4)), 1, "aligned")])
def test_indexer_queries_refusals(kw, status, text):
    assert _queries(**kw) == status and text in _err()


def _append(k=F, dt=0, ld=128, seq_len=F, off=F, seq=F, ent=F, n=2, B=1, m=4, rope=64, D=128,
            fmt=0, codes=F, scale=F, rows=8, lay=None):
    return lib.csa_indexer_append(k, dt, ld, seq_len, off, seq, ent, n, B, m, None, 1, rope, 1e4,
                                  1e-6, D, fmt, codes, scale, rows, lay, None, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(n=-1), 1, "n_items"), (dict(n=1 << 31), 1, "n_items"), (dict(B=0), 1, "B and m"),
    (dict(m=0), 1, "B and m"), (dict(rows=-1), 1, "ent_rows"), (dict(rows=1 << 31), 1, "ent_rows"),
    (dict(off=None), 1, "ent_off"), (dict(k=None), 1, "null"), (dict(ent=None), 1, "null"),
    (dict(ld=120), 1, "stride"), (dict(ld=130), 1, "stride"), (dict(D=32), 2, "indexer dim"),
    (dict(lay=ctypes.byref(L.CacheLayout(4096, 4, 0)), m=128), 1, "m = 4"),
    (dict(lay=ctypes.byref(L.CacheLayout(4096, 0, 0))), 1, "bt_stride")])
def test_indexer_append_refusals(kw, status, text):
    assert _append(**kw) == status and text in _err()


def test_binding_refuses_tensors_it_would_read_past():
    u8 = lambda *n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(L.CSAError, match="codes must be"):
        L.csa_mxfp4_quantize(x, u8(4, 31), u8(4, 2))
    with pytest.raises(L.CSAError, match="at least 8 bytes"):
        L.csa_mxfp4_quantize(x, u8(4, 32), u8(7))
    with pytest.raises(L.CSAError, match="contiguous rows"):
        L.csa_mxfp4_quantize(x.t(), u8(64, 2), u8(64))
    with pytest.raises(L.CSAError, match="bfloat16, float16 or float32"):
        L.csa_mxfp4_quantize(x.double(), u8(4, 32), u8(4, 2))
    with pytest.raises(L.CSAError, match="CUDA device"):
        L.csa_mxfp4_quantize(x, u8(4, 32), u8(4, 2))
    with pytest.raises(L.CSAError, match="b's codes"):
        L.csa_mxfp4_matmul(u8(4, 32), u8(512), u8(8, 16), u8(512), torch.zeros((4, 8)))
    with pytest.raises(L.CSAError, match="a's scales"):
        L.csa_mxfp4_matmul(u8(4, 32), u8(8), u8(8, 32), u8(512), torch.zeros((4, 8)))
    q, pos = torch.zeros((3, 2, 128)), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(L.CSAError, match="heads of q and k"):
        L.csa_qk_norm_rope(q, None, pos, q[:, :1], None)
    with pytest.raises(L.CSAError, match="one element type"):
        L.csa_qk_norm_rope(q, None, pos, q.half(), None)
    with pytest.raises(L.CSAError, match="pos must be"):
        L.csa_qk_norm_rope(q, None, pos.long(), q, None)
    with pytest.raises(L.CSAError, match="both None"):
        L.csa_qk_norm_rope(None, None, pos, None, None)
    with pytest.raises(L.CSAError, match="q_weight"):
        L.csa_qk_norm_rope(q, None, pos, q, None, q_weight=torch.ones(64))
    with pytest.raises(L.CSAError, match="scale must be"):
        L.csa_indexer_queries(q, pos, u8(3, 2, 128), torch.zeros((3, 1)))
    with pytest.raises(L.CSAError, match="codes must be"):
        L.csa_indexer_queries(q, pos, u8(3, 2, 128), u8(3, 2, 4), fmt=L.CSA_IDX_MXFP4)
    k, i32, i64 = torch.zeros((5, 128)), torch.zeros(5, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(L.CSAError, match="item_ent"):
        L.csa_indexer_append(k, i64, i64, i32, i32[:4], u8(9, 128), torch.zeros(9), B=2)
    with pytest.raises(L.CSAError, match="seq_len"):
        L.csa_indexer_append(k, i64, i64, i32, i32, u8(9, 128), torch.zeros(9), B=3)
    with pytest.raises(L.CSAError, match="scale must be"):
        L.csa_indexer_append(k, i64, i64, i32, i32, u8(9, 128), torch.zeros(8), B=2)


def test_append_reads_no_block_past_a_slice_of_the_table(monkeypatch):
    # what the library is handed: the bound it tests an entry's block against (the stride) is the
    # width of the table that the caller gave, and its rows are those of that table
    seen = []

    def call(*a):
        lay = a[20]._obj
        assert lay.bt_stride == table.shape[1]
        rows = ctypes.cast(lay.block_table, ctypes.POINTER(ctypes.c_int32))
        seen.extend(rows[i] for i in range(a[8] * lay.bt_stride))
        return 0

    monkeypatch.setattr(L, "_marshal", None)
    monkeypatch.setattr(L, "_idx_append", call)
    monkeypatch.setattr(L, "_is_current", lambda dev: True)
    monkeypatch.setattr(L, "_stream_on", lambda stream, dev: None)
    big = torch.arange(40, dtype=torch.int32).view(4, 10)
    for table, B in ((big, 4), (big[:, 2:], 4), (big[:, 3:6], 3), (big[2:, :4], 2), (big[3:, 7:], 1), (big[1:], 1)):
        k, i32 = torch.zeros((5, 128)), torch.zeros(5, dtype=torch.int32)
        L.csa_indexer_append(k, torch.zeros(B, dtype=torch.int64), None, i32, i32, torch.zeros((9, 128), dtype=torch.uint8),
                             torch.zeros(9), B=B, layout=L.cache_layout(table))
        assert seen == table[:B].flatten().tolist()
        seen.clear()


def test_marshalling_built_for_another_torch_is_not_used():
    # its accessors hold another torch's tensor layout: the package goes on without it
    code = ("import torch; torch.__version__ = '0.0.1'; import long_context_compressed_04_b200 as L; "
            "assert L._marshal is None")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr
    assert L._marshal is not None and L._marshal.torch_version == torch.__version__


@pytest.fixture
def marshal_build(monkeypatch, tmp_path):
    """build.build_marshal in a directory of its own, its compiler runs counted, not made."""
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_csa_marshal.so"))
    monkeypatch.setattr(build, "OBJ_DIR", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", run)
    return runs


def test_marshalling_is_built_again_for_another_torch(marshal_build, monkeypatch):
    build.build_marshal()
    build.build_marshal()
    assert len(marshal_build) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build.build_marshal()
    build.build_marshal()
    assert len(marshal_build) == 2


@pytest.mark.parametrize("fails", ["compiler", "compile", "headers"])
def test_library_builds_where_the_marshalling_cannot(marshal_build, monkeypatch, capfd, fails):
    # no host compiler, one that refuses the source, a torch without its paths: the library is built
    # all the same, and no marshalling of an older source is left behind
    open(build.MARSHAL, "w").close()
    run = build.subprocess.run

    def failing(cmd, **kw):
        if cmd[0].endswith("g++"):
            if fails == "compiler":
                raise FileNotFoundError("g++")
            if fails == "compile":
                return subprocess.CompletedProcess(cmd, 1, "", "no Python.h")
        return run(cmd, **kw)

    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(build.subprocess, "run", failing)
    monkeypatch.setattr(build, "OUT", os.path.join(build.OBJ_DIR, "libcsa.so"))
    if fails == "headers":
        monkeypatch.delattr(torch, "_C")
    assert build.build(force=True) == build.OUT and os.path.exists(build.OUT)
    assert not os.path.exists(build.MARSHAL) and "without it" in capfd.readouterr().err


@pytest.mark.parametrize("capturing", [False, True])
def test_projection_is_complete_when_built(monkeypatch, capturing):
    # the weight's quantisation reports to the projection's status and is waited for (not inside a
    # capture), so that a first call on another stream reads all of it
    events = []

    class Stream:
        def synchronize(self):
            events.append("wait")

    monkeypatch.setattr(pipeline, "csa_mxfp4_quantize", lambda x, c, s, **kw: events.append(kw["dev_status"]))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    p = pipeline.QueryProjection(torch.zeros((256, 64)), 2, 128, max_q=3)
    assert events[0] is p.dev_status and events[1:] == ([] if capturing else ["wait"])
