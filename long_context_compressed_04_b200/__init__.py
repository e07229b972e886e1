"""Hybrid compressed attention (CSA / HCA) on B200: Python binding of libcsa.

Argument marshalling only: every function here passes tensor pointers, sizes and the
current CUDA stream to the C ABI of ``libcsa.so`` (declared in ``include/csa.h``) and raises
``CSAError`` when it returns a non-zero status.  All computation happens in the CUDA
kernels.  There is no CPU fallback: importing this package fails if ``libcsa.so`` has not
been built (``python long_context_compressed_04_b200/build.py``).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import sys
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa.so")

CSA_KV_BF16 = 0
CSA_KV_FP8_576 = 1
CSA_DT_BF16 = 0
CSA_DT_F16 = 1
CSA_DT_F32 = 2
CSA_SF_ROWS = 0
CSA_SF_TILED = 1
CSA_IDX_FP8 = 0
CSA_IDX_MXFP4 = 1
CSA_DEV_OOB = 1
CSA_DEV_TIMEOUT = 2
CSA_DEV_NAN = 4
CSA_DEV_CAPACITY = 8

STATUS_NAMES = {0: "CSA_OK", 1: "CSA_ERR_INVALID_ARG", 2: "CSA_ERR_UNSUPPORTED",
                3: "CSA_ERR_CUDA", 4: "CSA_ERR_WORKSPACE"}


class CSAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python long_context_compressed_04_b200/build.py` (needs nvcc)")

_lib = ctypes.CDLL(LIB_PATH)
_P, _I32, _I64, _F32, _SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
_SIGS = {
    "csa_version": (ctypes.c_int, []),
    "csa_last_error": (ctypes.c_char_p, []),
    "csa_entry_row_bytes": (_I32, [_I32, _I32]),
    "csa_compress": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I32,
                                    _F32, _F32, _P, _P, _P, _P]),
    "hca_compress": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I32,
                                    _F32, _F32, _P, _P, _P, _P]),
    "csa_indexer_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "lightning_indexer_topk": (ctypes.c_int, [_P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _I32, _I32, _I32,
                                              _I32, _I32, _I32, _I32, _P, _P, _I64, _P, _SZ, _P,
                                              _P, _P]),
    "sparse_mqa_attn": (ctypes.c_int, [_P, _P, _I32, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _P,
                                       _I32, _I32, _I32, _I32, _I32, _F32, _F32, _F32, _P, _P,
                                       _P, _P]),
    "dense_hca_workspace_size": (_SZ, [_I32, _I32, _I32, _I32]),
    "dense_hca_attn": (ctypes.c_int, [_P, _P, _I32, _I64, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _I32, _I32,
                                      _I32, _I32, _I32, _F32, _F32, _F32, _I32, _P, _P, _SZ, _P,
                                      _P, _P]),
    "lightning_indexer_topk_noalloc": (ctypes.c_int, [_P, _P, _P, _P, _P, _I64, _P, _P, _P, _P,
                                                      _I32,
                                                      _I32, _I32, _I32, _I32, _I32, _I32, _P, _P,
                                                      _I64, _P, _P]),
    "csa_launch_count": (ctypes.c_longlong, []),
    "csa_profile_enable": (None, [ctypes.c_int]),
    "csa_profile_collect": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int]),
    "csa_debug_set_wait_limit": (ctypes.c_int, [ctypes.c_longlong]),
    "lightning_indexer_topk_mxfp4": (ctypes.c_int, [_P, _P, _P, _P, _P, _I64, _P, _P, _P, _P,
                                                    _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                                    _I32, _P, _P, _I64, _P, _SZ, _P, _P, _P]),
    "csa_cache_append": (ctypes.c_int, [_P, _P, _P, _P, _I32, _P, _P, _P, _I64, _P, _I64, _I32,
                                        _I32, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "csa_topk_merge": (ctypes.c_int, [_P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P]),
    "csa_cp_candidates": (ctypes.c_int, [_P, _P, _I64, _P, _P, _I32, _I32, _I32, _P, _P, _P,
                                         _P]),
    "csa_cp_pack_rows": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32,
                                        _P, _P, _P, _P]),
    "csa_mxfp4_sf_bytes": (_SZ, [_I64, _I64, _I32]),
    "csa_mxfp4_quantize": (ctypes.c_int, [_P, _I32, _I64, _I64, _I64, _P, _P, _I32, _P, _P]),
    "csa_mxfp4_dequantize": (ctypes.c_int, [_P, _P, _I32, _I64, _I64, _P, _I32, _I64, _P]),
    "csa_mxfp4_matmul": (ctypes.c_int, [_P, _P, _P, _P, _I64, _I64, _I64, _P, _I32, _I64, _P,
                                        _P]),
    "csa_qk_norm_rope": (ctypes.c_int, [_P, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _P, _I64,
                                        _I64, _P, _I64, _I64, _I32, _I32, _I32, _I32, _I32, _I32,
                                        _I32, _F32, _F32, _P]),
    "csa_indexer_queries": (ctypes.c_int, [_P, _I32, _I64, _I64, _P, _P, _I32, _I32, _F32, _F32,
                                           _I32, _I32, _I32, _I32, _P, _P, _P, _P]),
    "csa_indexer_append": (ctypes.c_int, [_P, _I32, _I64, _P, _P, _P, _P, _I64, _I32, _I32, _P,
                                          _I32, _I32, _F32, _F32, _I32, _I32, _P, _P, _I64, _P,
                                          _P, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)


class CacheLayout(ctypes.Structure):
    """csa_cache_layout_t (see include/csa.h): the classical cache's block table and the
    state cache's ring size."""
    _fields_ = [("block_table", ctypes.c_void_p), ("bt_stride", ctypes.c_int64),
                ("kv_ring", ctypes.c_int64)]


def cache_layout(block_table=None, kv_ring: int = 0):
    """A cache layout for the calls' ``layout`` argument, or None for the contiguous one.
    block_table: int32 [B, bt_stride] device tensor (blocks of 32 CSA entries); kv_ring:
    rows of each sequence's state-cache ring (0 = linear raw store)."""
    if block_table is None and not kv_ring:
        return None
    lay = CacheLayout(None if block_table is None else block_table.data_ptr(),
                      0 if block_table is None else block_table.stride(0), int(kv_ring))
    lay._block_table = block_table      # keeps the tensor alive with the struct
    return lay


def _lay(layout):
    return None if layout is None else ctypes.byref(layout)


def _p(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _s(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int):
    if status != 0:
        raise CSAError(status, _lib.csa_last_error().decode())


class _KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 40), ("launches", ctypes.c_longlong),
                ("total_ms", ctypes.c_double)]


def csa_launch_count() -> int:
    return _lib.csa_launch_count()


def csa_profile_enable(on: bool = True):
    _lib.csa_profile_enable(1 if on else 0)


def csa_profile_collect(keep_pending: bool = False) -> dict:
    """{kernel name: (timed launches, total device ms)} since the last collect.  With
    keep_pending, the recorded event pairs stay registered (for CUDA-graph replays)."""
    arr = (_KernelTime * 32)()
    n = _lib.csa_profile_collect(ctypes.cast(arr, ctypes.c_void_p), 32, 1 if keep_pending else 0)
    return {arr[i].name.decode(): (arr[i].launches, arr[i].total_ms) for i in range(n)}


def csa_debug_set_wait_limit(cycles: int = 0):
    """Test hook: limit (SM clocks) of the kernels' bounded waits; 0 restores the default.
    Synchronous; call it with no libcsa kernel in flight and outside stream capture."""
    _check(_lib.csa_debug_set_wait_limit(int(cycles)))


def csa_version() -> int:
    return _lib.csa_version()


def csa_entry_row_bytes(fmt: int, D: int) -> int:
    return _lib.csa_entry_row_bytes(fmt, D)


def csa_indexer_workspace_size(Q: int, max_n: int, k: int) -> int:
    return _lib.csa_indexer_workspace_size(Q, max_n, k)


def dense_hca_workspace_size(Q: int, H: int, D: int, max_n: int) -> int:
    return _lib.dense_hca_workspace_size(Q, H, D, max_n)


def csa_compress(kv, gate, pos_bias, seq_len, kv_off, kv_pos0, ent_off, item_seq, item_ent,
                 entries, *,
                 B: int, D: int, fmt: int = CSA_KV_BF16, rope_theta: float = 10000.0,
                 eps: float = 1e-6, layout=None, dev_status=None, stream=None):
    _check(_lib.csa_compress(_p(kv), _p(gate), _p(pos_bias), _p(seq_len), _p(kv_off), _p(kv_pos0),
                             _p(ent_off), _p(item_seq), _p(item_ent), item_seq.numel(), B, D, fmt,
                             rope_theta, eps, _p(entries), _lay(layout), _p(dev_status),
                             _s(stream)))


def hca_compress(kv, gate, pos_bias, seq_len, kv_off, kv_pos0, ent_off, item_seq, item_ent,
                 entries, *,
                 B: int, D: int, fmt: int = CSA_KV_BF16, rope_theta: float = 10000.0,
                 eps: float = 1e-6, layout=None, dev_status=None, stream=None):
    _check(_lib.hca_compress(_p(kv), _p(gate), _p(pos_bias), _p(seq_len), _p(kv_off), _p(kv_pos0),
                             _p(ent_off), _p(item_seq), _p(item_ent), item_seq.numel(), B, D, fmt,
                             rope_theta, eps, _p(entries), _lay(layout), _p(dev_status),
                             _s(stream)))


def lightning_indexer_topk(qI, qI_scale, w, kI, kI_scale, seq_len, ent_off, q_seq, q_pos, idx_out,
                           workspace, *, B: int, H_I: int, d_I: int, m: int, k: int, max_n: int,
                           scores_out=None, ld_scores: int = 0, layout=None, dev_status=None,
                           stream=None):
    _check(_lib.lightning_indexer_topk(
        _p(qI), _p(qI_scale), _p(w), _p(kI), _p(kI_scale), kI_scale.numel(), _p(seq_len),
        _p(ent_off), _p(q_seq),
        _p(q_pos),
        q_seq.numel(), B, H_I, d_I, m, k, max_n, _p(idx_out), _p(scores_out), ld_scores,
        _p(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
        _lay(layout), _p(dev_status), _s(stream)))


NOALLOC_SCRATCH_BYTES = 16 << 20


def lightning_indexer_topk_noalloc(qI, qI_scale, w, kI, kI_scale, seq_len, ent_off, q_seq, q_pos,
                                   idx_out, *, B: int, H_I: int, d_I: int, m: int, k: int,
                                   max_n: int, scores_out=None, ld_scores: int = 0,
                                   dev_status=None, stream=None):
    """lightning_indexer_topk without a workspace, for callers that cannot allocate device
    memory: the scratch lives in a fixed 16 MiB device array inside libcsa, shared by all
    calls on a device (calls that overlap on the GPU race on it)."""
    _check(_lib.lightning_indexer_topk_noalloc(
        _p(qI), _p(qI_scale), _p(w), _p(kI), _p(kI_scale), kI_scale.numel(), _p(seq_len),
        _p(ent_off), _p(q_seq),
        _p(q_pos), q_seq.numel(), B, H_I, d_I, m, k, max_n, _p(idx_out), _p(scores_out),
        ld_scores, _p(dev_status), _s(stream)))


def lightning_indexer_topk_mxfp4(qI, qI_sf, w, kI, kI_sf, seq_len, ent_off, q_seq, q_pos,
                                 idx_out, workspace, *, B: int, H_I: int, d_I: int, m: int,
                                 k: int, max_n: int, select_bf16: bool = False, scores_out=None,
                                 ld_scores: int = 0, layout=None, dev_status=None,
                                 stream=None):
    """MXFP4 indexer + top-k (see include/csa.h).  qI / kI: packed e2m1 bytes; qI_sf /
    kI_sf: UE8M0 bytes."""
    _check(_lib.lightning_indexer_topk_mxfp4(
        _p(qI), _p(qI_sf), _p(w), _p(kI), _p(kI_sf), kI.shape[0], _p(seq_len), _p(ent_off),
        _p(q_seq), _p(q_pos), q_seq.numel(), B, H_I, d_I, m, k, max_n, 1 if select_bf16 else 0,
        _p(idx_out), _p(scores_out), ld_scores, _p(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _lay(layout), _p(dev_status), _s(stream)))


def csa_cache_append(kv_new, gate_new, seq_len, kv_off, kv_pos0, kv, gate, *, B: int, D: int,
                     m: int, kI_new=None, kI_scale_new=None, ent_off=None, kI=None,
                     kI_scale=None, layout=None, dev_status=None, stream=None):
    """One decode token per sequence into the state cache (and, for the entries it
    completes, their indexer keys into the key store); see include/csa.h."""
    _check(_lib.csa_cache_append(
        _p(kv_new), _p(gate_new), _p(kI_new), _p(kI_scale_new),
        0 if kI is None else kI.shape[1], _p(seq_len), _p(kv_off), _p(kv_pos0), kv.shape[0],
        _p(ent_off), 0 if kI is None else kI.shape[0], B, D, m, _p(kv), _p(gate), _p(kI),
        _p(kI_scale), _lay(layout), _p(dev_status), _s(stream)))


def csa_topk_merge(cand_scores, cand_idx, idx_out, *, dev_status=None, stream=None):
    """Top-k of sequences from their slices' candidates, [W, Q, k_in] (see include/csa.h)."""
    W, Q, k_in = cand_idx.shape
    assert cand_scores.shape == cand_idx.shape
    assert cand_idx.stride() == cand_scores.stride() and cand_idx.stride()[1:] == (k_in, 1)
    _check(_lib.csa_topk_merge(_p(cand_scores), _p(cand_idx), cand_idx.stride(0), W, Q, k_in,
                               idx_out.shape[1], _p(idx_out), _p(dev_status), _s(stream)))


def csa_cp_candidates(idx, scores, q_seq, slice_lo, cand_idx, cand_scores, *, B: int,
                      dev_status=None, stream=None):
    """A slice's selection as candidates of the whole sequence (see include/csa.h)."""
    Q, k = idx.shape
    _check(_lib.csa_cp_candidates(_p(idx), _p(scores), scores.stride(0), _p(q_seq),
                                  _p(slice_lo), Q, B, k, _p(cand_idx), _p(cand_scores),
                                  _p(dev_status), _s(stream)))


def csa_cp_pack_rows(idx, q_seq, slice_lo, slice_n, ent_off, entries, out, local_idx=None, *,
                     B: int, dev_status=None, stream=None):
    """The selected rows this rank's slice holds, at their positions (see include/csa.h)."""
    Q, k = idx.shape
    _check(_lib.csa_cp_pack_rows(_p(idx), _p(q_seq), _p(slice_lo), _p(slice_n), _p(ent_off),
                                 _p(entries), entries.shape[0], entries.shape[1], Q, B, k,
                                 _p(out), _p(local_idx), _p(dev_status), _s(stream)))


def sparse_mqa_attn(q, entries, seq_len, ent_off, kv, kv_off, kv_pos0, q_seq, q_pos, idx, sink,
                    out, *,
                    fmt: int, B: int, H: int, D: int, W: int, m: int, k: int,
                    softmax_scale: float, rope_theta: float = 10000.0, eps: float = 1e-6,
                    layout=None, dev_status=None, stream=None):
    _check(_lib.sparse_mqa_attn(
        _p(q), _p(entries), fmt, entries.shape[0], _p(seq_len), _p(ent_off), _p(kv), _p(kv_off), _p(kv_pos0), _p(q_seq),
        _p(q_pos), _p(idx), k, m, _p(sink), q_seq.numel(), B, H, D, W, softmax_scale,
        rope_theta, eps, _p(out), _lay(layout), _p(dev_status), _s(stream)))


def dense_hca_attn(q, entries, seq_len, ent_off, kv, kv_off, kv_pos0, q_seq, q_pos, sink, out,
                   workspace, *, fmt: int, B: int, H: int, D: int, W: int, m: int, max_n: int,
                   softmax_scale: float, rope_theta: float = 10000.0, eps: float = 1e-6,
                   layout=None, dev_status=None, stream=None):
    _check(_lib.dense_hca_attn(
        _p(q), _p(entries), fmt, entries.shape[0], _p(seq_len), _p(ent_off), _p(kv), _p(kv_off), _p(kv_pos0), _p(q_seq),
        _p(q_pos), m, _p(sink), q_seq.numel(), B, H, D, W, softmax_scale, rope_theta, eps,
        max_n, _p(out), _p(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _lay(layout), _p(dev_status), _s(stream)))


# ---- the lightning indexer's inputs --------------------------------------------------
# These calls check their tensors' types, shapes and devices, since a wrong one would be
# read past its end; sizes and alignments are checked by the library.  Decode steps issue many
# small launches, and the host time per call is what bounds them: the tests and the
# conversion of the arguments are compiled (csrc/marshal.cpp).  Where a test fails, or that
# module was not built for this torch, the call below does the same in Python, finds the reason
# and raises.
_DTYPES = {torch.bfloat16: CSA_DT_BF16, torch.float16: CSA_DT_F16, torch.float32: CSA_DT_F32}
_U8, _I32T, _I64T, _F32T = torch.uint8, torch.int32, torch.int64, torch.float32
# The current stream's handle without a Stream object (3 us less per call) and the current
# device without the check that CUDA is initialised (a CUDA tensor is at hand), where torch has
# them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_mx_quantize, _mx_dequantize, _mx_matmul = (_lib.csa_mxfp4_quantize, _lib.csa_mxfp4_dequantize,
                                            _lib.csa_mxfp4_matmul)
_qk_norm_rope, _idx_queries, _idx_append = (_lib.csa_qk_norm_rope, _lib.csa_indexer_queries,
                                            _lib.csa_indexer_append)


def _load_marshal():
    """The compiled marshalling, or None where it was not built, or was built against another
    torch or Python, whose tensors it would read at the wrong places."""
    try:
        from . import _csa_marshal as m
    except ImportError:
        return None
    built = getattr(m, "torch_version", None), getattr(m, "python_tag", None)
    if built != (str(torch.__version__), sys.implementation.cache_tag):
        warnings.warn(f"_csa_marshal.so was built for torch {built[0]} ({built[1]}) and is not used: "
                      "build the package again")
        return None
    m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        _mx_quantize, _mx_dequantize, _mx_matmul, _qk_norm_rope, _idx_queries, _idx_append)))
    return m


_marshal = _load_marshal()


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def _bad(message: str):
    raise CSAError(1, message)


def _need_rows_dtype(t, name):
    if t.dtype not in _DTYPES:
        _bad(f"{name} must be bfloat16, float16 or float32, not {t.dtype}")


def _need(t, name, dtype, shape):
    """A contiguous tensor of this type and shape (None in the shape: any size there)."""
    if t.dtype != dtype or not t.is_contiguous() or t.dim() != len(shape) or \
            any(n is not None and n != m for n, m in zip(shape, t.shape)):
        want = "x".join("*" if n is None else str(n) for n in shape)
        _bad(f"{name} must be a contiguous {dtype} tensor of {want}, not {t.dtype} "
             f"{tuple(t.shape)} with strides {t.stride()}")


def _need_one_device(*tensors):
    """All tensors on the current CUDA device."""
    dev = tensors[0].device
    for t in tensors:
        if t is not None and t.device != dev:
            _bad(f"tensors on {dev} and {t.device}")
    if dev.type != "cuda" or dev.index != torch.cuda.current_device():
        _bad(f"tensors on {dev}: the current CUDA device is needed (torch.cuda.device)")


def _need_status(dev_status):
    if dev_status is not None and (dev_status.dtype != _I32T or dev_status.numel() < 1):
        _bad("dev_status must be an int32 tensor of at least one element")


def _need_2d(t, name):
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        _bad(f"{name} must be 2-D with contiguous rows, not {tuple(t.shape)} with strides "
             f"{t.stride()}")


def _is_current(dev):
    return dev >= 0 and dev == _device()


def _status_ok(t, dev):
    return t is None or (t.dtype is _I32T and t.numel() >= 1 and t.get_device() == dev)


def _dense_ok(t, dtype, n, dev):
    """n contiguous elements of this type."""
    return t.dtype is dtype and t.numel() == n and t.is_contiguous() and t.get_device() == dev


def _weight_ok(w, D, dev):
    return w is None or _dense_ok(w, _F32T, D, dev)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_on(stream, dev):
    if stream is not None:
        return stream.cuda_stream
    return torch.cuda.current_stream().cuda_stream if _raw_stream is None else _raw_stream(dev)


def csa_mxfp4_sf_bytes(rows: int, cols: int, sf_layout: int = CSA_SF_ROWS) -> int:
    return _lib.csa_mxfp4_sf_bytes(rows, cols, sf_layout)


def _mxfp4_ok(codes, sf, rows, cols, sf_layout, dev):
    need = (rows + 127) // 128 * ((cols + 127) // 128) * 512 if sf_layout else rows * (cols // 32)
    return (codes.dtype is _U8 and codes.numel() == rows * (cols // 2) and codes.is_contiguous()
            and sf.dtype is _U8 and sf.numel() >= need and sf.is_contiguous()
            and codes.get_device() == dev and sf.get_device() == dev)


def _need_mxfp4(codes, sf, rows, cols, sf_layout, what):
    _need(codes, f"{what} codes", _U8, (rows, cols // 2))
    need = csa_mxfp4_sf_bytes(rows, cols, sf_layout)
    if sf.dtype != _U8 or not sf.is_contiguous() or sf.numel() < need:
        _bad(f"{what} scales must be a contiguous uint8 tensor of at least {need} bytes")


def _need_quantized(x, name, codes, sf, sf_layout, dev_status=None):
    """The reason why x [rows, cols] and its MXFP4 form are refused."""
    _need_2d(x, name)
    _need_rows_dtype(x, name)
    _need_mxfp4(codes, sf, *x.shape, sf_layout, "the")
    _need_status(dev_status)
    _need_one_device(x, codes, sf, dev_status)


def csa_mxfp4_quantize(x, codes, sf, *, sf_layout: int = CSA_SF_ROWS, dev_status=None,
                       stream=None):
    """Rows of x (bf16, fp16 or fp32 [rows, cols], any row stride) to packed e2m1 codes and
    UE8M0 scales in blocks of 32 (see include/csa.h)."""
    if _marshal is not None:
        status = _marshal.quantize(x, codes, sf, sf_layout, dev_status, _handle(stream))
        if status == 0:
            return
        if status is not None:
            _check(status)
    dev, dtype = x.get_device(), _DTYPES.get(x.dtype)
    if x.dim() != 2:
        _need_2d(x, "x")
    rows, cols = x.shape
    ld, step = x.stride()
    if not ((step == 1 or cols <= 1) and dtype is not None
            and _mxfp4_ok(codes, sf, rows, cols, sf_layout, dev)
            and (dev_status is None or _status_ok(dev_status, dev)) and _is_current(dev)):
        _need_quantized(x, "x", codes, sf, sf_layout, dev_status)
    status = _mx_quantize(x.data_ptr(), dtype, rows, cols, ld if rows > 1 else cols,
                          codes.data_ptr(), sf.data_ptr(), sf_layout,
                          None if dev_status is None else dev_status.data_ptr(),
                          _stream_on(stream, dev))
    if status:
        _check(status)


def csa_mxfp4_dequantize(codes, sf, out, *, sf_layout: int = CSA_SF_ROWS, stream=None):
    """The values MXFP4 rows stand for, into out (bf16, fp16 or fp32 [rows, cols])."""
    if _marshal is not None:
        status = _marshal.dequantize(codes, sf, out, sf_layout, _handle(stream))
        if status == 0:
            return
        if status is not None:
            _check(status)
    dev, dtype = out.get_device(), _DTYPES.get(out.dtype)
    if out.dim() != 2:
        _need_2d(out, "out")
    rows, cols = out.shape
    ld, step = out.stride()
    if not ((step == 1 or cols <= 1) and dtype is not None
            and _mxfp4_ok(codes, sf, rows, cols, sf_layout, dev) and _is_current(dev)):
        _need_quantized(out, "out", codes, sf, sf_layout)
    status = _mx_dequantize(codes.data_ptr(), sf.data_ptr(), sf_layout, rows, cols,
                            out.data_ptr(), dtype, ld if rows > 1 else cols,
                            _stream_on(stream, dev))
    if status:
        _check(status)


def csa_mxfp4_matmul(a, a_sf, b, b_sf, out, *, dev_status=None, stream=None):
    """out[m, n] = sum_k A[m, k] B[n, k] of packed MXFP4 a [M, K / 2] and b [N, K / 2] with
    tiled scales (CSA_SF_TILED), out bf16, fp16 or fp32 [M, N] (any row stride)."""
    if _marshal is not None:
        status = _marshal.matmul(a, a_sf, b, b_sf, out, dev_status, _handle(stream))
        if status == 0:
            return
        if status is not None:
            _check(status)
    dev, dtype = out.get_device(), _DTYPES.get(out.dtype)
    if out.dim() != 2:
        _need_2d(out, "out")
    M, N = out.shape
    ld, step = out.stride()
    K = 2 * a.shape[-1]
    if not ((step == 1 or N <= 1) and dtype is not None
            and _mxfp4_ok(a, a_sf, M, K, CSA_SF_TILED, dev)
            and _mxfp4_ok(b, b_sf, N, K, CSA_SF_TILED, dev)
            and (dev_status is None or _status_ok(dev_status, dev)) and _is_current(dev)):
        _need_2d(out, "out")
        _need_rows_dtype(out, "out")
        _need_mxfp4(a, a_sf, M, K, CSA_SF_TILED, "a's")
        _need_mxfp4(b, b_sf, N, K, CSA_SF_TILED, "b's")
        _need_status(dev_status)
        _need_one_device(a, a_sf, b, b_sf, out, dev_status)
    status = _mx_matmul(a.data_ptr(), a_sf.data_ptr(), b.data_ptr(), b_sf.data_ptr(), M, N, K,
                        out.data_ptr(), dtype, ld if M > 1 else N,
                        None if dev_status is None else dev_status.data_ptr(),
                        _stream_on(stream, dev))
    if status:
        _check(status)


def _need_heads(t, name, T, D):
    if t.dim() != 3 or t.shape[0] != T or t.shape[2] != D or (D > 1 and t.stride(2) != 1):
        _bad(f"{name} must be [{T}, heads, {D}] with contiguous channels, not {tuple(t.shape)} "
             f"with strides {t.stride()}")


_NO_HEADS = (None, 0, 0, 0, None, 0, 0)


def _head_args(x, out, dtype, T, D, dev):
    """(pointer, token stride, head stride, heads, output's pointer and strides) of head rows
    [T, heads, D] and their output, None where they do not fit.  A lone token's or head's
    stride is never used."""
    if x is None:
        return _NO_HEADS
    if out is None or x.dim() != 3:
        return None
    t, n, d = shape = x.shape
    if (t != T or d != D or out.shape != shape or x.dtype is not dtype or out.dtype is not dtype
            or x.get_device() != dev or out.get_device() != dev):
        return None
    st, sh, se = x.stride()
    ost, osh, ose = out.stride()
    if se != 1 or ose != 1:
        return None
    if T <= 1:
        st = ost = 0
    if n <= 1:
        sh = osh = 0
    return x.data_ptr(), st, sh, n, out.data_ptr(), ost, osh


def csa_qk_norm_rope(q, k, pos, q_out, k_out, *, q_weight=None, k_weight=None, norm: bool = True,
                     rope_dims: int = 64, rope_theta: float = 10000.0, eps: float = 1e-6,
                     stream=None):
    """RMSNorm of the query heads q [T, H, D] and key heads k [T, Hk, D] (either may be None)
    and rotation of their last rope_dims channels at pos (int32 [T]), in one launch.  An
    output may be its own input.  sparse_mqa_attn and dense_hca_attn rotate their queries
    themselves: rope_dims=0 makes their input, the default would have them rotated twice."""
    if _marshal is not None:
        status = _marshal.qk_norm_rope(q, k, pos, q_out, k_out, q_weight, k_weight, norm, rope_dims,
                                       rope_theta, eps, _handle(stream))
        if status == 0:
            return
        if status is not None:
            _check(status)
    lead = q if q is not None else k
    if lead is None:
        _bad("q and k are both None")
    dev, dtype = lead.get_device(), lead.dtype
    shape = lead.shape
    T, D = shape[0], shape[-1]
    qa = _head_args(q, q_out, dtype, T, D, dev)
    ka = _head_args(k, k_out, dtype, T, D, dev)
    if not (qa is not None and ka is not None and dtype in _DTYPES
            and _dense_ok(pos, _I32T, T, dev) and _weight_ok(q_weight, D, dev)
            and _weight_ok(k_weight, D, dev) and _is_current(dev)):
        _need_rows_dtype(lead, "q" if q is not None else "k")
        for x, out, name in ((q, q_out, "q"), (k, k_out, "k")):
            if x is None:
                continue
            _need_heads(x, name, T, D)
            if out is None or out.dim() != 3 or out.shape[1] != x.shape[1]:
                _bad("q_out and k_out must have the heads of q and k")
            _need_heads(out, f"{name}_out", T, D)
            if x.dtype != dtype or out.dtype != dtype:
                _bad("q, k and their outputs must have one element type")
        _need(pos, "pos", _I32T, (T,))
        for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if w is not None:
                _need(w, name, _F32T, (D,))
        _need_one_device(lead, k, pos, None if q is None else q_out, None if k is None else k_out,
                         q_weight, k_weight)
        _bad("q, k and their outputs must be contiguous along the channels")
    qp, q_st, q_sh, H, qo, qo_st, qo_sh = qa
    kp, k_st, k_sh, Hk, ko, ko_st, ko_sh = ka
    status = _qk_norm_rope(qp, q_st, q_sh, kp, k_st, k_sh, pos.data_ptr(), _ptr(q_weight),
                           _ptr(k_weight), qo, qo_st, qo_sh, ko, ko_st, ko_sh, _DTYPES[dtype], T,
                           H, Hk, D, rope_dims, 1 if norm else 0, rope_theta, eps,
                           _stream_on(stream, dev))
    if status:
        _check(status)


def _indexer_rows_ok(codes, scale, rows, D, fmt, dev):
    """The codes and scales of `rows` indexer rows."""
    if fmt == CSA_IDX_FP8:
        return _dense_ok(codes, _U8, rows * D, dev) and _dense_ok(scale, _F32T, rows, dev)
    return _dense_ok(codes, _U8, rows * (D // 2), dev) and \
        _dense_ok(scale, _U8, rows * (D // 32), dev)


def _need_indexer_rows(codes, scale, lead, D, fmt):
    if fmt == CSA_IDX_FP8:
        _need(codes, "codes", _U8, (*lead, D))
        _need(scale, "scale", _F32T, lead)
    else:
        _need(codes, "codes", _U8, (*lead, D // 2))
        _need(scale, "scale", _U8, (*lead, D // 32))


def csa_indexer_queries(q, q_pos, codes, scale, *, fmt: int = CSA_IDX_FP8, weight=None,
                        norm: bool = True, rope_dims: int = 64, rope_theta: float = 10000.0,
                        eps: float = 1e-6, dev_status=None, stream=None):
    """The indexer's query heads q [Q, H, D] normed, rotated at q_pos and quantised: codes and
    scale are lightning_indexer_topk's qI and qI_scale (fmt CSA_IDX_FP8) or
    lightning_indexer_topk_mxfp4's qI and qI_sf (CSA_IDX_MXFP4)."""
    if _marshal is not None:
        status = _marshal.queries(q, q_pos, codes, scale, fmt, weight, norm, rope_dims, rope_theta,
                                  eps, dev_status, _handle(stream))
        if status == 0:
            return
        if status is not None:
            _check(status)
    if q.dim() != 3:
        _bad(f"q must be [Q, H, D], not {tuple(q.shape)}")
    Q, H, D = q.shape
    st, sh, step = q.stride()
    dev, dtype = q.get_device(), _DTYPES.get(q.dtype)
    if not (dtype is not None and step == 1 and _dense_ok(q_pos, _I32T, Q, dev)
            and _indexer_rows_ok(codes, scale, Q * H, D, fmt, dev) and _weight_ok(weight, D, dev)
            and _status_ok(dev_status, dev) and _is_current(dev)):
        _need_rows_dtype(q, "q")
        _need_heads(q, "q", Q, D)
        _need(q_pos, "q_pos", _I32T, (Q,))
        _need_indexer_rows(codes, scale, (Q, H), D, fmt)
        if weight is not None:
            _need(weight, "weight", _F32T, (D,))
        _need_status(dev_status)
        _need_one_device(q, q_pos, codes, scale, weight, dev_status)
    status = _idx_queries(q.data_ptr(), dtype, st if Q > 1 else 0, sh if H > 1 else 0, q_pos.data_ptr(), _ptr(weight),
                          1 if norm else 0, rope_dims, rope_theta, eps, Q, H, D, fmt,
                          codes.data_ptr(), scale.data_ptr(), _ptr(dev_status),
                          _stream_on(stream, dev))
    if status:
        _check(status)


def csa_indexer_append(k, seq_len, ent_off, item_seq, item_ent, codes, scale, *, B: int,
                       m: int = 4, fmt: int = CSA_IDX_FP8, weight=None, norm: bool = True,
                       rope_dims: int = 64, rope_theta: float = 10000.0, eps: float = 1e-6,
                       layout=None, dev_status=None, stream=None):
    """Indexer keys k [n, D] of the listed entries normed, rotated at their block ends,
    quantised and written to their rows of the key store (codes, scale), through the layout's
    block table or ent_off.  A block table that is a slice of columns is copied first."""
    bt, ring = None, 0
    if layout is not None:
        bt, ring = getattr(layout, "_block_table", None), layout.kv_ring
    if _marshal is not None and (bt is not None or layout is None or not layout.block_table):
        status = _marshal.append(k, seq_len, ent_off, item_seq, item_ent, codes, scale, B, m, fmt,
                                 weight, norm, rope_dims, rope_theta, eps, bt, ring, dev_status,
                                 _handle(stream))
        if status == 0:
            return
        if status is not None:
            _check(status)
    if bt is not None and bt.dim() == 2:
        # The kernel takes the table's stride for its width.  Rows with a gap between them (a
        # slice of columns) are copied: an entry past the slice would find the next row's
        # blocks, or, behind the last row, what is no table at all.
        if B > 1 and bt.stride(0) != bt.shape[1]:
            with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
                bt = bt[:B].contiguous()
        layout = CacheLayout(bt.data_ptr(), bt.shape[1], ring)
    dev, dtype = k.get_device(), _DTYPES.get(k.dtype)
    if k.dim() != 2:
        _need_2d(k, "k")
    n, D = k.shape
    ld, step = k.stride()
    ent_rows = codes.shape[0]
    if not (dtype is not None and step == 1 and codes.dim() == 2
            and _indexer_rows_ok(codes, scale, ent_rows, D, fmt, dev)
            and _dense_ok(item_seq, _I32T, n, dev) and _dense_ok(item_ent, _I32T, n, dev)
            and _dense_ok(seq_len, _I64T, B, dev)
            and (ent_off is None or _dense_ok(ent_off, _I64T, B, dev))
            and (bt is None or (bt.dtype is _I32T and bt.dim() == 2 and bt.shape[0] >= B
                                and bt.stride()[1] == 1 and bt.get_device() == dev))
            and _weight_ok(weight, D, dev) and _status_ok(dev_status, dev) and _is_current(dev)):
        _need_2d(k, "k")
        _need_rows_dtype(k, "k")
        _need(item_seq, "item_seq", _I32T, (n,))
        _need(item_ent, "item_ent", _I32T, (n,))
        _need(seq_len, "seq_len", _I64T, (B,))
        if ent_off is not None:
            _need(ent_off, "ent_off", _I64T, (B,))
        if bt is not None and (bt.dtype != _I32T or bt.dim() != 2 or bt.shape[0] < B
                               or (bt.shape[1] > 1 and bt.stride(1) != 1)):
            _bad("the block table must be int32 [B, bt_stride] with contiguous rows")
        _need_indexer_rows(codes, scale, (codes.shape[0],), D, fmt)
        if weight is not None:
            _need(weight, "weight", _F32T, (D,))
        _need_status(dev_status)
        _need_one_device(k, seq_len, ent_off, item_seq, item_ent, codes, scale, weight, bt,
                         dev_status)
    status = _idx_append(k.data_ptr(), dtype, ld if n > 1 else D,
                         seq_len.data_ptr(), _ptr(ent_off), item_seq.data_ptr(),
                         item_ent.data_ptr(), n, B, m, _ptr(weight), 1 if norm else 0, rope_dims,
                         rope_theta, eps, D, fmt, codes.data_ptr(), scale.data_ptr(),
                         ent_rows, _lay(layout), _ptr(dev_status),
                         _stream_on(stream, dev))
    if status:
        _check(status)
