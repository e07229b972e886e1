// Argument marshalling of the calls that make the lightning indexer's inputs, compiled: decode steps
// issue many small launches, and through ctypes the tests of the tensors and the conversion of
// up to 25 arguments took 3 to 7 us of host time per call against 2.3 for the launch itself.
//
// Each function takes the Python call's arguments in order, tests every tensor (type, size,
// contiguity, device) and calls the C entry point on the given or the current stream.  It returns
// the entry point's status, or None if a test failed: the Python side then finds the reason
// and raises.  Nothing here computes, allocates device memory or synchronises.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/csa.h"

namespace {

decltype(&csa_mxfp4_quantize) f_quantize;
decltype(&csa_mxfp4_dequantize) f_dequantize;
decltype(&csa_mxfp4_matmul) f_matmul;
decltype(&csa_qk_norm_rope) f_qk_norm_rope;
decltype(&csa_indexer_queries) f_queries;
decltype(&csa_indexer_append) f_append;

// The arguments of one call; `ok` turns false at the first one that does not fit.
struct Args {
    PyObject* const* a;
    bool ok = true;

    const at::Tensor* tensor(int i) {
        if (ok && THPVariable_Check(a[i])) return &THPVariable_Unpack(a[i]);
        ok = false;
        return nullptr;
    }
    bool none(int i) const { return a[i] == Py_None; }
    int64_t integer(int i) {
        if (!ok) return 0;
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }
    int32_t int32(int i) {
        const int64_t v = integer(i);
        if (v != (int32_t)v) ok = false;
        return (int32_t)v;
    }
    float real(int i) {
        if (!ok) return 0.f;
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return (float)v;
    }
    void need(bool cond) { ok = ok && cond; }
    int32_t truth(int i) {
        const int t = PyObject_IsTrue(a[i]);
        if (t < 0) {
            PyErr_Clear();
            ok = false;
        }
        return t > 0;
    }
    // n contiguous elements of a type on a device
    void* dense(int i, at::ScalarType type, int64_t n, int dev) {
        const at::Tensor* t = tensor(i);
        if (!t) return nullptr;
        need(t->scalar_type() == type && t->numel() == n && t->is_contiguous() && t->get_device() == dev);
        return ok ? t->data_ptr() : nullptr;
    }
    void* dense_or_none(int i, at::ScalarType type, int64_t n, int dev) {
        return none(i) ? nullptr : dense(i, type, n, dev);
    }
    int32_t* status(int i, int dev) {
        if (none(i)) return nullptr;
        const at::Tensor* t = tensor(i);
        if (!t) return nullptr;
        need(t->scalar_type() == at::kInt && t->numel() >= 1 && t->get_device() == dev);
        return ok ? static_cast<int32_t*>(t->data_ptr()) : nullptr;
    }
    // the stream: a handle, or None for the device's current one; the device has to be current
    void* stream(int i, int dev) {
        if (!ok) return nullptr;
        need(dev >= 0 && dev == c10::cuda::current_device());
        if (!ok) return nullptr;
        if (none(i)) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
        return reinterpret_cast<void*>(integer(i));
    }
};

int dtype_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return CSA_DT_BF16;
        case at::kHalf: return CSA_DT_F16;
        case at::kFloat: return CSA_DT_F32;
        default: return -1;
    }
}

PyObject* result(const Args& x, int status) {
    if (x.ok) return PyLong_FromLong(status);
    Py_RETURN_NONE;
}

// A 2-D tensor's rows: contiguous along a row, any stride between them.
struct Rows {
    void* p = nullptr;
    int64_t rows = 0, cols = 0, ld = 0;
    int dtype = -1, dev = -1;
    Rows(Args& x, int i) {
        const at::Tensor* t = x.tensor(i);
        if (!t) return;
        x.need(t->dim() == 2);
        if (!x.ok) return;
        dtype = dtype_of(*t);
        dev = (int)t->get_device();
        rows = t->size(0);
        cols = t->size(1);
        ld = rows > 1 ? t->stride(0) : cols;
        x.need(dtype >= 0 && (t->stride(1) == 1 || cols <= 1));
        if (x.ok) p = t->data_ptr();
    }
};

// Packed codes [rows, cols / 2] and their scale bytes.
void mxfp4(Args& x, int codes, int sf, int64_t rows, int64_t cols, int layout, int dev, uint8_t*& pc, uint8_t*& ps) {
    const int64_t need = layout ? (rows + 127) / 128 * ((cols + 127) / 128) * 512 : rows * (cols / 32);
    pc = static_cast<uint8_t*>(x.dense(codes, at::kByte, rows * (cols / 2), dev));
    const at::Tensor* t = x.tensor(sf);
    if (!t) return;
    x.need(t->scalar_type() == at::kByte && t->numel() >= need && t->is_contiguous() && t->get_device() == dev);
    if (x.ok) ps = static_cast<uint8_t*>(t->data_ptr());
}

// [T, heads, D] rows and their output; a lone token's or head's stride is never used.
struct Heads {
    void *p = nullptr, *out = nullptr;
    int64_t st = 0, sh = 0, ost = 0, osh = 0, heads = 0;
    Heads(Args& x, int i, int o, at::ScalarType type, int64_t T, int64_t D, int dev) {
        if (x.none(i)) return;
        const at::Tensor *a = x.tensor(i), *b = x.tensor(o);
        if (!a || !b) return;
        x.need(a->dim() == 3 && b->dim() == 3 && a->sizes() == b->sizes() && a->size(0) == T && a->size(2) == D &&
               a->scalar_type() == type && b->scalar_type() == type && a->get_device() == dev &&
               b->get_device() == dev && a->stride(2) == 1 && b->stride(2) == 1);
        if (!x.ok) return;
        heads = a->size(1);
        if (T > 1) {
            st = a->stride(0);
            ost = b->stride(0);
        }
        if (heads > 1) {
            sh = a->stride(1);
            osh = b->stride(1);
        }
        p = a->data_ptr();
        out = b->data_ptr();
    }
};

// The call itself, without the interpreter's lock: a launch may wait for room in the queue.
template <class F>
int unlocked(const Args& x, F call) {
    if (!x.ok) return 0;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = (int)call();
    Py_END_ALLOW_THREADS
    return status;
}

#define CSA_ARGS(count) \
    if (n != (count)) Py_RETURN_NONE; \
    Args x{a}

// x, codes, sf, sf_layout, dev_status, stream
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    CSA_ARGS(6);
    const Rows r(x, 0);
    const int32_t layout = x.int32(3);
    uint8_t *codes = nullptr, *sf = nullptr;
    mxfp4(x, 1, 2, r.rows, r.cols, layout, r.dev, codes, sf);
    int32_t* st = x.status(4, r.dev);
    void* s = x.stream(5, r.dev);
    return result(x, unlocked(x, [&] {
        return f_quantize(r.p, r.dtype, r.rows, r.cols, r.ld, codes, sf, layout, st, s);
    }));
}

// codes, sf, out, sf_layout, stream
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    CSA_ARGS(5);
    const Rows r(x, 2);
    const int32_t layout = x.int32(3);
    uint8_t *codes = nullptr, *sf = nullptr;
    mxfp4(x, 0, 1, r.rows, r.cols, layout, r.dev, codes, sf);
    void* s = x.stream(4, r.dev);
    return result(x, unlocked(x, [&] {
        return f_dequantize(codes, sf, layout, r.rows, r.cols, r.p, r.dtype, r.ld, s);
    }));
}

// a, a_sf, b, b_sf, out, dev_status, stream
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
    CSA_ARGS(7);
    const Rows r(x, 4);
    const at::Tensor* ta = x.tensor(0);
    x.need(ta && ta->dim() >= 1);
    const int64_t K = x.ok ? 2 * ta->size(-1) : 0;
    uint8_t *pa = nullptr, *sa = nullptr, *pb = nullptr, *sb = nullptr;
    mxfp4(x, 0, 1, r.rows, K, CSA_SF_TILED, r.dev, pa, sa);
    mxfp4(x, 2, 3, r.cols, K, CSA_SF_TILED, r.dev, pb, sb);
    int32_t* st = x.status(5, r.dev);
    void* s = x.stream(6, r.dev);
    return result(x, unlocked(x, [&] {
        return f_matmul(pa, sa, pb, sb, r.rows, r.cols, K, r.p, r.dtype, r.ld, st, s);
    }));
}

// q, k, pos, q_out, k_out, q_weight, k_weight, norm, rope_dims, rope_theta, eps, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    CSA_ARGS(12);
    const at::Tensor* lead = x.tensor(x.none(0) ? 1 : 0);
    x.need(lead && lead->dim() == 3 && dtype_of(*lead) >= 0);
    if (!x.ok) Py_RETURN_NONE;
    const int dev = (int)lead->get_device();
    const int64_t T = lead->size(0), D = lead->size(2);
    const Heads q(x, 0, 3, lead->scalar_type(), T, D, dev), k(x, 1, 4, lead->scalar_type(), T, D, dev);
    const void* pos = x.dense(2, at::kInt, T, dev);
    const void* qw = x.dense_or_none(5, at::kFloat, D, dev);
    const void* kw = x.dense_or_none(6, at::kFloat, D, dev);
    const int32_t norm = x.truth(7), rope = x.int32(8);
    const float theta = x.real(9), eps = x.real(10);
    x.need(T <= INT32_MAX && q.heads <= INT32_MAX && k.heads <= INT32_MAX && D <= INT32_MAX);
    void* s = x.stream(11, dev);
    const int dtype = dtype_of(*lead);
    return result(x, unlocked(x, [&] {
        return f_qk_norm_rope(q.p, q.st, q.sh, k.p, k.st, k.sh, (const int32_t*)pos, (const float*)qw,
                              (const float*)kw, q.out, q.ost, q.osh, k.out, k.ost, k.osh, dtype, (int32_t)T,
                              (int32_t)q.heads, (int32_t)k.heads, (int32_t)D, rope, norm, theta, eps, s);
    }));
}

// The codes and scales of `rows` indexer rows.
void indexer_rows(Args& x, int codes, int scale, int64_t rows, int64_t D, int32_t fmt, int dev, uint8_t*& pc,
                  void*& ps) {
    if (fmt == CSA_IDX_FP8) {
        pc = static_cast<uint8_t*>(x.dense(codes, at::kByte, rows * D, dev));
        ps = x.dense(scale, at::kFloat, rows, dev);
    } else {
        pc = static_cast<uint8_t*>(x.dense(codes, at::kByte, rows * (D / 2), dev));
        ps = x.dense(scale, at::kByte, rows * (D / 32), dev);
    }
}

// q, q_pos, codes, scale, fmt, weight, norm, rope_dims, rope_theta, eps, dev_status, stream
PyObject* queries(PyObject*, PyObject* const* a, Py_ssize_t n) {
    CSA_ARGS(12);
    const at::Tensor* q = x.tensor(0);
    x.need(q && q->dim() == 3 && dtype_of(*q) >= 0);
    if (!x.ok) Py_RETURN_NONE;
    const int dev = (int)q->get_device();
    const int64_t Q = q->size(0), H = q->size(1), D = q->size(2);
    x.need(q->stride(2) == 1 && Q <= INT32_MAX && H <= INT32_MAX && D <= INT32_MAX);
    const void* pos = x.dense(1, at::kInt, Q, dev);
    const int32_t fmt = x.int32(4);
    uint8_t* codes = nullptr;
    void* scale = nullptr;
    indexer_rows(x, 2, 3, Q * H, D, fmt, dev, codes, scale);
    const void* w = x.dense_or_none(5, at::kFloat, D, dev);
    const int32_t norm = x.truth(6), rope = x.int32(7);
    const float theta = x.real(8), eps = x.real(9);
    int32_t* st = x.status(10, dev);
    void* s = x.stream(11, dev);
    const void* qp = q->data_ptr();
    const int dtype = dtype_of(*q);
    const int64_t q_st = Q > 1 ? q->stride(0) : 0, q_sh = H > 1 ? q->stride(1) : 0;
    return result(x, unlocked(x, [&] {
        return f_queries(qp, dtype, q_st, q_sh, (const int32_t*)pos, (const float*)w, norm, rope, theta, eps,
                         (int32_t)Q, (int32_t)H, (int32_t)D, fmt, codes, scale, st, s);
    }));
}

// k, seq_len, ent_off, item_seq, item_ent, codes, scale, B, m, fmt, weight, norm, rope_dims,
// rope_theta, eps, block_table, kv_ring, dev_status, stream
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    CSA_ARGS(19);
    const Rows k(x, 0);
    const at::Tensor* c = x.tensor(5);
    x.need(c && c->dim() == 2);
    if (!x.ok) Py_RETURN_NONE;
    const int64_t ent_rows = c->size(0);
    const int32_t B = x.int32(7), m = x.int32(8), fmt = x.int32(9);
    const void* seq_len = x.dense(1, at::kLong, B, k.dev);
    const void* ent_off = x.dense_or_none(2, at::kLong, B, k.dev);
    const void* seq = x.dense(3, at::kInt, k.rows, k.dev);
    const void* ent = x.dense(4, at::kInt, k.rows, k.dev);
    uint8_t* codes = nullptr;
    void* scale = nullptr;
    indexer_rows(x, 5, 6, ent_rows, k.cols, fmt, k.dev, codes, scale);
    const void* w = x.dense_or_none(10, at::kFloat, k.cols, k.dev);
    const int32_t norm = x.truth(11), rope = x.int32(12);
    const float theta = x.real(13), eps = x.real(14);
    csa_cache_layout_t layout = {nullptr, 0, x.integer(16)};
    if (!x.none(15)) {
        const at::Tensor* bt = x.tensor(15);
        // the kernel takes the stride for a row's width: rows with a gap go to the Python side
        x.need(bt && bt->scalar_type() == at::kInt && bt->dim() == 2 && bt->size(0) >= B &&
               (bt->stride(1) == 1 || bt->size(1) <= 1) && (bt->stride(0) == bt->size(1) || B == 1) &&
               bt->get_device() == k.dev);
        if (!x.ok) Py_RETURN_NONE;
        layout.block_table = static_cast<const int32_t*>(bt->data_ptr());
        layout.bt_stride = bt->size(1);
    }
    x.need(k.cols <= INT32_MAX);
    int32_t* st = x.status(17, k.dev);
    void* s = x.stream(18, k.dev);
    return result(x, unlocked(x, [&] {
        return f_append(k.p, k.dtype, k.ld, (const int64_t*)seq_len, (const int64_t*)ent_off, (const int32_t*)seq,
                        (const int32_t*)ent, k.rows, B, m, (const float*)w, norm, rope, theta, eps, (int32_t)k.cols,
                        fmt, codes, scale, ent_rows, layout.block_table || layout.kv_ring ? &layout : nullptr, st,
                        s);
    }));
}

// The entry points' addresses, in the order of the pointers above.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
        return nullptr;
    }
    void* p[6];
    for (int i = 0; i < 6; i++) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    f_quantize = reinterpret_cast<decltype(f_quantize)>(p[0]);
    f_dequantize = reinterpret_cast<decltype(f_dequantize)>(p[1]);
    f_matmul = reinterpret_cast<decltype(f_matmul)>(p[2]);
    f_qk_norm_rope = reinterpret_cast<decltype(f_qk_norm_rope)>(p[3]);
    f_queries = reinterpret_cast<decltype(f_queries)>(p[4]);
    f_append = reinterpret_cast<decltype(f_append)>(p[5]);
    Py_RETURN_NONE;
}

// No C++ exception passes into the interpreter (torch's accessors may throw): it reads as a failed
// test, for which the Python side raises.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

#define CSA_METHOD(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
    CSA_METHOD(quantize), CSA_METHOD(dequantize), CSA_METHOD(matmul), CSA_METHOD(qk_norm_rope),
    CSA_METHOD(queries), CSA_METHOD(append), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_csa_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// CSA_TORCH, CSA_PYTHON: the versions compiled against, whose tensors' layout is compiled in.  The
// package takes the module under these alone.
PyMODINIT_FUNC PyInit__csa_marshal(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && (PyModule_AddStringConstant(m, "torch_version", CSA_TORCH) ||
              PyModule_AddStringConstant(m, "python_tag", CSA_PYTHON))) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
