// MXFP4 quantisation and its inverse ("DeepSeek-V4 深度分析报告" 3.4: MXFP4 on the QK path of
// CSA, FP4 weights; Figure 2, "Lightning Indexer FP4").
//
// A block is 32 consecutive elements of a row.  With amax its largest magnitude, the scale is
// 2^e, e = floor(log2(amax)) - 2 (2 = the exponent of e2m1's largest binade), stored as the
// byte e + 127 (clamped at 0); every element becomes the e2m1 value nearest to x / 2^e (ties
// to the even code, past 6 to 6).  The division is a multiplication by a power of two and so
// exact: the codes are those of the definition bit for bit, whatever the batch.
//
// Both kernels are bound by HBM.  A lane takes 8 consecutive elements (16 bytes of bf16, one
// 4-byte word of codes) and four lanes a block (its amax takes two shuffles); a warp takes 256
// elements of one row, or as many rows of fewer as fit.  Warps are persistent and work
// on kItems such pieces at once, whose loads go out together: one fence per warp instead of one per
// piece, one division per task.  An 8192 x 2048 fp32 weight quantised (76 MB) and read back as
// bf16 (42 MB): 23 us in all, 5.1 TB/s; 524288 rows of 128 read back as bf16 (170 MB): 28 us,
// 6.0 TB/s.
#include <type_traits>

#include "launchers.cuh"
#include "rows.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;

// Where the scale bytes lie: rows x blocks row-major, or tiles of 128 rows x 4 blocks of 512
// bytes (the tensor cores' layout: row r, block j of a tile at 16 (r mod 32) + 4 (r div 32)
// + j; tiles along the blocks first).
struct ScaleMap {
    int tiled;
    int64_t nblk;      // blocks per row
    int64_t ktiles;    // ceil(nblk / 4)
    __device__ __forceinline__ int64_t at(int64_t r, int64_t j) const {
        if (!tiled) return r * nblk + j;
        return ((r >> 7) * ktiles + (j >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (j & 3);
    }
    // from row r, block j to row r + dr, block j + dj (dj a multiple of 4; in the tiled layout both
    // rows lie in one group of 32)
    __device__ __forceinline__ int64_t step(int dr, uint32_t dj) const {
        return tiled ? dr * 16 + (int64_t)(dj >> 2) * 512 : dr * nblk + dj;
    }
};

// How a [rows, units] matrix of 8-element units is cut for warps.  A piece is 32 units: 2^lanes
// lanes to a row (32 at most), 32 >> lanes rows.  A task is kItems pieces: along a row where a row
// has that many, else down the rows; one division per task, and piece i of it lies at fixed
// strides from piece 0.
struct Tasks {
    int64_t rows;            // rows walked (the tiled layout's padding included)
    uint32_t units;          // units of a row, likewise
    uint32_t n, per_row;     // tasks, and how many a row (or group of rows) is cut into
    uint32_t mul;            // ceil(2^32 / per_row), 0 for 1
    int lanes, along;        // along: pieces of a task follow one another along the row
    __device__ __forceinline__ int row_step() const { return along ? 0 : 32 >> lanes; }
    __device__ __forceinline__ uint32_t unit_step() const { return along ? 32u : 0u; }
    // the row and unit of this lane in piece 0 of task i
    __device__ __forceinline__ void at(uint32_t i, int lane, int64_t& row, uint32_t& unit) const {
        uint32_t g = i, k = 0;
        if (per_row > 1) {
            g = __umulhi(i, mul);
            k = i - g * per_row;
            if ((int32_t)k < 0) {            // the rounded-up reciprocal may be one too far
                g--;
                k += per_row;
            }
        }
        unit = ((k * (along ? kItems : 1)) << lanes) + (lane & ((1 << lanes) - 1));
        row = (int64_t)g * ((32 >> lanes) * (along ? 1 : kItems)) + (lane >> lanes);
    }
};

Tasks make_tasks(int64_t rows_u, int64_t units_u) {
    Tasks t;
    t.rows = rows_u;
    t.units = (uint32_t)units_u;
    t.lanes = 2;
    while (t.lanes < 5 && (1 << t.lanes) < units_u) t.lanes++;
    const int64_t chunks = (units_u + (1 << t.lanes) - 1) >> t.lanes;
    t.along = chunks >= kItems;
    t.per_row = (uint32_t)(t.along ? (chunks + kItems - 1) / kItems : chunks);
    const int64_t rows_per = (32 >> t.lanes) * (t.along ? 1 : kItems);
    t.n = (uint32_t)((rows_u + rows_per - 1) / rows_per * t.per_row);
    t.mul = t.per_row > 1 ? (uint32_t)((((uint64_t)1 << 32) + t.per_row - 1) / t.per_row) : 0;
    return t;
}

// The magnitude bits of the largest of 8 elements as fp32 (a NaN above an infinity above the rest).
__device__ __forceinline__ uint32_t top_bits(const Row8<float>& v) {
    float f[8];
    v.get(f);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
    return top;
}
template <class T>
__device__ __forceinline__ uint32_t top_bits(const Row8<T>& v) {
    // 16-bit magnitudes compare as integers, two at a time
    uint32_t m = __vmaxu2(__vmaxu2(v.r.x & 0x7fff7fffu, v.r.y & 0x7fff7fffu),
                          __vmaxu2(v.r.z & 0x7fff7fffu, v.r.w & 0x7fff7fffu));
    m = max(m & 0xffffu, m >> 16);
    if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value)
        return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
    return m << 16;
}

// A task's strides from piece to piece: elements of the rows, words of the codes, scale bytes.
struct Steps {
    int64_t row_elems, code_words, scales;
};

// One task of the quantiser; kFull: all its pieces lie inside the matrix.
template <class T, bool kFull>
__device__ __forceinline__ void quantize_task(const T* src, uint32_t* dst, uint8_t* sfp, const Steps& step, int lane,
                                              int rstep, uint32_t ustep, int rows_left, uint32_t units_left,
                                              int pad_rows_left, uint32_t pad_units_left, int32_t* st) {
    Row8<T> v[kItems];
#pragma unroll
    for (int i = 0; i < kItems; i++) {
        if (kFull || (i * rstep < rows_left && i * ustep < units_left)) {
            v[i].load(src);
        } else {
            v[i].zero();
        }
        src += step.row_elems;
    }
#pragma unroll
    for (int i = 0; i < kItems; i++) {
        uint32_t top = top_bits(v[i]);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        uint32_t e = max(top >> 23, 2u) - 2u;
        const bool bad = e == 253u;                  // an infinity or a NaN in the block
        const float inv = __uint_as_float((254u - e) << 23);   // 2^(127 - e)
        const float inv2[2] = {inv, inv};
        float f[8];
        v[i].get(f);
#pragma unroll
        for (int j = 0; j < 8; j += 2) mul2(f + j, f + j, inv2);
        uint32_t c = pack_e2m1x8(f);
        if (bad) {
            c = 0u;
            e = 255u;
        }
        if (kFull || (i * rstep < rows_left && i * ustep < units_left)) *dst = c;
        if ((lane & 3) == 0 && (kFull || (i * rstep < pad_rows_left && i * ustep < pad_units_left))) {
            *sfp = (uint8_t)e;
            if (bad) flag(st, CSA_DEV_NAN);
        }
        dst += step.code_words;
        sfp += step.scales;
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) mxfp4_quantize_kernel(
    const T* __restrict__ x, int64_t rows, uint32_t units, int64_t ld, const Tasks tk,
    uint32_t* __restrict__ codes, uint8_t* __restrict__ sf, const ScaleMap sm, int32_t* __restrict__ st) {
    pdl_wait();
    // Rows in the tiled layout are read by the product and the inverse alone, which wait for this
    // grid before they read anything: the next kernel may start.  Rows in the indexer's layout
    // may be read ahead of that wait, so it may not.
    if (sm.tiled) pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int rstep = tk.row_step();
    const uint32_t ustep = tk.unit_step();
    const Steps step{rstep * ld + ustep * 8, (int64_t)rstep * units + ustep, sm.step(rstep, ustep >> 2)};
    for (uint32_t i0 = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i0 < tk.n;
         i0 += gridDim.x * (kThreads / 32)) {
        int64_t row;
        uint32_t unit;
        tk.at(i0, lane, row, unit);
        // what is left from here, at most a task's worth; past the end nothing is
        const int rows_left = (int)max(min(rows - row, (int64_t)64), (int64_t)0);
        const int pad_rows_left = (int)max(min(tk.rows - row, (int64_t)64), (int64_t)0);
        const uint32_t units_left = unit < units ? units - unit : 0u;
        const uint32_t pad_units_left = unit < tk.units ? tk.units - unit : 0u;
        const T* src = x + row * ld + unit * 8;
        uint32_t* dst = codes + row * units + unit;
        uint8_t* sfp = sf + sm.at(row, unit >> 2);
        const bool full = (kItems - 1) * rstep < rows_left && (kItems - 1) * ustep < units_left;
        if (__all_sync(0xffffffffu, full))
            quantize_task<T, true>(src, dst, sfp, step, lane, rstep, ustep, 0, 0, 0, 0, st);
        else
            quantize_task<T, false>(src, dst, sfp, step, lane, rstep, ustep, rows_left, units_left, pad_rows_left,
                                    pad_units_left, st);
    }
    __threadfence();   // visible before the next kernel's reads ahead of its own wait
}

template <class T, bool kFull>
__device__ __forceinline__ void dequantize_task(const uint32_t* src, const uint8_t* sfp, T* dst, const Steps& step,
                                                int rstep, uint32_t ustep, int rows_left, uint32_t units_left) {
    uint32_t c[kItems], e[kItems];
#pragma unroll
    for (int i = 0; i < kItems; i++) {
        c[i] = e[i] = 0;
        if (kFull || (i * rstep < rows_left && i * ustep < units_left)) {
            c[i] = *src;
            e[i] = *sfp;
        }
        src += step.code_words;
        sfp += step.scales;
    }
#pragma unroll
    for (int i = 0; i < kItems; i++) {
        // 2^(e - 127): the byte is the exponent field, 0 the subnormal 2^-127, 255 a NaN
        const float s = __uint_as_float(e[i] == 0 ? 0x00400000u : e[i] == 255u ? 0x7fffffffu : e[i] << 23);
        const float s2[2] = {s, s};
        float f[8];
        unpack_e2m1x8(c[i], f);
#pragma unroll
        for (int j = 0; j < 8; j += 2) mul2(f + j, f + j, s2);
        Row8<T> v;
        v.set(f);
        if (kFull || (i * rstep < rows_left && i * ustep < units_left)) v.store(dst);
        dst += step.row_elems;
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) mxfp4_dequantize_kernel(
    const uint32_t* __restrict__ codes, const uint8_t* __restrict__ sf, const ScaleMap sm, const Tasks tk,
    T* __restrict__ out, int64_t ld) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int rstep = tk.row_step();
    const uint32_t ustep = tk.unit_step();
    const Steps step{rstep * ld + ustep * 8, (int64_t)rstep * tk.units + ustep, sm.step(rstep, ustep >> 2)};
    for (uint32_t i0 = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i0 < tk.n;
         i0 += gridDim.x * (kThreads / 32)) {
        int64_t row;
        uint32_t unit;
        tk.at(i0, lane, row, unit);
        const int rows_left = (int)max(min(tk.rows - row, (int64_t)64), (int64_t)0);
        const uint32_t units_left = unit < tk.units ? tk.units - unit : 0u;
        const uint32_t* src = codes + row * tk.units + unit;
        const uint8_t* sfp = sf + sm.at(row, unit >> 2);
        T* dst = out + row * ld + unit * 8;
        const bool full = (kItems - 1) * rstep < rows_left && (kItems - 1) * ustep < units_left;
        if (__all_sync(0xffffffffu, full))
            dequantize_task<T, true>(src, sfp, dst, step, rstep, ustep, 0, 0);
        else
            dequantize_task<T, false>(src, sfp, dst, step, rstep, ustep, rows_left, units_left);
    }
    __threadfence();
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

// As many CTAs as are resident, or fewer where the tasks do not fill them.
dim3 grid_of(const Tasks& t, int per_sm) {
    const int64_t need = ((int64_t)t.n + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t most = (int64_t)sm_count() * per_sm;
    return dim3((unsigned)(need < most ? need : most));
}

template <class T>
cudaError_t quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                     uint8_t* sf, int tiled, int32_t* st, cudaStream_t stream) {
    const int64_t ktiles = (cols + 127) / 128;
    const Tasks p = make_tasks(tiled ? (rows + 127) / 128 * 128 : rows, tiled ? ktiles * 16 : cols / 8);
    LaunchScope scope(kKMxQuant, stream);
    return launch_pdl(mxfp4_quantize_kernel<T>, grid_of(p, 4), dim3(kThreads), 0, stream, (const T*)x, rows,
                      (uint32_t)(cols / 8), ld, p, (uint32_t*)codes, sf, ScaleMap{tiled, cols / 32, ktiles}, st);
}

template <class T>
cudaError_t dequantize(const uint8_t* codes, const uint8_t* sf, int tiled, int64_t rows,
                       int64_t cols, void* out, int64_t ld, cudaStream_t stream) {
    const Tasks p = make_tasks(rows, cols / 8);
    LaunchScope scope(kKMxDequant, stream);
    return launch_pdl(mxfp4_dequantize_kernel<T>, grid_of(p, 6), dim3(kThreads), 0, stream,
                      (const uint32_t*)codes, sf, ScaleMap{tiled, cols / 32, (cols + 127) / 128}, p, (T*)out, ld);
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld,
                                  uint8_t* codes, uint8_t* sf, int tiled, int32_t* st,
                                  cudaStream_t stream) {
    switch (dtype) {
        case CSA_DT_BF16: return quantize<__nv_bfloat16>(x, rows, cols, ld, codes, sf, tiled, st, stream);
        case CSA_DT_F16: return quantize<__half>(x, rows, cols, ld, codes, sf, tiled, st, stream);
        default: return quantize<float>(x, rows, cols, ld, codes, sf, tiled, st, stream);
    }
}

cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* sf, int tiled,
                                    int64_t rows, int64_t cols, void* out, int dtype, int64_t ld,
                                    cudaStream_t stream) {
    switch (dtype) {
        case CSA_DT_BF16: return dequantize<__nv_bfloat16>(codes, sf, tiled, rows, cols, out, ld, stream);
        case CSA_DT_F16: return dequantize<__half>(codes, sf, tiled, rows, cols, out, ld, stream);
        default: return dequantize<float>(codes, sf, tiled, rows, cols, out, ld, stream);
    }
}

}  // namespace csa
