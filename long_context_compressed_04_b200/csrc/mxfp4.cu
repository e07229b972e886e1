// MXFP4 quantisation and its inverse ("DeepSeek-V4 深度分析报告" 3.4: MXFP4 on the QK path of
// CSA, FP4 weights; Figure 2, "Lightning Indexer FP4").
//
// A block is 32 consecutive elements of a row.  With amax its largest magnitude, the scale is
// 2^e, e = floor(log2(amax)) - 2 (2 = the exponent of e2m1's largest binade), stored as the
// byte e + 127 (clamped at 0); every element becomes the e2m1 value nearest to x / 2^e (ties
// to the even code, past 6 to 6).  The division is a multiplication by a power of two and so
// exact: the codes are those of the definition bit for bit, whatever the batch.
//
// Both kernels are bound by HBM: a thread takes 8 consecutive elements (16 bytes of bf16, one
// 4-byte word of codes), so a warp's loads and stores are contiguous, and four lanes share a
// block (its amax takes two shuffles).  kUnits independent groups of 8 per thread keep
// enough bytes in flight.
#include "launchers.cuh"
#include "rows.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;

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
};

// u / d for u * d < 2^64, by a multiplication with ceil(2^64 / d); d = 1 apart.
struct FastDiv {
    uint64_t mul;
    uint32_t d;
    __device__ __forceinline__ uint64_t div(uint64_t u) const { return d == 1 ? u : __umul64hi(u, mul); }
};
FastDiv fast_div(uint32_t d) { return {d == 1 ? 0 : ~0ull / d + 1, d}; }

// Units of 8 elements over the grid of rows_u x units_u; the units past rows x cols are those
// of the tiled layout's padding, which only write a zero scale.
template <class T>
__global__ void __launch_bounds__(kThreads) mxfp4_quantize_kernel(
    const T* __restrict__ x, int64_t rows, int64_t cols, int64_t ld, int64_t n_units,
    FastDiv units_per_row, uint32_t* __restrict__ codes, uint8_t* __restrict__ sf, ScaleMap sm,
    int32_t* __restrict__ st) {
    pdl_wait();
    const int64_t u0 = (int64_t)blockIdx.x * (kThreads * kUnits) + threadIdx.x;
    Row8<T> v[kUnits];
    int64_t row[kUnits], unit[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; i++) {
        const int64_t u = u0 + (int64_t)i * kThreads;
        row[i] = (int64_t)units_per_row.div((uint64_t)u);
        unit[i] = u - row[i] * units_per_row.d;
        v[i].zero();
        if (row[i] < rows && unit[i] * 8 < cols) v[i].load(x + row[i] * ld + unit[i] * 8);
    }
#pragma unroll
    for (int i = 0; i < kUnits; i++) {
        float f[8];
        v[i].get(f);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; j++) top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int64_t u = u0 + (int64_t)i * kThreads;
        if (u >= n_units) continue;
        const uint32_t ex = top >> 23;
        const bool bad = ex == 255u;               // an infinity or a NaN in the block
        const uint32_t e = bad ? 255u : ex > 2u ? ex - 2u : 0u;
        const float inv = __uint_as_float((254u - (bad ? 127u : e)) << 23);   // 2^(127 - e)
        const bool in = row[i] < rows && unit[i] * 8 < cols;
        if (in) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; j++) y[j] = f[j] * inv;
            codes[row[i] * (cols >> 3) + unit[i]] = bad ? 0u : pack_e2m1x8(y);
        }
        if ((unit[i] & 3) == 0) {
            sf[sm.at(row[i], unit[i] >> 2)] = (uint8_t)e;
            if (bad) flag(st, CSA_DEV_NAN);
        }
    }
    __threadfence();   // visible before the next kernel's reads ahead of its own wait
}

template <class T>
__global__ void __launch_bounds__(kThreads) mxfp4_dequantize_kernel(
    const uint32_t* __restrict__ codes, const uint8_t* __restrict__ sf, ScaleMap sm, int64_t n_units,
    FastDiv units_per_row, T* __restrict__ out, int64_t ld) {
    pdl_wait();
    const int64_t u0 = (int64_t)blockIdx.x * (kThreads * kUnits) + threadIdx.x;
    uint32_t c[kUnits], e[kUnits];
    int64_t row[kUnits], unit[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; i++) {
        const int64_t u = u0 + (int64_t)i * kThreads;
        row[i] = (int64_t)units_per_row.div((uint64_t)u);
        unit[i] = u - row[i] * units_per_row.d;
        c[i] = e[i] = 0;
        if (u < n_units) {
            c[i] = codes[u];
            e[i] = sf[sm.at(row[i], unit[i] >> 2)];
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; i++) {
        if (u0 + (int64_t)i * kThreads >= n_units) continue;
        // 2^(e - 127): the byte is the exponent field, 0 the subnormal 2^-127, 255 a NaN
        const float s = __uint_as_float(e[i] == 0 ? 0x00400000u : e[i] == 255u ? 0x7fffffffu : e[i] << 23);
        float f[8];
        unpack_e2m1x8(c[i], f);
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] *= s;
        Row8<T> v;
        v.set(f);
        v.store(out + row[i] * ld + unit[i] * 8);
    }
    __threadfence();
}

template <class T>
cudaError_t quantize(const void* x, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                     uint8_t* sf, int tiled, int32_t* st, cudaStream_t stream) {
    const int64_t ktiles = (cols + 127) / 128;
    const int64_t units = tiled ? ktiles * 16 : cols / 8;
    const int64_t n = units * (tiled ? (rows + 127) / 128 * 128 : rows);
    LaunchScope scope(kKMxQuant, stream);
    return launch_pdl(mxfp4_quantize_kernel<T>,
                      dim3((unsigned)((n + kThreads * kUnits - 1) / (kThreads * kUnits))),
                      dim3(kThreads), 0, stream, (const T*)x, rows, cols, ld, n,
                      fast_div((uint32_t)units), (uint32_t*)codes, sf,
                      ScaleMap{tiled, cols / 32, ktiles}, st);
}

template <class T>
cudaError_t dequantize(const uint8_t* codes, const uint8_t* sf, int tiled, int64_t rows,
                       int64_t cols, void* out, int64_t ld, cudaStream_t stream) {
    const int64_t n = rows * (cols / 8);
    LaunchScope scope(kKMxDequant, stream);
    return launch_pdl(mxfp4_dequantize_kernel<T>,
                      dim3((unsigned)((n + kThreads * kUnits - 1) / (kThreads * kUnits))),
                      dim3(kThreads), 0, stream, (const uint32_t*)codes, sf,
                      ScaleMap{tiled, cols / 32, (cols + 127) / 128}, n,
                      fast_div((uint32_t)(cols / 8)), (T*)out, ld);
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
