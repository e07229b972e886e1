// Eight consecutive elements of a row in bf16, fp16 or fp32, and their e2m1 / e4m3 codes.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace csa {

// 16 (bf16, fp16) or 32 (fp32) bytes of a row, loaded and stored as 16-byte vectors.
template <class T>
struct Row8;

template <>
struct Row8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = r; }
    __device__ __forceinline__ void get(float* f) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 p = bf16x2_to_f32(w[i]);
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        }
    }
    __device__ __forceinline__ void set(const float* f) {
        // one packed conversion per pair: the single ones run on the slow conversion unit (the
        // 8192-token norm and rotation took 83 us with them, 27 % of that unit's rate)
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <>
struct Row8<__half> {
    uint4 r;
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __half* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(__half* p) const { *reinterpret_cast<uint4*>(p) = r; }
    __device__ __forceinline__ void get(float* f) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        }
    }
    __device__ __forceinline__ void set(const float* f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <>
struct Row8<float> {
    float4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void store(float* p) const {
        *reinterpret_cast<float4*>(p) = a;
        *reinterpret_cast<float4*>(p + 4) = b;
    }
    __device__ __forceinline__ void get(float* f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void set(const float* f) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// Eight e2m1 codes, element j in nibble j: nearest, ties to the even code, past 6 to 6.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float* y) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return r;
}

__device__ __forceinline__ void unpack_e2m1x8(uint32_t c, float* f) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

// Eight e4m3 codes, element j in byte j: nearest, ties to even, past 448 to 448.
__device__ __forceinline__ uint2 pack_e4m3x8(const float* y) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i], y[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2], y[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

// Two fp32 operations in one instruction, each rounded as its own.
__device__ __forceinline__ uint64_t bits2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void mul2(float* d, const float* a, const float* b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a[0], a[1])), "l"(bits2(b[0], b[1])));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d[0]), "=f"(d[1]) : "l"(r));
}
__device__ __forceinline__ void add2(float* d, const float* a, const float* b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a[0], a[1])), "l"(bits2(b[0], b[1])));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d[0]), "=f"(d[1]) : "l"(r));
}
__device__ __forceinline__ void fma2(float* d, const float* a, const float* b, const float* c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(bits2(a[0], a[1])), "l"(bits2(b[0], b[1])), "l"(bits2(c[0], c[1])));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d[0]), "=f"(d[1]) : "l"(r));
}

// z as an fp32 whose last bit is set where bits were cut off ("rounded to odd"): rounding the
// result to a format of at most 21 fraction bits gives what rounding z itself gives.
// Magnitudes below 2^-126 come back as one just above it (for the formats here both round to
// zero); |z| must be below 2^128.
// The sign is that of `sign`.
__device__ __forceinline__ float f64_to_f32_odd(double z, double sign) {
    const uint32_t hi = (uint32_t)__double2hiint(z), lo = (uint32_t)__double2loint(z);
    const uint32_t neg = (uint32_t)__double2hiint(sign) & 0x80000000u;
    const uint32_t mag = hi & 0x7fffffffu;
    const bool small = mag < (897u << 20);
    const uint32_t a = (small ? (897u << 20) : mag) - (896u << 20);
    uint32_t f = __funnelshift_l(lo, a, 3);
    f |= (lo & 0x1fffffffu) ? 1u : 0u;
    return __uint_as_float(z == 0.0 ? neg : (f | neg));
}
__device__ __forceinline__ float f64_to_f32_odd(double z) { return f64_to_f32_odd(z, z); }

}  // namespace csa
