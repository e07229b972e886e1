// Per-head norm and position rotation of query and key rows, and the lightning indexer's
// inputs made from them ("DeepSeek-V4 深度分析报告" "其他注意力技术细节": RMSNorm of queries and
// KV, partial RoPE on the last 64 dims; Figure 2 and 3.4: the indexer's query heads and keys
// in FP8 or MXFP4; 3.5: keys in the classical cache's blocks).
//
//   y = x / sqrt(mean(x^2) + eps) * weight;  the last `rope` channels rotated by
//   pos * theta^(-2j/rope) in interleaved pairs.
//
// A group of lanes holds one row, 8 consecutive channels a lane (4 rotation pairs), so the
// whole row stays in registers between its one load and its one store; a warp walks rows
// (heads) that share a position, whose cosines and sines it forms once, in fp64, and keeps.
#include "launchers.cuh"
#include "rows.cuh"

namespace csa {

namespace {

constexpr int kWarps = 4;

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int LPR>
__device__ __forceinline__ double group_sum(double v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// cos and sin of pos * freq, the angle formed in fp64 and reduced with a two-term 2 pi.
__device__ __forceinline__ void rotation(double pos, double freq, double& c, double& s) {
    const double a = pos * freq;
    const double k = rint(a * 0.15915494309189533577);
    const double r = fma(-k, 2.4492935982947064e-16, fma(-k, 6.283185307179586232, a));
    sincos(r, &s, &c);
}

// ---- rows kept in their type -------------------------------------------------------------
struct QkArgs {
    QkRows q, k;
    const int32_t* pos;
    int T, D, rope, norm;
    int heads_per_warp, warps_per_token;
    float eps;
};

__device__ __forceinline__ void load_weight8(const float* weight, int ch, float* w) {
    if (weight) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(weight + ch));
        const float4 b = __ldg(reinterpret_cast<const float4*>(weight + ch + 4));
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) w[j] = 1.f;
    }
}

// Heads [h0, h1) of one token, kU passes of 32 / LPR rows at a time: the loads of all kU go
// out before the first is used.
template <class T, int LPR, int C, int kU>
__device__ __forceinline__ void norm_rope_heads(const QkRows& x, int64_t t, int h0, int h1, int D,
                                                int lo, bool norm, float eps, int sub, int l,
                                                const float (&cs)[C][4], const float (&sn)[C][4]) {
    constexpr int kRows = 32 / LPR;
    float w[C][8];
#pragma unroll
    for (int c = 0; c < C; c++) {
        const int ch = 8 * (l + LPR * c);
        load_weight8(ch < D ? x.weight : nullptr, ch, w[c]);
    }
    const float inv_d = 1.f / (float)D;
    const T* src = (const T*)x.x + t * x.st + (h0 + sub) * x.sh + 8 * l;
    T* dst = (T*)x.out + t * x.ost + (h0 + sub) * x.osh + 8 * l;
    for (int hb = h0 + sub; hb - sub < h1; hb += kU * kRows) {
        Row8<T> r[kU][C];
#pragma unroll
        for (int u = 0; u < kU; u++)
#pragma unroll
            for (int c = 0; c < C; c++) {
                r[u][c].zero();
                if (hb + u * kRows < h1 && 8 * (l + LPR * c) < D)
                    r[u][c].load(src + u * kRows * x.sh + 8 * LPR * c);
            }
#pragma unroll
        for (int u = 0; u < kU; u++) {
            float f[C][8];
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int c = 0; c < C; c++) {
                r[u][c].get(f[c]);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    s0 = fmaf(f[c][j], f[c][j], s0);
                    s1 = fmaf(f[c][j + 1], f[c][j + 1], s1);
                }
            }
            float rs = 1.f;
            if (norm) rs = rsqrtf(fmaf(group_sum<LPR>(s0 + s1), inv_d, eps));
            const bool in = hb + u * kRows < h1;
#pragma unroll
            for (int c = 0; c < C; c++) {
                const int ch = 8 * (l + LPR * c);
#pragma unroll
                for (int j = 0; j < 8; j++) f[c][j] *= rs * w[c][j];
                if (ch + 8 > lo) {
#pragma unroll
                    for (int p = 0; p < 4; p++) {
                        const float a = f[c][2 * p], b = f[c][2 * p + 1];
                        // a chunk may hold the border: its first pairs stay as they are
                        if (ch >= lo || ch + 2 * p >= lo) {
                            f[c][2 * p] = a * cs[c][p] - b * sn[c][p];
                            f[c][2 * p + 1] = a * sn[c][p] + b * cs[c][p];
                        }
                    }
                }
                Row8<T> o;
                o.set(f[c]);
                if (in && ch < D) o.store(dst + u * kRows * x.osh + 8 * LPR * c);
            }
        }
        src += kU * kRows * x.sh;
        dst += kU * kRows * x.osh;
    }
}

// LPR lanes a row, C chunks of 8 channels a lane (chunk c of lane l: channels 8 (l + LPR c)).
template <class T, int LPR, int C>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_kernel(const QkArgs a, const RopeTable rt) {
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = task / a.warps_per_token;
    if (t >= a.T) return;
    const int h0 = (int)(task - t * a.warps_per_token) * a.heads_per_warp;
    const int h1 = min(h0 + a.heads_per_warp, a.q.heads + a.k.heads);
    const int lo = a.D - a.rope;              // first rotated channel (even)
    float cs[C][4], sn[C][4];
    const double pos = (double)a.pos[t];
#pragma unroll
    for (int c = 0; c < C; c++) {
#pragma unroll
        for (int p = 0; p < 4; p++) {
            const int ch = 8 * (l + LPR * c) + 2 * p;
            cs[c][p] = 1.f;
            sn[c][p] = 0.f;
            if (ch >= lo && ch < a.D) {
                double cd, sd;
                rotation(pos, rt.freq[(ch - lo) >> 1], cd, sd);
                cs[c][p] = (float)cd;
                sn[c][p] = (float)sd;
            }
        }
    }
    constexpr int kU = C == 1 ? 4 : 1;
    if (h0 < a.q.heads)
        norm_rope_heads<T, LPR, C, kU>(a.q, t, h0, min(h1, a.q.heads), a.D, lo, a.norm, a.eps, sub, l, cs, sn);
    if (h1 > a.q.heads)
        norm_rope_heads<T, LPR, C, 1>(a.k, t, max(h0 - a.q.heads, 0), h1 - a.q.heads, a.D, lo, a.norm, a.eps,
                                      sub, l, cs, sn);
    __threadfence();   // visible before the next kernel's reads ahead of its own wait
}

// ---- rows in the indexer's stored formats ----------------------------------------------------
// The codes are those of the definition, whatever the order of the sums: an e4m3 or e2m1 code
// (or a block's power-of-two scale) next to a rounding border is not left to fp32.  The fast
// path computes in fp32 and brackets every quotient z by its error bound: if the codes of z -
// margin and z + margin agree, that code is the one.  If they differ anywhere in the warp's
// rows (about 1 pass in 60 on normal data), or the values leave the range the bound holds in,
// the rows are done again in fp64.
//
// v = x * weight, rotated, is left without the norm's factor r, which joins the scale.  The
// bound, u = 2^-24, relative to |v1| + |v2| of a rotated pair before the rotation (|v|
// elsewhere): the product with the weight, cos or sin, the product with it, the sum: 4 u.
//   MXFP4: z = v * (r * 2^-e).  The sum of squares takes at most 5 roundings in a lane and
//   log2(LPR) <= 4 across, the mean and eps 1, of which rsqrt halves 5 u and adds its
//   2 ulp = 4 u; the product u, the bracket u: 15 u of |v1| + |v2| <= 2 max|v| (a rotation
//   keeps the pair's length).  The bracket is one margin per block, 2 max|z| kFp4Margin.
//   e4m3: z = v * (448 / max|v|), from which r drops out: 4 u, twice 4 u of the largest |v|, u
//   each of the division, the product, the definition's rounding of the scale to fp32 and the
//   bracket: 16 u.  The bracket is relative to each element, since the codes near zero are dense.
// With rows' sums of squares below 2^100, weights below 2^40 and results within 2^-60 .. 2^100
// nothing overflows, and an underflowed product is below 2^-34 of a quotient's unit, far from
// every border but zero's, whose sign it keeps.  (An exact zero beside other values always
// takes the fp64 path of MXFP4, where its bracket has both signs.)
constexpr float kU24 = 5.9604645e-08f;
constexpr float kFp4Margin = 20.f * kU24;
constexpr float kFp8Margin = 20.f * kU24;
constexpr float kTiny = 8.6736174e-19f, kHuge = 1.2676506e+30f;   // 2^-60, 2^100

struct RowQuant {
    uint8_t* codes;    // rows of D (e4m3) or D / 2 (e2m1) bytes
    float* scale;      // e4m3: one fp32 per row
    uint8_t* sf;       // MXFP4: D / 32 UE8M0 bytes per row
    int32_t* st;
};

// A row's result in a lane: its 8 codes (4 bytes for e2m1) and scale, and whether it is bad.
struct RowCodes {
    uint32_t c0, c1;
    uint32_t scale;    // fp32 bits, or the UE8M0 byte
    bool bad;
};

struct Eight {
    float v[8];
};

// The row in fp64 from the input's bits to the codes.  Out of line, its arguments by value: an
// array whose address is taken would live in local memory on the fast path too.
template <int LPR, bool FP4>
__device__ __noinline__ RowCodes quantize_row_f64(const Eight x, const Eight w, const double2* rot, bool norm,
                                                  double eps) {
    constexpr int D = 8 * LPR;
    double y[8];
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        y[j] = (double)x.v[j];
        ss = fma(y[j], y[j], ss);
    }
    double r = 1.0;
    if (norm) r = rsqrt(group_sum<LPR>(ss) * (1.0 / D) + eps);
#pragma unroll
    for (int j = 0; j < 8; j++) y[j] *= r * (double)w.v[j];
    if (rot) {
#pragma unroll
        for (int p = 0; p < 4; p++) {
            const double2 cs = rot[p];
            const double a = y[2 * p], b = y[2 * p + 1];
            y[2 * p] = a * cs.x - b * cs.y;
            y[2 * p + 1] = a * cs.y + b * cs.x;
        }
    }
    RowCodes o;
    float f[8];
    if constexpr (FP4) {
        // the block's scale needs the exponent of its largest magnitude only
        int top = 0;
#pragma unroll
        for (int j = 0; j < 8; j++) top = max(top, __double2hiint(y[j]) & 0x7fffffff);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = (top >> 20) - 1023;              // floor(log2(amax)); -1023 for zeros
        o.bad = ex > 129;                               // not finite, or past the scales' range
        const int e = o.bad ? 255 : max(ex - 2 + 127, 0);
        const double inv = __hiloint2double((1023 + 127 - (o.bad ? 127 : e)) << 20, 0);
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] = f64_to_f32_odd(o.bad ? 0.0 : y[j] * inv);
        o.c0 = pack_e2m1x8(f);
        o.c1 = 0;
        o.scale = (uint32_t)e;
    } else {
        double top = 0.0;
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            top = fmax(top, fabs(y[j]));
            nan |= y[j] != y[j];
        }
#pragma unroll
        for (int s = LPR / 2; s > 0; s >>= 1) {
            top = fmax(top, __shfl_xor_sync(0xffffffffu, top, s));
            nan |= __shfl_xor_sync(0xffffffffu, (int)nan, s) != 0;
        }
        float scale = (float)(top / 448.0);
        o.bad = nan || !(scale <= 3.402823466e38f);
        if (!(scale > 0.f) || o.bad) scale = 1.f;
        // y / scale: the product with the rounded reciprocal, mended once by its remainder, so
        // that a quotient fp64 holds (a tie between two codes, say) comes out exactly
        const double sd = (double)scale, inv = 1.0 / sd;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const double z = y[j] * inv;
            f[j] = f64_to_f32_odd(o.bad ? 0.0 : fma(fma(-z, sd, y[j]), inv, z));
        }
        const uint2 c = pack_e4m3x8(f);
        o.c0 = c.x;
        o.c1 = c.y;
        o.scale = o.bad ? 0x7fffffffu : __float_as_uint(scale);
    }
    return o;
}

// One row over LPR = D / 8 lanes (all lanes of the warp call it): norm, rotation (cs, sn of
// this lane's 4 pairs where rot is given, rot the same in fp64), codes and scale to row `dst`.
// near: whether this lane's weights are past the fast path's range.
template <int LPR, bool FP4>
__device__ __forceinline__ void quantize_row(const float* x, int l, const float* cs, const float* sn,
                                             const double2* rot, const float* w, bool near, bool norm, float eps,
                                             const RowQuant& o, int64_t dst, bool in) {
    constexpr int D = 8 * LPR;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 8; j += 2) fma2(s, x + j, x + j, s);
    const float ss = group_sum<LPR>(s[0] + s[1]);     // a NaN or infinity of the row shows here
    near |= !(ss < kHuge);
    float r = 1.f;
    if (norm) {
        const float ms = fmaf(ss, 1.f / D, eps);
        near |= !(ms > kTiny);
        r = rsqrtf(ms);
    }
    float v[8], mag[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) mul2(v + j, x + j, w + j);
    if constexpr (!FP4) {
#pragma unroll
        for (int j = 0; j < 8; j++) mag[j] = fabsf(v[j]);
    }
    if (rot) {
#pragma unroll
        for (int p = 0; p < 4; p++) {
            const float a = v[2 * p], b = v[2 * p + 1];
            if constexpr (!FP4) mag[2 * p] = mag[2 * p + 1] = fabsf(a) + fabsf(b);
            v[2 * p] = fmaf(a, cs[p], -(b * sn[p]));
            v[2 * p + 1] = fmaf(a, sn[p], b * cs[p]);
        }
    }
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j++) amax = fmaxf(amax, fabsf(v[j]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    if constexpr (!FP4) {
#pragma unroll
        for (int m = 4; m < LPR; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    }
    const bool zero = amax == 0.f;
    near |= !zero && !(amax > kTiny);
    RowCodes c;
    c.bad = false;
    float lo[8], hi[8];
    if constexpr (FP4) {
        const float top = amax * r;
        const uint32_t ex = __float_as_uint(top) >> 23;
        // the largest magnitude may itself lie next to a power of two
        near |= !zero && (!(top > kTiny && top < kHuge) ||
                          __float_as_uint(fmaf(top, 2.1f * kFp4Margin, top)) >> 23 != ex ||
                          __float_as_uint(fmaf(top, -2.1f * kFp4Margin, top)) >> 23 != ex);
        // a non-finite block is `near`: the minimum only keeps the shift in range
        const uint32_t e = zero ? 0u : max(min(ex, 250u), 2u) - 2u;
        c.scale = e;
        const float inv = zero ? 1.f : r * __uint_as_float((254u - e) << 23);     // r * 2^(127 - e)
        const float inv2[2] = {inv, inv};
        const float m = 2.f * kFp4Margin * (amax * inv), up[2] = {m, m}, down[2] = {-m, -m};
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float z[2];
            mul2(z, v + j, inv2);
            add2(lo + j, z, down);
            add2(hi + j, z, up);
        }
        c.c0 = pack_e2m1x8(lo);
        c.c1 = 0;
        near |= !zero && pack_e2m1x8(hi) != c.c0;     // zeros keep their sign in lo
    } else {
        const float inv = zero ? 1.f : 448.f / amax;
        const float inv2[2] = {inv, inv};
        const float m = kFp8Margin * inv, up[2] = {m, m}, down[2] = {-m, -m};
        c.scale = __float_as_uint(zero ? 1.f : (amax * r) * (1.f / 448.f));
        near |= !zero && !(amax * r > kTiny && amax * r < kHuge);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float z[2];
            mul2(z, v + j, inv2);
            fma2(lo + j, mag + j, down, z);
            fma2(hi + j, mag + j, up, z);
        }
        const uint2 a = pack_e4m3x8(lo), b = pack_e4m3x8(hi);
        c.c0 = a.x;
        c.c1 = a.y;
        near |= !zero && (a.x != b.x || a.y != b.y);
    }
    if (__any_sync(0xffffffffu, near)) {
        Eight xv, wv;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            xv.v[j] = x[j];
            wv.v[j] = w[j];
        }
        c = quantize_row_f64<LPR, FP4>(xv, wv, rot, norm, (double)eps);
    }
    if (!in) return;
    if constexpr (FP4) {
        reinterpret_cast<uint32_t*>(o.codes)[dst * (D / 8) + l] = c.c0;
        if ((l & 3) == 0) {
            o.sf[dst * (D / 32) + (l >> 2)] = (uint8_t)c.scale;
            if (c.bad) flag(o.st, CSA_DEV_NAN);
        }
    } else {
        reinterpret_cast<uint2*>(o.codes)[dst * LPR + l] = make_uint2(c.c0, c.c1);
        if (l == 0) {
            o.scale[dst] = __uint_as_float(c.scale);
            if (c.bad) flag(o.st, CSA_DEV_NAN);
        }
    }
}

// Whether a weight is not finite or past what the fast path's bound holds for.
__device__ __forceinline__ bool weight_past_range(const float* w) {
    bool past = false;
#pragma unroll
    for (int j = 0; j < 8; j++) past |= !(fabsf(w[j]) < 1.0995116e+12f);   // 2^40
    return past;
}

// This lane's 4 rotation pairs: fp32 in registers, fp64 in shared memory for the fp64 path
// (nullptr where the lane's channels are not rotated).
template <int LPR>
__device__ __forceinline__ const double2* lane_rotation(double pos, const RopeTable& rt, int l, int rope,
                                                        double2* mine, float* cs, float* sn) {
    const int first = 4 * l - (8 * LPR - rope) / 2;
#pragma unroll
    for (int p = 0; p < 4; p++) {
        cs[p] = 1.f;
        sn[p] = 0.f;
    }
    if (first < 0) return nullptr;
#pragma unroll
    for (int p = 0; p < 4; p++) {
        double c, s;
        rotation(pos, rt.freq[first + p], c, s);
        mine[p] = make_double2(c, s);
        cs[p] = (float)c;
        sn[p] = (float)s;
    }
    return mine;
}

struct QueryArgs {
    const void* q;
    const float* weight;
    const int32_t* pos;
    int64_t st, sh;           // strides of q, elements
    int Q, H, rope, norm;
    int heads_per_warp, warps_per_token;
    float eps;
    RowQuant o;
};

template <class T, int LPR, bool FP4>
__global__ void __launch_bounds__(32 * kWarps) indexer_queries_kernel(const QueryArgs a, const RopeTable rt) {
    __shared__ double2 rot64[32 * kWarps][4];
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    constexpr int kRows = 32 / LPR;
    const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = task / a.warps_per_token;
    if (t >= a.Q) return;
    const int h0 = (int)(task - t * a.warps_per_token) * a.heads_per_warp;
    const int h1 = min(h0 + a.heads_per_warp, a.H);
    float w[8], cs[4], sn[4];
    load_weight8(a.weight, 8 * l, w);
    const bool past = weight_past_range(w);
    const T* src = (const T*)a.q + t * a.st + (h0 + sub) * a.sh + 8 * l;
    constexpr int kU = 2;                // rows a lane loads ahead of the one it works on
    Row8<T> r[kU];
#pragma unroll
    for (int u = 0; u < kU; u++) {
        r[u].zero();
        if (h0 + sub + u * kRows < h1) r[u].load(src + u * kRows * a.sh);
    }
    const double2* rot = lane_rotation<LPR>((double)a.pos[t], rt, l, a.rope, rot64[threadIdx.x], cs, sn);
    int64_t dst = t * a.H + h0 + sub;
    for (int hb = h0; hb < h1; hb += kRows) {
        const int h = hb + sub;
        float x[8];
        r[0].get(x);
#pragma unroll
        for (int u = 0; u + 1 < kU; u++) r[u] = r[u + 1];
        r[kU - 1].zero();
        src += kRows * a.sh;
        if (h + kU * kRows < h1) r[kU - 1].load(src + (kU - 1) * kRows * a.sh);
        quantize_row<LPR, FP4>(x, l, cs, sn, rot, w, past, a.norm, a.eps, a.o, dst, h < h1);
        dst += kRows;
    }
    __threadfence();
}

struct AppendArgs {
    const void* k;
    const float* weight;
    int64_t ld;
    const int64_t* seq_len;
    EntryRows er;
    const int32_t* item_seq;
    const int32_t* item_ent;
    int64_t n, ent_rows;
    int B, m, rope, norm;
    float eps;
    RowQuant o;
};

// One listed entry per row: its position is the block end (i + 1) m - 1.
template <class T, int LPR, bool FP4>
__global__ void __launch_bounds__(32 * kWarps) indexer_append_kernel(const AppendArgs a, const RopeTable rt) {
    __shared__ double2 rot64[32 * kWarps][4];
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    constexpr int kRows = 32 / LPR;
    const int64_t it = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRows + sub;
    bool in = it < a.n;
    int64_t dst = 0, pos = 0;
    Row8<T> r;
    r.zero();
    if (in) {
        r.load((const T*)a.k + it * a.ld + 8 * l);
        const int b = a.item_seq[it];
        const int64_t i = a.item_ent[it];
        bool ok = b >= 0 && b < a.B && i >= 0;
        if (ok) {
            pos = (i + 1) * a.m - 1;
            ok = pos < a.seq_len[b] && (!a.er.bt || (i >> a.er.pe_shift) < a.er.bt_stride);
            if (ok) dst = a.er.row(b, i);
            ok = ok && dst >= 0 && dst < a.ent_rows;
        }
        if (!ok) {
            if (l == 0) flag(a.o.st, CSA_DEV_OOB);
            in = false;
            pos = 0;
            r.zero();
        }
    }
    float w[8], x[8], cs[4], sn[4];
    load_weight8(a.weight, 8 * l, w);
    const double2* rot = lane_rotation<LPR>((double)pos, rt, l, a.rope, rot64[threadIdx.x], cs, sn);
    r.get(x);
    quantize_row<LPR, FP4>(x, l, cs, sn, rot, w, weight_past_range(w), a.norm, a.eps, a.o, dst, in);
    __threadfence();
}

// theta^(-2j / rope) for the pairs j of the rotated channels.  A thread keeps its last table:
// its 32 powers took 1.0 us of a call's 4.
const RopeTable& rope_table(int rope, double theta) {
    static thread_local RopeTable t = {};
    static thread_local int last_rope = -1;
    static thread_local double last_theta = 0.0;
    if (rope != last_rope || theta != last_theta) {
        for (int j = 0; j < rope / 2; j++) t.freq[j] = pow(theta, -2.0 * j / rope);
        last_rope = rope;
        last_theta = theta;
    }
    return t;
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

// Heads one warp walks: all of a token's when the tokens alone give every SM 8 warps (the
// cosines are then formed once per token), fewer when there are few tokens.
void split_heads(int tokens, int heads, int rows_per_pass, int& per_warp, int& warps) {
    const int64_t want = (int64_t)sm_count() * 8;
    const int passes = (heads + rows_per_pass - 1) / rows_per_pass;
    int64_t split = (want + tokens - 1) / tokens;
    if (split > passes) split = passes;
    if (split < 1) split = 1;
    const int p = (int)((passes + split - 1) / split);
    per_warp = p * rows_per_pass;
    warps = (heads + per_warp - 1) / per_warp;
}

unsigned blocks_of(int64_t tasks) { return (unsigned)((tasks + kWarps - 1) / kWarps); }

template <class T, int LPR, int C>
cudaError_t run_qk(QkArgs a, const RopeTable& rt, cudaStream_t stream) {
    split_heads(a.T, a.q.heads + a.k.heads, 32 / LPR, a.heads_per_warp, a.warps_per_token);
    LaunchScope scope(kKQkNormRope, stream);
    return launch_pdl(qk_norm_rope_kernel<T, LPR, C>, dim3(blocks_of((int64_t)a.T * a.warps_per_token)),
                      dim3(32 * kWarps), 0, stream, a, rt);
}

template <class T>
cudaError_t run_qk_dims(const QkArgs& a, const RopeTable& rt, cudaStream_t stream) {
    const int chunks = a.D / 8;
    if (chunks <= 8) return run_qk<T, 8, 1>(a, rt, stream);
    if (chunks <= 16) return run_qk<T, 16, 1>(a, rt, stream);
    if (chunks <= 32) return run_qk<T, 32, 1>(a, rt, stream);
    if (chunks <= 64) return run_qk<T, 32, 2>(a, rt, stream);
    if (chunks <= 96) return run_qk<T, 32, 3>(a, rt, stream);
    return run_qk<T, 32, 4>(a, rt, stream);
}

template <class T, int LPR, bool FP4>
cudaError_t run_queries(QueryArgs a, const RopeTable& rt, cudaStream_t stream) {
    split_heads(a.Q, a.H, 32 / LPR, a.heads_per_warp, a.warps_per_token);
    LaunchScope scope(kKIndexerQueries, stream);
    return launch_pdl(indexer_queries_kernel<T, LPR, FP4>,
                      dim3(blocks_of((int64_t)a.Q * a.warps_per_token)), dim3(32 * kWarps), 0, stream,
                      a, rt);
}

template <class T, int LPR, bool FP4>
cudaError_t run_append(const AppendArgs& a, const RopeTable& rt, cudaStream_t stream) {
    constexpr int kRows = 32 / LPR;
    LaunchScope scope(kKIndexerAppend, stream);
    return launch_pdl(indexer_append_kernel<T, LPR, FP4>, dim3(blocks_of((a.n + kRows - 1) / kRows)),
                      dim3(32 * kWarps), 0, stream, a, rt);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkRows& q, const QkRows& k, const int32_t* pos, int dtype, int T,
                                int D, int rope, int norm, float theta, float eps,
                                cudaStream_t stream) {
    const QkArgs a{q, k, pos, T, D, rope, norm, 0, 0, eps};
    const RopeTable& rt = rope_table(rope, theta);
    switch (dtype) {
        case CSA_DT_BF16: return run_qk_dims<__nv_bfloat16>(a, rt, stream);
        case CSA_DT_F16: return run_qk_dims<__half>(a, rt, stream);
        default: return run_qk_dims<float>(a, rt, stream);
    }
}

#define CSA_ROWS_DISPATCH(RUN, ARGS)                                                      \
    do {                                                                                  \
        const bool fp4 = fmt == CSA_IDX_MXFP4;                                            \
        if (dtype == CSA_DT_BF16) {                                                       \
            using T = __nv_bfloat16;                                                      \
            if (D == 128) return fp4 ? RUN<T, 16, true>(ARGS, rt, stream) : RUN<T, 16, false>(ARGS, rt, stream); \
            return fp4 ? RUN<T, 8, true>(ARGS, rt, stream) : RUN<T, 8, false>(ARGS, rt, stream); \
        }                                                                                 \
        if (dtype == CSA_DT_F16) {                                                        \
            using T = __half;                                                             \
            if (D == 128) return fp4 ? RUN<T, 16, true>(ARGS, rt, stream) : RUN<T, 16, false>(ARGS, rt, stream); \
            return fp4 ? RUN<T, 8, true>(ARGS, rt, stream) : RUN<T, 8, false>(ARGS, rt, stream); \
        }                                                                                 \
        if (D == 128) return fp4 ? RUN<float, 16, true>(ARGS, rt, stream) : RUN<float, 16, false>(ARGS, rt, stream); \
        return fp4 ? RUN<float, 8, true>(ARGS, rt, stream) : RUN<float, 8, false>(ARGS, rt, stream); \
    } while (0)

cudaError_t launch_indexer_queries(const void* q, int dtype, int64_t st, int64_t sh, const int32_t* pos,
                                   const float* weight, int norm, int rope, float theta, float eps,
                                   int Q, int H, int D, int fmt, uint8_t* codes, void* scale,
                                   int32_t* dev_status, cudaStream_t stream) {
    QueryArgs a{q, weight, pos, st, sh, Q, H, rope, norm, 0, 0, eps,
                RowQuant{codes, (float*)scale, (uint8_t*)scale, dev_status}};
    const RopeTable& rt = rope_table(rope, theta);
    CSA_ROWS_DISPATCH(run_queries, a);
}

cudaError_t launch_indexer_append(const void* k, int dtype, int64_t ld, const int64_t* seq_len,
                                  const EntryRows& er, const int32_t* item_seq,
                                  const int32_t* item_ent, int64_t n, int64_t ent_rows, int B, int m,
                                  const float* weight, int norm, int rope, float theta, float eps,
                                  int D, int fmt, uint8_t* codes, void* scale, int32_t* dev_status,
                                  cudaStream_t stream) {
    AppendArgs a{k, weight, ld, seq_len, er, item_seq, item_ent, n, ent_rows, B, m, rope, norm,
                 eps, RowQuant{codes, (float*)scale, (uint8_t*)scale, dev_status}};
    const RopeTable& rt = rope_table(rope, theta);
    CSA_ROWS_DISPATCH(run_append, a);
}

}  // namespace csa
