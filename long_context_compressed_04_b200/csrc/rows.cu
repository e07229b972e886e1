// Per-head norm and position rotation of query and key rows, and the lightning indexer's
// inputs made from them ("DeepSeek-V4 深度分析报告" "其他注意力技术细节": RMSNorm of queries and
// KV, partial RoPE on the last 64 dims; Figure 2 and 3.4: the indexer's query heads and keys
// in FP8 or MXFP4; 3.5: keys in the classical cache's blocks).
//
//   y = x / sqrt(mean(x^2) + eps) * weight;  the last `rope` channels rotated by
//   pos * theta^(-2j/rope) in interleaved pairs.
//
// A group of lanes holds one row, chunks of 8 consecutive channels a lane (4 rotation pairs), so
// the whole row stays in registers between its one load and its one store; a warp walks rows
// (heads) that share a position, whose cosines and sines its lanes form once, in fp64, a pair
// each.  8192 tokens of 64 + 1 heads x 128 in bf16 (273 MB): norm and rotation 50 us, 5.4 TB/s,
// bound by HBM; query heads to MXFP4 (170 MB) 50 us, to FP8 (203 MB) 62, bound by instructions
// (256 per lane and 16 channels for MXFP4, half of them the scale, the brackets and the codes; FP8
// converts two values of a bracket to each code and has more passes in fp64).
#include <type_traits>

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

// Its two top bits are 0 if a mean square lies in 2^-64 .. 2^64; beyond, squares of the row may have
// left fp32's range.  (Bits of several may be joined.)
__device__ __forceinline__ uint32_t range_bits(float ms) { return __float_as_uint(ms) - (63u << 23); }

// Mean of a row's squares over its lanes, plus eps.
template <int LPR, int C>
__device__ __forceinline__ float mean_square(const float (&f)[C][8], float inv_d, float eps) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            s0 = fmaf(f[c][j], f[c][j], s0);
            s1 = fmaf(f[c][j + 1], f[c][j + 1], s1);
        }
    return fmaf(group_sum<LPR>(s0 + s1), inv_d, eps);
}

// Rows whose squares leave fp32's range (all lanes of the warp call it): a row whose mean square lies
// outside 2^-64 .. 2^64 is multiplied by the power of two that brings the larger of its greatest
// magnitude and sqrt(eps) near 1, which its norm undoes.  Rows in range keep their bits.
template <int LPR, int C>
__device__ __forceinline__ float rescaled_mean_square(float (&f)[C][8], float ms, float inv_d, float eps) {
    float top = sqrtf(eps);
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
        for (int j = 0; j < 8; j++) top = fmaxf(top, fabsf(f[c][j]));
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -120), 120);
    const float k = range_bits(ms) >> 30 == 0u ? 1.f : __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
        for (int j = 0; j < 8; j++) f[c][j] *= k;
    return mean_square<LPR, C>(f, inv_d, eps * k * k);
}

// A row's values, normed by rs, weighted and rotated, into its output.
template <class T, int LPR, int C>
__device__ __forceinline__ void finish_row(float (&f)[C][8], float rs, const float (&w)[C][8], const float (&cs)[C][4],
                                           const float (&sn)[C][4], int D, int lo, int l, T* dst, bool write) {
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
        if (write && ch < D) o.store(dst + 8 * LPR * c);
    }
}

// Heads [h0, h1) of one token, kU passes of 32 / LPR rows at a time: the loads of all kU go
// out before the first is used.
template <class T, int LPR, int C, int kU>
__device__ __forceinline__ void norm_rope_heads(const QkRows& x, int64_t t, int h0, int h1, int D,
                                                int lo, bool norm, float eps, int sub, int l,
                                                const float (&cs)[C][4], const float (&sn)[C][4]) {
    constexpr int kRows = 32 / LPR;
    constexpr bool kRanged = !std::is_same<T, __half>::value;     // fp16's squares stay in range
    float w[C][8];
#pragma unroll
    for (int c = 0; c < C; c++) {
        const int ch = 8 * (l + LPR * c);
        load_weight8(ch < D ? x.weight : nullptr, ch, w[c]);
    }
    const float inv_d = 1.f / (float)D;
    const int64_t step = kRows * x.sh, ostep = kRows * x.osh;
    const T* src = (const T*)x.x + t * x.st + (h0 + sub) * x.sh + 8 * l;
    T* dst = (T*)x.out + t * x.ost + (h0 + sub) * x.osh + 8 * l;
    for (int hb = h0; hb < h1; hb += kU * kRows) {
        Row8<T> r[kU][C];
        // lanes past the last head load the last one again: no zeroing, no predicate
        const bool full = hb + kU * kRows <= h1;
        const auto load = [&](Row8<T>(&row)[C], int u) {
            const T* from = src + u * step;
            if (!full) from -= max(hb + sub + u * kRows - (h1 - 1), 0) * x.sh;
#pragma unroll
            for (int c = 0; c < C; c++)
                if (8 * (l + LPR * c) < D) row[c].load(from + 8 * LPR * c);
        };
        const auto values = [&](Row8<T>(&row)[C], float(&f)[C][8]) {
#pragma unroll
            for (int c = 0; c < C; c++) {
                if (8 * (l + LPR * c) >= D) row[c].zero();
                row[c].get(f[c]);
            }
        };
#pragma unroll
        for (int u = 0; u < kU; u++) load(r[u], u);
        if constexpr (kU == 1) {
            float f[C][8];
            values(r[0], f);
            float rs = 1.f;
            if (norm) {
                float ms = mean_square<LPR, C>(f, inv_d, eps);
                if (kRanged && __any_sync(0xffffffffu, range_bits(ms) >> 30))
                    ms = rescaled_mean_square<LPR, C>(f, ms, inv_d, eps);
                rs = rsqrtf(ms);
            }
            finish_row<T, LPR, C>(f, rs, w, cs, sn, D, lo, l, dst, full | (hb + sub < h1));
        } else {
            // every mean square before the first row is done: one test of their range and the
            // shuffles of all kU in flight (4096 tokens of 33 heads x 64 in bf16 10.8 -> 9.0 us)
            float ms[kU];
            uint32_t far = 0;
#pragma unroll
            for (int u = 0; u < kU; u++) {
                float f[C][8];
                values(r[u], f);
                ms[u] = norm ? mean_square<LPR, C>(f, inv_d, eps) : 1.f;
                far |= range_bits(ms[u]);
            }
            if (kRanged && __any_sync(0xffffffffu, far >> 30)) {
                // from the inputs again (nothing of these rows is written yet), and not unrolled: it
                // costs the others no registers
#pragma unroll 1
                for (int u = 0; u < kU; u++) {
                    Row8<T> row[C];
                    float f[C][8];
                    load(row, u);
                    values(row, f);
                    const float m = rescaled_mean_square<LPR, C>(f, mean_square<LPR, C>(f, inv_d, eps), inv_d, eps);
                    finish_row<T, LPR, C>(f, rsqrtf(m), w, cs, sn, D, lo, l, dst + u * ostep,
                                          hb + sub + u * kRows < h1);
                }
            } else {
#pragma unroll
                for (int u = 0; u < kU; u++) {
                    float f[C][8];
                    values(r[u], f);
                    finish_row<T, LPR, C>(f, norm ? rsqrtf(ms[u]) : 1.f, w, cs, sn, D, lo, l, dst + u * ostep,
                                          full | (hb + sub + u * kRows < h1));
                }
            }
        }
        src += kU * step;
        dst += kU * ostep;
    }
}

// Resident CTAs that the registers have to allow: what the kernels took before their rows' range was
// tested, without which 8192 x 65 x 128 took 50.5 us instead of 49.6.
template <class T, int C>
constexpr int qk_blocks() {
    return sizeof(T) == 2 ? (C == 1 ? 7 : C == 2 ? 5 : 4) : (C == 1 ? 5 : C <= 3 ? 4 : 3);
}

// LPR lanes a row, C chunks of 8 channels a lane (chunk c of lane l: channels 8 (l + LPR c)).
template <class T, int LPR, int C>
__global__ void __launch_bounds__(32 * kWarps, qk_blocks<T, C>()) qk_norm_rope_kernel(const QkArgs a, const RopeTable rt) {
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = task / a.warps_per_token;
    if (t >= a.T) return;
    const int h0 = (int)(task - t * a.warps_per_token) * a.heads_per_warp;
    const int h1 = min(h0 + a.heads_per_warp, a.q.heads + a.k.heads);
    const int lo = a.D - a.rope;              // first rotated channel (even)
    // each pair's cosine and sine by one lane, handed on through shared memory
    __shared__ float2 tables[kWarps][kMaxRopePairs];
    float2* table = tables[threadIdx.x >> 5];
    const double pos = (double)a.pos[t];
    for (int j = lane; j < a.rope / 2; j += 32) {
        double cd, sd;
        rotation(pos, rt.freq[j], cd, sd);
        table[j] = make_float2((float)cd, (float)sd);
    }
    __syncwarp();
    float cs[C][4], sn[C][4];
#pragma unroll
    for (int c = 0; c < C; c++) {
#pragma unroll
        for (int p = 0; p < 4; p++) {
            const int ch = 8 * (l + LPR * c) + 2 * p;
            const float2 r = ch >= lo && ch < a.D ? table[(ch - lo) >> 1] : make_float2(1.f, 0.f);
            cs[c][p] = r.x;
            sn[c][p] = r.y;
        }
    }
    // (four rows of fp32 in flight per lane: 4096 x 65 x 128 55 us against 50 with one)
    constexpr int kU = sizeof(T) == 4 ? 1 : C == 1 ? 4 : C == 2 ? 2 : 1;
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
// margin and z + margin agree, that code is the one.  If they differ anywhere in the warp's rows,
// or the values leave the range the bound holds in, the rows are done again in fp64.
//
// v = x * weight, rotated, is left without the norm's factor r, which joins the scale.  The
// bound, u = 2^-24: v is off by 4 u of |v1| + |v2| of its pair before the rotation, or of |v|
// without one (the product with the weight, cos or sin, the product with it, the sum); the rest
// is relative to z:
//   MXFP4: z = v * (r * 2^-e).  The sum of squares takes at most 6 roundings in a lane and
//   log2(LPR) <= 3 across, the mean and eps 1, of which rsqrt halves 5 u and adds its
//   2 ulp = 4 u; the product u: 10 u.  The block's largest |v| is off by 8 u of itself (|v1| +
//   |v2| <= 2 max|v|, since a rotation keeps the pair's length), and 10 u with r.
//   e4m3: z = v * (448 / max|v|), from which r drops out: 8 u of the largest |v|, u each of the
//   division, the product, the definition's rounding of the scale to fp32: 11 u.
// The bracket's own roundings add 2 u.  Counted whole against |v1| + |v2|, the bound of e4m3, whose
// codes are dense near zero, sent 1 pass in 15 to fp64, where this sends 1 in 38 (4 us of 72 for 8192
// tokens of 64 x 128 with a random weight; MXFP4 sends 1 in 200 either way; bf16 rows without a
// weight lie on borders more often).  The angle's own error, pos 2^-52 of |v1| + |v2|, finds u of
// room in the bound: positions below 2^28.  With rows' sums of squares below
// 2^100, weights below 2^40 and results within 2^-60 .. 2^100 nothing overflows, and an
// underflowed product is below 2^-34 of a quotient's unit, far from every border but zero's,
// whose sign it keeps without a rotation.  Where every product is zero in fp32 (values below 2^-148),
// the norm may lift them back: a block then counts as zero if the mean square is above 2^-36,
// which leaves them below 2^-130, an eighth of the least scale; a row in e4m3, whose scales reach
// down to 2^-149, only if its inputs are zeros.  (Both tests on every row: 8192 tokens of 64 x 128
// to MXFP4 50.6 -> 51.7 us.)
constexpr float kU24 = 5.9604645e-08f;
constexpr float kAbsMargin = 5.f * kU24, kRelMargin = 15.f * kU24, kTopMargin = 24.f * kU24;
constexpr float kTiny = 8.6736174e-19f, kHuge = 1.2676506e+30f;   // 2^-60, 2^100
constexpr float kLeastMean = 1.4551915e-11f;                      // 2^-36

struct RowQuant {
    uint8_t* codes;    // rows of D (e4m3) or D / 2 (e2m1) bytes
    float* scale;      // e4m3: one fp32 per row
    uint8_t* sf;       // MXFP4: D / 32 UE8M0 bytes per row
    int32_t* st;
};

// Which of a lane's two chunks are rotated: the second (rope = D / 2), both (rope = D), or as
// the lane's pair numbers say.
enum RotMode { kRotAny = 0, kRotUpper = 1, kRotAll = 2 };

// A row's (or a lane's) values: kC chunks of 8 channels, chunk c of lane l at 8 (l + LPR c).
constexpr int kC = 2;
struct Lane {
    float v[kC][8];
};

// Codes of one lane's chunks (e2m1: the first word of each), their scales, what is bad.
struct RowCodes {
    uint32_t c[kC][2];
    uint32_t scale[kC];   // UE8M0 byte per chunk's block, or the row's fp32 bits
    bool bad[kC];
};

// The row in fp64 from the input's bits to the codes.  Out of line, its arguments by value: an
// array whose address is taken would live in local memory on the fast path too.
template <int LPR, bool FP4>
__device__ __noinline__ RowCodes quantize_row_f64(const Lane x, const float* weight, const double2* rot0,
                                                  const double2* rot1, bool norm, double eps) {
    constexpr int D = 8 * kC * LPR;
    double y[kC][8];
    double s4[4] = {};         // four chains: a call's time is that of its dependent instructions
#pragma unroll
    for (int c = 0; c < kC; c++)
#pragma unroll
        for (int j = 0; j < 8; j++) {
            y[c][j] = (double)x.v[c][j];
            s4[j & 3] = fma(y[c][j], y[c][j], s4[j & 3]);
        }
    const double ss = (s4[0] + s4[1]) + (s4[2] + s4[3]);
    double r = 1.0;
    if (norm) r = rsqrt(group_sum<LPR>(ss) * (1.0 / D) + eps);
#pragma unroll
    for (int c = 0; c < kC; c++) {
        const double2* rot = c ? rot1 : rot0;
#pragma unroll
        for (int j = 0; j < 8; j++) y[c][j] *= r * (double)__ldg(weight + 8 * LPR * c + j);
        if (rot) {
#pragma unroll
            for (int p = 0; p < 4; p++) {
                const double2 cs = rot[p];
                const double a = y[c][2 * p], b = y[c][2 * p + 1];
                y[c][2 * p] = a * cs.x - b * cs.y;
                y[c][2 * p + 1] = a * cs.y + b * cs.x;
            }
        }
    }
    RowCodes o;
    if constexpr (FP4) {
#pragma unroll
        for (int c = 0; c < kC; c++) {
            // the block's scale needs the exponent of its largest magnitude only
            int top = 0;
#pragma unroll
            for (int j = 0; j < 8; j++) top = max(top, __double2hiint(y[c][j]) & 0x7fffffff);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = (top >> 20) - 1023;              // floor(log2(amax)); -1023 for zeros
            const bool bad = ex > 129;                      // not finite, or past the scales' range
            const int e = bad ? 255 : max(ex - 2 + 127, 0);
            const double inv = __hiloint2double((1023 + 127 - (bad ? 127 : e)) << 20, 0);
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; j++) f[j] = f64_to_f32_odd(bad ? 0.0 : y[c][j] * inv);
            o.c[c][0] = pack_e2m1x8(f);
            o.c[c][1] = 0;
            o.scale[c] = (uint32_t)e;
            o.bad[c] = bad;
        }
    } else {
        // magnitudes compare as integers, a NaN above an infinity above the rest
        unsigned long long top = 0;
#pragma unroll
        for (int c = 0; c < kC; c++)
#pragma unroll
            for (int j = 0; j < 8; j++)
                top = max(top, (unsigned long long)__double_as_longlong(fabs(y[c][j])));
#pragma unroll
        for (int s = LPR / 2; s > 0; s >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
        float scale = (float)(__longlong_as_double((long long)top) / 448.0);
        const bool bad = !(scale <= 3.402823466e38f);
        if (!(scale > 0.f) || bad) scale = 1.f;
        // y / scale: the product with the rounded reciprocal, mended once by its remainder, so
        // that a quotient fp64 holds (a tie between two codes, say) comes out exactly
        const double sd = (double)scale, inv = 1.0 / sd;
#pragma unroll
        for (int c = 0; c < kC; c++) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const double z = y[c][j] * inv;
                // (a zero's remainder would lose its sign)
                f[j] = f64_to_f32_odd(bad ? 0.0 : fma(fma(-z, sd, y[c][j]), inv, z), bad ? 0.0 : z);
            }
            const uint2 q = pack_e4m3x8(f);
            o.c[c][0] = q.x;
            o.c[c][1] = q.y;
            o.scale[c] = bad ? 0x7fffffffu : __float_as_uint(scale);
            o.bad[c] = bad;
        }
    }
    return o;
}

// cos and sin of a position's pairs (at most 64 of a 128-channel row), in shared memory: fp32 for
// the fast path, fp64 for the other.  Kept out of registers: with them and the weights there
// a thread took 128 and the SM held 16 warps.
struct RotTable {
    double2 f64[64];
    float2 f32[64];
};

// Weights of a call without any (read like the others: no branch per row, 16 bytes at a time, which
// a bare array of floats would not be aligned for).
#define CSA_ONES_8 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f
#define CSA_ONES_32 CSA_ONES_8, CSA_ONES_8, CSA_ONES_8, CSA_ONES_8
constexpr int kMaxIndexerDim = 128;
struct alignas(sizeof(float4)) UnitWeights {
    float v[kMaxIndexerDim];
};
static_assert(alignof(UnitWeights) >= alignof(float4), "read through float4");
__device__ const UnitWeights kOnes = {{CSA_ONES_32, CSA_ONES_32, CSA_ONES_32, CSA_ONES_32}};

// What a lane needs of a position: its weights, its chunks' pairs in the table, whether a weight
// is past what the fast path's bound holds for.
template <RotMode RM>
struct LaneParams {
    const float* weight;
    const RotTable* table;
    int pair[kC];      // first pair of the chunk, negative: not rotated
    bool past;
    __device__ __forceinline__ bool rotated(int c) const {
        return RM == kRotAll || (RM == kRotUpper ? c == 1 : pair[c] >= 0);
    }
    __device__ __forceinline__ const double2* rot(int c) const { return rotated(c) ? table->f64 + pair[c] : nullptr; }
};

// The brackets of a chunk's quotients z = v * inv: kAbsMargin times the pair's magnitude before the
// rotation (scaled alike) plus kRelMargin |z| to each side, or without a rotation both times |z|;
// for e2m1, whose codes are few, both times the pair's magnitude (cheaper: 50 us against 51).
template <bool FP4>
__device__ __forceinline__ void bracket(const float* v, const float* mag, bool rotated, float inv, float* lo,
                                        float* hi) {
    if (FP4 && rotated) {
        const float inv2[2] = {inv, inv}, m = (kAbsMargin + kRelMargin) * inv;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float d = mag[i] * m, down[2] = {-d, -d}, up[2] = {d, d};
            float z[2];
            mul2(z, v + 2 * i, inv2);
            add2(lo + 2 * i, z, down);
            add2(hi + 2 * i, z, up);
        }
    } else if (rotated) {
        const float inv2[2] = {inv, inv}, m = kAbsMargin * inv;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float z[2];
            mul2(z, v + 2 * i, inv2);
            const float d = mag[i] * m;
            const float up[2] = {fmaf(fabsf(z[0]), kRelMargin, d), fmaf(fabsf(z[1]), kRelMargin, d)};
            add2(hi + 2 * i, z, up);
            lo[2 * i] = z[0] - up[0];
            lo[2 * i + 1] = z[1] - up[1];
        }
    } else {
        constexpr float eps = kAbsMargin + kRelMargin;
        const float a = fmaf(inv, -eps, inv), b = fmaf(inv, eps, inv), a2[2] = {a, a}, b2[2] = {b, b};
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            mul2(lo + j, v + j, a2);
            mul2(hi + j, v + j, b2);
        }
    }
}

// Whether any of a chunk's inputs is not a zero.
__device__ __forceinline__ bool any_nonzero(const float* x) {
    uint32_t bits = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) bits |= __float_as_uint(x[j]);
    return (bits & 0x7fffffffu) != 0u;
}

// One row over LPR = D / 16 lanes (all lanes of the warp call it): norm, rotation, codes and
// scale.  codes, scale: this lane's first word and its row's scales.
template <int LPR, bool FP4, RotMode RM>
__device__ __forceinline__ void quantize_row(const Lane& x, int l, const LaneParams<RM>& p, bool norm, float eps,
                                             void* codes, void* scale, int32_t* st, bool in) {
    constexpr int D = 8 * kC * LPR;
    bool near = p.past;         // not settled in fp32
    float s[kC][2] = {};
#pragma unroll
    for (int c = 0; c < kC; c++)
#pragma unroll
        for (int j = 0; j < 8; j += 2) fma2(s[c], x.v[c] + j, x.v[c] + j, s[c]);
    const float ss = group_sum<LPR>((s[0][0] + s[0][1]) + (s[1][0] + s[1][1]));   // NaNs and infinities show here
    near |= !(ss < kHuge);
    const float ms = fmaf(ss, 1.f / D, eps);
    near |= norm & !(ms > (FP4 ? kLeastMean : kTiny));
    const float r = norm ? rsqrtf(ms) : 1.f;
    Lane v;
    float mag[kC][4], amax[kC];      // of a rotated pair: |v1| + |v2| before the rotation
#pragma unroll
    for (int c = 0; c < kC; c++) {
        const float4 w0 = __ldg(reinterpret_cast<const float4*>(p.weight + 8 * LPR * c));
        const float4 w1 = __ldg(reinterpret_cast<const float4*>(p.weight + 8 * LPR * c + 4));
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int j = 0; j < 8; j += 2) mul2(v.v[c] + j, x.v[c] + j, w + j);
        if (p.rotated(c)) {
            const float4* t = reinterpret_cast<const float4*>(p.table->f32 + p.pair[c]);
            const float4 t0 = t[0], t1 = t[1];
            const float cs[4] = {t0.x, t0.z, t1.x, t1.z}, sn[4] = {t0.y, t0.w, t1.y, t1.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float a = v.v[c][2 * i], b = v.v[c][2 * i + 1];
                mag[c][i] = fabsf(a) + fabsf(b);
                v.v[c][2 * i] = fmaf(a, cs[i], -(b * sn[i]));
                v.v[c][2 * i + 1] = fmaf(a, sn[i], b * cs[i]);
            }
        }
        amax[c] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; j++) amax[c] = fmaxf(amax[c], fabsf(v.v[c][j]));
    }
    RowCodes q;
    bool blank = false;          // e4m3: every product of the row is zero
    if constexpr (FP4) {
#pragma unroll
        for (int c = 0; c < kC; c++) {
            amax[c] = fmaxf(amax[c], __shfl_xor_sync(0xffffffffu, amax[c], 1));
            amax[c] = fmaxf(amax[c], __shfl_xor_sync(0xffffffffu, amax[c], 2));
            const bool zero = amax[c] == 0.f;
            const float top = amax[c] * r;
            const uint32_t ex = __float_as_uint(top) >> 23;
            // the largest magnitude may itself lie next to a power of two
            const float above = fmaf(top, kTopMargin, top), below = fmaf(top, -kTopMargin, top);
            near |= !zero & (!(fminf(amax[c], top) > kTiny) | !(top < kHuge) |
                             ((__float_as_uint(above) ^ __float_as_uint(below)) >> 23 != 0u));
            // a non-finite block is `near`: the bounds only keep the shift in range
            const uint32_t e = zero ? 0u : max(min(ex, 250u), 2u) - 2u;
            q.scale[c] = e;
            q.bad[c] = false;
            const float inv = zero ? 1.f : r * __uint_as_float((254u - e) << 23);     // r * 2^(127 - e)
            float lo[8], hi[8];
            bracket<true>(v.v[c], mag[c], p.rotated(c), inv, lo, hi);
            q.c[c][0] = pack_e2m1x8(lo);
            q.c[c][1] = 0;
            near |= !zero & (pack_e2m1x8(hi) != q.c[c][0]);     // zeros keep their sign in lo
        }
    } else {
        float top = fmaxf(amax[0], amax[1]);
#pragma unroll
        for (int m = 1; m < LPR; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        const bool zero = top == 0.f;
        near |= !zero & (!(fminf(top, top * r) > kTiny) | !(top * r < kHuge));
        blank = zero;
        const float inv = zero ? 1.f : 448.f / top;
#pragma unroll
        for (int c = 0; c < kC; c++) {
            float lo[8], hi[8];
            bracket<false>(v.v[c], mag[c], p.rotated(c), inv, lo, hi);
            const uint2 a = pack_e4m3x8(lo), b = pack_e4m3x8(hi);
            q.c[c][0] = a.x;
            q.c[c][1] = a.y;
            q.scale[c] = __float_as_uint(zero ? 1.f : (top * r) * (1.f / 448.f));
            q.bad[c] = false;
            near |= !zero & ((a.x != b.x) | (a.y != b.y));
        }
    }
    unsigned unsettled = __ballot_sync(0xffffffffu, near | blank);
    if (unsettled) {
        if constexpr (!FP4) {
            if (blank) near |= any_nonzero(x.v[0]) | any_nonzero(x.v[1]);
            unsettled = __ballot_sync(0xffffffffu, near);
        }
        if (unsettled) {
            const RowCodes d = quantize_row_f64<LPR, FP4>(x, p.weight, p.rot(0), p.rot(1), norm, (double)eps);
            // by row: the fp32 scale of a settled neighbour may differ from the fp64 one in its
            // last bits, and a row's result must not depend on the rows beside it
            if (unsettled >> ((threadIdx.x & 31) & ~(LPR - 1)) & ((1u << LPR) - 1u)) {
                q = d;
                if (in && ((FP4 ? l & 3 : l) == 0) && (q.bad[0] | q.bad[1])) flag(st, CSA_DEV_NAN);
            }
        }
    }
    if (!in) return;
    if constexpr (FP4) {
#pragma unroll
        for (int c = 0; c < kC; c++) {
            reinterpret_cast<uint32_t*>(codes)[LPR * c] = q.c[c][0];
            if ((l & 3) == 0) reinterpret_cast<uint8_t*>(scale)[LPR / 4 * c] = (uint8_t)q.scale[c];
        }
    } else {
#pragma unroll
        for (int c = 0; c < kC; c++) reinterpret_cast<uint2*>(codes)[LPR * c] = make_uint2(q.c[c][0], q.c[c][1]);
        if (l == 0) *reinterpret_cast<float*>(scale) = __uint_as_float(q.scale[0]);
    }
}

// Where a lane writes row `dst`: its first word of codes, its (first block's) scale.
template <int LPR, bool FP4>
__device__ __forceinline__ void lane_out(const RowQuant& o, int64_t dst, int l, uint8_t*& codes, uint8_t*& scale) {
    constexpr int D = 8 * kC * LPR;
    codes = o.codes + dst * (FP4 ? D / 2 : D) + l * (FP4 ? 4 : 8);
    scale = FP4 ? o.sf + dst * (D / 32) + (l >> 2) : reinterpret_cast<uint8_t*>(o.scale + dst);
}

// The table of a position by `n` lanes (this one is number i of them): a pair per lane.  The lanes
// that read it synchronise their warp first.
__device__ __forceinline__ void fill_table(RotTable& t, const RopeTable& rt, double pos, int pairs, int i, int n) {
    for (int j = i; j < pairs; j += n) {
        double c, s;
        rotation(pos, rt.freq[j], c, s);
        t.f64[j] = make_double2(c, s);
        t.f32[j] = make_float2((float)c, (float)s);
    }
}

template <int LPR, RotMode RM>
__device__ __forceinline__ LaneParams<RM> lane_params(const float* weight, const RotTable& table, int l, int rope) {
    static_assert(8 * kC * LPR <= kMaxIndexerDim, "a row's channels each have a unit weight");
    LaneParams<RM> p;
    p.weight = (weight ? weight : kOnes.v) + 8 * l;
    p.table = &table;
    p.past = false;
#pragma unroll
    for (int c = 0; c < kC; c++) {
        float w[8];
        load_weight8(p.weight, 8 * LPR * c, w);
#pragma unroll
        for (int j = 0; j < 8; j++) p.past |= !(fabsf(w[j]) < 1.0995116e+12f);   // 2^40, or a NaN
        p.pair[c] = 4 * (l + LPR * c) - (8 * kC * LPR - rope) / 2;
    }
    return p;
}

template <class T, int LPR>
struct RawLane {
    Row8<T> r[kC];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int c = 0; c < kC; c++) r[c].load(p + 8 * LPR * c);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int c = 0; c < kC; c++) r[c].zero();
    }
    __device__ __forceinline__ void get(Lane& x) const {
#pragma unroll
        for (int c = 0; c < kC; c++) r[c].get(x.v[c]);
    }
};

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

template <class T, int LPR, bool FP4, RotMode RM>
__global__ void __launch_bounds__(32 * kWarps, 7) indexer_queries_kernel(const QueryArgs a, const RopeTable rt) {
    __shared__ RotTable tables[kWarps];
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    constexpr int kRows = 32 / LPR;
    const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = task / a.warps_per_token;
    if (t >= a.Q) return;
    const int h0 = (int)(task - t * a.warps_per_token) * a.heads_per_warp;
    const int h1 = min(h0 + a.heads_per_warp, a.H);
    // the row worked on and the one after it; lanes past the last head load the last one again
    const T* src = (const T*)a.q + t * a.st + 8 * l;
    RawLane<T, LPR> cur, nxt;
    cur.load(src + min(h0 + sub, h1 - 1) * a.sh);
    RotTable& table = tables[threadIdx.x >> 5];
    fill_table(table, rt, (double)a.pos[t], a.rope / 2, lane, 32);
    const LaneParams<RM> p = lane_params<LPR, RM>(a.weight, table, l, a.rope);
    __syncwarp();
    uint8_t *codes, *scale;
    lane_out<LPR, FP4>(a.o, t * a.H + h0 + sub, l, codes, scale);
    src += min(h0 + sub + kRows, h1 - 1) * a.sh;
    const int64_t step = kRows * a.sh;
#pragma unroll 1
    for (int hb = h0; hb < h1; hb += kRows) {
        nxt.load(src);
        if (hb + 3 * kRows <= h1) src += step;
        else src += max(min(kRows, h1 - 1 - (hb + sub + kRows)), 0) * a.sh;
        Lane x;
        cur.get(x);
        quantize_row<LPR, FP4, RM>(x, l, p, a.norm, a.eps, codes, scale, a.o.st, hb + sub < h1);
        cur = nxt;
        codes += kRows * 8 * kC * LPR / (FP4 ? 2 : 1);
        scale += kRows * (FP4 ? kC * LPR / 4 : 4);
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
template <class T, int LPR, bool FP4, RotMode RM>
__global__ void __launch_bounds__(32 * kWarps) indexer_append_kernel(const AppendArgs a, const RopeTable rt) {
    constexpr int kRows = 32 / LPR;
    __shared__ RotTable tables[kWarps * kRows];
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    const int64_t it = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRows + sub;
    bool in = it < a.n;
    int64_t dst = 0, pos = 0;
    RawLane<T, LPR> r;
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
        }
    }
    RotTable& table = tables[threadIdx.x / LPR];
    fill_table(table, rt, (double)pos, a.rope / 2, l, LPR);
    const LaneParams<RM> p = lane_params<LPR, RM>(a.weight, table, l, a.rope);
    __syncwarp();
    uint8_t *codes, *scale;
    lane_out<LPR, FP4>(a.o, dst, l, codes, scale);
    Lane x;
    r.get(x);
    quantize_row<LPR, FP4, RM>(x, l, p, a.norm, a.eps, codes, scale, a.o.st, in);
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

template <class T, int LPR, bool FP4, RotMode RM>
cudaError_t run(QueryArgs a, const RopeTable& rt, cudaStream_t stream) {
    split_heads(a.Q, a.H, 32 / LPR, a.heads_per_warp, a.warps_per_token);
    LaunchScope scope(kKIndexerQueries, stream);
    return launch_pdl(indexer_queries_kernel<T, LPR, FP4, RM>,
                      dim3(blocks_of((int64_t)a.Q * a.warps_per_token)), dim3(32 * kWarps), 0, stream,
                      a, rt);
}

template <class T, int LPR, bool FP4, RotMode RM>
cudaError_t run(const AppendArgs& a, const RopeTable& rt, cudaStream_t stream) {
    constexpr int kRows = 32 / LPR;
    LaunchScope scope(kKIndexerAppend, stream);
    return launch_pdl(indexer_append_kernel<T, LPR, FP4, RM>, dim3(blocks_of((a.n + kRows - 1) / kRows)),
                      dim3(32 * kWarps), 0, stream, a, rt);
}

// The rotation of half a 128-channel row or of a whole 64-channel one has kernels of its own.
template <class T, bool FP4, class Args>
cudaError_t run_dims(int D, const Args& a, const RopeTable& rt, cudaStream_t stream) {
    if (D == 128)
        return a.rope == 64 ? run<T, 8, FP4, kRotUpper>(a, rt, stream) : run<T, 8, FP4, kRotAny>(a, rt, stream);
    return a.rope == 64 ? run<T, 4, FP4, kRotAll>(a, rt, stream) : run<T, 4, FP4, kRotAny>(a, rt, stream);
}

template <class Args>
cudaError_t run_types(int dtype, int fmt, int D, const Args& a, const RopeTable& rt, cudaStream_t stream) {
    const bool fp4 = fmt == CSA_IDX_MXFP4;
    if (dtype == CSA_DT_BF16)
        return fp4 ? run_dims<__nv_bfloat16, true>(D, a, rt, stream) : run_dims<__nv_bfloat16, false>(D, a, rt, stream);
    if (dtype == CSA_DT_F16)
        return fp4 ? run_dims<__half, true>(D, a, rt, stream) : run_dims<__half, false>(D, a, rt, stream);
    return fp4 ? run_dims<float, true>(D, a, rt, stream) : run_dims<float, false>(D, a, rt, stream);
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

cudaError_t launch_indexer_queries(const void* q, int dtype, int64_t st, int64_t sh, const int32_t* pos,
                                   const float* weight, int norm, int rope, float theta, float eps,
                                   int Q, int H, int D, int fmt, uint8_t* codes, void* scale,
                                   int32_t* dev_status, cudaStream_t stream) {
    QueryArgs a{q, weight, pos, st, sh, Q, H, rope, norm, 0, 0, eps,
                RowQuant{codes, (float*)scale, (uint8_t*)scale, dev_status}};
    const RopeTable& rt = rope_table(rope, theta);
    return run_types(dtype, fmt, D, a, rt, stream);
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
    return run_types(dtype, fmt, D, a, rt, stream);
}

}  // namespace csa
