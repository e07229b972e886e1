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
    const void* q;
    const void* k;
    void* q_out;
    void* k_out;
    const float* q_weight;
    const float* k_weight;
    const int32_t* pos;
    int64_t q_st, q_sh, k_st, k_sh, qo_st, qo_sh, ko_st, ko_sh;   // strides, elements
    int T, H, Hk, D, rope, norm;
    int heads_per_warp, warps_per_token;
    float eps;
};

// LPR lanes a row, C chunks of 8 channels a lane (chunk c of lane l: channels 8 (l + LPR c)).
template <class T, int LPR, int C>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_kernel(const QkArgs a, const RopeTable rt) {
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    constexpr int kRows = 32 / LPR;
    const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = task / a.warps_per_token;
    if (t >= a.T) return;
    const int h0 = (int)(task % a.warps_per_token) * a.heads_per_warp;
    const int heads = a.H + a.Hk;
    const int h1 = min(h0 + a.heads_per_warp, heads);
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
    for (int hb = h0; hb < h1; hb += kRows) {
        const int h = hb + sub;
        const bool in = h < h1;
        const bool isq = h < a.H;
        const T* src = isq ? (const T*)a.q + t * a.q_st + h * a.q_sh
                           : (const T*)a.k + t * a.k_st + (h - a.H) * a.k_sh;
        Row8<T> r[C];
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int ch = 8 * (l + LPR * c);
            r[c].zero();
            if (in && ch < a.D) r[c].load(src + ch);
        }
#pragma unroll
        for (int c = 0; c < C; c++) {
            float f[8];
            r[c].get(f);
#pragma unroll
            for (int j = 0; j < 8; j++) ss = fmaf(f[j], f[j], ss);
        }
        float rs = 1.f;
        if (a.norm) rs = rsqrtf(group_sum<LPR>(ss) / (float)a.D + a.eps);
        if (!in) continue;
        const float* w = isq ? a.q_weight : a.k_weight;
        T* dst = isq ? (T*)a.q_out + t * a.qo_st + h * a.qo_sh
                     : (T*)a.k_out + t * a.ko_st + (h - a.H) * a.ko_sh;
#pragma unroll
        for (int c = 0; c < C; c++) {
            const int ch = 8 * (l + LPR * c);
            if (ch >= a.D) continue;
            float f[8];
            r[c].get(f);
            if (w) {
                const float4 w0 = __ldg(reinterpret_cast<const float4*>(w + ch));
                const float4 w1 = __ldg(reinterpret_cast<const float4*>(w + ch + 4));
                const float ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int j = 0; j < 8; j++) f[j] *= rs * ww[j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++) f[j] *= rs;
            }
#pragma unroll
            for (int p = 0; p < 4; p++) {
                if (ch + 2 * p < lo) continue;
                const float x = f[2 * p], y = f[2 * p + 1];
                f[2 * p] = x * cs[c][p] - y * sn[c][p];
                f[2 * p + 1] = x * sn[c][p] + y * cs[c][p];
            }
            Row8<T> o;
            o.set(f);
            o.store(dst + ch);
        }
    }
    __threadfence();   // visible before the next kernel's reads ahead of its own wait
}

// ---- rows in the indexer's stored formats ----------------------------------------------------
// The arithmetic is fp64 from the input's bits to the code: an e4m3 or e2m1 code (and a
// block's power-of-two scale) next to a rounding border would depend on the order of fp32
// sums, and the index sets with it.  In fp64 the codes are those of the definition.
struct RowQuant {
    uint8_t* codes;    // rows of D (e4m3) or D / 2 (e2m1) bytes
    float* scale;      // e4m3: one fp32 per row
    uint8_t* sf;       // MXFP4: D / 32 UE8M0 bytes per row
    int32_t* st;
};

// One row over LPR = D / 8 lanes (all lanes of the warp call it): norm, rotation (cs, sn of
// this lane's 4 pairs), codes and scale to row `dst`.
template <int LPR, bool FP4>
__device__ __forceinline__ void quantize_row(const float* x, int l, const double* cs,
                                             const double* sn, bool rot, const float* w, bool norm,
                                             double eps, const RowQuant& o, int64_t dst, bool in) {
    constexpr int D = 8 * LPR;
    double y[8];
    double r = 1.0;
    if (norm) {
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            y[j] = (double)x[j];
            ss = fma(y[j], y[j], ss);
        }
        r = rsqrt(group_sum<LPR>(ss) * (1.0 / D) + eps);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = (double)x[j];
    }
#pragma unroll
    for (int j = 0; j < 8; j++) y[j] *= r * (double)w[j];
    if (rot) {
#pragma unroll
        for (int p = 0; p < 4; p++) {
            const double u = y[2 * p], v = y[2 * p + 1];
            y[2 * p] = u * cs[p] - v * sn[p];
            y[2 * p + 1] = u * sn[p] + v * cs[p];
        }
    }
    if constexpr (FP4) {
        // the block's scale needs the exponent of its largest magnitude only
        int top = 0;
#pragma unroll
        for (int j = 0; j < 8; j++) top = max(top, __double2hiint(y[j]) & 0x7fffffff);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = (top >> 20) - 1023;              // floor(log2(amax)); -1023 for zeros
        const bool bad = ex > 129;                      // not finite, or past the scales' range
        const int e = bad ? 255 : max(ex - 2 + 127, 0);
        const double inv = __hiloint2double((1023 + 127 - (bad ? 127 : e)) << 20, 0);
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] = f64_to_f32_odd(bad ? 0.0 : y[j] * inv);
        const uint32_t c = pack_e2m1x8(f);
        if (in) {
            reinterpret_cast<uint32_t*>(o.codes)[dst * (D / 8) + l] = c;
            if ((l & 3) == 0) {
                o.sf[dst * (D / 32) + (l >> 2)] = (uint8_t)e;
                if (bad) flag(o.st, CSA_DEV_NAN);
            }
        }
    } else {
        double top = 0.0;
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            top = fmax(top, fabs(y[j]));
            nan |= y[j] != y[j];
        }
#pragma unroll
        for (int s = LPR / 2; s > 0; s >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, s));
        float scale = (float)(top * (1.0 / 448.0));
        const unsigned group = (LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u)) << ((threadIdx.x & 31) & ~(LPR - 1));
        const bool bad = (__ballot_sync(0xffffffffu, nan) & group) != 0 || !(scale <= 3.402823466e38f);
        if (!(scale > 0.f)) scale = 1.f;
        // y / scale: the product with the rounded reciprocal, mended once by its remainder, so
        // that a quotient fp64 holds (a tie between two codes, say) comes out exactly
        const double sd = (double)scale, inv = 1.0 / sd;
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const double z = y[j] * inv;
            f[j] = f64_to_f32_odd(bad ? 0.0 : fma(fma(-z, sd, y[j]), inv, z));
        }
        const uint2 c = pack_e4m3x8(f);
        if (in) {
            reinterpret_cast<uint2*>(o.codes)[dst * LPR + l] = c;
            if (l == 0) {
                o.scale[dst] = bad ? __int_as_float(0x7fffffff) : scale;
                if (bad) flag(o.st, CSA_DEV_NAN);
            }
        }
    }
}

template <class T>
__device__ __forceinline__ void load_weight(const float* weight, int ch, float* w) {
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

struct QueryArgs {
    const void* q;
    const float* weight;
    const int32_t* pos;
    int64_t st, sh;           // strides of q, elements
    int Q, H, rope, norm;
    int heads_per_warp, warps_per_token;
    double eps;
    RowQuant o;
};

template <class T, int LPR, bool FP4>
__global__ void __launch_bounds__(32 * kWarps) indexer_queries_kernel(const QueryArgs a, const RopeTable rt) {
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    constexpr int kRows = 32 / LPR, D = 8 * LPR;
    const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = task / a.warps_per_token;
    if (t >= a.Q) return;
    const int h0 = (int)(task % a.warps_per_token) * a.heads_per_warp;
    const int h1 = min(h0 + a.heads_per_warp, a.H);
    const T* src = (const T*)a.q + t * a.st + 8 * l;
    float w[8];
    load_weight<T>(a.weight, 8 * l, w);
    const bool rot = 8 * l >= D - a.rope;
    double cs[4], sn[4];
    if (rot) {
        const double pos = (double)a.pos[t];
#pragma unroll
        for (int p = 0; p < 4; p++) rotation(pos, rt.freq[4 * l + p - (D - a.rope) / 2], cs[p], sn[p]);
    }
    Row8<T> cur, nxt;
    cur.zero();
    if (h0 + sub < h1) cur.load(src + (h0 + sub) * a.sh);
    for (int hb = h0; hb < h1; hb += kRows) {
        const int h = hb + sub;
        nxt.zero();
        if (h + kRows < h1) nxt.load(src + (h + kRows) * a.sh);
        float x[8];
        cur.get(x);
        quantize_row<LPR, FP4>(x, l, cs, sn, rot, w, a.norm, a.eps, a.o, t * a.H + h, h < h1);
        cur = nxt;
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
    double eps;
    RowQuant o;
};

// One listed entry per row: its position is the block end (i + 1) m - 1.
template <class T, int LPR, bool FP4>
__global__ void __launch_bounds__(32 * kWarps) indexer_append_kernel(const AppendArgs a, const RopeTable rt) {
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    constexpr int kRows = 32 / LPR, D = 8 * LPR;
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
            r.zero();
        }
    }
    float w[8], x[8];
    load_weight<T>(a.weight, 8 * l, w);
    const bool rot = 8 * l >= D - a.rope;
    double cs[4], sn[4];
    if (rot) {
#pragma unroll
        for (int p = 0; p < 4; p++) rotation((double)pos, rt.freq[4 * l + p - (D - a.rope) / 2], cs[p], sn[p]);
    }
    r.get(x);
    quantize_row<LPR, FP4>(x, l, cs, sn, rot, w, a.norm, a.eps, a.o, dst, in);
    __threadfence();
}

// theta^(-2j / rope) for the pairs j of the rotated channels.
RopeTable rope_table(int rope, double theta) {
    RopeTable t = {};
    for (int j = 0; j < rope / 2; j++) t.freq[j] = pow(theta, -2.0 * j / rope);
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
    split_heads(a.T, a.H + a.Hk, 32 / LPR, a.heads_per_warp, a.warps_per_token);
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
    QkArgs a{q.x, k.x, q.out, k.out, q.weight, k.weight, pos, q.st, q.sh, k.st, k.sh, q.ost, q.osh,
             k.ost, k.osh, T, q.heads, k.heads, D, rope, norm, 0, 0, eps};
    const RopeTable rt = rope_table(rope, theta);
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
    QueryArgs a{q, weight, pos, st, sh, Q, H, rope, norm, 0, 0, (double)eps,
                RowQuant{codes, (float*)scale, (uint8_t*)scale, dev_status}};
    const RopeTable rt = rope_table(rope, theta);
    CSA_ROWS_DISPATCH(run_queries, a);
}

cudaError_t launch_indexer_append(const void* k, int dtype, int64_t ld, const int64_t* seq_len,
                                  const EntryRows& er, const int32_t* item_seq,
                                  const int32_t* item_ent, int64_t n, int64_t ent_rows, int B, int m,
                                  const float* weight, int norm, int rope, float theta, float eps,
                                  int D, int fmt, uint8_t* codes, void* scale, int32_t* dev_status,
                                  cudaStream_t stream) {
    AppendArgs a{k, weight, ld, seq_len, er, item_seq, item_ent, n, ent_rows, B, m, rope, norm,
                 (double)eps, RowQuant{codes, (float*)scale, (uint8_t*)scale, dev_status}};
    const RopeTable rt = rope_table(rope, theta);
    CSA_ROWS_DISPATCH(run_append, a);
}

}  // namespace csa
