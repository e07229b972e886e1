// MXFP4 product on the 5th-generation tensor cores: out[m, n] = sum_k A[m, k] B[n, k]
// ("DeepSeek-V4 深度分析报告" 3.4: MXFP4 weights and activations; batch-invariant GEMMs without
// split-K, 3.3).
//
// Two kernels, one structure: a decode step's few tokens lie on the accumulator's columns and the
// weight's rows on its 128 lanes, so that the weight streams 128 (or RT) rows at a time; a
// batch of more than 96 has its tokens on the lanes and 64 to 256 weight rows on the columns.
// In both a result is summed over K ascending, K = 64 an instruction, so that its bits do
// not depend on the batch (tested over both kernels and every tile width).
//
//   warp 0         TMA producer: per stage of K = 256 the rows of both operands (128 bytes
//                  each, 128-byte swizzle) and their scale tiles (bulk copies: the tiled
//                  scale layout is the tensor cores' own);
//   warp 1         TMEM allocation; it copies the scales into TMEM (one slot of columns
//                  per stage: a slot is refilled only after the MMAs that read it) and
//                  issues tcgen05.mma kind::mxf4.block_scale;
//   other warps    epilogue (see the kernels).
// Warps 0 and 1 walk their loops converged and one elected lane issues: from a branch of one lane
// each tcgen05 instruction took some 70 clocks to issue (a stage has up to ten).
//
// Every wait is bounded; a timeout aborts the CTA, drains its copies and MMAs, frees TMEM and
// reports CSA_DEV_TIMEOUT.
#include <atomic>

#include "launchers.cuh"
#include "rows.cuh"
#include "sm100.cuh"

namespace csa {

namespace {

constexpr int kThreads = 192;
constexpr int kStageK = 256;             // elements of K per stage: 128 bytes a row
constexpr int kRowB = kStageK / 2;
constexpr int kWTile = 128 * kRowB;      // a stage's weight rows (the MMA reads 128)
constexpr int kSfTile = 512;             // scales of 128 rows x 4 blocks

// A stage: 128 rows for the accumulator's lanes and NT for its columns, with their scale tiles.
template <int NT>
constexpr int column_tiles() { return NT > 128 ? 2 : 1; }   // 128-row scale tiles of the columns
template <int NT>
constexpr int stage_bytes() { return kWTile + NT * kRowB + 2 * kSfTile * (1 + column_tiles<NT>()); }
template <int NT>
constexpr int stages() {
    const int s = (220 * 1024) / stage_bytes<NT>();
    return s > 10 ? 10 : s;
}
// TMEM columns: NT of accumulator, then per stage 8 of the lanes' scales and 8 per column tile.
template <int NT>
constexpr int sf_cols() { return 8 * (1 + column_tiles<NT>()); }
template <int NT>
constexpr uint32_t tmem_cols() {
    const int c = NT + stages<NT>() * sf_cols<NT>();
    return c <= 128 ? 128u : c <= 256 ? 256u : 512u;
}

// One lane of a converged warp, the same each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
    return p != 0;
}

// A tile of shared memory to global memory by the TMA unit (rows and bytes outside the map are
// dropped), in a bulk group of its own; the waits are for the issuing lane's groups: all read
// from shared memory, or all written.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\t"
        "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(sm100::smem_addr(src)), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void bulk_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

struct GemmArgs {
    const uint8_t* a_sf;
    const uint8_t* b_sf;
    void* out;
    int64_t ld;
    int32_t* st;
    int M, N, K, dtype;
    int kt128;        // scale tiles along K
};

__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// ---- tokens on the columns -----------------------------------------------------------------
// One CTA per RT weight rows (NT >= M): it keeps up to 10 stages in flight and has no second
// tile.  Four epilogue warps: a thread holds one output feature and walks the tokens, the 32
// lanes of a warp writing consecutive features (the type chosen outside the walk and one running
// pointer: 64 tokens 7.1 -> 5.6 us).  An MMA of 128 lanes takes some 70 clocks however few
// columns it has and a scale copy some 40, so at RT = 64 a stage's 8 KB of weights take about
// 450 clocks: 8 tokens x 8192 x 2048 in 5.3 us, of which 3.2 are the launch and one stage (8.9 MB:
// 1.4 us at the copy rate).
template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
    mxfp4_gemm_kernel(const __grid_constant__ CUtensorMap tmap_b,
                      const __grid_constant__ CUtensorMap tmap_a, const GemmArgs g, const int RT) {
    using namespace sm100;
    constexpr int S = stages<NT>();
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint8_t* sW = smem;                                  // [S][128 rows x 128 B]
    uint8_t* sX = sW + S * kWTile;                       // [S][NT rows x 128 B]
    uint8_t* sSw = sX + S * NT * kRowB;                  // [S][2][512]
    uint8_t* sSx = sSw + S * 2 * kSfTile;                // [S][2][512]
    uint64_t* full = reinterpret_cast<uint64_t*>(sSx + S * 2 * kSfTile);
    uint64_t* empty = full + S;
    uint64_t* accfull = empty + S;
    uint64_t* drain = accfull + 1;
    uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_smem + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = blockIdx.x * RT;
    const int row0 = n0 & 127;                // the tile's first lane: its place in its scale tile
    const int nk = (g.K + kStageK - 1) / kStageK;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(accfull, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        mbar_fence_init();
        prefetch_tmap(&tmap_b);
        prefetch_tmap(&tmap_a);
    }
    if (warp == 1) {
        tmem_alloc(tmem_base_smem, tmem_cols<NT>());
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_base_smem;
    pdl_wait();

    if (warp == 0) {
        const uint8_t* bsf = g.b_sf + (int64_t)(n0 >> 7) * g.kt128 * kSfTile;
        int n_load = 0;
        for (int i = 0; i < nk; i++) {
            const int s = i % S;
            if (!mbar_wait_warp(&empty[s], ((i / S) & 1) ^ 1, abort_flag, g.st)) break;
            const uint32_t sfb = (uint32_t)min(2, g.kt128 - 2 * i) * kSfTile;
            if (elect_one()) {
                mbar_arrive_expect_tx(&full[s], RT * kRowB + NT * kRowB + 2 * sfb);
                tma_load_2d(sW + s * kWTile + row0 * kRowB, &tmap_b, &full[s], i * kRowB, n0);
                tma_load_2d(sX + s * NT * kRowB, &tmap_a, &full[s], i * kRowB, 0);
                bulk_load(sSw + s * 2 * kSfTile, bsf + (int64_t)2 * i * kSfTile, sfb, &full[s]);
                bulk_load(sSx + s * 2 * kSfTile, g.a_sf + (int64_t)2 * i * kSfTile, sfb, &full[s]);
            }
            __syncwarp();
            n_load++;
        }
        if (lane == 0)
            for (int s = 0; s < S; s++) {
                const int cnt = n_load / S + (s < n_load % S ? 1 : 0);
                if (cnt) mbar_drain(&full[s], (cnt - 1) & 1, g.st);
            }
        __syncwarp();
    } else if (warp == 1) {
        // the whole warp walks the loop, so that the operands of one elected lane's instructions
        // are uniform
        bool ok = true;
        for (int i = 0; i < nk; i++) {
            const int s = i % S;
            if (!mbar_wait_warp(&full[s], (i / S) & 1, abort_flag, g.st)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int kleft = g.K - i * kStageK;
            const uint32_t sfw = tmem + (uint32_t)(NT + s * sf_cols<NT>()), sfx = sfw + 8;
            const uint64_t wd = smem_desc_k_sw128(sW + s * kWTile);
            const uint64_t xd = smem_desc_k_sw128(sX + s * NT * kRowB);
            const uint64_t swd = smem_desc_rows16(sSw + s * 2 * kSfTile);
            const uint64_t sxd = smem_desc_rows16(sSx + s * 2 * kSfTile);
            if (elect_one()) {
#pragma unroll
                for (int kt = 0; kt < 2; kt++)
                    if (128 * kt < kleft) {
                        tmem_cp_32x128b_x4(sfw + 4 * kt, swd + (kt * kSfTile >> 4));
                        tmem_cp_32x128b_x4(sfx + 4 * kt, sxd + (kt * kSfTile >> 4));
                    }
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (64 * j < kleft) {
                        const uint32_t id = 2 * (j & 1), sel = id << 30;
                        mma_mxf4(tmem, wd + 2 * j, xd + 2 * j, instr_desc_mxf4(128, NT, id, id),
                                 (sfw + 4 * (j >> 1)) | sel, (sfx + 4 * (j >> 1)) | sel,
                                 i > 0 || j > 0 ? 1u : 0u);
                    }
                mma_commit(&empty[s]);
            }
            __syncwarp();
        }
        if (elect_one()) {
            if (ok) mma_commit(accfull);
            mma_commit(drain);
            mbar_drain(drain, 0, g.st);
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;       // accumulator lane
        const int n = n0 - row0 + r;
        if (mbar_wait_warp(accfull, 0, abort_flag, g.st)) {
            tc_fence_after();
            const bool in = r >= row0 && r < row0 + RT && n < g.N;
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16);
            const auto walk = [&](auto* out) {
                out += n;
                for (int c = 0; c < g.M; c += 16) {
                    uint32_t d[16];
                    tmem_ld16(taddr + (uint32_t)c, d);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        if (in && c + j < g.M) {
                            put(out, __uint_as_float(d[j]));
                            out += g.ld;
                        }
                }
            };
            if (g.dtype == CSA_DT_BF16) walk(reinterpret_cast<__nv_bfloat16*>(g.out));
            else if (g.dtype == CSA_DT_F16) walk(reinterpret_cast<__half*>(g.out));
            else walk(reinterpret_cast<float*>(g.out));
            tc_fence_before();
        }
        __threadfence();   // visible before the next kernel's reads ahead of its own wait
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, tmem_cols<NT>());
    }
}

// ---- tokens on the lanes -------------------------------------------------------------------
// Persistent: CTA c takes the 128-token x CT-feature tiles c, c + grid, ... (tokens fastest, so
// that neighbours share the weight's rows in L2).  Eight epilogue warps, two per lane quarter,
// take the accumulator into registers at once (CT / 2 columns a thread) and hand it back, so
// the next tile's MMAs wait for those loads only; the conversion, a 2 KB transposition per warp
// in shared memory and the stores of 64 contiguous bytes a row (TMA where rows allow) run beside
// them.  8192 x 8192 x 2048 to bf16: 66 us, 4.2 PFLOP/s, at 1965 MHz (bursts of 100 calls); 77 us in a
// loop, which the power cap holds at 1590 MHz and 987 W.  Without the stores 50, whose traffic
// (134 MB) competes with the operands' loads; 5.5 PFLOP/s per further stage.  Tried and slower:
// two accumulators of 192 columns (75 us), scales written to TMEM by four warps instead of
// copies in the MMA warp's stream (71), streaming stores (69), features fastest (71).
constexpr int kWideThreads = 320;
constexpr int kStageRowB = 64;           // bytes of a row per transposition

template <int CT>
constexpr int wide_stages() {
    const int s = (224 * 1024 - 8 * 32 * kStageRowB) / stage_bytes<CT>();
    return s > 8 ? 8 : s;
}
template <int CT>
constexpr int wide_accs() { return CT <= 128 ? 2 : 1; }
template <int CT>
constexpr uint32_t wide_tmem_cols() {
    const int c = wide_accs<CT>() * CT + wide_stages<CT>() * sf_cols<CT>();
    return c <= 128 ? 128u : c <= 256 ? 256u : 512u;
}

template <class T>
__device__ __forceinline__ void pack16(const uint32_t* d, uint4& v) {   // 16 bytes of T from fp32 bits
    if constexpr (sizeof(T) == 4) {
        v = make_uint4(d[0], d[1], d[2], d[3]);
    } else {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] = __uint_as_float(d[j]);
        Row8<T> r;
        r.set(f);
        v = r.r;
    }
}

template <class T, int CT>
__global__ void __launch_bounds__(kWideThreads, 1)
    mxfp4_gemm_wide_kernel(const __grid_constant__ CUtensorMap tmap_a,
                           const __grid_constant__ CUtensorMap tmap_b,
                           const __grid_constant__ CUtensorMap tmap_out, const GemmArgs g, const int mtiles,
                           const int tiles, const int tma_out) {
    using namespace sm100;
    constexpr int S = wide_stages<CT>(), kTT = column_tiles<CT>(), kAcc = wide_accs<CT>();
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint8_t* sA = smem;                                  // [S][128 tokens x 128 B]
    uint8_t* sB = sA + S * kWTile;                       // [S][CT features x 128 B]
    uint8_t* sSa = sB + S * CT * kRowB;                  // [S][2][512]
    uint8_t* sSb = sSa + S * 2 * kSfTile;                // [S][kTT][2][512]
    uint8_t* sOut = sSb + S * kTT * 2 * kSfTile;         // [8][32 x 64 B]
    uint64_t* full = reinterpret_cast<uint64_t*>(sOut + 8 * 32 * kStageRowB);
    uint64_t* empty = full + S;
    uint64_t* accfull = empty + S;
    uint64_t* accempty = accfull + kAcc;
    uint64_t* drain = accempty + kAcc;
    uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_smem + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nk = (g.K + kStageK - 1) / kStageK;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < kAcc; i++) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accempty[i], 8);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        mbar_fence_init();
        prefetch_tmap(&tmap_a);
        prefetch_tmap(&tmap_b);
    }
    if (warp == 1) {
        tmem_alloc(tmem_base_smem, wide_tmem_cols<CT>());
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_base_smem;
    pdl_wait();

    if (warp == 0) {
        int s = 0, n_load = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
            const int m0 = (tile % mtiles) * 128, n0 = (tile / mtiles) * CT;
            const uint8_t* asf = g.a_sf + (int64_t)(m0 >> 7) * g.kt128 * kSfTile;
            const uint8_t* bsf = g.b_sf + (int64_t)(n0 >> 7) * g.kt128 * kSfTile;
            const int tt = kTT == 2 && n0 + 128 < g.N ? 2 : 1;       // weight scale tiles that exist
            for (int i = 0; i < nk; i++) {
                if (!mbar_wait_warp(&empty[s], phase ^ 1, abort_flag, g.st)) {
                    ok = false;
                    break;
                }
                const uint32_t sfb = (uint32_t)min(2, g.kt128 - 2 * i) * kSfTile;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&full[s], 128 * kRowB + CT * kRowB + sfb * (1 + tt));
                    tma_load_2d(sA + s * kWTile, &tmap_a, &full[s], i * kRowB, m0);
                    tma_load_2d(sB + s * CT * kRowB, &tmap_b, &full[s], i * kRowB, n0);
                    bulk_load(sSa + s * 2 * kSfTile, asf + (int64_t)2 * i * kSfTile, sfb, &full[s]);
                    for (int t = 0; t < tt; t++)
                        bulk_load(sSb + (s * kTT + t) * 2 * kSfTile,
                                  bsf + ((int64_t)t * g.kt128 + 2 * i) * kSfTile, sfb, &full[s]);
                }
                __syncwarp();
                n_load++;
                if (++s == S) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        if (lane == 0)
            for (int i = 0; i < S; i++) {
                const int cnt = n_load / S + (i < n_load % S ? 1 : 0);
                if (cnt) mbar_drain(&full[i], (cnt - 1) & 1, g.st);
            }
        __syncwarp();
    } else if (warp == 1) {
        int s = 0, n_tile = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x, n_tile++) {
            const int acc = n_tile % kAcc;
            // a 64-feature tile may begin in the middle of its scale tile: 32 rows a column
            const uint32_t sf_shift = CT < 128 ? (uint32_t)((tile / mtiles) * CT & 127) >> 5 : 0u;
            const uint32_t d = tmem + (uint32_t)(acc * CT);
            if (!mbar_wait_warp(&accempty[acc], ((n_tile / kAcc) & 1) ^ 1, abort_flag, g.st)) break;
            tc_fence_after();
            for (int i = 0; i < nk; i++) {
                if (!mbar_wait_warp(&full[s], phase, abort_flag, g.st)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int kleft = g.K - i * kStageK;
                const uint32_t sfa = tmem + (uint32_t)(kAcc * CT + s * sf_cols<CT>()), sfb = sfa + 8;
                const uint64_t ad = smem_desc_k_sw128(sA + s * kWTile);
                const uint64_t bd = smem_desc_k_sw128(sB + s * CT * kRowB);
                const uint64_t sad = smem_desc_rows16(sSa + s * 2 * kSfTile);
                const uint64_t sbd = smem_desc_rows16(sSb + s * kTT * 2 * kSfTile);
                if (elect_one()) {
#pragma unroll
                    for (int kt = 0; kt < 2; kt++)
                        if (128 * kt < kleft) {
                            tmem_cp_32x128b_x4(sfa + 4 * kt, sad + (kt * kSfTile >> 4));
#pragma unroll
                            for (int t = 0; t < kTT; t++)
                                tmem_cp_32x128b_x4(sfb + 4 * (kt * kTT + t), sbd + ((t * 2 + kt) * kSfTile >> 4));
                        }
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        if (64 * j < kleft) {
                            const uint32_t id = 2 * (j & 1), sel = id << 30;
                            mma_mxf4(d, ad + 2 * j, bd + 2 * j, instr_desc_mxf4(128, CT, id, id),
                                     (sfa + 4 * (j >> 1)) | sel, (sfb + 4 * kTT * (j >> 1) + sf_shift) | sel,
                                     i > 0 || j > 0 ? 1u : 0u);
                        }
                    mma_commit(&empty[s]);
                }
                __syncwarp();
                if (++s == S) {
                    s = 0;
                    phase ^= 1;
                }
            }
            if (ok && elect_one()) mma_commit(&accfull[acc]);
            __syncwarp();
        }
        if (elect_one()) {
            mma_commit(drain);
            mbar_drain(drain, 0, g.st);
        }
        __syncwarp();
    } else {
        constexpr int kCols = CT / 2;                        // columns of this warp
        constexpr int kPiece = 16 / (int)sizeof(T);          // elements of 16 bytes
        constexpr int kChunk = kStageRowB / (int)sizeof(T);  // columns per transposition
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        uint8_t* stage = sOut + (warp - 2) * 32 * kStageRowB;
        T* out = reinterpret_cast<T*>(g.out);
        const bool vec = (reinterpret_cast<uintptr_t>(g.out) | (uintptr_t)(g.ld * (int64_t)sizeof(T))) % 16 == 0;
        int n_tile = 0;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, n_tile++) {
            const int acc = n_tile % kAcc;
            if (!mbar_wait_warp(&accfull[acc], (n_tile / kAcc) & 1, abort_flag, g.st)) break;
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * CT + half * kCols);
            uint32_t d[kCols];
#pragma unroll
            for (int c = 0; c < kCols; c += 32) tmem_ld32(taddr + c, d + c);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&accempty[acc]);
            const int m0 = (tile % mtiles) * 128 + quarter * 32, n0 = (tile / mtiles) * CT + half * kCols;
#pragma unroll
            for (int c = 0; c < kCols; c += kChunk) {
                // lane = token row: its 4 pieces of 16 bytes, spread over the banks
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    uint4 v;
                    pack16<T>(d + c + p * kPiece, v);
                    *reinterpret_cast<uint4*>(stage + lane * kStageRowB + ((p ^ ((lane >> 1) & 3)) << 4)) = v;
                }
                if (tma_out) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (m0 < g.M && n0 + c < g.N) {
                        if (elect_one()) tma_store_2d(&tmap_out, stage, (n0 + c) * (int)sizeof(T), m0);
                    }
                    bulk_store_wait_read();
                    __syncwarp();
                    continue;
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int r = i * 8 + (lane >> 2), p = lane & 3;
                    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * kStageRowB + ((p ^ ((r >> 1) & 3)) << 4));
                    const int n = n0 + c + p * kPiece;
                    if (m0 + r < g.M && n < g.N) {
                        T* o = out + (int64_t)(m0 + r) * g.ld + n;
                        if (vec && n + kPiece <= g.N) {
                            *reinterpret_cast<uint4*>(o) = v;
                        } else {
                            const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
                            for (int j = 0; j < kPiece; j++)
                                if (n + j < g.N) o[j] = e[j];
                        }
                    }
                }
                __syncwarp();
            }
        }
        bulk_store_wait_all();
        __threadfence();   // visible before the next kernel's reads ahead of its own wait
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, wide_tmem_cols<CT>());
    }
}

template <int CT>
size_t wide_smem_bytes() {
    return 1024 + (size_t)wide_stages<CT>() * stage_bytes<CT>() + 8 * 32 * kStageRowB +
           (2 * wide_stages<CT>() + 2 * wide_accs<CT>() + 1) * 8 + 16;
}

template <int NT>
size_t smem_bytes() {
    return 1024 + (size_t)stages<NT>() * stage_bytes<NT>() + (2 * stages<NT>() + 2) * 8 + 16;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Row-major [rows x row_bytes] byte matrix, boxes of box_rows x 128 bytes, 128-byte swizzle;
// bytes past a row or the last row read as zeros.
bool make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t row_bytes, uint32_t box_rows,
              uint64_t pitch = 0, uint32_t box_bytes = kRowB,
              CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    EncodeFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {row_bytes, rows};
    const cuuint64_t strides[1] = {pitch ? pitch : row_bytes};
    const cuuint32_t box[2] = {box_bytes, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    auto encode = [&] {
        return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
                   estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (encode()) return true;
    // a host thread that has made no runtime call yet has no current context, which the driver's
    // call needs: make the device's current and try again
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}

// Raises a kernel's shared-memory limit once per device (`done`: a bit per device).
template <class Kernel>
cudaError_t allow_smem(Kernel* kernel, size_t bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <int NT>
cudaError_t run(const uint8_t* a, const uint8_t* b, const GemmArgs& g, int RT, cudaStream_t stream) {
    CUtensorMap mb, ma;
    if (!make_map(&mb, b, (uint64_t)g.N, (uint64_t)g.K / 2, (uint32_t)RT) ||
        !make_map(&ma, a, (uint64_t)g.M, (uint64_t)g.K / 2, (uint32_t)NT))
        return cudaErrorInvalidValue;
    const size_t sm = smem_bytes<NT>();
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(mxfp4_gemm_kernel<NT>, sm, done);
    if (e != cudaSuccess) return e;
    LaunchScope scope(kKMxMatmul, stream);
    return launch_pdl(mxfp4_gemm_kernel<NT>, dim3((g.N + RT - 1) / RT),
                      dim3(kThreads), sm, stream, mb, ma, g, RT);
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

template <class T, int CT>
cudaError_t run_wide(const uint8_t* a, const uint8_t* b, const GemmArgs& g, int sms, cudaStream_t stream) {
    CUtensorMap mb, ma, mo = {};
    if (!make_map(&mb, b, (uint64_t)g.N, (uint64_t)g.K / 2, (uint32_t)CT) ||
        !make_map(&ma, a, (uint64_t)g.M, (uint64_t)g.K / 2, 128u))
        return cudaErrorInvalidValue;
    // The TMA unit stores where it can: rows 16-byte aligned and whole 16-byte pieces (it writes a
    // row's last piece whole, past the row's end), byte columns within an int32.  512 x 8192 x
    // 2048: 7.9 us, with the threads' own stores 8.4; 128 x 8192 x 2048: 6.2 and 5.9.
    const uint64_t pitch = (uint64_t)g.ld * sizeof(T);
    const int tma_out = (reinterpret_cast<uintptr_t>(g.out) | pitch | (uint64_t)g.N * sizeof(T)) % 16 == 0 &&
                        (uint64_t)g.N * sizeof(T) < (1ull << 31) && pitch < (1ull << 40);
    if (tma_out && !make_map(&mo, g.out, (uint64_t)g.M, (uint64_t)g.N * sizeof(T), 32u, pitch, kStageRowB,
                             CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    const size_t sm = wide_smem_bytes<CT>();
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(mxfp4_gemm_wide_kernel<T, CT>, sm, done);
    if (e != cudaSuccess) return e;
    const int mtiles = (g.M + 127) / 128;
    const int64_t tiles = (int64_t)mtiles * ((g.N + CT - 1) / CT);
    if (tiles > 0x7fffffff - 1024) return cudaErrorInvalidValue;
    LaunchScope scope(kKMxMatmul, stream);
    return launch_pdl(mxfp4_gemm_wide_kernel<T, CT>, dim3((unsigned)(tiles < sms ? tiles : sms)),
                      dim3(kWideThreads), sm, stream, ma, mb, mo, g, mtiles, (int)tiles, tma_out);
}

template <int CT>
cudaError_t run_wide_type(const uint8_t* a, const uint8_t* b, const GemmArgs& g, int sms, cudaStream_t stream) {
    if (g.dtype == CSA_DT_BF16) return run_wide<__nv_bfloat16, CT>(a, b, g, sms, stream);
    if (g.dtype == CSA_DT_F16) return run_wide<__half, CT>(a, b, g, sms, stream);
    return run_wide<float, CT>(a, b, g, sms, stream);
}

}  // namespace

cudaError_t launch_mxfp4_matmul(const uint8_t* a, const uint8_t* a_sf, const uint8_t* b,
                                const uint8_t* b_sf, int M, int N, int K, void* out, int dtype,
                                int64_t ld, int32_t* st, cudaStream_t stream) {
    const GemmArgs g{a_sf, b_sf, out, ld, st, M, N, K, dtype, (K + 127) / 128};
    const int sms = sm_count();
    // Up to 96 tokens lie on the columns: 8192 x 2048 takes 5.3 us for 32 tokens (7.1 on the lanes),
    // 5.9 against 6.4 for 65, 6.0 against 6.0 (16384 x 2048: 6.0, 6.7) for 96; 128 tokens would take
    // 6.3 against 6.2.
    if (M > 96) {
        // The feature tile that takes the least time: rounds of tiles over the SMs, each a fixed part
        // and a part per stage of K (in 10 ns, from 8192 x 8192 at K = 512 and 4096: 256 columns
        // 1.6 + 0.41 per stage, 128 0.7 + 0.28, 64 0.45 + 0.27; the narrow tiles are bound by the
        // stage's issue, not its bytes).  512 x 8192 x 2048: 7.8 us at 256, 9.1 at 128, 13.5 at 64;
        // 197 x 4104 x 1504: 9.6, 7.3 and 6.4.
        const int64_t mt = (M + 127) / 128, nk = (K + kStageK - 1) / kStageK;
        auto cost = [&](int ct, int64_t fixed, int64_t per_stage) {
            return (mt * ((N + ct - 1) / ct) + sms - 1) / sms * (fixed + per_stage * nk);
        };
        const int64_t c256 = cost(256, 160, 41), c128 = cost(128, 70, 28), c64 = cost(64, 45, 27);
        if (c256 <= c128 && c256 <= c64) return run_wide_type<256>(a, b, g, sms, stream);
        if (c128 <= c64) return run_wide_type<128>(a, b, g, sms, stream);
        return run_wide_type<64>(a, b, g, sms, stream);
    }
    // weight rows a CTA takes: 128, or fewer while the tiles leave SMs without one (8 x 8192 x 2048:
    // 5.3 us at 64, 5.5 at 128, and 9.8 at 32 in two rounds; 8 x 16384 x 2048: 5.5 at 128, 10.0 at 64)
    int RT = 128;
    while (RT > 32 && (N + RT / 2 - 1) / (RT / 2) <= sms) RT /= 2;
    if (M <= 16) return run<16>(a, b, g, RT, stream);
    if (M <= 32) return run<32>(a, b, g, RT, stream);
    if (M <= 64) return run<64>(a, b, g, RT, stream);
    return run<96>(a, b, g, RT, stream);
}

}  // namespace csa
