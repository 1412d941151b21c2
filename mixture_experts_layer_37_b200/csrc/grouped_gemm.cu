// Grouped matrix products over rows sorted by expert, and their gradients, on
// the 5th-generation tensor cores (bf16, fp32 accumulation).
//
//   FWD  y[r,n]    = sum_k x[r,k] W[e,k,n] (+ b[e,n])     rows r of expert e
//   GX   dx[r,k]   = sum_n dy[r,n] W[e,k,n]
//   GW   dW[e,k,n] = sum_{r of e} x[r,k] dy[r,n]
//
// with rows [offsets[e], offsets[e+1]) belonging to expert e.  The matrix
// products of the expert FFNs and their gradients ("MoE: gating, experts, load
// balancing, capacity factor" (dpshk.com/news/6005940) §2.2, §4.4; gradients
// from the product rule).
//
// One persistent CTA per SM, 192 threads: warp 0 loads by TMA, warp 1 issues
// tcgen05.mma (M=128, N=256, K=16, two TMEM accumulators of 256 columns), warps
// 2-5 read the accumulators and store.  What differs between the three forms
// is which operand is contiguous along the contraction:
//   FWD  A = x rows, contraction-major; B = W[e], output-major (four boxes
//        [64 k x 64 n]);
//   GX   A = dy rows, contraction-major; B = W[e], contraction-major (one box
//        [256 k x 64 n]): the weights are read as they lie, nothing is transposed;
//   GW   both output-major: A = x (two boxes [64 rows x 64 k]), B = dy (four
//        boxes [64 rows x 64 n]); the contraction runs over the expert's rows.
// Weights and weight gradients are addressed as 3-D tensors [E, K, N], so a K
// or N that fills no tile is cut at the expert's own edge (zero fill on loads)
// and never mixes with the next expert's values.
//
// Ragged edges.  FWD, GX: a tile that runs past its expert's last row reads
// the next rows and does not store them (rows do not mix).  GW: rows of the
// next expert in the last block of 64 would be summed, and 0 * inf is not 0, so
// they are not multiplied by zero but overwritten: the MMA warp clears the rows
// of both operands behind the expert's end up to the next multiple of 16 in
// shared memory (at most 15 rows, once per tile) and issues only that many
// K=16 steps.  GW tiles are taken expert by expert in order of falling row
// count, so that the last wave holds the cheapest tiles.
// Every wait is bounded in time, as in the other kernels.
#include "gemm_common.cuh"
#include "grouped.h"

namespace moe {
namespace {

using namespace gemm;

constexpr int BM = 128;
constexpr int kStages = 4;
constexpr int kAStageBytes = BM * BK * 2;                 // 16 KB
constexpr int kBStageBytes = 4 * kBBoxBytes;              // 32 KB
constexpr int kStageBytes = kAStageBytes + kBStageBytes;  // 48 KB
constexpr int kSmemBytes = kStages * kStageBytes + 1024 /*barriers, tables*/ + 1024 /*alignment*/;

enum { FORM_FWD = 0, FORM_GX = 1, FORM_GW = 2 };
// What the epilogue does with the fp32 accumulators: round to bf16 (with a
// bias in FWD, added to what is there in GW on request), store as fp32, or, in
// FWD, the backward pass of the expert activation (below).
enum { EPI_BF16 = 0, EPI_F32 = 1, EPI_SWIGLU_GRAD = 2, EPI_GELU_GRAD = 3 };

struct GroupedParams {
    const int32_t* offsets = nullptr;  // [E+1]
    int rows = 0;                      // rows of the buffers
    int E = 0;
    int M = 0;                         // GW: output rows per expert (K of the weights)
    int N = 0;                         // output columns
    int kblocks = 0, kblocks2 = 0;     // FWD, GX: blocks of 64 of the first and of a second operand pair
    int bn_out = 256, n_tiles = 0, m_tiles = 0;
    void* out = nullptr;
    const __nv_bfloat16* bias = nullptr;  // [E, N] or null
    int accumulate = 0;                   // GW
    const float* dh = nullptr;            // activation gradients: [rows, N] fp32
    __nv_bfloat16* h = nullptr;           // [rows, N] outputs
    __nv_bfloat16* d0 = nullptr;
    __nv_bfloat16* d1 = nullptr;
    DevStatus st;
};

constexpr uint32_t make_idesc_majors(int m, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const void* map, uint64_t* bar, int32_t c0, int32_t c1,
                                            int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

struct Tile {
    int e, m0, row0, rows, nt;  // FWD, GX: rows of this tile from row0; GW: m0 in the output, rows to sum from row0
};

// Expert by expert; inside an expert groups of kGroupM m-tiles, n-tile-major
// inside a group, so that the CTAs running together share operands in L2.
template <int FORM>
__device__ __forceinline__ Tile decode(int tile, const GroupedParams& p, const GroupTables* t) {
    int i = 0;
    while (t->start[i + 1] * p.n_tiles <= tile) ++i;
    const int local = tile - t->start[i] * p.n_tiles;
    const int mt_e = t->start[i + 1] - t->start[i];
    const int grp = local / (kGroupM * p.n_tiles);
    const int gm = min(kGroupM, mt_e - grp * kGroupM);
    const int r = local - grp * kGroupM * p.n_tiles;
    Tile o;
    o.nt = r / gm;
    const int mt = grp * kGroupM + (r - o.nt * gm);
    o.e = t->expert[i];
    o.m0 = mt * BM;
    if (FORM == FORM_GW) {
        o.row0 = t->row0[i];
        o.rows = t->nrows[i];
    } else {
        o.row0 = t->row0[i] + o.m0;
        o.rows = min(BM, t->nrows[i] - o.m0);
    }
    return o;
}

template <int FORM>
__device__ __forceinline__ int tile_kblocks(const GroupedParams& p, const Tile& t) {
    return FORM == FORM_GW ? (t.rows + BK - 1) / BK : p.kblocks + p.kblocks2;
}

__device__ __forceinline__ void store16_bf16(__nv_bfloat16* row, int col, int N, const float* x) {
#pragma unroll
    for (int hlf = 0; hlf < 2; ++hlf)
        if (col + 8 * hlf < N) {
            const float* v = x + 8 * hlf;
            *reinterpret_cast<uint4*>(row + col + 8 * hlf) =
                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                           pack_bf16x2(v[6], v[7]));
        }
}

// x += 16 bf16 values at row + col (those inside N).
__device__ __forceinline__ void add16_bf16(const __nv_bfloat16* row, int col, int N, float* x) {
#pragma unroll
    for (int hlf = 0; hlf < 2; ++hlf)
        if (col + 8 * hlf < N) {
            const uint4 b = *reinterpret_cast<const uint4*>(row + col + 8 * hlf);
            const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[8 * hlf + 2 * i] += bf16_lo(w[i]);
                x[8 * hlf + 2 * i + 1] += bf16_hi(w[i]);
            }
        }
}

// The activation's backward pass for 16 columns of one row, from the fp32
// accumulators of its own products and the fp32 gradient dh.  Only what the
// next products read is rounded to bf16 (their operand type), once.
//   SwiGLU  s = sigmoid(g): h = g s u, dg = dh u s (1 + g (1 - s)), du = dh g s
//   GELU    h = p Phi(p), dp = dh (Phi(p) + p phi(p))
__device__ __forceinline__ void swiglu_grad(float g, float u, float dh, float& h, float& dg, float& du) {
    const float s = 1.0f / (1.0f + __expf(-g));
    const float gs = g * s;
    h = gs * u;
    dg = dh * u * (s + gs * (1.0f - s));
    du = dh * gs;
}
__device__ __forceinline__ void gelu_grad(float p, float dh, float& h, float& dp) {
    const float cdf = 0.5f * (1.0f + erff(p * 0.70710678118654752f));
    const float pdf = 0.39894228040143268f * __expf(-0.5f * p * p);
    h = p * cdf;
    dp = dh * (cdf + p * pdf);
}

template <int FORM, int EPI>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmA2, const __grid_constant__ CUtensorMap tmB2,
                   GroupedParams p) {
    constexpr bool kTwoB = EPI == EPI_SWIGLU_GRAD;  // gate and up halves of the 256 columns
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sA = smem;
    uint8_t* sB = smem + kStages * kAStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    __shared__ GroupTables tab;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&tfull[0], 1);
        mbar_init(&tfull[1], 1);
        mbar_init(&tempty[0], 4);
        mbar_init(&tempty[1], 4);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    // the prologue above overlaps the launch before; from here on its results are read
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 2) build_group_tables<FORM == FORM_GW>(p.offsets, p.rows, p.E, BM, p.m_tiles, p.st, &tab, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int total_tiles = tab.start[p.E] * p.n_tiles;
    const uint64_t tmo = p.st.timeout_ns;

    auto give_up = [&](uint32_t site) {
        report_timeout(p.st, site);
        *abort_flag = 1;
    };

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0;
            uint32_t phase = 0, issued_mask = 0, issued_par = 0;
            bool stop = false;
            for (int tile = blockIdx.x; tile < total_tiles && !stop; tile += gridDim.x) {
                const Tile t = decode<FORM>(tile, p, &tab);
                const int n0 = t.nt * p.bn_out;
                const int kbs = tile_kblocks<FORM>(p, t);
                for (int kb = 0; kb < kbs; ++kb) {
                    if (*abort_flag) { stop = true; break; }
                    if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, tmo)) {
                        give_up(SITE_GEMM_PRODUCER_EMPTY);
                        stop = true;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[stage], kStageBytes);
                    uint8_t* a_dst = sA + stage * kAStageBytes;
                    uint8_t* b_dst = sB + stage * kBStageBytes;
                    if (FORM == FORM_GW) {
                        const int r = t.row0 + kb * BK;
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            tma_load_2d(a_dst + i * kBBoxBytes, &tmA, &full[stage], t.m0 + 64 * i, r);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            tma_load_2d(b_dst + i * kBBoxBytes, &tmB, &full[stage], n0 + 64 * i, r);
                    } else if (FORM == FORM_GX) {
                        const bool second = kb >= p.kblocks;
                        const int c = (second ? kb - p.kblocks : kb) * BK;
                        tma_load_2d(a_dst, second ? &tmA2 : &tmA, &full[stage], c, t.row0);
                        tma_load_3d(b_dst, second ? &tmB2 : &tmB, &full[stage], c, n0, t.e);
                    } else {
                        tma_load_2d(a_dst, &tmA, &full[stage], kb * BK, t.row0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (kTwoB)
                                tma_load_3d(b_dst + i * kBBoxBytes, i < 2 ? &tmB : &tmB2, &full[stage],
                                            n0 + 64 * (i & 1), kb * BK, t.e);
                            else
                                tma_load_3d(b_dst + i * kBBoxBytes, &tmB, &full[stage], n0 + 64 * i, kb * BK, t.e);
                        }
                    }
                    issued_mask |= 1u << stage;
                    issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // no copy may still be landing in shared memory when the CTA exits
            for (int s = 0; s < kStages; ++s)
                if ((issued_mask >> s) & 1u)
                    if (!mbar_wait_bounded(&full[s], (issued_par >> s) & 1u, tmo)) give_up(SITE_GEMM_PRODUCER_DRAIN);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer
        // the whole warp walks the tiles (it clears rows in GW); lane 0 issues
        int stage = 0;
        uint32_t phase = 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool stop = false;
        constexpr bool kAMn = FORM == FORM_GW, kBMn = FORM != FORM_GX;
        for (int tile = blockIdx.x; tile < total_tiles && !stop; tile += gridDim.x) {
            const Tile t = decode<FORM>(tile, p, &tab);
            const int kbs = tile_kblocks<FORM>(p, t);
            if (kbs == 0) continue;  // GW, an expert without rows: the epilogue stores zeros by itself
            const bool m64 = FORM != FORM_GW && t.rows <= BM / 2;
            const uint32_t idesc =
                m64 ? make_idesc_majors(BM / 2, BN_MMA, kAMn, kBMn) : make_idesc_majors(BM, BN_MMA, kAMn, kBMn);
            bool ok = mbar_wait_bounded(&tempty[acc], acc_phase ^ 1u, tmo);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) give_up(SITE_GEMM_MMA_TMEM_EMPTY);
                break;
            }
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN_MMA);
            for (int kb = 0; kb < kbs; ++kb) {
                if (__shfl_sync(0xffffffffu, *abort_flag, 0)) { stop = true; break; }
                ok = mbar_wait_bounded(&full[stage], phase, tmo);
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0) give_up(SITE_GEMM_MMA_FULL);
                    stop = true;
                    break;
                }
                uint8_t* a_st = sA + stage * kAStageBytes;
                uint8_t* b_st = sB + stage * kBStageBytes;
                int steps = BK / 16;
                if (FORM == FORM_GW) {
                    const int held = t.rows - kb * BK;
                    if (held < BK) {
                        steps = (held + 15) / 16;
                        // rows [held, 16 steps) of the six boxes: 128 bytes each
                        const int nz = (16 * steps - held) * 8;
                        for (int i = lane; i < nz; i += 32) {
                            const int off = held * 128 + i * 16;
#pragma unroll
                            for (int b = 0; b < 6; ++b)
                                *reinterpret_cast<uint4*>((b < 2 ? a_st + b * kBBoxBytes : b_st + (b - 2) * kBBoxBytes) +
                                                          off) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t a_addr = smem_u32(a_st), b_addr = smem_u32(b_st);
                    for (int kk = 0; kk < steps; ++kk) {
                        // contraction-major: +32 bytes per K=16 step inside the 128-byte swizzle row;
                        // output-major: +16 rows of 128 bytes per step, 64-column boxes 8 KB apart
                        const uint64_t adesc = kAMn ? smem_desc_sw128(a_addr + kk * 2048, kBBoxBytes, 1024)
                                                    : smem_desc_sw128(a_addr + kk * 32, 16, 1024);
                        const uint64_t bdesc = kBMn ? smem_desc_sw128(b_addr + kk * 2048, kBBoxBytes, 1024)
                                                    : smem_desc_sw128(b_addr + kk * 32, 16, 1024);
                        tc_mma_f16(d_tmem, adesc, bdesc, idesc, (kb | kk) != 0 ? 1u : 0u);
                    }
                    tc_commit(&empty[stage]);
                }
                __syncwarp();
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (stop) break;
            if (lane == 0) tc_commit(&tfull[acc]);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
        // every MMA issued by this thread has completed before TMEM is freed
        if (lane == 0) {
            tc_commit(drain);
            if (!mbar_wait_bounded(drain, 0, tmo)) give_up(SITE_GEMM_DRAIN);
        }
    } else {
        // ---------------------------------------------------- epilogue
        const int q = warp & 3;  // TMEM lanes 32q..32q+31 are reachable from this warp
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int tile = blockIdx.x; tile < total_tiles; tile += gridDim.x) {
            const int ab = __shfl_sync(0xffffffffu, *abort_flag, 0);
            if (ab) break;
            const Tile t = decode<FORM>(tile, p, &tab);
            const int n0 = t.nt * p.bn_out;
            const bool none = tile_kblocks<FORM>(p, t) == 0;
            if (!none) {
                const bool ok = mbar_wait_bounded(&tfull[acc], acc_phase, tmo);
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0) give_up(SITE_GEMM_EPI_TMEM_FULL);
                    break;
                }
                tc_fence_after();
            }
            // M=128: row 32q + lane.  M=64: rows 16q..16q+15 sit in lanes 0-15 of this warp's quarter
            const bool m64 = FORM != FORM_GW && t.rows <= BM / 2;
            const int r = m64 ? 16 * q + lane : q * 32 + lane;
            const bool valid = FORM == FORM_GW ? t.m0 + r < p.M : r < t.rows && (!m64 || lane < 16);
            const int64_t orow = FORM == FORM_GW ? (int64_t)t.e * p.M + t.m0 + (valid ? r : 0) : t.row0 + (valid ? r : 0);
            const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN_MMA);
            if (EPI == EPI_SWIGLU_GRAD) {
                for (int c = 0; c < 128; c += 16) {
                    uint32_t g[16], u[16];
                    tmem_ld_16(tbase + c, g);
                    tmem_ld_16(tbase + 128 + c, u);
                    const int col = n0 + c;
                    float d[16];
                    if (valid && col < p.N) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<float4*>(d + 4 * i) =
                                *reinterpret_cast<const float4*>(p.dh + orow * p.N + col + 4 * i);
                    }
                    tmem_ld_wait();
                    if (valid && col < p.N) {
                        float h[16], dg[16], du[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            swiglu_grad(__uint_as_float(g[i]), __uint_as_float(u[i]), d[i], h[i], dg[i], du[i]);
                        store16_bf16(p.h + orow * p.N, col, p.N, h);
                        store16_bf16(p.d0 + orow * p.N, col, p.N, dg);
                        store16_bf16(p.d1 + orow * p.N, col, p.N, du);
                    }
                }
            } else {
                for (int c = 0; c < BN_MMA; c += 16) {
                    uint32_t v[16];
                    if (!none) {
                        tmem_ld_16(tbase + c, v);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = 0u;
                    }
                    const int col = n0 + c;
                    if (!valid || col >= p.N || (none && p.accumulate)) continue;
                    float x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(v[i]);
                    if (FORM == FORM_FWD && p.bias != nullptr) add16_bf16(p.bias + (int64_t)t.e * p.N, col, p.N, x);
                    if (EPI == EPI_GELU_GRAD) {
                        float h[16], dp[16];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 d = *reinterpret_cast<const float4*>(p.dh + orow * p.N + col + 4 * i);
                            gelu_grad(x[4 * i], d.x, h[4 * i], dp[4 * i]);
                            gelu_grad(x[4 * i + 1], d.y, h[4 * i + 1], dp[4 * i + 1]);
                            gelu_grad(x[4 * i + 2], d.z, h[4 * i + 2], dp[4 * i + 2]);
                            gelu_grad(x[4 * i + 3], d.w, h[4 * i + 3], dp[4 * i + 3]);
                        }
                        store16_bf16(p.h + orow * p.N, col, p.N, h);
                        store16_bf16(p.d0 + orow * p.N, col, p.N, dp);
                    } else if (EPI == EPI_F32) {
                        float* dst = static_cast<float*>(p.out) + orow * p.N + col;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (col + 4 * i < p.N) {
                                float4 w = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                                if (FORM == FORM_GW && p.accumulate) {
                                    const float4 old = *reinterpret_cast<const float4*>(dst + 4 * i);
                                    w.x += old.x;
                                    w.y += old.y;
                                    w.z += old.z;
                                    w.w += old.w;
                                }
                                *reinterpret_cast<float4*>(dst + 4 * i) = w;
                            }
                    } else {
                        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + orow * p.N;
                        if (FORM == FORM_GW && p.accumulate) add16_bf16(dst, col, p.N, x);
                        store16_bf16(dst, col, p.N, x);
                    }
                }
            }
            if (!none) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[acc]);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

// ------------------------------------------------------------------ host side
template <int FORM, int EPI>
cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& a2, const CUtensorMap& b2,
                   const GroupedParams& p, int64_t tiles_upper, cudaStream_t s) {
    static std::atomic<bool> attr_set[64];
    const cudaError_t err = ensure_smem_attr(attr_set, grouped_kernel<FORM, EPI>, kSmemBytes);
    if (err != cudaSuccess) return err;
    const int grid = (int)min64(tiles_upper, (int64_t)sm_count());
    if (grid <= 0) return cudaSuccess;
    return launch_kernel(grouped_kernel<FORM, EPI>, dim3(grid), dim3(kThreads), kSmemBytes, s, a, b, a2, b2, p);
}

// Activations [rows, cols], boxes [box_rows, 64].
bool act_map(CUtensorMap* m, const void* base, int64_t rows, int cols, int box_rows) {
    return make_map(m, base, (uint64_t)cols, (uint64_t)rows, (uint64_t)cols * 2, 64, (uint32_t)box_rows);
}

GroupedParams params(const GroupedArgs& a) {
    GroupedParams p;
    p.offsets = a.offsets;
    p.rows = (int)a.rows;
    p.E = a.E;
    p.st = a.st;
    return p;
}

int64_t row_tiles_upper(const GroupedArgs& a) { return a.rows / BM + a.E; }

}  // namespace

cudaError_t launch_grouped_fwd_bf16(const GroupedArgs& a, cudaStream_t s) {
    CUtensorMap mA, mB, mB2;
    bool ok = act_map(&mA, a.x, a.rows, a.K, 128);
    ok = ok && make_map_3d(&mB, a.w, a.E, a.K, a.N, 64, BK);
    const bool two = a.grad_act == GRAD_SWIGLU;
    if (two)
        ok = ok && make_map_3d(&mB2, a.w2, a.E, a.K, a.N, 64, BK);
    else
        mB2 = mB;
    if (!ok) return cudaErrorInvalidValue;
    GroupedParams p = params(a);
    p.N = a.N;
    p.kblocks = (a.K + BK - 1) / BK;
    p.bn_out = two ? 128 : 256;
    p.n_tiles = (a.N + p.bn_out - 1) / p.bn_out;
    p.out = a.y;
    p.bias = static_cast<const __nv_bfloat16*>(a.bias);
    p.dh = static_cast<const float*>(a.dh);
    p.h = static_cast<__nv_bfloat16*>(a.h);
    p.d0 = static_cast<__nv_bfloat16*>(a.d0);
    p.d1 = static_cast<__nv_bfloat16*>(a.d1);
    const int64_t tiles = row_tiles_upper(a) * p.n_tiles;
    if (two) return launch<FORM_FWD, EPI_SWIGLU_GRAD>(mA, mB, mA, mB2, p, tiles, s);
    if (a.grad_act == GRAD_GELU) return launch<FORM_FWD, EPI_GELU_GRAD>(mA, mB, mA, mB2, p, tiles, s);
    return launch<FORM_FWD, EPI_BF16>(mA, mB, mA, mB2, p, tiles, s);
}

cudaError_t launch_grouped_gx_bf16(const GroupedArgs& a, cudaStream_t s) {
    CUtensorMap mA, mB, mA2, mB2;
    bool ok = act_map(&mA, a.dy, a.rows, a.N, 128);
    ok = ok && make_map_3d(&mB, a.w, a.E, a.K, a.N, 64, 256);
    if (a.dy2 != nullptr) {
        ok = ok && act_map(&mA2, a.dy2, a.rows, a.N, 128);
        ok = ok && make_map_3d(&mB2, a.w2, a.E, a.K, a.N, 64, 256);
    } else {
        mA2 = mA;
        mB2 = mB;
    }
    if (!ok) return cudaErrorInvalidValue;
    GroupedParams p = params(a);
    p.N = a.K;
    p.kblocks = (a.N + BK - 1) / BK;
    p.kblocks2 = a.dy2 != nullptr ? p.kblocks : 0;
    p.n_tiles = (a.K + 255) / 256;
    p.out = a.dx;
    const int64_t tiles = row_tiles_upper(a) * p.n_tiles;
    return a.out_f32 ? launch<FORM_GX, EPI_F32>(mA, mB, mA2, mB2, p, tiles, s)
                     : launch<FORM_GX, EPI_BF16>(mA, mB, mA2, mB2, p, tiles, s);
}

cudaError_t launch_grouped_gw_bf16(const GroupedArgs& a, cudaStream_t s) {
    CUtensorMap mA, mB;
    bool ok = act_map(&mA, a.x, a.rows, a.K, BK);
    ok = ok && act_map(&mB, a.dy, a.rows, a.N, BK);
    if (!ok) return cudaErrorInvalidValue;
    GroupedParams p = params(a);
    p.M = a.K;
    p.N = a.N;
    p.m_tiles = (a.K + BM - 1) / BM;
    p.n_tiles = (a.N + 255) / 256;
    p.out = a.dw;
    p.accumulate = a.accumulate ? 1 : 0;
    const int64_t tiles = (int64_t)a.E * p.m_tiles * p.n_tiles;
    return a.out_f32 ? launch<FORM_GW, EPI_F32>(mA, mB, mA, mB, p, tiles, s)
                     : launch<FORM_GW, EPI_BF16>(mA, mB, mA, mB, p, tiles, s);
}

}  // namespace moe
