// Expert products with 4-bit weights: quantisation, the grouped product
//   y[r,n] = sum_g s[e,g,n] sum_{k in g} x[r,k] q[e,k,n]  (+ b[e,n]),  q in [-8, 7],
// and the expert FFNs built from it, for batches of single tokens, where the
// time is the time to stream the weights ("Hand-building a LLaMA4-MoE" (dpshk.com/
// news/5809432) §5.2 names 4-bit experts; the scales per group of K as the
// INT8 form's per column).  bf16 activations, fp32 sums and scales.
//
// Storage of the codes: [E, N, ceil(K/128) * 64 bytes], K-contiguous per output
// column, a code q stored as q + 8.  A block of 128 codes is 16 words of 32 bits;
// word 4 t + i holds the eight codes of k = 32 i + 8 t .. + 7 in the order k,
// k+2, k+4, k+6, k+1, k+3, k+5, k+7 (low bits first): (w >> 4j) & 0x000F000F,
// or'ed with 0x4300 in both halves, is the bf16 pair (128 + c[2j], 128 + c[2j+1]),
// exactly; minus 136, exactly, two neighbouring codes.
//
// Method: the weights are the 128-row operand of the matrix instruction and come
// from tensor memory: a thread that owns a column n widens its codes in registers
// and stores them with tcgen05.st, so that the four times larger bf16 form never
// passes through shared memory (written and read there it would take 4 x 32 KB
// of its bandwidth where the codes' own 8 KB arrive in the time of 2).  The
// tokens are the other operand, read by TMA as they lie.  Each group of 32, 64 or
// 128 k gets a fresh accumulator, and the thread that owns column n multiplies the
// finished sums by the group's scale in fp32: weights are never rounded to
// bf16 products with their scale.
//
// One persistent CTA per SM, tiles of 128 columns x TN tokens:
//   warp 0     TMA producer: 256 k of codes [128 rows x 128 bytes] and their
//              scales (SwiGLU: of gate and of up) and of tokens [TN rows x 256 k]
//              per stage, across tiles without a pause;
//   warp 1     issues tcgen05.mma (A in TMEM, M=128, N=TN, K=16);
//   then two or three groups of four warps that widen, taking units (I4Smem) in turn;
//   last four warps (eight from 32 tokens on) that scale and add each group's
//              sums, and at the tile's end activation, bias and the store.
// TN = 16 for batches of few rows per expert, 64 (SwiGLU, or groups of 32: 32)
// for more: the host chooses by the mean.  Every wait is bounded in time, as in the other kernels.
//
// Measured: 128 rows over 64 experts of 2048 x 2048, groups of 64, 35 to 39 us, where the codes and scales take 20 at
// the memory's rate (without the widening 32: the rest is the hand-over and 7 rounds of tiles for 6.2); 500 rows over
// 8 experts of 4096 x 4096, groups of 128, 44 us, 33 if even (12): an expert of more than 64 rows takes its codes again.  (Tiles of
// 128 tokens fit tensor memory for groups of 128 but leave two stages, fewer than the waits below need; 54 us was
// measured so, which settles nothing.)
#include <math.h>

#include "gemm_common.cuh"
#include "grouped.h"

namespace moe {
namespace {

using namespace gemm;

constexpr int kBlockK = 128;                  // codes of a storage block
constexpr int kCols = 128;                    // output columns of a tile
constexpr int kCodeStage = kCols * 128;       // 16 KB: two blocks of each column

enum { I4_PLAIN = 0, I4_SWIGLU = 1, I4_GELU = 2 };

struct Int4Params {
    const float* s0 = nullptr;            // [E, groups, N] scales (SwiGLU: gate)
    const float* s1 = nullptr;            // SwiGLU: up
    const __nv_bfloat16* bias = nullptr;  // [E, N] or null
    __nv_bfloat16* out = nullptr;         // [rows, N]
    const int32_t* offsets = nullptr;     // [E+1]
    int rows = 0, E = 0, N = 0, groups = 0, blocks = 0, n_tiles = 0;
    DevStatus st;
};

template <int MODE, int GS, int TN>
struct I4Smem {
    static constexpr int kMats = MODE == I4_SWIGLU ? 2 : 1;
    static constexpr int kX = TN * 512;  // 256 k of TN tokens: four boxes of 64 k
    static constexpr int kScales = 2 * (4 / GS) * kCols * 4;  // the groups of 256 k of 128 columns
    static constexpr int kXOff = kMats * kCodeStage, kScaleOff = kXOff + kX;
    static constexpr int kStage = kScaleOff + kMats * kScales;
    // What is handed on at a time: kUnit blocks of 128 k of one matrix, its widened codes (64 columns a block) in one
    // of kABufs buffers in TMEM and its groups' accumulators (TN columns each) in one of kDBufs.  Handing on 256 k
    // at TN = 16 halves the issuer's waits and commits (64 experts of 2048 x 2048, 128 rows: 60 -> 38 us).
    static constexpr int kUnit = TN == 16 ? 2 : 1;
    static constexpr int kPerStage = 2 / kUnit * kMats;  // units of a stage: by half, then by matrix
    static constexpr int kACols = kUnit * 64, kDCols = kUnit * (4 / GS) * TN;
    static constexpr int kABufs = TN != 16 ? 4 : GS == 1 ? 2 : 3;
    // No more accumulators than A buffers: a buffer's `done` must not complete again before the warps that wait for
    // it have seen it, and a unit kABufs later waits for their `taken` only if there are no more of these.
    static constexpr int kDFit = (512 - kABufs * kACols) / kDCols, kDBufs = kDFit < kABufs ? kDFit : kABufs;
    static_assert(kDBufs >= 2 && kABufs * kACols + kDBufs * kDCols <= 512, "the buffers fit tensor memory");
    static constexpr int kGroupsOfWarps = kABufs == 3 ? 3 : 2;  // four widening warps each
    // A group comes back to a buffer that it filled itself the last time: only then does the parity that it waits
    // for tell that use from the one before.
    static_assert(kABufs % kGroupsOfWarps == 0, "each buffer belongs to one group of warps");
    static constexpr int kWidenWarps = 4 * kGroupsOfWarps;
    // Four for each kTokens of the tile's tokens.  Four for all 64 held the products up (500 rows over 8 even experts
    // of 4096 x 4096, groups of 128: 34.7 us against 33.0; 1024 rows of 2048 x 2048, groups of 64: 24.7 against 21.6;
    // SwiGLU FFN of 512 tokens, 16 experts of 2048 x 2048: 61 against 56).
    static constexpr int kScaleWarps = TN == 16 ? 4 : 8;
    static constexpr int kTokens = TN / (kScaleWarps / 4);
    static constexpr int kThreads = 32 * (2 + kWidenWarps + kScaleWarps);
    static constexpr int kStages = 200 * 1024 / kStage < 8 ? 200 * 1024 / kStage : 8;
    // A widening group skips the stages that hold none of its units and waits for `full` by parity. Before it waits for
    // unit u it has seen the products of unit u - kGroupsOfWarps - kABufs done, so their stage and all before it were
    // full; if that one lies less than kStages behind, the fill before the awaited one is over and cannot be taken for it.
    static_assert(kStages * kPerStage >= kGroupsOfWarps + kABufs, "stages enough to wait for a fill by its parity");
    static constexpr int kBytes = kStages * kStage + 512 + 1024 /*alignment*/;
};

// The codes 2j, 2j+1 of a word as a bf16 pair.
__device__ __forceinline__ uint32_t widen(uint32_t w, int j) {
    uint32_t v;  // (shifted & mask) | bits of 128, as one three-input operation
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w >> (4 * j)), "r"(0x000F000Fu), "r"(0x43004300u));
    const __nv_bfloat162 m = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));  // 136
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), m);
    return *reinterpret_cast<const uint32_t*>(&d);
}

// 16 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16.
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// A place in a ring of N buffers and the parity of its current turn.
template <int N>
struct Ring {
    uint32_t i = 0, par = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            par ^= 1u;
        }
    }
};

struct I4Tile {
    int e, row0, rows, n0;
};
__device__ __forceinline__ I4Tile i4_tile(int tile, const Int4Params& p, const GroupTables* t, int tn, int& i) {
    while (t->start[i + 1] * p.n_tiles <= tile) ++i;
    const int local = tile - t->start[i] * p.n_tiles;
    const int pass = local / p.n_tiles;
    I4Tile o;
    o.e = t->expert[i];
    o.row0 = t->row0[i] + pass * tn;
    o.rows = min(tn, t->nrows[i] - pass * tn);
    o.n0 = (local - pass * p.n_tiles) * kCols;
    return o;
}

// tmQ0, tmQ1: codes as uint8 [E*N, blocks*64], box [128 rows, 128 bytes], 128-byte swizzle; tmX: tokens
// [rows, K] bf16, box [TN rows, 64 k], 128-byte swizzle; tmS0, tmS1: scales [E, groups, N], box [1, the groups
// of 256 k, 128 columns], zeros past an expert's last group.  GS: steps of 32 k per group.
template <int MODE, int GS, int TN>
__global__ void __launch_bounds__(I4Smem<MODE, GS, TN>::kThreads, 1)
    int4_kernel(const __grid_constant__ CUtensorMap tmQ0, const __grid_constant__ CUtensorMap tmQ1,
                const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmS0,
                const __grid_constant__ CUtensorMap tmS1, Int4Params p) {
    using S = I4Smem<MODE, GS, TN>;
    constexpr int kMats = S::kMats, kStages = S::kStages, kGroups = 4 / GS, kUnit = S::kUnit;
    constexpr int kABufs = S::kABufs, kDBufs = S::kDBufs;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * S::kStage);
    uint64_t* empty = full + kStages;
    uint64_t* ready = empty + kStages;  // [A buffer] widened, by four warps
    uint64_t* done = ready + kABufs;    // [A buffer] its products are done: codes free, sums readable
    uint64_t* taken = done + kABufs;    // [D buffer] its sums are read
    uint64_t* drain = taken + kDBufs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    __shared__ GroupTables tab;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], S::kScaleWarps);  // the last readers: they wait for the products
        }
        for (int b = 0; b < kABufs; ++b) {
            mbar_init(&ready[b], 4);
            mbar_init(&done[b], 1);
        }
        for (int b = 0; b < kDBufs; ++b) mbar_init(&taken[b], S::kScaleWarps);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
        tma_prefetch_desc(&tmQ0);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    // the prologue above overlaps the launch before; from here on its results are read
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 2) build_group_tables<false>(p.offsets, p.rows, p.E, TN, 0, p.st, &tab, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t a_base = tmem_base, d_base = tmem_base + kABufs * S::kACols;
    const int total = tab.start[p.E] * p.n_tiles;
    // A tile is nst stages; a block of 128 k behind the last one is worked on like the others (codes, tokens and
    // scales are zeros there), so that every stage holds the same units and only the producer and the last warps
    // need to know the tiles.
    const int nst = (p.blocks + 1) / 2;
    const int tiles = total > (int)blockIdx.x ? (total - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;  // of this CTA
    const int stages = tiles * nst;
    const uint64_t tmo = p.st.timeout_ns;
    auto give_up = [&](uint32_t site) {
        report_timeout(p.st, site);
        *abort_flag = 1;
    };

    if (warp == 0) {
        if (elect_one()) {
            // ------------------------------------------------ TMA producer
            int stage = 0, place = 0;
            uint32_t phase = 0, issued_mask = 0, issued_par = 0;
            bool stop = false;
            for (int tile = blockIdx.x; tile < total && !stop; tile += gridDim.x) {
                if (*abort_flag) break;
                const I4Tile t = i4_tile(tile, p, &tab, TN, place);
                for (int st = 0; st < nst; ++st) {
                    if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, tmo)) {
                        give_up(SITE_GEMM_PRODUCER_EMPTY);
                        stop = true;
                        break;
                    }
                    uint8_t* s = smem + stage * S::kStage;
                    mbar_arrive_expect_tx(&full[stage], S::kStage);
                    tma_load_2d(s, &tmQ0, &full[stage], st * 128, t.e * p.N + t.n0);
                    if (kMats == 2) tma_load_2d(s + kCodeStage, &tmQ1, &full[stage], st * 128, t.e * p.N + t.n0);
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        tma_load_2d(s + S::kXOff + b * TN * 128, &tmX, &full[stage], st * 256 + 64 * b, t.row0);
                    tma_load_3d(s + S::kScaleOff, &tmS0, &full[stage], t.n0, st * 2 * kGroups, t.e);
                    if (kMats == 2) tma_load_3d(s + S::kScaleOff + S::kScales, &tmS1, &full[stage], t.n0, st * 2 * kGroups, t.e);
                    issued_mask |= 1u << stage;
                    issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // the loads land before the MMAs that read them complete: wait for the last release of every stage
            for (int s = 0; s < kStages; ++s)
                if ((issued_mask >> s) & 1u)
                    if (!mbar_wait_bounded(&empty[s], (issued_par >> s) & 1u, tmo)) give_up(SITE_GEMM_PRODUCER_DRAIN);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            // ------------------------------------------------ MMA issuer
            constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(TN >> 3) << 17) | ((128u >> 4) << 24);
            Ring<kStages> sb;
            Ring<kABufs> ab;
            Ring<kDBufs> db;
            bool stop = false;
            for (int st = 0; st < stages && !stop; ++st, sb.next()) {
                if (!mbar_wait_bounded(&full[sb.i], sb.par, tmo)) {
                    give_up(SITE_GEMM_MMA_FULL);
                    break;
                }
                const uint64_t xd = smem_desc_sw128(smem_u32(smem + sb.i * S::kStage + S::kXOff), 16, 1024);
#pragma unroll
                for (int v = 0; v < S::kPerStage; ++v) {
                    if (!mbar_wait_bounded(&ready[ab.i], ab.par, tmo) || !mbar_wait_bounded(&taken[db.i], db.par ^ 1u, tmo)) {
                        give_up(SITE_INT4_MMA_WIDENED);
                        stop = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = a_base + ab.i * S::kACols, d = d_base + db.i * S::kDCols;
#pragma unroll
                    for (int kk = 0; kk < 8 * kUnit; ++kk) {  // K=16 steps, 2 GS of them in a group
                        const int k = v / kMats * 8 + kk;     // of the stage's 16
                        tc_mma_f16_ta(d + kk / (2 * GS) * TN, a + kk * 8,
                                      xd + (uint32_t)((k / 4 * TN * 128 + k % 4 * 32) >> 4), kIdesc,
                                      kk % (2 * GS) != 0 ? 1u : 0u);
                    }
                    tc_commit(&done[ab.i]);
                    ab.next();
                    db.next();
                }
            }
            // every MMA issued by this thread has completed before TMEM is freed
            tc_commit(drain);
            if (!mbar_wait_bounded(drain, 0, tmo)) give_up(SITE_GEMM_DRAIN);
        }
        __syncwarp();
    } else if (warp < 2 + S::kWidenWarps) {
        // ---------------------------------------------------- widening
        const int q = warp & 3;                    // TMEM lanes 32q..32q+31: columns n0 + 32q + lane
        const int row = 32 * q + lane;
        const uint32_t lanes = (uint32_t)(32 * q) << 16;
        for (int u = (warp - 2) >> 2; u < stages * S::kPerStage; u += S::kGroupsOfWarps) {
            const int st = u / S::kPerStage, v = u % S::kPerStage, ab = u % kABufs;
            const uint8_t* c = smem + st % kStages * S::kStage + v % kMats * kCodeStage + row * 128;
            // only the stages of its own units are waited for: they cannot be filled again before those are done
            bool ok = mbar_wait_bounded(&full[st % kStages], (st / kStages) & 1, tmo);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) give_up(SITE_INT4_WIDEN_FULL);
                break;
            }
            uint4 w[kUnit][4];
#pragma unroll
            for (int h = 0; h < kUnit; ++h)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    w[h][t] = *reinterpret_cast<const uint4*>(c + (((4 * (v / kMats + h) + t) ^ (row & 7)) << 4));
            ok = mbar_wait_bounded(&done[ab], ((u / kABufs) & 1) ^ 1, tmo);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) give_up(SITE_INT4_WIDEN_FREE);
                break;
            }
            tc_fence_after();
            const uint32_t dst = a_base + lanes + ab * S::kACols;
#pragma unroll
            for (int h = 0; h < kUnit; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t r[16];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) r[4 * t + j] = widen(word_of(w[h][t], i), j);
                    tmem_st_16(dst + 64 * h + 16 * i, r);
                }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ready[ab]);
        }
    } else {
        // ---------------------------------------------------- scales, sums and the store
        const int q = warp & 3;
        constexpr int kTok = S::kTokens;
        const int tok0 = ((warp - 2 - S::kWidenWarps) >> 2) * kTok;
        Ring<kStages> sb;
        Ring<kABufs> ab;
        Ring<kDBufs> db;
        int place = 0;
        bool stop = false;
        for (int tile = blockIdx.x; tile < total && !stop; tile += gridDim.x) {
            if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
            const I4Tile t = i4_tile(tile, p, &tab, TN, place);
            const int n = t.n0 + 32 * q + lane;
            float acc[kMats][kTok];
#pragma unroll
            for (int m = 0; m < kMats; ++m)
#pragma unroll
                for (int j = 0; j < kTok; ++j) acc[m][j] = 0.f;
#pragma unroll 1
            for (int st = 0; st < nst && !stop; ++st, sb.next()) {
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[sb.i], sb.par, tmo))) stop = true;
                const float* scales = reinterpret_cast<const float*>(smem + sb.i * S::kStage + S::kScaleOff) + 32 * q + lane;
#pragma unroll
                for (int v = 0; v < S::kPerStage; ++v) {
                    constexpr int kG = kUnit * kGroups;  // groups of a unit
                    const int m = v % kMats;
                    float sc[kG];
#pragma unroll
                    for (int g = 0; g < kG; ++g) sc[g] = scales[m * (S::kScales / 4) + (v / kMats * kGroups + g) * kCols];
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&done[ab.i], ab.par, tmo))) stop = true;
                    tc_fence_after();
                    const uint32_t src = d_base + ((uint32_t)(32 * q) << 16) + db.i * S::kDCols + tok0;
#pragma unroll
                    for (int g = 0; g < kG; ++g)
#pragma unroll
                        for (int c = 0; c < kTok; c += 16) {
                            uint32_t r[16];
                            tmem_ld_16(src + g * TN + c, r);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) acc[m][c + j] = fmaf(sc[g], __uint_as_float(r[j]), acc[m][c + j]);
                        }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&taken[db.i]);
                    ab.next();
                    db.next();
                }
                if (lane == 0) mbar_arrive(&empty[sb.i]);
            }
            if (stop) {
                if (lane == 0) give_up(SITE_GEMM_EPI_TMEM_FULL);
                break;
            }
            if (n < p.N) {
                const float bias = p.bias != nullptr ? __bfloat162float(p.bias[(int64_t)t.e * p.N + n]) : 0.f;
                __nv_bfloat16* o = p.out + (int64_t)(t.row0 + tok0) * p.N + n;
#pragma unroll
                for (int j = 0; j < kTok; ++j)
                    if (tok0 + j < t.rows) {
                        float v = acc[0][j] + bias;
                        if (MODE == I4_SWIGLU) v = silu_f(v) * acc[kMats - 1][j];
                        if (MODE == I4_GELU) {
                            float cdf, pdf;
                            normal_cdf_pdf(v, cdf, pdf);
                            v *= cdf;
                        }
                        o[(int64_t)j * p.N] = __float2bfloat16_rn(v);
                    }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

struct Int4Operands {
    const void* x = nullptr;   // [rows, K]
    const void* q0 = nullptr;  // codes
    const void* q1 = nullptr;
    int K = 0;
};

template <int MODE, int GS, int TN>
cudaError_t launch_shape(const Int4Operands& o, Int4Params p, cudaStream_t s) {
    static std::atomic<bool> attr[64];
    const cudaError_t err = ensure_smem_attr(attr, int4_kernel<MODE, GS, TN>, I4Smem<MODE, GS, TN>::kBytes);
    if (err != cudaSuccess) return err;
    CUtensorMap q0, q1, x;
    bool ok = make_map_u8(&q0, o.q0, (int64_t)p.E * p.N, (int64_t)p.blocks * 64, 128, kCols);
    ok = ok && make_map_u8(&q1, MODE == I4_SWIGLU ? o.q1 : o.q0, (int64_t)p.E * p.N, (int64_t)p.blocks * 64, 128, kCols);
    ok = ok && make_map(&x, o.x, (uint64_t)o.K, (uint64_t)p.rows, (uint64_t)o.K * 2, 64, TN);
    CUtensorMap s0, s1;
    ok = ok && make_map_3d_f32_plain(&s0, p.s0, p.E, p.groups, p.N, kCols, 2 * (4 / GS));
    ok = ok && make_map_3d_f32_plain(&s1, MODE == I4_SWIGLU ? p.s1 : p.s0, p.E, p.groups, p.N, kCols, 2 * (4 / GS));
    if (!ok) return cudaErrorInvalidValue;
    p.n_tiles = (p.N + kCols - 1) / kCols;
    // experts that can hold a row, and the passes of TN rows
    const int64_t tiles = (min64(p.E, p.rows) + p.rows / TN) * p.n_tiles;
    return launch_kernel(int4_kernel<MODE, GS, TN>, dim3((unsigned)min64(tiles, sm_count())), dim3(I4Smem<MODE, GS, TN>::kThreads),
                         I4Smem<MODE, GS, TN>::kBytes, s, q0, q1, x, s0, s1, p);
}

template <int MODE, int GS>
cudaError_t launch_group(const Int4Operands& o, const Int4Params& p, cudaStream_t s) {
    // Measured, tiles of 16 tokens against 64: 8 experts of 4096 x 4096, 16 rows each 29.4 against 31.2 us, 20 rows
    // 36.5 against 31.7; 64 experts of 2048 x 2048, 16 rows each 54.9 against 60.5 us, 20 rows 62.7 against 61.3 (groups
    // of 32, against 32: 60.7 and 55.8, 70.2 and 56.3).  Where 64 leave two fifths of the SMs without a tile, 16 are
    // faster for any number of rows (2 of 1024 x 1024, 64 rows: 7.1 against 7.9; 4 of 1024 x 2048, 24 rows: 6.9 against
    // 8.4, but 32 rows, 96 tiles: 9.3 against 8.6).
    const int64_t tiles64 = ((int64_t)p.rows / 64 + p.E) * ((p.N + kCols - 1) / kCols);
    if ((int64_t)p.rows <= 16 * (int64_t)p.E || 5 * tiles64 <= 3 * sm_count()) return launch_shape<MODE, GS, 16>(o, p, s);
    return launch_shape<MODE, GS, MODE == I4_SWIGLU || GS == 1 ? 32 : 64>(o, p, s);
}

template <int MODE>
cudaError_t launch_int4(const Int4Operands& o, const Int4Params& p, int group, cudaStream_t s) {
    if (group == 32) return launch_group<MODE, 1>(o, p, s);
    if (group == 64) return launch_group<MODE, 2>(o, p, s);
    return launch_group<MODE, 4>(o, p, s);
}

Int4Params int4_params(const int32_t* offsets, int64_t rows, int E, int K, int N, int group, DevStatus st) {
    Int4Params p;
    p.offsets = offsets;
    p.rows = (int)rows;
    p.E = E;
    p.N = N;
    p.groups = (K + group - 1) / group;
    p.blocks = (K + kBlockK - 1) / kBlockK;
    p.st = st;
    return p;
}

// ------------------------------------------------------------ quantisation
// One thread per (expert, block of 128 k, column): the groups' scales from
// w (or given codes, PACK), then the block's 16 words.
template <bool BF16, bool PACK>
__global__ void __launch_bounds__(128) quantize4_kernel(const void* __restrict__ w, const int8_t* __restrict__ given,
                                                        int K, int N, int group, uint8_t* __restrict__ codes,
                                                        float* __restrict__ scale) {
    const int n = blockIdx.x * 128 + threadIdx.x;
    if (n >= N) return;
    const int64_t e = blockIdx.z;
    const int b = blockIdx.y, blocks = gridDim.y, groups = (K + group - 1) / group;
    auto load = [&](int k) -> float {
        const int64_t i = (e * K + k) * N + n;
        if constexpr (BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
        return static_cast<const float*>(w)[i];
    };
    uint32_t words[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) words[i] = 0x88888888u;  // codes behind K: zero
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // steps of 32 k
        const int k0 = b * kBlockK + 32 * i;
        if (k0 >= K) break;
        if (!PACK && (32 * i) % group == 0) {
            float amax = 0.f;
            bool finite = true;
            for (int k = k0; k < min(k0 + group, K); ++k) {
                const float a = fabsf(load(k));
                finite = finite && a < INFINITY;  // false for NaN, which fmaxf drops
                amax = fmaxf(amax, a);
            }
            s = finite ? amax / 7.0f : NAN;  // no code stands for infinity or NaN: the products show it
            scale[(e * groups + k0 / group) * N + n] = s;
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            uint32_t word = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) {  // place c of the word: k + 2c, or k + 2(c - 4) + 1
                const int k = k0 + 8 * t + (c < 4 ? 2 * c : 2 * (c - 4) + 1);
                int q = 0;
                if (k < K) {
                    if (PACK)
                        q = given[(e * K + k) * N + n];
                    else if (s > 0.f)
                        q = (int)fminf(fmaxf(rintf(load(k) / s), -7.f), 7.f);
                }
                word |= (uint32_t)(min(max(q, -8), 7) + 8) << (4 * c);
            }
            words[4 * t + i] = word;
        }
    }
    uint4* dst = reinterpret_cast<uint4*>(codes + ((e * N + n) * blocks + b) * 64);
#pragma unroll
    for (int t = 0; t < 4; ++t) dst[t] = make_uint4(words[4 * t], words[4 * t + 1], words[4 * t + 2], words[4 * t + 3]);
}

}  // namespace

cudaError_t launch_quantize_int4(const void* w, bool bf16, const int8_t* given, int E, int K, int N, int group,
                                 uint8_t* codes, float* scale, cudaStream_t s) {
    const dim3 grid((unsigned)((N + 127) / 128), (unsigned)((K + kBlockK - 1) / kBlockK), (unsigned)E);
    if (given != nullptr)
        quantize4_kernel<false, true><<<grid, 128, 0, s>>>(nullptr, given, K, N, group, codes, scale);
    else if (bf16)
        quantize4_kernel<true, false><<<grid, 128, 0, s>>>(w, nullptr, K, N, group, codes, scale);
    else
        quantize4_kernel<false, false><<<grid, 128, 0, s>>>(w, nullptr, K, N, group, codes, scale);
    return cudaGetLastError();
}

cudaError_t launch_grouped_int4(const GroupedArgs& a, const float* scale, int group, cudaStream_t s) {
    Int4Params p = int4_params(a.offsets, a.rows, a.E, a.K, a.N, group, a.st);
    p.s0 = scale;
    p.bias = static_cast<const __nv_bfloat16*>(a.bias);
    p.out = static_cast<__nv_bfloat16*>(a.y);
    Int4Operands o;
    o.x = a.x;
    o.q0 = a.w;
    o.K = a.K;
    return launch_int4<I4_PLAIN>(o, p, group, s);
}

cudaError_t launch_ffn_int4(const FfnArgs& a, cudaStream_t s) {
    if (a.rows_cap <= 0) return cudaSuccess;
    const bool swiglu = a.act == 0;
    Int4Params p = int4_params(a.offsets, a.rows_cap, a.E, a.d, a.ffn, a.int4_group, a.st);
    p.s0 = a.w1_scale;
    p.s1 = a.w_up_scale;
    p.bias = swiglu ? nullptr : static_cast<const __nv_bfloat16*>(a.b1);
    p.out = static_cast<__nv_bfloat16*>(a.h);
    Int4Operands o;
    o.x = a.x_perm;
    o.q0 = a.w1;
    o.q1 = a.w_up;
    o.K = a.d;
    cudaError_t err = swiglu ? launch_int4<I4_SWIGLU>(o, p, a.int4_group, s) : launch_int4<I4_GELU>(o, p, a.int4_group, s);
    if (err != cudaSuccess) return err;
    if (a.between != nullptr && (err = record_mark(a.between, s)) != cudaSuccess) return err;
    Int4Params r = int4_params(a.offsets, a.rows_cap, a.E, a.ffn, a.d, a.int4_group, a.st);
    r.s0 = a.w2_scale;
    r.bias = swiglu ? nullptr : static_cast<const __nv_bfloat16*>(a.b2);
    r.out = static_cast<__nv_bfloat16*>(a.y_perm);
    o.x = a.h;
    o.q0 = a.w2;
    o.K = a.ffn;
    return launch_int4<I4_PLAIN>(o, r, a.int4_group, s);
}

}  // namespace moe
