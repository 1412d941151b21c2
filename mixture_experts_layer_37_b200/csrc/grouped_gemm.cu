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
// Persistent CTA pairs (tcgen05 cta_group::2): a cluster of two CTAs computes
// one 256 x 256 tile, each holding 128 of its rows and 128 of its columns in
// shared memory; 352 threads per CTA: warp 0 loads by TMA, one lane of warp 1
// of the leader issues the MMAs (M=256, N=256, K=16, two TMEM accumulators of
// 256 columns), warps 2-9 read the CTA's 128 accumulator rows and store, warp
// 10 clears rows (GW, below).
// Why pairs: one CTA with a 128 x 256 tile reads 12 KB of operands from shared
// memory for each MMA of 128 clocks and receives as much by TMA, 24 KB where
// the memory moves 16; a pair moves 8 KB + 8 KB per SM for the same work.
// Measured alone the change gave 126 -> 121 us at 8192 x 2048 x 4096; elected
// issuers in place of lane 0 give 101 -> 93 us there and 1440 -> 1370 us (1.61
// PFLOP/s) at 65536 rows of 4096 x 4096 (even experts, in a graph).  With uneven
// experts 107 us (of 83 us at the tensor cores' peak), tensor pipe busy 76 % of it;
// fp32 GW that adds to 268 MB of gradients, same sizes: 157 us (98 us at the memory's
// rate, 138 without adding).  There neither memory (47 %) nor the tensor pipe (46 %)
// is full: a tile's sums pass registers and slabs in turn.  Runs of a few milliseconds
// meet the power cap: 16384 x 4096 x 4096 GX takes 482 us at first, 560 in a long row.
// What differs between the three forms is which operand is contiguous along
// the contraction:
//   FWD  A = x rows, contraction-major; B = W[e], output-major (two boxes
//        [64 k x 64 n] per CTA);
//   GX   A = dy rows, contraction-major; B = W[e], contraction-major (one box
//        [128 k x 64 n] per CTA): the weights are read as they lie;
//   GW   both output-major: A = x (two boxes [64 rows x 64 k] per CTA), B = dy
//        (two boxes [64 rows x 64 n]); the contraction runs over the expert's rows.
// Weights and weight gradients are addressed as 3-D tensors [E, K, N], so a K
// or N that fills no tile is cut at the expert's own edge (zero fill on loads,
// clipping on stores) and never mixes with the next expert's values.
//
// Ragged edges.  FWD, GX: a tile that runs past its expert's last row reads
// the next rows and does not store them (rows do not mix).  GW: rows of the
// next expert in the last block of 64 would be summed, and 0 * inf is not 0, so
// they are not multiplied by zero but overwritten: warp 10 of each CTA clears
// the rows of its operands behind the expert's end up to the next multiple of
// 16 in shared memory (at most 15 rows, once per tile) and only that many K=16
// steps are issued.  The last block of an expert therefore lands on a barrier
// of each CTA's own, and the leader waits for the clearing warps of both CTAs
// instead of the copies.  GW tiles are taken expert by expert in order
// of falling row count, so that the last wave holds the cheapest tiles.
// A last tile of at most 128 rows (GW: output rows) runs as an M=128 pair: 64
// rows per CTA, its accumulator in TMEM lanes 0-63 for the first 128 columns
// and 64-127 for the others.
//
// Stores go through shared memory: a warp's 32 rows of 128 bytes, then one TMA
// store, or, for a warp with fewer rows, whole lines by eight lanes per row.  (Lanes storing their own rows 16 bytes
// at a time moved three times the sectors.)
// Every wait is bounded in time, as in the other kernels.
#include <type_traits>

#include "gemm_common.cuh"
#include "grouped.h"

namespace moe {
namespace {

using namespace gemm;

constexpr int BM = 256;                                   // tile rows (128 per CTA)
constexpr int kGroupM2 = 16;                              // m-tiles per raster group
constexpr int kABytes = 128 * BK * 2;                     // 16 KB: this CTA's rows of A
constexpr int kBBytes = 2 * kBBoxBytes;                   // 16 KB: this CTA's columns of B
constexpr int kStageBytes = kABytes + kBBytes;            // 32 KB
constexpr int kEpiWarps = 8;                              // two per 32 TMEM lanes: one for each half of the columns
constexpr int kClearWarp = 2 + kEpiWarps;                // GW: clears the rows behind an expert's end
constexpr int kThreadsG = 32 * (kClearWarp + 1);
constexpr int kSlabBytes = 32 * 128;                      // an epilogue warp's staging: 32 rows of 128 bytes
constexpr int kRunRows = 512;                             // GW, fp32 output: rows summed in TMEM before a promotion

enum { FORM_FWD = 0, FORM_GX = 1, FORM_GW = 2 };
// What the epilogue does with the fp32 accumulators: round to bf16 (with a
// bias in FWD, added to what is there in GW on request), store as fp32, or, in
// FWD, the backward pass of the expert activation (below).
enum { EPI_BF16 = 0, EPI_F32 = 1, EPI_SWIGLU_GRAD = 2, EPI_GELU_GRAD = 3 };

// fp32 outputs take twice the stores of a bf16 tile: two staging slabs per warp, one stage less (fp32 GW that adds to
// 8 x 2048 x 4096 gradients, 8192 rows, measured together: 160 us; three slabs, four stages 187; four, three 208).
template <int EPI>
struct Smem {
    static constexpr int kSlabs = EPI != EPI_F32 ? 1 : 2;
    static_assert(EPI != EPI_F32 || kSlabs == 2, "an accumulating tile refills its slabs two at a time");
    static constexpr int kStages = EPI != EPI_F32 ? 6 : 5;
    static constexpr int kSlabOff = kStages * kStageBytes;
    static constexpr int kBarOff = kSlabOff + kEpiWarps * kSlabs * kSlabBytes;
    static constexpr int kBytes = kBarOff + 512 + 1024 /*alignment*/;
};

struct GroupedParams {
    const int32_t* offsets = nullptr;  // [E+1]
    int rows = 0;                      // rows of the buffers
    int E = 0;                         // GW: parts of the experts' rows
    int split = 1;                     // GW: parts of each expert
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
    float* sums = nullptr;                // GELU: [slabs, N] column sums of d0 before its rounding, or null
    DevStatus st;
};

constexpr uint32_t make_idesc_majors(int m, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// tma_load_2d_pair with three coordinates.
__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const void* map, uint32_t bar_cluster_addr, int32_t c0,
                                                 int32_t c1, int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
        "%5}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

struct Tile {
    int e, m0, row0, rows, nt;  // FWD, GX: rows of this tile from row0; GW: m0 in the output, rows to sum from row0
    bool half;                  // an M=128 pair
};

// Expert by expert; inside an expert groups of kGroupM2 m-tiles, n-tile-major
// inside a group, so that the pairs running together share operands in L2.
// `i`: the caller's place in the tables; its tiles only grow.
template <int FORM>
__device__ __forceinline__ Tile decode(int tile, const GroupedParams& p, const GroupTables* t, int& i) {
    while (t->start[i + 1] * p.n_tiles <= tile) ++i;
    const int local = tile - t->start[i] * p.n_tiles;
    const int mt_e = t->start[i + 1] - t->start[i];
    const int grp = local / (kGroupM2 * p.n_tiles);
    const int gm = min(kGroupM2, mt_e - grp * kGroupM2);
    const int r = local - grp * kGroupM2 * p.n_tiles;
    Tile o;
    o.nt = r / gm;
    const int mt = grp * kGroupM2 + (r - o.nt * gm);
    o.e = t->expert[i];
    o.m0 = mt * BM;
    if (FORM == FORM_GW) {
        o.row0 = t->row0[i];
        o.rows = t->nrows[i];
        o.half = p.M - o.m0 <= BM / 2;
    } else {
        o.row0 = t->row0[i] + o.m0;
        o.rows = min(BM, t->nrows[i] - o.m0);
        o.half = o.rows <= BM / 2;
    }
    return o;
}

template <int FORM>
__device__ __forceinline__ int tile_kblocks(const GroupedParams& p, const Tile& t) {
    return FORM == FORM_GW ? (t.rows + BK - 1) / BK : p.kblocks + p.kblocks2;
}

// 8 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld_8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// A slab: 32 rows (one per lane) of 128 bytes in shared memory, 16-byte pieces
// permuted by the row so that both a lane writing its row and eight lanes
// reading one row touch all banks once.
__device__ __forceinline__ uint4* slab_piece(uint8_t* slab, int row, int piece) {
    return reinterpret_cast<uint4*>(slab + row * 128 + ((piece ^ (row & 7)) << 4));
}
__device__ __forceinline__ uint4 pack8_bf16(const float* v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ uint4 pack4_f32(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
// The slab to memory by eight lanes per row.  row(r) says where row r's first
// column lies, or null where the row is not stored; n = columns left from there.
template <class T, class Row>
__device__ __forceinline__ void store_slab(uint8_t* slab, int lane, int n, Row&& row) {
    __syncwarp();
    const int piece = lane & 7;
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + (lane >> 3);
        const uint4 v = *slab_piece(slab, r, piece);
        T* dst = row(r);
        if (dst != nullptr && piece * kPer < n) *reinterpret_cast<uint4*>(dst + piece * kPer) = v;
    }
    __syncwarp();
}
// The reverse: 32 rows of 128 bytes into registers (zeros where there is no
// row or column), and from there into the slab.
template <class T, class Row>
__device__ __forceinline__ void fetch_rows(uint4 (&v)[8], int lane, int n, Row&& row) {
    const int piece = lane & 7;
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const T* src = row(4 * i + (lane >> 3));
        v[i] = make_uint4(0, 0, 0, 0);
        if (src != nullptr && piece * kPer < n) v[i] = *reinterpret_cast<const uint4*>(src + piece * kPer);
    }
}
__device__ __forceinline__ void put_rows(uint8_t* slab, int lane, const uint4 (&v)[8]) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) *slab_piece(slab, 4 * i + (lane >> 3), lane & 7) = v[i];
    __syncwarp();
}

// A slab by TMA to [.., col..] of row `row` (of expert e where the tensor has
// three dimensions).  One lane.
template <bool THREE>
__device__ __forceinline__ void tma_store(const void* map, const uint8_t* slab, int col, int row, int e) {
    const uint64_t m = reinterpret_cast<uint64_t>(map);
    const uint32_t sa = smem_u32(slab);
    if (THREE)
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(m),
                     "r"(sa), "r"(col), "r"(row), "r"(e)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(m), "r"(sa),
                     "r"(col), "r"(row)
                     : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// At most N of this thread's stores still read their slabs.
template <int N>
__device__ __forceinline__ void tma_store_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// mbar_arrive_cluster without releasing this thread's writes.  For "accumulator read": the reads are done
// (tcgen05.wait::ld) and ordered by the tcgen05 fence, and whoever waits reads nothing that this thread wrote,
// while a releasing arrival waits for the tile's own global stores (1,850 clocks in a one-tile call).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// mbar_wait_bounded for a phase that the other CTA's threads complete after
// writing its shared memory: acquires at cluster scope.
__device__ __forceinline__ bool mbar_wait_bounded_cluster(uint64_t* bar, uint32_t parity, uint64_t timeout_ns) {
    const uint64_t t0 = globaltimer_ns();
    uint32_t n = 0;
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((++n & 15u) == 0 && globaltimer_ns() - t0 > timeout_ns) return false;
    }
}

// The activation's backward pass, from the fp32
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
    float cdf, pdf;
    normal_cdf_pdf(p, cdf, pdf);
    h = p * cdf;
    dp = dh * (cdf + p * pdf);
}

// The sums over a warp's lanes of eight values each, value lane / 4 in this lane: every step but the last two halves
// the values that a lane keeps.
__device__ __forceinline__ float sum_lanes_8(float (&v)[8], int lane) {
#pragma unroll
    for (int w = 16, n = 4; w >= 4; w >>= 1, n >>= 1)
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = lane & w ? v[i] : v[i + n], keep = lane & w ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

template <int FORM, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreadsG, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmA2, const __grid_constant__ CUtensorMap tmB2,
                   const __grid_constant__ CUtensorMap tmO, GroupedParams p) {
    using S = Smem<EPI>;
    constexpr int kStages = S::kStages;
    constexpr bool kTwoB = EPI == EPI_SWIGLU_GRAD;  // gate and up halves of each CTA's columns
    constexpr bool kGw = FORM == FORM_GW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sA = smem;
    uint8_t* sB = smem + kStages * kABytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBarOff);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint64_t* tail = drain + 1;  // [stage] GW: this CTA's part of an expert's last, partly filled block
    uint64_t* ready = tail + kStages;  // [stage] GW, leader: both CTAs have cleared such a block
    uint64_t* olds = ready + kStages;  // [epilogue warp][kSlabs] GW, fp32: what is there, in the warp's slabs
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(olds + S::kSlabs * kEpiWarps);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    __shared__ GroupTables tab;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&tail[s], 1);
            mbar_init(&ready[s], 2);
        }
        mbar_init(&tfull[0], 1);
        mbar_init(&tfull[1], 1);
        mbar_init(&tempty[0], 2 * kEpiWarps);
        mbar_init(&tempty[1], 2 * kEpiWarps);
        mbar_init(drain, 1);
        for (int i = 0; i < S::kSlabs * kEpiWarps; ++i) mbar_init(&olds[i], 1);
        *abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, kTmemCols);
        tmem_relinquish_pair();
    }
    // the prologue above overlaps the launch before; from here on its results are read
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 2) build_group_tables<kGw>(p.offsets, p.rows, p.E, BM, p.m_tiles, p.st, &tab, lane, kGw ? p.split : 1);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA signal
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int total_tiles = tab.start[p.E] * p.n_tiles;
    const uint64_t tmo = p.st.timeout_ns;
    const uint32_t full_lead = mapa_shared(smem_u32(full), 0);      // the leader's full[0]
    const uint32_t ready_lead = mapa_shared(smem_u32(ready), 0);    // the leader's ready[0]
    const uint32_t tempty_lead = mapa_shared(smem_u32(tempty), 0);  // the leader's tempty[0]

    auto give_up = [&](uint32_t site) {
        report_timeout(p.st, site);
        *abort_flag = 1;
    };

    if (warp == 0) {
        if (elect_one()) {
            // ------------------------------------------------ TMA producer (both CTAs)
            int stage = 0, place = 0;
            uint32_t phase = 0, issued_mask = 0, issued_par = 0;
            bool stop = false;
            for (int tile = pair; tile < total_tiles && !stop; tile += npairs) {
                const Tile t = decode<FORM>(tile, p, &tab, place);
                const int kbs = tile_kblocks<FORM>(p, t);
                const int own = (t.half ? 64 : 128) * rank;                    // this CTA's rows of the tile
                const int n0 = t.nt * p.bn_out + (kTwoB ? 64 : 128) * rank;    // and its columns
                if (*abort_flag) break;
                for (int kb = 0; kb < kbs; ++kb) {
                    if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, tmo)) {
                        give_up(SITE_GEMM_PRODUCER_EMPTY);
                        stop = true;
                        break;
                    }
                    uint8_t* a_dst = sA + stage * kABytes;
                    uint8_t* b_dst = sB + stage * kBBytes;
                    const uint32_t bar = full_lead + 8u * stage;
                    if (kGw) {
                        const int r = t.row0 + kb * BK;
                        if (t.rows - kb * BK < BK) {
                            // the expert's last, partly filled block: cleared before it counts as full
                            mbar_arrive_expect_tx(&tail[stage], kStageBytes);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                tma_load_2d(a_dst + i * kBBoxBytes, &tmA, &tail[stage], t.m0 + own + 64 * i, r);
                                tma_load_2d(b_dst + i * kBBoxBytes, &tmB, &tail[stage], n0 + 64 * i, r);
                            }
                        } else {
                            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                tma_load_2d_pair(a_dst + i * kBBoxBytes, &tmA, bar, t.m0 + own + 64 * i, r);
                                tma_load_2d_pair(b_dst + i * kBBoxBytes, &tmB, bar, n0 + 64 * i, r);
                            }
                        }
                    } else {
                        if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
                        if (FORM == FORM_GX) {
                            const bool second = kb >= p.kblocks;
                            const int c = (second ? kb - p.kblocks : kb) * BK;
                            tma_load_2d_pair(a_dst, second ? &tmA2 : &tmA, bar, c, t.row0 + own);
                            tma_load_3d_pair(b_dst, second ? &tmB2 : &tmB, bar, c, n0, t.e);
                        } else {
                            tma_load_2d_pair(a_dst, &tmA, bar, kb * BK, t.row0 + own);
                            tma_load_3d_pair(b_dst, &tmB, bar, n0, kb * BK, t.e);
                            tma_load_3d_pair(b_dst + kBBoxBytes, kTwoB ? &tmB2 : &tmB, bar, kTwoB ? n0 : n0 + 64, kb * BK,
                                             t.e);
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
            // the loads land before the MMAs that read them complete: wait for the last release of every stage
            for (int s = 0; s < kStages; ++s)
                if ((issued_mask >> s) & 1u)
                    if (!mbar_wait_bounded(&empty[s], (issued_par >> s) & 1u, tmo)) give_up(SITE_GEMM_PRODUCER_DRAIN);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            if (rank == 0) {
                // -------------------------------------------- MMA issuer (leader)
                // Its loop is kept short: with warp-wide votes and an abort check in every block, 236 of a
                // block's 695 clocks passed between the MMAs (512 of work).
                int stage = 0, place = 0, acc = 0;
                uint32_t full_par = 0, ready_par = 0;  // parity of each stage's next use of that barrier
                uint32_t acc_phase = 0;
                bool stop = false;
                constexpr bool kAMn = kGw, kBMn = FORM != FORM_GX;
                // blocks of 64 that one accumulator sums: all, or (GW, fp32 output) a run
                constexpr int kRun = kGw && EPI == EPI_F32 ? kRunRows / BK : 1 << 30;
                // contraction-major: +32 bytes per K=16 step inside the 128-byte swizzle row;
                // output-major: +16 rows of 128 bytes per step, 64-column boxes 8 KB apart
                const uint64_t a_desc0 = smem_desc_sw128(smem_u32(sA), kAMn ? kBBoxBytes : 16, 1024);
                const uint64_t b_desc0 = smem_desc_sw128(smem_u32(sB), kBMn ? kBBoxBytes : 16, 1024);
                constexpr uint32_t kAStep = (kAMn ? 2048 : 32) >> 4, kBStep = (kBMn ? 2048 : 32) >> 4;
                for (int tile = pair; tile < total_tiles && !stop; tile += npairs) {
                    if (*abort_flag) break;
                    const Tile t = decode<FORM>(tile, p, &tab, place);
                    const int kbs = tile_kblocks<FORM>(p, t);
                    if (kbs == 0) continue;  // GW, an expert without rows: the epilogue stores zeros by itself
                    const uint32_t idesc = t.half ? make_idesc_majors(BM / 2, BN_MMA, kAMn, kBMn)
                                                  : make_idesc_majors(BM, BN_MMA, kAMn, kBMn);
                    for (int kb = 0; kb < kbs; ++kb) {
                        const int kr = kb % kRun;  // block of this run
                        if (kr == 0) {             // a new accumulator
                            if (kb > 0) {
                                tc_commit_pair_mc(&tfull[acc], 0x3);
                                acc ^= 1;
                                if (acc == 0) acc_phase ^= 1u;
                            }
                            if (!mbar_wait_bounded(&tempty[acc], acc_phase ^ 1u, tmo)) {
                                give_up(SITE_GEMM_MMA_TMEM_EMPTY);
                                stop = true;
                                break;
                            }
                        }
                        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN_MMA);
                        int steps = BK / 16;
                        bool ok;
                        if (kGw && t.rows - kb * BK < BK) {
                            steps = (t.rows - kb * BK + 15) / 16;
                            ok = mbar_wait_bounded_cluster(&ready[stage], (ready_par >> stage) & 1u, tmo);
                            ready_par ^= 1u << stage;
                        } else {
                            ok = mbar_wait_bounded(&full[stage], (full_par >> stage) & 1u, tmo);
                            full_par ^= 1u << stage;
                        }
                        if (!ok) {
                            give_up(SITE_GEMM_MMA_FULL);
                            stop = true;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t a0 = a_desc0 + (uint32_t)stage * (kABytes >> 4);
                        const uint64_t b0 = b_desc0 + (uint32_t)stage * (kBBytes >> 4);
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            if (!kGw || kk < steps)
                                tc_mma_f16_pair(d_tmem, a0 + kk * kAStep, b0 + kk * kBStep, idesc,
                                                (kr | kk) != 0 ? 1u : 0u);
                        tc_commit_pair_mc(&empty[stage], 0x3);
                        if (++stage == kStages) stage = 0;
                    }
                    if (stop) break;
                    tc_commit_pair_mc(&tfull[acc], 0x3);
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1u;
                }
                // every pair MMA has completed before either CTA frees its TMEM
                tc_commit_pair_mc(drain, 0x3);
            }
            if (!mbar_wait_bounded(drain, 0, tmo)) give_up(SITE_GEMM_DRAIN);
        }
        __syncwarp();
    } else if (warp == kClearWarp) {
        // ---------------------------------------------------- clearing (GW, both CTAs)
        if (kGw) {
            int stage = 0, place = 0;
            uint32_t tail_par = 0;  // parity of each stage's next tail
            for (int tile = pair; tile < total_tiles; tile += npairs) {
                if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
                const Tile t = decode<FORM>(tile, p, &tab, place);
                const int kbs = tile_kblocks<FORM>(p, t);
                const int held = t.rows % BK;
                if (held != 0) {
                    const int st = (stage + kbs - 1) % kStages;
                    const bool ok = mbar_wait_bounded(&tail[st], (tail_par >> st) & 1u, tmo);
                    if (!__all_sync(0xffffffffu, ok)) {
                        if (lane == 0) give_up(SITE_GROUPED_TAIL);
                        break;
                    }
                    tail_par ^= 1u << st;
                    // rows [held, next multiple of 16) of this CTA's four boxes, 128 bytes each
                    const int n = ((held + 15) / 16 * 16 - held) * 8;
                    uint8_t* a = sA + st * kABytes + held * 128;
                    uint8_t* b = sB + st * kBBytes + held * 128;
                    for (int i = lane; i < n; i += 32)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            *reinterpret_cast<uint4*>(a + x * kBBoxBytes + i * 16) = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4*>(b + x * kBBoxBytes + i * 16) = make_uint4(0, 0, 0, 0);
                        }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(ready_lead + 8u * st);
                }
                stage = (stage + kbs) % kStages;
            }
        }
    } else {
        // ---------------------------------------------------- epilogue (both CTAs)
        const int q = warp & 3;            // TMEM lanes 32q..32q+31 are reachable from this warp
        const int hc = (warp - 2) >> 2;    // which half of the columns it takes
        uint8_t* slabs = smem + S::kSlabOff + (warp - 2) * S::kSlabs * kSlabBytes;
        uint64_t* old = olds + S::kSlabs * (warp - 2);
        int acc = 0, place = 0, turn = 0;
        uint32_t acc_phase = 0, old_par = 0;
        // the next accumulator, complete; false: gave up
        auto acquire = [&]() -> bool {
            const bool ok = mbar_wait_bounded(&tfull[acc], acc_phase, tmo);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) give_up(SITE_GEMM_EPI_TMEM_FULL);
                return false;
            }
            tc_fence_after();
            return true;
        };
        auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(tempty_lead + 8u * acc);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        };
        // a slab that no earlier store still reads
        auto next_slab = [&]() -> uint8_t* {
            if (lane == 0) tma_store_wait_read<S::kSlabs - 1>();
            __syncwarp();
            uint8_t* slab = slabs + turn * kSlabBytes;
            turn = (turn + 1) % S::kSlabs;
            return slab;
        };
        for (int tile = pair; tile < total_tiles; tile += npairs) {
            const int ab = __shfl_sync(0xffffffffu, *abort_flag, 0);
            if (ab) break;
            const Tile t = decode<FORM>(tile, p, &tab, place);
            // full tile: rows 32q.. of this CTA's 128, TMEM columns [128 hc, +128); half tile: rows 32 (q & 1)..
            // of its 64, output columns from 128 (q >> 1), TMEM columns [64 hc, +64)
            const int r0 = t.half ? 64 * rank + 32 * (q & 1) : 128 * rank + 32 * q;
            const int rn = min(32, (kGw ? p.M - t.m0 : t.rows) - r0);  // rows of this warp (none: <= 0)
            const int row = (kGw ? t.m0 : t.row0) + r0;                // the first of them (GW: of the expert's matrix)
            const int64_t first = kGw ? (int64_t)t.e * p.M + row : row;
            const int tc0 = t.half ? 64 * hc : 128 * hc;               // its TMEM columns
            const int ncols = t.half ? 64 : 128;
            // output column of TMEM column tc0 (SwiGLU: of output tc0 / 2, see below)
            const int col0 = t.nt * p.bn_out + (t.half ? 128 * (q >> 1) : 0) + tc0;
            // row r of this warp at column col of a [.., N] tensor
            auto at_col = [&](auto* base, int col) {
                return [=](int r) { return r < rn ? base + (first + r) * p.N + col : nullptr; };
            };
            const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16) + tc0;
            if (kGw && EPI == EPI_F32) {
                // runs of kRunRows rows are summed in TMEM and the runs in registers (round to nearest): the
                // tensor cores' own fp32 sums lose toward zero.  Relative norm of the error at 16384 rows, normal
                // inputs: 1.9e-5 in one run, 4.8e-7 in these; at 1024 rows 9.9e-7 and 4.7e-7
                float x[128];
#pragma unroll
                for (int i = 0; i < 128; ++i) x[i] = 0.f;
                // Accumulating: what is there waits in the slabs and is added once, to the finished sums (sums begun
                // from it would be rounded at its magnitude by every run: 67 units in the last place after 32).  The
                // first slabs are loaded while the products run, the others when these are stored: 8192 x 2048 x
                // 4096, 8 experts, 160 us (uneven) and 142 (even); sums begun from the old values, all of them loaded
                // meanwhile, 167 and 160; added by the memory (TMA reduction) 187 and 192.
                const bool add = p.accumulate && rn > 0 && t.rows > 0;
                auto load_old = [&](int c) {  // columns c.. into their slab (one lane)
                    const int s = c / 32 % S::kSlabs;
                    if (c >= ncols || col0 + c >= p.N) return;
                    mbar_arrive_expect_tx(&old[s], kSlabBytes);
                    tma_load_3d(slabs + s * kSlabBytes, &tmO, &old[s], col0 + c, row, t.e);
                };
                if (add) {
                    if (lane == 0) {
                        tma_store_wait_read<0>();
#pragma unroll
                        for (int s = 0; s < S::kSlabs; ++s) load_old(32 * s);
                    }
                    __syncwarp();
                }
                const int runs = (tile_kblocks<FORM>(p, t) * BK + kRunRows - 1) / kRunRows;
                bool ok = true;
#pragma unroll 1
                for (int run = 0; run < runs && ok; ++run) {
                    ok = acquire();
                    const uint32_t tb = tq + (uint32_t)(acc * BN_MMA);
#pragma unroll
                    for (int c = 0; c < 128; c += 16) {
                        if (c >= ncols) break;
                        uint32_t v[16];
                        tmem_ld_16(tb + c, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[c + i] += __uint_as_float(v[i]);
                    }
                    release();
                }
                if (!ok) {
                    if (add)  // the loads in flight land before the CTA leaves
                        for (int s = 0; s < S::kSlabs; ++s)
                            if (32 * s < ncols && col0 + 32 * s < p.N) mbar_wait_bounded(&old[s], (old_par >> s) & 1u, tmo);
                    break;
                }
                if (rn <= 0 || (runs == 0 && p.accumulate)) continue;
                if (add) {
                    bool in = true;
#pragma unroll
                    for (int c = 0; c < 128; c += 32) {
                        if (c >= ncols || col0 + c >= p.N) break;
                        const int s = c / 32 % S::kSlabs;
                        uint8_t* slab = slabs + s * kSlabBytes;
                        in = __all_sync(0xffffffffu, mbar_wait_bounded(&old[s], (old_par >> s) & 1u, tmo));
                        old_par ^= 1u << s;
                        if (!in) {
                            // the load into the other slab, issued with this one, lands before the CTA leaves
                            if (s == 0 && c + 32 < ncols && col0 + c + 32 < p.N)
                                mbar_wait_bounded(&old[1], (old_par >> 1) & 1u, tmo);
                            break;
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float4* v = reinterpret_cast<float4*>(slab_piece(slab, lane, j));
                            const float4 o = *v;
                            const float* a = x + c + 4 * j;
                            *v = make_float4(o.x + a[0], o.y + a[1], o.z + a[2], o.w + a[3]);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store<true>(&tmO, slab, col0 + c, row, t.e);
                            if (s == S::kSlabs - 1) {
                                // the next columns into the slabs, each once its store has read it
                                tma_store_wait_read<1>();
                                load_old(c + 32);
                                tma_store_wait_read<0>();
                                load_old(c + 64);
                            }
                        }
                        __syncwarp();
                    }
                    if (!in) {
                        if (lane == 0) give_up(SITE_GROUPED_OLD);
                        break;
                    }
                    continue;
                }
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    if (c >= ncols || col0 + c >= p.N) break;
                    uint8_t* slab = next_slab();
#pragma unroll
                    for (int j = 0; j < 8; ++j) *slab_piece(slab, lane, j) = pack4_f32(x + c + 4 * j);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) tma_store<true>(&tmO, slab, col0 + c, row, t.e);
                }
                continue;
            }
            const bool none = tile_kblocks<FORM>(p, t) == 0;  // GW, an expert without rows
            // what the epilogue reads from memory is fetched before the accumulator is waited for
            constexpr bool kGrad = EPI == EPI_SWIGLU_GRAD || EPI == EPI_GELU_GRAD;
            constexpr int kGradUnroll = EPI == EPI_SWIGLU_GRAD ? 4 : 1;
            constexpr bool kFetch = kGrad || (kGw && EPI == EPI_BF16);
            // SwiGLU: each CTA's 128 columns are [gate 64 | up 64] of the same 64 outputs; a warp takes the
            // 64 outputs of its half (full tile) or 32 of them (half tile)
            const int gcol0 = t.nt * 128 + (t.half ? 64 * (q >> 1) + 32 * hc : 64 * hc);
            uint4 seen[kFetch ? 2 : 1][8];
            if (kGw && EPI == EPI_BF16) {
                if (p.accumulate && !none) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const int col = col0 + 64 * s;
                        fetch_rows<__nv_bfloat16>(seen[s], lane, 64 * s < ncols ? p.N - col : 0,
                                                  at_col(static_cast<const __nv_bfloat16*>(p.out), col));
                    }
                }
            }
            uint2 bias = make_uint2(0, 0);  // FWD: lane i holds the bias of the warp's columns 4i..4i+3
            if (FORM == FORM_FWD && EPI == EPI_BF16 && p.bias != nullptr && col0 + 4 * lane < p.N)
                bias = __ldg(reinterpret_cast<const uint2*>(p.bias + (int64_t)t.e * p.N + col0 + 4 * lane));
            if (kGrad) {
                const int g0 = EPI == EPI_SWIGLU_GRAD ? gcol0 : col0;
#pragma unroll
                for (int s = 0; s < 2; ++s) fetch_rows<float>(seen[s], lane, p.N - (g0 + 32 * s), at_col(p.dh, g0 + 32 * s));
            }
            if (!none && !acquire()) break;
            const uint32_t tb = tq + (uint32_t)(acc * BN_MMA);
            // fp32 accumulators of 32 columns
            auto load32 = [&](uint32_t taddr, float* x) {
                uint32_t v[2][16];
                tmem_ld_16(taddr, v[0]);
                tmem_ld_16(taddr + 16, v[1]);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(v[i >> 4][i & 15]);
            };
            if (kGrad) {
                // N is a multiple of 32 here (bf16 layers have ffn % 64 == 0): every step of 32 columns is whole.
                // dh comes in and h, the gradients go out through the slab, 32 columns at a time and 8 of them in
                // registers.  Kept in loops: unrolled over a tile's columns, the activations came to more code than
                // the instruction caches hold (GELU backward of 259 tokens, six launches: 82 us, in loops 73).
                const int n = EPI == EPI_SWIGLU_GRAD ? ncols / 2 : ncols;
                const uint32_t ta = EPI == EPI_SWIGLU_GRAD && t.half ? tb - tc0 + 32 * hc : tb;
                const int g0 = EPI == EPI_SWIGLU_GRAD ? gcol0 : col0;
                uint8_t* slab = slabs;
#pragma unroll 1
                for (int c = 0; c < n && g0 + c < p.N; c += 32) {
                    const int col = g0 + c;
                    put_rows(slab, lane, seen[0]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) seen[0][i] = seen[1][i];
                    if (c + 64 < n) fetch_rows<float>(seen[1], lane, p.N - (col + 64), at_col(p.dh, col + 64));
                    uint4 du[4];  // SwiGLU: the gradient of up waits here for the slab
                    uint4 bias[4];
                    if (EPI == EPI_GELU_GRAD) {
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            bias[s] = __ldg(reinterpret_cast<const uint4*>(p.bias + (int64_t)t.e * p.N + col) + s);
                    }
#pragma unroll kGradUnroll
                    for (int s = 0; s < 4; ++s) {
                        uint32_t av[8], uv[8];
                        tmem_ld_8(ta + c + 8 * s, av);
                        if (EPI == EPI_SWIGLU_GRAD) tmem_ld_8(ta + 64 + c + 8 * s, uv);
                        float d[8], h[8], x[8], y[8];
                        *reinterpret_cast<uint4*>(d) = *slab_piece(slab, lane, 2 * s);
                        *reinterpret_cast<uint4*>(d + 4) = *slab_piece(slab, lane, 2 * s + 1);
                        tmem_ld_wait();
                        if (EPI == EPI_GELU_GRAD) {
                            const uint32_t bw[4] = {bias[0].x, bias[0].y, bias[0].z, bias[0].w};
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                x[i] = __uint_as_float(av[i]) + (i & 1 ? bf16_hi(bw[i / 2]) : bf16_lo(bw[i / 2]));
#pragma unroll
                            for (int i = 0; i < 8; ++i) gelu_grad(x[i], d[i], h[i], x[i]);
                            bias[0] = bias[1];
                            bias[1] = bias[2];
                            bias[2] = bias[3];
                            if (p.sums != nullptr) {  // b1's gradient: d0 summed as it is before its rounding
                                float v[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) v[i] = lane < rn ? x[i] : 0.f;
                                const float sum = sum_lanes_8(v, lane);
                                const int64_t at = first_slab(t.row0 - t.m0, t.e) + ((t.m0 + r0) >> 5);
                                if (rn > 0 && (lane & 3) == 0) p.sums[at * p.N + col + 8 * s + (lane >> 2)] = sum;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                swiglu_grad(__uint_as_float(av[i]), __uint_as_float(uv[i]), d[i], h[i], x[i], y[i]);
                            du[s] = pack8_bf16(y);
                        }
                        // into the two pieces just read: h, then the gradient
                        *slab_piece(slab, lane, 2 * s) = pack8_bf16(h);
                        *slab_piece(slab, lane, 2 * s + 1) = pack8_bf16(x);
                    }
                    auto h_row = at_col(p.h, col), g_row = at_col(p.d0, col);
                    const int piece = lane & 7, shift = (piece >> 1) * 8 - piece * 8;  // columns of a piece; the slab's own
                    store_slab<__nv_bfloat16>(slab, lane, 64, [&](int r) {
                        __nv_bfloat16* o = piece & 1 ? g_row(r) : h_row(r);
                        return o != nullptr ? o + shift : nullptr;
                    });
                    if (EPI == EPI_SWIGLU_GRAD) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) *slab_piece(slab, lane, j) = du[j];
                        store_slab<__nv_bfloat16>(slab, lane, 32, at_col(p.d1, col));
                    }
                }
            } else {
                constexpr int kCols = EPI == EPI_F32 ? 32 : 64;  // columns of a slab
                // not unrolled: a call of one tile fetches every instruction that it executes
#pragma unroll 1
                for (int c = 0; c < ncols; c += kCols) {
                    const int col = col0 + c;
                    if (col >= p.N || rn <= 0 || (none && p.accumulate)) break;
                    float x[kCols];
                    if (none) {
#pragma unroll
                        for (int i = 0; i < kCols; ++i) x[i] = 0.f;
                    } else {
                        load32(tb + c, x);
                        if (kCols == 64) load32(tb + c + 32, x + 32);
                    }
                    uint8_t* slab = next_slab();
                    if (FORM == FORM_FWD && EPI == EPI_BF16 && p.bias != nullptr) {
#pragma unroll
                        for (int i = 0; i < kCols / 4; ++i) {
                            const uint32_t b0 = __shfl_sync(0xffffffffu, bias.x, c / 4 + i);
                            const uint32_t b1 = __shfl_sync(0xffffffffu, bias.y, c / 4 + i);
                            x[4 * i] += bf16_lo(b0);
                            x[4 * i + 1] += bf16_hi(b0);
                            x[4 * i + 2] += bf16_lo(b1);
                            x[4 * i + 3] += bf16_hi(b1);
                        }
                    }
                    if (EPI == EPI_F32) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) *slab_piece(slab, lane, j) = pack4_f32(x + 4 * j);
                    } else {
                        if (kGw && p.accumulate) {
                            // what is there, through the slab; added in fp32, one rounding
                            put_rows(slab, lane, seen[0]);
#pragma unroll
                            for (int i = 0; i < 8; ++i) seen[0][i] = seen[kFetch ? 1 : 0][i];
#pragma unroll
                            for (int j = 0; j < kCols / 8; ++j) {
                                const uint4 v = *slab_piece(slab, lane, j);
                                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    x[8 * j + 2 * i] += bf16_lo(w[i]);
                                    x[8 * j + 2 * i + 1] += bf16_hi(w[i]);
                                }
                            }
                            __syncwarp();
                        }
#pragma unroll
                        for (int j = 0; j < kCols / 8; ++j) *slab_piece(slab, lane, j) = pack8_bf16(x + 8 * j);
                    }
                    using Out = typename std::conditional<EPI == EPI_F32, float, __nv_bfloat16>::type;
                    if (kGw || rn == 32) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) tma_store<kGw>(&tmO, slab, col, row, t.e);
                    } else {
                        store_slab<Out>(slab, lane, p.N - col, at_col(static_cast<Out*>(p.out), col));
                        // an empty group, so that the groups count the slabs' uses
                        if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                }
            }
            if (!none) release();
        }
        // the stores have read their slabs; what they write is complete with the grid
        if (lane == 0) tma_store_wait_read<0>();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

// ------------------------------------------------------------------ host side
template <int FORM, int EPI>
cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& a2, const CUtensorMap& b2,
                   const CUtensorMap& o, const GroupedParams& p, int64_t tiles_upper, cudaStream_t s) {
    static std::atomic<int> max_pairs[64];  // resident clusters per device, 0 until measured
    int dev = 0;
    cudaGetDevice(&dev);
    int pairs_cap = dev < 64 ? max_pairs[dev].load(std::memory_order_acquire) : 0;
    if (pairs_cap <= 0) {
        cudaError_t err = cudaFuncSetAttribute(grouped_kernel<FORM, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Smem<EPI>::kBytes);
        if (err != cudaSuccess) return err;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (unsigned)(sm_count() / 2));
        cfg.blockDim = dim3(kThreadsG);
        cfg.dynamicSmemBytes = Smem<EPI>::kBytes;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        err = cudaOccupancyMaxActiveClusters(&n, grouped_kernel<FORM, EPI>, &cfg);
        if (err != cudaSuccess || n <= 0) n = sm_count() / 2;
        pairs_cap = n;
        if (dev < 64) max_pairs[dev].store(n, std::memory_order_release);
    }
    const int pairs = (int)min64(tiles_upper, (int64_t)pairs_cap);
    if (pairs <= 0) return cudaSuccess;
    return launch_kernel(grouped_kernel<FORM, EPI>, dim3(2 * pairs), dim3(kThreadsG), Smem<EPI>::kBytes, s, a, b, a2, b2,
                         o, p);
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
    CUtensorMap mA, mB, mB2, mO;
    if (a.grad_act != GRAD_NONE && a.N % 32 != 0) return cudaErrorInvalidValue;  // its epilogue stores 32 columns whole
    const bool two = a.grad_act == GRAD_SWIGLU;
    bool ok = act_map(&mA, a.x, a.rows, a.K, 128);
    ok = ok && make_map_3d(&mB, a.w, a.E, a.K, a.N, false, 64, BK);
    if (two)
        ok = ok && make_map_3d(&mB2, a.w2, a.E, a.K, a.N, false, 64, BK);
    else
        mB2 = mB;
    if (a.grad_act == GRAD_NONE)
        ok = ok && act_map(&mO, a.y, a.rows, a.N, 32);
    else
        mO = mA;  // three outputs, stored by the warps
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
    p.sums = a.sums;
    const int64_t tiles = row_tiles_upper(a) * p.n_tiles;
    if (two) return launch<FORM_FWD, EPI_SWIGLU_GRAD>(mA, mB, mA, mB2, mO, p, tiles, s);
    if (a.grad_act == GRAD_GELU) return launch<FORM_FWD, EPI_GELU_GRAD>(mA, mB, mA, mB2, mO, p, tiles, s);
    return launch<FORM_FWD, EPI_BF16>(mA, mB, mA, mB2, mO, p, tiles, s);
}

cudaError_t launch_grouped_gx_bf16(const GroupedArgs& a, cudaStream_t s) {
    CUtensorMap mA, mB, mA2, mB2, mO;
    bool ok = act_map(&mA, a.dy, a.rows, a.N, 128);
    ok = ok && make_map_3d(&mB, a.w, a.E, a.K, a.N, false, 64, 128);
    if (a.dy2 != nullptr) {
        ok = ok && act_map(&mA2, a.dy2, a.rows, a.N, 128);
        ok = ok && make_map_3d(&mB2, a.w2, a.E, a.K, a.N, false, 64, 128);
    } else {
        mA2 = mA;
        mB2 = mB;
    }
    ok = ok && (a.out_f32 ? make_map_2d_f32(&mO, a.dx, a.rows, a.K, 32, 32) : act_map(&mO, a.dx, a.rows, a.K, 32));
    if (!ok) return cudaErrorInvalidValue;
    GroupedParams p = params(a);
    p.N = a.K;
    p.kblocks = (a.N + BK - 1) / BK;
    p.kblocks2 = a.dy2 != nullptr ? p.kblocks : 0;
    p.n_tiles = (a.K + 255) / 256;
    p.out = a.dx;
    const int64_t tiles = row_tiles_upper(a) * p.n_tiles;
    return a.out_f32 ? launch<FORM_GX, EPI_F32>(mA, mB, mA2, mB2, mO, p, tiles, s)
                     : launch<FORM_GX, EPI_BF16>(mA, mB, mA2, mB2, mO, p, tiles, s);
}

cudaError_t launch_grouped_gw_bf16(const GroupedArgs& a, cudaStream_t s) {
    CUtensorMap mA, mB, mO;
    bool ok = act_map(&mA, a.x, a.rows, a.K, BK);
    ok = ok && act_map(&mB, a.dy, a.rows, a.N, BK);
    ok = ok && make_map_3d(&mO, a.dw, (int64_t)a.E * a.split, a.K, a.N, a.out_f32, a.out_f32 ? 32 : 64, 32);
    if (!ok) return cudaErrorInvalidValue;
    GroupedParams p = params(a);
    p.E = a.E * a.split;
    p.split = a.split;
    p.M = a.K;
    p.N = a.N;
    p.m_tiles = (a.K + BM - 1) / BM;
    p.n_tiles = (a.N + 255) / 256;
    p.out = a.dw;
    p.accumulate = a.accumulate ? 1 : 0;
    const int64_t tiles = (int64_t)p.E * p.m_tiles * p.n_tiles;
    return a.out_f32 ? launch<FORM_GW, EPI_F32>(mA, mB, mA, mB, mO, p, tiles, s)
                     : launch<FORM_GW, EPI_BF16>(mA, mB, mA, mB, mO, p, tiles, s);
}

}  // namespace moe
