// Grouped matrix products over rows sorted by expert and their gradients in
// fp32 FMA (no TF32): the precision-reference path of float32 configurations,
// and two small kernels of the backward pass (bias gradients; the expert
// activation's gradient on fp32 buffers).  The three forms are those of
// grouped_gemm.cu.
//
// One CTA per output tile, 256 threads, each TM/16 x TN/16 outputs; operands
// staged TK deep through shared memory, the next TK loaded into registers
// while the current ones are used; the FMAs run two at a time (f32x2, each
// rounded as a scalar fmaf).  Every output is one sum in ascending order of
// the contraction.  Rows and columns outside the expert are never read.
// Measured at 2048 rows, 8 experts of 1024 x 1024 (57 us at a nominal 75
// TFLOP/s): GW 102 to 107 us (42 TFLOP/s), the FMA pipe busy 67 % of a CTA's life
// and 57 % of the kernel's (1.7 rounds of resident CTAs), and waiting for it the
// largest stall; FWD 123 and GX 132 us, 52 and 50 % (47 and 44), behind loads from
// memory and shared memory (its wavefronts 68 %).
#include <math.h>

#include "grouped.h"

namespace moe {
namespace {

constexpr int kF32Threads = 256;

enum { FORM_FWD = 0, FORM_GX = 1, FORM_GW = 2 };

struct F32Params {
    const float* A = nullptr;   // FWD: x [rows, K]; GX: dy [rows, N]; GW: x
    const float* B = nullptr;   // FWD, GX: w [E, K, N]; GW: dy
    const float* bias = nullptr;
    float* out = nullptr;
    const int32_t* offsets = nullptr;
    int rows = 0, E = 0, K = 0, N = 0, n_tiles = 0, m_tiles = 0;
    int accumulate = 0;
    int split = 1;              // GW: parts of each expert's rows; E counts them
    DevStatus st;
};

// One operand's [TK x T] piece: PER float4 per thread, from memory that is
// contiguous along the tile (KC = false) or along the contraction (KC = true).
// base points at tile element 0, contraction element 0; ld is the stride of
// the other axis; t_n, k_n say how many of each exist from here.
template <int T, int TK, bool KC>
struct Piece {
    static constexpr int PER = T * TK / 4 / kF32Threads;
    static_assert(PER * 4 * kF32Threads == T * TK, "whole pieces");
    float4 v[PER];
    __device__ __forceinline__ void load(const float* base, int64_t ld, int t_n, int k0, int k_n) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int id = threadIdx.x + i * kF32Threads;
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int k = k0 + (KC ? id % (TK / 4) * 4 : id / (T / 4));
            const int t = KC ? id / (TK / 4) : id % (T / 4) * 4;
            if (k < k_n && t < t_n)
                v[i] = *reinterpret_cast<const float4*>(base + (KC ? t * ld + k : k * ld + t));
        }
    }
    __device__ __forceinline__ void store(float (*s)[T + 4]) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int id = threadIdx.x + i * kF32Threads;
            if (KC) {
                const int k = id % (TK / 4) * 4, t = id / (TK / 4);
                s[k][t] = v[i].x;
                s[k + 1][t] = v[i].y;
                s[k + 2][t] = v[i].z;
                s[k + 3][t] = v[i].w;
            } else {
                *reinterpret_cast<float4*>(&s[id / (T / 4)][id % (T / 4) * 4]) = v[i];
            }
        }
    }
};

// A thread's outputs: rows ty*RM + 64*i.. in groups of at most 4, columns the same.
template <int FORM, int TM, int TN, int TK>
__global__ void __launch_bounds__(kF32Threads, 2) grouped_f32_kernel(F32Params p) {
    constexpr int RM = TM / 16, RN = TN / 16;          // outputs per thread: RM rows, RN columns
    constexpr int GM = RM < 4 ? RM : 4, GN = RN < 4 ? RN : 4;  // contiguous run of each
    __shared__ GroupTables tab;
    __shared__ __align__(16) float sA[2][TK][TM + 4];
    __shared__ __align__(16) float sB[2][TK][TN + 4];
    griddep_wait();
    griddep_launch_dependents();
    if (threadIdx.x < 32)
        build_group_tables<FORM == FORM_GW>(p.offsets, p.rows, p.E, TM, p.m_tiles, p.st, &tab, threadIdx.x,
                                            FORM == FORM_GW ? p.split : 1);
    __syncthreads();
    const int tile = blockIdx.x;
    if (tile >= tab.start[p.E] * p.n_tiles) return;
    int i = 0;
    while (tab.start[i + 1] * p.n_tiles <= tile) ++i;
    const int local = tile - tab.start[i] * p.n_tiles;
    const int m0 = local / p.n_tiles * TM, n0 = local % p.n_tiles * TN;
    const int e = tab.expert[i];
    const int out_n = FORM == FORM_GX ? p.K : p.N;                                   // output columns
    const int m_n = (FORM == FORM_GW ? p.K : tab.nrows[i]) - m0, n_n = out_n - n0;   // outputs from here
    const int k_n = FORM == FORM_FWD ? p.K : FORM == FORM_GX ? p.N : tab.nrows[i];   // contraction length
    const int64_t row0 = tab.row0[i];
    const float *a, *b;
    int64_t lda, ldb;
    if (FORM == FORM_FWD) {
        a = p.A + (row0 + m0) * p.K;
        lda = p.K;
        b = p.B + (int64_t)e * p.K * p.N + n0;
        ldb = p.N;
    } else if (FORM == FORM_GX) {
        a = p.A + (row0 + m0) * p.N;
        lda = p.N;
        b = p.B + (int64_t)e * p.K * p.N + (int64_t)n0 * p.N;
        ldb = p.N;
    } else {
        a = p.A + row0 * p.K + m0;
        lda = p.K;
        b = p.B + row0 * p.N + n0;
        ldb = p.N;
    }
    Piece<TM, TK, FORM != FORM_GW> pa;
    Piece<TN, TK, FORM == FORM_GX> pb;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    uint64_t acc[RM][RN / 2];
#pragma unroll
    for (int r = 0; r < RM; ++r)
#pragma unroll
        for (int c = 0; c < RN / 2; ++c) acc[r][c] = 0ull;
    pa.load(a, lda, m_n, 0, k_n);
    pb.load(b, ldb, n_n, 0, k_n);
    int buf = 0;
    for (int k0 = 0; k0 < k_n; k0 += TK) {
        pa.store(sA[buf]);
        pb.store(sB[buf]);
        __syncthreads();
        if (k0 + TK < k_n) {
            pa.load(a, lda, m_n, k0 + TK, k_n);
            pb.load(b, ldb, n_n, k0 + TK, k_n);
        }
#pragma unroll
        for (int k = 0; k < TK; ++k) {
            float av[RM];
            uint64_t bv[RN / 2];
#pragma unroll
            for (int g = 0; g < RM / GM; ++g)
#pragma unroll
                for (int j = 0; j < GM; ++j) av[g * GM + j] = sA[buf][k][g * 16 * GM + ty * GM + j];
#pragma unroll
            for (int g = 0; g < RN / GN; ++g)
#pragma unroll
                for (int j = 0; j < GN / 2; ++j)
                    bv[g * GN / 2 + j] =
                        *reinterpret_cast<const uint64_t*>(&sB[buf][k][g * 16 * GN + tx * GN + 2 * j]);
#pragma unroll
            for (int r = 0; r < RM; ++r) {
                const uint64_t ar = pack2(av[r], av[r]);
#pragma unroll
                for (int c = 0; c < RN / 2; ++c) acc[r][c] = fma2(ar, bv[c], acc[r][c]);
            }
        }
        buf ^= 1;  // the other buffer was last read before this iteration's barrier
    }
#pragma unroll
    for (int r = 0; r < RM; ++r) {
        const int m = r / GM * 16 * GM + ty * GM + r % GM;
        if (m >= m_n) continue;
        float* orow = p.out + (FORM == FORM_GW ? (int64_t)e * p.K + m0 + m : row0 + m0 + m) * out_n;
#pragma unroll
        for (int c = 0; c < RN; c += 2) {
            const int n = c / GN * 16 * GN + tx * GN + c % GN;
            if (n >= n_n) continue;  // sizes are multiples of 4: pairs are whole
            float v0, v1;
            unpack2(acc[r][c / 2], v0, v1);
            if (FORM == FORM_FWD && p.bias != nullptr) {
                v0 += p.bias[(int64_t)e * p.N + n0 + n];
                v1 += p.bias[(int64_t)e * p.N + n0 + n + 1];
            }
            float2* dst = reinterpret_cast<float2*>(orow + n0 + n);
            if (FORM != FORM_FWD && p.accumulate) {
                const float2 old = *dst;
                v0 += old.x;
                v1 += old.y;
            }
            *dst = make_float2(v0, v1);
        }
    }
}

template <int FORM, int TM, int TN, int TK>
cudaError_t launch_tiles(F32Params p, int out_m, int out_n, cudaStream_t s) {
    p.n_tiles = (out_n + TN - 1) / TN;
    p.m_tiles = (out_m + TM - 1) / TM;
    const int64_t row_tiles = FORM == FORM_GW ? (int64_t)p.E * p.m_tiles : (int64_t)p.rows / TM + p.E;
    return launch_kernel(grouped_f32_kernel<FORM, TM, TN, TK>, dim3((unsigned)(row_tiles * p.n_tiles)),
                         dim3(kF32Threads), 0, s, p);
}

template <int FORM>
cudaError_t launch_form(const GroupedArgs& a, const F32Params& p, int out_m, int out_n, cudaStream_t s) {
    auto tiles = [&](int tm, int tn) {
        return (FORM == FORM_GW ? (int64_t)p.E * ((out_m + tm - 1) / tm) : (a.rows + tm - 1) / tm) * ((out_n + tn - 1) / tn);
    };
    const int64_t sms = sm_count();
    // The largest tile that still gives every SM work: 1024 x 1024 weights, 8 experts, 2048 rows, FWD 119 us with
    // 64 x 128 (256 tiles), 146 us with 64 x 64, 200 us with 128 x 128 (128); GW 101 us with 128 x 128 (512 tiles),
    // 107 us with 64 x 128; 512 x 512, 512 rows, FWD 24 us with 64 x 64 (64 tiles), 35 us with 64 x 128, 30 us with
    // 32 x 32; 128 x 256, 4 experts, 128 rows, 4.9 us with 32 x 32, 7.4 us with 64 x 64 (8 tiles).
    if constexpr (FORM == FORM_GW)
        if (tiles(128, 128) >= 2 * sms) return launch_tiles<FORM, 128, 128, 16>(p, out_m, out_n, s);
    if (tiles(64, 128) >= sms) return launch_tiles<FORM, 64, 128, 16>(p, out_m, out_n, s);
    if (tiles(64, 64) >= sms / 3) return launch_tiles<FORM, 64, 64, 32>(p, out_m, out_n, s);
    return launch_tiles<FORM, 32, 32, 32>(p, out_m, out_n, s);
}

F32Params params(const GroupedArgs& a) {
    F32Params p;
    p.offsets = a.offsets;
    p.rows = (int)a.rows;
    p.E = a.E;
    p.K = a.K;
    p.N = a.N;
    p.accumulate = a.accumulate ? 1 : 0;
    p.st = a.st;
    return p;
}

// ------------------------------------------------------------ bias gradients
constexpr int kColWarps = 16;  // a lane holds 4 columns

struct ColsumJob {
    const void* dy = nullptr;  // [rows, N], or fp32 sums of slabs of its rows
    void* db = nullptr;        // [E, N], or [E, split, N]
    int N = 0;
    bool slabs = false;
};
struct ColsumParams {
    ColsumJob job[2];
    int tiles0 = 0;  // tiles of 128 columns of the first job; the second's follow
    const int32_t* offsets = nullptr;
    int rows = 0, E = 0, accumulate = 0, split = 1;
    DevStatus st;
};

template <bool IN_BF16>
__device__ __forceinline__ float4 load4(const void* base, int64_t i) {
    if (IN_BF16) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + i);
        return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
    }
    return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
}

// One CTA per (expert or part of its rows, 128 columns): warp w adds the rows w,
// w+16, ... in two interleaved sums, eight rows loaded at a time (the loads'
// latency bounds this kernel), and the warps' sums are added in a fixed order.
// b1's gradient of a bf16 GELU FFN takes, instead of rows, the sums of 32 rows
// each that the activation's epilogue left (unrounded, where the rows themselves
// are rounded for the products).
template <bool IN_BF16, bool OUT_BF16>
__global__ void __launch_bounds__(kColWarps * 32) colsum_kernel(ColsumParams p) {
    __shared__ float4 part[kColWarps][32];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool second = (int)blockIdx.x >= p.tiles0;
    const ColsumJob j = second ? p.job[1] : p.job[0];
    const int n0 = (blockIdx.x - (second ? p.tiles0 : 0)) * 128;
    const int e = blockIdx.y, col = n0 + lane * 4;
    int o[2], cnt[2];
    group_rows(p.offsets, p.rows, p.E, p.st, lane, o, cnt);  // by every warp for itself
    const int ex = e / p.split;
    int row0 = __shfl_sync(0xffffffffu, ex < 32 ? o[0] : o[1], ex & 31);
    int n = __shfl_sync(0xffffffffu, ex < 32 ? cnt[0] : cnt[1], ex & 31);
    const int first = row0;
    if (p.split > 1) part_rows(p.split, e % p.split, row0, n);
    if (j.slabs) {  // parts are whole slabs
        row0 = first_slab(first, ex) + ((row0 - first) >> 5);
        n = (n + 31) >> 5;
    }
    float4 s[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (col < j.N)
        for (int r = warp; r < n; r += 8 * kColWarps) {
            float4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                const int64_t at = (int64_t)(row0 + r + kColWarps * i) * j.N + col;
                if (r + kColWarps * i < n) v[i] = j.slabs ? load4<false>(j.dy, at) : load4<IN_BF16>(j.dy, at);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[i & 1].x += v[i].x;
                s[i & 1].y += v[i].y;
                s[i & 1].z += v[i].z;
                s[i & 1].w += v[i].w;
            }
        }
    part[warp][lane] = make_float4(s[0].x + s[1].x, s[0].y + s[1].y, s[0].z + s[1].z, s[0].w + s[1].w);
    __syncthreads();
    if (threadIdx.x < 128) {
        const int c = n0 + threadIdx.x;
        if (c >= j.N) return;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kColWarps; ++w) v += reinterpret_cast<const float*>(part[w])[threadIdx.x];
        const int64_t o = (int64_t)e * j.N + c;
        if (OUT_BF16) {
            __nv_bfloat16* d = static_cast<__nv_bfloat16*>(j.db) + o;
            if (p.accumulate) v += __bfloat162float(*d);
            *d = __float2bfloat16_rn(v);
        } else {
            float* d = static_cast<float*>(j.db) + o;
            if (p.accumulate) v += *d;
            *d = v;
        }
    }
}

// ------------------------------------------------------------ parts joined
// Four neighbouring values per thread; bound by reading the parts, which the kernel before has left in L2.
template <bool OUT_BF16>
__global__ void __launch_bounds__(256) join_kernel(const float* __restrict__ part, void* __restrict__ out, int accumulate,
                                                   int split, int64_t n) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const float* src = part + (int64_t)blockIdx.y * split * n + i;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int z = 0; z < split; ++z) {
        const float4 a = *reinterpret_cast<const float4*>(src + z * n);
        v.x += a.x;
        v.y += a.y;
        v.z += a.z;
        v.w += a.w;
    }
    if (OUT_BF16) {
        uint2* d = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + (int64_t)blockIdx.y * n + i);
        if (accumulate) {
            const uint2 o = *d;
            v.x += bf16_lo(o.x);
            v.y += bf16_hi(o.x);
            v.z += bf16_lo(o.y);
            v.w += bf16_hi(o.y);
        }
        *d = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    } else {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(out) + (int64_t)blockIdx.y * n + i);
        if (accumulate) {
            const float4 o = *d;
            v.x += o.x;
            v.y += o.y;
            v.z += o.z;
            v.w += o.w;
        }
        *d = v;
    }
}

// ------------------------------------------------------- fp32 activation gradient
template <bool SWIGLU>
__global__ void __launch_bounds__(256) act_grad_f32_kernel(int64_t n, float* g, float* u, float* dh) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const float x = g[i], d = dh[i];
    if (SWIGLU) {
        const float s = 1.0f / (1.0f + expf(-x)), xs = x * s, uv = u[i];
        dh[i] = xs * uv;
        g[i] = d * uv * (s + xs * (1.0f - s));
        u[i] = d * xs;
    } else {
        const float cdf = normal_cdf(x);
        dh[i] = x * cdf;
        g[i] = d * (cdf + x * 0.39894228040143268f * expf(-0.5f * x * x));
    }
}

}  // namespace

cudaError_t launch_grouped_fwd_f32(const GroupedArgs& a, cudaStream_t s) {
    F32Params p = params(a);
    p.accumulate = 0;
    p.A = static_cast<const float*>(a.x);
    p.B = static_cast<const float*>(a.w);
    p.bias = static_cast<const float*>(a.bias);
    p.out = static_cast<float*>(a.y);
    return launch_form<FORM_FWD>(a, p, 0, a.N, s);
}

cudaError_t launch_grouped_gx_f32(const GroupedArgs& a, cudaStream_t s) {
    F32Params p = params(a);
    p.A = static_cast<const float*>(a.dy);
    p.B = static_cast<const float*>(a.w);
    p.out = static_cast<float*>(a.dx);
    return launch_form<FORM_GX>(a, p, 0, a.K, s);
}

cudaError_t launch_grouped_gw_f32(const GroupedArgs& a, cudaStream_t s) {
    F32Params p = params(a);
    p.A = static_cast<const float*>(a.x);
    p.B = static_cast<const float*>(a.dy);
    p.out = static_cast<float*>(a.dw);
    p.E = a.E * a.split;
    p.split = a.split;
    return launch_form<FORM_GW>(a, p, a.K, a.N, s);
}

cudaError_t launch_grouped_colsum(const GroupedArgs& a, const GroupedArgs* also, bool dy_bf16, cudaStream_t s) {
    ColsumParams p;
    int tiles = 0;
    for (int i = 0; i < (also != nullptr ? 2 : 1); ++i) {
        const GroupedArgs& g = i == 0 ? a : *also;
        p.job[i].dy = g.sums != nullptr ? g.sums : g.dy;
        p.job[i].slabs = g.sums != nullptr;
        p.job[i].db = g.db;
        p.job[i].N = g.N;
        tiles += (g.N + 127) / 128;
        if (i == 0) p.tiles0 = tiles;
    }
    p.offsets = a.offsets;
    p.rows = (int)a.rows;
    p.E = a.E;
    p.accumulate = a.accumulate ? 1 : 0;
    p.split = a.split;
    p.st = a.st;
    const dim3 grid((unsigned)tiles, (unsigned)(a.E * a.split)), block(kColWarps * 32);
    if (!dy_bf16) return launch_kernel(colsum_kernel<false, false>, grid, block, 0, s, p);
    return a.out_f32 ? launch_kernel(colsum_kernel<true, false>, grid, block, 0, s, p)
                     : launch_kernel(colsum_kernel<true, true>, grid, block, 0, s, p);
}

cudaError_t launch_join(const float* part, void* out, bool out_f32, bool accumulate, int E, int split, int64_t n,
                        cudaStream_t s) {
    const dim3 grid((unsigned)((n / 4 + 255) / 256), (unsigned)E);
    return out_f32 ? launch_kernel(join_kernel<false>, grid, dim3(256), 0, s, part, out, accumulate ? 1 : 0, split, n)
                   : launch_kernel(join_kernel<true>, grid, dim3(256), 0, s, part, out, accumulate ? 1 : 0, split, n);
}

cudaError_t launch_act_grad_f32(int act, int64_t n, float* g, float* u, float* dh, cudaStream_t s) {
    if (n <= 0) return cudaSuccess;
    const dim3 grid((unsigned)((n + 255) / 256));
    return act == 0 ? launch_kernel(act_grad_f32_kernel<true>, grid, dim3(256), 0, s, n, g, u, dh)
                    : launch_kernel(act_grad_f32_kernel<false>, grid, dim3(256), 0, s, n, g, u, dh);
}

}  // namespace moe
