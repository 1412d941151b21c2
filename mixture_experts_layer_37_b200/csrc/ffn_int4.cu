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
// k+2, k+4, k+6, k+1, k+3, k+5, k+7 (low bits first).  One 16-byte load then
// gives lane (g, t) of a warp its operands of the warp-level MMA (m16n8k16, the
// weights as the 16-row operand, eight tokens as columns) for four steps of 32 k:
//   - (w >> 4j) & 0x000F000F, or'ed with 0x4300 in both halves, is the bf16 pair
//     (128 + c[2j], 128 + c[2j+1]), exactly; minus 136, exactly, the codes;
//   - the same lane's tokens' values for those k are eight neighbours in x: one
//     16-byte load, no shuffle.
// The four lanes of a row cover 32 neighbouring k in each step, so a group of
// 32, 64 or 128 ends with a step and its scale multiplies the fp32 sum of the
// group: the weights are never rounded to bf16 products with their scale.
//
// Two shapes of a warp's work, chosen on the host from the mean rows per expert:
// eight tokens by 16 columns, many warps per SM (decode), or 32 tokens by 32
// columns (a batch), where each widened code is used four times.  Warps of a CTA
// split K and are joined in a fixed order through shared memory.  Codes are
// loaded several blocks ahead into registers, past L1 (each is read once).
// An expert with more rows than a pass holds streams its codes again from L2.
#include <math.h>

#include "grouped.h"

namespace moe {
namespace {

constexpr int kBlockK = 128;  // codes of a storage block
constexpr int kWarps = 8;

enum { I4_PLAIN = 0, I4_SWIGLU = 1, I4_GELU = 2 };

struct Int4Params {
    const __nv_bfloat16* x = nullptr;     // [rows, K]
    const uint8_t* q0 = nullptr;          // codes (SwiGLU: gate)
    const uint8_t* q1 = nullptr;          // SwiGLU: up
    const float* s0 = nullptr;            // [E, groups, N]
    const float* s1 = nullptr;
    const __nv_bfloat16* bias = nullptr;  // [E, N] or null
    __nv_bfloat16* out = nullptr;         // [rows, N]
    const int32_t* offsets = nullptr;     // [E+1]
    int rows = 0, K = 0, N = 0, groups = 0, blocks = 0;
    DevStatus st;
};

__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The codes 2j, 2j+1 of a word as a bf16 pair.
__device__ __forceinline__ uint32_t widen(uint32_t w, int j) {
    const uint32_t v = ((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 m = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));  // 136
    __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), m);
    return *reinterpret_cast<uint32_t*>(&d);
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ float silu_i4(float x) { return x / (1.0f + __expf(-x)); }
__device__ __forceinline__ float gelu_i4(float x) { return 0.5f * x * (1.0f + erff(x * 0.70710678118654752f)); }

// GS: steps of 32 k per group.  NT: tokens / 8.  MT: 16-column tiles of a warp
// (SwiGLU: tile 0 of gate, tile 1 of up, the same columns).  KS: warps that
// split K; the kWarps / KS others stand side by side along N.  DEPTH: blocks of
// codes in flight per warp.
template <int MODE, int GS, int NT, int MT, int KS, int DEPTH>
__global__ void __launch_bounds__(kWarps * 32) int4_kernel(Int4Params p) {
    constexpr bool TWO = MODE == I4_SWIGLU;
    constexpr int kMats = TWO ? 2 : 1;
    constexpr int kColTiles = MT / kMats;                        // distinct 16-column tiles of a warp
    constexpr int kCtaCols = kWarps / KS * kColTiles * 16;
    constexpr int kTok = 8 * NT;
    __shared__ float red[KS][kMats][kTok][kCtaCols + 4];
    griddep_wait();  // the rows and offsets of the launches before
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int e = blockIdx.y;
    int row0, nrows;
    group_rows(p.offsets, p.rows, e, p.st, row0, nrows);
    if (nrows == 0) return;
    const int ks = warp % KS, wn = warp / KS;
    const int n_cta = blockIdx.x * kCtaCols;
    // this warp's blocks of K
    const int per = (p.blocks + KS - 1) / KS;
    const int b0 = min(ks * per, p.blocks), b1 = min(b0 + per, p.blocks);
    // code rows and scales of this lane: columns g and g + 8 of each tile (past N: the last column, not stored)
    const uint8_t* code[MT][2];
    const float* scale[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = min(n_cta + (wn * kColTiles + m / kMats) * 16 + g + 8 * h, p.N - 1);
            const bool up = TWO && (m & 1);
            code[m][h] = (up ? p.q1 : p.q0) + ((int64_t)e * p.N + n) * p.blocks * 64 + t * 16;
            scale[m][h] = (up ? p.s1 : p.s0) + (int64_t)e * p.groups * p.N + n;
        }
    for (int r0 = 0; r0 < nrows; r0 += kTok) {
        uint4 buf[DEPTH][MT][2];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (b0 + d < b1)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) buf[d][m][h] = load_stream(code[m][h] + (int64_t)(b0 + d) * 64);
        // tokens of this lane as columns of the MMA: r0 + 8 j + g
        const __nv_bfloat16* xr[NT];
        bool held[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            held[j] = r0 + 8 * j + g < nrows;
            xr[j] = p.x + (int64_t)(row0 + (held[j] ? r0 + 8 * j + g : 0)) * p.K + 8 * t;
        }
        auto load_x = [&](uint4 (&v)[NT], int k0) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                v[j] = make_uint4(0, 0, 0, 0);
                if (held[j] && k0 + 8 * t < p.K) v[j] = __ldg(reinterpret_cast<const uint4*>(xr[j] + k0));
            }
        };
        float sum[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) sum[m][j][c] = 0.f;
        uint4 xa[2][NT];
        if (b0 < b1) load_x(xa[0], b0 * kBlockK);
        for (int b = b0; b < b1; b += DEPTH) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                if (b + d >= b1) break;
                const int k0 = (b + d) * kBlockK;
                float part[MT][NT][4];
                float sc[MT][2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = k0 + 32 * i;
                    // the next step's tokens (past the end: zeros, not loaded)
                    load_x(xa[(i + 1) & 1], k + 32 < b1 * kBlockK ? k + 32 : p.K);
                    if (i % GS == 0) {
                        const int gi = min(k / (32 * GS), p.groups - 1);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int h = 0; h < 2; ++h) sc[m][h] = __ldg(scale[m][h] + (int64_t)gi * p.N);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int j = 0; j < NT; ++j)
#pragma unroll
                                for (int c = 0; c < 4; ++c) part[m][j][c] = 0.f;
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const uint32_t w0 = word_of(buf[d][m][0], i), w1 = word_of(buf[d][m][1], i);
                        uint32_t a[2][4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            a[0][j] = widen(w0, j);
                            a[1][j] = widen(w1, j);
                        }
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const uint4& xv = xa[i & 1][j];
                            mma_bf16(part[m][j], a[0][0], a[1][0], a[0][1], a[1][1], xv.x, xv.y);
                            mma_bf16(part[m][j], a[0][2], a[1][2], a[0][3], a[1][3], xv.z, xv.w);
                        }
                    }
                    if (i % GS == GS - 1) {
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int j = 0; j < NT; ++j)
#pragma unroll
                                for (int c = 0; c < 4; ++c) sum[m][j][c] = fmaf(sc[m][c >> 1], part[m][j][c], sum[m][j][c]);
                    }
                }
                if (b + d + DEPTH < b1)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) buf[d][m][h] = load_stream(code[m][h] + (int64_t)(b + d + DEPTH) * 64);
            }
        }
        // the K parts of each output, then added in order
        __syncthreads();  // the last pass's values are read
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    red[ks][TWO ? m & 1 : 0][8 * j + 2 * t + (c & 1)][(wn * kColTiles + m / kMats) * 16 + g + 8 * (c >> 1)] =
                        sum[m][j][c];
        __syncthreads();
        const int ntok = min(kTok, nrows - r0);
        // two neighbouring columns per thread (N is even)
        for (int i = threadIdx.x; i < ntok * (kCtaCols / 2); i += kWarps * 32) {
            const int tok = i / (kCtaCols / 2), c = i % (kCtaCols / 2) * 2, n = n_cta + c;
            if (n >= p.N) continue;
            float v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float a = 0.f, u = 0.f;
#pragma unroll
                for (int z = 0; z < KS; ++z) {
                    a += red[z][0][tok][c + h];
                    if (TWO) u += red[z][kMats - 1][tok][c + h];
                }
                if (p.bias != nullptr) a += __bfloat162float(p.bias[(int64_t)e * p.N + n + h]);
                v[h] = MODE == I4_SWIGLU ? silu_i4(a) * u : MODE == I4_GELU ? gelu_i4(a) : a;
            }
            *reinterpret_cast<uint32_t*>(p.out + (int64_t)(row0 + r0 + tok) * p.N + n) = pack_bf16x2(v[0], v[1]);
        }
    }
}

template <int MODE, int GS, int NT, int MT, int KS, int DEPTH>
cudaError_t launch_shape(const Int4Params& p, int E, cudaStream_t s) {
    constexpr int kCtaCols = kWarps / KS * (MT / (MODE == I4_SWIGLU ? 2 : 1)) * 16;
    const dim3 grid((unsigned)((p.N + kCtaCols - 1) / kCtaCols), (unsigned)E);
    return launch_kernel(int4_kernel<MODE, GS, NT, MT, KS, DEPTH>, grid, dim3(kWarps * 32), 0, s, p);
}

template <int MODE, int GS>
cudaError_t launch_group(const Int4Params& p, int E, cudaStream_t s) {
    if ((int64_t)p.rows <= 6 * (int64_t)E) return launch_shape<MODE, GS, 1, MODE == I4_SWIGLU ? 2 : 1, 4, 4>(p, E, s);
    return launch_shape<MODE, GS, 4, 2, 2, 2>(p, E, s);
}

template <int MODE>
cudaError_t launch_int4(const Int4Params& p, int group, int E, cudaStream_t s) {
    if (group == 32) return launch_group<MODE, 1>(p, E, s);
    if (group == 64) return launch_group<MODE, 2>(p, E, s);
    return launch_group<MODE, 4>(p, E, s);
}

Int4Params int4_params(const int32_t* offsets, int64_t rows, int K, int N, int group, DevStatus st) {
    Int4Params p;
    p.offsets = offsets;
    p.rows = (int)rows;
    p.K = K;
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
            for (int k = k0; k < min(k0 + group, K); ++k) amax = fmaxf(amax, fabsf(load(k)));
            s = amax / 7.0f;
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
    Int4Params p = int4_params(a.offsets, a.rows, a.K, a.N, group, a.st);
    p.x = static_cast<const __nv_bfloat16*>(a.x);
    p.q0 = static_cast<const uint8_t*>(a.w);
    p.s0 = scale;
    p.bias = static_cast<const __nv_bfloat16*>(a.bias);
    p.out = static_cast<__nv_bfloat16*>(a.y);
    return launch_int4<I4_PLAIN>(p, group, a.E, s);
}

cudaError_t launch_ffn_int4(const FfnArgs& a, cudaStream_t s) {
    if (a.rows_cap <= 0) return cudaSuccess;
    const bool swiglu = a.act == 0;
    Int4Params p = int4_params(a.offsets, a.rows_cap, a.d, a.ffn, a.int4_group, a.st);
    p.x = static_cast<const __nv_bfloat16*>(a.x_perm);
    p.q0 = static_cast<const uint8_t*>(a.w1);
    p.q1 = static_cast<const uint8_t*>(a.w_up);
    p.s0 = a.w1_scale;
    p.s1 = a.w_up_scale;
    p.bias = swiglu ? nullptr : static_cast<const __nv_bfloat16*>(a.b1);
    p.out = static_cast<__nv_bfloat16*>(a.h);
    cudaError_t err = swiglu ? launch_int4<I4_SWIGLU>(p, a.int4_group, a.E, s)
                             : launch_int4<I4_GELU>(p, a.int4_group, a.E, s);
    if (err != cudaSuccess) return err;
    if (a.between != nullptr && (err = record_mark(a.between, s)) != cudaSuccess) return err;
    Int4Params r = int4_params(a.offsets, a.rows_cap, a.ffn, a.d, a.int4_group, a.st);
    r.x = static_cast<const __nv_bfloat16*>(a.h);
    r.q0 = static_cast<const uint8_t*>(a.w2);
    r.s0 = a.w2_scale;
    r.bias = swiglu ? nullptr : static_cast<const __nv_bfloat16*>(a.b2);
    r.out = static_cast<__nv_bfloat16*>(a.y_perm);
    return launch_int4<I4_PLAIN>(r, a.int4_group, a.E, s);
}

}  // namespace moe
