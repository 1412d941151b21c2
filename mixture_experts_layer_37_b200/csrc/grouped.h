// Launch interfaces of the grouped products and their gradients.  Internal to
// libmoe.
#pragma once

#include "internal.h"

namespace moe {

// Which tiles belong to which expert, built by every CTA in shared memory from
// the offsets on the device (the host never reads the routing).
struct GroupTables {
    int start[kMaxExperts + 1];  // first row tile (or, of the weight gradients, output tile) of the i-th expert taken
    int row0[kMaxExperts];       // its first row
    int nrows[kMaxExperts];      // its rows
    int expert[kMaxExperts];     // which expert it is
};

#ifdef __CUDACC__
// The normal distribution Phi and its density phi, each to its own relative precision.  (1 + erf(x / sqrt 2)) / 2
// cancels for negative x: at -5 it is off by a tenth, behind -5.5 it is noise or zero, and so are x Phi(x) and its
// gradients.
// fp32: by erfc.
__device__ __forceinline__ float normal_cdf(float x) { return 0.5f * erfcf(x * -0.70710678118654752f); }
// Where results are rounded to bf16: from phi, which the gradient needs anyway, and the Mills ratio
// Phi(-z) / phi(z) = t P(t), t = 1 / (1 + 0.35 z), P a polynomial fitted here for the least relative error over
// 0 <= z <= 14.6 (3.2e-8, evaluated in fp32 3.4e-7; phi has the fast exponential's error).  With erfc the GELU
// backward pass of 8192 rows, 8 experts of 2048 x 4096, took 732 us where this takes 668, 777 rows of 192 x 320 59 for 51.
__device__ __forceinline__ void normal_cdf_pdf(float x, float& cdf, float& pdf) {
    pdf = 0.39894228040143268f * __expf(-0.5f * x * x);
    const float t = __fdividef(1.0f, fmaf(0.35f, fabsf(x), 1.0f));
    float q = -0.0730919167f;
    q = fmaf(q, t, 0.3610515f);
    q = fmaf(q, t, -0.641334414f);
    q = fmaf(q, t, 0.399403274f);
    q = fmaf(q, t, -0.0582185797f);
    q = fmaf(q, t, 0.264595568f);
    q = fmaf(q, t, 0.300343603f);
    q = fmaf(q, t, 0.350586385f);
    q = fmaf(q, t, 0.349978685f);
    const float tail = pdf * (q * t);
    cdf = x < 0.0f ? tail : 1.0f - tail;
}

// The rows of experts lane and lane + 32, by a whole warp.  Offsets that decrease
// or leave the buffers are refused: such an expert has no rows, and the status
// word says so.  So has one that begins below the end of an expert before it
// (possible only behind offsets that decrease): its rows are the other's, and two
// tiles would write them.
__device__ __forceinline__ void group_rows(const int32_t* offsets, int rows, int E, const DevStatus& st, int lane,
                                           int (&row0)[2], int (&n)[2]) {
    int carry = 0;  // the largest end so far
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = lane + 32 * i;
        int a = 0, b = 0;
        if (e < E) {
            a = offsets[e];
            b = offsets[e + 1];
        }
        const bool in = a >= 0 && b >= a && b <= rows;
        int end = in ? b : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, end, d);
            if (lane >= d) end = max(end, u);
        }
        int before = __shfl_up_sync(0xffffffffu, end, 1);
        before = lane > 0 ? max(before, carry) : carry;
        const bool ok = in && (a >= before || a == b);
        if (e < E && !ok) report_range(st, SITE_GROUPED_OFFSETS);
        row0[i] = ok ? a : 0;
        n[i] = ok ? b - a : 0;
        carry = max(carry, __shfl_sync(0xffffffffu, end, 31));
    }
}

// The part z of S of expert e's rows (whole blocks of 64, the last parts may be empty).
__device__ __forceinline__ void part_rows(int S, int z, int& row0, int& n) {
    const int per = ((n + S - 1) / S + 63) / 64 * 64, from = min(z * per, n);
    row0 += from;
    n = min(per, n - from);
}

// Column sums of 32 rows each ("slabs", counted from an expert's first row): where expert e's begin. Experts' rows do
// not overlap and come in order, so their slabs do not either; rows / 32 + E of them at most.
__host__ __device__ __forceinline__ int64_t max_slabs(int64_t rows, int E) { return rows / 32 + E; }
__device__ __forceinline__ int first_slab(int row0, int e) { return (row0 >> 5) + e; }

// One warp; each lane holds experts `lane` and `lane + 32`.  BY_ROWS: experts
// in order of falling row count (ties: lower id) with m_tiles tiles each; else
// in their own order with one tile per bm rows.  split > 1: E counts the parts
// of the experts' rows, part e % split of expert e / split.
template <bool BY_ROWS>
__device__ __forceinline__ void build_group_tables(const int32_t* offsets, int rows, int E, int bm, int m_tiles,
                                                   const DevStatus& st, GroupTables* t, int lane, int split = 1) {
    int o[2], n[2];
    group_rows(offsets, rows, E / split, st, lane, o, n);
    if (split > 1) {  // every expert's rows, then each part's own
        const int oe[2] = {o[0], o[1]}, ne[2] = {n[0], n[1]};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = (lane + 32 * i) / split;  // 32 experts at most are split
            o[i] = __shfl_sync(0xffffffffu, oe[0], e & 31);
            n[i] = __shfl_sync(0xffffffffu, ne[0], e & 31);
            part_rows(split, (lane + 32 * i) % split, o[i], n[i]);
        }
    }
    int rank[2] = {lane, lane + 32};
    if (BY_ROWS) {
        rank[0] = rank[1] = 0;
        for (int j = 0; j < E; ++j) {
            const int nj = __shfl_sync(0xffffffffu, j < 32 ? n[0] : n[1], j & 31);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (nj > n[i] || (nj == n[i] && j < lane + 32 * i)) ++rank[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (lane + 32 * i < E) {
            t->row0[rank[i]] = o[i];
            t->nrows[rank[i]] = n[i];
            t->expert[rank[i]] = lane + 32 * i;
        }
    if (BY_ROWS) {
        for (int e = lane; e <= E; e += 32) t->start[e] = e * m_tiles;
    } else {
        int carry = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int v = (n[i] + bm - 1) / bm;
            int s = v;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, s, d);
                if (lane >= d) s += u;
            }
            if (lane + 32 * i < E) t->start[lane + 32 * i] = carry + s - v;
            carry += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0) t->start[E] = carry;
    }
    __syncwarp();
}
#endif

enum { GRAD_NONE = 0, GRAD_SWIGLU = 1, GRAD_GELU = 2 };

// Weights w [E, K, N]; x [rows, K]; dy [rows, N] (see grouped_gemm.cu).
struct GroupedArgs {
    const int32_t* offsets = nullptr;  // [E+1]
    int64_t rows = 0;                  // rows of the row buffers
    int E = 0, K = 0, N = 0;
    const void* x = nullptr;
    const void* w = nullptr;
    const void* bias = nullptr;        // [E, N] or null
    void* y = nullptr;                 // [rows, N]
    const void* dy = nullptr;
    void* dx = nullptr;                // [rows, K]
    void* dw = nullptr;                // [E, K, N]
    void* db = nullptr;                // [E, N] or null
    bool out_f32 = false;              // GX, GW: fp32 output
    bool accumulate = false;           // GW: dw += , db +=
    // GW, bias gradients: each expert's rows in `split` parts whose sums are written one after the other
    // ([E, split, ..], fp32, not accumulated) and joined by launch_join
    int split = 1;
    // GX with a second pair: dx = dy w^T + dy2 w2^T
    const void* dy2 = nullptr;
    const void* w2 = nullptr;          // also: the up matrix of GRAD_SWIGLU
    // FWD with the activation's backward pass in its epilogue (y is not written)
    int grad_act = GRAD_NONE;
    const void* dh = nullptr;          // [rows, N] fp32
    void* h = nullptr;                 // [rows, N] activation
    void* d0 = nullptr;                // [rows, N] gradient of gate (SwiGLU) or of the pre-activation (GELU)
    void* d1 = nullptr;                // [rows, N] gradient of up (SwiGLU)
    // GELU: d0's column sums by slabs of 32 rows, [max_slabs, N] fp32, written by FWD with the activation's backward
    // pass and read instead of dy by the bias gradient; or null
    float* sums = nullptr;
    DevStatus st;
};

cudaError_t launch_grouped_fwd_bf16(const GroupedArgs& a, cudaStream_t s);
cudaError_t launch_grouped_gx_bf16(const GroupedArgs& a, cudaStream_t s);
cudaError_t launch_grouped_gw_bf16(const GroupedArgs& a, cudaStream_t s);
cudaError_t launch_grouped_fwd_f32(const GroupedArgs& a, cudaStream_t s);
cudaError_t launch_grouped_gx_f32(const GroupedArgs& a, cudaStream_t s);
cudaError_t launch_grouped_gw_f32(const GroupedArgs& a, cudaStream_t s);
// y = x W (+ bias) with W as 4-bit codes (a.w, see ffn_int4.cu) and scales [E, ceil(K/group), N]; bf16.
cudaError_t launch_grouped_int4(const GroupedArgs& a, const float* scale, int group, cudaStream_t s);
// Codes and scales of w [E, K, N], or, with `given` [E, K, N] (values -8..7), its storage form alone.
cudaError_t launch_quantize_int4(const void* w, bool bf16, const int8_t* given, int E, int K, int N, int group,
                                 uint8_t* codes, float* scale, cudaStream_t s);
// out[e, i] (+)= sum over z of part[e, z, i] in ascending z, i < n; out in fp32 or bf16.
cudaError_t launch_join(const float* part, void* out, bool out_f32, bool accumulate, int E, int split, int64_t n,
                        cudaStream_t s);
// db[e,n] (+)= sum over the rows of e of dy[r,n]; db in fp32 (a.out_f32) or bf16.
// `also` (or null): a second one in the same launch, for the same rows and with the same options.
cudaError_t launch_grouped_colsum(const GroupedArgs& a, const GroupedArgs* also, bool dy_bf16, cudaStream_t s);
// Elementwise over all rows in fp32: from g, u and dh to h (over dh), dg (over g), du (over u).
cudaError_t launch_act_grad_f32(int act, int64_t n, float* g, float* u, float* dh, cudaStream_t s);

}  // namespace moe
