// The 4-bit weight format (kmoe_w4 in kmoe.h): helpers shared by its kernels.
//
//   W[r][c] = (q[r][c] - z[r][c / group]) * s[r][c / group]
// A block of 128 columns of a row is 64 bytes: the sixteen 8-column words of
// the block as a transposed 4 x 4 square. Lane t (0..3) of a matrix fragment
// so finds in 16 consecutive bytes its 8 columns of each 32-column slice:
// word jj of the 16 bytes holds columns 32 jj + 8 t .. + 7.
#pragma once

#include "common.cuh"

namespace kmoe {

constexpr int kW4Block = 128;                     // columns of one 64-byte block

// Place of 8-column word v (0..15) in its block.
__host__ __device__ constexpr int w4_place(int v) { return 4 * (v & 3) + (v >> 2); }

// One stack of 4-bit matrices, as seen by the kernels.
struct W4Ptrs {
    const uint8_t *q;
    const __nv_bfloat16 *s;
    const uint8_t *z;     // NULL: 8 everywhere
};

__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t *>(&v); }

}  // namespace kmoe

namespace kmoe {

kmoe_status launch_quant_w4(const void *w, int w_dtype, int rows, int cols, int group, uint8_t *codes,
                            __nv_bfloat16 *scales, uint8_t *zeros, cudaStream_t st);
kmoe_status launch_dequant_w4(const W4Ptrs &w, int group, int rows, int cols, void *out, int out_dtype,
                              cudaStream_t st);

// One launch of the 4-bit products: y[p] = W_e x[row(p)], or with `up` set
// H[p] = SiLU(W x) * (up x). Rows p in [offsets[e], offsets[e + 1]) belong to
// expert e < E; with `shared` rows P .. P + n_shared - 1 belong to the shared
// expert. x row of p: perm[p] below P (p itself without perm), p - P
// for the shared expert, or p itself everywhere with x_by_row.
struct W4Product {
    const void *x;
    int x_rows, P, n_shared, rows, cols, E;
    const int32_t *perm, *offsets;       // offsets NULL: E == 1, all P rows
    W4Ptrs w, up, w_shared, up_shared;   // up.q NULL: no SwiGLU
    int group;
    bool x_by_row;                       // x is indexed by p, the shared rows behind the P routed ones
    bool x_f32;                          // x (H) in FP32
    void *y, *y_shared;                  // y [P (+ n_shared for SwiGLU), rows]
    int y_dtype;
    int *status;                         // set to 0 (NULL: none)
};
kmoe_status launch_w4(const W4Product &a, cudaStream_t st);
// The tensor-core kernel; y is BF16 (H: FP32). x16 and x_scale: scratch for x in
// FP16 ([x_rows, cols], for FP32 x its own memory) and a float for each of its
// rows. wait_limit: SM cycles before a pipeline wait gives up and sets *err (the
// device status word; may be NULL) to 1.
kmoe_status launch_w4_tc(const W4Product &a, void *x16, float *x_scale, int *err, long long wait_limit, cudaStream_t st);

// Routing by the rule of kmoe_routing. hist as in launch_topk.
kmoe_status launch_route(const void *logits, int l_dtype, const float *bias, int N, int E, int K,
                         const kmoe_routing &r, int32_t *idx, float *w, cudaStream_t st, int32_t *hist = nullptr);

// Division by a number that the host knows: the high word of n * ceil(2^64 / d),
// exact for n < 2^32 and 1 < d < 2^32.
struct DivideBy {
    unsigned long long m;     // 0 stands for d = 1
    static DivideBy make(uint32_t d) { return {d > 1 ? ~0ull / d + 1 : 0}; }
    __device__ __forceinline__ int operator()(int n) const { return m ? (int)__umul64hi((unsigned long long)(uint32_t)n, m) : n; }
};

// Whether ranges that overlap, as descending offsets give them (which no dispatch
// makes), could add up to more blocks of `tokens` rows than the kernels' sums hold.
inline bool may_overflow(const W4Product &p, int tokens) { return p.offsets && (long long)p.E * (p.P / tokens + 1) >= 1LL << 28; }
// By a whole CTA: whether offsets descend somewhere.
__device__ __forceinline__ bool offsets_descend(const W4Product &p)
{
    bool down = false;
    for (int g = threadIdx.x; g < p.E; g += blockDim.x) down = down || p.offsets[g + 1] < p.offsets[g];
    return __syncthreads_or(down);
}

// Rows [start, start + count) of group g (expert or shared expert), cut to the batch.
__device__ __forceinline__ void group_rows(const W4Product &p, int g, int *start, int *count)
{
    if (g >= p.E) {
        *start = p.P;
        *count = p.n_shared;
        return;
    }
    int a = 0, b = p.P;
    if (p.offsets) {
        a = max(p.offsets[g], 0);
        b = min(p.offsets[g + 1], p.P);
    }
    *start = a;
    *count = max(b - a, 0);
}

// Largest j in [0, n) with v[j] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int last_not_above(const int *v, int n, int x)
{
    int lo = 0;
    for (int w = 1 << (31 - __clz(n)); w > 0; w >>= 1)
        if (lo + w < n && v[lo + w] <= x) lo += w;
    return lo;
}

}  // namespace kmoe
