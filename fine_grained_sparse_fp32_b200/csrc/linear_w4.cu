// Products with 4-bit weights and group scales: dense, grouped by expert, and
// the gate/up half of the experts' FFN.
//
//   y[p][r] = sum_G s[r][G] * ( sum_{c in G} (q[r][c] - z[r][G]) x[p][c] )
// over the groups G of 32, 64 or 128 columns. The inner sums run on the tensor
// cores (mma.sync m16n8k16, weights as M, tokens as N): codes minus zero
// points are whole numbers below 16 in magnitude, exact in BF16, so the
// weights are never rounded; the group scale multiplies the FP32 sum.
// A fragment's 16 columns may be any 16 of a group, as long as both operands
// agree. Lane (g, t) holds rows g and g + 8 and, of every 32 columns, columns
// 8t .. 8t + 7: one 32-bit word of codes per row and, for token g, 16 bytes of
// x. Both come straight from global memory: no shared memory holds operands.
//
// With `up` weights, rows 0-7 of the fragment are eight gate features and rows
// 8-15 the same eight up features, so a thread has both sums of its feature
// and token and writes SiLU(gate) * up.
//
// A unit is one fragment row tile (16 rows; 8 features) of one expert for up
// to 32 tokens. The units of all experts that have rows are numbered through,
// and every team of kWarps warps takes a contiguous share of them; the warps
// of a team split the columns of a unit and add their sums in a fixed order.
#include "w4.cuh"
#include "permute_dev.cuh"

#include <algorithm>

namespace kmoe {

constexpr int kW4Warps = 4;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4Tokens = 32;                     // tokens of a unit: up to four n-tiles of 8
constexpr int kW4MaxGroups = 1025;

struct W4Args {
    W4Product p;
    int tiles;          // row tiles of one expert
    int groups;         // experts, the shared one included
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// One unit: NT n-tiles of tokens. pa / pb: this lane's rows of the two
// fragment halves (code rows, scale rows, zero rows).
struct RowPtr {
    const uint8_t *q;
    const __nv_bfloat16 *s;
    const uint8_t *z;
};

template <int G, bool kZeros, int NT>
__device__ __forceinline__ void unit_sums(const RowPtr &ra, const RowPtr &rb, const __nv_bfloat16 *const (&xr)[NT],
                                          int blocks, int warp, float (&acc)[NT][4])
{
    constexpr int GB = kW4Block / G;              // groups of a 128-column block
    const int t = threadIdx.x & 3;
    const __nv_bfloat162 z8 = w4_zero(8);
    for (int b = warp; b < blocks; b += kW4Warps) {
        const uint4 qa = *reinterpret_cast<const uint4 *>(ra.q + (size_t)b * 64 + t * 16);
        const uint4 qb = *reinterpret_cast<const uint4 *>(rb.q + (size_t)b * 64 + t * 16);
#pragma unroll
        for (int gi = 0; gi < GB; ++gi) {
            const float sa = __bfloat162float(ra.s[b * GB + gi]), sb = __bfloat162float(rb.s[b * GB + gi]);
            __nv_bfloat162 za = z8, zb = z8;
            if (kZeros) {
                za = w4_zero(ra.z[b * GB + gi]);
                zb = w4_zero(rb.z[b * GB + gi]);
            }
            float part[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[n][i] = 0.f;
#pragma unroll
            for (int j = gi * (G / 32); j < (gi + 1) * (G / 32); ++j) {
                const uint32_t wa = word_of(qa, j), wb = word_of(qb, j);
                uint32_t fa[4], fb[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    fa[i] = w4_codes(wa, i, za);
                    fb[i] = w4_codes(wb, i, zb);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (xr[n]) x = *reinterpret_cast<const uint4 *>(xr[n] + (size_t)b * kW4Block + j * 32 + t * 8);
                    mma_bf16(part[n], fa[0], fb[0], fa[1], fb[1], x.x, x.y);
                    mma_bf16(part[n], fa[2], fb[2], fa[3], fb[3], x.z, x.w);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] = fmaf(sa, part[n][0], acc[n][0]);
                acc[n][1] = fmaf(sa, part[n][1], acc[n][1]);
                acc[n][2] = fmaf(sb, part[n][2], acc[n][2]);
                acc[n][3] = fmaf(sb, part[n][3], acc[n][3]);
            }
        }
    }
}

template <bool kUp, int G, bool kZeros, class YT>
__global__ void __launch_bounds__(kW4Threads)
w4_kernel(const W4Args a)
{
    __shared__ int pre[kW4MaxGroups + 1];         // token blocks of the groups before
    __shared__ int scan_tmp[32];
    __shared__ __align__(16) float red[kW4Warps][kW4Tokens / 8][32][4];
    pdl_wait();
    pdl_trigger();
    const W4Product &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t = lane & 3;

    // token blocks of every group, as an exclusive prefix
    const int per = (a.groups + kW4Threads - 1) / kW4Threads;
    int mine = 0;
    for (int i = 0; i < per; ++i) {
        const int g = threadIdx.x * per + i;
        int start, count = 0;
        if (g < a.groups) group_rows(p, g, &start, &count);
        mine += (count + kW4Tokens - 1) / kW4Tokens;
    }
    int run = block_exclusive_scan(mine, scan_tmp);
    for (int i = 0; i < per; ++i) {
        const int g = threadIdx.x * per + i;
        if (g >= a.groups) break;
        int start, count;
        group_rows(p, g, &start, &count);
        pre[g] = run;
        run += (count + kW4Tokens - 1) / kW4Tokens;
        if (g == a.groups - 1) pre[a.groups] = run;
    }
    __syncthreads();

    const long long total = (long long)pre[a.groups] * a.tiles;
    const long long u0 = total * blockIdx.x / gridDim.x, u1 = total * (blockIdx.x + 1) / gridDim.x;
    const int blocks = p.cols / kW4Block, gpr = p.cols / G;
    for (long long u = u0; u < u1; ++u) {
        const int tb = (int)(u / a.tiles), tile = (int)(u - (long long)tb * a.tiles);
        int lo = 1, hi = a.groups;                // smallest j with pre[j] > tb
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] > tb) hi = mid;
            else lo = mid + 1;
        }
        const int grp = lo - 1;
        const bool shared = grp >= p.E;
        int start, count;
        group_rows(p, grp, &start, &count);
        const int first = (tb - pre[grp]) * kW4Tokens;
        const int row0 = start + first, n = min(kW4Tokens, count - first);

        // this lane's two weight rows; rows past the end repeat the last one
        RowPtr ra, rb;
        {
            const W4Ptrs &w = shared ? p.w_shared : p.w;
            const W4Ptrs &w2 = kUp ? (shared ? p.up_shared : p.up) : w;
            const int r_a = min(kUp ? tile * 8 + g8 : tile * 16 + g8, p.rows - 1);
            const int r_b = kUp ? r_a : min(tile * 16 + g8 + 8, p.rows - 1);
            const size_t at = shared ? 0 : (size_t)grp * p.rows;
            ra = {w.q + (at + r_a) * (p.cols / 2), w.s + (at + r_a) * gpr, kZeros ? w.z + (at + r_a) * gpr : nullptr};
            rb = {w2.q + (at + r_b) * (p.cols / 2), w2.s + (at + r_b) * gpr,
                  kZeros ? w2.z + (at + r_b) * gpr : nullptr};
        }
        const __nv_bfloat16 *xr[kW4Tokens / 8];
#pragma unroll
        for (int nt = 0; nt < kW4Tokens / 8; ++nt) {
            const int i = nt * 8 + g8;
            int xi = -1;
            if (i < n) {
                xi = row0 + i;
                if (!p.x_by_row) xi = shared ? xi - p.P : p.perm ? p.perm[xi] : xi;
                if ((unsigned)xi >= (unsigned)p.x_rows) xi = -1;
            }
            xr[nt] = xi < 0 ? nullptr : p.x + (size_t)xi * p.cols;
        }
        float acc[kW4Tokens / 8][4];
#pragma unroll
        for (int nt = 0; nt < kW4Tokens / 8; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
        const int nts = (n + 7) / 8;
        if (nts == 1) {
            const __nv_bfloat16 *const x1[1] = {xr[0]};
            float a1[1][4] = {};
            unit_sums<G, kZeros, 1>(ra, rb, x1, blocks, warp, a1);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[0][i] = a1[0][i];
        } else {
            const __nv_bfloat16 *const x4[4] = {xr[0], xr[1], xr[2], xr[3]};
            unit_sums<G, kZeros, 4>(ra, rb, x4, blocks, warp, acc);
        }
        // the warps' sums, added in order by warp nt for n-tile nt
#pragma unroll
        for (int nt = 0; nt < kW4Tokens / 8; ++nt)
            if (nt < nts) *reinterpret_cast<float4 *>(red[warp][nt][lane]) = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
        __syncthreads();
        if (warp < nts) {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kW4Warps; ++w) {
                const float4 r = *reinterpret_cast<const float4 *>(red[w][warp][lane]);
                v[0] += r.x; v[1] += r.y; v[2] += r.z; v[3] += r.w;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {         // tokens 2t, 2t + 1 of the n-tile
                const int i = warp * 8 + 2 * t + j;
                if (i >= n) continue;
                const size_t row = (size_t)row0 + i;
                if (kUp) {
                    const int f = tile * 8 + g8;
                    if (f < p.rows) store_val(static_cast<YT *>(p.y) + row * p.rows + f, silu_mul(v[j], v[2 + j]));
                } else {
                    YT *y = shared ? static_cast<YT *>(p.y_shared) + (row - p.P) * p.rows
                                   : static_cast<YT *>(p.y) + row * p.rows;
                    const int r = tile * 16 + g8;
                    if (r < p.rows) store_val(y + r, v[j]);
                    if (r + 8 < p.rows) store_val(y + r + 8, v[2 + j]);
                }
            }
        }
        __syncthreads();
    }
}

static int sm_count_w4()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        n = 148;
    return n;
}

template <bool kUp, int G, bool kZeros, class YT>
static kmoe_status run_w4(const W4Args &a, cudaStream_t st)
{
    // no more teams than units there can be: every routed row adds at most one token block
    const long long most = ((long long)std::min(a.p.E, a.p.P) + (a.p.P + a.p.n_shared) / kW4Tokens + 1) * a.tiles;
    const int grid = (int)std::min<long long>(sm_count_w4() * 4, most);
    launch_pdl(w4_kernel<kUp, G, kZeros, YT>, grid, kW4Threads, 0, st, a);
    return check_launch("w4");
}

template <bool kUp, class YT>
static kmoe_status pick_w4(const W4Args &a, cudaStream_t st)
{
    const bool z = a.p.w.z != nullptr;
    switch (a.p.group) {
    case 32: return z ? run_w4<kUp, 32, true, YT>(a, st) : run_w4<kUp, 32, false, YT>(a, st);
    case 64: return z ? run_w4<kUp, 64, true, YT>(a, st) : run_w4<kUp, 64, false, YT>(a, st);
    default: return z ? run_w4<kUp, 128, true, YT>(a, st) : run_w4<kUp, 128, false, YT>(a, st);
    }
}

kmoe_status launch_w4(const W4Product &p, cudaStream_t st)
{
    W4Args a{p, 0, p.E + (p.n_shared > 0 ? 1 : 0)};
    if (a.groups > kW4MaxGroups) return fail(KMOE_ERR_UNSUPPORTED, "4-bit products: too many experts");
    const bool up = p.up.q != nullptr;
    a.tiles = up ? (p.rows + 7) / 8 : (p.rows + 15) / 16;
    if (up) return pick_w4<true, __nv_bfloat16>(a, st);
    return p.y_dtype == KMOE_F32 ? pick_w4<false, float>(a, st) : pick_w4<false, __nv_bfloat16>(a, st);
}

}  // namespace kmoe
