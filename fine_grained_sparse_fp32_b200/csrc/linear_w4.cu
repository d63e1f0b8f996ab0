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
// to 16 tokens. The units of all experts that have rows are numbered through
// and every CTA takes a contiguous share of them; a unit's columns are steps of
// 128, and the CTA's steps are again shared out evenly and contiguously among
// its warps. So a warp streams one long run of weights with no barrier in it:
// each lane copies its own 16 bytes of both rows kW4Stages - 1 steps ahead into
// its own shared memory (cp.async), which keeps about 100 KB of an SM's weight
// traffic in flight without registers. Units that two or more warps share are
// added in warp order at the end, so results do not depend on timing.
#include "w4.cuh"
#include "permute_dev.cuh"
#include "sm100.cuh"

#include <algorithm>

namespace kmoe {
using namespace sm100;

constexpr int kW4Warps = 8;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4CtasPerSm = 2;
constexpr int kW4Tiles = 2;                       // n-tiles of 8 tokens in a unit
constexpr int kW4Tokens = 8 * kW4Tiles;
constexpr int kW4Stages = 8;                      // steps of a warp's copies in flight, plus the one in use
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

// A walk over (unit, 128-column block) steps: the unit's expert and rows, and
// this lane's two weight rows of the fragment.
template <bool kUp, int G, bool kZeros>
struct Walk {
    int tb, tile, grp, block;                     // token block, row tile, expert, block of the row
    const uint8_t *qa, *qb;                       // this lane's code bytes of the row in the upper / lower half
    size_t at_a, at_b;                            // row index of both (for scales and zero points)
    const uint8_t *za, *zb;
    const __nv_bfloat16 *sa, *sb;

    __device__ __forceinline__ void rows(const W4Args &a)
    {
        const W4Product &p = a.p;
        const int g8 = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
        const bool shared = grp >= p.E;
        const W4Ptrs &w = shared ? p.w_shared : p.w;
        const W4Ptrs &w2 = kUp ? (shared ? p.up_shared : p.up) : w;
        // rows past the end repeat the last one; their results are not stored
        const int r_a = min(kUp ? tile * 8 + g8 : tile * 16 + g8, p.rows - 1);
        const int r_b = kUp ? r_a : min(tile * 16 + g8 + 8, p.rows - 1);
        const size_t e0 = shared ? 0 : (size_t)grp * p.rows;
        const int pitch = p.cols / 2, gpr = p.cols / G;
        qa = w.q + (e0 + r_a) * pitch + t * 16;
        qb = w2.q + (e0 + r_b) * pitch + t * 16;
        sa = w.s + (e0 + r_a) * gpr;
        sb = w2.s + (e0 + r_b) * gpr;
        if (kZeros) {
            za = w.z + (e0 + r_a) * gpr;
            zb = w2.z + (e0 + r_b) * gpr;
        }
    }
    __device__ __forceinline__ void start(const W4Args &a, const int *pre, long long unit, int blk)
    {
        tb = (int)(unit / a.tiles);
        tile = (int)(unit - (long long)tb * a.tiles);
        block = blk;
        int lo = 1, hi = a.groups;                // smallest j with pre[j] > tb
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] > tb) hi = mid;
            else lo = mid + 1;
        }
        grp = lo - 1;
        rows(a);
    }
    __device__ __forceinline__ void next_unit(const W4Args &a, const int *pre)
    {
        block = 0;
        if (++tile == a.tiles) {
            tile = 0;
            ++tb;
            while (grp + 1 < a.groups && pre[grp + 1] <= tb) ++grp;
        }
        rows(a);
    }
};

// One step: a 128-column block of 16 rows times NT n-tiles of tokens.
template <int G, bool kZeros, int NT>
__device__ __forceinline__ void w4_step(const uint4 qa, const uint4 qb, const float (&sa)[kW4Block / G],
                                        const float (&sb)[kW4Block / G], const uint32_t (&za)[kW4Block / G],
                                        const uint32_t (&zb)[kW4Block / G], const uint4 (&x)[NT][4],
                                        float (&acc)[kW4Tiles][4])
{
#pragma unroll
    for (int gi = 0; gi < kW4Block / G; ++gi) {
        const __nv_bfloat162 z0 = w4_zero(kZeros ? za[gi] : 8u), z1 = w4_zero(kZeros ? zb[gi] : 8u);
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
                fa[i] = w4_codes(wa, i, z0);
                fb[i] = w4_codes(wb, i, z1);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma_bf16(part[n], fa[0], fb[0], fa[1], fb[1], x[n][j].x, x[n][j].y);
                mma_bf16(part[n], fa[2], fb[2], fa[3], fb[3], x[n][j].z, x[n][j].w);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            acc[n][0] = fmaf(sa[gi], part[n][0], acc[n][0]);
            acc[n][1] = fmaf(sa[gi], part[n][1], acc[n][1]);
            acc[n][2] = fmaf(sb[gi], part[n][2], acc[n][2]);
            acc[n][3] = fmaf(sb[gi], part[n][3], acc[n][3]);
        }
    }
}

// The scales (or zero points) of a 128-column block of one row.
template <int GB>
__device__ __forceinline__ void load_scales(const __nv_bfloat16 *s, float (&v)[GB])
{
    if constexpr (GB == 1) {
        v[0] = __bfloat162float(*s);
    } else if constexpr (GB == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(s);
        v[0] = bf16_lo(w);
        v[1] = bf16_hi(w);
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(s);
        v[0] = bf16_lo(w.x);
        v[1] = bf16_hi(w.x);
        v[2] = bf16_lo(w.y);
        v[3] = bf16_hi(w.y);
    }
}
template <int GB>
__device__ __forceinline__ void load_zeros(const uint8_t *z, uint32_t (&v)[GB])
{
    const uint32_t w = GB == 1   ? *z
                       : GB == 2 ? *reinterpret_cast<const uint16_t *>(z)
                                 : *reinterpret_cast<const uint32_t *>(z);
#pragma unroll
    for (int i = 0; i < GB; ++i) v[i] = (w >> (8 * i)) & 15u;
}

// Stores this lane's sums of unit (row0, n, tile): rows g and g + 8 of the
// fragment, tokens 2t, 2t + 1 of each n-tile.
template <bool kUp, class YT>
__device__ __forceinline__ void store_unit(const W4Product &p, bool shared, int row0, int n, int tile,
                                           const float (&acc)[kW4Tiles][4])
{
    const int lane = threadIdx.x & 31, g8 = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < kW4Tiles; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int i = nt * 8 + 2 * t + j;
            if (i >= n) continue;
            const size_t row = (size_t)row0 + i;
            if (kUp) {
                const int f = tile * 8 + g8;
                if (f < p.rows) store_val(static_cast<YT *>(p.y) + row * p.rows + f, silu_mul(acc[nt][j], acc[nt][2 + j]));
            } else {
                YT *y = shared ? static_cast<YT *>(p.y_shared) + (row - p.P) * p.rows
                               : static_cast<YT *>(p.y) + row * p.rows;
                const int r = tile * 16 + g8;
                if (r < p.rows) store_val(y + r, acc[nt][j]);
                if (r + 8 < p.rows) store_val(y + r + 8, acc[nt][2 + j]);
            }
        }
}

struct W4Smem {
    uint4 ring[kW4Warps][kW4Stages][2][32];       // [lane]: a lane reads back only what it copied
    float4 part[kW4Warps][2][kW4Tiles][32];       // sums of units shared with earlier (0) or later (1) warps
    int pre[kW4MaxGroups + 1];                    // token blocks of the experts before
    int scan_tmp[32];
};

template <bool kUp, int G, bool kZeros, class YT>
__global__ void __launch_bounds__(kW4Threads, kW4CtasPerSm)
w4_kernel(const W4Args a)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    W4Smem &sm = *reinterpret_cast<W4Smem *>(smem_raw);
    constexpr int GB = kW4Block / G;
    pdl_wait();
    pdl_trigger();
    const W4Product &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t = lane & 3;

    // token blocks of every expert, as an exclusive prefix
    const int per = (a.groups + kW4Threads - 1) / kW4Threads;
    int mine = 0;
    for (int i = 0; i < per; ++i) {
        const int g = threadIdx.x * per + i;
        int start, count = 0;
        if (g < a.groups) group_rows(p, g, &start, &count);
        mine += (count + kW4Tokens - 1) / kW4Tokens;
    }
    int run = block_exclusive_scan(mine, sm.scan_tmp);
    for (int i = 0; i < per; ++i) {
        const int g = threadIdx.x * per + i;
        if (g >= a.groups) break;
        int start, count;
        group_rows(p, g, &start, &count);
        sm.pre[g] = run;
        run += (count + kW4Tokens - 1) / kW4Tokens;
        if (g == a.groups - 1) sm.pre[a.groups] = run;
    }
    __syncthreads();

    // this CTA's units, and this warp's steps (local numbers) of them
    const long long total = (long long)sm.pre[a.groups] * a.tiles;
    const long long u0 = total * blockIdx.x / gridDim.x, u1 = total * (blockIdx.x + 1) / gridDim.x;
    const int blocks = p.cols / kW4Block;
    const long long steps = (u1 - u0) * blocks;
    const long long s0 = steps * warp / kW4Warps, s1 = steps * (warp + 1) / kW4Warps;
    bool tail_open = false;                       // the last unit goes on in the next warp
    int e_row0 = 0, e_n = 0, e_tile = 0;
    bool e_shared = false;
    if (s0 < s1) {
        Walk<kUp, G, kZeros> pf, cu;              // copies ahead, and the step in use
        cu.start(a, sm.pre, u0 + s0 / blocks, (int)(s0 % blocks));
        pf = cu;
        long long issued = s0;
        auto copy = [&](int stage) {
            if (issued < s1) {
                cp_async16(smem_u32(&sm.ring[warp][stage][0][lane]), pf.qa + (size_t)pf.block * 64, 16);
                cp_async16(smem_u32(&sm.ring[warp][stage][1][lane]), pf.qb + (size_t)pf.block * 64, 16);
                ++issued;
                if (++pf.block == blocks && issued < s1) pf.next_unit(a, sm.pre);
            }
            cp_async_commit();                    // an empty group past the end keeps the count
        };
        for (int i = 0; i < kW4Stages - 1; ++i) copy(i);
        int stage = 0;
        bool whole = cu.block == 0;               // the unit's first step is this warp's
        float acc[kW4Tiles][4];
        const __nv_bfloat16 *xr[kW4Tiles];
        bool fresh = true;
        for (long long s = s0; s < s1; ++s) {
            if (fresh) {                          // a new unit: its tokens
                fresh = false;
                int start, count;
                e_shared = cu.grp >= p.E;
                group_rows(p, cu.grp, &start, &count);
                const int first = (cu.tb - sm.pre[cu.grp]) * kW4Tokens;
                e_row0 = start + first;
                e_n = min(kW4Tokens, count - first);
                e_tile = cu.tile;
#pragma unroll
                for (int nt = 0; nt < kW4Tiles; ++nt) {
                    const int i = nt * 8 + g8;
                    int xi = -1;
                    if (i < e_n) {
                        xi = e_row0 + i;
                        if (!p.x_by_row) xi = e_shared ? xi - p.P : p.perm ? p.perm[xi] : xi;
                        if ((unsigned)xi >= (unsigned)p.x_rows) xi = -1;
                    }
                    xr[nt] = xi < 0 ? nullptr : p.x + (size_t)xi * p.cols + t * 8;
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
                }
            }
            uint4 x[kW4Tiles][4];
#pragma unroll
            for (int nt = 0; nt < kW4Tiles; ++nt)
                if (nt == 0 || e_n > 8)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[nt][j] = xr[nt] ? *reinterpret_cast<const uint4 *>(xr[nt] + cu.block * kW4Block + j * 32)
                                          : make_uint4(0, 0, 0, 0);
            float sa[GB], sb[GB];
            uint32_t za[GB], zb[GB];
            load_scales<GB>(cu.sa + cu.block * GB, sa);
            load_scales<GB>(cu.sb + cu.block * GB, sb);
            if (kZeros) {
                load_zeros<GB>(cu.za + cu.block * GB, za);
                load_zeros<GB>(cu.zb + cu.block * GB, zb);
            }
            cp_async_wait<kW4Stages - 2>();       // this lane's own copies: no other thread to wait for
            const uint4 qa = sm.ring[warp][stage][0][lane], qb = sm.ring[warp][stage][1][lane];
            // the stage used one step ago takes the copy kW4Stages - 1 steps ahead
            copy(stage == 0 ? kW4Stages - 1 : stage - 1);
            stage = stage + 1 == kW4Stages ? 0 : stage + 1;
            if (e_n > 8) {
                w4_step<G, kZeros, 2>(qa, qb, sa, sb, za, zb, x, acc);
            } else {
                const uint4 x1[1][4] = {{x[0][0], x[0][1], x[0][2], x[0][3]}};
                w4_step<G, kZeros, 1>(qa, qb, sa, sb, za, zb, x1, acc);
            }
            if (++cu.block == blocks) {           // the unit ends here
                if (whole) {
                    store_unit<kUp, YT>(p, e_shared, e_row0, e_n, e_tile, acc);
                } else {
#pragma unroll
                    for (int nt = 0; nt < kW4Tiles; ++nt)
                        sm.part[warp][0][nt][lane] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
                }
                whole = fresh = true;
                if (s + 1 < s1) cu.next_unit(a, sm.pre);
            }
        }
        if (!fresh) {                             // the last unit goes on in later warps
            tail_open = whole;
#pragma unroll
            for (int nt = 0; nt < kW4Tiles; ++nt)
                sm.part[warp][whole ? 1 : 0][nt][lane] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
        }
    }
    __syncthreads();
    if (tail_open) {                              // the warp that began a shared unit adds it up
        float acc[kW4Tiles][4];
        const long long end = ((s1 - 1) / blocks + 1) * blocks;     // the unit's last step + 1
#pragma unroll
        for (int nt = 0; nt < kW4Tiles; ++nt) {
            float4 v = sm.part[warp][1][nt][lane];
            for (int w = warp + 1; w < kW4Warps && steps * w / kW4Warps < end; ++w) {
                if (steps * w / kW4Warps == steps * (w + 1) / kW4Warps) continue;      // a warp without steps
                const float4 o = sm.part[w][0][nt][lane];
                v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
            }
            acc[nt][0] = v.x; acc[nt][1] = v.y; acc[nt][2] = v.z; acc[nt][3] = v.w;
        }
        store_unit<kUp, YT>(p, e_shared, e_row0, e_n, e_tile, acc);
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
    // no more CTAs than units there can be: an expert with rows has at least one token block
    const long long most = ((long long)std::min(a.p.E, a.p.P) + (a.p.P + a.p.n_shared) / kW4Tokens + 1) * a.tiles;
    const int grid = (int)std::min<long long>(sm_count_w4() * kW4CtasPerSm, most);
    cudaFuncSetAttribute(w4_kernel<kUp, G, kZeros, YT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(W4Smem));
    launch_pdl(w4_kernel<kUp, G, kZeros, YT>, grid, kW4Threads, sizeof(W4Smem), st, a);
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
