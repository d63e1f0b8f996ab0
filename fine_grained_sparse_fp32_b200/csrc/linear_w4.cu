// Products with 4-bit weights and group scales: dense, grouped by expert, and
// the two halves of the experts' FFN.
//
//   y[p][r] = sum_G s[r][G] * ( sum_{c in G} (q[r][c] - z[r][G]) x[p][c] )
// over the groups G of 32, 64 or 128 columns. The bound is the weights' way
// through HBM, about 46 weights per clock and SM, so what counts is how few
// instructions a weight costs. The inner sums are whole numbers on the integer
// tensor cores (mma.sync m16n8k32, u8 x s8 -> s32; weights as M, x as N): four
// codes become four operand bytes with one AND (and half a shift), where BF16
// operands took 2.75 instructions per two codes and left the kernel bound by
// its integer pipe (28% of HBM's rate). For that x is cut into digits: for
// each token and 128 columns, with 2^E the power of two below the largest |x|,
//   x = 2^(E - 21) * (65536 t0 + 256 t1 + t2) + r,   |r| <= 2^(E - 22),
// with t in -128..127. r is 0 for every BF16 x within 2^14 of the block's
// largest value, so sums are at least as exact as with FP32 products. The
// digits of a token are three columns of the fragment, and the integer sums of
// a group are exact; zero points come off as -z * (sum of the digits), the
// start value of the sum. Group scale and 2^(E - 21) multiply the sums in FP32.
//
// With `up` weights, rows 0-7 of a fragment are eight gate features and rows
// 8-15 the same eight up features, and SiLU(gate) * up is written.
//
// A unit is one fragment row tile (16 rows; 8 features) of one expert for up
// to 8 tokens. The units of all experts that have rows are numbered through
// and every CTA (one per SM) takes a contiguous share of them, in phases: as
// many units as the digits of their tokens fit into shared memory (nearly
// always all). A unit's columns are steps of 128, and a phase's steps are
// shared out evenly and contiguously among the warps. So a warp streams one
// long run of weights with no barrier in it: each lane copies its 16 bytes of
// both its rows (and lanes 0 to 3 of a row its scales and zero points)
// kW4Stages - 1 steps ahead into the warp's shared memory (cp.async), which
// keeps about 64 KB of an SM's weight traffic in flight without registers.
// Units that two or more warps share are added in warp order at the end, so
// results do not depend on timing. A unit of more tokens costs more
// instructions for the same weights; the CTAs' shares are cut by that cost.
#include "w4.cuh"
#include "sm100.cuh"

#include <algorithm>

namespace kmoe {
using namespace sm100;

constexpr int kW4Warps = 16;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4Tiles = 4;                       // fragments of two tokens (three digits each) in a unit
constexpr int kW4Tokens = 2 * kW4Tiles;
constexpr int kW4Stages = 5;                      // steps of a warp's copies in flight, plus the one in use
constexpr int kW4MaxGroups = 1025;
constexpr int kW4Entries = 64;                    // token blocks of a phase
constexpr int kW4SmemMax = 226 * 1024;

// Instructions of a step by its token pairs, in units of about 25: what the
// CTAs' shares are cut by.
__host__ __device__ constexpr int w4_cost(int tokens) { return 3 + (tokens + 1) / 2; }

struct W4Args {
    W4Product p;
    int tiles;          // row tiles of one expert
    int groups;         // experts, the shared one included
    int x_tiles;        // token pairs whose digits fit into shared memory
    int tokens;         // tokens of a unit: 2 * kW4Tiles, fewer where x_tiles is less
    int q_jump, s_jump; // from the end of a row to the row of the next tile: code bytes, groups
};

// D += A B with unsigned codes and signed digits, 16 rows x 8 columns, 32 deep.
__device__ __forceinline__ void mma_u8s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One token block of a phase.
struct W4Entry {
    int grp, row0, n, tile0;                      // expert, first row, rows, first staged token pair
};

// One step's copies of a warp: code bytes by lane, then the words that hold the
// scales and zero points of the row pair g: {scale g, scale g + 8, zero g,
// zero g + 8}, of 4 bytes each (8 with groups of 32).
template <int G>
struct W4Stage {
    uint4 q[2][32];
    uint4 aux[8][G == 32 ? 2 : 1];
};

struct W4Smem {
    float head[kW4Warps][kW4Tiles][32];           // sums of a unit that an earlier warp began
    long long cost[kW4MaxGroups + 1];             // cost of the experts before
    long long scan_tmp[32];
    W4Entry ent[kW4Entries];
    int row[kW4Entries * kW4Tokens];              // x row of every staged token (two per pair), -1: none
    int pre[kW4MaxGroups + 1];                    // token blocks of the experts before
    int start[kW4MaxGroups + 1], count[kW4MaxGroups + 1];     // rows of every expert
};
// behind it: W4Stage [kW4Warps][kW4Stages], digits uint4 [pair][block][2][32], digit sums int [pair][block][128 / G][8], scales float [pair][block][2]
__host__ __device__ constexpr size_t w4_x_bytes(int cols, int G) { return (size_t)(cols / kW4Block) * (1024 + 32 * (kW4Block / G) + 8); }
constexpr size_t kW4Tables = (sizeof(W4Smem) + 127) / 128 * 128;
template <int G>
constexpr size_t kW4FixedSmem = kW4Tables + sizeof(W4Stage<G>) * kW4Warps * kW4Stages;

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

// Block-wide exclusive scan over threadIdx.x, of counts and costs at once.
__device__ __forceinline__ void scan2(int *count, long long *cost, W4Smem &sm)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long mine = *cost << 30 | *count;  // counts stay below 2^30, costs below 2^33
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
    }
    if (lane == 31) sm.scan_tmp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        long long v = lane < kW4Warps ? sm.scan_tmp[lane] : 0;
#pragma unroll
        for (int o = 1; o < kW4Warps; o <<= 1) {
            const long long n = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += n;
        }
        if (lane < kW4Warps) sm.scan_tmp[lane] = v;
    }
    __syncthreads();
    const long long before = incl - mine + (warp ? sm.scan_tmp[warp - 1] : 0);
    *count = (int)(before & 0x3fffffff);
    *cost = before >> 30;
}

// Largest j in [0, n) with v[j] <= x (v ascending, v[0] <= x, n <= 1056), by a
// whole warp in two looks.
template <class T>
__device__ __forceinline__ int last_not_above(const T *v, int n, T x)
{
    const int lane = threadIdx.x & 31, chunk = (n + 31) >> 5;
    const unsigned c = __ballot_sync(0xffffffffu, lane * chunk < n && v[lane * chunk] <= x);
    const int base = (31 - __clz(c)) * chunk;
    unsigned f = __ballot_sync(0xffffffffu, lane < chunk && base + lane < n && v[base + lane] <= x);
    const int at = base + 31 - __clz(f);
    return chunk > 32 && base + 32 < n && v[base + 32] <= x ? base + 32 : at;
}

// The unit at which a share that begins at cost c starts (by a whole warp).
__device__ __forceinline__ long long unit_at(const W4Args &a, const W4Smem &sm, long long c)
{
    if (c >= sm.cost[a.groups]) return (long long)sm.pre[a.groups] * a.tiles;
    const int g = last_not_above(sm.cost, a.groups, c), count = sm.count[g];
    long long rem = c - sm.cost[g];
    const long long full = (long long)a.tiles * w4_cost(a.tokens);
    const int tb = (int)min(rem / full, (long long)((count - 1) / a.tokens));
    rem -= tb * full;
    return ((long long)sm.pre[g] + tb) * a.tiles + min(rem / w4_cost(min(a.tokens, count - tb * a.tokens)), (long long)a.tiles);
}

// This lane's weight rows of a unit: rows g and g + 8 of its fragment.
template <bool kUp, int G>
struct UnitRows {
    const W4Ptrs *wa, *wb;
    size_t ra, rb;

    __device__ __forceinline__ UnitRows(const W4Args &a, int grp, int tile)
    {
        const W4Product &p = a.p;
        const int g8 = (threadIdx.x & 31) >> 2;
        const bool shared = grp >= p.E;
        wa = shared ? &p.w_shared : &p.w;
        wb = kUp ? (shared ? &p.up_shared : &p.up) : wa;
        // rows past the end repeat the last one; their results are not stored
        const int r_a = min(kUp ? tile * 8 + g8 : tile * 16 + g8, p.rows - 1);
        const int r_b = kUp ? r_a : min(tile * 16 + g8 + 8, p.rows - 1);
        const size_t e0 = shared ? 0 : (size_t)grp * p.rows;
        ra = e0 + r_a;
        rb = e0 + r_b;
    }
};

constexpr int aux_word(int G) { return G == 32 ? 8 : 4; }

// The copies ahead: a walk over (unit, 128-column block) steps.
template <bool kUp, int G, bool kZeros>
struct Copier {
    int ent, tile, left;                          // left: blocks of the unit still to copy
    int a_jump;                                   // aux: from the end of a row to the next tile's row
    const uint8_t *qa, *qb, *aux;                 // aux: lanes 0, 1 of a row scales of rows g, g + 8; 2, 3 zero points

    __device__ __forceinline__ void unit(const W4Args &a, const W4Smem &sm, int block)
    {
        const UnitRows<kUp, G> r(a, sm.ent[ent].grp, tile);
        const int t = threadIdx.x & 3, pitch = a.p.cols / 2, gpr = a.p.cols / G;
        qa = r.wa->q + r.ra * pitch + t * 16 + (size_t)block * 64;
        qb = r.wb->q + r.rb * pitch + t * 16 + (size_t)block * 64;
        const size_t at = (t & 1 ? r.rb : r.ra) * gpr + (size_t)block * (kW4Block / G);
        const W4Ptrs *w = t & 1 ? r.wb : r.wa;
        aux = t < 2 ? reinterpret_cast<const uint8_t *>(w->s + at) : kZeros ? w->z + at : nullptr;
        left = a.p.cols / kW4Block - block;
        a_jump = a.s_jump * (t < 2 ? 2 : 1);
    }
    // One step into `st`, which ends the unit's walk or goes on in it.
    __device__ __forceinline__ void step(const W4Args &a, const W4Smem &sm, W4Stage<G> &st, bool more)
    {
        constexpr int GB = kW4Block / G, W = aux_word(G);
        const int lane = threadIdx.x & 31, t = lane & 3;
        cp_async16(smem_u32(&st.q[0][lane]), qa, 16);
        cp_async16(smem_u32(&st.q[1][lane]), qb, 16);
        if (kZeros || t < 2) {                    // the aligned word that holds them, no byte past the last one
            const uint32_t in = (uint32_t)reinterpret_cast<uintptr_t>(aux) & (W - 1);
            const uint32_t n = in + (t < 2 ? 2 * GB : GB);
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(
                             smem_u32(reinterpret_cast<uint8_t *>(st.aux[lane >> 2]) + t * W)),
                         "l"(aux - in), "n"(W), "r"(n)
                         : "memory");
        }
        qa += 64;
        qb += 64;
        aux += t < 2 ? 2 * GB : GB;
        if (--left == 0 && more) {
            if (++tile < a.tiles - 1) {           // whole tiles of one matrix lie at equal distances
                qa += a.q_jump;
                qb += a.q_jump;
                aux += a_jump;
                left = a.p.cols / kW4Block;
            } else {
                if (tile == a.tiles) {
                    tile = 0;
                    ++ent;
                }
                unit(a, sm, 0);
            }
        }
    }
};

// Scales (FP32) and zero points of a step from its copied words. la, lb, lz,
// lzb: low address bits of the values, which say where in the word they are.
template <int G, bool kZeros>
__device__ __forceinline__ void read_aux(const uint4 (&aux)[G == 32 ? 2 : 1], uint32_t la, uint32_t lb, uint32_t lza, uint32_t lzb,
                                         float (&sa)[kW4Block / G], float (&sb)[kW4Block / G], int (&za)[kW4Block / G],
                                         int (&zb)[kW4Block / G])
{
    if constexpr (G == 32) {
        const uint4 s = aux[0];
        sa[0] = bf16_lo(s.x); sa[1] = bf16_hi(s.x); sa[2] = bf16_lo(s.y); sa[3] = bf16_hi(s.y);
        sb[0] = bf16_lo(s.z); sb[1] = bf16_hi(s.z); sb[2] = bf16_lo(s.w); sb[3] = bf16_hi(s.w);
        if (kZeros) {
            const uint4 z = aux[1];
            const uint32_t a = lza & 4 ? z.y : z.x, b = lzb & 4 ? z.w : z.z;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                za[i] = (a >> (8 * i)) & 15;
                zb[i] = (b >> (8 * i)) & 15;
            }
        }
    } else {
        const uint4 w = aux[0];
        if constexpr (G == 64) {
            sa[0] = bf16_lo(w.x); sa[1] = bf16_hi(w.x); sb[0] = bf16_lo(w.y); sb[1] = bf16_hi(w.y);
        } else {
            sa[0] = la & 2 ? bf16_hi(w.x) : bf16_lo(w.x);
            sb[0] = lb & 2 ? bf16_hi(w.y) : bf16_lo(w.y);
        }
        if (kZeros) {
            const uint32_t a = w.z >> (8 * (lza & 3)), b = w.w >> (8 * (lzb & 3));
#pragma unroll
            for (int i = 0; i < kW4Block / G; ++i) {
                za[i] = (a >> (8 * i)) & 15;
                zb[i] = (b >> (8 * i)) & 15;
            }
        }
    }
}

// One step: a 128-column block of 16 rows times NT token pairs. dig, sums and
// sx point to this lane's share of the first pair's block.
template <int G, bool kZeros, int NT>
__device__ __forceinline__ void w4_step(const uint4 qa, const uint4 qb, const float (&sa)[kW4Block / G],
                                        const float (&sb)[kW4Block / G], const int (&za)[kW4Block / G],
                                        const int (&zb)[kW4Block / G], const uint4 *dig, const int2 *sums,
                                        const float *sx, int blocks, float (&acc)[NT][4])
{
    constexpr int GB = kW4Block / G;
    uint32_t a[4][4];                             // operand bytes of each 32-column slice
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t wa = word_of(qa, j), wb = word_of(qb, j);
        a[j][0] = wa & 0x0f0f0f0fu;
        a[j][1] = wb & 0x0f0f0f0fu;
        a[j][2] = (wa >> 4) & 0x0f0f0f0fu;
        a[j][3] = (wb >> 4) & 0x0f0f0f0fu;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const uint4 d0 = dig[n * blocks * 64], d1 = dig[n * blocks * 64 + 32];
        const float x = sx[n * blocks * 2];
        int part[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j % (G / 32) == 0) {
                const int2 c = sums[n * blocks * GB * 4 + (j / (G / 32)) * 4];
                if (kZeros) {
                    const int gi = j / (G / 32);
                    part[0] = -za[gi] * c.x;
                    part[1] = -za[gi] * c.y;
                    part[2] = -zb[gi] * c.x;
                    part[3] = -zb[gi] * c.y;
                } else {                          // staged as -8 times the digit sum
                    part[0] = part[2] = c.x;
                    part[1] = part[3] = c.y;
                }
            }
            const uint4 &d = j < 2 ? d0 : d1;
            mma_u8s8(part, a[j][0], a[j][1], a[j][2], a[j][3], j & 1 ? d.z : d.x, j & 1 ? d.w : d.y);
            if (j % (G / 32) == G / 32 - 1) {
                const int gi = j / (G / 32);
                const float fa = sa[gi] * x, fb = sb[gi] * x;
                acc[n][0] = fmaf(fa, (float)part[0], acc[n][0]);
                acc[n][1] = fmaf(fa, (float)part[1], acc[n][1]);
                acc[n][2] = fmaf(fb, (float)part[2], acc[n][2]);
                acc[n][3] = fmaf(fb, (float)part[3], acc[n][3]);
            }
        }
    }
}

// The digits' sums of a token pair joined: lane (g, t) gets row g + 8 (t & 1)
// of token t >> 1. Even lanes hold digits 0 and 1, odd lanes digit 2.
__device__ __forceinline__ float join_digits(const float (&acc)[4])
{
    const bool odd = threadIdx.x & 1;
    const float a = odd ? acc[0] : fmaf(acc[0], 65536.f, acc[1] * 256.f);
    const float b = odd ? acc[2] : fmaf(acc[2], 65536.f, acc[3] * 256.f);
    const float other = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
    return (odd ? b : a) + other;
}

// Stores the joined sums v[pair] of a unit.
template <bool kUp, class YT, int NT>
__device__ __forceinline__ void store_unit(const W4Product &p, const W4Entry &e, int tile, const float (&v)[NT])
{
    const int lane = threadIdx.x & 31, g8 = lane >> 2, t = lane & 3;
    const bool shared = e.grp >= p.E;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int i = nt * 2 + (t >> 1);
        const size_t row = (size_t)e.row0 + i;
        if (kUp) {
            const float up = __shfl_xor_sync(0xffffffffu, v[nt], 1);
            const int f = tile * 8 + g8;
            if (i < e.n && !(t & 1) && f < p.rows)
                store_val(static_cast<YT *>(p.y) + row * p.rows + f, silu_mul(v[nt], up));
        } else {
            const int r = tile * 16 + g8 + 8 * (t & 1);
            if (i < e.n && r < p.rows) {
                YT *y = shared ? static_cast<YT *>(p.y_shared) + (row - p.P) * p.rows
                               : static_cast<YT *>(p.y) + row * p.rows;
                store_val(y + r, v[nt]);
            }
        }
    }
}

// Two 4-byte operand words per digit from eight fixed-point values: bytes of
// columns 0 4 1 5 and 2 6 3 7. v + 0x808080 has the balanced digits + 128 as its
// bytes, and flipping their top bits makes them signed bytes.
__device__ __forceinline__ void split_digits(const int (&v)[8], uint32_t (&w)[3][2])
{
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = ((uint32_t)v[i] + 0x808080u) ^ 0x808080u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {                 // columns 2h, 2h + 4, 2h + 1, 2h + 5
        const uint32_t lo = __byte_perm(b[2 * h], b[2 * h + 4], 0x5140), lo1 = __byte_perm(b[2 * h + 1], b[2 * h + 5], 0x5140);
        const uint32_t hi = __byte_perm(b[2 * h], b[2 * h + 4], 0x0062), hi1 = __byte_perm(b[2 * h + 1], b[2 * h + 5], 0x0062);
        w[2][h] = __byte_perm(lo, lo1, 0x5410);
        w[1][h] = __byte_perm(lo, lo1, 0x7632);
        w[0][h] = __byte_perm(hi, hi1, 0x5410);
    }
}

// Digits of the phase's tokens: 16 lanes take 128 columns of one token, eight
// each. Pairs without a second token get zeros in its place.
template <int G, bool kZeros, class XT>
__device__ __forceinline__ void stage_digits(const W4Args &a, const W4Smem &sm, int pairs, uint4 *dig, int *sums, float *sx)
{
    constexpr int GB = kW4Block / G, GL = G / 8;  // groups of a block; lanes of a group
    constexpr int kAhead = 4, kItems = kW4Threads / 16;
    const W4Product &p = a.p;
    const int blocks = p.cols / kW4Block, items = pairs * 2 * blocks;
    const int l16 = threadIdx.x & 15, jj = l16 >> 2, t = l16 & 3;
    for (int it0 = threadIdx.x >> 4; it0 - (int)(threadIdx.x >> 4) < items; it0 += kItems * kAhead) {
        float v[kAhead][8];                       // all loads first: their latencies overlap
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int it = it0 + k * kItems, slot = it / blocks, b = it - slot * blocks;
            const int xi = it < items ? sm.row[slot] : -1;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = 0.f;
            if (xi >= 0) load8(static_cast<const XT *>(p.x) + (size_t)xi * p.cols + b * kW4Block + l16 * 8, v[k]);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int it = it0 + k * kItems, slot = it / blocks, b = it - slot * blocks, tok = slot & 1;
            if (it - (int)(threadIdx.x >> 4) % 2 >= items) break;     // both halves of the warp are past the end
            uint32_t top = 0;                     // bits of the largest |x|; NaN and infinity are the largest
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[k][i]) & 0x7fffffffu);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            // exponent field of 2^E; below 2^-105 the digits stay at that scale (off by less than 2^-127)
            const uint32_t ex = max(top >> 23, 22u);
            const float mul = __uint_as_float((275u - ex) << 23);     // 2^(21 - E)
            int q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = __float2int_rn(v[k][i] * mul);
            uint32_t w[3][2];
            split_digits(q, w);
            int sum[3];
#pragma unroll
            for (int j = 0; j < 3; ++j) sum[j] = __dp4a((int)w[j][0], 0x01010101, __dp4a((int)w[j][1], 0x01010101, 0));
#pragma unroll
            for (int o = 1; o < GL; o <<= 1)
#pragma unroll
                for (int j = 0; j < 3; ++j) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
            if (it >= items) continue;
            const int at = (slot >> 1) * blocks + b;
            uint2 *out = reinterpret_cast<uint2 *>(dig + (at * 2 + (jj >> 1)) * 32) + (jj & 1);
#pragma unroll
            for (int j = 0; j < 3; ++j) out[((tok * 4 + j) * 4 + t) * 2] = make_uint2(w[j][0], w[j][1]);
            out[((tok * 4 + 3) * 4 + t) * 2] = make_uint2(0, 0);
            if (l16 % GL == 0) {
                int *c = sums + (at * GB + l16 / GL) * 8 + tok * 4;
                const int f = kZeros ? 1 : -8;
                *reinterpret_cast<int4 *>(c) = make_int4(f * sum[0], f * sum[1], f * sum[2], 0);
            }
            // a block with an infinity or a NaN makes this token's results NaN, and no other's
            if (l16 == 0) sx[at * 2 + tok] = (top >> 23) == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((ex - 21u) << 23);
        }
    }
}

// What a warp carries from unit to unit of a phase.
struct WarpRun {
    int s, s1, issued, stage;                     // step, end, steps copied, ring stage of this step
    int block;                                    // first block of the unit at hand
    bool open;                                    // the last unit goes on in later warps; v holds its sums so far
    int ent, tile;                                // the unit at hand
    float v[kW4Tiles];
};

// The units of one token block that are this warp's, for its NT token pairs.
template <bool kUp, int G, bool kZeros, class YT, int NT>
__device__ __forceinline__ void run_entry(const W4Args &a, W4Smem &sm, W4Stage<G> *ring, const uint4 *dig, const int *sums,
                                          const float *sx, WarpRun &r, Copier<kUp, G, kZeros> &cp)
{
    constexpr int GB = kW4Block / G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3;
    const int blocks = a.p.cols / kW4Block;
    const W4Entry e = sm.ent[r.ent];
    const int at = e.tile0 * blocks;
    const uint4 *d0 = dig + at * 64 + lane;
    const int2 *c0 = reinterpret_cast<const int2 *>(sums) + at * GB * 4 + t;
    const float *x0 = sx + at * 2 + (t >> 1);
    uint32_t ia = 0, ib = 0;                      // low bits of the group's index, which tell the place in its copied word
    bool fresh = true;
    while (true) {
        if (fresh || r.tile == a.tiles - 1) {     // the last tile of a matrix may repeat rows
            const UnitRows<kUp, G> w(a, e.grp, r.tile);
            const uint32_t gpr = a.p.cols / G;
            ia = (uint32_t)w.ra * gpr + r.block * GB;
            ib = (uint32_t)w.rb * gpr + r.block * GB;
            fresh = false;
        }
        const uint4 *d = d0 + r.block * 64;
        const int2 *c = c0 + r.block * GB * 4;
        const float *x = x0 + r.block * 2;
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
        const int n_steps = min(blocks - r.block, r.s1 - r.s);
        for (int i = 0; i < n_steps; ++i) {
            W4Stage<G> &st = ring[r.stage];
            cp_async_wait<kW4Stages - 2>();
            __syncwarp();                         // every lane's copies of this step; reads of the last one are done
            const uint4 qa = st.q[0][lane], qb = st.q[1][lane];
            float sa[GB], sb[GB];
            int za[GB], zb[GB];
            read_aux<G, kZeros>(st.aux[lane >> 2], 2 * ia, 2 * ib, ia, ib, sa, sb, za, zb);
            // the stage used one step ago takes the copy kW4Stages - 1 steps ahead
            const int prev = r.stage == 0 ? kW4Stages - 1 : r.stage - 1;
            if (r.issued < r.s1) {
                ++r.issued;
                cp.step(a, sm, ring[prev], r.issued < r.s1);
            }
            cp_async_commit();                    // an empty group past the end keeps the count
            r.stage = r.stage + 1 == kW4Stages ? 0 : r.stage + 1;
            w4_step<G, kZeros, NT>(qa, qb, sa, sb, za, zb, d, c, x, blocks, acc);
            d += 64;
            c += GB * 4;
            x += 2;
            ia += GB;
            ib += GB;
        }
        r.s += n_steps;
        const bool whole = r.block == 0, ends = r.block + n_steps == blocks;
        r.block = 0;
        float v[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) v[n] = join_digits(acc[n]);
        if (whole && ends) {
            store_unit<kUp, YT, NT>(a.p, e, r.tile, v);
        } else if (!whole) {                      // begun by an earlier warp
#pragma unroll
            for (int n = 0; n < NT; ++n) sm.head[warp][n][lane] = v[n];
        } else {
            r.open = true;
#pragma unroll
            for (int n = 0; n < NT; ++n) r.v[n] = v[n];
        }
        if (r.s >= r.s1) return;
        ia += a.s_jump;
        ib += a.s_jump;
        if (++r.tile == a.tiles) {
            r.tile = 0;
            ++r.ent;
            return;
        }
    }
}

template <bool kUp, int G, bool kZeros, class XT, class YT>
__global__ void __launch_bounds__(kW4Threads, 1)
w4_kernel(const __grid_constant__ W4Args a)
{
    extern __shared__ __align__(128) uint8_t smem_raw[];
    W4Smem &sm = *reinterpret_cast<W4Smem *>(smem_raw);
    constexpr int GB = kW4Block / G;
    const W4Product &p = a.p;
    const int blocks = p.cols / kW4Block;
    W4Stage<G> *ring = reinterpret_cast<W4Stage<G> *>(smem_raw + kW4Tables) + (threadIdx.x >> 5) * kW4Stages;
    uint4 *dig = reinterpret_cast<uint4 *>(smem_raw + kW4FixedSmem<G>);
    int *sums = reinterpret_cast<int *>(dig + (size_t)a.x_tiles * blocks * 64);
    float *sx = reinterpret_cast<float *>(sums + (size_t)a.x_tiles * blocks * GB * 8);
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (a.p.status && blockIdx.x == 0 && threadIdx.x == 0) *a.p.status = 0;

    // rows, token blocks and cost of every expert, the latter as exclusive prefixes
    {
        const int per = (a.groups + kW4Threads - 1) / kW4Threads;     // 1 to 3
        int n_blocks[3], cost[3], run = 0;
        long long run_cost = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int g = threadIdx.x * per + i;
            n_blocks[i] = cost[i] = 0;
            if (i < per && g < a.groups) {
                int start, count;
                group_rows(p, g, &start, &count);
                sm.start[g] = start;
                sm.count[g] = count;
                const int full = count / a.tokens, rest = count - full * a.tokens;
                n_blocks[i] = full + (rest > 0);
                cost[i] = full * w4_cost(a.tokens) + (rest ? w4_cost(rest) : 0);
            }
            run += n_blocks[i];
            run_cost += cost[i];
        }
        if (a.groups > 1) scan2(&run, &run_cost, sm);
        else run = 0, run_cost = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int g = threadIdx.x * per + i;
            if (i >= per || g >= a.groups) break;
            sm.pre[g] = run;
            sm.cost[g] = run_cost * a.tiles;
            run += n_blocks[i];
            run_cost += cost[i];
            if (g == a.groups - 1) {
                sm.pre[a.groups] = run;
                sm.cost[a.groups] = run_cost * a.tiles;
            }
        }
    }
    __syncthreads();
    // this CTA's share of the cost c: from c b / gridDim.x on, in parts that stay below 2^63
    const long long c = sm.cost[a.groups];
    auto at_share = [&](int b) { return unit_at(a, sm, c / gridDim.x * b + c % gridDim.x * b / gridDim.x); };
    const long long u1 = at_share(blockIdx.x + 1);
    for (long long u0 = at_share(blockIdx.x); u0 < u1;) {
        // the phase's token blocks: every warp works them out, each writes its share
        int n_ent = 0, used = 0;
        long long phase_end;
        {
            int tb = (int)(u0 / a.tiles), g = last_not_above(sm.pre, a.groups, tb);
            for (; n_ent < kW4Entries && (long long)tb * a.tiles < u1; ++n_ent, ++tb) {
                while (sm.pre[g + 1] <= tb) ++g;
                const int first = (tb - sm.pre[g]) * a.tokens, n = min(a.tokens, sm.count[g] - first);
                const int pairs = (n + 1) / 2, row0 = sm.start[g] + first;
                if (n_ent && used + pairs > a.x_tiles) break;
                if (n_ent % kW4Warps == warp) {
                    if (lane == 0) sm.ent[n_ent] = {g, row0, n, used};
                    if (lane < 2 * pairs) {       // x rows; a token that is not there stands for zeros
                        int xi = row0 + lane;
                        if (lane < n && !p.x_by_row) xi = g >= p.E ? xi - p.P : p.perm ? p.perm[xi] : xi;
                        sm.row[used * 2 + lane] = lane < n && (unsigned)xi < (unsigned)p.x_rows ? xi : -1;
                    }
                }
                used += pairs;
            }
            phase_end = min((long long)tb * a.tiles, u1);
        }
        __syncthreads();
        const int first_tile = (int)(u0 % a.tiles), steps = (int)(phase_end - u0) * blocks;
        const int s0 = (int)((long long)steps * warp / kW4Warps);
        WarpRun r{s0, (int)((long long)steps * (warp + 1) / kW4Warps), s0, 0, s0 % blocks, false, 0, 0, {}};
        Copier<kUp, G, kZeros> cp{};
        if (r.s < r.s1) {
            r.ent = (first_tile + s0 / blocks) / a.tiles;
            r.tile = first_tile + s0 / blocks - r.ent * a.tiles;
            cp.ent = r.ent;
            cp.tile = r.tile;
            cp.unit(a, sm, r.block);
        }
        for (int i = 0; i < kW4Stages - 1; ++i) {
            if (r.issued < r.s1) {
                ++r.issued;
                cp.step(a, sm, ring[i], r.issued < r.s1);
            }
            cp_async_commit();
        }
        stage_digits<G, kZeros, XT>(a, sm, used, dig, sums, sx);
        __syncthreads();
        while (r.s < r.s1) {
            const int nt = (sm.ent[r.ent].n + 1) / 2;
            if (nt == 1) run_entry<kUp, G, kZeros, YT, 1>(a, sm, ring, dig, sums, sx, r, cp);
            else if (nt == 2) run_entry<kUp, G, kZeros, YT, 2>(a, sm, ring, dig, sums, sx, r, cp);
            else if (nt == 3) run_entry<kUp, G, kZeros, YT, 3>(a, sm, ring, dig, sums, sx, r, cp);
            else run_entry<kUp, G, kZeros, YT, 4>(a, sm, ring, dig, sums, sx, r, cp);
        }
        __syncthreads();
        if (r.open) {                             // the warp that began a shared unit adds it up
            const W4Entry e = sm.ent[r.ent];
            const int end = ((r.s1 - 1) / blocks + 1) * blocks;       // the unit's last step + 1
            for (int w = warp + 1; w < kW4Warps; ++w) {
                const int w0 = (int)((long long)steps * w / kW4Warps), w1 = (int)((long long)steps * (w + 1) / kW4Warps);
                if (w0 >= end) break;
                if (w0 == w1) continue;           // a warp without steps
#pragma unroll
                for (int k = 0; k < kW4Tiles; ++k)
                    if (2 * k < e.n) r.v[k] += sm.head[w][k][lane];
            }
            store_unit<kUp, YT, kW4Tiles>(p, e, r.tile, r.v);
        }
        u0 = phase_end;
        if (u0 < u1) __syncthreads();             // tables and digits are free for the next phase
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

template <bool kUp, int G, bool kZeros, class XT, class YT>
static kmoe_status run_w4(W4Args a, cudaStream_t st)
{
    const size_t x_bytes = w4_x_bytes(a.p.cols, G);
    a.x_tiles = (int)std::min<size_t>((kW4SmemMax - kW4FixedSmem<G>) / x_bytes, kW4Entries * kW4Tiles);
    if (a.x_tiles < 1) return fail(KMOE_ERR_UNSUPPORTED, "4-bit products: cols=%d", a.p.cols);
    a.tokens = 2 * std::min(a.x_tiles, kW4Tiles);
    constexpr int kTileRows = kUp ? 8 : 16;
    a.q_jump = (kTileRows - 1) * (a.p.cols / 2);
    a.s_jump = (kTileRows - 1) * (a.p.cols / G);
    // no more CTAs than units there can be: an expert with rows has at least one token block
    const long long most = ((long long)std::min(a.p.E, a.p.P) + (a.p.P + a.p.n_shared) / a.tokens + 1) * a.tiles;
    const int grid = (int)std::min<long long>(sm_count_w4(), most);
    const size_t smem = kW4FixedSmem<G> + a.x_tiles * x_bytes;
    cudaFuncSetAttribute(w4_kernel<kUp, G, kZeros, XT, YT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    launch_pdl(w4_kernel<kUp, G, kZeros, XT, YT>, grid, kW4Threads, smem, st, a);
    return check_launch("w4");
}

template <bool kUp, class XT, class YT>
static kmoe_status pick_w4(const W4Args &a, cudaStream_t st)
{
    const bool z = a.p.w.z != nullptr;
    switch (a.p.group) {
    case 32: return z ? run_w4<kUp, 32, true, XT, YT>(a, st) : run_w4<kUp, 32, false, XT, YT>(a, st);
    case 64: return z ? run_w4<kUp, 64, true, XT, YT>(a, st) : run_w4<kUp, 64, false, XT, YT>(a, st);
    default: return z ? run_w4<kUp, 128, true, XT, YT>(a, st) : run_w4<kUp, 128, false, XT, YT>(a, st);
    }
}

kmoe_status launch_w4(const W4Product &p, cudaStream_t st)
{
    W4Args a{p, 0, p.E + (p.n_shared > 0 ? 1 : 0), 0, 0, 0, 0};
    if (a.groups > kW4MaxGroups) return fail(KMOE_ERR_UNSUPPORTED, "4-bit products: too many experts");
    const bool up = p.up.q != nullptr;
    a.tiles = up ? (p.rows + 7) / 8 : (p.rows + 15) / 16;
    if (up) return pick_w4<true, __nv_bfloat16, float>(a, st);
    if (p.x_f32) return pick_w4<false, float, __nv_bfloat16>(a, st);
    return p.y_dtype == KMOE_F32 ? pick_w4<false, __nv_bfloat16, float>(a, st)
                                 : pick_w4<false, __nv_bfloat16, __nv_bfloat16>(a, st);
}

}  // namespace kmoe
