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
// its integer pipe (28% of HBM's rate). For that x is cut into digits: for each
// token and 128 columns, with 2^E the power of two below the largest |x|,
//   x = 2^(E - 21) * (65536 t0 + 256 t1 + t2) + r,      |r| <= 2^(E - 22),
// with t in -128..127, which is exact for every BF16 x within 2^14 of the block's
// largest value. (Two digits, exact within 2^6 of it, would put four tokens into a
// fragment, which 200 tokens and more would gain by; but one x 1000 times the others would
// cost those 2% of their value, for all to see where its own weight is 0.) The
// digits of a token are three columns of the fragment, so it holds two
// tokens. The integer sums of a group are exact, as is 256 t0 + t1 of
// them (below 2^27). Zero points come off as -z times the sum of the digits.
// Group scale and power of two multiply the sums in FP32.
//
// With `up` weights, rows 0-7 of a fragment are eight gate features and rows
// 8-15 the same eight up features, and SiLU(gate) * up is written.
//
// A unit is two fragments (32 rows; 16 features) of one expert for up to 4
// tokens: the digits read for one fragment serve both. The units of all experts
// that have rows are numbered through and every CTA (one per SM) takes a
// contiguous share of them, in phases: as many units as the digits of their
// tokens fit into shared memory (nearly always all). A unit of more tokens
// costs more instructions for the same weights; shares are cut by that cost. A
// unit's columns are steps of 128, and a phase's steps are shared out evenly
// and contiguously among the warps. So a warp streams one long run of weights
// with no barrier in it: each lane copies its 16 bytes of four rows, and its
// share of their scales and zero points, kW4Stages - 1 steps ahead into the
// warp's shared memory (cp.async), which keeps 64 KB of an SM's weight traffic
// in flight without registers. Units that two or more warps share are added in
// warp order at the end, so results do not depend on timing.
//
// Measured on the layer's experts (384 of 512 x 2560, groups of 128, K = 6 and a
// shared one), cold: 32 tokens take 50 us for gate and up (208 MB: 4.2 TB/s) and 30
// us for down (104 MB: 3.5 TB/s). The steps run at HBM's rate; some 10 us of each
// launch go by before the first one (tables, plan, first copies, digits), of
// which the copies into L2 hide a part.
#include "w4.cuh"
#include "sm100.cuh"

#include <algorithm>

namespace kmoe {
using namespace sm100;

constexpr int kW4Warps = 16;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4Frags = 2;                       // row fragments of a unit
constexpr int kW4Cols = 2;                        // column fragments of a unit
constexpr int kW4FragTokens = 2;                  // tokens of a column fragment, three digits each
constexpr int kW4Pieces = 2 * 4 * 3 * kW4FragTokens;       // 16-byte pieces of a fragment's block
constexpr int kW4Stages = 3;                      // steps of a warp's copies in flight, plus the one in use
constexpr int kW4MaxGroups = 1025;
constexpr int kW4Entries = 32;                    // token blocks of a phase
constexpr int kW4Perm = kW4Threads;               // rows whose token is looked up in a table
constexpr int kW4Ahead = 3;                       // tokens' blocks a half-warp loads before it cuts the first into digits
constexpr int kW4Known = 1024;                    // token blocks whose expert is looked up in a table
constexpr int kW4SmemMax = 226 * 1024;

// Cost of a step by its tokens: what the CTAs' shares are cut by.
__host__ __device__ constexpr int w4_cost(int tokens) { return 3 + (tokens + kW4FragTokens - 1) / kW4FragTokens; }

struct W4Args {
    W4Product p;
    int tiles;              // units of one expert and token block
    int groups;             // experts, the shared one included
    int x_frags;            // column fragments whose digits fit into shared memory
    int tokens;             // tokens of a unit: those of kW4Cols fragments, fewer where x_frags is less
    int q_jump, s_jump;     // from the end of a row to the row of the next tile: code bytes, groups
    DivideBy by_blocks, by_tiles, by_tokens, by_grid;
    bool check;             // look whether offsets descend
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
    int grp, row0, n, tile0;                      // expert, first row, rows, first staged fragment
};

// One step's copies of a warp: code bytes of rows g, g + 8 (gate, up) of both
// fragments by lane, then for each g the words that hold the four rows' scales
// (4 bytes; 8 with groups of 32) and the words that hold their zero points.
template <int G, bool kZeros>
struct W4Stage {
    uint4 q[2 * kW4Frags][32];
    uint4 s[8][G == 32 ? 2 : 1];
    uint4 z[kZeros ? 8 : 1];
};

struct alignas(16) W4Smem {
    float head[kW4Warps][kW4Cols][kW4Frags][32];  // sums of a unit that an earlier warp began
    long long scan_tmp[32];
    W4Entry ent[kW4Entries];
    int share[4];                                 // this CTA's first unit and the one behind its last: token block, tile
    int n_ent, used;                              // the phase's token blocks, their column fragments
    uint8_t frag_ent[kW4Entries * kW4Cols];       // token block of every staged fragment
    uint16_t known[kW4Known];                     // expert of the first token blocks
    int perm[kW4Perm];                            // token of the first rows
};
static_assert(sizeof(W4Smem) % 16 == 0, "what follows is 16-byte aligned");
// Behind it: W4Stage [kW4Warps][kW4Stages], digits uint4 [fragment][block][2][digit columns][4], digit sums int
// [fragment][block][128 / G][4], powers of two float [fragment][block][4], and four tables of the experts.
__host__ __device__ constexpr size_t w4_x_bytes(int cols, int G)
{
    return (size_t)(cols / kW4Block) * (16 * kW4Pieces + 16 * (kW4Block / G) + 16);
}
template <int G, bool kZeros>
__host__ __device__ constexpr size_t w4_ring_bytes() { return sizeof(W4Stage<G, kZeros>) * kW4Warps * kW4Stages; }

// The experts' tables in shared memory, groups + 1 entries each.
struct W4Tables {
    int *pre, *cost;                              // token blocks of the experts before, and their cost
    int *start, *count;                           // rows of every expert
};

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
    long long v = lane < kW4Warps ? sm.scan_tmp[lane] : 0;
#pragma unroll
    for (int o = 1; o < kW4Warps; o <<= 1) {
        const long long n = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += n;
    }
    const long long up = __shfl_sync(0xffffffffu, v, warp ? warp - 1 : 0);
    const long long before = incl - mine + (warp ? up : 0);
    *count = (int)(before & 0x3fffffff);
    *cost = before >> 30;
}

// The unit (token block, numbered through all experts, and tile) at which share
// b of gridDim.x begins: the place b / gridDim.x of the total cost, in whole
// units of cost and a rest over gridDim.x, so that everything fits into 32 bits.
__device__ __forceinline__ int2 share_begin(const W4Args &a, const W4Tables &tab, int b)
{
    const int c = tab.cost[a.groups], grid = gridDim.x;
    if (b >= grid) return make_int2(tab.pre[a.groups], 0);
    const int q = a.by_grid(c), r = (c - q * grid) * b, rq = a.by_grid(r), whole = q * b + rq, rest = r - rq * grid;
    const int g = last_not_above(tab.cost, a.groups, whole), count = tab.count[g];
    const int full = w4_cost(a.tokens), tb = min((whole - tab.cost[g]) / full, a.by_tokens(count - 1));
    const int left = whole - tab.cost[g] - tb * full, w = w4_cost(min(a.tokens, count - tb * a.tokens));
    // left < 8, rest < grid, tiles <= 4096
    const int tile = (int)((uint32_t)(left * grid + rest) * (uint32_t)a.tiles / (uint32_t)(w * grid));
    return tile < a.tiles ? make_int2(tab.pre[g] + tb, tile) : make_int2(tab.pre[g] + tb + 1, 0);
}

// The token blocks of a phase that begins in token block `first`, by one warp:
// lane k takes block first + k, as many as there are up to the share's last
// (`last`, inclusive) and as fit into shared memory.
__device__ __forceinline__ void plan_phase(const W4Args &a, W4Smem &sm, const W4Tables &tab, int first, int last)
{
    const int lane = threadIdx.x & 31, tb = first + lane;
    const bool in = tb <= last;
    const int g = !in ? 0 : tb < kW4Known ? sm.known[tb] : last_not_above(tab.pre, a.groups, tb);
    const int skip = in ? (tb - tab.pre[g]) * a.tokens : 0, n = in ? min(a.tokens, tab.count[g] - skip) : 0;
    const int frags = (n + kW4FragTokens - 1) / kW4FragTokens, row0 = in ? tab.start[g] + skip : 0;
    int upto = frags;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    const bool take = in && upto <= a.x_frags;    // the first always fits
    const unsigned m = __ballot_sync(0xffffffffu, take);
    if (take) {
        sm.ent[lane] = {g, row0, n, upto - frags};
        for (int i = upto - frags; i < upto; ++i) sm.frag_ent[i] = lane;
    }
    if (lane == __popc(m) - 1) {
        sm.n_ent = lane + 1;
        sm.used = upto;
    }
}

// This lane's four weight rows of a unit: rows g and g + 8 of each fragment, in
// the order gate f, up f, gate f + 8, up f + 8 with `up` weights.
template <bool kUp>
__device__ __forceinline__ size_t unit_row(const W4Args &a, int grp, int tile, int i)
{
    const int g8 = (threadIdx.x & 31) >> 2;
    int r = kUp ? tile * 16 + g8 + 8 * (i >> 1) : tile * 32 + g8 + 8 * i;
    // rows past the end repeat an earlier one, a multiple of 8 rows before (or
    // the last); their results are not stored
    if (r >= a.p.rows) {
        r -= (r - a.p.rows + 8) & ~7;
        if (r < 0) r = a.p.rows - 1;
    }
    return (grp >= a.p.E ? 0 : (size_t)grp * a.p.rows) + r;
}
// The copies ahead: a walk over (unit, 128-column block) steps.
template <bool kUp, int G, bool kZeros>
struct Copier {
    int ent, tile, left;                          // left: blocks of the unit still to copy
    const uint8_t *q[4], *s, *z;                  // s, z: of row t of the four

    __device__ __forceinline__ void unit(const W4Args &a, const W4Smem &sm, int block)
    {
        constexpr int GB = kW4Block / G;
        const int grp = sm.ent[ent].grp, t = threadIdx.x & 3, pitch = a.p.cols / 2, gpr = a.p.cols / G;
        const W4Product &p = a.p;
        const bool shared = grp >= p.E, second = kUp && (t & 1);
        // plain selects: the pointers come from the constant bank
        const uint8_t *q0 = shared ? p.w_shared.q : p.w.q, *q1 = kUp ? (shared ? p.up_shared.q : p.up.q) : q0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = (i & 1 ? q1 : q0) + unit_row<kUp>(a, grp, tile, i) * pitch + t * 16 + (size_t)block * 64;
        const size_t at = unit_row<kUp>(a, grp, tile, t) * gpr + block * GB;
        const __nv_bfloat16 *s0 = second ? (shared ? p.up_shared.s : p.up.s) : (shared ? p.w_shared.s : p.w.s);
        s = reinterpret_cast<const uint8_t *>(s0 + at);
        if (kZeros) z = (second ? (shared ? p.up_shared.z : p.up.z) : (shared ? p.w_shared.z : p.w.z)) + at;
        left = a.p.cols / kW4Block - block;
    }
    // The aligned word that holds n bytes at p: from its start, no byte past them.
    template <int W>
    __device__ __forceinline__ static void word(void *dst, const uint8_t *p, int n)
    {
        const uint32_t in = (uint32_t)reinterpret_cast<uintptr_t>(p) & (W - 1);
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(p - in), "n"(W),
                     "r"(in + n)
                     : "memory");
    }
    // One step into `st`, which ends the unit's walk or goes on in it.
    __device__ __forceinline__ void step(const W4Args &a, const W4Smem &sm, W4Stage<G, kZeros> &st, bool more)
    {
        constexpr int GB = kW4Block / G, W = G == 32 ? 8 : 4;
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(smem_u32(&st.q[i][lane])), "l"(q[i])
                         : "memory");
            q[i] += 64;
        }
        word<W>(reinterpret_cast<uint8_t *>(st.s) + lane * W, s, 2 * GB);
        s += 2 * GB;
        if (kZeros) {
            word<4>(reinterpret_cast<uint8_t *>(st.z) + lane * 4, z, GB);
            z += GB;
        }
        if (--left == 0 && more) {
            if (++tile < a.tiles - 1) {           // whole tiles of one matrix lie at equal distances
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] += a.q_jump;
                s += 2 * a.s_jump;
                if (kZeros) z += a.s_jump;
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

// Asks for the weights behind a warp's first copies to be brought into L2: up
// to 16 KB, row by row. They arrive while the digits are made, when HBM would
// otherwise wait.
template <bool kUp>
__device__ __forceinline__ void prefetch_units(const W4Args &a, const W4Smem &sm, int ent, int tile, int block, int steps)
{
    const W4Product &p = a.p;
    const int lane = threadIdx.x & 31, blocks = p.cols / kW4Block;
    block += kW4Stages - 1;
    steps -= kW4Stages - 1;
    for (int left = 8; left > 0 && steps > 0;) {
        while (block >= blocks) {
            block -= blocks;
            if (++tile == a.tiles) {
                tile = 0;
                ++ent;
            }
        }
        const int n = min(min(blocks - block, left), steps), grp = sm.ent[ent].grp;
        const bool shared = grp >= p.E, second = kUp && lane >= 16;
        const int r = kUp ? tile * 16 + (lane & 15) : tile * 32 + lane;
        const uint8_t *q = second ? (shared ? p.up_shared.q : p.up.q) : (shared ? p.w_shared.q : p.w.q);
        q += ((shared ? 0 : (size_t)grp * p.rows) + r) * (p.cols / 2) + (size_t)block * 64;
        if (r < p.rows)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(q), "r"(n * 64) : "memory");
        block += n;
        left -= n;
        steps -= n;
    }
}

// Scales (FP32) of a step's four rows, and zero points, from their copied words.
// at: index of a row's first group in its array, whose low bits say where in
// the word it is; they are the same for the four rows, which lie multiples of
// eight rows apart.
template <int G>
__device__ __forceinline__ void read_scales(const uint4 *w, uint32_t at, float (&s)[4][kW4Block / G])
{
    const uint32_t lo[4] = {w[0].x, G == 32 ? w[0].z : w[0].y, G == 32 ? w[G == 32].x : w[0].z, G == 32 ? w[G == 32].z : w[0].w};
    const uint32_t hi[4] = {w[0].y, w[0].w, w[G == 32].y, w[G == 32].w};      // groups of 32 only
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (G == 128) {
            s[i][0] = at & 1 ? bf16_hi(lo[i]) : bf16_lo(lo[i]);
        } else {
            s[i][0] = bf16_lo(lo[i]);
            s[i][1] = bf16_hi(lo[i]);
        }
        if constexpr (G == 32) {
            s[i][2] = bf16_lo(hi[i]);
            s[i][3] = bf16_hi(hi[i]);
        }
    }
}
template <int G>
__device__ __forceinline__ void read_zeros(const uint4 &w, uint32_t at, int (&z)[4][kW4Block / G])
{
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = G == 32 ? v[i] : v[i] >> (8 * (at & 3));
#pragma unroll
        for (int k = 0; k < kW4Block / G; ++k) z[i][k] = (b >> (8 * k)) & 15;
    }
}

// One step: a 128-column block of two row fragments times NT column fragments.
// dig, sums and sx point to this lane's share of the first one's block.
// acc[column fragment][row fragment][half]: rows g and g + 8 of token t >> 1, digits
// 0 and 1 in even lanes, digit 2 in odd ones.
template <int G, bool kZeros, int NT>
__device__ __forceinline__ void w4_step(const uint4 (&q)[4], const float (&s)[4][kW4Block / G],
                                        const int (&z)[4][kW4Block / G], const uint4 *dig, const int *sums,
                                        const float *sx, int blocks, float (&acc)[NT][kW4Frags][2])
{
    constexpr int GB = kW4Block / G, GS = G / 32; // groups of a block; 32-column slices of a group
    constexpr int P = kW4Pieces;
    const int second = 1 - (threadIdx.x & 1);     // odd lanes hold digit 2 and a column without meaning
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const uint4 d0 = dig[n * blocks * P], d1 = dig[n * blocks * P + P / 2];
        const float x = sx[n * blocks * 4];
        int part[kW4Frags][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int gi = j / GS;
            if (j % GS == 0)
#pragma unroll
                for (int f = 0; f < kW4Frags; ++f) part[f][0] = part[f][1] = part[f][2] = part[f][3] = 0;
            const uint4 &d = j < 2 ? d0 : d1;
#pragma unroll
            for (int f = 0; f < kW4Frags; ++f) {
                const uint32_t wa = word_of(q[2 * f], j), wb = word_of(q[2 * f + 1], j);
                mma_u8s8(part[f], wa & 0x0f0f0f0fu, wb & 0x0f0f0f0fu, (wa >> 4) & 0x0f0f0f0fu, (wb >> 4) & 0x0f0f0f0fu,
                         j & 1 ? d.z : d.x, j & 1 ? d.w : d.y);
            }
            if (j % GS == GS - 1) {
                const int c = sums[n * blocks * GB * 4 + gi * 4];     // of this lane's digits; times -8 without zero points
#pragma unroll
                for (int f = 0; f < kW4Frags; ++f)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int sum = part[f][2 * h] * 256 + part[f][2 * h + 1] * second + (kZeros ? -z[2 * f + h][gi] * c : c);
                        acc[n][f][h] = fmaf(s[2 * f + h][gi] * x, (float)sum, acc[n][f][h]);
                    }
            }
        }
    }
}

// Joins the digits of a unit's fragments: lane (g, t) gets row g + 8 (t & 1) of
// token t >> 1.
__device__ __forceinline__ float join_digits(const float (&acc)[2])
{
    const bool odd = threadIdx.x & 1;
    const float mine = odd ? acc[1] : acc[0], other = __shfl_xor_sync(0xffffffffu, odd ? acc[0] : acc[1], 1);
    return fmaf(odd ? other : mine, 256.f, (odd ? mine : other) * (1.f / 256.f));
}

// Stores the sums v[column fragment][row fragment] of a unit.
template <bool kUp, class YT, int NT>
__device__ __forceinline__ void store_unit(const W4Product &p, const W4Entry &e, int tile, const float (&v)[NT][kW4Frags])
{
    const int lane = threadIdx.x & 31, g8 = lane >> 2, t = lane & 3;
    const bool shared = e.grp >= p.E;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int i = n * kW4FragTokens + (t >> 1);
        const size_t row = (size_t)e.row0 + i;
        if constexpr (kUp) {                      // even lanes hold gates, odd ones ups: they take feature f of the two fragments
            const float o = __shfl_xor_sync(0xffffffffu, t & 1 ? v[n][0] : v[n][1], 1);
            const float gate = t & 1 ? o : v[n][0], up = t & 1 ? v[n][1] : o;
            const int f = tile * 16 + g8 + 8 * (t & 1);
            if (i < e.n && f < p.rows) store_val(static_cast<YT *>(p.y) + row * p.rows + f, silu_mul(gate, up));
        } else {
            if (i >= e.n) continue;
            YT *y = shared ? static_cast<YT *>(p.y_shared) + (row - p.P) * p.rows : static_cast<YT *>(p.y) + row * p.rows;
#pragma unroll
            for (int f = 0; f < kW4Frags; ++f) {
                const int r = tile * 32 + 16 * f + g8 + 8 * (t & 1);
                if (r < p.rows) store_val(y + r, v[n][f]);
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

// Eight columns of kW4Ahead staged tokens' blocks, from item it0 on (16 lanes
// take the 128 columns of an item). A token that is not there stands for zeros.
template <class XT>
__device__ __forceinline__ void load_items(const W4Args &a, const W4Smem &sm, int it0, int items, float (&v)[kW4Ahead][8])
{
    const W4Product &p = a.p;
    const int blocks = p.cols / kW4Block;
#pragma unroll
    for (int k = 0; k < kW4Ahead; ++k) {
        const int it = it0 + k * (kW4Threads / 16), slot = a.by_blocks(it), b = it - slot * blocks;
        int xi = -1;
        if (it < items) {
            const W4Entry e = sm.ent[sm.frag_ent[slot / kW4FragTokens]];
            const int i = slot - kW4FragTokens * e.tile0;
            if (i < e.n) {
                xi = e.row0 + i;
                if (!p.x_by_row) xi = e.grp >= p.E ? xi - p.P : !p.perm ? xi : xi < kW4Perm ? sm.perm[xi] : p.perm[xi];
                if ((unsigned)xi >= (unsigned)p.x_rows) xi = -1;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = 0.f;
        if (xi >= 0) load8(static_cast<const XT *>(p.x) + (size_t)xi * p.cols + b * kW4Block + (threadIdx.x & 15) * 8, v[k]);
    }
}

// Digits of the phase's tokens; v holds the first items' values.
template <int G, bool kZeros, class XT>
__device__ __forceinline__ void stage_digits(const W4Args &a, const W4Smem &sm, int frags, float (&v)[kW4Ahead][8], uint4 *dig,
                                             int *sums, float *sx)
{
    constexpr int GB = kW4Block / G, GL = G / 8;  // groups of a block; lanes of a group
    constexpr int kItems = kW4Threads / 16, kPer = kW4FragTokens, kShift = 21;
    const int blocks = a.p.cols / kW4Block, items = frags * kPer * blocks;
    const int l16 = threadIdx.x & 15, jj = l16 >> 2, t = l16 & 3;
#pragma unroll 1
    for (int it0 = threadIdx.x >> 4;;) {
#pragma unroll 1
        for (int k = 0; k < kW4Ahead; ++k) {
            const int it = it0 + k * kItems, slot = a.by_blocks(it), b = it - slot * blocks, tok = slot % kPer;
            if (it - (int)(threadIdx.x >> 4) % 2 >= items) break;     // both halves of the warp are past the end
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = k == 0 ? v[0][i] : k == 1 ? v[1][i] : v[2][i];
            uint32_t top = 0;                     // bits of the largest |x|; NaN and infinity are the largest
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            // exponent field of 2^E; below 2^-105 the digits stay at that scale (off by less than 2^-118)
            const uint32_t ex = max(top >> 23, 22u);
            const float mul = __uint_as_float((254u + kShift - ex) << 23);    // 2^(kShift - E)
            int q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = __float2int_rn(x[i] * mul);
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
            const int at = slot / kPer * blocks + b;
            uint2 *out = reinterpret_cast<uint2 *>(dig + at * kW4Pieces + (jj >> 1) * (kW4Pieces / 2)) + (jj & 1);
#pragma unroll
            for (int j = 0; j < 3; ++j) out[((tok * 3 + j) * 4 + t) * 2] = make_uint2(w[j][0], w[j][1]);
            if (l16 % GL == 0) {
                const int f = kZeros ? 1 : -8;
                *reinterpret_cast<int2 *>(sums + (at * GB + l16 / GL) * 4 + tok * 2) = make_int2(f * (256 * sum[0] + sum[1]), f * 256 * sum[2]);
            }
            // a block with an infinity or a NaN makes this token's results NaN, and no other's
            if (l16 == 0)
                sx[at * 4 + tok] = (top >> 23) == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((ex - kShift) << 23);
        }
        it0 += kItems * kW4Ahead;
        if (it0 - (int)(threadIdx.x >> 4) % 2 >= items) break;
        load_items<XT>(a, sm, it0, items, v);
    }
}

// What a warp carries from unit to unit of a phase.
struct WarpRun {
    int s, s1, issued, stage;                     // step, end, steps copied, ring stage of this step
    int block;                                    // first block of the unit at hand
    bool open;                                    // the last unit goes on in later warps; its sums so far lie in the ring
    int ent, tile;                                // the unit at hand
};

// The units of one token block that are this warp's, for its NT column fragments.
template <bool kUp, int G, bool kZeros, class YT, int NT>
__device__ __forceinline__ void run_entry(const W4Args &a, W4Smem &sm, W4Stage<G, kZeros> *ring, const uint4 *dig, const int *sums,
                                          const float *sx, WarpRun &r, Copier<kUp, G, kZeros> &cp)
{
    constexpr int GB = kW4Block / G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3;
    const int blocks = a.p.cols / kW4Block;
    const W4Entry e = sm.ent[r.ent];
    const int at0 = e.tile0 * blocks;
    // column g of a fragment: digit g & 3 of token g >> 2 (there is no fourth digit: its column repeats the third)
    const int column = (lane >> 4) * 3 + min((lane >> 2) & 3, 2);
    const uint4 *d0 = dig + at0 * kW4Pieces + column * 4 + t;
    const int *c0 = sums + at0 * GB * 4 + t;
    const float *x0 = sx + at0 * 4 + (t >> 1);
    uint32_t at = 0;                              // index of the first row's group at hand, modulo 2^32
    bool fresh = true;
    while (true) {
        if (fresh || r.tile == a.tiles - 1) {     // the last tile of a matrix may repeat rows
            at = (uint32_t)unit_row<kUp>(a, e.grp, r.tile, 0) * (uint32_t)(a.p.cols / G) + r.block * GB;
            fresh = false;
        }
        const uint4 *d = d0 + r.block * kW4Pieces;
        const int *c = c0 + r.block * GB * 4;
        const float *x = x0 + r.block * 4;
        float acc[NT][kW4Frags][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int f = 0; f < kW4Frags; ++f)
#pragma unroll
                for (int i = 0; i < 2; ++i) acc[n][f][i] = 0.f;
        const int n_steps = min(blocks - r.block, r.s1 - r.s);
        for (int i = 0; i < n_steps; ++i) {
            W4Stage<G, kZeros> &st = ring[r.stage];
            cp_async_wait<kW4Stages - 2>();
            __syncwarp();                         // every lane's copies of this step; reads of the last one are done
            const uint4 q[4] = {st.q[0][lane], st.q[1][lane], st.q[2][lane], st.q[3][lane]};
            float s[4][GB];
            int z[4][GB];
            read_scales<G>(st.s[lane >> 2], at, s);
            if (kZeros) read_zeros<G>(st.z[lane >> 2], at, z);
            // the stage used one step ago takes the copy kW4Stages - 1 steps ahead
            const int prev = r.stage == 0 ? kW4Stages - 1 : r.stage - 1;
            if (r.issued < r.s1) {
                ++r.issued;
                cp.step(a, sm, ring[prev], r.issued < r.s1);
            }
            cp_async_commit();                    // an empty group past the end keeps the count
            r.stage = r.stage + 1 == kW4Stages ? 0 : r.stage + 1;
            w4_step<G, kZeros, NT>(q, s, z, d, c, x, blocks, acc);
            d += kW4Pieces;
            c += GB * 4;
            x += 4;
            at += GB;
        }
        r.s += n_steps;
        const bool whole = r.block == 0, ends = r.block + n_steps == blocks;
        r.block = 0;
        float v[NT][kW4Frags];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int f = 0; f < kW4Frags; ++f) v[n][f] = join_digits(acc[n][f]);
        if (whole && ends) {
            store_unit<kUp, YT, NT>(a.p, e, r.tile, v);
        } else {
            // begun by an earlier warp; or later warps go on with it: the warp's last step, its ring is free
            if (whole) r.open = true;
            __syncwarp();
            float *to = whole ? reinterpret_cast<float *>(ring) : &sm.head[warp][0][0][0];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int f = 0; f < kW4Frags; ++f) to[(n * kW4Frags + f) * 32 + lane] = v[n][f];
        }
        if (r.s >= r.s1) return;
        at += a.s_jump;
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
    uint8_t *behind = smem_raw + sizeof(W4Smem);
    W4Stage<G, kZeros> *ring = reinterpret_cast<W4Stage<G, kZeros> *>(behind) + (threadIdx.x >> 5) * kW4Stages;
    uint4 *dig = reinterpret_cast<uint4 *>(behind + w4_ring_bytes<G, kZeros>());
    int *sums = reinterpret_cast<int *>(dig + a.x_frags * blocks * kW4Pieces);
    float *sx = reinterpret_cast<float *>(sums + a.x_frags * blocks * GB * 4);
    W4Tables tab;
    tab.pre = reinterpret_cast<int *>(sx + a.x_frags * blocks * 4);
    tab.cost = tab.pre + a.groups + 1;
    tab.start = tab.cost + a.groups + 1;
    tab.count = tab.start + a.groups + 1;
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (a.p.status && blockIdx.x == 0 && threadIdx.x == 0) *a.p.status = 0;

    if (a.check && offsets_descend(p)) return;     // then nothing is done
    // rows, token blocks and cost of every expert, the latter as exclusive prefixes
    if (p.perm && threadIdx.x < min(p.P, kW4Perm)) sm.perm[threadIdx.x] = p.perm[threadIdx.x];
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
                tab.start[g] = start;
                tab.count[g] = count;
                const int full = a.by_tokens(count), rest = count - full * a.tokens;
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
            tab.pre[g] = run;
            tab.cost[g] = (int)run_cost;
            for (int k = run; k < min(run + n_blocks[i], kW4Known); ++k) sm.known[k] = g;
            run += n_blocks[i];
            run_cost += cost[i];
            if (g == a.groups - 1) {
                // ranges that overlap could count beyond 32 bits: then nothing is done
                const bool fits = run_cost < 0x7fffffffLL;
                tab.pre[a.groups] = fits ? run : 0;
                tab.cost[a.groups] = fits ? (int)run_cost : 0;
            }
        }
    }
    __syncthreads();
    if (tab.cost[a.groups] == 0) return;           // no rows
    if (warp == 0) {
        if (lane < 2) reinterpret_cast<int2 *>(sm.share)[lane] = share_begin(a, tab, blockIdx.x + lane);
        __syncwarp();
        plan_phase(a, sm, tab, sm.share[0], sm.share[2] - (sm.share[3] == 0));
    }
    __syncthreads();
    const int2 u1 = make_int2(sm.share[2], sm.share[3]);
    for (int2 u0 = make_int2(sm.share[0], sm.share[1]); u0.x < u1.x || (u0.x == u1.x && u0.y < u1.y);) {
        const int n_ent = sm.n_ent, used = sm.used;
        int units = n_ent * a.tiles - u0.y;
        int2 next = make_int2(u0.x + n_ent, 0);
        if (next.x > u1.x) {                      // the share ends inside the last token block
            units -= a.tiles - u1.y;
            next = u1;
        }
        const int steps = units * blocks;
        const int s0 = (int)((long long)steps * warp / kW4Warps);
        const int unit0 = a.by_blocks(s0);
        float v[kW4Ahead][8];
        load_items<XT>(a, sm, threadIdx.x >> 4, used * kW4FragTokens * blocks, v);
        WarpRun r{s0, (int)((long long)steps * (warp + 1) / kW4Warps), s0, 0, s0 - unit0 * blocks, false, 0, 0};
        Copier<kUp, G, kZeros> cp{};
        if (r.s < r.s1) {
            r.ent = a.by_tiles(u0.y + unit0);
            r.tile = u0.y + unit0 - r.ent * a.tiles;
            cp.ent = r.ent;
            cp.tile = r.tile;
            cp.unit(a, sm, r.block);
        }
#pragma unroll 1
        for (int i = 0; i < kW4Stages - 1; ++i) {
            if (r.issued < r.s1) {
                ++r.issued;
                cp.step(a, sm, ring[i], r.issued < r.s1);
            }
            cp_async_commit();
        }
        prefetch_units<kUp>(a, sm, r.ent, r.tile, r.block, r.s1 - r.s);
        stage_digits<G, kZeros, XT>(a, sm, used, v, dig, sums, sx);
        __syncthreads();
        while (r.s < r.s1) {
            if (sm.ent[r.ent].n <= kW4FragTokens) run_entry<kUp, G, kZeros, YT, 1>(a, sm, ring, dig, sums, sx, r, cp);
            else run_entry<kUp, G, kZeros, YT, 2>(a, sm, ring, dig, sums, sx, r, cp);
        }
        __syncthreads();
        if (r.open) {                             // the warp that began a shared unit adds it up
            const W4Entry e = sm.ent[r.ent];
            const int end = a.by_blocks(r.s1 - 1) * blocks + blocks;     // the unit's last step + 1
            float v[kW4Cols][kW4Frags];
            const float *mine = reinterpret_cast<const float *>(ring);
#pragma unroll
            for (int i = 0; i < kW4Cols * kW4Frags; ++i)          // (fragments that the unit does not have: no token is stored)
                v[i / kW4Frags][i % kW4Frags] = mine[i * 32 + lane];
            for (int w = warp + 1; w < kW4Warps; ++w) {
                const int w0 = (int)((long long)steps * w / kW4Warps), w1 = (int)((long long)steps * (w + 1) / kW4Warps);
                if (w0 >= end) break;
                if (w0 == w1) continue;           // a warp without steps
#pragma unroll
                for (int i = 0; i < kW4Cols * kW4Frags; ++i) v[i / kW4Frags][i % kW4Frags] += (&sm.head[w][0][0][0])[i * 32 + lane];
            }
            store_unit<kUp, YT, kW4Cols>(p, e, r.tile, v);
        }
        u0 = next;
        if (u0.x < u1.x || (u0.x == u1.x && u0.y < u1.y)) {
            __syncthreads();                      // tables and digits are free again
            if (warp == 0) plan_phase(a, sm, tab, u0.x, u1.x - (u1.y == 0));
            __syncthreads();
        }
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
    const size_t fixed = sizeof(W4Smem) + w4_ring_bytes<G, kZeros>() + 4 * sizeof(int) * (a.groups + 1);
    a.x_frags = (int)std::min<size_t>((kW4SmemMax - fixed) / x_bytes, kW4Entries * kW4Cols);
    if (a.x_frags < 1) return fail(KMOE_ERR_UNSUPPORTED, "4-bit products: cols=%d", a.p.cols);
    a.tokens = kW4FragTokens * std::min(a.x_frags, kW4Cols);
    // the units' cost is counted in 31 bits
    if (((long long)(a.p.P + a.p.n_shared) / a.tokens + a.groups) * w4_cost(a.tokens) >= 0x7fffffffLL)
        return fail(KMOE_ERR_UNSUPPORTED, "4-bit products: %d rows of %d columns", a.p.P, a.p.cols);
    a.check = may_overflow(a.p, a.tokens);
    constexpr int kTileRows = kUp ? 16 : 32;
    a.tiles = (a.p.rows + kTileRows - 1) / kTileRows;
    a.q_jump = (kTileRows - 1) * (a.p.cols / 2);
    a.s_jump = (kTileRows - 1) * (a.p.cols / G);
    const int blocks = a.p.cols / kW4Block;
    a.by_blocks = DivideBy::make(blocks);
    a.by_tiles = DivideBy::make(a.tiles);
    a.by_tokens = DivideBy::make(a.tokens);
    // no more CTAs than units there can be: an expert with rows has at least one token block
    const long long most = ((long long)std::min(a.p.E, a.p.P) + (a.p.P + a.p.n_shared) / a.tokens + 1) * a.tiles;
    const int grid = (int)std::min<long long>(sm_count_w4(), most);
    a.by_grid = DivideBy::make(grid);
    const size_t smem = fixed + a.x_frags * x_bytes;
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
    W4Args a{};
    a.p = p;
    a.groups = p.E + (p.n_shared > 0 ? 1 : 0);
    if (a.groups > kW4MaxGroups) return fail(KMOE_ERR_UNSUPPORTED, "4-bit products: too many experts");
    if (p.up.q != nullptr) return pick_w4<true, __nv_bfloat16, float>(a, st);
    if (p.x_f32) return pick_w4<false, float, __nv_bfloat16>(a, st);
    return p.y_dtype == KMOE_F32 ? pick_w4<false, __nv_bfloat16, float>(a, st)
                                 : pick_w4<false, __nv_bfloat16, __nv_bfloat16>(a, st);
}

}  // namespace kmoe
