// Products with 4-bit weights on the 5th-generation tensor cores, for batches
// whose experts see many tokens (linear_w4.cu is the kernel for few).
//
//   y[p][r] = sum_c (q[r][c] - z[r][c / group]) s[r][c / group] x[p][c]
// Weights are the M operand (128 rows), tokens the N operand (up to 128), both
// in FP16 with FP32 sums. With powers of two taken out, FP16 holds more of both
// than BF16 would: 2^-a times x, a from the largest value of its row, is exact
// for every BF16 x within 2^30 of that value, and (q - z) times the row's
// scale over the power of two below its largest scale is exact for |q - z| <= 8 and
// off by at most 2^-11 of the weight otherwise (a BF16 weight would be off by
// 2^-8, the rounding of the result). That holds for scales within 2^8 of the row's
// largest; CTAs that meet others start anew in a pass that moves the power of
// two along the row (`wide`, below).
// The powers of two come back in FP32 with the sums.
//
// Unpacking costs this kernel most of its instructions (9 for 8 weights), so a weight is
// unpacked once for up to 128 tokens, scale included, and the sums stay in
// tensor memory for a unit's whole depth; and unpacked weights take no
// shared-memory bandwidth: the unpacking threads write them straight into
// tensor memory, from where the MMA reads its A operand. A unit is two M tiles
// (256 rows of one expert, or 128 gate and the same 128 up features) and a
// block of tokens. Units are dealt to the CTAs (one per SM) in turn.
//   warps 0-7    results: sums from tensor memory, SiLU(gate) * up or y (warps
//                0-3 and 4-7 take turns in steps of 16 tokens, so that a slot is
//                soon free)
//   warps 8-15   unpack: 64 bytes of codes of a row and 128 columns into 64
//                columns of tensor memory (8-11 tile 0, 12-15 tile 1)
//   warp 16      loads code tiles by TMA (64-byte swizzle: the unpackers' reads
//                have no bank conflicts)
//   warp 17      issues tcgen05.mma
//   warps 18-19  gather token rows with cp.async (a TMA gather of four rows
//                costs its issuer 80 clocks, too much for 64 tokens)
// Measured on the layer's experts (384 of 512 x 2560, groups of 128, K = 6 and a
// shared one), cold and alone: 4096 tokens take 224 us for gate and up (150 GFLOP: 670
// TFLOP/s; the tensor pipe was 43% busy at 218) and 145 us for down (75 GFLOP: 520 TFLOP/s,
// 30%). Call after call the FFN takes 450 us in all, since the power limit lowers the clock.
// Instruction issue bounds it: 2.3 a clock over warps that wait for one another,
// with room for two buffers of unpacked weights only. Unpacking by 16 warps took
// 408 us in all, not 372: their reads hold up the token rows' copies.
//
// Tensor memory: sums 2 tiles x 2 slots x 64 columns (a unit of more than 64
// tokens takes both slots), unpacked weights 2 tiles x 2 buffers x 64 columns.
#include "sm100.cuh"
#include "swap_units.cuh"
#include "w4.cuh"

#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <type_traits>

namespace kmoe {
using namespace sm100;

namespace w4tc {

constexpr int kThreads = 20 * 32;
constexpr int kTokens = 128;                      // tokens of a unit
constexpr int kRows = 128;                        // rows of an M tile
constexpr int kCodeTile = kRows * 64;             // bytes of one tile's codes of a 128-column block
constexpr int kPanel = kTokens * 128;             // bytes of 64 columns of a token block
constexpr int kStages = 4;                        // 128-column blocks in flight: codes 16 KB, tokens 32 KB each
constexpr int kMaxGroups = 1025;
constexpr int kKnown = 2048;                      // token blocks whose expert is looked up in a table
constexpr int kLoadWarp = 16, kMmaWarp = 17, kGatherWarp = 18;
constexpr int kGatherThreads = 64;

struct Maps {
    CUtensorMap w[2], w_shared[2];                // codes (gate, up with SwiGLU)
};

struct Args {
    W4Product p;
    int tiles, groups;                            // units of a token block; experts, the shared one included
    DivideBy by_tiles;
    bool check;                                   // look whether offsets descend
    const void *x16;                              // x in FP16, rows x_pitch bytes apart
    size_t x_pitch;
    const float *x_scale;                         // its rows' powers of two
    int *err;
    long long wait_limit;
};

struct Barriers {
    uint64_t cfull[kStages], cempty[kStages], bfull[kStages], bempty[kStages];
    uint64_t afull[2], aempty[2], dfull[2], dempty[2], drain;          // dfull: every second unit's sums; dempty: a slot read
};

enum { kGoOn = 0, kGaveUp = 1, kStartAnew = 2 };      // a wait ran out; a row's scales differ widely: the wide pass follows

struct Tail {
    Barriers bars[2];                             // of the usual pass and of the wide one
    uint32_t tmem_base;
    int abort, total, sums[kThreads / 32];        // abort: kGoOn, or why every role leaves its units
    int pre[kMaxGroups + 1], start[kMaxGroups], count[kMaxGroups], size[kMaxGroups];   // size: tokens of a block
    uint16_t known[kKnown];
    uint8_t field[4][2][kRows];                   // exponent fields of the rows' bases, of units in turn
    // Wide pass: whether an unpacking warp has a row whose groups need a base each, of blocks in
    // turn (the MMA warp is at most two buffers behind), and when all of them have said so.
    alignas(8) uint8_t split[8][8];
    uint64_t vote;
    // result warps: the tokens' powers of two, and 16 tokens' results of 32 rows
    alignas(16) float tok[8][kTokens];
    alignas(16) uint32_t turn[8][8 * 32];

    __device__ __forceinline__ bool any_split(uint32_t it) const
    {
        return *reinterpret_cast<const volatile unsigned long long *>(split[it & 7]) != 0;
    }
};
constexpr size_t kSmem = 1024 + (size_t)kStages * (2 * kCodeTile + 2 * kPanel) + sizeof(Tail);

// mbar_wait by a whole warp: true in every lane, or false in every lane. Past
// the first look the warp is suspended for up to 4 us at a time, so a shorter
// limit counts as that.
__device__ __forceinline__ bool wait_slowly(uint64_t *bar, uint32_t parity, volatile int *abort, int *err, long long limit)
{
    const long long t0 = clock64();
    bool done = false, give_up = false;
    while (!done && !give_up) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(4000)
            : "memory");
        done = ok != 0;
        if (!done && clock64() - t0 > limit) {
            *abort = kGaveUp;
            if (err) atomicCAS(err, kErrNone, kErrWaitTimeout);
        }
        give_up = !done && *abort;
    }
    return __all_sync(0xffffffffu, done);
}
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort, int *err, long long limit)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return wait_slowly(bar, parity, abort, err, limit);
}

struct Unit {
    int grp, row0, n, tile;
};

__device__ __forceinline__ Unit unit_of(const Args &a, const Tail &T, int u)
{
    const int tb = a.by_tiles(u), g = tb < kKnown ? T.known[tb] : last_not_above(T.pre, a.groups, tb);
    const int first = (tb - T.pre[g]) * T.size[g];
    return {g, T.start[g] + first, min(T.size[g], T.count[g] - first), u - tb * a.tiles};
}

// Tokens of a block of a group with `count` rows: equal blocks of at most 128.
__device__ __forceinline__ int block_size(int count)
{
    const int n = (count + kTokens - 1) / kTokens;
    return n > 1 ? (((count + n - 1) / n) + 3) & ~3 : kTokens;
}

// Tables of the groups. Each thread has one group of a step, its number of
// blocks is added up over the warp, and then over the warps before.
__device__ __forceinline__ void build_tables(const Args &a, Tail &T)
{
    constexpr int kWarps = kThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (a.check && offsets_descend(a.p)) {        // then nothing is done
        if (threadIdx.x == 0) T.total = 0;
        __syncthreads();
        return;
    }
    int run = 0;
    for (int g0 = 0; g0 < a.groups; g0 += kThreads) {
        const int g = g0 + threadIdx.x;
        int n = 0;
        if (g < a.groups) {
            int start, count;
            group_rows(a.p, g, &start, &count);
            const int size = block_size(count);
            T.start[g] = start;
            T.count[g] = count;
            T.size[g] = size;
            n = (count + size - 1) / size;
        }
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) T.sums[warp] = incl;
        __syncthreads();
        int before = run + incl - n;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int v = T.sums[w];
            before += w < warp ? v : 0;
            run += v;
        }
        if (g < a.groups) {
            T.pre[g] = before;
            for (int k = before; k < min(before + n, kKnown); ++k) T.known[k] = g;
        }
        __syncthreads();                          // sums are read
    }
    if (threadIdx.x == 0) {
        T.pre[a.groups] = run;
        // ranges that overlap could count beyond the units' 32 bits: then nothing is done
        T.total = (long long)run * a.tiles < 0x7fff0000LL ? run * a.tiles : 0;
    }
    __syncthreads();
}

// Asks L2 for bytes that lie at p, but for parts of 16 at the ends.
__device__ __forceinline__ void prefetch_l2(const void *p, size_t bytes)
{
    const uintptr_t from = (reinterpret_cast<uintptr_t>(p) + 15) & ~uintptr_t(15), to = (reinterpret_cast<uintptr_t>(p) + bytes) & ~uintptr_t(15);
    if (to > from) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"((uint32_t)(to - from)) : "memory");
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, FP16 inputs, FP32 accumulation.
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Instruction descriptor: FP16 A and B (both K-major), FP32 sums, M x N tile.
__device__ __forceinline__ constexpr uint32_t idesc_f16_f32(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<__half2 *>(&v); }
__device__ __forceinline__ uint32_t half2_bits(__half2 v) { return *reinterpret_cast<uint32_t *>(&v); }

// The eight columns of a word as FP16 weights, in column order and in 9
// instructions: a code in the low bits of a half is that many times 2^-24, or
// 2^-20 four bits further up (so one shift serves the word), and one FMA takes it
// to (q - z) s, rounded once. s24 = 2^24 s and s20 = 2^20 s are exact, and so is
// minus_z = -z s for z <= 8, a product of 11 bits. With a zero point of 9 to 15 it
// would have 12, and a code equal to z would leave a weight of up to 2^-7 s: there
// every code is flipped, q' = 15 - q, z' = 15 - z, and (q' - z') (-s) is the same weight.
// The flip is part of the mask's instruction. For s24 to be an FP16 number, s lies below
// 2^-8, which the token's factor gives back. Below 2^-14 FP16's places are 2^-24
// wide: none is lost where s has its 8 bits above that.
constexpr float kTokenFactor = 512.f;
// (a ^ b) & c in one instruction: the compiler shares a ^ b among the masks, which costs one more a word.
__device__ __forceinline__ uint32_t flip_and_mask(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x28;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ void unpack_word(uint32_t word, uint32_t flip, __half2 s24, __half2 s20, __half2 minus_z, uint32_t *out)
{
    const uint32_t up = word >> 8;
    out[0] = half2_bits(__hfma2(as_half2(flip_and_mask(word, flip, 0x000f000fu)), s24, minus_z));
    out[1] = half2_bits(__hfma2(as_half2(flip_and_mask(word, flip, 0x00f000f0u)), s20, minus_z));
    out[2] = half2_bits(__hfma2(as_half2(flip_and_mask(up, flip, 0x000f000fu)), s24, minus_z));
    out[3] = half2_bits(__hfma2(as_half2(flip_and_mask(up, flip, 0x00f000f0u)), s20, minus_z));
}
// Four groups' zero points, one a byte, after the flips, and those: the top bit of each byte.
struct ZeroPoints {
    uint32_t z = 0x08080808u, flips = 0;
    __device__ __forceinline__ void set(uint32_t zeros)
    {
        z = zeros & 0x0f0f0f0fu;
        flips = z + 0x77777777u;
        z ^= ((flips >> 7) & 0x01010101u) * 15u;
    }
    __device__ __forceinline__ uint32_t flip(int gi) const        // that bit 32 times
    {
        uint32_t r;
        asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(flips), "r"(0x8888u + 0x1111u * gi));
        return r;
    }
    // of groups gi and gi + 1, at the top of two halves (other bits, too)
    __device__ __forceinline__ uint32_t signs(int gi) const { return __byte_perm(flips, 0, 0x1010 * gi + 0x1000); }
    __device__ __forceinline__ __half2 minus(int gi) const { return as_half2(__byte_perm(z, 0x80808080u, 0x4040u + 0x0101u * gi)); }      // -z 2^-24
};

// A few blocks' scales and zero points of a row, read at once: a load whose lanes
// read a row each takes 32 clocks of the load unit, however few
// bytes it brings (groups of 32, 1024 tokens: one load a block took 336 us, two
// blocks' at a time 308).
struct Scales {
    uint4 s;
    uint2 z;
};
// n (1, 2, 4 or 8) of them, of rows that start at multiples of n.
template <bool kZeros>
__device__ __forceinline__ Scales load_scales(const __nv_bfloat16 *s, const uint8_t *z, int n)
{
    Scales r{};
    if (n == 8) {                                 // (groups of 32)
        r.s = *reinterpret_cast<const uint4 *>(s);
        if (kZeros) r.z = *reinterpret_cast<const uint2 *>(z);
    } else if (n == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(s);
        r.s.x = v.x;
        r.s.y = v.y;
        if (kZeros) r.z.x = *reinterpret_cast<const uint32_t *>(z);
    } else if (n == 2) {
        r.s.x = *reinterpret_cast<const uint32_t *>(s);
        if (kZeros) r.z.x = *reinterpret_cast<const uint16_t *>(z);
    } else {
        r.s.x = *reinterpret_cast<const uint16_t *>(s);
        if (kZeros) r.z.x = *z;
    }
    return r;
}
// The first n of 2n taken off.
template <int n, bool kZeros>
__device__ __forceinline__ void next_scales(Scales &r)
{
    if constexpr (n == 4) {
        r.s.x = r.s.z;
        r.s.y = r.s.w;
        if (kZeros) r.z.x = r.z.y;
    } else if constexpr (n == 2) {
        r.s.x = r.s.y;
        if (kZeros) r.z.x >>= 16;
    }
}
// The largest magnitudes so far (two halves of 15 bits) with some scales' among them.
__device__ __forceinline__ uint32_t larger_scale(uint32_t top, uint4 s)
{
    return __vmaxu2(__vmaxu2(top, __vmaxu2(s.x & 0x7fff7fffu, s.y & 0x7fff7fffu)), __vmaxu2(s.z & 0x7fff7fffu, s.w & 0x7fff7fffu));
}
__device__ __forceinline__ uint32_t larger_half(uint32_t v) { return max(v & 0xffffu, v >> 16); }
// Exponent field of a magnitude's 15 bits: 1 to 254.
__device__ __forceinline__ uint32_t scale_field(uint32_t bits) { return min(max(bits >> 7, 1u), 254u); }
// 2^(127 - field) as FP32.
__device__ __forceinline__ float over_field(uint32_t field) { return __uint_as_float(field == 254u ? 0x00400000u : (254u - field) << 23); }

// This thread's row of M tile c of a unit, and its matrix.
template <bool kUp>
__device__ __forceinline__ size_t tile_row(const Args &a, const Unit &u, int c, int row)
{
    const int r = kUp ? u.tile * kRows + row : u.tile * 2 * kRows + c * kRows + row;
    return (u.grp >= a.p.E ? 0 : (size_t)u.grp * a.p.rows) + min(r, a.p.rows - 1);
}

// A row's weights are held over one power of two, its base: the one below the
// row's largest scale. A scale within 2^kSpread of that keeps its 8 bits above FP16's
// last place, 2^-24, and so does each |q - z| <= 8 times it. A row with a
// smaller scale is `wide`, which the unpacking warps see at the end of a unit: then every
// role leaves its units as if a wait had run out, and the CTA takes all of them
// again in the wide pass. There the base moves along the row: it is the power of
// two kRoom above the first groups' scales and serves those from its own
// down to kSpread below; for groups outside, the row's sums so far, FP32 numbers, are
// multiplied in tensor memory by the quotient of old base and new. A group whose codes are
// all z adds nothing, whatever its scale (the quantiser gives a group of zeros the
// scale 1), and is left out. A base stays within 2^-kFall of the highest so far, and the
// sums so within FP32's range. Where the groups of a block need a base each in one of the
// unit's rows, they go to the tensor core one by one.
// 1024 tokens, all rows with a block of zeros behind scales of 2^-11: 349 us, not 247, with
// groups of 128, 520, not 305, with groups of 32. Deciding unit by unit, with no second
// pass, cost the usual pass 5 to 15%: by registers in the unpacking warps, by the scales'
// latency in others.
constexpr uint32_t kSpread = 8, kRoom = 4, kFall = 96;

// The base's field of a row from some groups on, whose scales have fields low to
// high, at most kSpread apart; 0: none so far.
__device__ __forceinline__ uint32_t next_base(uint32_t base, uint32_t highest, uint32_t low, uint32_t high)
{
    if (base != 0 && high <= base && low + kSpread >= base) return base;
    return max(min((low + high) / 2 + kRoom, 254u), highest > kFall ? highest - kFall : 1u);
}

// A group's factors for unpack_word. scale: 2^24 s with s below 2^-8, that is 2^15
// times the scale over its row's base, negative where codes are flipped; minus: -z 2^-24.
struct GroupFactors {
    __half2 s24, s20, minus_z;
    __device__ __forceinline__ void set(__half2 scale, __half2 minus)
    {
        s24 = scale;
        s20 = __hmul2(s24, as_half2(0x2c002c00u));                    // 2^-4
        minus_z = __hmul2(s24, minus);
    }
};

// What an unpacking warp needs to know of a unit.
struct UnpackAt {
    const __nv_bfloat16 *sc, *sc_after;           // scales and zero points of this thread's row, and of the next unit's
    const uint8_t *zr, *zr_after, *codes;         // its codes in stage 0
    Scales ahead;                                 // of the first block; then of the next unit's
    uint32_t d, to;                               // its warp's sums of the unit and buffer 0 in tensor memory
    uint32_t it, step;                            // blocks and buffers so far
    int blocks, n;                                // n: the unit's tokens
    uint8_t *field;                               // where the result warps find its last base
};

// A unit of the wide pass. False in every lane of a warp whose wait gave up.
template <int G, bool kZeros>
__device__ __forceinline__ bool unpack_wide(Tail &T, Barriers &B, int *err, long long limit, UnpackAt &at)
{
    constexpr int GB = kW4Block / G;              // groups of a block
    const int lane = threadIdx.x & 31, swizzle = (lane >> 1) & 3;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_warp(bar, parity, &T.abort, err, limit); };
    uint32_t base = 0, highest = 0;               // exponent fields (0: none so far)
    for (int kb = 0; kb < at.blocks; ++kb, ++at.it) {
        const Scales now = at.ahead;
        if (kb + 1 < at.blocks) at.ahead = load_scales<kZeros>(at.sc + (kb + 1) * GB, at.zr + (kb + 1) * GB, GB);
        else at.ahead = load_scales<kZeros>(at.sc_after, at.zr_after, GB);
        const int st = at.it % kStages;
        if (!wait(&B.cfull[st], (at.it / kStages) & 1)) return false;
        uint4 w[4];                               // w[t]: words of columns 8t of each 32-column slice
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = *reinterpret_cast<const uint4 *>(at.codes + (size_t)st * 2 * kCodeTile + ((t ^ swizzle) << 4));
        uint32_t bits[GB], low = 255u, high = 0;  // scales, 0 where a group adds nothing; fields of the others
#pragma unroll
        for (int gi = 0; gi < GB; ++gi) {
            const uint32_t two = gi < 2 ? now.s.x : now.s.y, z = kZeros ? (now.z.x >> (8 * gi)) & 15u : 8u;
            uint32_t differ = 0;
#pragma unroll
            for (int jj = gi * (G / 32); jj < (gi + 1) * (G / 32); ++jj)
#pragma unroll
                for (int t = 0; t < 4; ++t) differ |= word_of(w[t], jj) ^ z * 0x11111111u;
            bits[gi] = differ == 0 ? 0u : gi & 1 ? two & 0xffff0000u : two << 16;
            if ((bits[gi] & 0x7fffffffu) == 0) continue;
            low = min(low, scale_field((bits[gi] & 0x7fffffffu) >> 16));
            high = max(high, scale_field((bits[gi] & 0x7fffffffu) >> 16));
        }
        bool split = false;                       // some row's groups need a base each
        if constexpr (GB > 1) {
            const bool mine = __any_sync(0xffffffffu, high > low + kSpread);
            if (lane == 0) {
                T.split[at.it & 7][(threadIdx.x >> 5) - 8] = mine;
                mbar_arrive(&T.vote);
            }
            if (!wait(&T.vote, at.it & 1)) return false;
            split = T.any_split(at.it);
        }
#pragma unroll 1
        for (int pass = 0; pass < (split ? GB : 1); ++pass, ++at.step) {
            const uint32_t ab = at.step & 1;
            if (split) {
                uint32_t f = 0;
#pragma unroll
                for (int gi = 0; gi < GB; ++gi) f = gi == pass ? bits[gi] & 0x7fffffffu : f;
                high = f ? scale_field(f >> 16) : 0u;
                low = f ? high : 255u;
            }
            const uint32_t next = high != 0 ? next_base(base, highest, low, high) : base;
            if (!wait(&B.aempty[ab], ((at.step >> 1) & 1) ^ 1)) return false;
            const bool moves = base != 0 && next != base;
            if (__any_sync(0xffffffffu, moves)) {
                // the MMAs of the step before, too, which is one of this unit
                if (!wait(&B.aempty[ab ^ 1], ((at.step - 1) >> 1) & 1)) return false;
                tc_fence_after();
                const int e = 127 + (int)base - (int)next;
                const float by = !moves ? 1.f : e > 0 ? __uint_as_float((uint32_t)e << 23) : 0.f;
#pragma unroll 1
                for (int t0 = 0; t0 < at.n; t0 += 16) {
                    uint32_t v[16];
                    tmem_ld16(at.d + t0, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * by);
                    tmem_st16(at.d + t0, v);
                }
            }
            tc_fence_after();
            base = next;
            highest = max(highest, base);
            ZeroPoints zp;
            if (kZeros) zp.set(now.z.x);
#pragma unroll
            for (int gi = 0; gi < GB; ++gi) {
                if (split && gi != pass) continue;
                const uint32_t flip = kZeros ? zp.flip(gi) : 0u;
                GroupFactors f;
                const float scale = bits[gi] ? __uint_as_float(bits[gi]) * over_field(base) * 0x1p15f : 0.f;
                f.set(__float2half2_rn(flip ? -scale : scale), zp.minus(gi));
#pragma unroll
                for (int jj = gi * (G / 32); jj < (gi + 1) * (G / 32); ++jj) {
                    uint32_t r[16];
#pragma unroll
                    for (int t = 0; t < 4; ++t) unpack_word(word_of(w[t], jj), flip, f.s24, f.s20, f.minus_z, r + 4 * t);
                    tmem_st16(at.to + ab * 64 + jj * 16, r);
                }
            }
            const bool last = !split || pass + 1 == GB;
            if (last && kb + 1 == at.blocks) *at.field = (uint8_t)max(base, 1u);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&B.afull[ab]);
                if (last) mbar_arrive(&B.cempty[st]);
            }
        }
    }
    return true;
}

// Tensor memory: sums of tile c in a slot, unpacked weights of tile c in a buffer.
__device__ __forceinline__ uint32_t d_col(int c, int slot) { return c * 128 + slot * 64; }
__device__ __forceinline__ uint32_t a_col(int c, int b) { return 256 + c * 128 + b * 64; }

// 32 rows (one per lane) by 16 tokens of results to y [token][row] in BF16. They
// turn in shared memory, two tokens a word, so that a lane stores 16 bytes of two
// tokens' rows: 4-byte stores, four times as many, took up to 300 clocks each. at:
// the first token's row of lane 0; left: rows from there to the end; n: tokens that
// are there.
__device__ __forceinline__ void store_turned(__nv_bfloat16 *at, int pitch, int left, int n, uint32_t *turn, const float (&o)[16])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 8; ++i) turn[i * 32 + lane] = as_u32(__floats2bfloat162_rn(o[2 * i], o[2 * i + 1]));
    __syncwarp();
    const int i = lane >> 2, r = (lane & 3) * 8;
    const uint4 a = *reinterpret_cast<const uint4 *>(turn + i * 32 + r), b = *reinterpret_cast<const uint4 *>(turn + i * 32 + r + 4);
    __syncwarp();                                 // read, before the next ones are written
    const uint32_t w[2][4] = {{__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410), __byte_perm(b.x, b.y, 0x5410), __byte_perm(b.z, b.w, 0x5410)},
                              {__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632), __byte_perm(b.x, b.y, 0x7632), __byte_perm(b.z, b.w, 0x7632)}};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        __nv_bfloat16 *dst = at + (size_t)(2 * i + h) * pitch + r;
        if (2 * i + h >= n) continue;
        if (r + 8 <= left && pitch % 8 == 0) {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(w[h][0], w[h][1], w[h][2], w[h][3]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (r + k < left) dst[k] = __ushort_as_bfloat16((unsigned short)(w[h][k >> 1] >> (16 * (k & 1))));
        }
    }
}

// Results of 16 tokens (n of them there) from both tiles' sums v0, v1. at: the
// first token's row r of y. All: every token is there and has an x row, and the rows'
// powers of two, whole then in row_scale[.][0], are within 2^+-100.
template <bool kUp, bool kAll, class YT>
__device__ __forceinline__ void store_step(const W4Product &p, YT *at, int r, int n, const float *tok, const float (&row_scale)[2][2],
                                           uint32_t *turn, const uint32_t (&v0)[16], const uint32_t (&v1)[16])
{
    float o0[16], o1[16];
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        const float4 f4 = *reinterpret_cast<const float4 *>(tok + i);
        const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            o0[i + k] = __uint_as_float(v0[i + k]) * row_scale[0][0] * f[k];
            o1[i + k] = __uint_as_float(v1[i + k]) * row_scale[1][0] * f[k];
            // (in halves: weights of 2^100 and tokens of 2^-100 must not meet infinity on the way)
            if (!kAll) o0[i + k] *= row_scale[0][1];
            if (!kAll) o1[i + k] *= row_scale[1][1];
            if (!kAll && f[k] == 0.f) o0[i + k] = o1[i + k] = 0.f;    // a token without an x row stands for zeros
        }
    }
    if constexpr (kUp) {
#pragma unroll
        for (int i = 0; i < 16; ++i) o0[i] = silu_mul(o0[i], o1[i]);
        if (r < p.rows)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (kAll || i < n) at[(size_t)i * p.rows] = o0[i];
    } else {
        const int lane = threadIdx.x & 31, left = p.rows - (r - lane);
        store_turned(at - lane, p.rows, left, n, turn, o0);
        store_turned(at - lane + kRows, p.rows, left - kRows, n, turn, o1);
    }
}

// Slots that units take in turn: a unit of up to 64 tokens takes the next one,
// a larger one both (the first of which is read, and free, first). `phase` holds, for each slot, the parity of its uses (the
// MMA warp's: it waits for every use of a slot).
struct Slots {
    uint32_t phase = 0;
    int next = 0, first = 0, n = 1;
    __device__ __forceinline__ void take(int tokens)
    {
        n = tokens > 64 ? 2 : 1;
        first = n == 2 ? 0 : next;
        next = n == 1 ? first ^ 1 : 0;
    }
    __device__ __forceinline__ uint32_t parity(int slot) const { return (phase >> slot) & 1; }
    __device__ __forceinline__ void done() { phase ^= n == 2 ? 3u : 1u << first; }
};

template <int N>
using Const = std::integral_constant<int, N>;

// Every unit of this CTA, by roles of its warps; kWide: in the wide pass.
template <bool kUp, int G, bool kZeros, class YT, bool kWide>
__device__ __forceinline__ void run_units(const Maps &maps, const Args &a, Tail &T, uint8_t *codes, uint8_t *toks)
{
    constexpr int GB = kW4Block / G;
    const W4Product &p = a.p;
    Barriers &B = T.bars[kWide];
    volatile int *abort = &T.abort;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);    // known to be uniform
    const int lane = threadIdx.x & 31, blocks = p.cols / kW4Block;
    const int total = T.total;
    const uint32_t tmem = T.tmem_base;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_warp(bar, parity, abort, a.err, a.wait_limit); };

    if (warp == kLoadWarp) {
        // ---------------------------------------------------------- loads
        const uint64_t pol_w = policy_evict_first();
        uint32_t it = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
            const Unit U = unit_of(a, T, u);
            const bool shared = U.grp >= p.E;
            const int y0 = (shared ? 0 : U.grp * p.rows) + (kUp ? U.tile * kRows : U.tile * 2 * kRows);
            const int y1 = kUp ? y0 : y0 + kRows;
            // The next unit's scales and zero points, whose rows the unpackers read a few
            // bytes at a time, and each 32 bytes anew from memory otherwise.
            if (u + (int)gridDim.x < total) {
                const Unit V = unit_of(a, T, u + gridDim.x);
                const bool vs = V.grp >= p.E;
                const int r0 = V.tile * (kUp ? 1 : 2) * kRows, n = min(p.rows - r0, (kUp ? 1 : 2) * kRows), gpr = p.cols / G;
                const size_t at = ((vs ? 0 : (size_t)V.grp * p.rows) + r0) * gpr;
                if (elect_one()) {
                    prefetch_l2((vs ? p.w_shared.s : p.w.s) + at, (size_t)n * gpr * 2);
                    if (kUp) prefetch_l2((vs ? p.up_shared.s : p.up.s) + at, (size_t)n * gpr * 2);
                    if (kZeros) prefetch_l2((vs ? p.w_shared.z : p.w.z) + at, (size_t)n * gpr);
                    if (kZeros && kUp) prefetch_l2((vs ? p.up_shared.z : p.up.z) + at, (size_t)n * gpr);
                }
                __syncwarp();
            }
            const CUtensorMap *m0 = shared ? &maps.w_shared[0] : &maps.w[0], *m1 = shared ? &maps.w_shared[1] : &maps.w[1];
            for (int kb = 0; kb < blocks; ++kb, ++it) {
                const int s = it % kStages;
                ok = wait(&B.cempty[s], ((it / kStages) & 1) ^ 1);
                if (!ok) break;
                uint8_t *C = codes + (size_t)s * 2 * kCodeTile;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&B.cfull[s], 2 * kCodeTile);
                    tma_load_2d_hint(C, m0, &B.cfull[s], kb * 64, y0, pol_w);
                    tma_load_2d_hint(C + kCodeTile, m1, &B.cfull[s], kb * 64, y1, pol_w);
                }
                __syncwarp();
            }
        }
        // let loads in flight land, whichever role has left its units
        for (uint32_t j = it > (uint32_t)kStages ? it - kStages : 0; j < it; ++j)
            mbar_wait_drain(&B.cfull[j % kStages], (j / kStages) & 1, kDefaultWaitLimit);
    } else if (warp >= kGatherWarp) {
        // --------------------------------------------------------- gather
        // 16 threads take the 256 bytes of a row's 128 columns: warp w the rows
        // 4j + 2w and the next one. Lane k holds where the k-th and the (32 + k)-th
        // of the warp's rows start and hands them out: held by every thread for
        // itself, 32 places and a copy each were unrolled, and the fetching of
        // those instructions took 60 clocks a copy.
        const int w = warp - kGatherWarp, piece = lane & 15, second = lane >> 4, r8 = 2 * w + second;
        const uint32_t panel = (uint32_t)(piece >> 3) * kPanel;
        uint32_t it = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
            const Unit U = unit_of(a, T, u);
            const bool shared = U.grp >= p.E;
            // x rows, in 16-byte pieces from x; row 0 for tokens that are not there (their results are not used)
            uint32_t row[2];
            const uint32_t pieces = (uint32_t)(a.x_pitch >> 4);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = 32 * h + lane, i = 4 * (k >> 1) + 2 * w + (k & 1);
                int xi = 0;
                if (i < U.n) {
                    xi = U.row0 + i;
                    if (!p.x_by_row) xi = shared ? xi - p.P : p.perm ? p.perm[xi] : xi;
                    if ((unsigned)xi >= (unsigned)p.x_rows) xi = 0;
                }
                row[h] = (uint32_t)xi * pieces;
            }
            const int passes = (U.n + 3) / 4;
            for (int kb = 0; kb < blocks; ++kb, ++it) {
                const int s = it % kStages;
                ok = wait(&B.bempty[s], ((it / kStages) & 1) ^ 1);
                if (!ok) break;
                const uint32_t dst = smem_u32(toks) + s * 2 * kPanel + panel + r8 * 128;
                // the swizzle takes the row's low three bits: 4 (j & 1) + r8
                const uint32_t dst0 = dst + (((piece & 7) ^ r8) << 4), dst1 = dst + (((piece & 7) ^ (4 + r8)) << 4);
                const uint4 *src = static_cast<const uint4 *>(a.x16) + kb * (kW4Block * 2 / 16) + piece;
#pragma unroll 1
                for (int j0 = 0; j0 < passes; j0 += 8) {
                    const uint32_t held = j0 < 16 ? row[0] : row[1];
                    uint32_t from[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) from[j] = __shfl_sync(0xffffffffu, held, (2 * (j0 + j) + second) & 31);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j0 + j < passes) cp_async16((j & 1 ? dst1 : dst0) + (j0 + j) * 512, src + from[j], 16);
                }
                cp_async_arrive_noinc(&B.bfull[s]);       // once this thread's copies have landed
            }
        }
        cp_async_wait_all();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA
        // The whole warp walks; one elected lane issues. Kept converged, the
        // descriptors live in uniform registers and an MMA costs 11 clocks at 16
        // tokens; issued under `lane == 0` each took 170.
        uint32_t it = 0, step = 0;                // step: buffers
        Slots sl;
        bool ok = true;
        for (int u = blockIdx.x, turn = 0; u < total && ok; u += gridDim.x, turn ^= 1) {
            const Unit U = unit_of(a, T, u);
            const uint32_t idesc = idesc_f16_f32(kRows, (U.n + 15) & ~15);
            sl.take(U.n);
            for (int k = 0; k < sl.n; ++k) ok = ok && wait(&B.dempty[sl.first + k], sl.parity(sl.first + k) ^ 1);
            for (int kb = 0; kb < blocks && ok; ++kb, ++it) {
                const int s = it % kStages;
                ok = wait(&B.bfull[s], (it / kStages) & 1);
                // a buffer holds a block, in the wide pass sometimes one group of it
                int passes = 1;
#pragma unroll 1
                for (int g = 0; g < passes && ok; ++g, ++step) {
                    const int ab = step & 1;
                    ok = wait(&B.afull[ab], (step >> 1) & 1);
                    if (!ok) break;
                    if (kWide && GB > 1 && g == 0 && __shfl_sync(0xffffffffu, (int)T.any_split(it), 0)) passes = GB;
                    fence_proxy_async();          // the gathered rows, for the tensor core
                    tc_fence_after();
                    const uint32_t b0 = smem_u32(toks) + s * 2 * kPanel;
                    const uint64_t bd0 = sw128_kmajor_desc(b0), bd1 = sw128_kmajor_desc(b0 + kPanel);
                    // 16 columns each of both tiles, from the k0-th on
                    auto issue = [&](auto k0, auto n) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t dt = tmem + d_col(c, sl.first), at = tmem + a_col(c, ab);
#pragma unroll
                            for (int k = k0.value; k < k0.value + n.value; ++k)
                                umma_f16_ts(dt, at + k * 8, (k < 4 ? bd0 : bd1) + (uint64_t)((k & 3) * 2), idesc, (kb | k) != 0);
                        }
                    };
                    if (elect_one()) {
                        constexpr int kAll = kW4Block / 16, kOne = G / 16;
                        if (!kWide || passes == 1) issue(Const<0>{}, Const<kAll>{});
                        else if (g == 0) issue(Const<0>{}, Const<kOne>{});
                        else if (g == 1) issue(Const<kOne % kAll>{}, Const<kOne>{});
                        else if (g == 2) issue(Const<2 * kOne % kAll>{}, Const<kOne>{});
                        else issue(Const<3 * kOne % kAll>{}, Const<kOne>{});
                        umma_commit(&B.aempty[ab]);
                        if (g + 1 == passes) umma_commit(&B.bempty[s]);
                        if (g + 1 == passes && kb + 1 == blocks) umma_commit(&B.dfull[turn]);
                    }
                    __syncwarp();
                }
            }
            sl.done();
        }
        if (elect_one()) umma_commit(&B.drain);   // every MMA done before tensor memory is released
        __syncwarp();
        mbar_wait_drain(&B.drain, 0, kDefaultWaitLimit);
        __syncwarp();
    } else if (kWide && warp >= 8) {
        // ---------------------------------------------------- unpack, wide
        const int c = (warp - 8) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        uint32_t nth = 0;
        Slots sl;
        UnpackAt at{};
        at.codes = codes + c * kCodeTile + row * 64;
        at.to = lanes + a_col(c, 0);
        at.blocks = blocks;
        auto rows_of = [&](int u) {
            const Unit U = unit_of(a, T, u);
            const bool shared = U.grp >= p.E;
            const size_t first = tile_row<kUp>(a, U, c, row) * (p.cols / G);
            at.sc_after = (kUp && c ? (shared ? p.up_shared.s : p.up.s) : (shared ? p.w_shared.s : p.w.s)) + first;
            if (kZeros) at.zr_after = (kUp && c ? (shared ? p.up_shared.z : p.up.z) : (shared ? p.w_shared.z : p.w.z)) + first;
        };
        if (blockIdx.x < total) {
            rows_of(blockIdx.x);
            at.ahead = load_scales<kZeros>(at.sc_after, at.zr_after, GB);
        }
        for (int u = blockIdx.x; u < total; u += gridDim.x, ++nth) {
            at.sc = at.sc_after;
            at.zr = at.zr_after;
            at.n = unit_of(a, T, u).n;
            at.field = &T.field[nth & 3][c][row];
            sl.take(at.n);
            at.d = lanes + d_col(c, sl.first);
            if (u + (int)gridDim.x < total) rows_of(u + gridDim.x);
            if (!unpack_wide<G, kZeros>(T, B, a.err, a.wait_limit, at)) break;
        }
    } else if (warp >= 8) {
        // --------------------------------------------------------- unpack
        const int c = (warp - 8) >> 2, row = (warp & 3) * 32 + lane, gpr = p.cols / G;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        uint32_t it = 0, nth = 0;
        bool ok = true;
        const __nv_bfloat16 *sc = nullptr, *sc_after = nullptr;      // this unit's scales and the next one's
        const uint8_t *zr = nullptr, *zr_after = nullptr;
        auto rows_of = [&](int u) {
            const Unit U = unit_of(a, T, u);
            const bool shared = U.grp >= p.E;
            const size_t at = tile_row<kUp>(a, U, c, row) * gpr;
            sc_after = (kUp && c ? (shared ? p.up_shared.s : p.up.s) : (shared ? p.w_shared.s : p.w.s)) + at;
            if (kZeros) zr_after = (kUp && c ? (shared ? p.up_shared.z : p.up.z) : (shared ? p.w_shared.z : p.w.z)) + at;
        };
        // Scales at a time: two blocks' where every row is aligned to that. (One scale a
        // block is read alone: four at a time took 255 us for 1024 tokens, not 246.)
        const int n_blocks = GB > 1 && blocks % 2 == 0 ? 2 : 1, n_scales = n_blocks * GB;
        uint32_t top = 0;                         // of the next unit's scales, read along with this one's
        Scales now{}, later{};                    // at work, and read ahead
        uint4 s_after{};                          // of the next unit, for `top`
        if (blockIdx.x < total) {
            rows_of(blockIdx.x);
            for (int kb = 0; kb < blocks; kb += n_blocks) top = larger_scale(top, load_scales<false>(sc_after + kb * GB, nullptr, n_scales).s);
            later = load_scales<kZeros>(sc_after, zr_after, n_scales);
        }
        for (int u = blockIdx.x; u < total && ok; u += gridDim.x, ++nth) {
            // scales over the power of two below the row's largest: 2^(127 - field) as FP32
            const uint32_t field = scale_field(larger_half(top));
            const uint32_t to_half = (30u - field) * (128u * 0x00010001u);
            uint32_t low = GB == 1 ? 0x7fffu : 0x7fff7fffu;           // the smallest magnitudes
            sc = sc_after;
            zr = zr_after;
            const bool more = u + (int)gridDim.x < total;
            if (more) rows_of(u + gridDim.x);
            top = 0;
            s_after = make_uint4(0u, 0u, 0u, 0u);
            for (int kb = 0; kb < blocks; ++kb, ++it) {
                const int st = it % kStages, ab = it & 1;
                if ((kb & (n_blocks - 1)) == 0) {
                    const int ahead = kb + n_blocks;
                    now = later;
                    if (ahead < blocks) later = load_scales<kZeros>(sc + ahead * GB, zr + ahead * GB, n_scales);
                    else if (more) later = load_scales<kZeros>(sc_after, zr_after, n_scales);
                    top = larger_scale(top, s_after);
                    if (more) s_after = load_scales<false>(sc_after + kb * GB, nullptr, n_scales).s;
                }
                GroupFactors fac[GB];
                ZeroPoints zp;
                if (kZeros) zp.set(now.z.x);
#pragma unroll
                for (int gi = 0; gi < GB; gi += 2) {
                    const uint32_t two = gi < 2 ? now.s.x : now.s.y, size = two & 0x7fff7fffu;
                    low = GB == 1 ? min(low, size) : __vminu2(low, size);
                    // 2^15 over the base, for two scales at once: exponents in FP16's field
                    const uint32_t half2 = (size + to_half) << 3, sign = two ^ (kZeros ? zp.signs(gi) : 0u);
                    const uint32_t both = half2 | (sign & 0x80008000u);
                    fac[gi].set(as_half2(__byte_perm(both, 0, 0x1010)), zp.minus(gi));
                    if (gi + 1 < GB) fac[gi + 1].set(as_half2(__byte_perm(both, 0, 0x3232)), zp.minus(gi + 1));
                }
                next_scales<GB, kZeros>(now);
                ok = wait(&B.cfull[st], (it / kStages) & 1);
                if (!ok) break;
                const uint8_t *src = codes + (size_t)st * 2 * kCodeTile + c * kCodeTile + row * 64;
                uint4 w[4];                       // w[t]: words of columns 8t of each 32-column slice
#pragma unroll
                for (int t = 0; t < 4; ++t) w[t] = *reinterpret_cast<const uint4 *>(src + ((t ^ ((row >> 1) & 3)) << 4));
                ok = wait(&B.aempty[ab], ((it >> 1) & 1) ^ 1);
                if (!ok) break;
                tc_fence_after();
                // for the results. The block two before is done, so at the earliest the
                // last unit but one, whose sums took the place of the last but three's.
                if (kb == 0) T.field[nth & 3][c][row] = (uint8_t)field;
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {  // 32 columns: 16 columns of tensor memory
                    const int gi = jj / (G / 32);
                    uint32_t r[16];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        unpack_word(word_of(w[t], jj), kZeros ? zp.flip(gi) : 0u, fac[gi].s24, fac[gi].s20, fac[gi].minus_z, r + 4 * t);
                    tmem_st16(tmem + lanes + a_col(c, ab) + jj * 16, r);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&B.afull[ab]);
                    mbar_arrive(&B.cempty[st]);
                }
            }
            top = larger_scale(top, s_after);
            // scales that are wide, or 0 or below 2^-126, whose exponents the addition did not take right
            const uint32_t least = (GB == 1 ? low : min(low & 0xffffu, low >> 16)) >> 7;
            if (__any_sync(0xffffffffu, least == 0 || field > least + kSpread)) {
                *abort = kStartAnew;
                break;                            // (the others run out of work then, and look)
            }
        }
    } else {
        // -------------------------------------------------------- results
        const int half = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        // Units take turns in two barriers: a unit's sums can be complete before the
        // last one's are read, but the next but one's cannot, since three units
        // never fit into two slots.
        Slots sl;
        uint32_t nth = 0;
        bool ok = true;
        float f_after[kTokens / 32];              // the next unit's tokens' powers of two; 0 for one without an x row
        auto factors_of = [&](int u) {
            const Unit U = unit_of(a, T, u);
#pragma unroll
            for (int j = 0; j < kTokens / 32; ++j) {
                const int i = lane + 32 * j;
                int xi = 0;
                if (i < U.n) {
                    xi = U.row0 + i;
                    if (!p.x_by_row) xi = U.grp >= p.E ? xi - p.P : p.perm ? p.perm[xi] : xi;
                }
                f_after[j] = (unsigned)xi < (unsigned)p.x_rows ? a.x_scale[xi] : 0.f;
            }
        };
        if (blockIdx.x < total) factors_of(blockIdx.x);
        for (int u = blockIdx.x; u < total && ok; u += gridDim.x, ++nth) {
            const Unit U = unit_of(a, T, u);
            const bool shared = U.grp >= p.E;
            sl.take(U.n);
            float *tok = T.tok[warp];             // 0 for a token that is not there
            bool there = !kWide;                  // nothing out of the ordinary
#pragma unroll
            for (int j = 0; j < kTokens / 32; ++j) {
                tok[lane + 32 * j] = f_after[j] * kTokenFactor;
                there = there && f_after[j] != 0.f;
            }
            __syncwarp();
            if (u + (int)gridDim.x < total) factors_of(u + gridDim.x);
            ok = wait(&B.dfull[nth & 1], (nth >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            float row_scale[2][2];                // the rows' powers of two, halved
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint32_t field = T.field[nth & 3][c][row], half = (field + 127u) >> 1;
                there = there && field >= 27u && field <= 227u;
                row_scale[c][0] = __uint_as_float(half << 23);
                row_scale[c][1] = __uint_as_float((field + 127u - half) << 23);
            }
            there = __all_sync(0xffffffffu, there);
            float row_whole[2][2] = {{row_scale[0][0] * row_scale[0][1]}, {row_scale[1][0] * row_scale[1][1]}};
            YT *y = !kUp && shared ? static_cast<YT *>(p.y_shared) + (size_t)(U.row0 - p.P) * p.rows
                                   : static_cast<YT *>(p.y) + (size_t)U.row0 * p.rows;
            const int r = kUp ? U.tile * kRows + row : U.tile * 2 * kRows + row;
            auto release = [&](int slot) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.dempty[slot]);
            };
            // a group without a step in it leaves the last slot at once (the first one of two never)
            if (U.n - (sl.n - 1) * 64 <= 16 * half) release(sl.first + sl.n - 1);
            for (int t0 = 16 * half; t0 < U.n; t0 += 32) {
                uint32_t v0[16], v1[16];
                tmem_ld16(tmem + lanes + d_col(0, sl.first) + t0, v0);
                tmem_ld16(tmem + lanes + d_col(1, sl.first) + t0, v1);
                tmem_ld_wait();
                // the slot's last step is in registers
                if (t0 + 32 >= U.n || (t0 & 32)) release(sl.first + (t0 >> 6));
                // a whole step of tokens that are all there has no branch in it
                if (t0 + 16 <= U.n && there)
                    store_step<kUp, true>(p, y + (size_t)t0 * p.rows + r, r, 16, tok + t0, row_whole, T.turn[warp], v0, v1);
                else
                    store_step<kUp, false>(p, y + (size_t)t0 * p.rows + r, r, U.n - t0, tok + t0, row_scale, T.turn[warp], v0, v1);
            }
            __syncwarp();                         // tok is read
        }
    }
}

__device__ __forceinline__ void init_barriers(Barriers &B)
{
    for (int s = 0; s < kStages; ++s) {
        mbar_init(&B.cfull[s], 1);
        mbar_init(&B.cempty[s], 8);               // one arrival per unpacking warp
        mbar_init(&B.bfull[s], kGatherThreads);
        mbar_init(&B.bempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
        mbar_init(&B.afull[b], 8);                // one arrival per unpacking warp
        mbar_init(&B.aempty[b], 1);
        mbar_init(&B.dfull[b], 1);
        mbar_init(&B.dempty[b], 8);               // one arrival per result warp
    }
    mbar_init(&B.drain, 1);
}

template <bool kUp, int G, bool kZeros, class YT>
__global__ void __launch_bounds__(kThreads, 1)
w4_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *codes = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *toks = codes + (size_t)kStages * 2 * kCodeTile;
    Tail &T = *reinterpret_cast<Tail *>(toks + (size_t)kStages * 2 * kPanel);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);    // known to be uniform
    if (threadIdx.x == 0) {
        init_barriers(T.bars[0]);
        T.abort = kGoOn;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&T.tmem_base, 512);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();
    tc_fence_before();
    build_tables(a, T);                           // its barriers also publish the mbarriers and the allocation
    tc_fence_after();
    run_units<kUp, G, kZeros, YT, false>(maps, a, T, codes, toks);
    tc_fence_before();
    __syncthreads();
    if (T.abort == kStartAnew) {
        tc_fence_after();
        __syncthreads();
        if (threadIdx.x == 0) {
            init_barriers(T.bars[1]);
            mbar_init(&T.vote, 8);
            T.abort = kGoOn;
            fence_mbar_init();
        }
        __syncthreads();
        run_units<kUp, G, kZeros, YT, true>(maps, a, T, codes, toks);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(T.tmem_base, 512);
    }
}

// ------------------------------------------------------------------- host
static PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *q = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &q, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(q);
    }
    return fn;
}

// Codes [rows, bytes] as boxes of 128 rows x 64 bytes, 64-byte swizzle; rows
// behind the last read as zeros.
static bool make_map(CUtensorMap *m, const void *base, uint64_t rows, uint64_t bytes)
{
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {bytes, rows};
    cuuint64_t strides[1] = {bytes};
    cuuint32_t box[2] = {64, kRows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kUp, int G, bool kZeros, class YT>
static kmoe_status run(const Maps &maps, const Args &a, int grid, cudaStream_t st)
{
    cudaFuncSetAttribute(w4_tc_kernel<kUp, G, kZeros, YT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    launch_pdl(w4_tc_kernel<kUp, G, kZeros, YT>, grid, kThreads, kSmem, st, maps, a);
    return check_launch("w4_tc");
}

template <bool kUp, class YT>
static kmoe_status pick(const Maps &m, const Args &a, int grid, cudaStream_t st)
{
    const bool z = a.p.w.z != nullptr;
    switch (a.p.group) {
    case 32: return z ? run<kUp, 32, true, YT>(m, a, grid, st) : run<kUp, 32, false, YT>(m, a, grid, st);
    case 64: return z ? run<kUp, 64, true, YT>(m, a, grid, st) : run<kUp, 64, false, YT>(m, a, grid, st);
    default: return z ? run<kUp, 128, true, YT>(m, a, grid, st) : run<kUp, 128, false, YT>(m, a, grid, st);
    }
}

}  // namespace w4tc

// x (BF16 or FP32) in FP16 over a power of two per row: the largest magnitude
// of a row lies in [2^14, 2^15). One warp per row, two passes (the second reads
// L1). `out` may start where x starts, with rows the same bytes apart (H, FP32):
// a step's values are read before any of its results is written.
template <class XT>
__global__ void __launch_bounds__(256) to_f16_kernel(const XT *x, int rows, int cols, __half *out, size_t out_pitch, float *scale, int *status)
{
    pdl_wait();
    pdl_trigger();
    // here, not in the products' launch, whose CTAs may report in it before its first one starts
    if (status && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
    const int lane = threadIdx.x & 31, row = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const XT *src = x + (size_t)row * cols;
    uint32_t top = 0;
    for (int c = lane * 8; c < cols; c += 256) {
        float v[8];
        load8(src + c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const uint32_t ex = max(top >> 23, 15u);      // a row below 2^-112 stays at that scale
    const float mul = __uint_as_float((268u - ex) << 23);             // 2^(14 - E)
    __half *dst = out + (size_t)row * out_pitch;
    for (int c0 = 0; c0 < cols; c0 += 256) {
        const int c = c0 + lane * 8;
        float v[8];
        if (c < cols) load8(src + c, v);
        __syncwarp();
        if (c < cols) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 h = __floats2half2_rn(v[2 * i] * mul, v[2 * i + 1] * mul);
                o[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
            *reinterpret_cast<uint4 *>(dst + c) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        __syncwarp();
    }
    if (lane == 0) scale[row] = __uint_as_float((ex - 14u) << 23);
}

kmoe_status launch_w4_tc(const W4Product &p, void *x16, float *x_scale, int *err, long long wait_limit, cudaStream_t st)
{
    using namespace w4tc;
    Args a{};
    a.x16 = x16;
    a.x_pitch = (size_t)p.cols * (p.x_f32 ? 4 : 2);
    a.x_scale = x_scale;
    const int x_grid = (p.x_rows + 7) / 8;
    __half *out = static_cast<__half *>(x16);
    if (p.x_f32) launch_pdl(to_f16_kernel<float>, x_grid, 256, 0, st, static_cast<const float *>(p.x), p.x_rows, p.cols, out, (size_t)p.cols * 2, x_scale, p.status);
    else launch_pdl(to_f16_kernel<__nv_bfloat16>, x_grid, 256, 0, st, static_cast<const __nv_bfloat16 *>(p.x), p.x_rows, p.cols, out, (size_t)p.cols, x_scale, p.status);
    const kmoe_status conv = check_launch("to_f16");
    if (conv != KMOE_OK) return conv;
    a.p = p;
    a.check = may_overflow(p, kTokens);
    a.groups = p.E + (p.n_shared > 0 ? 1 : 0);
    if (a.groups > kMaxGroups) return fail(KMOE_ERR_UNSUPPORTED, "4-bit products: too many experts");
    const bool up = p.up.q != nullptr;
    const int unit_rows = up ? kRows : 2 * kRows;
    a.tiles = (p.rows + unit_rows - 1) / unit_rows;
    a.by_tiles = DivideBy::make(a.tiles);
    a.err = err;
    a.wait_limit = wait_limit;
    Maps m{};
    const uint64_t bytes = (uint64_t)p.cols / 2;
    auto codes = [&](CUtensorMap *map, const W4Ptrs &w, uint64_t rows) {
        return make_map(map, w.q, rows, bytes);
    };
    const bool shared = p.n_shared > 0;
    const uint64_t all_rows = (uint64_t)p.E * p.rows;
    const W4Ptrs &w1 = up ? p.up : p.w, &s0 = shared ? p.w_shared : p.w, &s1 = shared ? (up ? p.up_shared : p.w_shared) : w1;
    const bool ok = codes(&m.w[0], p.w, all_rows) && codes(&m.w[1], w1, all_rows) && codes(&m.w_shared[0], s0, p.rows) &&
                    codes(&m.w_shared[1], s1, p.rows);
    if (!ok) return fail(KMOE_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const long long most = ((long long)std::min(p.E, p.P) + (p.P + p.n_shared) / 64 + 1) * a.tiles;
    const int grid = (int)std::min<long long>(sms, most);
    return up ? pick<true, float>(m, a, grid, st) : pick<false, __nv_bfloat16>(m, a, grid, st);
}

}  // namespace kmoe
