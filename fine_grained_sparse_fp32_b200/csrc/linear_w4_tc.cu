// Products with 4-bit weights on the 5th-generation tensor cores, for batches
// whose experts see several tokens (linear_w4.cu is the kernel for few).
//
//   y[p][r] = sum_G s[r][G] * ( sum_{c in G} (q[r][c] - z[r][G]) x[p][c] )
// Weights are the M operand (128 rows), tokens the N operand (up to 64). A
// code minus its zero point is a whole number below 16 in magnitude, exact in
// BF16, so the weights are never rounded: the tensor cores sum one group's
// products of BF16 codes and BF16 x in FP32, and the group scale, which belongs
// to a row and so to one thread's lane of tensor memory, multiplies that sum as
// it is added up in registers.
//
// Unpacking bounds this kernel (1.4 instructions a weight on the integer pipe),
// so a CTA unpacks a weight once for up to 64 tokens, and unpacked weights take
// no shared-memory bandwidth: the unpacking threads write them straight into
// tensor memory, from where the MMA reads its A operand. A unit is two M tiles
// (256 rows of one expert, or 128 gate and the same 128 up features) and a
// block of tokens; the tiles' phases alternate, so one is unpacked and added up
// while the MMA works on the other. Units are dealt to the CTAs (one per SM)
// in turn.
//   warps 0-7    add up: tcgen05.ld of a group's sums, times the scale
//                (warps 0-3 tile 0, 4-7 tile 1); SiLU(gate) * up or the output
//   warps 8-15   unpack: 64 bytes of codes of a row and 128 columns into 64
//                columns of tensor memory (8-11 tile 0, 12-15 tile 1)
//   warp 16      loads code tiles by TMA (64-byte swizzle: the unpackers' reads
//                have no bank conflicts)
//   warp 17      issues tcgen05.mma
//   warps 18-19  gather token rows with cp.async (a TMA gather of four rows
//                costs its issuer 80 clocks: 32 of them for 64 tokens and 128
//                columns bounded the kernel)
// Tensor memory: sums 2 tiles x 2 buffers x 64 columns, unpacked weights
// 2 tiles x 2 buffers x 64 columns.
#include "sm100.cuh"
#include "swap_units.cuh"
#include "w4.cuh"

#include <cudaTypedefs.h>

#include <algorithm>

namespace kmoe {
using namespace sm100;

namespace w4tc {

constexpr int kThreads = 20 * 32;
constexpr int kTokens = 64;                       // tokens of a unit
constexpr int kRows = 128;                        // rows of an M tile
constexpr int kCodeTile = kRows * 64;             // bytes of one tile's codes of a 128-column block
constexpr int kPanel = kTokens * 128;             // bytes of 64 columns of a token block
constexpr int kStages = 4;                        // 128-column blocks in flight: codes 16 KB, tokens 16 KB each
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
    int *err;
    long long wait_limit;
};

struct Tail {
    uint64_t cfull[kStages], cempty[kStages], bfull[kStages], bempty[kStages];
    uint64_t afull[2][2], aempty[2][2], dfull[2][2], dempty[2][2], up_full, up_empty, drain;
    uint32_t tmem_base;
    int abort, total;
    int pre[kMaxGroups + 1], start[kMaxGroups], count[kMaxGroups], size[kMaxGroups];   // size: tokens of a block
    uint16_t known[kKnown];
};
constexpr size_t kSmem = 1024 + (size_t)kStages * (2 * kCodeTile + 2 * kPanel) + sizeof(Tail);

struct Unit {
    int grp, row0, n, tile;
};

__device__ __forceinline__ Unit unit_of(const Args &a, const Tail &T, int u)
{
    const int tb = a.by_tiles(u), g = tb < kKnown ? T.known[tb] : last_not_above(T.pre, a.groups, tb);
    const int first = (tb - T.pre[g]) * T.size[g];
    return {g, T.start[g] + first, min(T.size[g], T.count[g] - first), u - tb * a.tiles};
}

// Tokens of a block of a group with `count` rows: equal blocks of at most 64.
__device__ __forceinline__ int block_size(int count)
{
    const int n = (count + kTokens - 1) / kTokens;
    return n > 1 ? (((count + n - 1) / n) + 3) & ~3 : kTokens;
}

// Tables of the groups; one warp adds up the blocks.
__device__ __forceinline__ void build_tables(const Args &a, Tail &T)
{
    for (int g = threadIdx.x; g < a.groups; g += kThreads) {
        int start, count;
        group_rows(a.p, g, &start, &count);
        T.start[g] = start;
        T.count[g] = count;
        T.size[g] = block_size(count);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int run = 0;
        for (int g0 = 0; g0 < a.groups; g0 += 32) {
            const int g = g0 + threadIdx.x;
            const int n = g < a.groups ? (T.count[g] + T.size[g] - 1) / T.size[g] : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if ((int)threadIdx.x >= o) incl += v;
            }
            const int before = run + incl - n;
            if (g < a.groups) {
                T.pre[g] = before;
                for (int k = before; k < min(before + n, kKnown); ++k) T.known[k] = g;
            }
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (threadIdx.x == 0) {
            T.pre[a.groups] = run;
            // ranges that overlap (which no dispatch makes) could count beyond the units' 32 bits: then nothing is done
            T.total = (long long)run * a.tiles < 0x7fffffffLL ? run * a.tiles : 0;
        }
    }
    __syncthreads();
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, BF16 inputs, FP32 accumulation.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
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

// {128 + z, 128 + z} in BF16 (the low mantissa bits of 128.0 count ones).
__device__ __forceinline__ __nv_bfloat162 zero_pair(uint32_t z)
{
    const uint32_t v = (0x4300u | z) * 0x00010001u;
    return *reinterpret_cast<const __nv_bfloat162 *>(&v);
}
// Columns 2i, 2i + 1 of a word as BF16 q - z: 128 + q (the code as mantissa
// bits), minus 128 + z; exact.
__device__ __forceinline__ uint32_t code_pair(uint32_t word, int i, __nv_bfloat162 zz)
{
    const uint32_t v = ((word >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    return as_u32(__hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), zz));
}

// This thread's row of M tile c of a unit, and its matrix.
template <bool kUp>
__device__ __forceinline__ size_t tile_row(const Args &a, const Unit &u, int c, int row)
{
    const int r = kUp ? u.tile * kRows + row : u.tile * 2 * kRows + c * kRows + row;
    return (u.grp >= a.p.E ? 0 : (size_t)u.grp * a.p.rows) + min(r, a.p.rows - 1);
}

template <bool kUp, int G, bool kZeros, class YT>
__global__ void __launch_bounds__(kThreads, 1)
kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a)
{
    constexpr int GB = kW4Block / G;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *codes = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *toks = codes + (size_t)kStages * 2 * kCodeTile;
    Tail &T = *reinterpret_cast<Tail *>(toks + (size_t)kStages * 2 * kPanel);
    volatile int *abort = &T.abort;
    const W4Product &p = a.p;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);    // known to be uniform
    const int lane = threadIdx.x & 31, blocks = p.cols / kW4Block;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&T.cfull[s], 1);
            mbar_init(&T.cempty[s], 8);           // one arrival per unpacking warp
            mbar_init(&T.bfull[s], kGatherThreads);
            mbar_init(&T.bempty[s], 1);
        }
        for (int c = 0; c < 2; ++c)
            for (int b = 0; b < 2; ++b) {
                mbar_init(&T.afull[c][b], 4);
                mbar_init(&T.aempty[c][b], 1);
                mbar_init(&T.dfull[c][b], 1);
                mbar_init(&T.dempty[c][b], 4);
            }
        mbar_init(&T.up_full, 4);
        mbar_init(&T.up_empty, 4);
        mbar_init(&T.drain, 1);
        T.abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&T.tmem_base, 512);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();
    if (p.status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
    tc_fence_before();
    build_tables(a, T);                           // its barriers also publish the mbarriers and the allocation
    tc_fence_after();
    const int total = T.total;
    const uint32_t tmem = T.tmem_base;
    auto all = [](bool ok) { return __all_sync(0xffffffffu, ok); };
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, abort, a.err, a.wait_limit); };
    auto d_col = [](int c, int b) { return (uint32_t)(c * 128 + b * 64); };
    auto a_col = [](int c, int b) { return (uint32_t)(256 + c * 128 + b * 64); };

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
            const CUtensorMap *m0 = shared ? &maps.w_shared[0] : &maps.w[0], *m1 = shared ? &maps.w_shared[1] : &maps.w[1];
            for (int kb = 0; kb < blocks; ++kb, ++it) {
                const int s = it % kStages;
                ok = all(wait(&T.cempty[s], ((it / kStages) & 1) ^ 1));
                if (!ok) break;
                uint8_t *C = codes + (size_t)s * 2 * kCodeTile;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&T.cfull[s], 2 * kCodeTile);
                    tma_load_2d_hint(C, m0, &T.cfull[s], kb * 64, y0, pol_w);
                    tma_load_2d_hint(C + kCodeTile, m1, &T.cfull[s], kb * 64, y1, pol_w);
                }
                __syncwarp();
            }
        }
        if (!ok)                                  // let loads in flight land before the CTA exits
            for (uint32_t j = it > (uint32_t)kStages ? it - kStages : 0; j < it; ++j)
                mbar_wait_drain(&T.cfull[j % kStages], (j / kStages) & 1, kDefaultWaitLimit);
    } else if (warp >= kGatherWarp) {
        // --------------------------------------------------------- gather
        // 16 threads take the 256 bytes of a row's 128 columns, 4 rows a pass.
        const int th = threadIdx.x - kGatherWarp * 32, piece = th & 15;
        const uint32_t panel = (uint32_t)(piece >> 3) * kPanel;
        uint32_t it = 0;
        bool ok = true;
        auto landed = [&](uint32_t j) {           // this thread's copies of block j are in place: tell the MMA
            fence_proxy_async();
            mbar_arrive(&T.bfull[j % kStages]);
        };
        for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
            const Unit U = unit_of(a, T, u);
            const bool shared = U.grp >= p.E;
            int row[kTokens / 4];                 // x rows; row 0 for tokens that are not there (their results are not used)
#pragma unroll
            for (int j = 0; j < kTokens / 4; ++j) {
                const int i = 4 * j + (th >> 4);
                int xi = 0;
                if (i < U.n) {
                    xi = U.row0 + i;
                    if (!p.x_by_row) xi = shared ? xi - p.P : p.perm ? p.perm[xi] : xi;
                    if ((unsigned)xi >= (unsigned)p.x_rows) xi = 0;
                }
                row[j] = xi;
            }
            for (int kb = 0; kb < blocks; ++kb, ++it) {
                const int s = it % kStages;
                ok = all(wait(&T.bempty[s], ((it / kStages) & 1) ^ 1));
                if (!ok) break;
                const uint32_t dst = smem_u32(toks) + s * 2 * kPanel + panel;
                const char *src = static_cast<const char *>(p.x) + kb * (kW4Block * 2) + piece * 16;
#pragma unroll
                for (int j = 0; j < kTokens / 4; ++j) {
                    const int i = 4 * j + (th >> 4);
                    if (4 * j < U.n)
                        cp_async16(dst + i * 128 + (((piece & 7) ^ (i & 7)) << 4), src + (size_t)row[j] * (p.cols * 2), 16);
                }
                cp_async_commit();
                if (it > 0) {                     // one block behind, so that copies overlap
                    cp_async_wait<1>();
                    landed(it - 1);
                }
            }
        }
        cp_async_wait_all();
        if (it > 0) landed(it - 1);
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA
        // The whole warp walks; one elected lane issues. Kept converged, the
        // descriptors live in uniform registers and an MMA costs 11 clocks at 16
        // tokens; issued under `lane == 0` each took 170.
        uint32_t it = 0, dn = 0;                  // blocks; groups' sums per tile
        bool ok = true;
        for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
            const Unit U = unit_of(a, T, u);
            const uint32_t idesc = idesc_bf16_f32(kRows, (U.n + 15) & ~15);
            for (int kb = 0; kb < blocks && ok; ++kb, ++it) {
                const int s = it % kStages, ab = it & 1;
                ok = all(wait(&T.bfull[s], (it / kStages) & 1));
                const uint32_t b0 = smem_u32(toks) + s * 2 * kPanel;
                const uint64_t bd0 = sw128_kmajor_desc(b0), bd1 = sw128_kmajor_desc(b0 + kPanel);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    ok = ok && all(wait(&T.afull[c][ab], (it >> 1) & 1));
#pragma unroll
                    for (int gi = 0; gi < GB; ++gi) {
                        const uint32_t d = dn + gi;
                        ok = ok && all(wait(&T.dempty[c][d & 1], ((d >> 1) & 1) ^ 1));
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t dt = tmem + d_col(c, d & 1), at = tmem + a_col(c, ab);
#pragma unroll
                            for (int k = gi * (G / 16); k < (gi + 1) * (G / 16); ++k)
                                umma_bf16_ts(dt, at + k * 8, (k < 4 ? bd0 : bd1) + (uint64_t)((k & 3) * 2), idesc,
                                             k != gi * (G / 16));
                            umma_commit(&T.dfull[c][d & 1]);
                            if (gi + 1 == GB) umma_commit(&T.aempty[c][ab]);
                            if (gi + 1 == GB && c == 1) umma_commit(&T.bempty[s]);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                }
                dn += GB;
            }
        }
        if (elect_one()) umma_commit(&T.drain);   // every MMA done before tensor memory is released
        __syncwarp();
        mbar_wait_drain(&T.drain, 0, kDefaultWaitLimit);
        __syncwarp();
    } else if (warp >= 8) {
        // --------------------------------------------------------- unpack
        const int c = (warp - 8) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        uint32_t it = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
            const Unit U = unit_of(a, T, u);
            const uint8_t *zr = nullptr;
            if (kZeros) {
                const bool shared = U.grp >= p.E;
                const uint8_t *z = kUp && c ? (shared ? p.up_shared.z : p.up.z) : (shared ? p.w_shared.z : p.w.z);
                zr = z + tile_row<kUp>(a, U, c, row) * (p.cols / G);
            }
            for (int kb = 0; kb < blocks; ++kb, ++it) {
                const int s = it % kStages, ab = it & 1;
                uint32_t z = 0x08080808u;
                if (kZeros) {
                    const uint8_t *at = zr + kb * GB;
                    z = GB == 1 ? *at : GB == 2 ? *reinterpret_cast<const uint16_t *>(at) : *reinterpret_cast<const uint32_t *>(at);
                }
                if (!all(wait(&T.cfull[s], (it / kStages) & 1))) { ok = false; break; }
                const uint8_t *src = codes + (size_t)s * 2 * kCodeTile + c * kCodeTile + row * 64;
                uint4 w[4];                       // w[t]: words of columns 8t of each 32-column slice
#pragma unroll
                for (int t = 0; t < 4; ++t) w[t] = *reinterpret_cast<const uint4 *>(src + ((t ^ ((row >> 1) & 3)) << 4));
                if (!all(wait(&T.aempty[c][ab], ((it >> 1) & 1) ^ 1))) { ok = false; break; }
                tc_fence_after();
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {  // 32 columns: 16 columns of tensor memory
                    const __nv_bfloat162 zz = zero_pair((z >> (8 * (jj / (G / 32)))) & 15u);
                    uint32_t r[16];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) r[4 * t + i] = code_pair(word_of(w[t], jj), i, zz);
                    tmem_st16(tmem + lanes + a_col(c, ab) + jj * 16, r);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&T.afull[c][ab]);
                    mbar_arrive(&T.cempty[s]);
                }
            }
        }
    } else {
        // --------------------------------------------------------- add up
        const int c = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        uint32_t dn = 0, un = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < total && ok; u += gridDim.x, ++un) {
            const Unit U = unit_of(a, T, u);
            const bool shared = U.grp >= p.E;
            const __nv_bfloat16 *sc = kUp && c ? (shared ? p.up_shared.s : p.up.s) : (shared ? p.w_shared.s : p.w.s);
            sc += tile_row<kUp>(a, U, c, row) * (p.cols / G);
            float acc[kTokens];
#pragma unroll
            for (int i = 0; i < kTokens; ++i) acc[i] = 0.f;
            __nv_bfloat16 nxt[GB];                // scales of the next block, loaded one block ahead
#pragma unroll
            for (int gi = 0; gi < GB; ++gi) nxt[gi] = sc[gi];
            for (int kb = 0; kb < blocks && ok; ++kb) {
                float s[GB];
#pragma unroll
                for (int gi = 0; gi < GB; ++gi) s[gi] = __bfloat162float(nxt[gi]);
                if (kb + 1 < blocks)
#pragma unroll
                    for (int gi = 0; gi < GB; ++gi) nxt[gi] = sc[(kb + 1) * GB + gi];
#pragma unroll
                for (int gi = 0; gi < GB; ++gi, ++dn) {
                    if (ok && !all(wait(&T.dfull[c][dn & 1], (dn >> 1) & 1))) ok = false;
                    if (!ok) continue;
                    tc_fence_after();
                    const uint32_t d = tmem + lanes + d_col(c, dn & 1);
#pragma unroll
                    for (int q = 0; q < kTokens / 16; ++q)
                        if (q * 16 < U.n) {
                            uint32_t v[16];
                            tmem_ld16(d + q * 16, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) acc[q * 16 + i] = fmaf(s[gi], __uint_as_float(v[i]), acc[q * 16 + i]);
                        }
                    // the up tile's last sums stay: their place takes the up values
                    if (kUp && c && kb + 1 == blocks && gi + 1 == GB) continue;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&T.dempty[c][dn & 1]);
                }
            }
            if (!ok) break;
            const int last = (dn - 1) & 1;
            if (kUp && c) {                       // up values to the gates' warps, in the same lanes of tensor memory
                if (!all(wait(&T.up_empty, (un & 1) ^ 1))) break;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < kTokens / 16; ++q)
                    if (q * 16 < U.n) tmem_st16(tmem + lanes + d_col(1, last) + q * 16, reinterpret_cast<const uint32_t *>(acc) + q * 16);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&T.up_full);
                continue;
            }
            uint32_t there[2] = {~0u, ~0u};       // a token that is not there stands for a row of zeros
            if (p.perm && !p.x_by_row && !shared)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    there[h] = __ballot_sync(0xffffffffu, h * 32 + lane < U.n &&
                                                              (unsigned)p.perm[U.row0 + h * 32 + lane] < (unsigned)p.x_rows);
            const int r = kUp ? U.tile * kRows + row : U.tile * 2 * kRows + c * kRows + row;
            YT *y = !kUp && shared ? static_cast<YT *>(p.y_shared) + (size_t)(U.row0 - p.P) * p.rows
                                   : static_cast<YT *>(p.y) + (size_t)U.row0 * p.rows;
            if (kUp) {
                if (!all(wait(&T.up_full, un & 1))) break;
                tc_fence_after();
            }
#pragma unroll
            for (int q = 0; q < kTokens / 16; ++q)
                if (q * 16 < U.n) {
                    uint32_t v[16];
                    if (kUp) {
                        tmem_ld16(tmem + lanes + d_col(1, last) + q * 16, v);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float o = kUp ? silu_mul(acc[q * 16 + i], __uint_as_float(v[i])) : acc[q * 16 + i];
                        if (!((there[q >> 1] >> ((q & 1) * 16 + i)) & 1)) o = 0.f;
                        if (q * 16 + i < U.n && r < p.rows) store_val(y + (size_t)(q * 16 + i) * p.rows + r, o);
                    }
                }
            if (kUp) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&T.dempty[1][last]);
                    mbar_arrive(&T.up_empty);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
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
    cudaFuncSetAttribute(kernel<kUp, G, kZeros, YT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    launch_pdl(kernel<kUp, G, kZeros, YT>, grid, kThreads, kSmem, st, maps, a);
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

kmoe_status launch_w4_tc(const W4Product &p, int *err, long long wait_limit, cudaStream_t st)
{
    using namespace w4tc;
    Args a{};
    a.p = p;
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
    const long long most = ((long long)std::min(p.E, p.P) + (p.P + p.n_shared) / 32 + 1) * a.tiles;
    const int grid = (int)std::min<long long>(sms, most);
    if (up) return pick<true, __nv_bfloat16>(m, a, grid, st);
    return p.y_dtype == KMOE_F32 ? pick<false, float>(m, a, grid, st) : pick<false, __nv_bfloat16>(m, a, grid, st);
}

}  // namespace kmoe
