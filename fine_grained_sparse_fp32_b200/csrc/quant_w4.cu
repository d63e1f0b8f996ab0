// Weights into the 4-bit format with group scales, and back.
//
// Symmetric:    s = bf16(max |w| / 7),     q = clamp(rint(w / s), -8, 7) + 8
// Zero points:  s = bf16((hi - lo) / 15),  z = clamp(rint(-lo / s), 0, 15),
//               q = clamp(rint(w / s) + z, 0, 15),  lo <= 0 <= hi
// A thread owns one 8-column word, so a group of 32, 64 or 128 columns is 4, 8
// or 16 neighbouring lanes, its extremes come from two to four shuffles, and
// sixteen lanes write the 64 bytes of a 128-column block. Instruction issue bounds the
// quantiser: 83.9 M FP32 values (groups of 32, zero points) take 82 us at 3.25 of 4
// instructions a clock and SM, the ALU pipe at 62% (4.7 TB/s of reads and writes). HBM bounds
// the way back: 64 us, 6.0 TB/s at 1.9 instructions. CTAs of 128 threads: of 256, both took 150 us
// together; two words a thread: one took 91 us, four 82.
#include "w4.cuh"

namespace kmoe {

constexpr int kQuantW4Threads = 128, kQuantW4Words = 2, kDequantW4Parts = 4;

// rint(v / s) of the IEEE quotient, r = 1 / s rounded. v * r is within
// 3 * 2^-24 * 16 < 3e-6 of that quotient where the quotient is below 16, so
// both round to the same whole number unless v * r lies next to a half; there,
// and where a product is not finite, the division is done (about one value in
// 5000; all by division: 83.9 M FP32 values in 116 us).
__device__ __forceinline__ float rint_quotient(float v, float s, float r)
{
    const float t = v * r, q = rintf(t);
    return fabsf(t - q) < 0.4999f ? q : rintf(__fdiv_rn(v, s));
}

// words: rows * cols / 8, a multiple of 16, so the lanes of a group are all
// inside or all outside.
template <class T, bool kZeros>
__global__ void __launch_bounds__(kQuantW4Threads)
quant_w4_kernel(const T *__restrict__ w, long long words, int lanes_log2, uint32_t *__restrict__ codes,
                __nv_bfloat16 *__restrict__ scales, uint8_t *__restrict__ zeros)
{
    const long long first = (long long)blockIdx.x * (kQuantW4Words * kQuantW4Threads) + threadIdx.x;
    float v[kQuantW4Words][8];
#pragma unroll
    for (int u = 0; u < kQuantW4Words; ++u) {
        const long long i = first + u * kQuantW4Threads;
        if (i < words) {
            load8(w + i * 8, v[u]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] = 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < kQuantW4Words; ++u) {
        const long long i = first + u * kQuantW4Threads;
        float lo = 0.f, hi = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            lo = fminf(lo, v[u][e]);
            hi = fmaxf(hi, v[u][e]);
        }
        for (int o = 0; o < lanes_log2; ++o) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, 1 << o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, 1 << o));
        }
        const __nv_bfloat16 sb =
            __float2bfloat16_rn(kZeros ? __fdiv_rn(hi - lo, 15.f) : __fdiv_rn(fmaxf(hi, -lo), 7.f));
        const float sf = __bfloat162float(sb), s = sf == 0.f ? 1.f : sf, r = __frcp_rn(s);
        const float z = kZeros ? fminf(fmaxf(rint_quotient(-lo, s, r), 0.f), 15.f) : 8.f;
        uint32_t word = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = fminf(fmaxf(rint_quotient(v[u][e], s, r) + z, 0.f), 15.f);
            word |= ((uint32_t)q & 15u) << (4 * (e >> 1) + 16 * (e & 1));
        }
        if (i >= words) continue;
        codes[(i & ~15LL) + w4_place((int)(i & 15))] = word;
        if ((threadIdx.x & ((1 << lanes_log2) - 1)) == 0) {
            scales[i >> lanes_log2] = __float2bfloat16_rn(s);
            if (kZeros) zeros[i >> lanes_log2] = (uint8_t)z;
        }
    }
}

// 16 bytes of the result for each thread and step, so that a warp's store is
// one contiguous run: half a word's columns in FP32, a whole word's in BF16.
template <class T>
__global__ void __launch_bounds__(kQuantW4Threads)
dequant_w4_kernel(const uint32_t *__restrict__ codes, const __nv_bfloat16 *__restrict__ scales,
                  const uint8_t *__restrict__ zeros, long long words, int lanes_log2, T *__restrict__ out)
{
    constexpr int kHalves = sizeof(T) == 4 ? 2 : 1, kCols = 8 / kHalves;
    const long long parts = words * kHalves;
    const long long first = (long long)blockIdx.x * (kDequantW4Parts * kQuantW4Threads) + threadIdx.x;
    uint32_t word[kDequantW4Parts];
    float s[kDequantW4Parts], z[kDequantW4Parts];
#pragma unroll
    for (int u = 0; u < kDequantW4Parts; ++u) {
        const long long p = first + u * kQuantW4Threads, i = p / kHalves;
        if (p >= parts) break;
        word[u] = codes[(i & ~15LL) + w4_place((int)(i & 15))];
        s[u] = __bfloat162float(scales[i >> lanes_log2]);
        z[u] = zeros ? (float)zeros[i >> lanes_log2] : 8.f;
    }
#pragma unroll
    for (int u = 0; u < kDequantW4Parts; ++u) {
        const long long p = first + u * kQuantW4Threads;
        if (p >= parts) break;
        const uint32_t x = kHalves == 2 ? word[u] >> (8 * (int)(p & 1)) : word[u];
        float v[kCols];
#pragma unroll
        for (int e = 0; e < kCols; ++e) v[e] = ((float)((x >> (4 * (e >> 1) + 16 * (e & 1))) & 15u) - z[u]) * s[u];
        uint4 o;
        if constexpr (kHalves == 2) {
            o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        } else {
            o = make_uint4(as_u32(__floats2bfloat162_rn(v[0], v[1])), as_u32(__floats2bfloat162_rn(v[2], v[3])),
                           as_u32(__floats2bfloat162_rn(v[4], v[5])), as_u32(__floats2bfloat162_rn(v[6], v[7])));
        }
        *reinterpret_cast<uint4 *>(out + p * kCols) = o;
    }
}

static kmoe_status grid_for(long long items, int per_cta, unsigned *grid)
{
    const long long g = (items + per_cta - 1) / per_cta;
    if (g > 0x7fffffffLL) return fail(KMOE_ERR_UNSUPPORTED, "4-bit weights: %lld CTAs", g);
    *grid = (unsigned)g;
    return KMOE_OK;
}

kmoe_status launch_quant_w4(const void *w, int w_dtype, int rows, int cols, int group, uint8_t *codes,
                            __nv_bfloat16 *scales, uint8_t *zeros, cudaStream_t st)
{
    const long long words = (long long)rows * (cols / 8);
    const int lanes_log2 = group == 128 ? 4 : group == 64 ? 3 : 2;
    unsigned grid;
    const kmoe_status g = grid_for(words, kQuantW4Words * kQuantW4Threads, &grid);
    if (g != KMOE_OK) return g;
    uint32_t *c = reinterpret_cast<uint32_t *>(codes);
#define KMOE_QUANT_W4(T, Z)                                                                                     \
    quant_w4_kernel<T, Z><<<grid, kQuantW4Threads, 0, st>>>(static_cast<const T *>(w), words, lanes_log2, c, scales, \
                                                               zeros)
    if (w_dtype == KMOE_F32) {
        if (zeros) KMOE_QUANT_W4(float, true);
        else KMOE_QUANT_W4(float, false);
    } else {
        if (zeros) KMOE_QUANT_W4(__nv_bfloat16, true);
        else KMOE_QUANT_W4(__nv_bfloat16, false);
    }
#undef KMOE_QUANT_W4
    return check_launch("quant_w4");
}

kmoe_status launch_dequant_w4(const W4Ptrs &w, int group, int rows, int cols, void *out, int out_dtype,
                              cudaStream_t st)
{
    const long long words = (long long)rows * (cols / 8);
    const int lanes_log2 = group == 128 ? 4 : group == 64 ? 3 : 2, halves = out_dtype == KMOE_F32 ? 2 : 1;
    unsigned grid;
    const kmoe_status g = grid_for(words * halves, kDequantW4Parts * kQuantW4Threads, &grid);
    if (g != KMOE_OK) return g;
    const uint32_t *c = reinterpret_cast<const uint32_t *>(w.q);
    if (out_dtype == KMOE_F32)
        dequant_w4_kernel<float><<<grid, kQuantW4Threads, 0, st>>>(c, w.s, w.z, words, lanes_log2,
                                                                   static_cast<float *>(out));
    else
        dequant_w4_kernel<__nv_bfloat16><<<grid, kQuantW4Threads, 0, st>>>(c, w.s, w.z, words, lanes_log2,
                                                                          static_cast<__nv_bfloat16 *>(out));
    return check_launch("dequant_w4");
}

}  // namespace kmoe
