// Weights into the 4-bit format with group scales, and back.
//
// Symmetric:    s = bf16(max |w| / 7),     q = clamp(rint(w / s), -8, 7) + 8
// Zero points:  s = bf16((hi - lo) / 15),  z = clamp(rint(-lo / s), 0, 15),
//               q = clamp(rint(w / s) + z, 0, 15),  lo <= 0 <= hi
// A thread owns one 8-column word, so a group of 32, 64 or 128 columns is 4, 8
// or 16 neighbouring lanes, its extremes come from two to four shuffles, and
// sixteen lanes write the 64 bytes of a 128-column block.
#include "w4.cuh"

namespace kmoe {

constexpr int kQuantW4Threads = 256;

template <class T>
__device__ __forceinline__ void store8(T *p, const float *v);
template <>
__device__ __forceinline__ void store8<float>(float *p, const float *v)
{
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16 *p, const float *v)
{
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = as_u32(__floats2bfloat162_rn(v[2 * i], v[2 * i + 1]));
    *reinterpret_cast<uint4 *>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}

// words: rows * cols / 8, a multiple of 16, so the lanes of a group are all
// inside or all outside.
template <class T, bool kZeros>
__global__ void __launch_bounds__(kQuantW4Threads)
quant_w4_kernel(const T *__restrict__ w, long long words, int group, uint32_t *__restrict__ codes,
                __nv_bfloat16 *__restrict__ scales, uint8_t *__restrict__ zeros)
{
    const int lanes = group / 8;
    const long long i = (long long)blockIdx.x * kQuantW4Threads + threadIdx.x;
    float v[8], lo = 0.f, hi = 0.f;
    if (i < words) {
        load8(w + i * 8, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            lo = fminf(lo, v[e]);
            hi = fmaxf(hi, v[e]);
        }
    }
    for (int o = 1; o < lanes; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (i >= words) return;
    const __nv_bfloat16 sb =
        __float2bfloat16_rn(kZeros ? __fdiv_rn(hi - lo, 15.f) : __fdiv_rn(fmaxf(hi, -lo), 7.f));
    const float sf = __bfloat162float(sb), s = sf == 0.f ? 1.f : sf;
    const float z = kZeros ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f) : 8.f;
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = fminf(fmaxf(rintf(__fdiv_rn(v[e], s)) + z, 0.f), 15.f);
        word |= ((uint32_t)q & 15u) << (4 * (e >> 1) + 16 * (e & 1));
    }
    codes[(i & ~15LL) + w4_place((int)(i & 15))] = word;
    if ((threadIdx.x & (lanes - 1)) == 0) {
        scales[i / lanes] = __float2bfloat16_rn(s);
        if (kZeros) zeros[i / lanes] = (uint8_t)z;
    }
}

template <class T>
__global__ void __launch_bounds__(kQuantW4Threads)
dequant_w4_kernel(const uint32_t *__restrict__ codes, const __nv_bfloat16 *__restrict__ scales,
                  const uint8_t *__restrict__ zeros, long long words, int group, T *__restrict__ out)
{
    const long long i = (long long)blockIdx.x * kQuantW4Threads + threadIdx.x;
    if (i >= words) return;
    const uint32_t word = codes[(i & ~15LL) + w4_place((int)(i & 15))];
    const long long at = i / (group / 8);
    const float s = __bfloat162float(scales[at]), z = zeros ? (float)zeros[at] : 8.f;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ((float)((word >> (4 * (e >> 1) + 16 * (e & 1))) & 15u) - z) * s;
    store8(out + i * 8, v);
}

static kmoe_status grid_for(long long words, unsigned *grid)
{
    const long long g = (words + kQuantW4Threads - 1) / kQuantW4Threads;
    if (g > 0x7fffffffLL) return fail(KMOE_ERR_UNSUPPORTED, "4-bit weights: %lld words", words);
    *grid = (unsigned)g;
    return KMOE_OK;
}

kmoe_status launch_quant_w4(const void *w, int w_dtype, int rows, int cols, int group, uint8_t *codes,
                            __nv_bfloat16 *scales, uint8_t *zeros, cudaStream_t st)
{
    const long long words = (long long)rows * (cols / 8);
    unsigned grid;
    const kmoe_status g = grid_for(words, &grid);
    if (g != KMOE_OK) return g;
    uint32_t *c = reinterpret_cast<uint32_t *>(codes);
#define KMOE_QUANT_W4(T, Z)                                                                                     \
    quant_w4_kernel<T, Z><<<grid, kQuantW4Threads, 0, st>>>(static_cast<const T *>(w), words, group, c, scales, zeros)
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
    unsigned grid;
    const kmoe_status g = grid_for(words, &grid);
    if (g != KMOE_OK) return g;
    const uint32_t *c = reinterpret_cast<const uint32_t *>(w.q);
    if (out_dtype == KMOE_F32)
        dequant_w4_kernel<float><<<grid, kQuantW4Threads, 0, st>>>(c, w.s, w.z, words, group, static_cast<float *>(out));
    else
        dequant_w4_kernel<__nv_bfloat16><<<grid, kQuantW4Threads, 0, st>>>(c, w.s, w.z, words, group,
                                                                          static_cast<__nv_bfloat16 *>(out));
    return check_launch("dequant_w4");
}

}  // namespace kmoe
