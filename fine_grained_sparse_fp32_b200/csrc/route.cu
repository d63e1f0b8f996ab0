// Routing from logits: scores, groups, top-K and weights (kmoe_routing).
//
//   s = sigmoid(l) or softmax(l);  c = s + bias
//   groups by the largest c or the sum of the two largest; the best stay
//   idx = top-K of c in the groups that stayed;  w = s[idx] (/ sum) * scale
// One warp per token. The 32 lanes are shared out evenly among the groups
// (L = 32 / n_groups rounded down to a power of two, so a group's lanes are
// neighbours), and lane j of a group holds its experts j, j + L, ... in
// registers. Each keeps the two best of them in hand, so that a round of the
// selection is two warp reductions, whatever the number of experts.
//
// The choice is the one that FP64 scores make, at the cost of FP32 ones. FP32
// scores are off by at most D = 2^-20 max s + 2^-22 max |c| (the hardware
// exponential and reciprocal; the error of s is s (1 - s) times that of
// the exponential, or s times it, whose growth with the exponent s outweighs). In a softmax,
// in units of 2^-24 max s, two scores are off by 5.4 each (exponential 4, its argument 0.9,
// the product 0.5), and all of them by one factor, that of their sum: 5 + NPL + 5 of its
// terms, NPL additions in a lane and 5 over the warp. Their difference is off by
// less than NPL + 24 of them, and D takes half of that. Where a bias lies outside
// +-kFarBias, each score's own |c| counts instead of the largest: with that, one expert switched
// off by -1e9 sends every token to FP64 (65536 tokens: 343 us, not 95).
// Where the K + 1 best are further than 2 D apart, and the last group that stays
// further than 4 D from the first that goes, every exact score has the same
// order. Any other token (about one in 300) is decided again in FP64. Without a
// bias the order of scores is that of the logits, which are exact: equal ones
// are equal in FP64 too, and only logits whose FP64 scores may round to the same
// number go to FP64: closer than 1e-13, with scores below e^-600, or above 20
// under a sigmoid. Two equal ones at the end of the choice can hide a third that is
// such a neighbour of both; it takes scores like those, or logits below 2e-6, whose
// places are that close.
#include "permute_dev.cuh"
#include "w4.cuh"

#include <algorithm>
#include <cfloat>
#include <climits>
#include <type_traits>

namespace kmoe {

constexpr float kFarBias = 4.f;
constexpr int kRouteWarps = 8, kRouteCtas = 4;       // tokens in work of a CTA, CTAs of an SM

struct RouteArgs {
    const float *bias;
    int N, E, K, n_groups, topk_groups, size, lanes;   // size: experts of a group; lanes: lanes of a group
    bool softmax, top2, renormalise;
    float scale;
    int exact_places;                     // doubles of shared memory for a warp's FP64 choice
    int32_t *idx;
    float *w;
    int32_t *hist;
};

// Whole-number keys in the order of floats. Masked experts and empty places
// have the key of -inf, chosen ones and groups that go one below every float.
constexpr int kGoneKey = INT_MIN, kMaskedKey = (int)(0xff800000u ^ 0x7fffffffu);
__device__ __forceinline__ int key_of(float v)    // v is not -0
{
    const int b = __float_as_int(v);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float value_of(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

// Hardware exponential and reciprocal, for the choice: results below 2^-126
// become 0, which D allows for.
__device__ __forceinline__ float quick_exp(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
    return y;
}
__device__ __forceinline__ float quick_sigmoid(float l)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + quick_exp(-l)));
    return y;
}

// ------------------------------------------------- FP64 choice of one token
__device__ __forceinline__ double warp_max(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// One token's choice by FP64 scores, which lie in shared memory (c, one place
// for each lane and expert). Lane k returns choice k and its score.
template <class LT>
__device__ __noinline__ int route_exact(const LT *lr, const RouteArgs &a, double *c, double *score_out)
{
    constexpr double kMasked = -DBL_MAX, kGone = -INFINITY;
    const int lane = threadIdx.x & 31, group = lane / a.lanes, sub = lane % a.lanes, base = group * a.size;
    const int per = group < a.n_groups ? (a.size - sub + a.lanes - 1) / a.lanes : 0;
    auto logit = [&](int e) {
        const double l = (double)to_f32(lr[e]);
        return isnan(l) ? -INFINITY : l;
    };
    double top = -INFINITY, sum = 0;
    if (a.softmax) {
#pragma unroll 1
        for (int i = 0; i < per; ++i) top = fmax(top, logit(base + sub + a.lanes * i));
        top = warp_max(top);
    }
    auto weight = [&](double l) {                 // before the division by `sum`
        if (!a.softmax) return 1.0 / (1.0 + exp(-l));
        return l == -INFINITY ? 0.0 : l == top ? 1.0 : exp(l - top);
    };
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
        const double w = weight(logit(base + sub + a.lanes * i));
        c[i * 32 + lane] = w;
        sum += w;
    }
    if (a.softmax) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    } else {
        sum = 1.0;
    }
    double m1 = kMasked, m2 = kMasked;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
        const int e = base + sub + a.lanes * i;
        const double b = a.bias ? (double)a.bias[e] : 0.0, w = c[i * 32 + lane];
        const double v = logit(e) == -INFINITY || isnan(b) || b == -INFINITY ? kMasked
                         : (a.softmax ? (sum > 0 ? w / sum : 0.0) : w) + b;
        c[i * 32 + lane] = v;
        m2 = fmax(m2, fmin(m1, v));
        m1 = fmax(m1, v);
    }
    bool stays = true;
    if (a.topk_groups < a.n_groups) {
        for (int o = 1; o < a.lanes; o <<= 1) {
            const double p1 = __shfl_xor_sync(0xffffffffu, m1, o), p2 = __shfl_xor_sync(0xffffffffu, m2, o);
            m2 = fmax(fmin(m1, p1), fmax(m2, p2));
            m1 = fmax(m1, p1);
        }
        const double mine = a.top2 && m2 != kMasked ? m1 + m2 : m1;
        int before = 0;
        for (int g = 0; g < a.n_groups; ++g) {
            const double o = __shfl_sync(0xffffffffu, mine, g * a.lanes);
            before += o > mine || (o == mine && g < group);
        }
        stays = before < a.topk_groups;
    }
    int chosen = 0;
    bool ok = false;
    for (int k = 0; k < a.K; ++k) {
        double bc = kGone;
        int bi = 0;
        if (stays) {
#pragma unroll 4
            for (int i = 0; i < per; ++i) {
                const double v = c[i * 32 + lane];
                if (v > bc) { bc = v; bi = i; }
            }
        }
        const double best = warp_max(bc);
        const int be = base + sub + a.lanes * bi, e = __reduce_min_sync(0xffffffffu, bc == best ? be : INT_MAX);
        if (bc == best && be == e) c[bi * 32 + lane] = kGone;
        if (lane == k) { chosen = e; ok = best != kMasked; }
    }
    *score_out = lane < a.K && ok ? (sum > 0 ? weight(logit(chosen)) / sum : 0.0) : 0.0;
    return chosen;
}

// ------------------------------------------------------------------ kernel
// The two best of a lane's keys, ties to the lower index.
template <int NPL>
__device__ __forceinline__ void best_two(const int (&key)[NPL], uint64_t gone, int &m1, int &m2, int &i1, int &i2)
{
    m1 = m2 = kGoneKey;
    i1 = i2 = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int k = gone >> i & 1 ? kGoneKey : key[i];
        const bool first = k > m1, second = k > m2;
        if (second) { m2 = first ? m1 : k; i2 = first ? i1 : i; }
        if (first) { m1 = k; i1 = i; }
    }
}

// Instructions bound it: 65536 tokens of 384 experts in 8 groups, K = 6, FP32
// logits, bias, take 94 us (1.1 TB/s), 941 instructions a token at 92, the integer pipe
// (comparisons, selects) at 65% of its rate. Four CTAs an SM (64 registers): two
// (120 registers) took 127 us where four took 111.
template <class LT, int NPL, bool kBias>
__global__ void __launch_bounds__(32 * kRouteWarps, NPL <= 16 ? kRouteCtas : 2)
route_kernel(const LT *__restrict__ logits, const RouteArgs a)
{
    extern __shared__ double exact_c[];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int group = lane / a.lanes, sub = lane % a.lanes, base = group * a.size;
    const int per = group < a.n_groups ? (a.size - sub + a.lanes - 1) / a.lanes : 0;      // this lane's experts
    float b[kBias ? NPL : 1], b_max = 0.f;
    if (kBias) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            b[i] = fmaxf(i < per ? a.bias[base + sub + a.lanes * i] : 0.f, -INFINITY);    // NaN becomes -inf
            if (b[i] > -INFINITY) b_max = fmaxf(b_max, fabsf(b[i]));
        }
        b_max = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(b_max)));
    }
    const bool far = kBias && b_max > kFarBias;
    const int step = gridDim.x * kRouteWarps;
    for (int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5); t < a.N; t += step) {
        const LT *lr = logits + (size_t)t * a.E, *mine_of = lr + base + sub;
        int key[NPL];
        float s_max = 1.f, top = -INFINITY, sum = 0.f;
        {
            float l[NPL];
#pragma unroll
            for (int i = 0; i < NPL; ++i) l[i] = i < per ? to_f32(mine_of[a.lanes * i]) : -INFINITY;
            if (a.softmax) {
#pragma unroll
                for (int i = 0; i < NPL; ++i) top = fmaxf(top, l[i]);         // fmaxf drops NaN
                top = value_of(__reduce_max_sync(0xffffffffu, key_of(top + 0.f)));
                if (kBias || !a.renormalise) {
#pragma unroll
                    for (int i = 0; i < NPL; ++i) {
                        const float e = l[i] > -INFINITY ? (l[i] == top ? 1.f : quick_exp(l[i] - top)) : 0.f;
                        sum += e;
                        if (kBias) key[i] = __float_as_int(e);
                    }
                    sum = warp_sum(sum);
                    s_max = sum > 0.f ? 1.f / sum : 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                float c = fmaxf(l[i], -INFINITY) + 0.f;                       // no NaN, no -0
                if (kBias) {
                    c = (a.softmax ? __int_as_float(key[i]) * s_max : quick_sigmoid(l[i])) + b[kBias ? i : 0];
                    c = l[i] > -INFINITY ? c : -INFINITY;
                }
                key[i] = key_of(c);
            }
        }
        const float D = s_max * (a.softmax ? (NPL + 24) * 0x1p-25f : 0x1p-20f) + (far ? 0.f : (s_max + b_max) * 0x1p-22f) + 1e-36f;
        // whether two neighbours' order is not the exact one for sure (hi >= lo)
        auto unsure = [&](float hi, float lo, float width) {
            const float d = hi - lo;
            if (kBias) return !(d > width);
            const bool ties = a.softmax ? hi - top < -600.f : lo > 20.f || hi < -600.f;
            return ties || (d == 0.f ? fabsf(hi) < 2e-6f : !(d > 1e-13f));
        };
        int m1, m2, i1, i2;
        best_two(key, 0, m1, m2, i1, i2);
        bool again = false;
        if (a.topk_groups < a.n_groups) {
            int g1 = m1, g2 = m2;
            for (int o = 1; o < a.lanes; o <<= 1) {
                const int p1 = __shfl_xor_sync(0xffffffffu, g1, o), p2 = __shfl_xor_sync(0xffffffffu, g2, o);
                g2 = max(min(g1, p1), max(g2, p2));
                g1 = max(g1, p1);
            }
            int mine = g1;                        // group score as a key
            const bool sums = a.top2 && g1 > kMaskedKey;
            if (sums) {
                float v1 = value_of(g1), v2 = value_of(g2);
                if (!kBias) {                     // logits: their scores, the softmax's up to its divisor
                    v1 = a.softmax ? (v1 == top ? 1.f : quick_exp(v1 - top)) : quick_sigmoid(v1);
                    v2 = a.softmax ? (v2 == top ? 1.f : quick_exp(v2 - top)) : quick_sigmoid(v2);
                }
                mine = key_of((g2 > kMaskedKey ? v1 + v2 : v1) + 0.f);
            }
            if (group >= a.n_groups) mine = kGoneKey;
            int before = 0;
            for (int g = 0; g < a.n_groups; ++g) {
                const int o = __shfl_sync(0xffffffffu, mine, g * a.lanes);
                before += o > mine || (o == mine && g < group);
            }
            const bool stays = group < a.n_groups && before < a.topk_groups;
            int low = mine, high = mine;          // what a group score's own size leaves open
            if (far && mine > kMaskedKey) {
                const float own = (fabsf(value_of(g1)) + (a.top2 && g2 > kMaskedKey ? fabsf(value_of(g2)) : 0.f)) * 0x1p-22f;
                low = key_of(value_of(mine) - own + 0.f);
                high = key_of(value_of(mine) + own + 0.f);
            }
            const int last = __reduce_min_sync(0xffffffffu, stays ? low : INT_MAX);
            const int next = __reduce_max_sync(0xffffffffu, stays ? kGoneKey : high);
            if (next > kMaskedKey) {              // (masked groups come last in order of their index)
                const float hi = value_of(last), lo = value_of(next);
                if (kBias || !a.top2) again = unsure(hi, lo, 4 * D);
                else again = !(hi - lo > 4 * (0x1p-20f + 0x1p-22f));
            }
            if (!stays) m1 = m2 = kGoneKey;
        }
        uint64_t gone = 0;
        int chosen = 0;
        float prev = INFINITY, gap = INFINITY;    // gap: between neighbours in the order
        auto choose = [&](auto each) {            // each: every score's own share counts
            for (int k = 0;; ++k) {
                const int best = __reduce_max_sync(0xffffffffu, m1);
                const float v = value_of(best);
                if (best > kMaskedKey) {
                    // (infinities: NaN, and sure)
                    if (each.value) gap = fminf(gap, fmaf(fabsf(prev) + fabsf(v), -0x1p-23f, prev - v));
                    else if (kBias) gap = fminf(gap, prev - v);
                    else if (k > 0) again |= unsure(prev, v, 0.f);
                }
                if (k == a.K) break;
                if (best <= kMaskedKey) {             // fewer than K experts to choose from: masked ones in order
                    again = true;
                    break;
                }
                const int mine = base + sub + a.lanes * i1;
                const int e = __reduce_min_sync(0xffffffffu, m1 == best ? mine : INT_MAX);
                if (lane == k) chosen = e;
                prev = v;
                const bool owner = m1 == best && mine == e;
                if (owner) {
                    gone |= 1ull << i1;
                    m1 = m2;
                    i1 = i2;
                    m2 = kGoneKey;
                }
                // a lane whose two best are both gone looks for the next ones
                if (__any_sync(0xffffffffu, owner && m1 == kGoneKey)) {
                    int n1, n2, j1, j2;
                    best_two(key, gone, n1, n2, j1, j2);
                    if (owner) { m1 = n1; m2 = n2; i1 = j1; i2 = j2; }
                }
            }
        };
        if (far) choose(std::true_type{});
        else choose(std::false_type{});
        if (kBias) again |= !(gap > 2 * D);
        float s = 0.f;                            // score of choice `lane`
        if (!again) {
            const float l = lane < a.K ? to_f32(lr[chosen]) : -INFINITY;
            if (!a.softmax) {
                const float e = expf(-fabsf(l));          // (not e^-l, which is infinite where the score is not yet 0)
                s = lane < a.K ? (l < 0.f ? e : 1.f) / (1.f + e) : 0.f;
            } else {
                // weights that are renormalised need no common divisor, and over the largest
                // choice, not the largest logit, none of them is lost below 2^-126
                const float over = a.renormalise ? value_of(__reduce_max_sync(0xffffffffu, key_of(l + 0.f))) : top;
                s = lane < a.K ? (l == over ? 1.f : expf(l - over)) / (a.renormalise ? 1.f : sum) : 0.f;
            }
        }
        const float total = warp_sum(s);          // 0 from lanes without a choice
        // Scores that FP32 cannot weigh against each other, too: below 2^-126 a score is off by up
        // to 2^-150, which over a sum of 1e-8 is less than 1e-37 of weight.
        if (again || (a.renormalise && total < 1e-8f)) {
            double exact;
            chosen = route_exact(lr, a, exact_c + (threadIdx.x >> 5) * a.exact_places, &exact);
            if (a.renormalise) {
                double all = lane < a.K ? exact : 0.0;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
                exact = all > 0 ? exact / all : 0.0;
            }
            s = (float)exact;
        } else if (a.renormalise) {
            s /= total;
        }
        if (lane < a.K) {
            a.idx[(size_t)t * a.K + lane] = chosen;
            a.w[(size_t)t * a.K + lane] = s * a.scale;
            if (a.hist) atomicAdd(a.hist + (size_t)(t / kChunk) * a.E + chosen, 1);   // whole numbers: exact in any order
        }
    }
}

template <class LT, bool kBias>
static kmoe_status run_route(const LT *logits, RouteArgs a, cudaStream_t st)
{
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // each warp takes the same number of tokens, so that the bias is read once for them
    const int ctas = (a.N + kRouteWarps - 1) / kRouteWarps, room = sms * kRouteCtas, each = (ctas + room - 1) / room;
    const int grid = (ctas + each - 1) / each, npl = (a.size + a.lanes - 1) / a.lanes;
    a.exact_places = npl * 32;
    const int smem = kRouteWarps * a.exact_places * (int)sizeof(double);
#define KMOE_ROUTE(n)                                                                                                 \
    do {                                                                                                              \
        if (smem > 48 << 10)                                                                                          \
            cudaFuncSetAttribute(route_kernel<LT, n, kBias>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);      \
        launch_pdl(route_kernel<LT, n, kBias>, grid, 32 * kRouteWarps, smem, st, logits, a);                          \
    } while (0)
    if (npl <= 2) KMOE_ROUTE(2);
    else if (npl <= 4) KMOE_ROUTE(4);
    else if (npl <= 8) KMOE_ROUTE(8);
    else if (npl <= 12) KMOE_ROUTE(12);
    else if (npl <= 16) KMOE_ROUTE(16);
    else if (npl <= 32) KMOE_ROUTE(32);
    else KMOE_ROUTE(64);
#undef KMOE_ROUTE
    return check_launch("route");
}

kmoe_status launch_route(const void *logits, int l_dtype, const float *bias, int N, int E, int K,
                         const kmoe_routing &r, int32_t *idx, float *w, cudaStream_t st, int32_t *hist)
{
    RouteArgs a{};
    a.bias = bias;
    a.N = N;
    a.E = E;
    a.K = K;
    a.n_groups = r.topk_groups < r.n_groups ? r.n_groups : 1;      // all groups stay: no groups
    a.topk_groups = r.topk_groups < r.n_groups ? r.topk_groups : 1;
    a.size = E / a.n_groups;
    a.lanes = 32;
    while (a.lanes * a.n_groups > 32) a.lanes >>= 1;
    a.softmax = r.score == KMOE_ROUTE_SOFTMAX;
    a.top2 = r.group_score == KMOE_GROUP_TOP2;
    a.renormalise = r.renormalise != 0;
    a.scale = r.scale;
    a.idx = idx;
    a.w = w;
    a.hist = hist;
    if (l_dtype == KMOE_F32) {
        const float *l = static_cast<const float *>(logits);
        return bias ? run_route<float, true>(l, a, st) : run_route<float, false>(l, a, st);
    }
    const __nv_bfloat16 *l = static_cast<const __nv_bfloat16 *>(logits);
    return bias ? run_route<__nv_bfloat16, true>(l, a, st) : run_route<__nv_bfloat16, false>(l, a, st);
}

}  // namespace kmoe
