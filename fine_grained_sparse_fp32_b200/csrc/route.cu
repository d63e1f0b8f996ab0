// Routing from logits: scores, groups, top-K and weights (kmoe_routing).
//
//   s = sigmoid(l) or softmax(l);  c = s + bias
//   groups by the largest c or the sum of the two largest; the best stay
//   idx = top-K of c in the groups that stayed;  w = s[idx] (/ sum) * scale
// One warp per token. The 32 lanes are shared out evenly among the groups
// (L = 32 / n_groups rounded down to a power of two, so a group's lanes are
// neighbours), and lane j of a group holds its experts j, j + L, ... in
// registers, in ascending order.
#include "permute_dev.cuh"
#include "w4.cuh"

#include <cfloat>
#include <climits>

namespace kmoe {

constexpr int kRouteTokens = 8;       // tokens (warps) of a CTA

struct RouteArgs {
    const float *bias;
    int N, E, K, n_groups, topk_groups, size, lanes;   // size: experts of a group; lanes: lanes of a group
    bool softmax, top2, renormalise;
    float scale;
    int32_t *idx;
    float *w;
    int32_t *hist;
};

// FP64 value of a selection score: masked experts sort behind all others.
constexpr double kMasked = -DBL_MAX, kGone = -INFINITY;

__device__ __forceinline__ double warp_max(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

template <class LT, int NPL>
__global__ void __launch_bounds__(32 * kRouteTokens)
route_kernel(const LT *__restrict__ logits, const RouteArgs a)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kRouteTokens + (threadIdx.x >> 5);
    if (t >= a.N) return;
    const int group = lane / a.lanes, sub = lane % a.lanes;
    const int base = group * a.size;
    const LT *lr = logits + (size_t)t * a.E;
    double s[NPL], c[NPL];
    uint64_t masked = 0;
    static_assert(NPL <= 64, "mask bits");
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = sub + a.lanes * i;
        const bool in = group < a.n_groups && e < a.size;
        s[i] = in ? (double)to_f32(lr[base + e]) : -INFINITY;
        c[i] = in && a.bias ? (double)a.bias[base + e] : 0.0;
        if (isnan(s[i])) s[i] = -INFINITY;
        if (s[i] == -INFINITY || isnan(c[i]) || c[i] == -INFINITY) masked |= 1ull << i;
    }
    if (a.softmax) {
        double top = -INFINITY, sum = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) top = fmax(top, s[i]);
        top = warp_max(top);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            s[i] = s[i] == -INFINITY ? 0.0 : s[i] == top ? 1.0 : exp(s[i] - top);
            sum += s[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] = sum > 0 ? s[i] / sum : 0.0;
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] = 1.0 / (1.0 + exp(-s[i]));
    }
    double m1 = kMasked, m2 = kMasked;            // the two largest unmasked of this lane, then of the group
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = sub + a.lanes * i;
        const bool in = group < a.n_groups && e < a.size;
        c[i] = !in ? kGone : (masked >> i & 1) ? kMasked : s[i] + c[i];
        if ((masked >> i & 1)) s[i] = 0;
        if (c[i] > m1) { m2 = m1; m1 = c[i]; }
        else if (c[i] > m2) m2 = c[i];
    }
    if (a.topk_groups < a.n_groups) {
        for (int o = 1; o < a.lanes; o <<= 1) {
            const double p1 = __shfl_xor_sync(0xffffffffu, m1, o), p2 = __shfl_xor_sync(0xffffffffu, m2, o);
            m2 = fmax(fmin(m1, p1), m1 > p1 ? m2 : p2);
            m1 = fmax(m1, p1);
        }
        const double score = a.top2 && m2 != kMasked ? m1 + m2 : m1;
        int before = 0;                           // groups that come before this one
        for (int g = 0; g < a.n_groups; ++g) {
            const double o = __shfl_sync(0xffffffffu, score, g * a.lanes);
            before += o > score || (o == score && g < group);
        }
        if (before >= a.topk_groups)
#pragma unroll
            for (int i = 0; i < NPL; ++i) c[i] = kGone;
    }
    double sel = 0, sum = 0;                      // lane k keeps choice k
    int chosen = 0;
    for (int k = 0; k < a.K; ++k) {
        double bc = kGone, bs = 0;
        int be = INT_MAX;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (c[i] > bc) { bc = c[i]; be = base + sub + a.lanes * i; bs = s[i]; }
        const double top = warp_max(bc);
        const int e = __reduce_min_sync(0xffffffffu, bc == top ? be : INT_MAX);
        const int owner = __ffs(__ballot_sync(0xffffffffu, bc == top && be == e)) - 1;
        bs = __shfl_sync(0xffffffffu, bs, owner);
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (base + sub + a.lanes * i == e && lane == owner) c[i] = kGone;
        if (lane == k) { sel = bs; chosen = e; }
        sum += bs;
    }
    if (lane < a.K) {
        if (a.renormalise) sel = sum > 0 ? sel / sum : 0.0;
        a.idx[(size_t)t * a.K + lane] = chosen;
        a.w[(size_t)t * a.K + lane] = (float)(sel * (double)a.scale);
        if (a.hist) atomicAdd(a.hist + (size_t)(t / kChunk) * a.E + chosen, 1);   // whole numbers: exact in any order
    }
}

template <class LT>
static kmoe_status run_route(const LT *logits, const RouteArgs &a, cudaStream_t st)
{
    const int grid = (a.N + kRouteTokens - 1) / kRouteTokens, npl = (a.size + a.lanes - 1) / a.lanes;
#define KMOE_ROUTE(n) launch_pdl(route_kernel<LT, n>, grid, 32 * kRouteTokens, 0, st, logits, a)
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
    if (l_dtype == KMOE_F32) return run_route(static_cast<const float *>(logits), a, st);
    return run_route(static_cast<const __nv_bfloat16 *>(logits), a, st);
}

}  // namespace kmoe
