// Choice of experts by score: softmax or sigmoid scores, a bias that only the
// choice sees, groups of experts of which the best stay, the k best experts of
// those, weights renormalised and scaled.
//
// One warp takes one token; lane l holds experts l, l + 32, ...  Whether a
// choice is made is decided by the exact values: where neither a bias nor a
// sum of two scores is involved, scores are compared through the logits, whose
// order they have; else they are computed in fp32 with a bound on their error,
// and where two values that the result depends on (neighbours among the chosen
// experts, the last chosen and the first left out, the same two groups) are not
// further apart than that, the token is chosen again with scores in fp64.
#include <limits.h>

#include "common.cuh"

namespace moe {
namespace {

constexpr unsigned ALL = 0xffffffffu;
constexpr int WARPS = 4;

struct ScoredArgs {
    const float *logits, *bias;
    int32_t* ids;
    float* weights;
    float scale;
    int T, E, k, sigmoid, renorm, groups, top_groups, group_top;
    int size;   // experts of a group
    int magic;  // ceil(2^20 / size): e / size = e * magic >> 20 below 1024
};

// Order-preserving keys: 0 = absent, 1 = NaN, then -infinity .. infinity
// (-0 as +0).  value() is the inverse (of a key above 1).
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    if (v != v) return 1u;
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k); }
__device__ __forceinline__ uint64_t key_of(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    if (v != v) return 1u;
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double value_of(uint64_t k) {
    return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(ALL, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
    const uint32_t hi = __reduce_max_sync(ALL, (uint32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(ALL, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (uint64_t)hi << 32 | lo;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(ALL, v, off);
    return v;
}

template <typename Key>
struct Chosen {
    Key key;  // lane j < k: the j-th best choice
    int id;
    Key left;     // the best one left out (0: none)
    Key in, out;  // groups: the worst that stays, the best that does not (0: none)
};

// The choice itself, among c[i] = the choice value of expert lane + 32 i.
// room: E values of the warp's own in shared memory (groups > 1).
template <int NPER, typename F, typename Key>
__device__ __forceinline__ Chosen<Key> choose(const F (&c)[NPER], const ScoredArgs& a, F* room) {
    const int lane = threadIdx.x & 31;
    Chosen<Key> r;
    r.in = r.out = 0;
    uint32_t stay = ALL;
    int per = 32;  // lanes to a group
    if (a.groups > 1) {
        while (per * a.groups > 32) per >>= 1;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (lane + 32 * i < a.E) room[lane + 32 * i] = c[i];
        __syncwarp();
        const int g = lane / per;
        Key b1 = 0, b2 = 0;
        if (g < a.groups)
            for (int m = lane % per; m < a.size; m += per) {
                const Key k = key_of(room[g * a.size + m]);
                b2 = max(b2, min(b1, k));
                b1 = max(b1, k);
            }
        __syncwarp();
        for (int off = 1; off < per; off <<= 1) {
            const Key o1 = __shfl_xor_sync(ALL, b1, off), o2 = __shfl_xor_sync(ALL, b2, off);
            b2 = max(max(b2, o2), min(b1, o1));
            b1 = max(b1, o1);
        }
        // (a NaN among a group's best makes its sum one, and ranks it last)
        Key mine = b1;
        if (a.group_top == 2) mine = b1 > 1 && b2 > 1 ? key_of(value_of(b1) + value_of(b2)) : (Key)1;
        if (g >= a.groups) mine = 0;
        int rank = 0;
        for (int o = 0; o < a.groups; ++o) {
            const Key k = __shfl_sync(ALL, mine, o * per);
            rank += k > mine || (k == mine && o < g);
        }
        const bool stays = g < a.groups && rank < a.top_groups;
        stay = __ballot_sync(ALL, stays);
        r.in = ~warp_max(stays ? (Key)~mine : (Key)0);
        r.out = warp_max(stays ? (Key)0 : mine);
    }
    Key key[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        const int e = lane + 32 * i;
        const bool in = e < a.E && (a.groups == 1 || (stay >> ((e * a.magic >> 20) * per) & 1));
        key[i] = in ? key_of(c[i]) : (Key)0;
    }
    Key best = 0;
    int be = INT_MAX;
    auto rescan = [&]() {
        best = 0, be = INT_MAX;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (key[i] > best) best = key[i], be = lane + 32 * i;  // (of equal ones the lowest number)
    };
    rescan();
    r.key = 0, r.id = 0;
    for (int j = 0; j < a.k; ++j) {
        const Key most = warp_max(best);
        const int e = __reduce_min_sync(ALL, best == most ? be : INT_MAX);
        if (lane == j) r.key = most, r.id = e;
        if ((e & 31) == lane) {
#pragma unroll
            for (int i = 0; i < NPER; ++i)
                if (e == lane + 32 * i) key[i] = 0;
            rescan();
        }
    }
    r.left = warp_max(best);
    return r;
}

template <int NPER, typename F>
__device__ __forceinline__ void scores(const float (&l)[NPER], float top, const ScoredArgs& a, F (&c)[NPER]) {
    const int lane = threadIdx.x & 31;
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NPER; ++i) c[i] = F(1) / (F(1) + exp(-F(l[i])));
    } else {
        F sum = 0;
#pragma unroll
        for (int i = 0; i < NPER; ++i) {
            c[i] = lane + 32 * i < a.E ? exp(F(l[i]) - F(top)) : F(0);
            sum += c[i];
        }
        sum = warp_sum(sum);
#pragma unroll
        for (int i = 0; i < NPER; ++i) c[i] /= sum;
    }
    if (a.bias)
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (lane + 32 * i < a.E) c[i] += F(__ldg(a.bias + lane + 32 * i));
}

// The same choice with scores in fp64 (rare: kept out of the kernel's registers).
template <int NPER>
__device__ __noinline__ int choose_exactly(const float* logits, float top, const ScoredArgs& a, double* room) {
    const int lane = threadIdx.x & 31;
    float l[NPER];
    double c[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) l[i] = lane + 32 * i < a.E ? logits[lane + 32 * i] : 0.0f;
    scores<NPER, double>(l, top, a, c);
    return choose<NPER, double, uint64_t>(c, a, room).id;
}

template <int NPER>
__global__ void __launch_bounds__(32 * WARPS) route_scored_kernel(const __grid_constant__ ScoredArgs a) {
    extern __shared__ __align__(16) double room[];
    pdl_wait();
    pdl_launch_dependents();  // dependents may start their prologues now
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * WARPS + warp;
    if (t >= a.T) return;
    double* own = room + (size_t)warp * a.E;
    const float* logits = a.logits + t * a.E;
    float l[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) l[i] = lane + 32 * i < a.E ? logits[lane + 32 * i] : -INFINITY;

    float top = 0.0f, sum = 1.0f;
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < NPER; ++i)
        if (lane + 32 * i < a.E) most = max(most, key_of(l[i]));
    most = warp_max(most);
    top = most > 1 ? value_of(most) : NAN;
    if (!a.sigmoid) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (lane + 32 * i < a.E) sum += expf(l[i] - top);
        sum = warp_sum(sum);
    }
    auto score = [&](float v) { return a.sigmoid ? 1.0f / (1.0f + expf(-v)) : expf(v - top) / sum; };

    int id;
    const bool by_logit = !a.bias && (a.groups == 1 || a.group_top == 1);
    if (by_logit) {
        id = choose<NPER, float, uint32_t>(l, a, reinterpret_cast<float*>(own)).id;
    } else {
        float c[NPER];
        uint32_t large = 0;  // the largest finite magnitude's bits
#pragma unroll
        for (int i = 0; i < NPER; ++i) {
            c[i] = score(l[i]) + (a.bias && lane + 32 * i < a.E ? __ldg(a.bias + lane + 32 * i) : 0.0f);
            const uint32_t m = __float_as_uint(c[i]) & 0x7fffffffu;
            if (m < 0x7f800000u) large = max(large, m);
        }
        large = warp_max(large);
        const Chosen<uint32_t> r = choose<NPER, float, uint32_t>(c, a, reinterpret_cast<float*>(own));
        id = r.id;
        // A score is off by less than 2^-20 of the row's largest: expf and the
        // division by 4 units of 2^-24 each at most, the softmax' sum of up to 32
        // terms a lane and 5 rounds by less than 2^-18, which moves all of a
        // row's scores by one factor.  The bias' addition and a group's sum round
        // by 2^-24 of a choice each.  Twice that for a difference, and some.
        const float near = (a.sigmoid ? 0x1p-18f : 0x1p-16f) * score(top) + 0x1p-21f * __uint_as_float(large);
        const float v = value_of(r.key), after = __shfl_down_sync(ALL, v, 1);
        bool unsure = lane < a.k && !(v - (lane + 1 < a.k ? after : value_of(r.left)) > near);
        if (lane == a.k - 1 && r.left == 0) unsure = false;
        if (r.out != 0) unsure |= !(value_of(r.in) - value_of(r.out) > 2.0f * near);
        if (__any_sync(ALL, unsure)) id = choose_exactly<NPER>(logits, top, a, own);
    }
    float w = lane < a.k ? score(logits[id]) : 0.0f;
    if (a.renorm) w /= warp_sum(w) + 1e-20f;
    if (lane < a.k) {
        a.ids[t * a.k + lane] = id;
        a.weights[t * a.k + lane] = w * a.scale;
    }
}

moe_status launch_route_scored(const ScoredArgs& a, cudaStream_t s) {
    const dim3 grid((unsigned)((a.T + WARPS - 1) / WARPS));
    const size_t smem = sizeof(double) * WARPS * a.E;  // (at most 32 KB)
    auto kern = a.E <= 32    ? route_scored_kernel<1>
                : a.E <= 64  ? route_scored_kernel<2>
                : a.E <= 128 ? route_scored_kernel<4>
                : a.E <= 256 ? route_scored_kernel<8>
                : a.E <= 512 ? route_scored_kernel<16>
                             : route_scored_kernel<32>;
    cudaError_t e = launch_pdl(kern, grid, dim3(32 * WARPS), smem, s, a);
    return e == cudaSuccess ? MOE_OK : cuda_status(e, "moe_route_scored: launch");
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_route_scored(const float* logits, int T, int E, int k, const moe_scoring* s, int32_t* ids, float* weights,
                            cudaStream_t stream) {
    MOE_CHECK_ARG(s, "moe_route_scored: scoring is null");
    MOE_CHECK_ARG(T >= 0 && E > 0, "moe_route_scored: T=%d E=%d", T, E);
    MOE_CHECK_SUPPORTED(E <= 1024, "moe_route_scored: E=%d above 1024", E);
    MOE_CHECK_ARG(s->scoring == MOE_SCORE_SOFTMAX || s->scoring == MOE_SCORE_SIGMOID, "moe_route_scored: unknown scoring %d",
                  s->scoring);
    MOE_CHECK_ARG(s->renormalize == 0 || s->renormalize == 1, "moe_route_scored: renormalize must be 0 or 1");
    MOE_CHECK_ARG(s->scale - s->scale == 0.0f, "moe_route_scored: scale must be finite");
    MOE_CHECK_ARG(s->groups >= 1 && s->groups <= E && E % s->groups == 0, "moe_route_scored: groups=%d must divide E=%d",
                  s->groups, E);
    MOE_CHECK_SUPPORTED(s->groups <= 32, "moe_route_scored: groups=%d above 32", s->groups);
    const int size = E / s->groups;
    MOE_CHECK_ARG(s->top_groups >= 1 && s->top_groups <= s->groups, "moe_route_scored: top_groups=%d must be in [1, groups=%d]",
                  s->top_groups, s->groups);
    MOE_CHECK_ARG((s->group_top == 1 || s->group_top == 2) && s->group_top <= size,
                  "moe_route_scored: group_top=%d must be 1 or 2, and no more than a group's %d experts", s->group_top, size);
    MOE_CHECK_ARG(k >= 1 && k <= 32 && k <= s->top_groups * size,
                  "moe_route_scored: k=%d must be in [1, min(32, the %d experts of top_groups)]", k, s->top_groups * size);
    if (T == 0) return MOE_OK;
    MOE_CHECK_ARG(logits && ids && weights, "moe_route_scored: null pointer");
    MOE_CHECK_SUPPORTED((((uintptr_t)logits | (uintptr_t)s->bias | (uintptr_t)ids | (uintptr_t)weights) & 3) == 0,
                        "moe_route_scored: a pointer is not aligned to its type");
    ScoredArgs a = {};
    a.logits = logits, a.bias = s->bias, a.ids = ids, a.weights = weights, a.scale = s->scale, a.T = T, a.E = E, a.k = k;
    a.sigmoid = s->scoring == MOE_SCORE_SIGMOID, a.renorm = s->renormalize, a.groups = s->groups;
    a.top_groups = s->top_groups, a.group_top = s->group_top, a.size = size, a.magic = ((1 << 20) + size - 1) / size;
    return launch_route_scored(a, stream);
}

}  // extern "C"
