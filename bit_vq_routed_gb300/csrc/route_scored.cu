// Choice of experts by score: softmax or sigmoid scores, a bias that only the
// choice sees, groups of experts of which the best stay, the k best experts of
// those, weights renormalised and scaled.
//
// One warp takes one token.  Each group belongs to 32 / (groups, rounded up to a
// power of two) lanes, each of which holds a run of the group's experts in
// registers, so that a group's best need a few shuffles and a group that goes
// takes its lanes with it.
//
// The k best: a value that at least k experts reach comes from the lanes' own
// best, k rounds of a warp-wide maximum; the experts that reach it, seldom many
// more than k, move to one lane each, and every lane counts those ahead of its
// own.
//
// The choice is that of the exact values.  Where neither a bias nor a sum of two
// scores is involved, scores are compared through the logits, whose order they
// have; else they are computed in fp32 with a bound on their error, and where
// two values that the result depends on are not further apart than that, the
// few experts that may be among the k best, or among a group's best two, are
// compared again: in pairs of fp32 numbers first, and what those cannot tell apart in
// fp64.
//
// Instructions bound it, not the logits' 8 MB (8192 tokens of 256 experts in 8 groups
// with a bias: 8.5 us, 730 instructions a token, 8 of 10 schedulers' slots while all
// run; without groups and bias 5.1; one token 2.6, of which 2 are the launch).  The
// first form, k rounds of a maximum over all with a new search in the winner's lane and
// fp64 for a whole token, took 28.
#include <limits.h>

#include <type_traits>

#include "permute.cuh"

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
    int per, log_per;  // lanes of a group: a power of two
    int chunk;  // experts of a lane
    int vec;    // whether a lane's experts can be loaded four by four
    int room;   // doubles of shared memory a warp has
};

// Order-preserving keys: 0 = absent, 1 = NaN, then -infinity .. infinity
// (-0 as +0).  value_of() is the inverse (NaN for 0 and 1).
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return v != v ? 1u : u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
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
// exp(-v) and 1 / v by the special function unit: off by 2^-22 of the value, and
// the first by 2^-24 of it for each unit of v log2(e) too
__device__ __forceinline__ float quick_exp_neg(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * -1.4426950408889634f));
    return r;
}
__device__ __forceinline__ float quick_rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(ALL, v, off);
    return v;
}

// Which groups stay, from the two largest keys that each lane saw of its group:
// true in the lanes of those.  in, out: the rank value of the worst that stays
// and of the best that goes (0: none goes).
template <typename Key>
__device__ __forceinline__ bool group_stays(const ScoredArgs& a, Key& b1, Key& b2, Key& in, Key& out) {
    const int lane = threadIdx.x & 31, g = lane >> a.log_per;
    for (int off = 1; off < a.per; off <<= 1) {
        const Key o1 = __shfl_xor_sync(ALL, b1, off), o2 = __shfl_xor_sync(ALL, b2, off);
        b2 = max(max(b2, o2), min(b1, o1));
        b1 = max(b1, o1);
    }
    // (a NaN among a group's best makes its sum one, and ranks it last)
    Key mine = b1;
    if (a.group_top == 2) mine = b1 > 1 && b2 > 1 ? key_of(value_of(b1) + value_of(b2)) : (Key)1;
    if (g >= a.groups) mine = 0;
    // the top_groups-th largest: that many rounds of a maximum, equal ones together
    Key left = (lane & (a.per - 1)) == 0 ? mine : 0;
    in = 0;
#pragma unroll 2
    for (int j = 0; j < a.top_groups; ++j) {
        in = warp_max(left);
        if (left == in) left = 0;
    }
    bool stays = mine >= in && mine != 0;
    out = warp_max(stays ? (Key)0 : mine);
    if (__popc(__ballot_sync(ALL, stays)) != a.top_groups * a.per) {
        // equal ones on both sides of the border: by their numbers
        int rank = 0;
#pragma unroll 1
        for (int o = 0; o < a.groups; ++o) {
            const Key k = __shfl_sync(ALL, mine, o * a.per);
            rank += k > mine || (k == mine && o < g);
        }
        stays = g < a.groups && rank < a.top_groups;
        in = ~warp_max(stays ? (Key)~mine : (Key)0);
        out = warp_max(stays ? (Key)0 : mine);
    }
    return stays;
}

// An expert's choice value in fp64; total: the softmax' sum.  (Rare work: kept out
// of the kernel's registers.)
__device__ __noinline__ double choice64(const ScoredArgs& a, float l, float top, int e, double total) {
    const double x = exp(a.sigmoid ? -(double)l : (double)l - (double)top);
    const double s = a.sigmoid ? 1.0 / (1.0 + x) : x / total;
    return a.bias ? s + (double)a.bias[e] : s;
}

// exp(u + ul) = (z + zl) 2^n in pairs of fp32 numbers (a value and what its rounding
// left), |u| <= 80, |ul| at most u's rounding: off by less than 2^-28 of it.  (fp64
// arithmetic comes at a 64th of the rate.)
//   u = n ln 2 + r (Cody and Waite's way: n 355/512 comes off exactly, the rest of ln
//   2 in two pieces), exp(r) = 1 + r + r^2/2 as pairs and the series from r^3/6 on in
//   fp32.
__device__ __forceinline__ void exp_pair(float u, float ul, float& z, float& zl, float& two_n) {
    const float n = rintf(u * 1.4426950408889634f);
    const float r1 = fmaf(n, -0x1.63p-1f, u);
    const float p = __fmul_rn(n, -0x1.bd0106p-13f), pe = fmaf(n, -0x1.bd0106p-13f, -p);
    const float r = __fsub_rn(r1, p), back = __fsub_rn(r, r1);
    const float rl = __fsub_rn(__fsub_rn(r1, __fsub_rn(r, back)), __fadd_rn(p, back)) - pe - n * 0x1.cf79acp-40f + ul;
    const float h = __fmul_rn(r, r), hl = fmaf(r, r, -h);
    float q = 1.0f / 40320;
    q = fmaf(q, r, 1.0f / 5040);
    q = fmaf(q, r, 1.0f / 720);
    q = fmaf(q, r, 1.0f / 120);
    q = fmaf(q, r, 1.0f / 24);
    q = fmaf(q, r, 1.0f / 6) * h * r;
    const float x = __fadd_rn(1.0f, r), xl = __fsub_rn(r, __fsub_rn(x, 1.0f));
    const float y = __fadd_rn(x, 0.5f * h), yl = __fsub_rn(0.5f * h, __fsub_rn(y, x));
    const float low = ((0.5f * hl + rl * (y + q)) + (xl + yl)) + q;
    z = __fadd_rn(y, low), zl = __fsub_rn(low, __fsub_rn(z, y));
    two_n = __int_as_float(((int)n + 127) << 23);
}
// A softmax' term exp(l - top).
__device__ __noinline__ double term_fine(float l, float top) {
    const float u = __fsub_rn(l, top), back = __fsub_rn(u, l);
    const float ul = __fsub_rn(__fsub_rn(l, __fsub_rn(u, back)), __fadd_rn(top, back));
    float z, zl, two_n;
    exp_pair(fmaxf(u, -80.0f), u >= -80.0f ? ul : 0.0f, z, zl, two_n);
    const double e = ((double)z + (double)zl) * (double)two_n;
    return u == u ? e : (double)u;
}
// A choice value by these (inv: 1 / the softmax' sum, or 1).  A sigmoid is t = 1 / (1 +
// exp(|v|)), with one correction by its remainder, or 1 - t where v > 0; off by less
// than 2^-30 (on 420000 values t by 2^-31.3), a softmax' term by 2^-28 of itself.
__device__ __noinline__ double choice_fine(const ScoredArgs& a, float v, float top, int e, double inv) {
    double c;
    if (a.sigmoid) {
        float z, zl, two_n;
        exp_pair(fminf(fabsf(v), 80.0f), 0.0f, z, zl, two_n);  // (t is 2^-115 there)
        const float big = z * two_n;
        const float d = __fadd_rn(big, 1.0f), dl = fmaf(zl, two_n, __fsub_rn(1.0f, __fsub_rn(d, big)));
        const float t = __frcp_rn(d), tl = t * fmaf(-t, dl, fmaf(-t, d, 1.0f));
        c = (double)t + (double)tl;
        if (v > 0.0f) c = 1.0 - c;
        if (v != v) c = (double)v;
    } else {
        c = term_fine(v, top) * inv;
    }
    return a.bias ? c + (double)a.bias[e] : c;
}
// 1 / the softmax' sum that goes with them (1 where only the order counts).
__device__ __noinline__ double inverse_fine(const ScoredArgs& a, const float* logits, float top) {
    if (a.sigmoid || !a.bias) return 1.0;
    double total = 0.0;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < a.E; e += 32) total += term_fine(logits[e], top);
    return 1.0 / warp_sum(total);
}
// How far two of those may be off against one another: a softmax' by its terms and
// the common factor's share of their difference (over: its largest score, 1 without a
// factor).
__device__ __forceinline__ double fine_margin(const ScoredArgs& a, float over) {
    return a.sigmoid ? 0x1p-29 : 0x1p-26 * (a.bias ? (double)over : 1.0);
}

// The sum that a softmax with a bias needs for them (without one only the order
// counts, and 1 will do).
__device__ __noinline__ double sum64(const ScoredArgs& a, const float* logits, float top) {
    if (a.sigmoid || !a.bias) return 1.0;
    double total = 0.0;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < a.E; e += 32) total += exp((double)logits[e] - (double)top);
    return warp_sum(total);
}

// The whole choice in fp64, by loops over shared memory (rare, and kept small:
// its instructions come from memory).  Lane j < k gets the j-th expert.
__device__ __noinline__ int choose_exactly(const ScoredArgs& a, const float* logits, float top, double* room) {
    const int lane = threadIdx.x & 31;
    const double total = sum64(a, logits, top);
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32) room[e] = choice64(a, logits[e], top, e, total);
    __syncwarp();
    uint32_t stay = ALL;
    if (a.groups > 1) {
        uint64_t b1 = 0, b2 = 0, in, out;
        const int g = lane >> a.log_per;
        if (g < a.groups)
#pragma unroll 1
            for (int m = lane & (a.per - 1); m < a.size; m += a.per) {
                const uint64_t k = key_of(room[g * a.size + m]);
                b2 = max(b2, min(b1, k));
                b1 = max(b1, k);
            }
        stay = __ballot_sync(ALL, group_stays(a, b1, b2, in, out));
    }
    uint32_t gone = 0;  // bit i: expert lane + 32 i is out or taken
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32)
        if (!(stay >> (e / a.size * a.per) & 1)) gone |= 1u << (e >> 5);
    uint64_t best = 0;
    int be = INT_MAX, id = 0;
    bool search = true;
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
        if (search) {
            best = 0, be = INT_MAX;
#pragma unroll 1
            for (int e = lane; e < a.E; e += 32) {
                const uint64_t k = gone >> (e >> 5) & 1 ? 0 : key_of(room[e]);
                if (k > best) best = k, be = e;
            }
        }
        const uint64_t most = warp_max(best);
        const int e = __reduce_min_sync(ALL, best == most ? be : INT_MAX);
        if (lane == j) id = e;
        search = e == be;
        if (search) gone |= 1u << (e >> 5);
    }
    __syncwarp();
    return id;
}

template <int NPER>
__device__ __forceinline__ void load_run(const float* p, int count, bool vec, float (&v)[NPER]) {
    if (NPER >= 4 && vec) {
#pragma unroll
        for (int i = 0; i < NPER; i += 4) {
            const float4 f = i < count ? *reinterpret_cast<const float4*>(p + i) : make_float4(0, 0, 0, 0);
            v[i] = f.x, v[(i + 1) % NPER] = f.y, v[(i + 2) % NPER] = f.z, v[(i + 3) % NPER] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPER; ++i) v[i] = i < count ? p[i] : 0.0f;
    }
}

// One token by one warp; own: its part of the shared memory.  Lane j < k returns
// the j-th expert.
template <int NPER>
__device__ __forceinline__ int choose_token(const ScoredArgs& a, int64_t t, double* own) {
    const int lane = threadIdx.x & 31;
    uint32_t* keys = reinterpret_cast<uint32_t*>(own);  // 32, and their experts
    int* experts = reinterpret_cast<int*>(own) + 32;
    double* values = own + 32;  // 32 and one that is not used
    const float* logits = a.logits + t * a.E;
    const int g = lane >> a.log_per, at = (lane & (a.per - 1)) * a.chunk, first = g * a.size + at;
    const int count = g < a.groups ? min(a.chunk, a.size - at) : 0;  // (below 1: none)
    float c[NPER];  // logits, then the choice values
    load_run<NPER>(logits + first, count, a.vec, c);
    // (NaN where one of the lane's logits is: a NaN ranks last and may leave no trace among
    // the chosen, but makes all of the token's weights NaN, as by itself in a softmax' sum)
    float lost = 0.0f;
#pragma unroll
    for (int i = 0; i < NPER; ++i) lost += fabsf(c[i]);

    // A softmax' largest logit and sum.
    float top = 0.0f, over = 1.0f;
    if (!a.sigmoid) {
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (i < count) most = max(most, key_of(c[i]));
        top = value_of(warp_max(most));
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (i < count) sum += expf(c[i] - top);
        over = 1.0f / warp_sum(sum);
    }
    auto score = [&](float v) {
        return a.sigmoid ? quick_rcp(1.0f + quick_exp_neg(v)) : expf(v - top) * over;
    };
    const bool by_logit = !a.bias && (a.groups == 1 || a.group_top == 1);
    // How far two choices may be off against one another, but for |choice| 2^-22
    // (the bias' addition).  A sigmoid s is off by less than 2^-21: s (1 - s) <= 1/4
    // times the exponential's 2^-22, |v| s (1 - s) < 1/4 times the 2^-23.4 of its
    // argument, the sum's 2^-24 and the quotient's 2^-23.  A softmax' term is off by
    // 2^-21 of the row's largest score, and all of them by one factor, the sum's
    // error of one unit of 2^-24 a term and round.
    const float near = by_logit ? 0.0f : a.sigmoid ? 0x1p-20f : over * (0x1p-20f + (NPER + 8) * 0x1p-23f);
    if (!by_logit) {
        float b[NPER];
        if (a.bias) load_run<NPER>(a.bias + first, count, a.vec, b);
#pragma unroll
        for (int i = 0; i < NPER; ++i) {
            c[i] = score(c[i]);
            if (a.bias) c[i] += b[i];
        }
    }
    uint32_t key[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) key[i] = i < count ? key_of(c[i]) : 0u;

    uint32_t best = 0;  // of the lane
    if (a.groups > 1) {
        uint32_t b1 = 0, b2 = 0, in, out;
#pragma unroll
        for (int i = 0; i < NPER; ++i) {
            b2 = max(b2, min(b1, key[i]));
            b1 = max(b1, key[i]);
        }
        best = b1;
        bool stays = group_stays(a, b1, b2, in, out);
        if (!by_logit && out != 0) {
            // (without a bias a score's bound; else the largest finite magnitude
            // of what the ranks are made of)
            float large = a.sigmoid ? 1.0f : over;
            if (a.bias) {
                uint32_t m1 = __float_as_uint(value_of(b1)) & 0x7fffffffu, m2 = __float_as_uint(value_of(b2)) & 0x7fffffffu;
                m1 = max(m1 < 0x7f800000u ? m1 : 0u, m2 < 0x7f800000u ? m2 : 0u);
                large = __uint_as_float(warp_max(m1));
            }
            if (!(value_of(in) - value_of(out) > 2.0f * near + 0x1p-20f * large)) {
                // the groups again, by closer values of the experts that may be their
                // best two
                const float v = value_of(a.group_top == 2 ? b2 : b1);
                const uint32_t least = key_of(v - (near + 0x1p-22f * fabsf(v)));
                uint64_t open = 0;
#pragma unroll
                for (int i = 0; i < NPER; ++i) open |= (uint64_t)(key[i] >= max(least, 1u)) << i;
                auto stays_by = [&](auto value, double& margin) {
                    uint64_t d1 = 0, d2 = 0, din, dout;
#pragma unroll 1
                    for (uint64_t left = open; left != 0; left &= left - 1) {
                        const int e = first + __ffsll((long long)left) - 1;
                        const uint64_t k = key_of(value(e));
                        d2 = max(d2, min(d1, k));
                        d1 = max(d1, k);
                    }
                    __syncwarp();
                    const bool r = group_stays(a, d1, d2, din, dout);
                    margin = value_of(din) - value_of(dout);
                    return r;
                };
                double margin = 0.0;
                const double inv = inverse_fine(a, logits, top);
                stays = stays_by([&](int e) { return choice_fine(a, logits[e], top, e, inv); }, margin);
                if (!(margin > 2.0 * fine_margin(a, over) + 0x1p-44 * large)) {
                    const double total = sum64(a, logits, top);
                    stays = stays_by([&](int e) { return choice64(a, logits[e], top, e, total); }, margin);
                }
            }
        }
        if (!stays) {
            best = 0;
#pragma unroll
            for (int i = 0; i < NPER; ++i) key[i] = 0;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPER; ++i) best = max(best, key[i]);
    }

    int id = 0;
    // k experts reach `least`, and so does what may come ahead of them
    uint32_t least = 0, left = best;
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
        least = warp_max(left);
        if (left == least) left = 0;
    }
    if (near > 0.0f && least > 1u) {
        const float v = value_of(least);
        least = key_of(v - (near + 0x1p-22f * fabsf(v)));
    }
    least = max(least, 1u);
    keys[lane] = 0;
    __syncwarp();
    int pos = 0, n;
#pragma unroll
    for (int i = 0; i < NPER; ++i) pos += key[i] >= least;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int below = __shfl_up_sync(ALL, pos, off);
        if (lane >= off) pos += below;
    }
    n = __shfl_sync(ALL, pos, 31);
    if (n <= 32) {
#pragma unroll
        for (int i = NPER - 1; i >= 0; --i)
            if (key[i] >= least) --pos, keys[pos] = key[i], experts[pos] = first + i;
    }
    __syncwarp();
    if (n <= 32) {
        const uint32_t k = keys[lane];
        const int e = lane < n ? experts[lane] : INT_MAX;
        int rank = 0;
        for (int j = 0; j < n; j += 4) {
            const uint4 o = *reinterpret_cast<const uint4*>(keys + j);
            rank += o.x > k;
            rank += o.y > k;
            rank += o.z > k;
            rank += o.w > k;
        }
        // (the ranks' sum is that of 0 .. n - 1 unless there are equal keys)
        const auto by_number = [&](auto own_key) {
            int r = 0;
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                const auto o = __shfl_sync(ALL, own_key, j);
                const int oe = __shfl_sync(ALL, e, j);
                r += o > own_key || (o == own_key && oe < e);
            }
            return r;
        };
        if (__reduce_add_sync(ALL, lane < n ? rank : 0) != n * (n - 1) / 2) rank = by_number(k);
        __syncwarp();
        if (lane < n) keys[rank] = k, experts[rank] = e;
        __syncwarp();
        id = lane < a.k ? experts[lane] : 0;
        const float v = value_of(keys[lane]), after = value_of(keys[min(lane + 1, 31)]);
        const bool close = near > 0.0f && lane < min(a.k, n - 1) && !(v - after > near + 0x1p-22f * fabsf(v));
        if (__any_sync(ALL, close)) {
            const double fine = fine_margin(a, over);
            auto order_by = [&](auto value) {  // whether two neighbours come too close
                const double d = lane < n ? value() : 0.0;
                rank = by_number(lane < n ? key_of(d) : (uint64_t)0);
                __syncwarp();
                if (lane < n) experts[rank] = e, values[rank] = d;
                __syncwarp();
                id = lane < a.k ? experts[lane] : 0;
                const double w = values[lane];
                return __any_sync(ALL, lane < min(a.k, n - 1) && !(w - values[lane + 1] > fine + 0x1p-45 * fabs(w)));
            };
            const double inv = inverse_fine(a, logits, top);
            if (order_by([&] { return choice_fine(a, logits[e], top, e, inv); })) {
                const double total = sum64(a, logits, top);
                order_by([&] { return choice64(a, logits[e], top, e, total); });
            }
        }
    } else {
        // many equal ones, or a k of many: one after another
        int be = INT_MAX;
        uint32_t mine = 0;
        auto search = [&]() {
            best = 0, be = INT_MAX;
#pragma unroll
            for (int i = 0; i < NPER; ++i)
                if (key[i] > best) best = key[i], be = first + i;  // (of equal ones the lowest number)
        };
        search();
        for (int j = 0; j < a.k; ++j) {
            const uint32_t most = warp_max(best);
            const int e = __reduce_min_sync(ALL, best == most ? be : INT_MAX);
            if (lane == j) mine = most, id = e;
            if (e == be) {
#pragma unroll
                for (int i = 0; i < NPER; ++i)
                    if (e == first + i) key[i] = 0;
                search();
            }
        }
        const uint32_t rest = warp_max(best);
        const float v = value_of(mine), after = __shfl_down_sync(ALL, v, 1);
        const float next = lane + 1 < a.k ? after : value_of(rest);
        const bool close = near > 0.0f && (lane + 1 < a.k || (lane + 1 == a.k && rest != 0)) &&
                 !(v - next > near + 0x1p-22f * fabsf(v));
        if (__any_sync(ALL, close)) id = choose_exactly(a, logits, top, own);
    }
    const float l = lane < a.k ? logits[id] : 0.0f;
    float w = lane < a.k ? (a.sigmoid ? __fdividef(1.0f, 1.0f + expf(-l)) : expf(l - top) * over) : 0.0f;
    if (lost != lost) w = lost;
    if (a.renorm)
        w = __fdividef(w, warp_sum(w) + 1e-20f);
    else if (__any_sync(ALL, lost != lost))
        w = __int_as_float(0x7fffffff);
    if (lane < a.k) {
        a.ids[t * a.k + lane] = id;
        a.weights[t * a.k + lane] = w * a.scale;
    }
    return id;
}

template <int NPER>
__global__ void __launch_bounds__(32 * WARPS) route_scored_kernel(const __grid_constant__ ScoredArgs a) {
    extern __shared__ __align__(16) double room[];
    pdl_wait();
    pdl_launch_dependents();  // dependents may start their prologues now
    const int warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * WARPS + warp;
    if (t < a.T) choose_token<NPER>(a, t, room + (size_t)warp * a.room);
}

// Few tokens: one block, which then also sorts the pairs by expert as moe_permute
// does (a pair's place: the pairs of lower experts, and those ahead of it of its own).
// Up to T E = 5120 (40 KB): above, the permutation's own kernel is as fast or faster (8
// tokens of 1024 experts, k = 8: 17.9 in one and 18.1, k = 32: 36.5 and 29.5).
constexpr int FEW_T = 8;
constexpr size_t FEW_SMEM = 40 * 1024;

template <int NPER>
__global__ void __launch_bounds__(32 * FEW_T) route_scored_few_kernel(const __grid_constant__ ScoredArgs a,
                                                                      int32_t* offsets, int32_t* sorted_pair,
                                                                      int32_t* pair_to_sorted) {
    extern __shared__ __align__(16) double room[];
    __shared__ int ids[FEW_T * 32];
    pdl_wait();
    pdl_launch_dependents();  // dependents may start their prologues now
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, pairs = a.T * a.k;
    if (warp < a.T) {
        const int id = choose_token<NPER>(a, warp, room + (size_t)warp * a.room);
        if (lane < a.k) ids[warp * a.k + lane] = id;
    }
    __syncthreads();
    if (threadIdx.x < pairs) {
        const int p = threadIdx.x, e = ids[p];
        int at = 0;
        for (int o = 0; o < pairs; ++o) at += ids[o] < e || (ids[o] == e && o < p);
        sorted_pair[at] = p;
        pair_to_sorted[p] = at;
    }
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) {
        int below = 0;
        for (int o = 0; o < pairs; ++o) below += ids[o] < e;
        offsets[e] = below;
    }
}

void lay_out(ScoredArgs& a) {
    a.log_per = 5;
    while (a.log_per > 0 && (32 >> a.log_per) < a.groups) --a.log_per;
    a.per = 1 << a.log_per;
    a.chunk = (a.size + a.per - 1) / a.per;  // (at most 64)
    a.vec = a.chunk % 4 == 0 && a.size % 4 == 0 && aligned16(a.logits) && aligned16(a.bias);
    a.room = (a.E > 66 ? a.E + 1 : 66) / 2 * 2;  // (whole 16 bytes)
}

// f(integral constant) for the experts a lane holds
template <typename F>
moe_status with_chunk(int chunk, F&& f) {
    return chunk <= 1    ? f(std::integral_constant<int, 1>())
           : chunk <= 2  ? f(std::integral_constant<int, 2>())
           : chunk <= 4  ? f(std::integral_constant<int, 4>())
           : chunk <= 8  ? f(std::integral_constant<int, 8>())
           : chunk <= 16 ? f(std::integral_constant<int, 16>())
           : chunk <= 32 ? f(std::integral_constant<int, 32>())
                         : f(std::integral_constant<int, 64>());
}

moe_status launch_route_scored(ScoredArgs a, cudaStream_t s) {
    lay_out(a);
    const dim3 grid((unsigned)((a.T + WARPS - 1) / WARPS));
    const size_t smem = sizeof(double) * WARPS * a.room;  // (at most 32 KB)
    return with_chunk(a.chunk, [&](auto n) {
        cudaError_t e = launch_pdl(route_scored_kernel<decltype(n)::value>, grid, dim3(32 * WARPS), smem, s, a);
        return e == cudaSuccess ? MOE_OK : cuda_status(e, "moe_route_scored: launch");
    });
}

// The choice and the sorted pairs.
moe_status launch_route_scored_sorted(ScoredArgs a, int32_t* offsets, int32_t* sorted_pair, int32_t* pair_to_sorted,
                                      void* ws, size_t ws_bytes, cudaStream_t s) {
    lay_out(a);
    const size_t smem = sizeof(double) * a.T * a.room;
    if (a.T <= FEW_T && smem <= FEW_SMEM)
        return with_chunk(a.chunk, [&](auto n) {
            cudaError_t e = launch_pdl(route_scored_few_kernel<decltype(n)::value>, dim3(1), dim3(32 * FEW_T), smem, s, a,
                                       offsets, sorted_pair, pair_to_sorted);
            return e == cudaSuccess ? MOE_OK : cuda_status(e, "moe_route_tokens_scored: launch");
        });
    moe_status st = launch_route_scored(a, s);
    if (st != MOE_OK) return st;
    return launch_permute_ws(a.ids, a.T * a.k, a.E, offsets, sorted_pair, pair_to_sorted, s, ws, ws_bytes);
}

}  // namespace
}  // namespace moe

using namespace moe;

// (what: the entry point's name, for messages)
static moe_status scored_args(const char* what, const float* logits, int T, int E, int k, const moe_scoring* s, int32_t* ids,
                              float* weights, ScoredArgs* out) {
    MOE_CHECK_ARG(s, "%s: scoring is null", what);
    MOE_CHECK_ARG(T >= 0 && E > 0, "%s: T=%d E=%d", what, T, E);
    MOE_CHECK_SUPPORTED(E <= 1024, "%s: E=%d above 1024", what, E);
    MOE_CHECK_SUPPORTED(T <= INT32_MAX - WARPS, "%s: T=%d past what one launch covers", what, T);
    MOE_CHECK_ARG(s->scoring == MOE_SCORE_SOFTMAX || s->scoring == MOE_SCORE_SIGMOID, "%s: unknown scoring %d", what,
                  s->scoring);
    MOE_CHECK_ARG(s->renormalize == 0 || s->renormalize == 1, "%s: renormalize must be 0 or 1", what);
    MOE_CHECK_ARG(s->scale - s->scale == 0.0f, "%s: scale must be finite", what);
    MOE_CHECK_ARG(s->groups >= 1 && s->groups <= E && E % s->groups == 0, "%s: groups=%d must divide E=%d", what, s->groups,
                  E);
    MOE_CHECK_SUPPORTED(s->groups <= 32, "%s: groups=%d above 32", what, s->groups);
    const int size = E / s->groups;
    MOE_CHECK_ARG(s->top_groups >= 1 && s->top_groups <= s->groups, "%s: top_groups=%d must be in [1, groups=%d]", what,
                  s->top_groups, s->groups);
    MOE_CHECK_ARG((s->group_top == 1 || s->group_top == 2) && s->group_top <= size,
                  "%s: group_top=%d must be 1 or 2, and no more than a group's %d experts", what, s->group_top, size);
    MOE_CHECK_ARG(k >= 1 && k <= 32 && k <= s->top_groups * size,
                  "%s: k=%d must be in [1, min(32, the %d experts of top_groups)]", what, k, s->top_groups * size);
    if (T == 0) return MOE_OK;
    MOE_CHECK_ARG(logits && ids && weights, "%s: null pointer", what);
    MOE_CHECK_SUPPORTED((((uintptr_t)logits | (uintptr_t)s->bias | (uintptr_t)ids | (uintptr_t)weights) & 3) == 0,
                        "%s: a pointer is not aligned to its type", what);
    // (where every group stays there is nothing to choose among them)
    const int groups = s->top_groups == s->groups ? 1 : s->groups;
    ScoredArgs a = {};
    a.logits = logits, a.bias = s->bias, a.ids = ids, a.weights = weights, a.scale = s->scale, a.T = T, a.E = E, a.k = k;
    a.sigmoid = s->scoring == MOE_SCORE_SIGMOID, a.renorm = s->renormalize, a.groups = groups;
    a.top_groups = groups == 1 ? 1 : s->top_groups, a.group_top = s->group_top, a.size = E / groups;
    *out = a;
    return MOE_OK;
}

extern "C" {

moe_status moe_route_scored(const float* logits, int T, int E, int k, const moe_scoring* s, int32_t* ids, float* weights,
                            cudaStream_t stream) {
    ScoredArgs a;
    moe_status st = scored_args("moe_route_scored", logits, T, E, k, s, ids, weights, &a);
    if (st != MOE_OK || T == 0) return st;
    return launch_route_scored(a, stream);
}

moe_status moe_route_scored_packed(const moe_route_scored_args* p, cudaStream_t stream) {
    MOE_CHECK_ARG(p, "moe_route_scored_packed: args is null");
    return moe_route_scored(p->logits, p->T, p->E, p->k, &p->scoring, p->ids, p->weights, stream);
}

moe_status moe_route_tokens_scored(const uint16_t* x, const uint16_t* w_router, const float* router_bias, int T, int H, int E,
                                   int k, const moe_scoring* s, int fresh, float* logits, int32_t* ids, float* weights,
                                   int32_t* expert_offsets, int32_t* sorted_pair, int32_t* pair_to_sorted, void* ws,
                                   size_t ws_bytes, cudaStream_t stream) {
    ScoredArgs a;
    moe_status st = scored_args("moe_route_tokens_scored", logits, T, E, k, s, ids, weights, &a);
    if (st != MOE_OK) return st;
    MOE_CHECK_ARG(H > 0, "moe_route_tokens_scored: H=%d", H);
    MOE_CHECK_SUPPORTED((long long)T * k <= (1 << 24), "moe_route_tokens_scored: T*k above 2^24");
    MOE_CHECK_ARG(expert_offsets, "moe_route_tokens_scored: expert_offsets is null");
    if (T == 0) return launch_permute(ids, 0, E, expert_offsets, sorted_pair, pair_to_sorted, stream);
    MOE_CHECK_ARG(x && w_router && sorted_pair && pair_to_sorted, "moe_route_tokens_scored: null pointer");
    MOE_CHECK_SUPPORTED(H % 256 == 0, "moe_route_tokens_scored: H=%d must be a multiple of 256", H);
    MOE_CHECK_SUPPORTED(aligned16(x) && aligned16(w_router) && aligned16(logits) && aligned16(router_bias),
                        "moe_route_tokens_scored: x, w_router, router_bias and logits must be 16-byte aligned");
    if ((st = launch_router_logits(x, w_router, router_bias, logits, T, H, E, stream, fresh != 0)) != MOE_OK) return st;
    return launch_route_scored_sorted(a, expert_offsets, sorted_pair, pair_to_sorted, ws, ws_bytes, stream);
}

}  // extern "C"
