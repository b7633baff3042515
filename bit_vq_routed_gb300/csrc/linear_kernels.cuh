// y = act(x W^T + bias) + residual on the tensor cores, x and W in 16 bits
// (linear.cu) or in 8 bits with a scale a row (linear_8bit.cu).
//
// All three kernels compute y^T tiles: the weights' rows are the tensor core's M,
// the tokens its N.  So one token needs no more than 8 or 16 columns.  In the two
// tcgen05 kernels the rows are the accumulator's TMEM lanes: whatever the number
// of tokens a warp's 32 lanes hold 32 consecutive outputs of one token, whose
// store is contiguous for every row stride.  Their operands come through TMA (128
// bytes a row = 64 inputs of 16 bits or 128 of 8, 128-byte swizzle; rows and inputs past the end read
// as zeros), so ragged sizes need no code in the main loop.  No kernel here lets its
// dependents start early: y may be the activations that a routing reads before
// its wait (the launch contract in common.cuh).
#pragma once

#include <type_traits>

#include "elem.cuh"
#include "tc05.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float quick_exp2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float quick_inverse(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// QUICK (8-bit products): the activations by the special function unit, within 2^-16 of
// themselves (2^-20 and, where exponentials are small, 2^-24 for each unit of the exponent).
// silu is z sigmoid(z), gelu's tanh form z sigmoid(2 u); gelu takes erfc(x) = exp(-x^2) t
// p(t), t = 1 / (1 + 0.46 x), whose p was fitted here to erfc(x) exp(x^2) / t with the least
// largest relative error, 7e-7 (in fp32 the product is off by 1.8e-6 of itself up to |z| =
// 5, 3e-6 up to 8).  (Divisions rounded exactly and erff leave the unrolled loop for their
// rare cases: silu at K = 4272, N = 1367, T = 1564: 27.5 and 16.1 us; gelu at K = 512, N =
// 2048, T = 8192: 33.3 and 25.5.)
template <int ACT, bool QUICK>
__device__ __forceinline__ float activate(float z) {
    constexpr float LOG2E = 1.44269504088896341f;
    if (QUICK && ACT == MOE_ACT_SILU) return z * quick_inverse(1.0f + quick_exp2(-LOG2E * z));
    if (QUICK && ACT == MOE_ACT_GELU_TANH) {
        const float c = -1.59576912160573071f * LOG2E;  // 2 sqrt(2 / pi)
        return z * quick_inverse(1.0f + quick_exp2(z * (c + c * 0.044715f * z * z)));
    }
    if (QUICK && ACT == MOE_ACT_GELU) {
        const float m = fabsf(z);  // (x = m / sqrt 2)
        const float t = quick_inverse(1.0f + (0.46f * 0.707106781186547524f) * m);
        float p = 0.033857141f;  // (halves of p's)
        p = p * t - 0.113314509f;
        p = p * t + 0.084595270f;
        p = p * t + 0.026305515f;
        p = p * t + 0.093423799f;
        p = p * t + 0.115590967f;
        p = p * t + 0.129778624f;
        p = p * t + 0.129763529f;
        const float h = p * t * quick_exp2(-0.5f * LOG2E * (z * z));  // erfc(x) / 2
        return fmaxf(z, 0.0f) - fminf(m, 16.0f) * h;  // (h is 0 beyond; infinity stays, NaN comes with h)
    }
    if (ACT == MOE_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if (ACT == MOE_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    if (ACT == MOE_ACT_GELU_TANH)
        return 0.5f * z * (1.0f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
    if (ACT == MOE_ACT_SILU) return z / (1.0f + expf(-z));
    return z;
}
// With a residual, in the pair kernel: of 16 bits gelu's last product and the sum are rounded
// once, as they always were there.
template <int ACT, bool QUICK>
__device__ __forceinline__ float activate_add(float z, float r) {
    if (!QUICK && ACT == MOE_ACT_GELU) return fmaf(0.5f * z, 1.0f + erff(z * 0.70710678118654752f), r);
    if (!QUICK && ACT == MOE_ACT_GELU_TANH)
        return fmaf(0.5f * z, 1.0f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)), r);
    return __fadd_rn(activate<ACT, QUICK>(z), r);
}
// f(integral constant) for the call's activation: the choice is made once,
// outside the loops over the outputs
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case MOE_ACT_RELU: f(std::integral_constant<int, MOE_ACT_RELU>()); break;
        case MOE_ACT_GELU: f(std::integral_constant<int, MOE_ACT_GELU>()); break;
        case MOE_ACT_GELU_TANH: f(std::integral_constant<int, MOE_ACT_GELU_TANH>()); break;
        case MOE_ACT_SILU: f(std::integral_constant<int, MOE_ACT_SILU>()); break;
        default: f(std::integral_constant<int, MOE_ACT_NONE>());
    }
}

struct LinearArgs {
    const uint16_t *bias, *res;
    const float *sx, *sw;  // 8 bits: the scales of x's and w's rows
    uint16_t* y;
    int64_t ldr, ldy;
    int T, N, kblocks, act;
    int n_tiles, t_tiles;
    bool wide;  // pair kernel: store 16 bytes at a time
    int* err;
};

// E8: inputs of 8 bits (e4m3), else 16
template <bool E8>
constexpr int BK = E8 ? 128 : 64;     // inputs of a block: 128 bytes a row
constexpr int ROW_BYTES = 128;
constexpr int A_BYTES = 128 * ROW_BYTES;  // 128 weight rows
constexpr int TMA_WARP = 0, MMA_WARP = 1;
constexpr int THREADS = 192;           // TMA, MMA and four epilogue warps

// Which kernel (times on a GB300, microseconds, weights from memory):
//   - up to FEW_T tokens (8 bits: up to 32 of few inputs) the weights stream through registers (K = 4096, N =
//     6144: 9.0 at 1 token and 9.1 at 8, 83 % of the copy rate; the split
//     kernel 11.5 and 11.6; 8 bits 4.9 and 5.7, the split kernel 6.3);
//   - inputs of 16 bits: up to SPLIT_T tokens, and above where 128 x 128 tiles
//     leave room for clusters of 8 over a long sum, the split kernel (T = 64, N =
//     4096: 9.7, pairs 13.2, but N = 6144: 15.5 and 14.7; T = 128, K = 8192, N = 512:
//     9.0, pairs 16.5; K = 1024: 5.9 and 5.3, hence SPLIT_K); CTA pairs for the
//     rest (T = 96, N = 6144: 14.6; T = 4096: 108, 100 % of the measured cuBLAS rate);
//   - inputs of 8 bits: the cheaper of the two by an estimate of their cycles, see
//     run_linear (K = 4096, T = 64, N = 4096: split 6.7, pairs 7.0; T = 128: 9.4 and
//     7.4; K = 8192: 14.2 and 13.0; T = 4096, N = 6144: 59 to 61).
constexpr int FEW_T = 8;
constexpr int SPLIT_T = 64;
constexpr int SPLIT_K = 2048;
// A stage of the pair kernel holds two blocks of inputs instead of one up to this
// token tile (K = 4096, N = 6144, T = 128: 15.4 against 18.4; T = 512, whose tile
// is 176: 23.3 against 21.1).
constexpr int WIDE_STAGE_NT = 128;

// ---------------------------------------------------------------- few tokens
// Up to 8 tokens, and up to 32 where few inputs make the start of anything longer the
// larger part: the weights' bytes are all there is, so they go straight
// from memory to registers, each read once, 16 bytes a lane.  One CTA takes 16
// outputs, its warps a share of the inputs each.  mma.sync m16n8k16 with the
// weights as A and the tokens as B: a lane's 16 bytes of a row are taken as
// the k's of two of its fragments, the same way in A and in B, so the sum
// only runs in another order.
constexpr int FEW_WARPS = 8, FEW_SM_WARPS = 24;  // of a CTA, and of those on an SM (up to 16 tokens)
constexpr int FEW_UNROLL = 4;  // 64-byte steps in flight a warp
// Weights of 8 bits are asked for ahead of the wait, to L2 (where all writes meet:
// one that comes later is seen by the load all the same), up to this many bytes an SM
// (K = 4096, N = 4096, 110 KB an SM: 5.2 against 5.6, behind moe_quantize_rows 6.2 and
// 7.0; K = 2048, N = 6144: 3.9 and 4.4; but N = 6144, K = 4096, 166 KB: 7.2 and 6.6).
constexpr int64_t FEW_AHEAD = 128 * 1024;

template <bool BF>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    if (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        mma_16816(d, a0, a1, a2, a3, b0, b1);
}

__device__ __forceinline__ void mma_16x8x32_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct FewArgs {
    const uint8_t *x, *w;
    int64_t ldx, ldw;   // in bytes
    int64_t row_bytes;  // of K inputs (below 2^32)
    bool ahead;         // see FEW_AHEAD
    LinearArgs a;
};

// TT: tokens by eights.  More of them take fewer steps at a time, 32 tokens
// also two CTAs of 8 warps an SM instead of three.
constexpr int few_unroll(int tt) { return FEW_UNROLL / tt; }
constexpr int few_sm_warps(int tt) { return tt < 4 ? FEW_SM_WARPS : 16; }

template <bool BF, bool E8, int WARPS, int TT>
__global__ void __launch_bounds__(32 * WARPS, few_sm_warps(TT) / WARPS) linear_few_kernel(const FewArgs f) {
    constexpr int UNROLL = few_unroll(TT);
    __shared__ float part[WARPS][8 * TT][16];
    const LinearArgs& a = f.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int n0 = blockIdx.x * 16;
    // steps of 64 bytes: 4 lanes x 16 bytes of a row
    const int steps = (int)((f.row_bytes + 63) / 64);
    const int s0 = (int)((int64_t)steps * warp / WARPS);
    const int s1 = (int)((int64_t)steps * (warp + 1) / WARPS);
    // (rows past the end read the last one again; their sums are dropped)
    const uint8_t* w0 = f.w + (int64_t)min(n0 + g, a.N - 1) * f.ldw + 16 * q;
    const uint8_t* w1 = f.w + (int64_t)min(n0 + g + 8, a.N - 1) * f.ldw + 16 * q;
    const uint8_t* xr[TT];
#pragma unroll
    for (int h = 0; h < TT; ++h) xr[h] = f.x + (int64_t)min(8 * h + g, a.T - 1) * f.ldx + 16 * q;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 u0[UNROLL], u1[UNROLL], b[UNROLL][TT];
    const int last = min(s1, (int)((f.row_bytes - 16 * q + 63) / 64));  // a lane's inputs end there
    auto inside = [&](int s) { return s < last; };
    auto load_w = [&](int s, int i) {
        u0[i] = inside(s) ? ldg_stream(w0 + 64u * s) : zero;
        u1[i] = inside(s) ? ldg_stream(w1 + 64u * s) : zero;
    };
    auto load_x = [&](int s, int i) {
#pragma unroll
        for (int h = 0; h < TT; ++h) b[i][h] = inside(s) ? *reinterpret_cast<const uint4*>(xr[h] + 64u * s) : zero;
    };
    if (E8 && f.ahead) {
        // the CTA's weights to L2, be it while x still goes to 8 bits
        for (int64_t i = threadIdx.x; i < 16 * ((f.row_bytes + 127) / 128); i += 32 * WARPS)
            prefetch_l2(f.w + min(n0 + (int)(i & 15), a.N - 1) * f.ldw + 128 * (i >> 4));
    }
    // (before the weights too: whatever ran before may have written them)
    pdl_wait();
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) load_w(s0 + i, i), load_x(s0 + i, i);
    // what the thread's result needs besides the sums: up to 8 tokens asked for with them
    // (one token, K = N = 1024, bias and residual: 1.8 against 2.0, 8 bits 1.86 and 1.90;
    // with more the registers do not hold it)
    const int n = n0 + (threadIdx.x & 15);
    uint16_t bias = 0, res = 0;
    float sx = 1.0f, sw = 1.0f;
    auto ask = [&](int t) {
        if (t >= min(8 * TT, a.T) || n >= a.N) return;
        if (a.bias) bias = a.bias[n];
        if (a.res) res = a.res[(int64_t)t * a.ldr + n];
        if (E8) sx = a.sx[t], sw = a.sw[n];
    };
    if constexpr (TT == 1) ask(threadIdx.x >> 4);
    float acc[TT][4] = {};
    for (int s = s0; s < s1; s += UNROLL) {
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
#pragma unroll
            for (int h = 0; h < TT; ++h) {
                const uint4& x = b[i][h];
                if (E8) {
                    mma_16x8x32_e4m3(acc[h], u0[i].x, u1[i].x, u0[i].y, u1[i].y, x.x, x.y);
                    mma_16x8x32_e4m3(acc[h], u0[i].z, u1[i].z, u0[i].w, u1[i].w, x.z, x.w);
                } else {
                    mma_16x8x16<BF>(acc[h], u0[i].x, u1[i].x, u0[i].y, u1[i].y, x.x, x.y);
                    mma_16x8x16<BF>(acc[h], u0[i].z, u1[i].z, u0[i].w, u1[i].w, x.z, x.w);
                }
            }
            load_w(s + i + UNROLL, i);
            load_x(s + i + UNROLL, i);
        }
    }
    // acc: rows g and g + 8, tokens 2q and 2q + 1
#pragma unroll
    for (int h = 0; h < TT; ++h) {
        part[warp][8 * h + 2 * q][g] = acc[h][0];
        part[warp][8 * h + 2 * q + 1][g] = acc[h][1];
        part[warp][8 * h + 2 * q][g + 8] = acc[h][2];
        part[warp][8 * h + 2 * q + 1][g + 8] = acc[h][3];
    }
    __syncthreads();
    if (n < a.N)
#pragma unroll
        for (int t = threadIdx.x >> 4; t < 8 * TT; t += 2 * WARPS)
            if (t < a.T) {
                if constexpr (TT > 1) ask(t);
                float z = 0.0f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) z += part[w][t][threadIdx.x & 15];
                if (E8) z *= sx * sw;
                z += to_f32<BF>(bias);
                with_act(a.act, [&](auto act) { z = activate<decltype(act)::value, E8>(z); });
                a.y[(int64_t)t * a.ldy + n] = from_f32<BF>(z + to_f32<BF>(res));
            }
}

// The warps of a CTA of the few-token kernel for inputs of 8 bits, or 0 where the other
// kernels take the call.  A warp waits for memory once per batch of few_unroll steps of
// 64 inputs: more warps save batches, and cost 0.2 us for 12 and 0.6 us for 16 instead
// of 8.  Each CTA reads all tokens' rows, which with many inputs costs more than the
// split kernel's copies and the join of its cluster.  Microseconds on a GB300, of weights
// from memory and L2 in turn:
inline int few_warps8(int T, int64_t ctas, int K, int sms) {
    const int64_t round = FEW_SM_WARPS / 8 * sms;  // CTAs of 8 warps that run at once
    const int steps = (K + 63) / 64;
    if (T > 32 || (T > 16 && ctas > 2 * sms)) return 0;
    // (8, 16 warps, split kernel at N = 1024.  K = 1024: 2.6, 2.8, 4.3; K = 2048: 4.2, 3.3, 4.0;
    // K = 4096: 6.6, 5.2, 4.2.  At N = 4096, K = 1536: 4.5 and 5.0 split)
    if (T > 16) return ctas > sms ? (K <= 1536 ? 8 : 0) : K <= 1024 ? 8 : K <= 2560 ? 16 : 0;
    if (T > 8) {
        // (8, 12, 16 warps, split.  N = 1024, K = 1024: 1.9, 2.2, 2.5, 3.6; K = 1536: 2.6, 2.3,
        // 2.6, 3.9; K = 4096: 5.0, 4.4, 3.6, 4.0; K = 8192: 16 warps 5.3, split 5.5; N = 256:
        // 5.1 and 4.7)
        if (ctas <= sms) return K <= 1024 ? 8 : K <= 1536 ? 12 : K <= 6144 || 3 * ctas >= sms ? 16 : 0;
        // (8, 12, split.  N = 4096, K = 2560: 4.3, 4.4, 6.5; K = 4096: 6.2, 5.8, 7.3; K = 8192: -,
        // 9.2, 9.2; N = 2560: -, 8.7, 8.0)
        if (ctas <= 2 * sms) return K <= 2560 ? 8 : K <= 7168 ? 12 : 0;
        // (8, split.  N = 6144, K = 5120: 8.6, 9.5; K = 8192: 12.6, 12.2.  In two rounds, 4 warps:
        // N = 8192, K = 1536: 5.0 and 7.0; K = 4096: 11.2 and 9.4)
        if (ctas <= round) return K <= 5120 ? 8 : 0;
        return ctas <= 2 * round && K <= 1536 ? 4 : 0;
    }
    // (8, 12, 16 warps at one token.  N = 1024, K = 2048: 2.2, 2.4, 2.7; K = 5120: 4.2, 3.9, 4.4;
    // K = 8192: 6.1, -, 4.8)
    if (ctas <= sms) return steps <= 32 ? 8 : steps <= 96 ? 12 : 16;
    // (8, 12.  N = 4096, K = 2560: 3.8, 3.6; K = 4096, no batch less: 5.0, 5.3; K = 8192: 8.8, 7.7)
    if (ctas <= 2 * sms) return (steps + 47) / 48 < (steps + 31) / 32 ? 12 : 8;
    // (4 warps where CTAs of 8 come in two rounds.  K = 4096, N = 8192: 8.8 against 9.6, N = 12288 10.3
    // and 11.1; where they come in four, N = 32768, 26.2 and 25.8)
    return ctas > round && ctas <= 2 * round ? 4 : 8;
}

// ---------------------------------------------------------------- split kernel
// One tile of 128 outputs x NT tokens per cluster, its sum over the inputs
// split over the cluster's S CTAs.  CTA r finishes the tile's outputs r * 128/S
// ..: each CTA sends its part of their sums from TMEM into that CTA's shared
// memory (distributed shared memory), and after one cluster barrier each adds
// the parts in rank order, so the result does not depend on timing.
template <int NT, int STAGES>
struct __align__(1024) SplitSmem {
    struct Stage {
        uint8_t a[2][A_BYTES];
        uint8_t b[2][NT * ROW_BYTES];
    } st[STAGES];
    float part[NT * 128];  // [source CTA][token][own output]
    uint64_t full[STAGES], empty[STAGES], acc_full;
    uint32_t tmem;
    int failed;
};

template <bool BF, bool E8, int NT, int STAGES>
__global__ void __launch_bounds__(THREADS)
    linear_split_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                        const LinearArgs a, const int S) {
    using Smem = SplitSmem<NT, STAGES>;
    extern __shared__ __align__(1024) uint8_t dyn[];
    Smem& sm = *reinterpret_cast<Smem*>(dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u));
    constexpr uint32_t COLS = NT < 32 ? 32 : NT;
    constexpr uint32_t BYTES = 2 * (A_BYTES + NT * ROW_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x / S, rank = blockIdx.x % S;
    const int n0 = (tile / a.t_tiles) * 128, t0 = (tile % a.t_tiles) * NT;
    // stages of two blocks of inputs
    const int steps = (a.kblocks + 1) / 2;
    const int k0 = (int)((int64_t)steps * rank / S), n_k = (int)((int64_t)steps * (rank + 1) / S) - k0;
    const int nt = min(NT, a.T - t0);
    const Waits wait{a.err, &sm.failed};
    const int pre = min(STAGES, n_k);
    auto load_w = [&](int s, int i) {
        for (int h = 0; h < 2; ++h)
            tma_2d(smem_u32(sm.st[s].a[h]), &wmap, ((k0 + i) * 2 + h) * BK<E8>, n0, smem_u32(&sm.full[s]));
    };
    auto load_x = [&](int s, int i) {
        for (int h = 0; h < 2; ++h)
            tma_2d(smem_u32(sm.st[s].b[h]), &xmap, ((k0 + i) * 2 + h) * BK<E8>, t0, smem_u32(&sm.full[s]));
    };

    if (warp == TMA_WARP) {
        if (elect_one()) {
            for (int s = 0; s < STAGES; ++s) {
                mbar_init(smem_u32(&sm.full[s]), 1);
                mbar_init(smem_u32(&sm.empty[s]), 1);
            }
            mbar_init(smem_u32(&sm.acc_full), 1);
            sm.failed = 0;
            mbar_fence_init();
            prefetch_map(&wmap);
            prefetch_map(&xmap);
            // the first stages, as soon as what ran before has finished
            pdl_wait();
            for (int i = 0; i < pre; ++i) {
                mbar_arrive_expect_tx(smem_u32(&sm.full[i]), BYTES);
                load_w(i, i);
                load_x(i, i);
            }
        }
        __syncwarp();
    }
    if (warp == MMA_WARP) tmem_alloc(smem_u32(&sm.tmem), COLS);
    tc_before();
    __syncthreads();
    if (S > 1) cluster_arrive();  // (waited for before the first access to a peer)
    tc_after();
    const uint32_t tmem = sm.tmem;
    pdl_wait();

    if (warp == TMA_WARP) {
        int s = 0, turn = 1, i = pre;
        for (; i < n_k; ++i) {
            if (!wait.warp(smem_u32(&sm.empty[s]), (turn - 1) & 1, MOE_DEVERR_WAIT_EMPTY)) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(smem_u32(&sm.full[s]), BYTES);
                load_w(s, i);
                load_x(s, i);
            }
            if (++s == STAGES) s = 0, ++turn;
        }
        // (after a wait that gave up: the copies in flight land before the CTA ends)
        if (i < n_k)
            for (int j = max(0, i - STAGES); j < i; ++j)
                mbar_wait_sleep_bounded(smem_u32(&sm.full[j % STAGES]), (j / STAGES) & 1, a.err, MOE_DEVERR_WAIT_FULL);
    } else if (warp == MMA_WARP) {
        constexpr uint32_t idesc = E8 ? umma_idesc_e4m3(128, NT) : umma_idesc(BF, 128, NT);
        int s = 0, turn = 0;
        for (int i = 0; i < n_k; ++i) {
            if (!wait.warp(smem_u32(&sm.full[s]), turn & 1, MOE_DEVERR_WAIT_FULL)) break;
            tc_after();
            const uint64_t ad = desc_k_inner(smem_u32(sm.st[s].a)), bd = desc_k_inner(smem_u32(sm.st[s].b));
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    umma<E8>(tmem, ad + (j / 4) * (A_BYTES >> 4) + 2 * (j % 4),
                             bd + (j / 4) * (NT * ROW_BYTES >> 4) + 2 * (j % 4), idesc, i > 0 || j > 0);
                umma_arrive(smem_u32(&sm.empty[s]));
            }
            if (++s == STAGES) s = 0, ++turn;
        }
        if (elect_one()) umma_arrive(smem_u32(&sm.acc_full));
    }
    __syncwarp();
    if (S > 1) cluster_wait();  // the peers run

    const int rows = 128 / S;  // outputs of a CTA's share
    // what a thread's results need besides the sums, asked for ahead of them (and not
    // looked at before: 32 tokens, K = N = 4096, 8 bits with residual 7.1 against 8.0, 64 tokens
    // 7.9 and 9.4): 4 consecutive outputs of a token at a time
    const int per_token = rows / 4;
    uint16_t bias[4] = {}, res[4] = {};
    float sw[4], sx;
    auto ask = [&](int e) {
        const int t = t0 + e / per_token, n = n0 + rank * rows + 4 * (e % per_token);
        const int m = e < nt * per_token ? a.N - n : 0;
        const uint16_t* r = a.res + (int64_t)t * a.ldr + n;
        sx = E8 && m > 0 ? a.sx[t] : 1.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            bias[j] = a.bias && j < m ? a.bias[n + j] : 0;
            res[j] = a.res && j < m ? r[j] : 0;
            sw[j] = E8 && j < m ? a.sw[n + j] : 1.0f;
        }
    };
    const bool asked = E8 || a.bias || a.res;
    if (asked) ask(threadIdx.x);
    if (warp >= 2) {
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t dst = peer_addr(smem_u32(&sm.part[rank * NT * rows + row % rows]), row / rows);
        if (wait.warp(smem_u32(&sm.acc_full), 0, MOE_DEVERR_WAIT_FULL)) {
            tc_after();
            for (int c = 0; c < nt; c += 16) {
                uint32_t r[16];
                tmem_ld16_async(tmem + ((uint32_t)(quarter * 32) << 16) + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) peer_st(dst + 4 * (c + j) * rows, r[j]);
            }
        }
        tc_before();
    }
    __syncwarp();
    if (S > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp == MMA_WARP) {
        tc_after();
        tmem_free(tmem, COLS);
    }
    with_act(a.act, [&](auto act) {
        for (int e = threadIdx.x; e < nt * per_token; e += THREADS) {
            const int r4 = 4 * (e % per_token), t = t0 + e / per_token;
            const int n = n0 + rank * rows + r4, m = min(4, a.N - n);
            uint16_t* dst = a.y + (int64_t)t * a.ldy + n;
            float v[4] = {};
            const float* p = &sm.part[(e / per_token) * rows + r4];
            for (int s = 0; s < S; ++s) {
                const float4 f = *reinterpret_cast<const float4*>(p + s * NT * rows);
                v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (E8) v[j] *= sx * sw[j];
                v[j] = activate<decltype(act)::value, E8>(v[j] + to_f32<BF>(bias[j])) + to_f32<BF>(res[j]);
            }
            if (asked && e + THREADS < nt * per_token) ask(e + THREADS);
            if (m == 4 && (reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF>(v[0], v[1]), pack2<BF>(v[2], v[3]));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < m) dst[j] = from_f32<BF>(v[j]);
            }
        }
    });
}

// ---------------------------------------------------------------- pair kernel
// Persistent CTA pairs, one tile of 256 outputs x 256 tokens after another:
// cta_group::2 lets each CTA of the pair fetch only half of each operand (128
// weight rows, 128 tokens per stage), so a tile's 32 KB per CTA and 64 inputs
// feed 512 cycles of tensor work.  Two accumulators of 256 columns: the
// epilogue of one tile runs during the next tile's products.
// Epilogue warps: 16 where residuals are read (K = 4096, N = 4096, T = 1024: 28.0
// against 30.8 with 8), else 8 (24.9 and 25.0; 8 bits, K = 1424, N = 2051, T = 333:
// 7.8 and 8.0).  Results of 8-bit products take longer than the products themselves up to
// P_EPI_ACT_K inputs: 16 for gelu and silu too where a pair has several tiles (N = 2048,
// T = 8192, gelu, K = 1024: 26.9 against 28.8; K = 2560: 35.7 and 34.9).
constexpr int P_EPI_RES = 16, P_EPI = 8;
constexpr int P_EPI_ACT_K = 2048;
constexpr int P_STAGE_BYTES = 6 * 2 * A_BYTES;
constexpr int P_MAX_STAGES = 10;

struct __align__(1024) PairSmem {
    uint8_t st[P_STAGE_BYTES];
    uint16_t out[P_EPI_RES][16][32];  // an epilogue warp's 16 tokens x 32 outputs
    float sx[2][256];                   // 8 bits: the scales of a tile's tokens
    uint64_t full[P_MAX_STAGES], empty[P_MAX_STAGES], acc_full[2], acc_empty[2], peer_ready;
    uint32_t tmem;
    int failed;
};

// Tiles in groups of 16 token tiles, tokens first: the CTAs that run at the
// same time share the group's tokens and a few weight tiles in L2.
__device__ __forceinline__ void pair_tile(const LinearArgs& a, int tile, int& tn, int& tt) {
    const int per_group = 16 * a.n_tiles, g = tile / per_group, r = tile - g * per_group;
    const int width = min(16, a.t_tiles - 16 * g);
    tn = r / width;
    tt = 16 * g + r % width;
}

template <bool BF, bool E8, int SUB, int EPI>
__global__ void __launch_bounds__(64 + 32 * EPI, 1) __cluster_dims__(2, 1, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                       const LinearArgs a, const int NT) {
    extern __shared__ __align__(1024) uint8_t dyn[];
    PairSmem& sm = *reinterpret_cast<PairSmem*>(dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1, tiles = a.n_tiles * a.t_tiles;
    const Waits wait{a.err, &sm.failed};
    // a stage: SUB blocks of inputs of 128 weight rows and nt / 2 tokens
    const int block_bytes = A_BYTES + NT * 64, stage_bytes = SUB * block_bytes;
    const int n_stages = min(P_MAX_STAGES, P_STAGE_BYTES / stage_bytes);
    const int steps = (a.kblocks + SUB - 1) / SUB;

    if (threadIdx.x == 0) {
        for (int s = 0; s < n_stages; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&sm.acc_full[s]), 1);
            mbar_init(smem_u32(&sm.acc_empty[s]), 2 * EPI);  // the epilogue warps of both CTAs
        }
        mbar_init(smem_u32(&sm.peer_ready), 1);  // the odd CTA has its columns
        sm.failed = 0;
        mbar_fence_init();
    }
    if (threadIdx.x == 32 * 2) {
        prefetch_map(&wmap);
        prefetch_map(&xmap);
    }
    // the copies start as soon as both CTAs have their barriers; the others wait
    // for the accumulators' columns too
    __syncwarp();
    cluster_arrive();
    if (warp == MMA_WARP) tmem_alloc_pair(smem_u32(&sm.tmem), 512);
    tc_before();
    cluster_wait();
    if (warp != TMA_WARP) named_barrier(2, 32 + 32 * EPI);
    tc_after();
    const uint32_t tmem = sm.tmem;
    pdl_wait();

    const uint32_t st0 = smem_u32(sm.st);
    if (warp == TMA_WARP) {
        int s = 0, turn = 0, issued = 0;
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step) {
            int tn, tt;
            pair_tile(a, tile, tn, tt);
            const int n0 = tn * 256 + (int)rank * 128, t0 = tt * NT + (int)rank * (NT / 2);
            for (int kb = 0; kb < steps; ++kb) {
                if (turn > 0 && !wait.warp(smem_u32(&sm.empty[s]), (turn - 1) & 1, MOE_DEVERR_WAIT_EMPTY)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    // the even CTA's barrier counts the bytes of both
                    const uint32_t full = smem_u32(&sm.full[s]), st = st0 + s * stage_bytes;
                    if (rank == 0) mbar_arrive_expect_tx(full, 2 * stage_bytes);
#pragma unroll
                    for (int h = 0; h < SUB; ++h) {
                        tma_2d_pair(st + h * block_bytes, &wmap, (kb * SUB + h) * BK<E8>, n0, full);
                        tma_2d_pair(st + h * block_bytes + A_BYTES, &xmap, (kb * SUB + h) * BK<E8>, t0, full);
                    }
                }
                issued = min(issued + 1, n_stages);
                if (++s == n_stages) s = 0, ++turn;
            }
        }
        // (after a wait that gave up: the copies in flight land before the CTAs end)
        if (!ok && rank == 0)
            for (int i = 0; i < issued; ++i) {
                if (--s < 0) s = n_stages - 1, --turn;
                mbar_wait_sleep_bounded(smem_u32(&sm.full[s]), turn & 1, a.err, MOE_DEVERR_WAIT_FULL);
            }
        __syncwarp();
    } else if (warp == MMA_WARP) {
        if (rank == 1 && lane == 0) mbar_arrive_peer(peer_addr(smem_u32(&sm.peer_ready), 0));
        if (rank == 0) {
            const uint32_t idesc = E8 ? umma_idesc_e4m3(256, NT) : umma_idesc(BF, 256, NT);
            int s = 0, turn = 0, nth = 0;
            bool ok = wait.warp(smem_u32(&sm.peer_ready), 0, MOE_DEVERR_WAIT_FULL);
            for (int tile = first; tile < tiles && ok; tile += step, ++nth) {
                const int buf = nth & 1;
                if (nth >= 2 && !wait.warp(smem_u32(&sm.acc_empty[buf]), (nth / 2 - 1) & 1, MOE_DEVERR_WAIT_EMPTY))
                    break;
                tc_after();
                const uint32_t d = tmem + buf * 256;
                for (int kb = 0; kb < steps; ++kb) {
                    if (!wait.warp(smem_u32(&sm.full[s]), turn & 1, MOE_DEVERR_WAIT_FULL)) {
                        ok = false;
                        break;
                    }
                    tc_after();
                    const uint32_t st = st0 + s * stage_bytes;
                    if (elect_one()) {
#pragma unroll
                        for (int h = 0; h < SUB; ++h) {
                            const uint64_t ad = desc_k_inner(st + h * block_bytes), bd = ad + (A_BYTES >> 4);
#pragma unroll
                            for (int j = 0; j < ROW_BYTES / 32; ++j)
                                umma_pair<E8>(d, ad + 2 * j, bd + 2 * j, idesc, kb > 0 || h > 0 || j > 0);
                        }
                        umma_arrive_pair(smem_u32(&sm.empty[s]));
                    }
                    if (++s == n_stages) s = 0, ++turn;
                }
                if (elect_one()) umma_arrive_pair(smem_u32(&sm.acc_full[buf]));
            }
        }
        __syncwarp();
    } else {
        // EPI / 4 warps to a quarter of the TMEM lanes, 16-token chunks in turn.
        // A lane's 16 results are 16 tokens of one output; wide: they go through
        // shared memory, so that a store takes 64 bytes of 8 tokens each.
        const int quarter = warp & 3, part = (warp - 2) >> 2;
        uint16_t(*out)[32] = sm.out[warp - 2];
        const bool has_res = EPI == P_EPI_RES && a.res;  // (see P_EPI_RES)
        int nth = 0;
        bool ok = true;
        with_act(a.act, [&](auto act) {
            for (int tile = first; tile < tiles; tile += step, ++nth) {
                const int buf = nth & 1;
                int tn, tt;
                pair_tile(a, tile, tn, tt);
                const int n_warp = tn * 256 + (int)rank * 128 + quarter * 32, n = n_warp + lane;
                const int t0 = tt * NT, nt = min(NT, a.T - t0);
                const bool in = n < a.N, wide = a.wide && n_warp + 32 <= a.N;
                const float bias = a.bias && in ? to_f32<BF>(a.bias[n]) : 0.0f;
                const float sw = E8 && in ? a.sw[n] : 1.0f;
                if (E8) {
                    // (the barrier: also every warp is done with the tile before the last)
                    const int e = threadIdx.x - 64;
                    static_assert(EPI >= 8, "a thread for each of up to 256 tokens");
                    if (e < 256) sm.sx[buf][e] = e < nt ? a.sx[t0 + e] : 0.0f;
                    named_barrier(1, 32 * EPI);
                }
                if (has_res) {
                    // the residual's lines (up to three a token) to L2 while the products
                    // run (K = 512, N = 2048, T = 8192: 27.6 against 30.5, 8 bits 28.1 and 32.4;
                    // K = N = 4096, T = 1024: 26.8 and 27.2, 18.1 and 19.2)
                    const int n_cta = tn * 256 + (int)rank * 128, n_last = min(n_cta + 127, a.N - 1);
                    const uint16_t* res = a.res + (int64_t)t0 * a.ldr;
                    for (int e = threadIdx.x - 64; e < 4 * nt; e += 32 * EPI)
                        if ((e & 3) < 3) prefetch_l2(res + (int64_t)(e >> 2) * a.ldr + min(n_cta + 64 * (e & 3), n_last));
                }
                // a chunk's residuals are asked for before its sums are there, and the next
                // one's before its results are stored (8 bits, K = 512, N = 2048, T = 8192: 23.6
                // against 26.0; K = 2048, N = 4096, T = 512: 8.4 and 9.4)
                uint16_t v[16];
                auto ask = [&](int c) {
                    const uint16_t* res = a.res + (int64_t)(t0 + c) * a.ldr + n;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        v[j] = in && j < nt - c ? *res : (uint16_t)0;
                        res += a.ldr;
                    }
                };
                if (has_res) ask(16 * part);
                // (after a wait that gave up the warp still comes to the barriers)
                ok = ok && wait.warp(smem_u32(&sm.acc_full[buf]), (nth / 2) & 1, MOE_DEVERR_WAIT_FULL);
                if (!ok) continue;
                tc_after();
                const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + buf * 256;
                for (int c = 16 * part; c < nt; c += 4 * EPI) {
                    uint32_t r[16];
                    tmem_ld16_async(src + c, r);
                    float sx[16];
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 f = E8 ? *reinterpret_cast<const float4*>(&sm.sx[buf][c + j]) : make_float4(1, 1, 1, 1);
                        sx[j] = f.x, sx[j + 1] = f.y, sx[j + 2] = f.z, sx[j + 3] = f.w;
                    }
                    tmem_wait_ld16(r);
                    uint16_t y[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float z = __uint_as_float(r[j]);
                        if (E8) z *= sx[j] * sw;
                        z = has_res ? activate_add<decltype(act)::value, E8>(z + bias, to_f32<BF>(v[j]))
                                    : activate<decltype(act)::value, E8>(z + bias);
                        y[j] = from_f32<BF>(z);
                    }
                    if (has_res && c + 4 * EPI < nt) ask(c + 4 * EPI);
                    if (wide) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) out[j][lane] = y[j];
                        __syncwarp();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int t = 8 * h + lane / 4, o = 8 * (lane % 4);
                            const uint4 u = *reinterpret_cast<const uint4*>(&out[t][o]);
                            if (t < nt - c) *reinterpret_cast<uint4*>(a.y + (int64_t)(t0 + c + t) * a.ldy + n_warp + o) = u;
                        }
                        __syncwarp();
                    } else {
                        uint16_t* dst = a.y + (int64_t)(t0 + c) * a.ldy + n;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (in && j < nt - c) *dst = y[j];
                            dst += a.ldy;
                        }
                    }
                }
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_peer_relaxed(peer_addr(smem_u32(&sm.acc_empty[buf]), 0));
            }
        });
        __syncwarp();
    }
    tc_before();
    __syncthreads();
    cluster_sync();
    if (warp == MMA_WARP) {
        tc_after();
        tmem_free_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------- launch
moe_status launch_clustered(const void* kern, int grid, int threads, int cluster, size_t smem, cudaStream_t s,
                            void** args, const char* what) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    count_launch();
    cudaError_t e = cudaLaunchKernelExC(&cfg, kern, args);
    return e == cudaSuccess ? MOE_OK : cuda_status(e, what);
}

// What a call is named in messages.
template <bool E8>
constexpr const char* LAUNCH = E8 ? "moe_linear_8bit: launch" : "moe_linear: launch";
template <bool E8>
constexpr const char* SMEM = E8 ? "moe_linear_8bit: shared memory" : "moe_linear: shared memory";
template <bool E8>
constexpr const char* MAPS = E8 ? "moe_linear_8bit: tensor map encoding failed" : "moe_linear: tensor map encoding failed";

// Clusters of `size` (2, 4 or 8) CTAs of a kernel that takes a whole SM each, that
// the device runs at once: fewer than its SMs would give, as a cluster stays
// within a GPC.  Asked once per device.
inline int max_clusters(const void* kern, int threads, size_t smem, int size) {
    constexpr int kMaxDev = 64;
    static int known[kMaxDev][9];
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return num_sms() / size;
    if (known[dev][size] == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)size);
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {(unsigned)size, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = num_sms() / size;
        }
        known[dev][size] = n;
    }
    return known[dev][size];
}

template <bool BF, bool E8, int NT, int STAGES>
moe_status run_split(CUtensorMap& wmap, CUtensorMap& xmap, LinearArgs& a, int S, cudaStream_t s) {
    auto kern = linear_split_kernel<BF, E8, NT, STAGES>;
    const size_t smem = sizeof(SplitSmem<NT, STAGES>) + 1024;
    cudaError_t e = ensure_smem_attr(kern, (int)smem);
    if (e != cudaSuccess) return cuda_status(e, SMEM<E8>);
    void* args[] = {&wmap, &xmap, &a, &S};
    return launch_clustered((const void*)kern, a.n_tiles * a.t_tiles * S, THREADS, S, smem, s, args, LAUNCH<E8>);
}

template <bool BF, bool E8>
moe_status run_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, int K, LinearArgs a, cudaStream_t s) {
    constexpr int SIZE = E8 ? 1 : 2;  // bytes of an input
    const int sms = num_sms();
    a.kblocks = (K + BK<E8> - 1) / BK<E8>;
    auto maps = [&](CUtensorMap* wmap, CUtensorMap* xmap, int box_t) {
        const int64_t wd[2] = {K, a.N}, xd[2] = {K, a.T};
        // (a single row's stride is never used, but has to be valid)
        const int64_t any = (K + 15) / 16 * 16;
        const int64_t ws = a.N == 1 ? any : ldw, xs = a.T == 1 ? any : ldx;
        const int wb[2] = {BK<E8>, 128}, xb[2] = {BK<E8>, box_t};
        if (E8) return make_map8(wmap, w, 2, wd, &ws, wb) && make_map8(xmap, x, 2, xd, &xs, xb);
        return make_map16(wmap, BF, w, 2, wd, &ws, wb) && make_map16(xmap, BF, x, 2, xd, &xs, xb);
    };
    const int64_t ctas = (a.N + 15) / 16;
    if (const int warps = E8 ? few_warps8(a.T, ctas, K, sms) : a.T <= FEW_T ? FEW_WARPS : 0) {
        FewArgs f = {(const uint8_t*)x,  (const uint8_t*)w, ldx * SIZE,
                     ldw * SIZE,         (int64_t)K * SIZE, E8 && (int64_t)a.N * K <= FEW_AHEAD * sms, a};
        auto kern = linear_few_kernel<BF, E8, FEW_WARPS, 1>;
        if constexpr (E8) {
            auto of_warps = [&](auto tt) {
                constexpr int TT = decltype(tt)::value;
                if (warps == 4) kern = linear_few_kernel<BF, E8, 4, TT>;
                if (warps == 8) kern = linear_few_kernel<BF, E8, 8, TT>;
                if (warps == 12) kern = linear_few_kernel<BF, E8, 12, TT>;
                if (warps == 16) kern = linear_few_kernel<BF, E8, 16, TT>;
            };
            if (a.T <= 8) of_warps(std::integral_constant<int, 1>());
            else if (a.T <= 16) of_warps(std::integral_constant<int, 2>());
            else kern = warps == 8 ? linear_few_kernel<BF, E8, 8, 4> : linear_few_kernel<BF, E8, 16, 4>;
        }
        cudaError_t e = launch_pdl(kern, dim3((unsigned)ctas), dim3(32 * warps), 0, s, f);
        return e == cudaSuccess ? MOE_OK : cuda_status(e, LAUNCH<E8>);
    }
    CUtensorMap wmap, xmap;
    // The pair kernel's token tile c whose rounds over the SM pairs cost least.  In
    // cycles, a block of inputs costs 256 + c: as many times 128 bytes of shared
    // memory as its copies write and its products read (an instruction of 256 x c
    // takes c / 2 of them, four a block, which is less up to c = 256); a round about
    // 1500 for its start, the last one 20 a token for its results.  (Against the
    // tokens alone: K = 4096, N = 8192, T = 1024 42.6 and 46.6, 8 bits 26.3 and 28.9;
    // N = 6144, T = 3000 79.9 and 88.4, 44.6 and 49.7.)
    const int pairs = sms > 1 ? sms / 2 : 1, n256 = (a.N + 255) / 256;
    int c_best = 0;
    int64_t pair_cost = INT64_MAX;
    for (int c = 256; c >= 32; c -= 16) {
        const int64_t tiles = (int64_t)n256 * ((a.T + c - 1) / c);
        const int64_t cost = (tiles + pairs - 1) / pairs * ((int64_t)a.kblocks * (256 + c) + 1500) + 20 * c;
        if (cost < pair_cost) pair_cost = cost, c_best = c;
    }
    // The split kernel's tile and cluster: the largest power of two that keeps the
    // CTAs within what the SMs hold at once, two each up to 32 tokens (clusters of 3
    // or 6 do not fill the GPCs: 22.5 against 13.3 at one token, K = 4096, N = 6144).
    const int nt = a.T <= 16 ? 16 : a.T <= 32 ? 32 : a.T <= 64 ? 64 : 128;
    const int n128 = (a.N + 127) / 128, t_tiles = (a.T + nt - 1) / nt;
    const int64_t tiles = (int64_t)n128 * t_tiles;
    int S = 1;
    bool split;
    if (E8) {
        // A second CTA on an SM needs 8 blocks of its own to pay (K = 4096, N = 4096, 16
        // tokens: clusters of 4 5.0, of 8 6.3), and clusters of 8 that do not
        // run at once take twice as long (K = 4096, N = 2048, 128 tokens: 13.0, of 4
        // 8.8).
        using Sm = SplitSmem<128, 2>;
        auto big = linear_split_kernel<BF, E8, 128, 2>;
        auto room = [&](int size) -> int64_t {
            if (nt <= 32) return (a.kblocks >= 8 * size ? 2 : 1) * sms / size;
            if (ensure_smem_attr(big, (int)sizeof(Sm) + 1024) != cudaSuccess) return sms / size;
            return max_clusters((const void*)big, THREADS, sizeof(Sm) + 1024, size);
        };
        while (S < 8 && 4 * S <= a.kblocks && tiles <= room(2 * S)) S *= 2;
        // Its time in the same cycles: its blocks' traffic, 3.2 (128 + nt) each, and 63
        // a token for the join (constants from 200 sizes, K from 1024 to 8192, N from
        // 512 to 12288, T from 16 to 256; there the choice is 1 % from the better one
        // on average).
        const int64_t rounds = (tiles * S + sms - 1) / sms;  // (two CTAs on an SM share its memory)
        const int64_t cost = rounds * (((int64_t)(a.kblocks + S - 1) / S) * 16 * (128 + nt) / 5 + 63 * (a.T < nt ? a.T : nt));
        split = cost < pair_cost;
    } else {
        while (S < 8 && 2 * S * tiles <= (nt <= 32 ? 2 : 1) * sms && 4 * S <= a.kblocks) S *= 2;
        const int64_t tiles128 = (int64_t)n128 * ((a.T + 127) / 128);
        split = a.T <= SPLIT_T || (8 * tiles128 <= sms && K >= SPLIT_K);
    }
    if (!split) {
        const int nt = c_best;
        a.n_tiles = n256;
        a.t_tiles = (a.T + nt - 1) / nt;
        // Results 16 bytes at a time where a pair has several tiles one after
        // another and its stores stand beside the next one's copies (8 bits, K = N =
        // 4096, T = 4096: 45.1, each output by itself 48.1); the way through shared
        // memory makes a last tile longer (T = 256: 9.6 and 9.4).
        a.wide = aligned16(a.y) && a.ldy % 8 == 0 && (int64_t)a.n_tiles * a.t_tiles > 2 * pairs;
        if (!maps(&wmap, &xmap, nt / 2)) {
            set_error("%s", MAPS<E8>);
            return MOE_ERR_CUDA;
        }
        const bool many = a.res || (E8 && a.act > MOE_ACT_RELU && K <= P_EPI_ACT_K && (int64_t)a.n_tiles * a.t_tiles > pairs);
        auto kern = many ? (nt <= WIDE_STAGE_NT ? linear_pair_kernel<BF, E8, 2, P_EPI_RES> : linear_pair_kernel<BF, E8, 1, P_EPI_RES>)
                          : (nt <= WIDE_STAGE_NT ? linear_pair_kernel<BF, E8, 2, P_EPI> : linear_pair_kernel<BF, E8, 1, P_EPI>);
        const size_t smem = sizeof(PairSmem) + 1024;
        cudaError_t e = ensure_smem_attr(kern, (int)smem);
        if (e != cudaSuccess) return cuda_status(e, SMEM<E8>);
        void* args[] = {&wmap, &xmap, &a, (void*)&nt};
        const int64_t tiles = (int64_t)a.n_tiles * a.t_tiles;
        return launch_clustered((const void*)kern, (int)(2 * (tiles < pairs ? tiles : pairs)),
                                64 + 32 * (many ? P_EPI_RES : P_EPI), 0, smem, s, args, LAUNCH<E8>);
    }
    if (!maps(&wmap, &xmap, nt)) {
        set_error("%s", MAPS<E8>);
        return MOE_ERR_CUDA;
    }
    a.n_tiles = n128, a.t_tiles = t_tiles;
    switch (nt) {
        case 16: return run_split<BF, E8, 16, 2>(wmap, xmap, a, S, s);
        case 32: return run_split<BF, E8, 32, 2>(wmap, xmap, a, S, s);
        case 64: return run_split<BF, E8, 64, 3>(wmap, xmap, a, S, s);
        default: return run_split<BF, E8, 128, 2>(wmap, xmap, a, S, s);
    }
}

}  // namespace
}  // namespace moe
