// y = act(x W^T + bias) + residual on the tensor cores.
//
// All three kernels compute y^T tiles: the weights' rows are the tensor core's M,
// the tokens its N.  So one token needs no more than 8 or 16 columns.  In the two
// tcgen05 kernels the rows are the accumulator's TMEM lanes: whatever the number
// of tokens a warp's 32 lanes hold 32 consecutive outputs of one token, whose
// store is contiguous for every row stride.  Their operands come through TMA (64
// inputs = 128 bytes a row, 128-byte swizzle; rows and inputs past the end read
// as zeros), so ragged sizes need no code in the main loop.  No kernel here lets its
// dependents start early: y may be the activations that a routing reads before
// its wait (the launch contract in common.cuh).
#include <type_traits>

#include "elem.cuh"
#include "tc05.cuh"

namespace moe {
namespace {

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if (ACT == MOE_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if (ACT == MOE_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    if (ACT == MOE_ACT_GELU_TANH)
        return 0.5f * z * (1.0f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
    if (ACT == MOE_ACT_SILU) return z / (1.0f + expf(-z));
    return z;
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
    uint16_t* y;
    int64_t ldr, ldy;
    int T, N, kblocks, act;
    int n_tiles, t_tiles;
    int* err;
};

constexpr int BK = 64;                 // inputs of one stage
constexpr int A_BYTES = 128 * BK * 2;  // 128 weight rows
constexpr int TMA_WARP = 0, MMA_WARP = 1;
constexpr int THREADS = 192;           // TMA, MMA and four epilogue warps

// Which kernel (times on a GB300, microseconds, weights from memory):
//   - up to FEW_T tokens the weights stream through registers (K = 4096, N =
//     6144: 9.0 at 1 token and 9.1 at 8, 83 % of the copy rate; the split
//     kernel 11.5 and 11.6);
//   - up to SPLIT_T tokens, and above where 128 x 128 tiles leave room for
//     clusters of 8 over a long sum, the split kernel (T = 64, N = 4096: 10.8,
//     pairs 13.1, but N = 6144: 15.3 and 14.5; T = 128, K = 8192, N = 512: 10.8,
//     pairs 18.6; K = 1024: 5.7 and 5.3, hence SPLIT_K);
//   - CTA pairs for the rest (T = 96, N = 6144: 14.3, split 19.4; T = 256: 17.0
//     and 31.9; T = 4096: 110, 97 % of the measured cuBLAS rate).
constexpr int FEW_T = 8;
constexpr int SPLIT_T = 64;
constexpr int SPLIT_K = 2048;
// A stage of the pair kernel holds 128 inputs instead of 64 up to this token
// tile (K = 4096, N = 6144, T = 128: 15.4 against 18.4; T = 512, whose tile
// is 176: 23.3 against 21.1).
constexpr int WIDE_STAGE_NT = 128;

// ---------------------------------------------------------------- few tokens
// Up to 8 tokens: the weights' bytes are all there is, so they go straight
// from memory to registers, each read once, 16 bytes a lane.  One CTA takes 16
// outputs, its warps a share of the inputs each.  mma.sync m16n8k16 with the
// weights as A and the tokens as B: a lane's 16 bytes of a row are taken as
// the k's of two of its fragments, the same way in A and in B, so the sum
// only runs in another order.
constexpr int FEW_WARPS = 8;
constexpr int FEW_UNROLL = 4;  // 32-input steps in flight a warp

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

struct FewArgs {
    const uint16_t *x, *w;
    int64_t ldx, ldw;
    int K;
    LinearArgs a;
};

template <bool BF>
__global__ void __launch_bounds__(32 * FEW_WARPS, 24 / FEW_WARPS) linear_few_kernel(const FewArgs f) {
    __shared__ float part[FEW_WARPS][8][16];
    const LinearArgs& a = f.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int n0 = blockIdx.x * 16;
    // steps of 32 inputs: 4 lanes x 16 bytes of a row
    const int steps = (f.K + 31) / 32;
    const int s0 = steps * warp / FEW_WARPS, s1 = steps * (warp + 1) / FEW_WARPS;
    // (rows past the end read the last one again; their sums are dropped)
    const uint16_t* w0 = f.w + (int64_t)min(n0 + g, a.N - 1) * f.ldw + 8 * q;
    const uint16_t* w1 = f.w + (int64_t)min(n0 + g + 8, a.N - 1) * f.ldw + 8 * q;
    const uint16_t* xr = f.x + (int64_t)min(g, a.T - 1) * f.ldx + 8 * q;
    const int last = f.K - 8 * q;  // a lane's inputs end there
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 u0[FEW_UNROLL], u1[FEW_UNROLL], b[FEW_UNROLL];
    auto inside = [&](int s) { return s < s1 && 32 * s < last; };
    auto load_w = [&](int s, int i) {
        u0[i] = inside(s) ? ldg_stream(w0 + 32 * s) : zero;
        u1[i] = inside(s) ? ldg_stream(w1 + 32 * s) : zero;
    };
    auto load_x = [&](int s, int i) { b[i] = inside(s) ? *reinterpret_cast<const uint4*>(xr + 32 * s) : zero; };
    // (before the weights too: whatever ran before may have written them)
    pdl_wait();
#pragma unroll
    for (int i = 0; i < FEW_UNROLL; ++i) load_w(s0 + i, i), load_x(s0 + i, i);
    float acc[4] = {};
    for (int s = s0; s < s1; s += FEW_UNROLL) {
#pragma unroll
        for (int i = 0; i < FEW_UNROLL; ++i) {
            mma_16x8x16<BF>(acc, u0[i].x, u1[i].x, u0[i].y, u1[i].y, b[i].x, b[i].y);
            mma_16x8x16<BF>(acc, u0[i].z, u1[i].z, u0[i].w, u1[i].w, b[i].z, b[i].w);
            load_w(s + i + FEW_UNROLL, i);
            load_x(s + i + FEW_UNROLL, i);
        }
    }
    // acc: rows g and g + 8, tokens 2q and 2q + 1
    part[warp][2 * q][g] = acc[0];
    part[warp][2 * q + 1][g] = acc[1];
    part[warp][2 * q][g + 8] = acc[2];
    part[warp][2 * q + 1][g + 8] = acc[3];
    __syncthreads();
    static_assert(FEW_WARPS >= 4, "a thread for each of 8 tokens x 16 outputs");
    const int t = threadIdx.x >> 4, n = n0 + (threadIdx.x & 15);
    if (t < min(8, a.T) && n < a.N) {
        const float bias = a.bias ? to_f32<BF>(a.bias[n]) : 0.0f;
        const float res = a.res ? to_f32<BF>(a.res[(int64_t)t * a.ldr + n]) : 0.0f;
        float z = 0.0f;
#pragma unroll
        for (int w = 0; w < FEW_WARPS; ++w) z += part[w][t][threadIdx.x & 15];
        z += bias;
        with_act(a.act, [&](auto act) { z = activate<decltype(act)::value>(z); });
        a.y[(int64_t)t * a.ldy + n] = from_f32<BF>(z + res);
    }
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
        uint8_t b[2][NT * BK * 2];
    } st[STAGES];
    float part[NT * 128];  // [source CTA][token][own output]
    uint64_t full[STAGES], empty[STAGES], acc_full;
    uint32_t tmem;
    int failed;
};

template <bool BF, int NT, int STAGES>
__global__ void __launch_bounds__(THREADS)
    linear_split_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                        const LinearArgs a, const int S) {
    using Smem = SplitSmem<NT, STAGES>;
    extern __shared__ __align__(1024) uint8_t dyn[];
    Smem& sm = *reinterpret_cast<Smem*>(dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u));
    constexpr uint32_t COLS = NT < 32 ? 32 : NT;
    constexpr uint32_t BYTES = 2 * (A_BYTES + NT * BK * 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x / S, rank = blockIdx.x % S;
    const int n0 = (tile / a.t_tiles) * 128, t0 = (tile % a.t_tiles) * NT;
    // stages of 128 inputs
    const int steps = (a.kblocks + 1) / 2;
    const int k0 = (int)((int64_t)steps * rank / S), n_k = (int)((int64_t)steps * (rank + 1) / S) - k0;
    const int nt = min(NT, a.T - t0);
    const Waits wait{a.err, &sm.failed};
    const int pre = min(STAGES, n_k);
    auto load_w = [&](int s, int i) {
        for (int h = 0; h < 2; ++h)
            tma_2d(smem_u32(sm.st[s].a[h]), &wmap, (k0 + i) * 2 * BK + h * BK, n0, smem_u32(&sm.full[s]));
    };
    auto load_x = [&](int s, int i) {
        for (int h = 0; h < 2; ++h)
            tma_2d(smem_u32(sm.st[s].b[h]), &xmap, (k0 + i) * 2 * BK + h * BK, t0, smem_u32(&sm.full[s]));
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
        constexpr uint32_t idesc = umma_idesc(BF, 128, NT);
        int s = 0, turn = 0;
        for (int i = 0; i < n_k; ++i) {
            if (!wait.warp(smem_u32(&sm.full[s]), turn & 1, MOE_DEVERR_WAIT_FULL)) break;
            tc_after();
            const uint64_t ad = desc_k_inner(smem_u32(sm.st[s].a)), bd = desc_k_inner(smem_u32(sm.st[s].b));
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    umma(tmem, ad + (j / 4) * (A_BYTES >> 4) + 2 * (j % 4), bd + (j / 4) * (NT * BK * 2 >> 4) + 2 * (j % 4),
                         idesc, i > 0 || j > 0);
                umma_arrive(smem_u32(&sm.empty[s]));
            }
            if (++s == STAGES) s = 0, ++turn;
        }
        if (elect_one()) umma_arrive(smem_u32(&sm.acc_full));
    }
    __syncwarp();
    if (S > 1) cluster_wait();  // the peers run

    const int rows = 128 / S;  // outputs of a CTA's share
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
        const int per_token = rows / 4;  // groups of 4 consecutive outputs
        for (int e = threadIdx.x; e < nt * per_token; e += THREADS) {
            const int r4 = 4 * (e % per_token), t = t0 + e / per_token;
            const int n = n0 + rank * rows + r4, m = min(4, a.N - n);
            if (m <= 0) continue;
            uint16_t* dst = a.y + (int64_t)t * a.ldy + n;
            float bias[4], res[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bias[j] = a.bias && j < m ? to_f32<BF>(a.bias[n + j]) : 0.0f;
                res[j] = a.res && j < m ? to_f32<BF>(a.res[(int64_t)t * a.ldr + n + j]) : 0.0f;
            }
            float v[4] = {};
            const float* p = &sm.part[(e / per_token) * rows + r4];
            for (int s = 0; s < S; ++s) {
                const float4 f = *reinterpret_cast<const float4*>(p + s * NT * rows);
                v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = activate<decltype(act)::value>(v[j] + bias[j]) + res[j];
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
constexpr int P_THREADS = 320;  // TMA, MMA and eight epilogue warps
constexpr int P_STAGE_BYTES = 6 * 2 * A_BYTES;
constexpr int P_MAX_STAGES = 10;

struct __align__(1024) PairSmem {
    uint8_t st[P_STAGE_BYTES];
    uint64_t full[P_MAX_STAGES], empty[P_MAX_STAGES], acc_full[2], acc_empty[2];
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

template <bool BF, int SUB>
__global__ void __launch_bounds__(P_THREADS) __cluster_dims__(2, 1, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                       const LinearArgs a, const int NT) {
    extern __shared__ __align__(1024) uint8_t dyn[];
    PairSmem& sm = *reinterpret_cast<PairSmem*>(dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1, tiles = a.n_tiles * a.t_tiles;
    const Waits wait{a.err, &sm.failed};
    // a stage: SUB times 64 inputs of 128 weight rows and nt / 2 tokens
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
            mbar_init(smem_u32(&sm.acc_empty[s]), 16);  // the epilogue warps of both CTAs
        }
        sm.failed = 0;
        prefetch_map(&wmap);
        prefetch_map(&xmap);
        mbar_fence_init();
    }
    if (warp == MMA_WARP) tmem_alloc_pair(smem_u32(&sm.tmem), 512);
    tc_before();
    __syncthreads();
    cluster_sync();
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
                        tma_2d_pair(st + h * block_bytes, &wmap, (kb * SUB + h) * BK, n0, full);
                        tma_2d_pair(st + h * block_bytes + A_BYTES, &xmap, (kb * SUB + h) * BK, t0, full);
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
        if (rank == 0) {
            const uint32_t idesc = umma_idesc(BF, 256, NT);
            int s = 0, turn = 0, nth = 0;
            bool ok = true;
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
                            for (int j = 0; j < BK / 16; ++j)
                                umma_pair(d, ad + 2 * j, bd + 2 * j, idesc, kb > 0 || h > 0 || j > 0);
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
        // two warps to a quarter of the TMEM lanes, 16-token chunks in turn
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        int nth = 0;
        with_act(a.act, [&](auto act) {
            for (int tile = first; tile < tiles; tile += step, ++nth) {
                const int buf = nth & 1;
                int tn, tt;
                pair_tile(a, tile, tn, tt);
                const int n = tn * 256 + (int)rank * 128 + quarter * 32 + lane;
                const int t0 = tt * NT, nt = min(NT, a.T - t0);
                const bool in = n < a.N;
                const float bias = a.bias && in ? to_f32<BF>(a.bias[n]) : 0.0f;
                if (!wait.warp(smem_u32(&sm.acc_full[buf]), (nth / 2) & 1, MOE_DEVERR_WAIT_FULL)) break;
                tc_after();
                const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + buf * 256;
                for (int c = 16 * half; c < nt; c += 32) {
                    uint32_t r[16];
                    tmem_ld16_async(src + c, r);
                    uint16_t* dst = a.y + (int64_t)(t0 + c) * a.ldy + n;
                    const int m = in ? nt - c : 0;
                    uint16_t rv[16];
                    if (a.res) {
                        const uint16_t* res = a.res + (int64_t)(t0 + c) * a.ldr + n;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            rv[j] = j < m ? *res : (uint16_t)0;
                            res += a.ldr;
                        }
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float z = activate<decltype(act)::value>(__uint_as_float(r[j]) + bias);
                        if (a.res) z += to_f32<BF>(rv[j]);
                        if (j < m) *dst = from_f32<BF>(z);
                        dst += a.ldy;
                    }
                }
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_peer(peer_addr(smem_u32(&sm.acc_empty[buf]), 0));
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
                            void** args) {
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
    return e == cudaSuccess ? MOE_OK : cuda_status(e, "moe_linear: launch");
}

template <bool BF, int NT, int STAGES>
moe_status run_split(CUtensorMap& wmap, CUtensorMap& xmap, LinearArgs& a, int S, cudaStream_t s) {
    auto kern = linear_split_kernel<BF, NT, STAGES>;
    const size_t smem = sizeof(SplitSmem<NT, STAGES>) + 1024;
    cudaError_t e = ensure_smem_attr(kern, (int)smem);
    if (e != cudaSuccess) return cuda_status(e, "moe_linear: shared memory");
    void* args[] = {&wmap, &xmap, &a, &S};
    return launch_clustered((const void*)kern, a.n_tiles * a.t_tiles * S, THREADS, S, smem, s, args);
}

template <bool BF>
moe_status run(const void* x, int64_t ldx, const void* w, int64_t ldw, int K, LinearArgs a, cudaStream_t s) {
    const int sms = num_sms();
    auto maps = [&](CUtensorMap* wmap, CUtensorMap* xmap, int box_t) {
        const int64_t wd[2] = {K, a.N}, xd[2] = {K, a.T};
        // (a single row's stride is never used, but has to be valid)
        const int64_t any = (K + 7) / 8 * 8;
        const int64_t ws = a.N == 1 ? any : ldw, xs = a.T == 1 ? any : ldx;
        const int wb[2] = {BK, 128}, xb[2] = {BK, box_t};
        return make_map16(wmap, BF, w, 2, wd, &ws, wb) && make_map16(xmap, BF, x, 2, xd, &xs, xb);
    };
    if (a.T <= FEW_T) {
        FewArgs f = {(const uint16_t*)x, (const uint16_t*)w, ldx, ldw, K, a};
        cudaError_t e = launch_pdl(linear_few_kernel<BF>, dim3((unsigned)((a.N + 15) / 16)), dim3(32 * FEW_WARPS), 0, s, f);
        return e == cudaSuccess ? MOE_OK : cuda_status(e, "moe_linear: launch");
    }
    CUtensorMap wmap, xmap;
    const int64_t tiles128 = (int64_t)((a.N + 127) / 128) * ((a.T + 127) / 128);
    if (a.T > SPLIT_T && !(8 * tiles128 <= sms && K >= SPLIT_K)) {
        // the token tile whose rounds of tiles over the SM pairs cost least
        // (a round costs its tile's tokens, and about 24 tokens' worth of
        // start and end)
        const int pairs = sms / 2;
        a.n_tiles = (a.N + 255) / 256;
        int nt = 0;
        int64_t best = INT64_MAX;
        for (int c = 256; c >= 32; c -= 16) {
            const int64_t tiles = (int64_t)a.n_tiles * ((a.T + c - 1) / c);
            const int64_t cost = (tiles + pairs - 1) / pairs * (c + 24);
            if (cost < best) best = cost, nt = c;
        }
        a.t_tiles = (a.T + nt - 1) / nt;
        if (!maps(&wmap, &xmap, nt / 2)) {
            set_error("moe_linear: tensor map encoding failed");
            return MOE_ERR_CUDA;
        }
        auto kern = nt <= WIDE_STAGE_NT ? linear_pair_kernel<BF, 2> : linear_pair_kernel<BF, 1>;
        const size_t smem = sizeof(PairSmem) + 1024;
        cudaError_t e = ensure_smem_attr(kern, (int)smem);
        if (e != cudaSuccess) return cuda_status(e, "moe_linear: shared memory");
        void* args[] = {&wmap, &xmap, &a, &nt};
        const int64_t tiles = (int64_t)a.n_tiles * a.t_tiles;
        return launch_clustered((const void*)kern, (int)(2 * (tiles < pairs ? tiles : pairs)), P_THREADS, 0, smem, s, args);
    }
    const int nt = a.T <= 16 ? 16 : a.T <= 32 ? 32 : a.T <= 64 ? 64 : 128;
    if (!maps(&wmap, &xmap, nt)) {
        set_error("moe_linear: tensor map encoding failed");
        return MOE_ERR_CUDA;
    }
    a.n_tiles = (a.N + 127) / 128, a.t_tiles = (a.T + nt - 1) / nt;
    const int64_t tiles = (int64_t)a.n_tiles * a.t_tiles;
    // the largest power of two that keeps the CTAs within what the SMs hold at
    // once, two each up to 32 tokens (clusters of 3 or 6 do not fill the GPCs:
    // 22.5 against 13.3 at one token, K = 4096, N = 6144)
    int S = 1;
    while (S < 8 && 2 * S * tiles <= (nt <= 32 ? 2 : 1) * sms && 4 * S <= a.kblocks) S *= 2;
    switch (nt) {
        case 16: return run_split<BF, 16, 2>(wmap, xmap, a, S, s);
        case 32: return run_split<BF, 32, 2>(wmap, xmap, a, S, s);
        case 64: return run_split<BF, 64, 3>(wmap, xmap, a, S, s);
        default: return run_split<BF, 128, 2>(wmap, xmap, a, S, s);
    }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_linear_workspace_size(int T, int N, int K) {
    if (T < 0 || N < 0 || K <= 0) return 0;
    return 256;  // (the error word)
}

moe_status moe_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                      const void* residual, int64_t ldr, void* y, int64_t ldy, int T, int N, int K, int dtype,
                      int act, void* ws, size_t ws_bytes, cudaStream_t stream) {
    MOE_CHECK_ARG(T >= 0 && N >= 0 && K > 0, "moe_linear: T=%d N=%d must not be negative, K=%d must be positive", T, N,
                  K);
    MOE_CHECK_ARG(known_dtype(dtype), "moe_linear: unknown dtype %d", dtype);
    MOE_CHECK_ARG(act >= MOE_ACT_NONE && act <= MOE_ACT_SILU, "moe_linear: unknown activation %d", act);
    if (T == 0 || N == 0) return MOE_OK;
    MOE_CHECK_ARG(x && w && y, "moe_linear: null pointer");
    MOE_CHECK_ARG((T == 1 || (ldx >= K && ldy >= N)) && (N == 1 || ldw >= K) && (T == 1 || !residual || ldr >= N),
                  "moe_linear: a row stride is shorter than its row");
    MOE_CHECK_SUPPORTED(K % 8 == 0, "moe_linear: K=%d must be a multiple of 8", K);
    MOE_CHECK_SUPPORTED((T == 1 || ldx % 8 == 0) && (N == 1 || ldw % 8 == 0),
                        "moe_linear: the row strides of x and w must be multiples of 8 elements");
    MOE_CHECK_SUPPORTED(aligned16(x) && aligned16(w), "moe_linear: x and w must be 16-byte aligned");
    MOE_CHECK_SUPPORTED((((uintptr_t)bias | (uintptr_t)residual | (uintptr_t)y) & 1) == 0,
                        "moe_linear: bias, residual and y must be 2-byte aligned");
    MOE_CHECK_SUPPORTED(K <= INT32_MAX - 64 && (int64_t)((N + 127) / 128) * ((T + 15) / 16) * 8 <= INT32_MAX &&
                            ldx < ((int64_t)1 << 38) && ldw < ((int64_t)1 << 38),
                        "moe_linear: sizes or strides past what one launch covers");
    if (!ws || ws_bytes < moe_linear_workspace_size(T, N, K)) {
        set_error("moe_linear: workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0,
                  moe_linear_workspace_size(T, N, K));
        return MOE_ERR_WORKSPACE;
    }
    MOE_CHECK_SUPPORTED(((uintptr_t)ws & 15) == 0, "moe_linear: ws must be 16-byte aligned");
    LinearArgs a = {};
    a.bias = (const uint16_t*)bias, a.res = (const uint16_t*)residual, a.y = (uint16_t*)y;
    a.ldr = ldr, a.ldy = ldy, a.T = T, a.N = N, a.kblocks = (K + BK - 1) / BK, a.act = act;
    a.err = (int*)ws + 2;
    return dtype == MOE_DT_BF16 ? run<true>(x, ldx, w, ldw, K, a, stream) : run<false>(x, ldx, w, ldw, K, a, stream);
}

}  // extern "C"
