// y = act(x W^T + bias) + residual on the tensor cores.
//
// Both kernels compute y^T tiles: the weights' rows are the tensor core's M
// (the accumulator's TMEM lanes), the tokens its N (the columns).  So one
// token needs no more than 16 columns, and whatever the number of tokens a
// warp's 32 lanes hold 32 consecutive outputs of one token, whose store is
// contiguous for every row stride.  Operands come through TMA (64 inputs = 128
// bytes a row, 128-byte swizzle; rows and inputs past the end read as zeros),
// so ragged sizes need no code in the main loop.
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
#ifndef LINEAR_SPLIT_T
#define LINEAR_SPLIT_T 64
#endif
#ifndef LINEAR_CTAS
#define LINEAR_CTAS 2
#endif

// ---------------------------------------------------------------- split kernel
// One tile of 128 outputs x NT tokens per cluster, its sum over the inputs
// split over the cluster's CTAs: each keeps its part of the sum in TMEM, puts
// it into its shared memory, and every CTA adds up (in rank order, so the
// result does not depend on timing) and finishes a share of the tile through
// distributed shared memory.
template <int NT, int STAGES>
struct __align__(1024) SplitSmem {
    struct Stage {
        uint8_t a[A_BYTES];
        uint8_t b[NT * BK * 2];
    };
    union {
        Stage st[STAGES];
        float part[NT][128];
    };
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
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x / S, rank = blockIdx.x % S;
    const int n0 = (tile / a.t_tiles) * 128, t0 = (tile % a.t_tiles) * NT;
    const int kb0 = (int)((int64_t)a.kblocks * rank / S), kb1 = (int)((int64_t)a.kblocks * (rank + 1) / S);
    const int nt = min(NT, a.T - t0);
    const Waits wait{a.err, &sm.failed};

    const int n_kb = kb1 - kb0;
    auto kblock = [&](int i) { return (kb0 + i) * BK; };
    const int pre = min(STAGES, n_kb);
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
        }
        mbar_init(smem_u32(&sm.acc_full), 1);
        sm.failed = 0;
        mbar_fence_init();
        // the first stages' weights do not depend on what runs before
        for (int i = 0; i < pre; ++i) {
            mbar_arrive_expect_tx(smem_u32(&sm.full[i]), A_BYTES + NT * BK * 2);
            tma_2d(smem_u32(sm.st[i].a), &wmap, kblock(i), n0, smem_u32(&sm.full[i]));
        }
        prefetch_map(&xmap);
    }
    if (warp == MMA_WARP) tmem_alloc(smem_u32(&sm.tmem), COLS);
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = sm.tmem;

    pdl_wait();
    if (warp == TMA_WARP) {
        if (elect_one())
            for (int i = 0; i < pre; ++i) tma_2d(smem_u32(sm.st[i].b), &xmap, kblock(i), t0, smem_u32(&sm.full[i]));
        int s = 0, turn = 1, i = pre;
        for (; i < n_kb; ++i) {
            if (!wait.warp(smem_u32(&sm.empty[s]), (turn - 1) & 1, MOE_DEVERR_WAIT_EMPTY)) break;
            if (elect_one()) {
                const uint32_t full = smem_u32(&sm.full[s]);
                mbar_arrive_expect_tx(full, A_BYTES + NT * BK * 2);
                tma_2d(smem_u32(sm.st[s].a), &wmap, kblock(i), n0, full);
                tma_2d(smem_u32(sm.st[s].b), &xmap, kblock(i), t0, full);
            }
            if (++s == STAGES) s = 0, ++turn;
        }
        // (after a wait that gave up: the copies in flight land before the CTA ends)
        if (i < n_kb)
            for (int j = max(0, i - STAGES); j < i; ++j)
                mbar_wait_sleep_bounded(smem_u32(&sm.full[j % STAGES]), (j / STAGES) & 1, a.err, MOE_DEVERR_WAIT_FULL);
    } else if (warp == MMA_WARP) {
        constexpr uint32_t idesc = umma_idesc(BF, 128, NT);
        int s = 0, turn = 0;
        for (int i = 0; i < n_kb; ++i) {
            if (!wait.warp(smem_u32(&sm.full[s]), turn & 1, MOE_DEVERR_WAIT_FULL)) break;
            tc_after();
            const uint64_t ad = desc_k_inner(smem_u32(sm.st[s].a)), bd = desc_k_inner(smem_u32(sm.st[s].b));
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < BK / 16; ++j) umma(tmem, ad + 2 * j, bd + 2 * j, idesc, i > 0 || j > 0);
                umma_arrive(smem_u32(&sm.empty[s]));
            }
            if (++s == STAGES) s = 0, ++turn;
        }
        if (elect_one()) umma_arrive(smem_u32(&sm.acc_full));
    }
    __syncwarp();

    if (warp >= 2) {
        const int quarter = warp & 3, row = quarter * 32 + lane;
        if (wait.warp(smem_u32(&sm.acc_full), 0, MOE_DEVERR_WAIT_FULL)) {
            tc_after();
            for (int c = 0; c < (nt + 15) / 16; ++c) {
                uint32_t r[16];
                tmem_ld16_async(tmem + ((uint32_t)(quarter * 32) << 16) + 16 * c, r);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) sm.part[16 * c + j][row] = __uint_as_float(r[j]);
            }
        }
        tc_before();
    }
    __syncwarp();
    if (S > 1)
        cluster_sync();
    else
        __syncthreads();
    with_act(a.act, [&](auto act) {
        const uint32_t part = smem_u32(&sm.part[0][0]);
        const int total = nt * 32;  // groups of 4 consecutive outputs of a token
        const int e1 = (int)((int64_t)total * (rank + 1) / S);
        for (int e = (int)((int64_t)total * rank / S) + threadIdx.x; e < e1; e += THREADS) {
            const int n = n0 + 4 * (e & 31), t = t0 + (e >> 5), m = min(4, a.N - n);
            if (m <= 0) continue;
            uint16_t* dst = a.y + (int64_t)t * a.ldy + n;
            float bias[4], res[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bias[j] = a.bias && j < m ? to_f32<BF>(a.bias[n + j]) : 0.0f;
                res[j] = a.res && j < m ? to_f32<BF>(a.res[(int64_t)t * a.ldr + n + j]) : 0.0f;
            }
            float v[4] = {};
            if (S > 1) {
                float4 p[8];
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (s < S) p[s] = peer_ld4(peer_addr(part + 16 * e, s));
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (s < S) v[0] += p[s].x, v[1] += p[s].y, v[2] += p[s].z, v[3] += p[s].w;
            } else {
                const float4 p = reinterpret_cast<const float4*>(&sm.part[0][0])[e];
                v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w;
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
    tc_before();
    __syncwarp();
    if (S > 1)
        cluster_sync();  // (the peers have read this CTA's part)
    else
        __syncthreads();
    if (warp == MMA_WARP) {
        tc_after();
        tmem_free(tmem, COLS);
    }
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
    uint8_t st[P_STAGE_BYTES];  // stages of 128 weight rows and nt / 2 tokens
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

template <bool BF>
__global__ void __launch_bounds__(P_THREADS) __cluster_dims__(2, 1, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                       const LinearArgs a, const int NT) {
    extern __shared__ __align__(1024) uint8_t dyn[];
    PairSmem& sm = *reinterpret_cast<PairSmem*>(dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1, tiles = a.n_tiles * a.t_tiles;
    const Waits wait{a.err, &sm.failed};
    const int stage_bytes = A_BYTES + (NT * 64 + 1023) / 1024 * 1024;
    const int n_stages = min(P_MAX_STAGES, P_STAGE_BYTES / stage_bytes);

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
            for (int kb = 0; kb < a.kblocks; ++kb) {
                if (turn > 0 && !wait.warp(smem_u32(&sm.empty[s]), (turn - 1) & 1, MOE_DEVERR_WAIT_EMPTY)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    // the even CTA's barrier counts the bytes of both
                    const uint32_t full = smem_u32(&sm.full[s]), st = st0 + s * stage_bytes;
                    if (rank == 0) mbar_arrive_expect_tx(full, 2 * A_BYTES + NT * 128);
                    tma_2d_pair(st, &wmap, kb * BK, n0, full);
                    tma_2d_pair(st + A_BYTES, &xmap, kb * BK, t0, full);
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
                for (int kb = 0; kb < a.kblocks; ++kb) {
                    if (!wait.warp(smem_u32(&sm.full[s]), turn & 1, MOE_DEVERR_WAIT_FULL)) {
                        ok = false;
                        break;
                    }
                    tc_after();
                    const uint32_t st = st0 + s * stage_bytes;
                    const uint64_t ad = desc_k_inner(st), bd = desc_k_inner(st + A_BYTES);
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < BK / 16; ++j) umma_pair(d, ad + 2 * j, bd + 2 * j, idesc, kb > 0 || j > 0);
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
    CUtensorMap wmap, xmap;
    if (a.T > LINEAR_SPLIT_T) {
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
        auto kern = linear_pair_kernel<BF>;
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
    // the largest power of two that keeps the CTAs within two for each SM
    // (clusters of other sizes do not fill the GPCs)
    int S = 1;
    while (S < 8 && 2 * S * tiles <= LINEAR_CTAS * sms && 2 * S <= a.kblocks) S *= 2;
    switch (nt) {
        case 16: return run_split<BF, 16, 6>(wmap, xmap, a, S, s);
        case 32: return run_split<BF, 32, 5>(wmap, xmap, a, S, s);
        case 64: return run_split<BF, 64, 4>(wmap, xmap, a, S, s);
        default: return run_split<BF, 128, 3>(wmap, xmap, a, S, s);
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
