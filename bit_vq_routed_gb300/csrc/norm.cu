// Root-mean-square norm of rows with the residual's addition, its result in 16
// bits and/or in 8 bits (e4m3) with a scale a row, and rows to 8 bits without a
// norm.
//
//   h = round16(x + residual)             (or x itself)
//   r = 1 / sqrt(mean h^2 + eps),   y = h r w
//   a = max(max |y|, 1e-30),   q = e4m3(y 448 / a),   scale = a / 448
//
// (q from h w 448 / max |h w|, in which r cancels out, rounded once in fp32: a bf16 row's
// values are those of the exact quotient.)  r is one number a row, so max |y| = r max
// |h w|: the sum of squares and the largest magnitude are reduced together, and a row
// passes through the registers of its block once.  Across lanes the largest magnitude
// is compared by its bits as an unsigned number, where NaN lies above infinity above
// everything finite: what is not finite in a row reaches its scale.
//
// Bytes are all there is (8192 rows of 4096, fp32 onto a bf16 stream, 8-bit
// result: 302 MB in 47.0 us, 6.4 TB/s, 95 % of the copy rate).  What carries them is
// the next row's loads in flight while a row is reduced, and one barrier a row.
#include <cuda_fp8.h>

#include "elem.cuh"

namespace moe {
namespace {

struct NormArgs {
    const void* x;  // 16 bits, or fp32
    const uint16_t *res, *w;
    uint16_t *h, *y;
    uint8_t* q;
    float* scales;
    int64_t ldx, ldr, ldh, ldy, ldq;
    float eps;
    int T, H;
};

constexpr float E4M3_MAX = 448.0f;
constexpr float LEAST = 1e-30f;
// From here on r = 1 / sqrt(mean + eps) is at most 7.5e5, so r 448 / LEAST, and 448 over
// an h w whose r h w reaches LEAST, are within fp32.  Below, rows next to zero take their
// products with r first.
constexpr float LOW_EPS = 1.8e-12f;

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// max(m, |v|), NaN where either is
__device__ __forceinline__ float max_abs(float m, float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
    return r;
}
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// v 448 / big: 448 / big as a number and what its rounding left, so that the sum of the
// two products is the quotient rounded once; exact quotients stay exact, and a 16-bit
// value halfway between two of e4m3 goes to the even one.
struct Quotient {
    float inv, left;
    __device__ __forceinline__ explicit Quotient(float big) : inv(E4M3_MAX / big) {
        left = fmaf(-inv, big, E4M3_MAX) * (inv / E4M3_MAX);
    }
    __device__ __forceinline__ float operator()(float v) const { return fmaf(v, inv, v * left); }
};

// Element i of thread `tid`'s share of a row: each 8 of them belong to 256 neighbours
// that the warp holds, VEC: 8 neighbours a lane (16-byte accesses of 16-bit values),
// else lane after lane.
template <bool VEC>
__device__ __forceinline__ int element(int i, int tid, int threads) {
    if (VEC) return 8 * ((i / 8) * threads + tid) + i % 8;
    return 8 * ((i / 8) * threads + (tid & ~31)) + 32 * (i % 8) + (tid & 31);
}

// A thread's N elements of a row as they lie in memory; single 16-bit ones in a
// register each, as joining two would wait for them.
template <bool X32, bool VEC, int N>
struct Raw {
    uint32_t x[X32 || !VEC ? N : N / 2];
    uint32_t r[VEC ? N / 2 : N];
};
__device__ __forceinline__ void put4(uint32_t* w, const uint4& u) { w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w; }

template <bool X32, bool VEC, int N>
__device__ __forceinline__ void load_row(const NormArgs& a, int64_t t, int tid, int threads, Raw<X32, VEC, N>& raw) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint16_t* x16 = (const uint16_t*)a.x + t * a.ldx;
    const float* x32 = (const float*)a.x + t * a.ldx;
    const uint16_t* res = a.res ? a.res + t * a.ldr : nullptr;
    if (VEC) {
#pragma unroll
        for (int v = 0; v < N / 8; ++v) {
            const int e = element<true>(8 * v, tid, threads);
            const bool in = e < a.H;
            if (X32) {
                put4(&raw.x[8 * v], in ? ldg_stream(x32 + e) : zero);
                put4(&raw.x[8 * v + 4], in ? ldg_stream(x32 + e + 4) : zero);
            } else {
                put4(&raw.x[4 * v], in ? ldg_stream(x16 + e) : zero);
            }
            put4(&raw.r[4 * v], in && res ? *reinterpret_cast<const uint4*>(res + e) : zero);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = element<false>(i, tid, threads);
            const bool in = e < a.H;
            if (X32)
                raw.x[i] = in ? __float_as_uint(x32[e]) : 0;
            else
                raw.x[i] = in ? x16[e] : 0;
            raw.r[i] = in && res ? res[e] : 0;
        }
    }
}

// N 16-bit values (packed in pairs) to a row, from `base` on
template <bool VEC, int N>
__device__ __forceinline__ void store_row(uint16_t* base, const uint32_t (&p)[N / 2], int H, int tid, int threads) {
    if (VEC) {
#pragma unroll
        for (int v = 0; v < N / 8; ++v) {
            const int e = element<true>(8 * v, tid, threads);
            if (e < H)
                *reinterpret_cast<uint4*>(base + e) = make_uint4(p[4 * v], p[4 * v + 1], p[4 * v + 2], p[4 * v + 3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = element<false>(i, tid, threads);
            if (e < H) base[e] = (uint16_t)(i % 2 ? p[i / 2] >> 16 : p[i / 2]);
        }
    }
}

// A row's h w at element e, from memory: the thread's own element, which it may have
// written (h).
template <bool BF, bool X32>
__device__ __forceinline__ float value_again(const NormArgs& a, int64_t t, int e) {
    float v;
    if (a.res && a.h) {
        v = to_f32<BF>(a.h[t * a.ldh + e]);
    } else {
        v = X32 ? ((const float*)a.x)[t * a.ldx + e] : to_f32<BF>(((const uint16_t*)a.x)[t * a.ldx + e]);
        if (a.res) v = to_f32<BF>(from_f32<BF>(v + to_f32<BF>(a.res[t * a.ldr + e])));
    }
    return a.w ? v * to_f32<BF>(a.w[e]) : v;
}

// NORM: the norm; else rows to 8 bits alone.  A block takes rows blockIdx.x,
// + gridDim.x, ..., one after another; the next row's loads are under way while
// one is reduced and stored.  LOW: rows next to zero are told from the others, for any
// eps (see LOW_EPS).
template <bool BF, bool X32, bool NORM, bool VEC, int N, bool LOW>
__global__ void __launch_bounds__(1024) rows_kernel(const NormArgs a) {
    // A row's sum is that of 8 neighbours a lane, of 32 lanes, of all warps' parts in
    // order, whether a thread holds one such run of 8 or two: a row's result
    // depends neither on N nor on the rows beside it.
    constexpr int RUNS = N / 8;
    __shared__ float part_s[2][32 * RUNS];
    __shared__ uint32_t part_m[2][32];
    const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    // (the norm writes 16-bit activations: no early start of its dependents, see the
    // launch contract in common.cuh; 8-bit rows are read behind a wait only)
    if (!NORM) pdl_launch_dependents();
    uint32_t w2[N / 2];
    if (NORM) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const int e0 = element<VEC>(i, tid, threads), e1 = element<VEC>(i + 1, tid, threads);
            const uint16_t one = from_f32<BF>(1.0f);
            w2[i / 2] = (uint32_t)(a.w && e0 < a.H ? a.w[e0] : one) | (uint32_t)(a.w && e1 < a.H ? a.w[e1] : one) << 16;
        }
    }
    Raw<X32, VEC, N> raw;
    // (not where the registers would not hold them)
    constexpr bool AHEAD_ROW = VEC || N == 8;
    if (AHEAD_ROW) load_row<X32, VEC, N>(a, blockIdx.x, tid, threads, raw);
    int buf = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, buf ^= 1) {
        float v[N];
        if (!AHEAD_ROW) load_row<X32, VEC, N>(a, t, tid, threads, raw);
        {
            uint32_t h2[N / 2];
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                if (X32) {
                    v[i] = __uint_as_float(raw.x[i]), v[i + 1] = __uint_as_float(raw.x[i + 1]);
                } else {
                    const float2 f = unpack2<BF>(VEC ? raw.x[i / 2] : raw.x[i] | raw.x[i + 1] << 16);
                    v[i] = f.x, v[i + 1] = f.y;
                }
                if (NORM && a.res) {
                    const float2 f = unpack2<BF>(VEC ? raw.r[i / 2] : raw.r[i] | raw.r[i + 1] << 16);
                    h2[i / 2] = pack2<BF>(v[i] + f.x, v[i + 1] + f.y);
                    const float2 g = unpack2<BF>(h2[i / 2]);
                    v[i] = g.x, v[i + 1] = g.y;
                }
            }
            if (NORM && a.res && a.h) store_row<VEC, N>(a.h + t * a.ldh, h2, a.H, tid, threads);
        }
        if (AHEAD_ROW && t + gridDim.x < a.T) load_row<X32, VEC, N>(a, t + gridDim.x, tid, threads, raw);
        float sums[RUNS] = {}, sum = 0.0f;
        // The largest |h w|: one instruction a value, or by its bits in two where the
        // registers are full (fp32 x, 1162 rows of 13328: 33.3 against 37.0; bf16 rows,
        // 8192 of 4096: 29.2 against 28.5).
        constexpr bool BY_BITS = X32 && VEC && N > 8;
        float top = 0.0f;
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (NORM) {
                sums[i / 8] = fmaf(v[i], v[i], sums[i / 8]);
                const float2 w = unpack2<BF>(w2[i / 2]);
                v[i] *= i % 2 ? w.y : w.x;
            }
            if (BY_BITS)
                most = max(most, abs_bits(v[i]));
            else
                top = max_abs(top, v[i]);
        }
        if (NORM) {
#pragma unroll
            for (int r = 0; r < RUNS; ++r) {
#pragma unroll
                for (int off = 16; off >= 1; off >>= 1) sums[r] += __shfl_xor_sync(0xffffffffu, sums[r], off);
                if (lane == 0) part_s[buf][r * warps + warp] = sums[r];
            }
        }
        most = __reduce_max_sync(0xffffffffu, BY_BITS ? most : abs_bits(top));
        if (lane == 0) part_m[buf][warp] = most;
        // (one barrier a row: the next row's parts go to the other buffer)
        __syncthreads();
        most = __reduce_max_sync(0xffffffffu, lane < warps ? part_m[buf][lane] : 0u);
        float r = 1.0f;
        if (NORM) {
            sum = lane < RUNS * warps ? part_s[buf][lane] : 0.0f;
            if (RUNS == 2 && lane + 32 < 2 * warps) sum += part_s[buf][lane + 32];
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            r = rsqrtf(sum / (float)a.H + a.eps);
        }
        if (NORM && a.y) {
            uint32_t y2[N / 2];
#pragma unroll
            for (int i = 0; i < N; i += 2) y2[i / 2] = pack2<BF>(v[i] * r, v[i + 1] * r);
            store_row<VEC, N>(a.y + t * a.ldy, y2, a.H, tid, threads);
        }
        if (!NORM || a.q) {
            const float largest = __uint_as_float(most);
            float big = r * largest;
            if (big < LEAST) big = LEAST;  // (not NaN)
            if (tid == 0) a.scales[t] = big / E4M3_MAX;
            uint8_t* q = a.q + t * a.ldq;
            if (NORM && LOW && !(largest >= LEAST && big > LEAST)) {
                const Quotient scaled(big);
#pragma unroll 1
                for (int i = 0; i < N; ++i) {
                    const int e = element<VEC>(i, tid, threads);
                    if (e < a.H) q[e] = (uint8_t)e4m3x2(scaled(value_again<BF, X32>(a, t, e) * r), 0.0f);
                }
            } else {
                // The norm's quotient y / max |y| is that of h w, without r and its rounding.
                Quotient scaled(NORM ? largest : big);
                if (NORM && !LOW && big == LEAST) scaled.inv = r * (E4M3_MAX / LEAST), scaled.left = 0.0f;
                uint16_t q2[N / 2];
#pragma unroll
                for (int i = 0; i < N; i += 2) q2[i / 2] = e4m3x2(scaled(v[i]), scaled(v[i + 1]));
                if (VEC) {
#pragma unroll
                    for (int g = 0; g < N / 8; ++g) {
                        const int e = element<true>(8 * g, tid, threads);
                        if (e < a.H)
                            *reinterpret_cast<uint2*>(q + e) = make_uint2(q2[4 * g] | (uint32_t)q2[4 * g + 1] << 16,
                                                                          q2[4 * g + 2] | (uint32_t)q2[4 * g + 3] << 16);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int e = element<false>(i, tid, threads);
                        if (e < a.H) q[e] = (uint8_t)(i % 2 ? q2[i / 2] >> 8 : q2[i / 2]);
                    }
                }
            }
        }
    }
}

// Rows to 8 bits that are too long for a block's registers (weights of long sums):
// read twice, element by element, the second time mostly from L2.
template <bool BF, bool X32>
__global__ void __launch_bounds__(1024) long_rows_kernel(const NormArgs a) {
    __shared__ uint32_t part[32];
    const int tid = threadIdx.x, threads = blockDim.x;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        auto value = [&](int e) {
            return X32 ? ((const float*)a.x)[t * a.ldx + e] : to_f32<BF>(((const uint16_t*)a.x)[t * a.ldx + e]);
        };
        uint32_t most = 0;
        for (int e = tid; e < a.H; e += threads) most = max(most, abs_bits(value(e)));
        most = __reduce_max_sync(0xffffffffu, most);
        __syncthreads();  // (the last row's parts are read)
        if (tid % 32 == 0) part[tid / 32] = most;
        __syncthreads();
        most = __reduce_max_sync(0xffffffffu, part[tid % 32]);
        float big = __uint_as_float(most);
        if (big < LEAST) big = LEAST;  // (not NaN)
        const Quotient scaled(big);
        if (tid == 0) a.scales[t] = big / E4M3_MAX;
        for (int e = tid; e < a.H; e += threads)
            a.q[t * a.ldq + e] = (uint8_t)e4m3x2(scaled(value(e)), 0.0f);
    }
}

// Elements of a row a thread holds: 8 as far as 1024 threads reach (8192 rows of
// 4096, fp32 onto a stream: 47.1 us, 16 each 54.5; 333 rows of 2051 element by element:
// 3.3 and 4.1), then 16; and 16 where many rows' loads would else keep less than
// AHEAD bytes of an SM under way (8192 rows of 4096 to 8 bits, 16 KB: 28.5 and, with 8, 32.9;
// 4750 rows of 4944 that sum, 20 KB: 31.5 and 35.5).
constexpr int FEW = 8, MANY = 16;
constexpr int MAX_H = 1024 * MANY;
constexpr int AHEAD = 32 * 1024;

template <bool BF, bool X32, bool NORM, int N>
moe_status run(const NormArgs& a, bool vec, const char* what, cudaStream_t s) {
    const int threads = ((a.H + N - 1) / N + 31) / 32 * 32;
    // blocks that stay: as many as an SM holds at 64 registers a thread (twice
    // that and they come in two rounds, 47.4; a block a row: 71)
    const int64_t fit = (int64_t)num_sms() * (1024 / threads);
    const dim3 grid((unsigned)(a.T < fit ? a.T : fit));
    // (element by element always LOW: the compiler's code is shorter there, 333 rows of 2051
    // 1.5 M instructions against 2.2 M, 4000 rows of 4098 37.2 against 42.1; whole pieces only where eps asks for it, 8192 rows of 4096
    // 28.6 to 30.9)
    auto kern = vec ? rows_kernel<BF, X32, NORM, true, N, false> : rows_kernel<BF, X32, NORM, false, N, NORM>;
    if constexpr (NORM)
        if (vec && a.q && a.eps < LOW_EPS) kern = rows_kernel<BF, X32, NORM, true, N, true>;
    cudaError_t e = launch_pdl(kern, grid, dim3(threads), 0, s, a);
    return e == cudaSuccess ? MOE_OK : cuda_status(e, what);
}
template <bool BF, bool X32, bool NORM>
moe_status run(const NormArgs& a, bool vec, const char* what, cudaStream_t s) {
    if (!NORM && a.H > MAX_H) {
        const dim3 grid((unsigned)(a.T < 2 * num_sms() ? a.T : 2 * num_sms()));
        cudaError_t e = launch_pdl(long_rows_kernel<BF, X32>, grid, dim3(1024), 0, s, a);
        return e == cudaSuccess ? MOE_OK : cuda_status(e, what);
    }
    const int threads = ((a.H + FEW - 1) / FEW + 31) / 32 * 32;
    const bool wide = threads > 1024 || (vec && a.T > 4 * num_sms() &&
                                         1024 / threads * a.H * ((X32 ? 4 : 2) + (a.res ? 2 : 0)) < AHEAD);
    return wide ? run<BF, X32, NORM, MANY>(a, vec, what, s) : run<BF, X32, NORM, FEW>(a, vec, what, s);
}

template <bool NORM>
moe_status run(const NormArgs& a, bool bf, bool x32, bool vec, const char* what, cudaStream_t s) {
    if (bf) return x32 ? run<true, true, NORM>(a, vec, what, s) : run<true, false, NORM>(a, vec, what, s);
    return x32 ? run<false, true, NORM>(a, vec, what, s) : run<false, false, NORM>(a, vec, what, s);
}

// whether rows can be moved in 16-byte pieces (q: 8-byte ones)
bool whole_pieces(const NormArgs& a, bool x32) {
    auto fits = [&](const void* p, int64_t ld, int unit, int bytes) {
        return !p || ((uintptr_t)p % bytes == 0 && (a.T == 1 || ld % unit == 0));
    };
    return a.H % 8 == 0 && fits(a.x, a.ldx, x32 ? 4 : 8, 16) && fits(a.res, a.ldr, 8, 16) && fits(a.h, a.ldh, 8, 16) &&
           fits(a.y, a.ldy, 8, 16) && fits(a.q, a.ldq, 8, 8);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_rms_norm(const void* x, int64_t ldx, int x_dtype, const void* residual, int64_t ldr, void* h, int64_t ldh,
                        const void* weight, float eps, void* y, int64_t ldy, uint8_t* q, int64_t ldq, float* scales,
                        int T, int H, int dtype, cudaStream_t stream) {
    MOE_CHECK_ARG(T >= 0 && H > 0, "moe_rms_norm: T=%d must not be negative, H=%d must be positive", T, H);
    MOE_CHECK_ARG(known_dtype(dtype), "moe_rms_norm: unknown dtype %d", dtype);
    MOE_CHECK_ARG(x_dtype == dtype || x_dtype == MOE_DT_F32, "moe_rms_norm: x_dtype=%d must be dtype=%d or MOE_DT_F32",
                  x_dtype, dtype);
    MOE_CHECK_ARG(eps >= 0.0f && eps <= 3.0e38f, "moe_rms_norm: eps=%g must be finite and not negative", (double)eps);
    MOE_CHECK_SUPPORTED(H <= MAX_H, "moe_rms_norm: H=%d above %d", H, MAX_H);
    if (T == 0) return MOE_OK;
    MOE_CHECK_ARG(x, "moe_rms_norm: null pointer");
    MOE_CHECK_ARG(y || q, "moe_rms_norm: y and q are both null");
    MOE_CHECK_ARG(!q == !scales, "moe_rms_norm: q and scales go together");
    MOE_CHECK_ARG(residual || !h, "moe_rms_norm: h without a residual");
    MOE_CHECK_ARG(T == 1 || (ldx >= H && (!residual || ldr >= H) && (!h || ldh >= H) && (!y || ldy >= H) && (!q || ldq >= H)),
                  "moe_rms_norm: a row stride is shorter than its row");
    const bool x32 = x_dtype == MOE_DT_F32;
    MOE_CHECK_SUPPORTED((((uintptr_t)x & (x32 ? 3 : 1)) | (((uintptr_t)residual | (uintptr_t)h | (uintptr_t)weight |
                        (uintptr_t)y) & 1) | ((uintptr_t)scales & 3)) == 0, "moe_rms_norm: a pointer is not aligned to its type");
    NormArgs a = {};
    a.x = x, a.res = (const uint16_t*)residual, a.w = (const uint16_t*)weight, a.h = (uint16_t*)h, a.y = (uint16_t*)y;
    a.q = q, a.scales = scales, a.ldx = ldx, a.ldr = ldr, a.ldh = ldh, a.ldy = ldy, a.ldq = ldq;
    a.eps = eps, a.T = T, a.H = H;
    return run<true>(a, dtype == MOE_DT_BF16, x32, whole_pieces(a, x32), "moe_rms_norm: launch", stream);
}

moe_status moe_rms_norm_packed(const moe_rms_norm_args* p, cudaStream_t stream) {
    MOE_CHECK_ARG(p, "moe_rms_norm_packed: args is null");
    return moe_rms_norm(p->x, p->ldx, p->x_dtype, p->residual, p->ldr, p->h, p->ldh, p->weight, p->eps, p->y, p->ldy, p->q,
                        p->ldq, p->scales, p->T, p->H, p->dtype, stream);
}

moe_status moe_quantize_rows(const void* x, int64_t ldx, int x_dtype, uint8_t* q, int64_t ldq, float* scales, int T, int H,
                             cudaStream_t stream) {
    MOE_CHECK_ARG(T >= 0 && H > 0, "moe_quantize_rows: T=%d must not be negative, H=%d must be positive", T, H);
    MOE_CHECK_ARG(known_dtype(x_dtype) || x_dtype == MOE_DT_F32, "moe_quantize_rows: unknown x_dtype %d", x_dtype);
    MOE_CHECK_SUPPORTED(H <= INT32_MAX - 1024, "moe_quantize_rows: H=%d past what one launch covers", H);
    if (T == 0) return MOE_OK;
    MOE_CHECK_ARG(x && q && scales, "moe_quantize_rows: null pointer");
    MOE_CHECK_ARG(T == 1 || (ldx >= H && ldq >= H), "moe_quantize_rows: a row stride is shorter than its row");
    const bool x32 = x_dtype == MOE_DT_F32;
    MOE_CHECK_SUPPORTED((((uintptr_t)x & (x32 ? 3 : 1)) | ((uintptr_t)scales & 3)) == 0,
                        "moe_quantize_rows: a pointer is not aligned to its type");
    NormArgs a = {};
    a.x = x, a.q = q, a.scales = scales, a.ldx = ldx, a.ldq = ldq, a.T = T, a.H = H;
    return run<false>(a, x_dtype != MOE_DT_F16, x32, whole_pieces(a, x32), "moe_quantize_rows: launch", stream);
}

moe_status moe_quantize_rows_packed(const moe_quantize_rows_args* p, cudaStream_t stream) {
    MOE_CHECK_ARG(p, "moe_quantize_rows_packed: args is null");
    return moe_quantize_rows(p->x, p->ldx, p->x_dtype, p->q, p->ldq, p->scales, p->T, p->H, stream);
}

}  // extern "C"
