// y = act(x W^T + bias) + residual.
#include "elem.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case MOE_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
        case MOE_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
        case MOE_ACT_GELU_TANH: return 0.5f * z * (1.0f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
        case MOE_ACT_SILU: return z / (1.0f + expf(-z));
        default: return z;
    }
}

struct LinearArgs {
    const uint16_t *x, *w, *bias, *res;
    uint16_t* y;
    int64_t ldx, ldw, ldr, ldy;
    int T, N, K, act;
};

template <bool BF>
__global__ void __launch_bounds__(256) linear_kernel(const LinearArgs a) {
    __shared__ float xs[16][65], wsm[16][65];
    pdl_wait();
    const int t0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += 16) {
        for (int i = threadIdx.x; i < 64 * 16; i += 256) {
            const int r = i >> 4, c = i & 15;
            xs[c][r] = t0 + r < a.T && k0 + c < a.K ? to_f32<BF>(a.x[(int64_t)(t0 + r) * a.ldx + k0 + c]) : 0.0f;
            wsm[c][r] = n0 + r < a.N && k0 + c < a.K ? to_f32<BF>(a.w[(int64_t)(n0 + r) * a.ldw + k0 + c]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 16; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += xs[c][ty * 4 + i] * wsm[c][tx + 16 * j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + ty * 4 + i, n = n0 + tx + 16 * j;
            if (t >= a.T || n >= a.N) continue;
            float z = acc[i][j];
            if (a.bias) z += to_f32<BF>(a.bias[n]);
            z = activate(z, a.act);
            if (a.res) z += to_f32<BF>(a.res[(int64_t)t * a.ldr + n]);
            a.y[(int64_t)t * a.ldy + n] = from_f32<BF>(z);
        }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_linear_workspace_size(int T, int N, int K) {
    if (T < 0 || N < 0 || K <= 0) return 0;
    return 256;
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
    if (!ws || ws_bytes < moe_linear_workspace_size(T, N, K)) {
        set_error("moe_linear: workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0,
                  moe_linear_workspace_size(T, N, K));
        return MOE_ERR_WORKSPACE;
    }
    LinearArgs a = {(const uint16_t*)x, (const uint16_t*)w, (const uint16_t*)bias, (const uint16_t*)residual,
                    (uint16_t*)y,       ldx,                ldw,                   ldr,
                    ldy,                T,                  N,                     K,
                    act};
    auto kern = dtype == MOE_DT_BF16 ? linear_kernel<true> : linear_kernel<false>;
    cudaError_t e = launch_pdl(kern, dim3((N + 63) / 64, (T + 63) / 64), dim3(256), 0, stream, a);
    return e == cudaSuccess ? MOE_OK : cuda_status(e, "moe_linear: launch");
}

}  // extern "C"
