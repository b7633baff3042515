// moe_linear: the kernels of linear_kernels.cuh on inputs of 16 bits.
#include "linear_kernels.cuh"

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
    MOE_CHECK_SUPPORTED(K <= INT32_MAX - 64 && ((int64_t)N + 127) / 128 * (((int64_t)T + 15) / 16) * 8 <= INT32_MAX &&
                            N <= INT32_MAX - 256 && T <= INT32_MAX - 256 &&
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
    a.ldr = ldr, a.ldy = ldy, a.T = T, a.N = N, a.act = act;
    a.err = (int*)ws + 2;
    return dtype == MOE_DT_BF16 ? run_linear<true, false>(x, ldx, w, ldw, K, a, stream)
                                : run_linear<false, false>(x, ldx, w, ldw, K, a, stream);
}

}  // extern "C"
