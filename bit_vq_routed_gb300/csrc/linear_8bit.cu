// moe_linear_8bit: the kernels of linear_kernels.cuh on inputs of 8 bits (e4m3)
// with a scale a row of x and of w.  The products of two e4m3 values are exact
// in the tensor core and summed there in fp32; both scales are applied to the
// finished sum, so they cost the main loop nothing.
#include "linear_kernels.cuh"

using namespace moe;

extern "C" {

size_t moe_linear_8bit_workspace_size(int T, int N, int K) {
    if (T < 0 || N < 0 || K <= 0) return 0;
    return 256;  // (the error word)
}

moe_status moe_linear_8bit(const uint8_t* x, int64_t ldx, const float* x_scales, const uint8_t* w, int64_t ldw,
                           const float* w_scales, const void* bias, const void* residual, int64_t ldr, void* y, int64_t ldy,
                           int T, int N, int K, int dtype, int act, void* ws, size_t ws_bytes, cudaStream_t stream) {
    MOE_CHECK_ARG(T >= 0 && N >= 0 && K > 0, "moe_linear_8bit: T=%d N=%d must not be negative, K=%d must be positive", T,
                  N, K);
    MOE_CHECK_ARG(known_dtype(dtype), "moe_linear_8bit: unknown dtype %d", dtype);
    MOE_CHECK_ARG(act >= MOE_ACT_NONE && act <= MOE_ACT_SILU, "moe_linear_8bit: unknown activation %d", act);
    if (T == 0 || N == 0) return MOE_OK;
    MOE_CHECK_ARG(x && x_scales && w && w_scales && y, "moe_linear_8bit: null pointer");
    MOE_CHECK_ARG((T == 1 || (ldx >= K && ldy >= N)) && (N == 1 || ldw >= K) && (T == 1 || !residual || ldr >= N),
                  "moe_linear_8bit: a row stride is shorter than its row");
    MOE_CHECK_SUPPORTED(K % 16 == 0, "moe_linear_8bit: K=%d must be a multiple of 16", K);
    MOE_CHECK_SUPPORTED((T == 1 || ldx % 16 == 0) && (N == 1 || ldw % 16 == 0),
                        "moe_linear_8bit: the row strides of x and w must be multiples of 16");
    MOE_CHECK_SUPPORTED(aligned16(x) && aligned16(w), "moe_linear_8bit: x and w must be 16-byte aligned");
    MOE_CHECK_SUPPORTED((((uintptr_t)bias | (uintptr_t)residual | (uintptr_t)y) & 1) == 0 &&
                            (((uintptr_t)x_scales | (uintptr_t)w_scales) & 3) == 0,
                        "moe_linear_8bit: bias, residual and y must be 2-byte aligned, the scales 4-byte");
    MOE_CHECK_SUPPORTED(K <= INT32_MAX - 256 && ((int64_t)N + 127) / 128 * (((int64_t)T + 15) / 16) * 8 <= INT32_MAX &&
                            N <= INT32_MAX - 256 && T <= INT32_MAX - 256 &&
                            ldx < ((int64_t)1 << 39) && ldw < ((int64_t)1 << 39),
                        "moe_linear_8bit: sizes or strides past what one launch covers");
    if (!ws || ws_bytes < moe_linear_8bit_workspace_size(T, N, K)) {
        set_error("moe_linear_8bit: workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0,
                  moe_linear_8bit_workspace_size(T, N, K));
        return MOE_ERR_WORKSPACE;
    }
    MOE_CHECK_SUPPORTED(((uintptr_t)ws & 15) == 0, "moe_linear_8bit: ws must be 16-byte aligned");
    LinearArgs a = {};
    a.bias = (const uint16_t*)bias, a.res = (const uint16_t*)residual, a.y = (uint16_t*)y;
    a.sx = x_scales, a.sw = w_scales;
    a.ldr = ldr, a.ldy = ldy, a.T = T, a.N = N, a.act = act;
    a.err = (int*)ws + 2;
    return dtype == MOE_DT_BF16 ? run_linear<true, true>(x, ldx, w, ldw, K, a, stream)
                                : run_linear<false, true>(x, ldx, w, ldw, K, a, stream);
}

moe_status moe_linear_8bit_packed(const moe_linear_8bit_args* p, cudaStream_t stream) {
    MOE_CHECK_ARG(p, "moe_linear_8bit_packed: args is null");
    return moe_linear_8bit(p->x, p->ldx, p->x_scales, p->w, p->ldw, p->w_scales, p->bias, p->residual, p->ldr, p->y, p->ldy,
                           p->T, p->N, p->K, p->dtype, p->act, p->ws, p->ws_bytes, stream);
}

}  // extern "C"
