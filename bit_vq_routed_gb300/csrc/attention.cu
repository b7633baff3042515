// Attention over a paged cache for a batch whose sequences share a prefix.
#include <math.h>

#include "elem.cuh"

namespace moe {
namespace {

struct AttnArgs {
    const uint16_t *q, *kc, *vc;
    uint16_t* out;
    float* lse;
    const int32_t *cu_q, *prefix_pages, *page_table, *seq_lens;
    int64_t qt, qh, ot, oh, kc_s[3], vc_s[3], table_stride, prefix_len, num_pages;
    int T, B, G, q_heads, kv_heads, D, page_size, max_pages;
    float scale;
};

// One warp per (token, query head): the keys one after another, lanes over D.
template <bool BF>
__global__ void __launch_bounds__(128) attention_kernel(const AttnArgs a) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)a.T * a.q_heads) return;
    const int t = (int)(row / a.q_heads), h = (int)(row % a.q_heads), hk = h / a.G;
    const bool real = t >= a.cu_q[0] && t < a.cu_q[a.B];
    int lo = 0, hi = a.B;  // the last b with cu_q[b] <= t
    while (real && hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        (a.cu_q[mid] <= t ? lo : hi) = mid;
    }
    int64_t own = 0;
    if (real) {
        const int64_t len = min((int64_t)max(a.seq_lens[lo], 0), (int64_t)a.max_pages * a.page_size);
        own = max((int64_t)0, len - (a.cu_q[lo + 1] - 1 - t));
    }
    float q[4], o[4] = {};
    for (int i = 0; i < 4; ++i)
        q[i] = lane + 32 * i < a.D ? to_f32<BF>(a.q[t * a.qt + h * a.qh + lane + 32 * i]) : 0.0f;
    float m = -INFINITY, l = 0.0f;
    const int64_t n = real ? a.prefix_len + own : 0;
    for (int64_t j = 0; j < n; ++j) {
        const bool pre = j < a.prefix_len;
        const int64_t jj = pre ? j : j - a.prefix_len;
        const int64_t page = pre ? a.prefix_pages[jj / a.page_size] : a.page_table[lo * a.table_stride + jj / a.page_size];
        const bool there = page >= 0 && page < a.num_pages;
        const uint16_t* kr = a.kc + page * a.kc_s[0] + (jj % a.page_size) * a.kc_s[1] + hk * a.kc_s[2];
        const uint16_t* vr = a.vc + page * a.vc_s[0] + (jj % a.page_size) * a.vc_s[1] + hk * a.vc_s[2];
        float s = 0.0f, v[4];
        for (int i = 0; i < 4; ++i) {
            const bool in = there && lane + 32 * i < a.D;
            s += q[i] * (in ? to_f32<BF>(kr[lane + 32 * i]) : 0.0f);
            v[i] = in ? to_f32<BF>(vr[lane + 32 * i]) : 0.0f;
        }
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale;
        const float m2 = fmaxf(m, s);
        const float c = m == m2 ? 1.0f : expf(m - m2), p = expf(s - m2);
        for (int i = 0; i < 4; ++i) o[i] = o[i] * c + p * v[i];
        l = l * c + p;
        m = m2;
    }
    for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < a.D)
            a.out[t * a.ot + h * a.oh + lane + 32 * i] = from_f32<BF>(n > 0 ? o[i] / l : 0.0f);
    if (a.lse && lane == 0) a.lse[row] = n > 0 ? m + logf(l) : -INFINITY;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_prefix_attention_workspace_size(int T, int q_heads, int kv_heads, int head_dim) {
    if (T < 0 || q_heads <= 0 || kv_heads <= 0 || head_dim <= 0) return 0;
    return 256;
}

moe_status moe_prefix_attention(const moe_kv_cache* cache, const void* q, int64_t q_token_stride,
                                int64_t q_head_stride, int q_heads, int T, const int32_t* cu_q, int B,
                                const int32_t* prefix_pages, int64_t prefix_len, const int32_t* page_table,
                                int64_t table_stride, int max_pages, const int32_t* seq_lens, float scale,
                                void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                                void* ws, size_t ws_bytes, cudaStream_t stream) {
    MOE_CHECK_ARG(T >= 0, "moe_prefix_attention: T=%d is negative", T);
    MOE_CHECK_ARG(B > 0 && prefix_len >= 0 && max_pages >= 0,
                  "moe_prefix_attention: B=%d must be positive, prefix_len=%lld and max_pages=%d not negative", B,
                  (long long)prefix_len, max_pages);
    MOE_CHECK_ARG(isfinite(scale) && scale > 0.0f, "moe_prefix_attention: scale must be positive and finite");
    if (T == 0) return MOE_OK;
    MOE_CHECK_ARG(cache && cache->k && cache->v && q && out && cu_q && seq_lens, "moe_prefix_attention: null pointer");
    MOE_CHECK_ARG(prefix_len == 0 || prefix_pages, "moe_prefix_attention: prefix_pages is null");
    MOE_CHECK_ARG(max_pages == 0 || (page_table && (B == 1 || table_stride >= max_pages)),
                  "moe_prefix_attention: page_table is null or its stride is shorter than max_pages");
    MOE_CHECK_ARG(known_dtype(cache->dtype), "moe_prefix_attention: unknown dtype %d", cache->dtype);
    MOE_CHECK_ARG(cache->num_pages > 0 && cache->page_size > 0 && cache->kv_heads > 0 && cache->head_dim > 0,
                  "moe_prefix_attention: cache of %lld pages of %d tokens, %d heads of %d: all must be positive",
                  (long long)cache->num_pages, cache->page_size, cache->kv_heads, cache->head_dim);
    const int D = cache->head_dim, hk = cache->kv_heads, ps = cache->page_size;
    MOE_CHECK_ARG(q_heads > 0 && q_heads % hk == 0,
                  "moe_prefix_attention: q_heads=%d must be a positive multiple of kv_heads=%d", q_heads, hk);
    MOE_CHECK_SUPPORTED(D % 8 == 0 && D <= 128, "moe_prefix_attention: head_dim=%d must be a multiple of 8 up to 128",
                        D);
    MOE_CHECK_SUPPORTED(q_heads / hk <= 128, "moe_prefix_attention: %d query heads per key head, at most 128",
                        q_heads / hk);
    MOE_CHECK_SUPPORTED(ps >= 8 && ps <= 1024 && (ps & (ps - 1)) == 0,
                        "moe_prefix_attention: page_size=%d must be a power of two from 8 to 1024", ps);
    MOE_CHECK_SUPPORTED(cache->num_pages <= INT32_MAX && prefix_len <= INT32_MAX &&
                            (int64_t)max_pages * ps <= INT32_MAX && (int64_t)T * q_heads <= INT32_MAX,
                        "moe_prefix_attention: pages, lengths or rows past 2^31");
    bool strides = q_token_stride % 8 == 0 && q_head_stride % 8 == 0 && out_token_stride % 8 == 0 &&
                   out_head_stride % 8 == 0;
    for (int i = 0; i < 3; ++i) strides = strides && cache->k_stride[i] % 8 == 0 && cache->v_stride[i] % 8 == 0;
    MOE_CHECK_SUPPORTED(strides, "moe_prefix_attention: strides must be multiples of 8 elements");
    MOE_CHECK_SUPPORTED(aligned16(q) && aligned16(out) && aligned16(cache->k) && aligned16(cache->v),
                        "moe_prefix_attention: pointers must be 16-byte aligned");
    const size_t need = moe_prefix_attention_workspace_size(T, q_heads, hk, D);
    if (!ws || ws_bytes < need) {
        set_error("moe_prefix_attention: workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
        return MOE_ERR_WORKSPACE;
    }
    AttnArgs a = {};
    a.q = (const uint16_t*)q, a.kc = (const uint16_t*)cache->k, a.vc = (const uint16_t*)cache->v;
    a.out = (uint16_t*)out, a.lse = lse;
    a.cu_q = cu_q, a.prefix_pages = prefix_pages, a.page_table = page_table, a.seq_lens = seq_lens;
    a.qt = q_token_stride, a.qh = q_head_stride, a.ot = out_token_stride, a.oh = out_head_stride;
    for (int i = 0; i < 3; ++i) a.kc_s[i] = cache->k_stride[i], a.vc_s[i] = cache->v_stride[i];
    a.table_stride = table_stride, a.prefix_len = prefix_len, a.num_pages = cache->num_pages;
    a.T = T, a.B = B, a.G = q_heads / hk, a.q_heads = q_heads, a.kv_heads = hk, a.D = D, a.page_size = ps;
    a.max_pages = max_pages, a.scale = scale;
    auto kern = cache->dtype == MOE_DT_BF16 ? attention_kernel<true> : attention_kernel<false>;
    const int64_t rows = (int64_t)T * q_heads;
    cudaError_t e = launch_pdl(kern, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream, a);
    return e == cudaSuccess ? MOE_OK : cuda_status(e, "moe_prefix_attention: launch");
}

}  // extern "C"
