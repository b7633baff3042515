// Append of new keys and values to a paged cache, with the position rotation
// of the keys (and of the queries) applied on the way.
//
// A token's rows are cut into units of two 16-byte chunks that turn together
// (16 of the rot_dim turned elements, with 8 angles) or that only pass (the
// rest of a row); one thread moves one unit: it loads its chunks, then the
// position and the 8 cosines and sines, turns in fp32, rounds once and stores.
// One block takes one token, so the position, the slot and the table row are
// read through L1 by the token's units.  The kernel is pure traffic: each
// input row read once, each output row written once.
#include "elem.cuh"

namespace moe {
namespace {

struct AppendArgs {
    const uint16_t *k, *v, *q;
    uint16_t *q_out, *kc, *vc;
    int64_t kt, kh, vt, vh, qt, qh, ot, oh;  // strides: token, head
    int64_t kc_s[3], vc_s[3];
    int64_t n_slots;
    const int32_t* positions;
    const int64_t* slots;
    const float* cos_sin;
    int max_pos, rot, page_size, kv_heads, q_heads, D;
};

// units of one head of q or k (turned ones first), and of v
__host__ __device__ inline int turn_units(int rot) { return rot / 16; }
__host__ __device__ inline int pass_units(int n) { return (n / 8 + 1) / 2; }

template <bool BF, bool PAIRS>
__global__ void __launch_bounds__(1024) kv_append_kernel(const AppendArgs a) {
    pdl_wait();
    const int t = blockIdx.x;
    const int n_turn = turn_units(a.rot), per_head = n_turn + pass_units(a.D - a.rot);
    const int n_q = a.q ? a.q_heads * per_head : 0, n_k = a.kv_heads * per_head;
    const int per_v = pass_units(a.D), n_units = n_q + n_k + a.kv_heads * per_v;
    const int64_t slot = a.slots[t];
    const int pos = a.rot ? a.positions[t] : 0;
    const bool pos_ok = a.rot == 0 || (pos >= 0 && pos < a.max_pos);
    const bool kept = slot >= 0 && slot < a.n_slots && pos_ok;
    const int64_t page = kept ? slot / a.page_size : 0, in_page = kept ? slot % a.page_size : 0;

    for (int u = threadIdx.x; u < n_units; u += blockDim.x) {
        // where the unit's two chunks are (c1 = -1: only one)
        int head, r;
        const uint16_t* src;
        uint16_t* dst;
        bool turns = false, is_q = false;
        int c0, c1;
        if (u < n_q + n_k) {
            is_q = u < n_q;
            const int w = is_q ? u : u - n_q;
            head = w / per_head;
            r = w - head * per_head;
            turns = r < n_turn;
            if (is_q) {
                src = a.q + t * a.qt + head * a.qh;
                dst = a.q_out + t * a.ot + head * a.oh;
            } else {
                src = a.k + t * a.kt + head * a.kh;
                dst = a.kc + page * a.kc_s[0] + in_page * a.kc_s[1] + head * a.kc_s[2];
            }
            if (turns) {
                c0 = PAIRS ? 16 * r : 8 * r;
                c1 = PAIRS ? 16 * r + 8 : 8 * r + a.rot / 2;
            } else {
                c0 = a.rot + 16 * (r - n_turn);
                c1 = c0 + 8 < a.D ? c0 + 8 : -1;
            }
        } else {
            const int w = u - n_q - n_k;
            head = w / per_v;
            r = w - head * per_v;
            src = a.v + t * a.vt + head * a.vh;
            dst = a.vc + page * a.vc_s[0] + in_page * a.vc_s[1] + head * a.vc_s[2];
            c0 = 16 * r;
            c1 = c0 + 8 < a.D ? c0 + 8 : -1;
        }
        if (!is_q && !kept) continue;
        uint4 x = *reinterpret_cast<const uint4*>(src + c0);
        uint4 y = c1 >= 0 ? *reinterpret_cast<const uint4*>(src + c1) : make_uint4(0, 0, 0, 0);
        if (turns && pos_ok) {
            const float* row = a.cos_sin + (int64_t)pos * a.rot + 8 * r;
            float cs[8], sn[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 c2 = __ldg(reinterpret_cast<const float2*>(row) + i);
                const float2 s2 = __ldg(reinterpret_cast<const float2*>(row + a.rot / 2) + i);
                cs[2 * i] = c2.x, cs[2 * i + 1] = c2.y;
                sn[2 * i] = s2.x, sn[2 * i + 1] = s2.y;
            }
            uint32_t* xv = reinterpret_cast<uint32_t*>(&x);
            uint32_t* yv = reinterpret_cast<uint32_t*>(&y);
            if (PAIRS) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t& w = i < 4 ? xv[i] : yv[i - 4];
                    const float2 p = unpack2<BF>(w);
                    w = pack2<BF>(p.x * cs[i] - p.y * sn[i], p.y * cs[i] + p.x * sn[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 p = unpack2<BF>(xv[i]), s = unpack2<BF>(yv[i]);
                    xv[i] = pack2<BF>(p.x * cs[2 * i] - s.x * sn[2 * i], p.y * cs[2 * i + 1] - s.y * sn[2 * i + 1]);
                    yv[i] = pack2<BF>(s.x * cs[2 * i] + p.x * sn[2 * i], s.y * cs[2 * i + 1] + p.y * sn[2 * i + 1]);
                }
            }
        } else if (is_q && !pos_ok) {
            x = y = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);  // NaN in both types
        }
        *reinterpret_cast<uint4*>(dst + c0) = x;
        if (c1 >= 0) *reinterpret_cast<uint4*>(dst + c1) = y;
    }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_kv_append(const moe_kv_cache* cache, const void* k, int64_t k_token_stride,
                                    int64_t k_head_stride, const void* v, int64_t v_token_stride,
                                    int64_t v_head_stride, const void* q, int64_t q_token_stride,
                                    int64_t q_head_stride, void* q_out, int64_t q_out_token_stride,
                                    int64_t q_out_head_stride, int q_heads, int T, const int32_t* positions,
                                    const int64_t* slots, const float* cos_sin, int max_position, int rot_dim,
                                    int interleaved, cudaStream_t stream) {
    MOE_CHECK_ARG(T >= 0, "moe_kv_append: T=%d is negative", T);
    MOE_CHECK_ARG(interleaved == 0 || interleaved == 1, "moe_kv_append: interleaved=%d must be 0 or 1", interleaved);
    if (T == 0) return MOE_OK;
    MOE_CHECK_ARG(cache && cache->k && cache->v && k && v && slots, "moe_kv_append: null pointer");
    MOE_CHECK_ARG(known_dtype(cache->dtype), "moe_kv_append: unknown dtype %d", cache->dtype);
    MOE_CHECK_ARG(cache->num_pages > 0 && cache->page_size > 0 && cache->kv_heads > 0 && cache->head_dim > 0,
                  "moe_kv_append: cache of %lld pages of %d tokens, %d heads of %d: all must be positive",
                  (long long)cache->num_pages, cache->page_size, cache->kv_heads, cache->head_dim);
    const int D = cache->head_dim;
    MOE_CHECK_SUPPORTED(D % 8 == 0 && D <= 256, "moe_kv_append: head_dim=%d must be a multiple of 8 up to 256", D);
    MOE_CHECK_ARG(rot_dim >= 0 && rot_dim <= D, "moe_kv_append: rot_dim=%d must be in [0, %d]", rot_dim, D);
    MOE_CHECK_SUPPORTED(rot_dim % 16 == 0, "moe_kv_append: rot_dim=%d must be a multiple of 16", rot_dim);
    MOE_CHECK_ARG(rot_dim == 0 || (positions && cos_sin && max_position > 0),
                  "moe_kv_append: a rotation needs positions, cos_sin and max_position > 0");
    MOE_CHECK_ARG(!q || (q_out && q_heads > 0), "moe_kv_append: q needs q_out and q_heads > 0");
    // (a dimension of one element has no stride that matters)
    auto mult8 = [](int64_t stride, int64_t n) { return n <= 1 || stride % 8 == 0; };
    const int hk = cache->kv_heads;
    bool strides = mult8(k_token_stride, T) && mult8(k_head_stride, hk) && mult8(v_token_stride, T) &&
                   mult8(v_head_stride, hk);
    if (q)
        strides = strides && mult8(q_token_stride, T) && mult8(q_head_stride, q_heads) &&
                  mult8(q_out_token_stride, T) && mult8(q_out_head_stride, q_heads);
    const int64_t size[3] = {cache->num_pages, cache->page_size, hk};
    for (int i = 0; i < 3; ++i)
        strides = strides && mult8(cache->k_stride[i], size[i]) && mult8(cache->v_stride[i], size[i]);
    MOE_CHECK_SUPPORTED(strides, "moe_kv_append: strides must be multiples of 8 elements");
    MOE_CHECK_SUPPORTED(aligned16(k) && aligned16(v) && aligned16(q) && aligned16(q_out) && aligned16(cache->k) &&
                            aligned16(cache->v),
                        "moe_kv_append: pointers must be 16-byte aligned");
    MOE_CHECK_SUPPORTED(((uintptr_t)positions & 3) == 0 && ((uintptr_t)slots & 7) == 0 && ((uintptr_t)cos_sin & 7) == 0,
                        "moe_kv_append: positions, slots or cos_sin misaligned");
    AppendArgs a = {};
    a.k = (const uint16_t*)k, a.v = (const uint16_t*)v, a.q = (const uint16_t*)q, a.q_out = (uint16_t*)q_out;
    a.kc = (uint16_t*)cache->k, a.vc = (uint16_t*)cache->v;
    a.kt = k_token_stride, a.kh = k_head_stride, a.vt = v_token_stride, a.vh = v_head_stride;
    a.qt = q_token_stride, a.qh = q_head_stride, a.ot = q_out_token_stride, a.oh = q_out_head_stride;
    for (int i = 0; i < 3; ++i) a.kc_s[i] = cache->k_stride[i], a.vc_s[i] = cache->v_stride[i];
    a.n_slots = cache->num_pages * cache->page_size;
    a.positions = positions, a.slots = slots, a.cos_sin = cos_sin;
    a.max_pos = max_position, a.rot = rot_dim, a.page_size = cache->page_size;
    a.kv_heads = cache->kv_heads, a.q_heads = q_heads, a.D = D;
    const int per_head = turn_units(rot_dim) + pass_units(D - rot_dim);
    const long long units = (long long)(q ? q_heads : 0) * per_head + (long long)cache->kv_heads * (per_head + pass_units(D));
    MOE_CHECK_SUPPORTED(units <= (1 << 30), "moe_kv_append: too many heads");
    const int threads = (int)(units < 1024 ? (units + 31) / 32 * 32 : 1024);
    const bool bf = cache->dtype == MOE_DT_BF16;
    auto kern = bf ? (interleaved ? kv_append_kernel<true, true> : kv_append_kernel<true, false>)
                   : (interleaved ? kv_append_kernel<false, true> : kv_append_kernel<false, false>);
    cudaError_t e = launch_pdl(kern, dim3((unsigned)T), dim3((unsigned)threads), 0, stream, a);
    return e == cudaSuccess ? MOE_OK : cuda_status(e, "moe_kv_append: launch");
}
