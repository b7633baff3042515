// Append of new keys and values to a paged cache, with the position rotation
// of the keys (and of the queries) applied on the way.
//
// A token's rows are cut into units of two 16-byte chunks that turn together
// (16 of the rot_dim turned elements, with 8 angles) or that only pass (the rest
// of a row); one thread moves one unit: it loads its chunks, then the cosines and
// sines, turns in fp32, rounds once and stores.  Where rot_dim is no multiple of
// 16 the chunks that turn are of VEC = 4, 2 or 1 elements (the largest with 2 VEC
// dividing rot_dim).  One block takes one token, so the position, the slot and
// the table row are read through L1 by the token's units.
//
// The kernel is pure traffic: each input row read once, each output row written
// once (8192 tokens of 32 + 8 + 8 heads of 128: 36.6 us, 5.6 TB/s, 84 % of the
// copy rate).  Blocks in flight carry it: at 32 registers five tokens fit an SM.
// Loads ahead of the slot's arrival cost more than they gave (60 registers, 59
// us; held to 32, 39 us), and so do conversions one by one (47 us).
#include <type_traits>

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
__host__ __device__ inline int turn_units(int rot, int vec) { return rot / (2 * vec); }
__host__ __device__ inline int pass_units(int n) { return (n + 15) / 16; }

template <int VEC>
struct Vec;
template <>
struct Vec<8> {
    using type = uint4;
};
template <>
struct Vec<4> {
    using type = uint2;
};
template <>
struct Vec<2> {
    using type = uint32_t;
};
template <>
struct Vec<1> {
    using type = uint16_t;
};
// (rows of the table are 8-byte aligned: rot_dim is even)
template <int N>
__device__ __forceinline__ void load_floats(float (&f)[N], const float* p) {
    if (N == 1) {
        f[0] = __ldg(p);
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 v = __ldg(reinterpret_cast<const float2*>(p) + i);
            f[2 * i] = v.x, f[(2 * i + 1) % N] = v.y;
        }
    }
}

template <bool BF, bool PAIRS, int VEC>
__global__ void __launch_bounds__(1024) kv_append_kernel(const AppendArgs a) {
    pdl_wait();  // (and no early start of dependents: the launch contract in common.cuh)
    const int t = blockIdx.x;
    const int n_turn = turn_units(a.rot, VEC), per_head = n_turn + pass_units(a.D - a.rot);
    const int n_q = a.q ? a.q_heads * per_head : 0, n_k = a.kv_heads * per_head;
    const int per_v = pass_units(a.D), n_units = n_q + n_k + a.kv_heads * per_v;
    const int64_t slot = a.slots[t];
    const int pos = a.rot ? a.positions[t] : 0;
    const bool pos_ok = a.rot == 0 || (pos >= 0 && pos < a.max_pos);
    const bool kept = slot >= 0 && slot < a.n_slots && pos_ok;
    const int64_t page = kept ? slot / a.page_size : 0, in_page = kept ? slot % a.page_size : 0;
    const uint32_t nan2 = 0x7fff7fffu;  // NaN in both types

    for (int u = threadIdx.x; u < n_units; u += blockDim.x) {
        // where the unit's two chunks are (c1 = -1: only one)
        int head, r, c0, c1;
        const uint16_t* src;
        uint16_t* dst;
        bool turns = false, is_q = false;
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
                c0 = PAIRS ? 2 * VEC * r : VEC * r;
                c1 = PAIRS ? c0 + VEC : c0 + a.rot / 2;
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
        if (VEC < 8 && u < n_q + n_k && !turns) {
            // rot_dim, and with it what passes behind it, may lie off the 16-byte
            // grid: by words
            const int n = min(16, a.D - c0);
            uint32_t x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (2 * i < n) x[i] = *reinterpret_cast<const uint32_t*>(src + c0 + 2 * i);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (2 * i < n) *reinterpret_cast<uint32_t*>(dst + c0 + 2 * i) = pos_ok ? x[i] : nan2;
            continue;
        }
        if (VEC < 8 && turns) {
            using V = typename Vec<VEC>::type;
            union {
                V v[2];
                uint16_t e[2 * VEC];
            } x;
            x.v[0] = *reinterpret_cast<const V*>(src + c0);
            x.v[1] = *reinterpret_cast<const V*>(src + c1);
            if (pos_ok) {
                const float* row = a.cos_sin + (int64_t)pos * a.rot + VEC * r;
                float cs[VEC], sn[VEC];
                load_floats<VEC>(cs, row);
                load_floats<VEC>(sn, row + a.rot / 2);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int ia = PAIRS ? 2 * i : i, ib = PAIRS ? 2 * i + 1 : i + VEC;
                    const float p = to_f32<BF>(x.e[ia]), q = to_f32<BF>(x.e[ib]);
                    x.e[ia] = from_f32<BF>(p * cs[i] - q * sn[i]);
                    x.e[ib] = from_f32<BF>(q * cs[i] + p * sn[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2 * VEC; ++i) x.e[i] = 0x7fff;
            }
            *reinterpret_cast<V*>(dst + c0) = x.v[0];
            *reinterpret_cast<V*>(dst + c1) = x.v[1];
            continue;
        }
        uint4 x = *reinterpret_cast<const uint4*>(src + c0);
        uint4 y = c1 >= 0 ? *reinterpret_cast<const uint4*>(src + c1) : make_uint4(0, 0, 0, 0);
        if (turns && pos_ok) {
            const float* row = a.cos_sin + (int64_t)pos * a.rot + 8 * r;
            float cs[8], sn[8];
            load_floats<8>(cs, row);
            load_floats<8>(sn, row + a.rot / 2);
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
            x = y = make_uint4(nan2, nan2, nan2, nan2);
        }
        *reinterpret_cast<uint4*>(dst + c0) = x;
        if (c1 >= 0) *reinterpret_cast<uint4*>(dst + c1) = y;
    }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_kv_append_packed(const moe_kv_append_args* c, cudaStream_t stream) {
    MOE_CHECK_ARG(c, "moe_kv_append: null pointer");
    const int T = c->T, q_heads = c->q_heads, max_position = c->max_position, rot_dim = c->rot_dim;
    const int interleaved = c->interleaved;
    const void *k = c->k, *v = c->v, *q = c->q;
    void* q_out = c->q_out;
    const int32_t* positions = c->positions;
    const int64_t* slots = c->slots;
    const float* cos_sin = c->cos_sin;
    MOE_CHECK_ARG(T >= 0, "moe_kv_append: T=%d is negative", T);
    MOE_CHECK_ARG(interleaved == 0 || interleaved == 1, "moe_kv_append: interleaved=%d must be 0 or 1", interleaved);
    if (T == 0) return MOE_OK;
    const moe_kv_cache* cache = &c->cache;
    MOE_CHECK_ARG(cache->k && cache->v && k && v && slots, "moe_kv_append: null pointer");
    MOE_CHECK_ARG(known_dtype(cache->dtype), "moe_kv_append: unknown dtype %d", cache->dtype);
    MOE_CHECK_ARG(cache->num_pages > 0 && cache->page_size > 0 && cache->kv_heads > 0 && cache->head_dim > 0,
                  "moe_kv_append: cache of %lld pages of %d tokens, %d heads of %d: all must be positive",
                  (long long)cache->num_pages, cache->page_size, cache->kv_heads, cache->head_dim);
    const int D = cache->head_dim;
    MOE_CHECK_SUPPORTED(D % 8 == 0 && D <= 256, "moe_kv_append: head_dim=%d must be a multiple of 8 up to 256", D);
    MOE_CHECK_ARG(rot_dim >= 0 && rot_dim <= D, "moe_kv_append: rot_dim=%d must be in [0, %d]", rot_dim, D);
    MOE_CHECK_SUPPORTED(rot_dim % 2 == 0, "moe_kv_append: rot_dim=%d must be even", rot_dim);
    MOE_CHECK_ARG(rot_dim == 0 || (positions && cos_sin && max_position > 0),
                  "moe_kv_append: a rotation needs positions, cos_sin and max_position > 0");
    MOE_CHECK_ARG(!q || (q_out && q_heads > 0), "moe_kv_append: q needs q_out and q_heads > 0");
    // (a dimension of one element has no stride that matters)
    auto mult8 = [](int64_t stride, int64_t n) { return n <= 1 || stride % 8 == 0; };
    const int hk = cache->kv_heads;
    auto rows8 = [&](const int64_t (&stride)[2], int heads) { return mult8(stride[0], T) && mult8(stride[1], heads); };
    bool strides = rows8(c->k_stride, hk) && rows8(c->v_stride, hk);
    if (q) strides = strides && rows8(c->q_stride, q_heads) && rows8(c->q_out_stride, q_heads);
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
    a.kt = c->k_stride[0], a.kh = c->k_stride[1], a.vt = c->v_stride[0], a.vh = c->v_stride[1];
    a.qt = c->q_stride[0], a.qh = c->q_stride[1], a.ot = c->q_out_stride[0], a.oh = c->q_out_stride[1];
    for (int i = 0; i < 3; ++i) a.kc_s[i] = cache->k_stride[i], a.vc_s[i] = cache->v_stride[i];
    a.n_slots = cache->num_pages * cache->page_size;
    a.positions = positions, a.slots = slots, a.cos_sin = cos_sin;
    a.max_pos = max_position, a.rot = rot_dim, a.page_size = cache->page_size;
    a.kv_heads = cache->kv_heads, a.q_heads = q_heads, a.D = D;
    const int vec = rot_dim % 16 == 0 ? 8 : rot_dim % 8 == 0 ? 4 : rot_dim % 4 == 0 ? 2 : 1;
    const int per_head = turn_units(rot_dim, vec) + pass_units(D - rot_dim);
    const long long units = (long long)(q ? q_heads : 0) * per_head + (long long)cache->kv_heads * (per_head + pass_units(D));
    MOE_CHECK_SUPPORTED(units <= (1 << 30), "moe_kv_append: too many heads");
    const int threads = (int)(units < 1024 ? (units + 31) / 32 * 32 : 1024);
    const bool bf = cache->dtype == MOE_DT_BF16;
    auto pick = [&](auto v) {
        constexpr int V = decltype(v)::value;
        return bf ? (interleaved ? kv_append_kernel<true, true, V> : kv_append_kernel<true, false, V>)
                  : (interleaved ? kv_append_kernel<false, true, V> : kv_append_kernel<false, false, V>);
    };
    auto kern = vec == 8   ? pick(std::integral_constant<int, 8>())
                : vec == 4 ? pick(std::integral_constant<int, 4>())
                : vec == 2 ? pick(std::integral_constant<int, 2>())
                           : pick(std::integral_constant<int, 1>());
    cudaError_t e = launch_pdl(kern, dim3((unsigned)T), dim3((unsigned)threads), 0, stream, a);
    return e == cudaSuccess ? MOE_OK : cuda_status(e, "moe_kv_append: launch");
}

moe_status moe_kv_append(const moe_kv_cache* cache, const void* k, int64_t k_token_stride,
                         int64_t k_head_stride, const void* v, int64_t v_token_stride,
                         int64_t v_head_stride, const void* q, int64_t q_token_stride,
                         int64_t q_head_stride, void* q_out, int64_t q_out_token_stride,
                         int64_t q_out_head_stride, int q_heads, int T, const int32_t* positions,
                         const int64_t* slots, const float* cos_sin, int max_position, int rot_dim,
                         int interleaved, cudaStream_t stream) {
    MOE_CHECK_ARG(cache || T == 0, "moe_kv_append: null pointer");
    moe_kv_append_args c = {};
    if (cache) c.cache = *cache;
    c.k = k, c.v = v, c.q = q, c.q_out = q_out;
    c.k_stride[0] = k_token_stride, c.k_stride[1] = k_head_stride;
    c.v_stride[0] = v_token_stride, c.v_stride[1] = v_head_stride;
    c.q_stride[0] = q_token_stride, c.q_stride[1] = q_head_stride;
    c.q_out_stride[0] = q_out_token_stride, c.q_out_stride[1] = q_out_head_stride;
    c.positions = positions, c.slots = slots, c.cos_sin = cos_sin;
    c.q_heads = q_heads, c.T = T, c.max_position = max_position, c.rot_dim = rot_dim, c.interleaved = interleaved;
    return moe_kv_append_packed(&c, stream);
}

}  // extern "C"
