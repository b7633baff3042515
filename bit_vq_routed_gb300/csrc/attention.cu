// Attention over a paged cache for a batch whose sequences share a prefix.
//
// The rows of a key head are its queries: token t, query head g of the head's
// G, as row t * G + g.  A tile is the rows of as many whole tokens as fit 128
// (the M of the tensor core), whatever sequences they belong to.  A tile sees
// the prefix, all of its rows alike, and then for each sequence that has
// tokens in it that sequence's own keys, masked for the other rows.  So the
// prefix is read once for all sequences' rows of a tile, a batch of single
// tokens fills the tile's rows, prompts are the same case with one sequence to
// a tile, and one softmax runs over prefix and suffix without a second pass.
//
// Work is cut into steps of 128 keys.  A unit of work (one key head, one tile
// or a pair of tiles) has as many steps as its prefix and suffixes need; all
// units' steps in a row are dealt out evenly, so that each CTA (one per SM)
// gets a contiguous range, whatever the lengths are: they are read on the
// device, and the host needs no plan.  A unit that falls to several CTAs
// leaves partial results that a second kernel joins, in CTA order.
//
// A CTA runs two streams of S = Q K^T -> softmax -> O += P V, each with its own
// S and O in TMEM (128 + 128 columns); while one stream's softmax runs on its
// four warps (a thread to a row), the tensor core works for the other.
//   - Pairs (prompts): the streams are two tiles, every key block is loaded
//     once for both.
//   - Single tiles (decode): both streams work for the same tile, on
//     alternate key blocks; the two results are joined from TMEM at the end.
// Warps 0-3 and 4-7: softmax of stream 0 and 1, warp 8: the order of steps and
// the keys' loads, warp 11: the values' loads, warps 9 and 10: the MMAs of stream
// 0 and 1.  Keys and values come page by page through a 4-D TMA
// map over the cache (pages past a sequence's end: an index past the cache,
// read as zeros).  P goes back to TMEM in the element type as the A operand of
// P V; V is the B operand with its N dimension innermost, as it lies in the
// cache.  O is rescaled only when a row's maximum has grown by more than 2^8,
// by the softmax warps themselves; the sum of the probabilities runs in fp32
// over the unrounded values.  In fp16 they are held times 2^7 (F16_SHIFT), so that
// what many keys far below a row's maximum add up to is not lost below the
// type's range.
//
// Bounds and times (32 query heads of 128 over 8 key heads, both kernels):
//   - decode, by the keys' and values' bytes: 8 users with 30000 tokens each 155
//     us, 6.3 TB/s or 94 % of the copy rate, with 9421 to 30000 (143044 in all) 101
//     us, 5.8 TB/s; 32 users behind 32768 shared tokens 58 us for 231 MB, of which
//     about 15 are the start, the result and the join; one user behind 1200 tokens
//     15.5 us, nothing but that;
//   - prompts, by the tensor cores: 16384 tokens 1.55 ms, 1.42 PFLOP/s; 4 prompts of
//     1024 behind 8192 tokens 368 us, 1.31 PFLOP/s.  S of a half (64 keys) takes
//     them 48 cycles an instruction, shared memory's rate, where 128 keys take 64;
//     but with S of all 128 keys at once nothing of a stream's own runs beside its
//     softmax (400 us).
#include <math.h>

#include <type_traits>

#include "elem.cuh"
#include "tc05.cuh"

namespace moe {
namespace {

constexpr int BLOCK = 128;        // keys of a step, rows of a tile
constexpr int HALF = BLOCK / 2;   // keys that S, softmax and P V take at a time
constexpr int MAX_UNITS = 2048;   // units of one launch (more tokens: more launches)
constexpr int SEQ_CACHE = 512;    // sequences whose bounds a CTA keeps in shared memory
constexpr int MAX_RING = 12;
constexpr int N_DESC = 8;
constexpr int THREADS = 384;
constexpr int TMA_WARP = 8, MMA_WARP = 9, V_WARP = 11;
constexpr int REG_SOFTMAX = 208, REG_OTHER = 88;
static_assert(8 * REG_SOFTMAX + 4 * REG_OTHER == 12 * 168, "registers of the launch");
constexpr int DATA_BYTES = 192 * 1024;  // Q tiles and the ring of K and V blocks
constexpr int MAX_CTAS = 256;

// Pairs of tiles from so many rows of a key head in all on, and so many for a
// sequence on average.  Measured, pairs against single tiles (4 query heads a key
// head, 4096 tokens of prefix): one prompt of 128 rows 23.2 against 20.5 us, of 512
// rows 28.2 and 27.5, of 1024 rows 36.8 and 38.9; 16 prompts of 64 rows 37 and 40, of
// 1024 rows 172 and 202.  256 users with 8 rows behind 16384 tokens 162 and 141, with
// 16 rows 184 and 173, 128 users with 32 rows (16 heads) 172 and 189.
constexpr int PAIR_ROWS = 1024, PAIR_SEQ_ROWS = 16;
constexpr int JOIN_THREADS = 256, JOIN_WARPS = JOIN_THREADS / 32;

// Places on the line of all units' work, that is dealt out evenly: a unit takes
// UNIT_COST places in which nothing is done (its queries' load, the look at its
// last values and its result take about that long: a 4096-token prompt 157 us at
// 2 and 148 at 3; 4 costs ragged batches more than it gives) and then one for each
// step.
constexpr int UNIT_COST = 3;

// fp16 probabilities (and with them the sums and O) are held times 2^7.  With a
// reference that lags behind by up to 2^8 that is 2^15 at most, and what the
// type rounds to zero lies more than 2^32 below the maximum: N such keys take no
// more than N 2^-32 of the largest value from the result.  (Without it N 2^-25,
// and nothing of keys 18 nats below the largest: behind a sink of small value they
// can be all there is.)
constexpr float F16_SHIFT = 7.0f;

// What a CTA did: the unit of its first step, from the unit's first step's place
// to its end (unit_begin = INT64_MAX: the CTA has no step).
struct CtaInfo {
    long long unit_begin, unit_end, total;
    int ctas, unit, head, pad;
};

struct AttnArgs {
    uint16_t* out;
    float* lse;
    const int32_t *cu_q, *prefix_pages, *page_table, *seq_lens;
    int64_t ot, oh, table_stride;
    int prefix_len, num_pages;
    int T, t_base, t_end;  // tokens of the call, and of this launch
    int B, G, q_heads, kv_heads, D, page_shift, max_pages;
    int tile_tokens, units, pair;
    float scale_log2;  // scale * log2(e)
    int* err;
    CtaInfo* info;
    float* part_m;  // [CTA][head/tail][tile][rows]
    float4* part_o; // [CTA][head/tail][tile][D/4][rows]
    int part_rows;
};

// A run of steps over consecutive blocks of one segment, told by the TMA warp
// to the others.
struct Run {
    int flags;  // bits 0, 1: streams that take part (pairs); 2: first, 3: last run of its unit here; 4: the unit is whole here
    int seq;    // -1: prefix
    int key0;   // first key of the first block in its segment
    int keys;   // keys of the segment
    int n;      // steps
    int before; // steps of the unit here before this run (single tiles: the streams take them in turn)
    int whole;  // keys, from key0 on, that all rows with the segment see
    int fresh;  // first steps of the run that may be a stream's first of the unit here
    int row0, row1;  // the unit's tokens whose segment it is
    int unit, head;
};
constexpr int RUN_FIRST = 4, RUN_LAST = 8, RUN_WHOLE = 16, RUN_END = 32;  // (END: the CTA's last run)

struct Control {
    long long cum[MAX_UNITS + 1];
    int cu[SEQ_CACHE + 1], len[SEQ_CACHE + 1];
    Run run[N_DESC];
    float xm[BLOCK], xl[BLOCK];
    uint4 bad_keys[MAX_RING];  // bits of the keys in a slot whose values are not all finite
    uint64_t ring_full[MAX_RING], ring_empty[MAX_RING], run_full[N_DESC], run_empty[N_DESC];
    uint64_t q_full, q_empty, scanned[2], s_full[2][2], p_full[2][2], pv_done[2][2], o_free[2], x_full, x_empty, drained[2];
    uint32_t tmem;
    int failed;
};

// quotient of non-negative numbers (bit by bit past 32 bits: rare, and small)
__device__ __forceinline__ long long quotient(long long x, long long y) {
    if (((x | y) >> 32) == 0) return (uint32_t)x / (uint32_t)y;
    long long q = 0, r = 0;
#pragma unroll 1
    for (int i = 62; i >= 0; --i) {
        r = 2 * r + (x >> i & 1);
        q <<= 1;
        if (r >= y) r -= y, ++q;
    }
    return q;
}
// The places of `total` dealt out to CTAs: the first `more` get each + 1, the others each.
struct Deal {
    long long each, more;
    __device__ Deal(long long total, int ctas) : each(quotient(total, ctas)), more(total - each * ctas) {}
    __device__ long long begin(int c) const { return c * each + min((long long)c, more); }
    // the CTA that has place s
    __device__ int of(long long s) const {
        const long long first = more * (each + 1);
        return (int)(s < first ? quotient(s, each + 1) : more + quotient(s - first, each));
    }
};
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float x, float y, float z) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(x), "f"(y), "f"(z));
    return d;
}
// two floats in one register pair
__device__ __forceinline__ uint64_t pair2(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ void unpair2(uint64_t v, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    return d;
}

// bits of the rows of a tile outside [r0, r1)
__device__ __forceinline__ uint4 rows_off(int r0, int r1) {
    uint32_t w[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int lo = min(max(r0 - 32 * g, 0), 32), hi = min(max(r1 - 32 * g, 0), 32);
        const uint32_t below = hi == 32 ? 0xffffffffu : (1u << hi) - 1u, under = lo == 32 ? 0xffffffffu : (1u << lo) - 1u;
        w[g] = ~(below & ~under);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// acc + 0 * x for both halves of a word
template <bool BF>
__device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t acc) {
    if (BF)
        asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0));
    else
        asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0));
    return acc;
}

// 32 bytes (the first 16 alone where !all) in as few stores as the address allows
__device__ __forceinline__ void store32(uint16_t* p, const uint32_t (&u)[8], bool all) {
    if (all && (reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                     "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                     : "memory");
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
        if (all) *reinterpret_cast<uint4*>(p + 8) = make_uint4(u[4], u[5], u[6], u[7]);
    }
}

// The sequences' token ranges and cached lengths, from shared memory where
// they fit.
struct Seqs {
    const int *cu, *len;
    int B, lo, hi, max_keys;  // tokens outside [lo, hi) do not count in this launch
    __device__ int begin(int b) const { return min(max(cu[b], lo), hi); }
    __device__ int end(int b) const { return min(max(cu[b + 1], lo), hi); }
    __device__ int keys(int b) const { return min(max(len[b], 0), max_keys); }
    // keys of b that its token t sees
    __device__ int seen(int b, int t) const { return max(0, keys(b) - (cu[b + 1] - 1 - t)); }
    // the last sequence that begins at or before t (its range may end before it)
    __device__ int of(int t) const {
        int l = 0, h = B;
        while (h - l > 1) {
            const int m = (l + h) >> 1;
            if (cu[m] <= t)
                l = m;
            else
                h = m;
        }
        return l;
    }
    // steps of b for the tokens [t0, t1)
    __device__ int steps(int b, int t0, int t1) const {
        const int x0 = max(begin(b), t0), x1 = min(end(b), t1);
        return x0 < x1 ? (seen(b, x1 - 1) + BLOCK - 1) / BLOCK : 0;
    }
};

template <bool BF, int DH>
__global__ void __launch_bounds__(THREADS, 1)
    attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const AttnArgs a) {
    extern __shared__ __align__(1024) uint8_t dyn[];
    uint8_t* data = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    Control& sm = *reinterpret_cast<Control*>(data + DATA_BYTES);
    constexpr int TILE_BYTES = DH * BLOCK * 128;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_q = a.pair ? 2 : 1;
    const int n_ring = min(MAX_RING, DATA_BYTES / TILE_BYTES - n_q);
    const uint32_t q_smem = smem_u32(data), ring = q_smem + n_q * TILE_BYTES;
    const Waits wait{a.err, &sm.failed};

    if (threadIdx.x < MAX_RING) {
        mbar_init(smem_u32(&sm.ring_full[threadIdx.x]), 1);
        mbar_init(smem_u32(&sm.ring_empty[threadIdx.x]), 2);  // (both streams' MMA warps)
    } else if (threadIdx.x < MAX_RING + N_DESC) {
        mbar_init(smem_u32(&sm.run_full[threadIdx.x - MAX_RING]), 1);
        mbar_init(smem_u32(&sm.run_empty[threadIdx.x - MAX_RING]), 11);
    } else if (threadIdx.x < MAX_RING + N_DESC + 2) {
        const int i = threadIdx.x - MAX_RING - N_DESC;
        for (int h = 0; h < 2; ++h) {
            mbar_init(smem_u32(&sm.s_full[i][h]), 1);
            mbar_init(smem_u32(&sm.p_full[i][h]), 4);
            mbar_init(smem_u32(&sm.pv_done[i][h]), 1);
        }
        mbar_init(smem_u32(&sm.o_free[i]), 4);
        mbar_init(smem_u32(&sm.drained[i]), 1);
        mbar_init(smem_u32(&sm.scanned[i]), 4);
    } else if (threadIdx.x == MAX_RING + N_DESC + 2) {
        mbar_init(smem_u32(&sm.q_full), 1);
        mbar_init(smem_u32(&sm.q_empty), 2);
        mbar_init(smem_u32(&sm.x_full), 4);
        mbar_init(smem_u32(&sm.x_empty), 4);
        sm.failed = 0;
    } else if (threadIdx.x == 32) {
        prefetch_map(&qmap);
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    if (threadIdx.x < 32) mbar_fence_init();
    static_assert(MAX_RING + N_DESC + 3 <= 32, "one warp sets the barriers up");
    if (warp == MMA_WARP) tmem_alloc(smem_u32(&sm.tmem), 512);
    tc_before();
    pdl_wait();
    // (the joining kernel, which waits for this one's end and lets nobody start before its own)
    pdl_launch_dependents();

    // ------------------------------------------------ the units' steps
    const bool cached = a.B <= SEQ_CACHE;
    if (cached)
        for (int i = threadIdx.x; i <= a.B; i += THREADS) {
            const int begin = a.cu_q[i], keys = a.seq_lens[min(i, a.B - 1)];  // (both in flight at once)
            sm.cu[i] = begin, sm.len[i] = keys;
        }
    for (int i = threadIdx.x; i <= a.units; i += THREADS) sm.cum[i] = 0;
    __syncthreads();
    tc_after();
    const uint32_t tmem = sm.tmem;
    const Seqs seqs{cached ? sm.cu : a.cu_q, cached ? sm.len : a.seq_lens, a.B, a.t_base, a.t_end,
                    a.max_pages << a.page_shift};
    const int unit_tokens = a.tile_tokens * n_q;
    // sequences of few units by a thread each, then long ones by a warp
#pragma unroll 1
    for (int is_long = 0; is_long <= (a.units > 8); ++is_long)
#pragma unroll 1
        for (int b = is_long ? warp : threadIdx.x; b < a.B; b += is_long ? THREADS / 32 : THREADS) {
            const int x0 = seqs.begin(b), x1 = seqs.end(b);
            if (x0 >= x1) continue;
            const int u0 = (x0 - a.t_base) / unit_tokens, u1 = (x1 - 1 - a.t_base) / unit_tokens;
            if ((u1 - u0 >= 8) != (is_long != 0)) continue;
#pragma unroll 1
            for (int u = u0 + (is_long ? lane : 0); u <= u1; u += is_long ? 32 : 1) {
                const int tu = a.t_base + u * unit_tokens;
                const int n = seqs.steps(b, tu, tu + unit_tokens);
                // (in the low word: a 64-bit atomic in shared memory is a loop, and
                // decode has all sequences on one unit)
                if (n) atomicAdd(reinterpret_cast<unsigned*>(&sm.cum[u + 1]), (unsigned)n);
            }
        }
    __syncthreads();
    const int prefix_steps = (a.prefix_len + BLOCK - 1) / BLOCK;
    if (warp == 0) {
        long long run = 0;
#pragma unroll 1
        for (int u0 = 0; u0 < a.units; u0 += 32) {
            const int u = u0 + lane;
            // (a unit without keys takes one step in which every key is masked)
            long long n = u < a.units ? UNIT_COST + max(prefix_steps + sm.cum[u + 1], 1ll) : 0;
#pragma unroll 1
            for (int d = 1; d < min(a.units, 32); d <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, n, d);
                if (lane >= d) n += o;
            }
            if (u < a.units) sm.cum[u + 1] = run + n;
            run += __shfl_sync(0xffffffffu, n, 31);
        }
    }
    __syncthreads();
    const long long per_head = sm.cum[a.units], total = per_head * a.kv_heads;
    // (a range of fewer than two steps would leave a stream idle)
    const int ctas = (int)min((long long)gridDim.x, (total + 1) / 2);
    const int cta = blockIdx.x;
    const Deal deal(total, ctas);
    const long long s_begin = cta < ctas ? deal.begin(cta) : 0;

    // A load of a block: this lane's box of min(page, 128) keys.  Page numbers
    // come 32 at a time, a lane each: `first` is the batch's first step of run r.
    const int box_shift = min(a.page_shift, 7), box = 1 << box_shift, n_box = BLOCK >> box_shift;
    const int my = lane & (n_box - 1), my_half = lane >> (7 - box_shift);
    const int per_batch = 32 >> (7 - box_shift);
    auto batch = [&](const Run& r, int first) {
        const int key = r.key0 + first * BLOCK + lane * box, k = key >> a.page_shift;
        if (first >= r.n || key >= r.keys) return a.num_pages;  // (past the cache: zeros)
        return __ldg(r.seq < 0 ? a.prefix_pages + k : a.page_table + r.seq * a.table_stride + k);
    };
    auto load_block = [&](const CUtensorMap* map, const Run& r, int i, int page, int slot) {
        const uint32_t full = smem_u32(&sm.ring_full[slot]);
        if (elect_one()) mbar_arrive_expect_tx(full, TILE_BYTES);
        __syncwarp();
        if (my_half < DH)
            tma_4d(ring + slot * TILE_BYTES + my_half * BLOCK * 128 + my * box * 128, map, my_half * 64,
                   (r.key0 + i * BLOCK) & ((1 << a.page_shift) - 1), r.head, page, full);
        __syncwarp();
    };

    // After a wait that gave up: this loader's copies in flight land before the
    // CTA ends.  (slot, turn): the next it would have used; it uses every other.
    auto drain_ring = [&](int slot, int turn) {
#pragma unroll 1
        for (int n = 0; n < n_ring; n += 2) {
            slot -= 2;
            if (slot < 0) slot += n_ring, --turn;
            if (turn < 0) break;
            mbar_wait_sleep_bounded(smem_u32(&sm.ring_full[slot]), turn & 1, a.err, MOE_DEVERR_WAIT_FULL);
        }
    };

    // a thread of the softmax holds a row's 128 scores: registers go from the
    // third warpgroup to the first two (8 x REG_SOFTMAX + 4 x REG_OTHER is the
    // launch's 12 x 168 a lane)
    if (warp >= TMA_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_OTHER));
        if (warp == TMA_WARP) {
            // ------------------------------------------------ order of steps, loads
            // The cursor: place in_unit of unit `unit`, of unit_n places; step j of
            // segment seq (-1: prefix), which has seg_n.  left: places of the CTA's
            // range from there on; before: steps of the unit done here.
            int head = 0, unit = 0, seq = -1, j = 0, seg_n = 0, t0 = 0, t1 = 0, before = 0;
            // (32 bits: a CTA with 2^31 steps would be at work for an hour)
            int in_unit = 0, unit_n = 0, left = cta < ctas ? (int)(deal.begin(cta + 1) - s_begin) : 0;
            bool enter = true;  // the cursor has just come to the unit
            int started = 0;    // streams that have had steps of the unit here (pairs)
            if (left > 0) {
                head = (int)quotient(s_begin, per_head);
                const long long r = s_begin - head * per_head;
                int h = a.units;
#pragma unroll 1
                while (h - unit > 1) {
                    const int m = (unit + h) >> 1;
                    if (sm.cum[m] <= r)
                        unit = m;
                    else
                        h = m;
                }
                in_unit = (int)(r - sm.cum[unit]);
                unit_n = (int)(sm.cum[unit + 1] - sm.cum[unit]);
                const int skip = min(max(UNIT_COST - in_unit, 0), left);
                in_unit += skip, left -= skip;
                if (left > 0 && in_unit == unit_n) left = 0;  // (a unit has a step: not reached)
            }
            if (lane == 0) {
                CtaInfo f;
                f.unit_begin = left > 0 ? head * per_head + sm.cum[unit] + UNIT_COST : INT64_MAX;
                f.unit_end = head * per_head + sm.cum[unit + 1];
                f.total = total;
                f.ctas = ctas;
                f.unit = unit;
                f.head = head;
                f.pad = 0;
                a.info[cta] = f;
            }
            // the next run, with the cursor moved behind its last step
            auto next_run = [&]() {
                if (in_unit == unit_n) {
                    if (++unit == a.units) unit = 0, ++head;
                    unit_n = (int)(sm.cum[unit + 1] - sm.cum[unit]);
                    in_unit = UNIT_COST, left -= UNIT_COST;
                    before = 0;
                    enter = true;
                }
                int from = seq + 1;  // where to look for the segment's sequence (none: < 0)
                int at = 0;
                if (enter) {
                    t0 = a.t_base + unit * unit_tokens;
                    t1 = min(t0 + unit_tokens, a.t_end);
                    at = in_unit - UNIT_COST;
                    seq = -1, j = at, seg_n = prefix_steps;
                    at -= prefix_steps;
                    from = at < 0 ? -1 : seqs.of(t0);
                    enter = false;
                } else if (j < seg_n) {
                    from = -1;
                } else if (seq < 0) {
                    from = seqs.of(t0);
                }
                if (from >= 0) {
                    // The first sequence from there on with more than `at` steps, the
                    // steps of those before it taken off; behind the first one a lane to a
                    // sequence (one by one, a CTA that begins at the last of 32 begins 3 us
                    // late: 16 users behind 2000 tokens 26.6 us, so 25.3; all by lanes, a
                    // ragged batch of 9 takes 21.9 us instead of 21.2).  Where
                    // there is none (a unit that sees no key) the rest of the unit goes
                    // on masked steps behind the prefix.
                    seq = from;
                    seg_n = seq < a.B ? seqs.steps(seq, t0, t1) : 0;
                    if (at >= seg_n) {
                        at -= seg_n;
                        ++seq;
#pragma unroll 1
                        for (; seq < a.B; seq += 32) {
                            const int n = seq + lane < a.B ? seqs.steps(seq + lane, t0, t1) : 0;
                            int to = n;  // steps up to this lane's sequence
                            if (at > 0) {
#pragma unroll
                                for (int d = 1; d < 32; d <<= 1) {
                                    const int o = __shfl_up_sync(0xffffffffu, to, d);
                                    if (lane >= d) to += o;
                                }
                            }
                            const uint32_t found = __ballot_sync(0xffffffffu, at < to);
                            const int l = found != 0 ? __ffs(found) - 1 : 31;
                            seg_n = __shfl_sync(0xffffffffu, n, l);
                            at -= __shfl_sync(0xffffffffu, found != 0 ? to - n : to, l);
                            if (found != 0) {
                                seq += l;
                                break;
                            }
                        }
                    }
                    j = at;
                    if (seq >= a.B) seq = -1, j = prefix_steps, seg_n = prefix_steps + unit_n - in_unit;
                }
                Run r;
                r.seq = seq, r.key0 = j * BLOCK, r.keys = seq < 0 ? a.prefix_len : seqs.keys(seq);
                r.unit = unit, r.head = head, r.before = before;
                r.row0 = seq < 0 ? 0 : max(seqs.begin(seq), t0) - t0;
                r.row1 = seq < 0 ? unit_tokens : min(seqs.end(seq), t1) - t0;
                r.whole = (seq < 0 ? r.keys : seqs.seen(seq, t0 + r.row0)) - r.key0;
                r.flags = before == 0 ? RUN_FIRST : 0;
                r.n = min(seg_n - j, left);
                r.fresh = max(0, 2 - before);
                if (a.pair) {
                    const int tm = min(t0 + a.tile_tokens, t1);
                    if (seq < 0) {
                        r.flags |= tm < t1 ? 3 : 1;
                    } else {  // up to where one of the tiles has seen its keys
                        const int n0 = seqs.steps(seq, t0, tm), n1 = seqs.steps(seq, tm, t1);
                        r.flags |= (n0 > j ? 1 : 0) | (n1 > j ? 2 : 0);
                        if (n0 > j && n1 > j) r.n = min(r.n, min(n0, n1) - j);
                    }
                    if (before == 0) started = 0;
                    r.fresh = (r.flags & 3 & ~started) != 0 ? 1 : 0;
                    started |= r.flags & 3;
                }
                left -= r.n, before += r.n, in_unit += r.n, j += r.n;
                if (in_unit == unit_n || left == 0) {
                    r.flags |= RUN_LAST;
                    if (before + UNIT_COST == unit_n) r.flags |= RUN_WHOLE;
                    if (left <= UNIT_COST) r.flags |= RUN_END;  // (no step among the places left)
                }
                return r;
            };
            int slot = 0, turn = 0, desc = 0, desc_turn = 0, q_n = 0, i = 0;
            // Page numbers a batch ahead of their use: `ids` of the batch from step
            // `i0` of run `now`, and `ids_next` of the one after it (of the run after it
            // at the run's end).
            int ids = 0, ids_next = 0, i0 = 0;
            Run now = {}, next = {};
            now.flags = left > 0 ? 0 : RUN_END;
            // Step i of run `now`.  (Starts on an empty run.)
#pragma unroll 1
            for (;;) {
                const bool last = i + 1 >= now.n;
                if (last) {
                    if (now.flags & RUN_END)
                        next.n = 0;
                    else
                        next = next_run();
                }
                if (last || i == i0) ids_next = batch(last ? next : now, last ? 0 : i0 + per_batch);
                if (now.n > 0) {
                    if (turn > 0 && !wait.warp(smem_u32(&sm.ring_empty[slot]), (turn - 1) & 1, MOE_DEVERR_WAIT_EMPTY)) break;
                    load_block(&kmap, now, i, __shfl_sync(0xffffffffu, ids, (i - i0) * n_box + my), slot);
                    slot += 2, turn += slot >= n_ring;
                    if (slot >= n_ring) slot -= n_ring;
                }
                if (!last) {
                    if (++i == i0 + per_batch) i0 = i, ids = ids_next;
                    continue;
                }
                if (now.n > 0 && (now.flags & RUN_END)) break;
                if (now.flags & RUN_END) next.flags = RUN_END, next.n = 0;  // (a CTA without steps says so)
                now = next;
                i = i0 = 0;
                ids = ids_next;
                if (desc_turn > 0 && !wait.warp(smem_u32(&sm.run_empty[desc]), (desc_turn - 1) & 1, MOE_DEVERR_WAIT_EMPTY)) break;
                if (lane == 0) {
                    sm.run[desc] = now;
                    mbar_arrive(smem_u32(&sm.run_full[desc]));
                }
                __syncwarp();
                if (++desc == N_DESC) desc = 0, ++desc_turn;
                if (now.n == 0) break;
                if (now.flags & RUN_FIRST) {
                    if (q_n > 0 && !wait.warp(smem_u32(&sm.q_empty), (q_n - 1) & 1, MOE_DEVERR_WAIT_EMPTY)) break;
                    if (elect_one()) {
                        const int tile0 = a.t_base + now.unit * unit_tokens;
                        mbar_arrive_expect_tx(smem_u32(&sm.q_full), n_q * DH * a.tile_tokens * a.G * 128);
#pragma unroll 1
                        for (int x = 0; x < n_q * DH; ++x)
                            tma_4d(q_smem + x * BLOCK * 128, &qmap, x % DH * 64, 0, now.head, tile0 + x / DH * a.tile_tokens,
                                   smem_u32(&sm.q_full));
                    }
                    __syncwarp();
                    ++q_n;
                }
            }
            // (after a wait that gave up: the copies in flight land before the CTA ends)
            if (sm.failed) {
                if (q_n > 0) mbar_wait_sleep_bounded(smem_u32(&sm.q_full), (q_n - 1) & 1, a.err, MOE_DEVERR_WAIT_FULL);
                drain_ring(slot, turn);
            }
            __syncwarp();
        } else if (warp == V_WARP) {
            // ------------------------------------------------ the values' loads
            int slot = 1, turn = 0, desc = 0, desc_turn = 0;
            bool ok = true;
#pragma unroll 1
            for (bool more = true; more && ok;) {
                if (!wait.warp(smem_u32(&sm.run_full[desc]), desc_turn & 1, MOE_DEVERR_WAIT_FULL)) break;
                const Run r = sm.run[desc];
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.run_empty[desc]));
                if (++desc == N_DESC) desc = 0, ++desc_turn;
                more = !(r.flags & RUN_END);
                int ids = batch(r, 0), ids_next = 0;
#pragma unroll 1
                for (int i = 0, i0 = 0; i < r.n; ++i) {
                    if (i == i0 + per_batch) i0 = i, ids = ids_next;
                    if (i == i0) ids_next = batch(r, i0 + per_batch);
                    ok = turn == 0 || wait.warp(smem_u32(&sm.ring_empty[slot]), (turn - 1) & 1, MOE_DEVERR_WAIT_EMPTY);
                    if (!ok) break;
                    if (lane == 0) sm.bad_keys[slot] = make_uint4(0, 0, 0, 0);
                    __syncwarp();
                    load_block(&vmap, r, i, __shfl_sync(0xffffffffu, ids, (i - i0) * n_box + my), slot);
                    slot += 2, turn += slot >= n_ring;
                    if (slot >= n_ring) slot -= n_ring;
                }
            }
            if (sm.failed) drain_ring(slot, turn);
            __syncwarp();
        } else if (warp == MMA_WARP || warp == MMA_WARP + 1) {
            // ------------------------------------------------ tensor core, a warp to a stream
            constexpr uint32_t s_idesc = umma_idesc(BF, BLOCK, HALF);
            const uint32_t o_idesc = umma_idesc(BF, BLOCK, (a.D + 15) & ~15, true);
            const int k_steps = (a.D + 15) / 16;
            const int stream = warp - MMA_WARP;
            const uint32_t s_tm = tmem + 128 * stream, o_tm = tmem + 256 + 128 * stream;
            const uint64_t qd = desc_k_inner(q_smem + (a.pair ? stream * TILE_BYTES : 0));
            int desc = 0, desc_turn = 0, q_n = 0;
            int n = 0;                            // steps of the stream so far
            int uses = 0;                         // units whose O it has held
            bool pend = false, pend_new = false;  // P V still to do, O starts there
            int v_at = 0, v_turn = 0;
            bool fresh = true;
            uint4 pend_off = make_uint4(0, 0, 0, 0);
            const int tile_first = a.pair ? stream * a.tile_tokens : 0;
            int slot = 0, turn = 0;  // of the step's K; its V is in the next slot
            bool ok = true;
#pragma unroll 1
            for (bool more = true; more && ok;) {
                if (!wait.warp(smem_u32(&sm.run_full[desc]), desc_turn & 1, MOE_DEVERR_WAIT_FULL)) break;
                const int flags = sm.run[desc].flags, steps = sm.run[desc].n, before = sm.run[desc].before;
                // this tile's rows that the segment is not for: P V leaves them alone
                const uint4 others = rows_off((sm.run[desc].row0 - tile_first) * a.G, (sm.run[desc].row1 - tile_first) * a.G);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.run_empty[desc]));
                if (++desc == N_DESC) desc = 0, ++desc_turn;
                more = !(flags & RUN_END);
                if (flags & RUN_FIRST) {
                    fresh = true;
                    if (!wait.warp(smem_u32(&sm.q_full), q_n & 1, MOE_DEVERR_WAIT_FULL)) break;
                    ++q_n;
                }
                // the run's steps, and after the unit's last one what is pending
                const int rounds = steps + (flags & RUN_LAST ? 1 : 0);
#pragma unroll 1
                for (int i = 0; i < rounds && ok; ++i) {
                    const bool step = i < steps;
                    const int v_slot = slot + 1 == n_ring ? 0 : slot + 1, vt = slot + 1 == n_ring ? turn + 1 : turn;
                    const bool mine = step && (a.pair ? flags >> stream & 1 : ((before + i) & 1) == stream);
                    if (!step) {  // (the queries are read by S alone)
                        if (elect_one()) umma_arrive(smem_u32(&sm.q_empty));
                        __syncwarp();
                    }
                    // Half by half: P V of the stream's last block (its n-th), then S of
                    // this one over the scores that this P V was the last to need.
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (pend) {
                            const uint32_t v = ring + v_at * TILE_BYTES;
                            if (h == 0) {
                                ok = wait.warp(smem_u32(&sm.ring_full[v_at]), v_turn & 1, MOE_DEVERR_WAIT_FULL);
                                if (ok && pend_new && uses++ > 0)
                                    ok = wait.warp(smem_u32(&sm.o_free[stream]), (uses - 2) & 1, MOE_DEVERR_WAIT_EMPTY);
                                if (!ok) break;
                            }
                            ok = wait.warp(smem_u32(&sm.p_full[stream][h]), (n - 1) & 1, MOE_DEVERR_WAIT_FULL);
                            if (!ok) break;
                            tc_after();
                            const uint64_t vd = desc_n_inner(v + h * HALF * 128, BLOCK * 128);
                            const uint32_t p = s_tm + HALF * h;
                            const bool add = !pend_new || h > 0;
                            if (elect_one()) {
#pragma unroll
                                for (int k = 0; k < HALF / 16; ++k)
                                    umma_ts(o_tm, p + 8 * k, vd + k * (2048 >> 4), o_idesc, pend_off, add || k > 0);
                                umma_arrive(smem_u32(&sm.pv_done[stream][h]));
                                if (h == 1) umma_arrive(smem_u32(&sm.ring_empty[v_at]));
                            }
                            __syncwarp();
                        }
                        if (mine) {
                            if (h == 0) {
                                ok = wait.warp(smem_u32(&sm.ring_full[slot]), turn & 1, MOE_DEVERR_WAIT_FULL);
                                if (!ok) break;
                            }
                            tc_after();
                            const uint64_t kd = desc_k_inner(ring + slot * TILE_BYTES + h * HALF * 128);
                            const uint32_t d = s_tm + HALF * h;
                            if (elect_one()) {
#pragma unroll
                                for (int k = 0; k < 4 * DH; ++k) {
                                    const uint32_t off = (k / 4) * (BLOCK * 128 >> 4) + 2 * (k % 4);
                                    if (k < 4 * DH - 4 || k < k_steps) umma(d, qd + off, kd + off, s_idesc, k > 0);
                                }
                                umma_arrive(smem_u32(&sm.s_full[stream][h]));
                                if (h == 1) umma_arrive(smem_u32(&sm.ring_empty[slot]));
                            }
                            __syncwarp();
                        }
                    }
                    pend = mine;
                    if (!step || !ok) break;
                    if (mine) {
                        // (O begins with a product for all rows: probabilities of zero for the others)
                        pend_off = fresh ? make_uint4(0, 0, 0, 0) : others;
                        pend_new = fresh, fresh = false;
                        v_at = v_slot, v_turn = vt;
                        ++n;
                    } else {
                        // A stream that sits a step out does not hold its values' slot
                        // meanwhile (decode: 116 us against 102 when it does).  It takes
                        // part in the release of every slot, after the slot is full: a
                        // warp that skipped phases of a barrier could take an older one
                        // of the same parity for the one it waits for.
                        ok = wait.warp(smem_u32(&sm.ring_full[slot]), turn & 1, MOE_DEVERR_WAIT_FULL) &&
                             wait.warp(smem_u32(&sm.ring_full[v_slot]), vt & 1, MOE_DEVERR_WAIT_FULL);
                        if (!ok) break;
                        if (lane == 0) {
                            mbar_arrive(smem_u32(&sm.ring_empty[slot]));
                            mbar_arrive(smem_u32(&sm.ring_empty[v_slot]));
                        }
                        __syncwarp();
                    }
                    slot += 2, turn += slot >= n_ring;
                    if (slot >= n_ring) slot -= n_ring;
                }
            }
            // Nothing of this warp is in flight when the CTA ends: neither products,
            // after a wait that gave up, nor the arrivals on barriers that nobody
            // waits for any more (one commit completes after all before it).
            __syncwarp();
            if (elect_one()) umma_arrive(smem_u32(&sm.drained[stream]));
            __syncwarp();
            mbar_wait_sleep_bounded(smem_u32(&sm.drained[stream]), 0, a.err, MOE_DEVERR_WAIT_FULL);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_SOFTMAX));
        // ------------------------------------------------ softmax
        const int stream = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_tm = tmem + lanes + 128 * stream, o_tm = tmem + lanes + 256 + 128 * stream;
        const float c = a.scale_log2;
        constexpr float shift = BF ? 0.0f : F16_SHIFT;
        int desc = 0, desc_turn = 0, n = 0, x_n = 0;
        int my_seq = -1, my_seen = 0;  // the row's sequence (-1: none) and its keys
        bool has_rows = false;         // the warp has rows at all
        float m = -INFINITY, l = 0.0f;
        int done = 0;                  // steps of the unit so far
        int token = 0;
        int steps = 0, scans = 0;      // the CTA's steps before the run; blocks scanned
        bool alive = true;
        // The values of a block, before they meet the probabilities, where a row's
        // probability of zero would have to keep out what is not finite (other
        // sequences' rows P V does not touch).  Keys past the segment's end (what
        // lies there may be anything) get values of zero.  With `scan`, so do keys
        // whose values are not all finite, and the rows that do see such a key become
        // NaN: what is wrong with one sequence stays with it, and what is wrong with
        // one token with those after it.  The stream's 128 threads take a key each.
        auto clean_values = [&](int step, int there, bool scan, int nv) {
            const int at = 2 * step + 1, slot = at % n_ring;
            if (!wait.warp(smem_u32(&sm.ring_full[slot]), at / n_ring & 1, MOE_DEVERR_WAIT_FULL)) return;
            const uint32_t v = ring + slot * TILE_BYTES + row * 128;
            bool bad = row >= there;
            if (scan) {
                uint32_t acc[4] = {0, 0, 0, 0};  // 0 * x summed up: NaN where an x is not finite
#pragma unroll 2
                for (int x = 0; x < 8 * DH; ++x) {
                    const uint4 u = lds_u128(v + x / 8 * BLOCK * 128 + ((x + lane) & 7) * 16);
                    acc[0] = times_zero<BF>(u.x, acc[0]), acc[1] = times_zero<BF>(u.y, acc[1]);
                    acc[2] = times_zero<BF>(u.z, acc[2]), acc[3] = times_zero<BF>(u.w, acc[3]);
                }
                bad = bad || ((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7fff7fffu) != 0;
                // (noted before they are cleared: of pairs, the other tile's threads
                // may find them cleared already)
                const uint32_t word = __ballot_sync(0xffffffffu, bad && row < there);
                if (word != 0) {
                    if (lane == 0) atomicOr(reinterpret_cast<uint32_t*>(&sm.bad_keys[slot]) + quarter, word);
                    __threadfence_block();
                    __syncwarp();
                }
            }
            if (bad) {
#pragma unroll 1
                for (int x = 0; x < 8 * DH; ++x)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + x / 8 * BLOCK * 128 +
                                                                                  ((x + lane) & 7) * 16),
                                 "r"(0)
                                 : "memory");
                async_smem_fence();
            }
            if (scan) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.scanned[stream]));
                wait.warp(smem_u32(&sm.scanned[stream]), scans++ & 1, MOE_DEVERR_WAIT_FULL);
                const volatile uint32_t* word = reinterpret_cast<const volatile uint32_t*>(&sm.bad_keys[slot]);
                uint32_t seen_bad = 0;
#pragma unroll 1
                for (int g = 0; g < 4; ++g)
                    seen_bad |= word[g] & (nv >= 32 * g + 32 ? 0xffffffffu : nv <= 32 * g ? 0u : (1u << (nv - 32 * g)) - 1u);
                if (seen_bad != 0) l = __int_as_float(0x7fffffff);
            }
        };
        for (bool more = true; more;) {
            if (!wait.warp(smem_u32(&sm.run_full[desc]), desc_turn & 1, MOE_DEVERR_WAIT_FULL)) break;
            const Run st = sm.run[desc];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.run_empty[desc]));
            if (++desc == N_DESC) desc = 0, ++desc_turn;
            more = !(st.flags & RUN_END);
            if (st.flags & RUN_FIRST) {
                const int t0 = a.t_base + st.unit * unit_tokens + (a.pair ? stream * a.tile_tokens : 0);
                const int in_tile = row / a.G;
                token = t0 + in_tile;
                const bool real = in_tile < a.tile_tokens && token < a.t_end;
                has_rows = __any_sync(0xffffffffu, real);
                my_seq = -1, my_seen = 0;
                if (real) {
                    const int b = seqs.of(token);
                    if (token >= seqs.begin(b) && token < seqs.end(b)) my_seq = b, my_seen = seqs.seen(b, token);
                } else {
                    token = -1;
                }
                m = -INFINITY, l = 0.0f, done = 0;
            }
            // keys of the segment, from the run's first on, that this row sees (a
            // row of no token takes what comes)
            int seen = token < 0 ? INT32_MAX - BLOCK : 0;
            if (my_seq >= 0 && (st.seq < 0 || st.seq == my_seq)) seen = (st.seq < 0 ? st.keys : my_seen) - st.key0;
            const bool has_segment = __any_sync(0xffffffffu, token >= 0 && (st.seq < 0 || st.seq == my_seq));
            const bool shared = st.row0 > 0 || st.row1 < min(unit_tokens, a.t_end - a.t_base - st.unit * unit_tokens);
            const int fresh_steps = shared ? st.fresh : 0;
            // (blocks before it need no look at their values)
            const int clean = st.seq >= 0 && fresh_steps > 0 ? 0 : max(st.whole, 0) / BLOCK;
            // the stream's steps of the run
            const int first = a.pair ? (st.flags >> stream & 1 ? 0 : st.n) : (st.before & 1) ^ stream;
            // blocks that every row sees whole, and that some row sees at all
            const int whole_blocks = __reduce_min_sync(0xffffffffu, max(seen, 0) / BLOCK);
            const int seen_blocks = __reduce_max_sync(0xffffffffu, token < 0 ? 0 : (max(seen, 0) + BLOCK - 1) / BLOCK);
            for (int i = first; i < st.n; i += a.pair ? 1 : 2) {
                const int nv = min(max(seen - i * BLOCK, 0), BLOCK);
                const bool some = i < seen_blocks, masked = i >= whole_blocks;
                if (i >= clean) {
                    // a row of the segment does not see all keys there are, or a row of
                    // another may be in the stream's first product
                    const int there = st.keys - st.key0 - i * BLOCK;
                    const bool scan = st.seq >= 0 && (st.whole - i * BLOCK < min(there, BLOCK) || i < fresh_steps);
                    // (S first: with it the slot's earlier phases are over, so that the
                    // wait for the values takes no older phase for theirs)
                    // (A wait that gives up makes the next one give up, which ends the loop.)
                    if (scan || there < BLOCK) {
                        if (wait.warp(smem_u32(&sm.s_full[stream][0]), n & 1, MOE_DEVERR_WAIT_FULL))
                            clean_values(steps + i, there, scan, nv);
                        __syncwarp();
                    }
                }
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    alive = wait.warp(smem_u32(&sm.s_full[stream][h]), n & 1, MOE_DEVERR_WAIT_FULL);
                    if (!alive) break;
                    tc_after();
                    const uint32_t at = s_tm + HALF * h;
                    if (some) {
                        uint32_t r[HALF];
                        tmem_ld32_async(at, r);
                        tmem_ld32_async(at + 32, r + 32);
                        tmem_wait_ld();
                        if (masked) {
                            // bits of the keys this row sees, 32 a word
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                const int k = nv - HALF * h - 32 * g;
                                const uint32_t bits = k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (!(bits >> i & 1)) r[32 * g + i] = 0xff800000u;
                            }
                        }
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < HALF; i += 2)
                            mx[i / 2 & 3] = max3(mx[i / 2 & 3], __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
                        const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                        // A maximum that has grown far brings O, with all that has been
                        // added to it so far, and l to the new ones.  The probabilities
                        // do not wait for that answer: they are computed for the old
                        // maxima first, and once more where it was yes.
                        bool grown = __any_sync(0xffffffffu, token >= 0 && (top - m) * c > 8.0f);
                        if (done + h == 0) m = top, grown = false;  // (there is no O yet)
                        uint64_t sum[2];
                        uint32_t p[HALF / 2];
#pragma unroll 1
                        for (;;) {
                            // (fp16: rounded down, so that a probability is never above its bound
                            // however large the product)
                            const float mc = m == -INFINITY ? shift : BF ? -(m * c) : __fmaf_rd(-m, c, shift);
                            const uint64_t c2 = pair2(c, c), mc2 = pair2(mc, mc);
                            sum[0] = sum[1] = pair2(0.0f, 0.0f);
#pragma unroll
                            for (int k = 0; k < HALF / 2; ++k) {
                                float p0, p1;
                                unpair2(fma2(pair2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])), c2, mc2), p0,
                                        p1);
                                p0 = ex2(p0), p1 = ex2(p1);
                                sum[k & 1] = add2(sum[k & 1], pair2(p0, p1));
                                p[k] = pack2<BF>(p0, p1);
                            }
                            if (!grown) break;
                            grown = false;
                            const float m2 = fmaxf(m, top);
                            const float f = m == -INFINITY ? 0.0f : ex2((m - m2) * c);
                            m = m2;
                            l *= f;
                            alive = wait.warp(smem_u32(&sm.pv_done[stream][h ^ 1]), (h ? n : n - 1) & 1, MOE_DEVERR_WAIT_FULL);
                            tc_after();
#pragma unroll 1
                            for (int i = 0; i < a.D; i += 16) {
                                uint32_t o[16];
                                tmem_ld16_async(o_tm + i, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                tmem_st16(o_tm + i, o);
                            }
                        }
                        tmem_st16(at, p);  // (over scores already read)
                        tmem_st16(at + 16, p + 16);
                        float s0, s1, s2, s3;
                        unpair2(sum[0], s0, s1);
                        unpair2(sum[1], s2, s3);
                        l += (s0 + s1) + (s2 + s3);
                        tmem_wait_st();
                    } else if (has_segment || (has_rows && done == 0)) {  // (else: rows that P V leaves alone)
                        const uint32_t zero[16] = {};
                        tmem_st16(at, zero);
                        tmem_st16(at + 16, zero);
                        tmem_wait_st();
                    }
                    tc_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[stream][h]));
                }
                if (!alive) break;
                ++n;
                ++done;
            }
            if (!alive) break;
            steps += st.n;
            if (!(st.flags & RUN_LAST)) continue;
            const int unit_steps = st.before + st.n;  // of the unit, here

            // ------------------------------------------------ the unit's result
            if (!a.pair) {
                // stream 1 hands its maximum and sum over; its O is read by stream 0
                if (stream == 1) {
                    if (done == 0) continue;
                    if (x_n > 0 && !wait.warp(smem_u32(&sm.x_empty), (x_n - 1) & 1, MOE_DEVERR_WAIT_EMPTY)) break;
                    ++x_n;
                    sm.xm[row] = m;
                    sm.xl[row] = l;
                    if (!wait.warp(smem_u32(&sm.pv_done[1][1]), (n - 1) & 1, MOE_DEVERR_WAIT_FULL)) break;
                    tc_after();
                    tc_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sm.x_full));
                    continue;
                }
            } else if (done == 0) {
                // (a tile without tokens, or none of whose rows sees a key here)
                m = -INFINITY;
            }
            const bool both = !a.pair && unit_steps > 1;
            if (done > 0 && !wait.warp(smem_u32(&sm.pv_done[stream][1]), (n - 1) & 1, MOE_DEVERR_WAIT_FULL)) break;
            // the streams' maxima and sums as one: weights of their O, log2 of the sum
            float m1 = -INFINITY, l1 = 0.0f;
            if (both) {
                if (!wait.warp(smem_u32(&sm.x_full), x_n & 1, MOE_DEVERR_WAIT_FULL)) break;
                ++x_n;
                m1 = sm.xm[row], l1 = sm.xl[row];
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.x_empty));
            }
            const float mm = fmaxf(m, m1);
            float f0 = m == -INFINITY ? 0.0f : ex2((m - mm) * c), f1 = m1 == -INFINITY ? 0.0f : ex2((m1 - mm) * c);
            if (l != l) f0 = 1.0f;  // (NaN scores have no maximum, but stay visible)
            if (l1 != l1) f1 = 1.0f;
            const float ll = l * f0 + l1 * f1;
            const float inv = ll == 0.0f ? 0.0f : __frcp_rn(ll);
            f0 = f0 == 0.0f ? 0.0f : f0 * inv;
            f1 = f1 == 0.0f ? 0.0f : f1 * inv;
            float lse2 = ll == 0.0f ? -INFINITY : ll != ll ? ll : fmaf(mm, c, __log2f(ll) - shift);
            if (my_seq < 0) f0 = f1 = 0.0f, lse2 = -INFINITY;
            tc_after();
            const bool whole = st.flags & RUN_WHOLE;
            const int q_head = st.head * a.G + row % a.G;
            // a partial result: in the CTA's first place if the unit began
            // before this CTA's range, else in its last
            const long long unit_first = (long long)st.head * sm.cum[a.units] + sm.cum[st.unit] + UNIT_COST;
            const int64_t part = ((int64_t)cta * 2 + (unit_first < s_begin ? 0 : 1)) * 2 + (a.pair ? stream : 0);
            if (has_rows) {
                uint16_t* out = a.out + (int64_t)max(token, 0) * a.ot + q_head * a.oh;
                float4* po = a.part_o + part * a.part_rows * (a.D / 4) + row;
#pragma unroll 1
                for (int i = 0; i < a.D; i += 32) {
                    uint32_t o[32], o1[32];
                    tmem_ld32_async(o_tm + i, o);
                    tmem_ld32_async(o_tm + (both ? 128 : 0) + i, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k += 16) {
                        float v[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x)  // (a weight of zero: nothing was ever put there)
                            v[x] = (f0 != 0.0f ? __uint_as_float(o[k + x]) * f0 : 0.0f) +
                                   (f1 != 0.0f ? __uint_as_float(o1[k + x]) * f1 : 0.0f);
                        if (token >= 0 && i + k < a.D) {
                            const bool all = i + k + 8 < a.D;
                            if (whole) {
                                uint32_t u[8];
#pragma unroll
                                for (int x = 0; x < 8; ++x) u[x] = pack2<BF>(v[2 * x], v[2 * x + 1]);
                                store32(out + i + k, u, all);
                            } else {
                                po[0] = make_float4(v[0], v[1], v[2], v[3]);
                                po[a.part_rows] = make_float4(v[4], v[5], v[6], v[7]);
                                if (all) {
                                    po[2 * a.part_rows] = make_float4(v[8], v[9], v[10], v[11]);
                                    po[3 * a.part_rows] = make_float4(v[12], v[13], v[14], v[15]);
                                }
                                po += 4 * a.part_rows;
                            }
                        }
                    }
                    __syncwarp();  // (the next TMEM read is the whole warp's)
                }
                if (token >= 0) {
                    if (!whole)  // (+infinity makes NaN of the joined row)
                        a.part_m[part * a.part_rows + row] = lse2 != lse2 ? INFINITY : lse2;
                    else if (a.lse)
                        a.lse[(int64_t)token * a.q_heads + q_head] = lse2 * 0.69314718055994531f;
                }
            }
            tc_before();
            __syncwarp();
            if (lane == 0) {
                if (done > 0) mbar_arrive(smem_u32(&sm.o_free[stream]));
                if (both) mbar_arrive(smem_u32(&sm.o_free[1]));
            }
        }
        __syncwarp();
    }
    tc_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_after();
        tmem_free(tmem, 512);
    }
}

// ---------------------------------------------------------------- joining
// Joins the partial results of the units that fell to several CTAs: with the
// parts' O normalised and M = log2 of their sums, out = sum 2^(M - max) O / sum
// 2^(M - max).  Every block finds the units in question from the CTAs' notes
// (a unit is one where a CTA's range begins inside it, told by the first such
// CTA).  Work goes by chunks of 32 rows x 4 outputs.  A pair of chunks to a warp
// for prompts (two to four parts), a chunk to a warp for up to FEW_PARTS; eight
// loads a thread in flight.  More parts (one long sequence over all CTAs), or few
// chunks: a block to a chunk, its warps a share of the parts each, whose results
// warp 0 adds in order.
constexpr int FEW_PARTS = 24;
constexpr int JOIN_BLOCKS = 3;  // of an SM's registers

// One more set of parts into (m, l, o)
template <int PARTS, int COLS>
__device__ __forceinline__ void join_into(float& m, float& l, float4 (&o)[COLS], const float (&pm)[PARTS],
                                          const float4 (&po)[PARTS][COLS]) {
    float top = m;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) top = fmaxf(top, pm[i]);
    if (top == -INFINITY) return;
    const float s = ex2(m - top);
    l *= s;
#pragma unroll
    for (int c = 0; c < COLS; ++c) o[c].x *= s, o[c].y *= s, o[c].z *= s, o[c].w *= s;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        const float e = ex2(pm[i] - top);
        l += e;
#pragma unroll
        for (int c = 0; c < COLS; ++c)
            o[c].x += e * po[i][c].x, o[c].y += e * po[i][c].y, o[c].z += e * po[i][c].z, o[c].w += e * po[i][c].w;
    }
    m = top;
}

template <bool BF>
__global__ void __launch_bounds__(JOIN_THREADS, JOIN_BLOCKS) attention_join_kernel(const AttnArgs a, const int n_ctas) {
    __shared__ int4 few[MAX_CTAS], many[MAX_CTAS];  // first CTA but one, parts, unit, head
    __shared__ int counts[2][JOIN_WARPS];
    __shared__ float wm[JOIN_WARPS][32], wl[JOIN_WARPS][32];
    __shared__ float4 wo[JOIN_WARPS][32];
    pdl_wait();  // (and no early start of dependents: the launch contract in common.cuh)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a thread to a CTA's note
    static_assert(MAX_CTAS <= JOIN_THREADS, "one note a thread");
    const int my = threadIdx.x;
    int4 note = make_int4(my, 0, 0, 0);
    if (my > 0 && my < n_ctas) {
        const CtaInfo f = a.info[my];
        const Deal deal(f.total, f.ctas);
        if (my < f.ctas && deal.begin(my) > f.unit_begin && deal.begin(my - 1) <= f.unit_begin)
            note = make_int4(my, deal.of(f.unit_end - 1) - my + 2, f.unit, f.head);
    }
    const int n_q = a.pair ? 2 : 1, cols = a.D / 4, groups = a.part_rows / 32;
    // (so few chunks that every one gets a block: then a block takes it from three parts on)
    const int split = __syncthreads_count(note.y > 0);
    const int few_parts = split * n_q * cols * groups <= gridDim.x ? 2 : FEW_PARTS;
    const bool is_few = note.y > 0 && note.y <= few_parts, is_many = note.y > few_parts;
    const uint32_t few_mask = __ballot_sync(0xffffffffu, is_few), many_mask = __ballot_sync(0xffffffffu, is_many);
    if (lane == 0) counts[0][warp] = __popc(few_mask), counts[1][warp] = __popc(many_mask);
    __syncthreads();
    int n_few = 0, n_many = 0, few_at = 0, many_at = 0;
#pragma unroll
    for (int i = 0; i < JOIN_WARPS; ++i) {
        if (i == warp) few_at = n_few, many_at = n_many;
        n_few += counts[0][i], n_many += counts[1][i];
    }
    const uint32_t before = (1u << lane) - 1;
    if (is_few) few[few_at + __popc(few_mask & before)] = note;
    if (is_many) many[many_at + __popc(many_mask & before)] = note;
    __syncthreads();

    // chunk: a group of 32 rows and COLS times 4 outputs.  A thread's parts are
    // first, first + step, ...
    auto join = [&](auto parts, auto columns, const int4& f, int tile, int chunk, int first, int step) {
        constexpr int PARTS = decltype(parts)::value, COLS = decltype(columns)::value;
        const int c = f.x, n = f.y, d4 = chunk % (cols / COLS) * COLS, row = chunk / (cols / COLS) * 32 + lane;
        const int token = a.t_base + f.z * a.tile_tokens * n_q + tile * a.tile_tokens + row / a.G;
        const bool real = row / a.G < a.tile_tokens && token < a.t_end;
        // part k: the unit began in the first CTA's range, before the others'
        const int64_t stride = (int64_t)4 * a.part_rows;
        const float* pm0 = a.part_m + (int64_t)(c - 1) * stride + tile * a.part_rows + row;
        const float4* po0 = a.part_o + ((int64_t)(c - 1) * stride + tile * a.part_rows) * cols + d4 * a.part_rows + row;
        float m = -INFINITY, l = 0.0f;
        float4 o[COLS];
#pragma unroll
        for (int x = 0; x < COLS; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k0 = first; k0 < n; k0 += PARTS * step) {
            float pm[PARTS];
            float4 po[PARTS][COLS];
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                const int k = k0 + i * step;
                const int64_t at = k * stride + (k == 0 ? 2 * a.part_rows : 0);
                const bool in = real && k < n;
                pm[i] = in ? pm0[at] : -INFINITY;
#pragma unroll
                for (int x = 0; x < COLS; ++x)
                    po[i][x] = in ? po0[at * cols + x * a.part_rows] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            join_into<PARTS, COLS>(m, l, o, pm, po);
        }
        if (step > 1) {
            wm[warp][lane] = m, wl[warp][lane] = l, wo[warp][lane] = o[0];
            __syncthreads();
            if (warp == 0) {
                for (int i = 1; i < JOIN_WARPS; ++i) m = fmaxf(m, wm[i][lane]);
                l = 0.0f, o[0] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (m > -INFINITY)
                    for (int i = 0; i < JOIN_WARPS; ++i) {
                        const float e = ex2(wm[i][lane] - m);
                        const float4 p = wo[i][lane];
                        l += e * wl[i][lane];
                        o[0].x += e * p.x, o[0].y += e * p.y, o[0].z += e * p.z, o[0].w += e * p.w;
                    }
            }
            __syncthreads();
        }
        if (real && (step == 1 || warp == 0)) {
            const float r = l > 0.0f ? 1.0f / l : 0.0f;
            const int q_head = f.w * a.G + row % a.G;
            uint16_t* out = a.out + (int64_t)token * a.ot + q_head * a.oh + 4 * d4;
#pragma unroll
            for (int x = 0; x < COLS; ++x) {
                uint2 u;
                u.x = pack2<BF>(o[x].x * r, o[x].y * r), u.y = pack2<BF>(o[x].z * r, o[x].w * r);
                *reinterpret_cast<uint2*>(out + 4 * x) = u;
            }
            if (a.lse && d4 == 0)
                a.lse[(int64_t)token * a.q_heads + q_head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        }
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    const std::integral_constant<int, 4> four;
    const std::integral_constant<int, 8> eight;
    const int warps = gridDim.x * JOIN_WARPS;
    if (a.pair) {
        const int chunks = cols / 2 * groups;
        for (int w = blockIdx.x * JOIN_WARPS + warp; w < n_few * 2 * chunks; w += warps)
            join(four, two, few[w / (2 * chunks)], w / chunks % 2, w % chunks, 0, 1);
    } else {
        const int chunks = cols * groups;
        for (int w = blockIdx.x * JOIN_WARPS + warp; w < n_few * chunks; w += warps)
            join(eight, one, few[w / chunks], 0, w % chunks, 0, 1);
    }
    const int chunks = cols * groups;
    for (int w = blockIdx.x; w < n_many * n_q * chunks; w += gridDim.x)
        join(four, one, many[w / (n_q * chunks)], w / chunks % n_q, w % chunks, warp, JOIN_WARPS);
}

// ---------------------------------------------------------------- host
int tile_tokens(int T, int G) { return T < BLOCK / G ? T : BLOCK / G; }
int part_rows(int T, int G) { return (tile_tokens(T, G) * G + 31) / 32 * 32; }
int main_ctas() { return num_sms() < MAX_CTAS ? num_sms() : MAX_CTAS; }

// the workspace: error word, the CTAs' notes, the parts' maxima, their outputs
constexpr size_t INFO_OFF = 256, PART_OFF = INFO_OFF + (sizeof(CtaInfo) * MAX_CTAS + 255) / 256 * 256;

template <bool BF, int DH>
moe_status run(const CUtensorMap* maps, AttnArgs a, cudaStream_t s) {
    auto kern = attention_kernel<BF, DH>;
    const size_t smem = DATA_BYTES + sizeof(Control) + 1024;
    cudaError_t e = ensure_smem_attr(kern, (int)smem);
    if (e != cudaSuccess) return cuda_status(e, "moe_prefix_attention: shared memory");
    const int ctas = main_ctas(), n_q = a.pair ? 2 : 1, T = a.T;
    const int unit_tokens = a.tile_tokens * n_q;
    const int64_t per_launch = (int64_t)unit_tokens * MAX_UNITS;
    for (int64_t base = 0; base < T; base += per_launch) {
        a.t_base = (int)base;
        a.t_end = (int)(base + per_launch < T ? base + per_launch : T);
        a.units = (a.t_end - a.t_base + unit_tokens - 1) / unit_tokens;
        e = launch_pdl(kern, dim3((unsigned)ctas), dim3(THREADS), smem, s, maps[0], maps[1], maps[2], a);
        if (e != cudaSuccess) return cuda_status(e, "moe_prefix_attention: launch");
        const int64_t work = (int64_t)a.units * a.kv_heads * n_q * (a.D / 4) * (a.part_rows / 32);
        const int grid = (int)(work < JOIN_BLOCKS * ctas ? work : JOIN_BLOCKS * ctas);
        e = launch_pdl(attention_join_kernel<BF>, dim3((unsigned)grid), dim3(JOIN_THREADS), 0, s, a, ctas);
        if (e != cudaSuccess) return cuda_status(e, "moe_prefix_attention: launch of the joining kernel");
    }
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_prefix_attention_workspace_size(int T, int q_heads, int kv_heads, int head_dim) {
    if (T < 0 || q_heads <= 0 || kv_heads <= 0 || head_dim <= 0) return 0;
    const int G = q_heads / kv_heads;
    if (T == 0 || G < 1 || G > BLOCK) return PART_OFF;
    const size_t rows = (size_t)main_ctas() * 4 * part_rows(T, G);
    return PART_OFF + rows * 4 * (1 + (size_t)head_dim);
}

moe_status moe_prefix_attention(const moe_kv_cache* cache, const void* q, int64_t q_token_stride,
                                int64_t q_head_stride, int q_heads, int T, const int32_t* cu_q, int B,
                                const int32_t* prefix_pages, int64_t prefix_len, const int32_t* page_table,
                                int64_t table_stride, int max_pages, const int32_t* seq_lens, float scale,
                                void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                                void* ws, size_t ws_bytes, cudaStream_t stream) {
    MOE_CHECK_ARG(T >= 0, "moe_prefix_attention: T=%d is negative", T);
    MOE_CHECK_ARG((B > 0 || (B == 0 && T == 0)) && prefix_len >= 0 && max_pages >= 0,
                  "moe_prefix_attention: B=%d must be positive (0 without tokens), prefix_len=%lld and max_pages=%d not negative", B,
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
    const int G = q_heads / hk;
    MOE_CHECK_SUPPORTED(G <= BLOCK, "moe_prefix_attention: %d query heads per key head, at most %d", G, BLOCK);
    MOE_CHECK_SUPPORTED(ps >= 8 && ps <= 1024 && (ps & (ps - 1)) == 0,
                        "moe_prefix_attention: page_size=%d must be a power of two from 8 to 1024", ps);
    MOE_CHECK_SUPPORTED(cache->num_pages < INT32_MAX && prefix_len <= INT32_MAX - 64 * BLOCK &&
                            (int64_t)max_pages * ps <= INT32_MAX - 64 * BLOCK && (int64_t)T * q_heads <= INT32_MAX,
                        "moe_prefix_attention: pages, lengths or rows past 2^31");
    // (a dimension of one element has no stride that matters)
    const int64_t lim = (int64_t)1 << 38;
    auto good = [&](int64_t stride, int64_t n) { return n <= 1 || (stride > 0 && stride < lim && stride % 8 == 0); };
    auto of = [](int64_t stride, int64_t n) { return n <= 1 ? (int64_t)128 : stride; };
    const bool strides = good(q_token_stride, T) && good(q_head_stride, q_heads) && good(out_token_stride, T) &&
                         good(out_head_stride, q_heads) && good(cache->k_stride[0], cache->num_pages) &&
                         good(cache->v_stride[0], cache->num_pages) && good(cache->k_stride[1], ps) &&
                         good(cache->v_stride[1], ps) && good(cache->k_stride[2], hk) && good(cache->v_stride[2], hk);
    MOE_CHECK_SUPPORTED(strides, "moe_prefix_attention: strides must be positive multiples of 8 elements");
    MOE_CHECK_SUPPORTED(aligned16(q) && aligned16(out) && aligned16(cache->k) && aligned16(cache->v),
                        "moe_prefix_attention: pointers must be 16-byte aligned");
    MOE_CHECK_SUPPORTED((((uintptr_t)cu_q | (uintptr_t)prefix_pages | (uintptr_t)page_table | (uintptr_t)seq_lens |
                          (uintptr_t)lse) & 3) == 0,
                        "moe_prefix_attention: cu_q, prefix_pages, page_table, seq_lens or lse misaligned");
    const size_t need = moe_prefix_attention_workspace_size(T, q_heads, hk, D);
    if (!ws || ws_bytes < need) {
        set_error("moe_prefix_attention: workspace of %zu bytes, %zu needed", ws ? ws_bytes : (size_t)0, need);
        return MOE_ERR_WORKSPACE;
    }
    MOE_CHECK_SUPPORTED(aligned16(ws), "moe_prefix_attention: ws must be 16-byte aligned");
    AttnArgs a = {};
    a.out = (uint16_t*)out, a.lse = lse;
    a.cu_q = cu_q, a.prefix_pages = prefix_pages, a.page_table = page_table, a.seq_lens = seq_lens;
    a.ot = out_token_stride, a.oh = out_head_stride, a.table_stride = table_stride;
    a.prefix_len = (int)prefix_len, a.num_pages = (int)cache->num_pages;
    a.T = T, a.B = B, a.G = G, a.q_heads = q_heads, a.kv_heads = hk, a.D = D;
    while (1 << a.page_shift < ps) ++a.page_shift;
    a.max_pages = max_pages, a.scale_log2 = scale * 1.4426950408889634f;
    a.tile_tokens = tile_tokens(T, G), a.part_rows = part_rows(T, G);
    a.pair = (int64_t)T * G >= PAIR_ROWS && (int64_t)T * G >= (int64_t)PAIR_SEQ_ROWS * B;
    a.err = (int*)ws + 2;
    a.info = (CtaInfo*)((char*)ws + INFO_OFF);
    a.part_o = (float4*)((char*)ws + PART_OFF);
    a.part_m = (float*)(a.part_o + (size_t)main_ctas() * 4 * a.part_rows * (D / 4));

    const bool bf = cache->dtype == MOE_DT_BF16;
    CUtensorMap maps[3];
    const int64_t qd[4] = {D, G, hk, T};
    const int64_t qs[3] = {of(q_head_stride, q_heads), of(q_head_stride * G, hk), of(q_token_stride, T)};
    const int qb[4] = {64, G, 1, a.tile_tokens};
    const int64_t cd[4] = {D, ps, hk, cache->num_pages};
    const int cb[4] = {64, ps < BLOCK ? ps : BLOCK, 1, 1};
    bool ok = make_map16(&maps[0], bf, q, 4, qd, qs, qb);
    for (int i = 0; i < 2; ++i) {
        const int64_t* st = i ? cache->v_stride : cache->k_stride;
        const int64_t cs[3] = {st[1], of(st[2], hk), of(st[0], cache->num_pages)};
        ok = ok && make_map16(&maps[1 + i], bf, i ? cache->v : cache->k, 4, cd, cs, cb);
    }
    if (!ok) {
        set_error("moe_prefix_attention: tensor map encoding failed");
        return MOE_ERR_CUDA;
    }
    if (bf) return D > 64 ? run<true, 2>(maps, a, stream) : run<true, 1>(maps, a, stream);
    return D > 64 ? run<false, 2>(maps, a, stream) : run<false, 1>(maps, a, stream);
}

}  // extern "C"
