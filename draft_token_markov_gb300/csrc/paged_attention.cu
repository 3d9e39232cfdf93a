// paged_attention.cu -- attention of a chunk of new tokens over a paged
// cache on tcgen05: one persistent launch for single tokens, draft chunks
// and prompt chunks alike.
//
// Rows.  The queries of a row's tokens that share a key head are stacked,
// row = token * group + head in group, so an MMA tile of 128 rows holds
// 128 / group whole tokens (one box of a TMA load), and keys and values are
// read once for all of them.  An item is (request, key head, up to two such tiles); its
// keys go by in tiles of 128:
//   S = Q K^T           128 x 128, fp32 in TMEM (both operands in shared memory)
//   m, p = 2^(S c - m c), l += sum p
//   O += P V            P rounded to the type into S's columns of TMEM, the
//                       A operand; V as it lies in the cache (MN-major B)
// with c = scale log2 e.  The maximum that p is taken against moves, and O is
// rescaled in TMEM, when a row's grows; in items of two row tiles only when it
// has grown by more than 2^8 (kLazy), the sums being exact all the same: 220 us
// against 258 us with 0 for 2048 tokens over 8192, 85 against 95 us for a mixed
// batch, for an output error of 1.38 instead of 1.13 times that of its own
// rounding.  With few rows p is kept against the true maximum, so that the
// weight that counts most is 1, without its rounding (0.5% of a decode step's
// time, 2% and 3% of drafts' and short windows'; the output's error 1.39 instead
// of 1.41 times that of its own rounding at worst).
//
// Two slots, each with its S, its O and a warpgroup, take turns on the tensor
// core: while one is in its MMAs the other is in its softmax.  An item of two
// row tiles has one in each; an item of one has its even key tiles in slot 0
// and its odd ones in slot 1, and the two are joined at its end (O of both
// slots lies in the same TMEM lanes).
//
// Work.  An item weighs one for each of its key tiles, two where it has two
// row tiles (a slot's turn then does one of them, not half of both), and a few
// more for its start and end.
// The items of the call, in order of request, key head and rows, lie end to
// end, and the whole is cut into one range of equal weight a block, whatever
// the lengths; a key tile belongs to the block that its last unit falls to.  A
// warp of every block finds its range from the lengths by itself (a scan over
// the rows).  An item cut between blocks leaves its parts, O, m and l in fp32,
// in the plan's scratch; a second launch, a programmatic dependent of the
// first, joins them in the order of the keys.  (Joined by the block that
// finished last instead, with its 128 threads' loads, a part of 72 rows took
// 3 to 5 us at the call's end.)
//
// Roles.  Warps 0-3 and 4-7: softmax and output of the two slots, a thread a
// row; warp 8 issues MMAs; warps 9 and 10 load key and value tiles by TMA, a
// page a box (a box of a page that nobody sees is read out of range, as
// zeros; at 16 keys a page one warp for both would take as long as the
// loads); warp 11 walks the block's items, leaves each for the others in a
// ring in shared memory and loads its queries.  (Nothing of an item stays in
// a register for long: shared memory takes nearly all of the L1 cache, so that
// a spilled register costs a trip to L2.)  Value rows that no row of the item
// sees can hold anything: they are zeroed in shared memory before the MMA
// (0 * NaN).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention_tc.cuh"
#include "common.cuh"
#include "f32x2.cuh"
#include "paged.h"
#include "tc.cuh"

namespace dtm {

constexpr int kPaThreads = 384;
constexpr int kRing = 4;                     // items that are known ahead
constexpr int kPaTile = 128;                 // keys of a tile, and rows
constexpr float kLazy = 8.0f;
// an item's start and end, in key tiles of one row tile.  In us, for 16 rows of
// 1-500 tokens (7 query heads a key head), 24 rows of 1-300 (8) and 32 rows of
// 5 drafts: 3 and 7 take 85.0, 81.3, 42.5; with another weight of one tile, 2:
// 87.8, 86.5, 42.7, 5: 88.7, 79.8, 44.7; with another of two, 5: 89.2, 82.2,
// 42.6, 9: 86.6, 84.0, 42.6, 11: 90.6, 81.9, 42.6; 6 for both: 84.4, 83.4, 46.3
constexpr int kWeightOne = 3, kWeightTwo = 7;
// What a unit of work may take at most (it takes 0.3 to 2 us), where a wait is
// for whole items and not for a step of one.
constexpr uint64_t kUnitNs = 20000;

template <int D>
struct PaShape {
    static constexpr int kQBytes = kPaTile * D * 2;          // one tile of queries
    static constexpr int kKvBytes = kPaTile * D * 2;         // one tile of keys or values
    static constexpr int kStages = D == 128 ? 5 : 12;
    static constexpr int kHalf = kPaTile * 128;              // 64 elements of every row
    static constexpr int kHalves = D / 64;
    // tiles, slot 1's m and l, barriers, the schedule
    static constexpr int kExchange = 2 * kQBytes + kStages * kKvBytes;
    static constexpr int kBars = kExchange + 2 * kPaTile * 4;
    static constexpr int kMisc = kBars + 8 * (2 * kStages + 13 + 2 * kRing);
    static constexpr int kSmem = kMisc + 512;
};

// ------------------------------------------------------------------- items

struct PaItem {
    int tokens, t0;            // tokens of the item (0: no more items), the first within the request
    int qs, pos0, state;       // the request's first token, its position; its table row, -1 for none
    int h;                     // key head
    int end, first, kept;      // some row sees keys [first, end) and [0, kept)
    int sink_tiles, w0;        // key tiles: [0, sink_tiles), then from w0 on
    int j0, steps;             // the block's share: key tiles from the j0-th on
    int c0, c1;                // blocks that share the item
};

struct PaReq {
    int np, qs;                // tokens that there are queries for, the first
    int pos0;                  // position of its token 0
    int state;                 // its table row, -1 for none
};

// A row's lengths as the caller gave them.
struct PaRaw {
    int64_t state;
    int qs, qe, len;
};

__device__ __forceinline__ PaRaw pa_load(const AttnArgs &a, int r) {
    return PaRaw{__ldg(a.idx + r), __ldg(a.query_start + r), __ldg(a.query_start + r + 1), __ldg(a.seq_lens + r)};
}

__device__ __forceinline__ PaReq pa_request(const AttnArgs &a, const PaRaw &w) {
    PaReq q;
    q.qs = w.qs;
    const int n = w.qe - w.qs;
    q.np = w.state < 0 || q.qs < 0 || q.qs >= a.T || n < 0 ? 0 : min(n, a.T - q.qs);
    q.pos0 = max(w.len, 0) - n;
    q.state = w.state < a.num_states ? (int)w.state : -1;
    return q;
}
__device__ __noinline__ PaReq pa_request(const AttnArgs &a, int r) { return pa_request(a, pa_load(a, r)); }

// The first key of the window of a token at `pos`.
__device__ __forceinline__ int pa_window(const AttnArgs &a, int pos) {
    return a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
}

// The m-th pair of row tiles of a request: its keys and its key tiles (none
// where nothing is seen; it counts as one unit then).
__device__ __forceinline__ void pa_span(const AttnArgs &a, const PaReq &q, int m, PaItem &it) {
    it.t0 = m * 2 * a.tile_tokens;
    it.tokens = min(q.np - it.t0, 2 * a.tile_tokens);
    const int p0 = q.pos0 + it.t0, p1 = p0 + it.tokens - 1;
    it.end = q.state < 0 ? 0 : max(0, min(p1 + 1, a.room));
    it.first = pa_window(a, p0);
    it.kept = min(min(a.sinks, it.first), it.end);
    it.w0 = it.first / kPaTile;
    const int nw = it.first < it.end ? (it.end + kPaTile - 1) / kPaTile - it.w0 : 0;
    it.sink_tiles = (it.kept + kPaTile - 1) / kPaTile;
    if (nw > 0 && it.sink_tiles > it.w0) it.sink_tiles = it.w0;
    it.steps = it.sink_tiles + nw;
}

// An item's weight: its start and end, its key tiles.
__device__ __forceinline__ int pa_tile_weight(const AttnArgs &a, const PaItem &it) {
    return it.tokens > a.tile_tokens ? 2 : 1;
}
__device__ __forceinline__ int pa_ends_weight(const AttnArgs &a, const PaItem &it) {
    return it.tokens > a.tile_tokens ? kWeightTwo : kWeightOne;
}
__device__ __forceinline__ uint32_t pa_weight(const AttnArgs &a, const PaItem &it) {
    return pa_ends_weight(a, it) + max(it.steps, 1) * pa_tile_weight(a, it);
}
// How many of its key tiles end before an offset.
__device__ __forceinline__ int pa_tile_at(const AttnArgs &a, const PaItem &it, uint32_t off) {
    const int past = (int)off - pa_ends_weight(a, it);
    return past <= 0 ? 0 : min(past / pa_tile_weight(a, it), max(it.steps, 1));
}
// The weight of an item and its key tiles.
__device__ __noinline__ uint2 pa_units(const AttnArgs &a, PaReq q, int m) {
    PaItem it;
    pa_span(a, q, m, it);
    return make_uint2(pa_weight(a, it), it.steps);
}

__device__ __forceinline__ int pa_pairs(const AttnArgs &a, const PaReq &q) {
    return (q.np + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
}

// What the block's warps share, in shared memory.
struct PaShared {
    uint32_t abort, tmem;
    PaItem ring[kRing];
};

// The call's units cut into ranges of equal length, the first `rem` one longer.
// Units are counted in 64 bits (an item's fit 32): 2^31 key tiles, which is what
// a call may have, weigh more than 2^32.
struct PaSplit {
    uint64_t base;
    uint32_t blocks, rem;

    __device__ __forceinline__ void cut(uint64_t total, uint32_t grid) {
        blocks = (uint32_t)min((uint64_t)grid, total / 2);   // a range holds a tile of either weight
        base = blocks ? total / blocks : 0;
        rem = (uint32_t)(total - base * blocks);
    }
    __device__ __forceinline__ uint64_t first(uint32_t c) const { return c * base + min(c, rem); }
    __device__ __forceinline__ int block_of(uint64_t u) const {
        const uint64_t longer = rem * (base + 1);
        return (int)(u < longer ? u / (base + 1) : rem + (u - longer) / base);
    }
};

// ----------------------------------------------------------------- helpers

// An item's part from a block, for one slot: [D / 4][128 rows] vectors of
// four columns, then m and l, so that a warp writes and reads rows side by
// side.  A block has two at most: its last item's if that goes on in the next
// block, and its first one's if that began in one before.
template <int D>
__device__ __forceinline__ float *pa_part(const AttnArgs &a, int block, bool begins, int slot) {
    return a.parts + ((int64_t)(block * 2 + (begins ? 1 : 0)) * 2 + slot) * kPaTile * (D + 2);
}

// What the joining launch has to know of the item that begins in a block and
// goes on in the next (c0 == c1: none).
struct PaJoin {
    int c0, c1;
    int token, tokens, head;   // its first token, its tokens, its first query head
};

template <bool F16>
__device__ __forceinline__ constexpr float pa_shift() { return F16 ? 7.0f : 0.0f; }

// m c + log2 l, less the weights' shift, as a natural logarithm.
template <bool F16>
__device__ __forceinline__ float pa_lse(float m, float l, float c) {
    return l == 0.0f ? -INFINITY : (m * c - pa_shift<F16>() + __log2f(l)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ kernel
//
// Bounds.  Single tokens and draft chunks read each key and value once: 64 rows
// of 2000 to 16000 keys (64 / 8 heads of 128) take 260 us for 1.66 GB, 94% of
// the copy rate.  Short calls are bound by their start and end: 8 rows of 9
// tokens over 1000 to 16000 keys (147 MB, 22 us at the copy rate) take 41 us,
// 32 rows of 9 with 1004 keys in sight (71 MB, fp16, heads of 64) 35 us with the
// tensor pipe 15% active.
// Long chunks are bound by the chain of a slot, scores - softmax - values, some
// 3000 cycles for 2 x 128 rows x 128 keys against 2048 of MMAs: 2048 tokens
// over 8192 keys (32 / 8 heads of 128) take 220 us with the tensor pipe 65%
// active (of 216 us, 199 were left without the exponentials, 209 without the
// maxima).

template <int D, bool F16>
__global__ void __launch_bounds__(kPaThreads, 1)
paged_attention_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap qmap,
                       const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using S = PaShape<D>;
    extern __shared__ __align__(1024) uint8_t base[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint8_t *q_smem = base, *kv_smem = base + 2 * S::kQBytes;
    float *exchange = reinterpret_cast<float *>(base + S::kExchange);
    PaShared &sh = *reinterpret_cast<PaShared *>(base + S::kMisc);
    static_assert(sizeof(PaShared) <= 512, "kSmem");

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t kv_full = tc::smem_u32(base + S::kBars), kv_empty = kv_full + 8 * S::kStages;
    const uint32_t q_full = kv_empty + 8 * S::kStages, q_empty = q_full + 16, s_full = q_full + 32,
                   p_full = q_full + 48, pv_done = q_full + 64,
                   merge_full = q_full + 80, merge_free = q_full + 88, leave = q_full + 96,
                   item_full = q_full + 104, item_empty = item_full + 8 * kRing;
    if (tid == 0) {
        sh.abort = 0;
        for (int i = 0; i < S::kStages; ++i) {
            tc::mbar_init(kv_full + 8 * i, 1);
            tc::mbar_init(kv_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(q_full + 8 * i, 1);
            tc::mbar_init(q_empty + 8 * i, 1);
            tc::mbar_init(s_full + 8 * i, 1);
            tc::mbar_init(p_full + 8 * i, 4);        // the slot's warps
            tc::mbar_init(pv_done + 8 * i, 1);
        }
        tc::mbar_init(merge_full, 4);                // slot 1's warps
        tc::mbar_init(merge_free, 4);                // slot 0's
        tc::mbar_init(leave, 1);
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(item_full + 8 * i, 1);
            tc::mbar_init(item_empty + 8 * i, 11);   // the warps that read it
        }
        tc::mbar_init_fence();
    }
    // the scan's first loads are on their way while the block sets up
    PaRaw raw{-1, 0, 0, 0};
    uint32_t pending = 0;
    if (warp == 11) {
        pending = __ldcg(a.status);                  // a pending status: nothing is done
        if (lane < a.rows) raw = pa_load(a, lane);
    }
    if (warp >= 9 && lane == 0) {
        const CUtensorMap *map = warp == 9 ? &kmap : warp == 10 ? &vmap : &qmap;
        asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    }
    if (warp == 8) tc::tmem_alloc(tc::smem_u32(&sh.tmem), 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;
    // a wait that some lane gives up is given up by the warp
    auto all_wait = [&](uint32_t bar, uint32_t parity, uint32_t where, uint64_t limit_ns) {
        if (__all_sync(0xffffffffu, tc::mbar_test(bar, parity))) return true;
        return (bool)__all_sync(0xffffffffu, tc::mbar_wait_or_abort(bar, parity, where, limit_ns, &sh.abort));
    };
    auto step_wait = [&](uint32_t bar, uint32_t parity, uint32_t where) {
        return all_wait(bar, parity, where, a.timeout_ns);
    };
    auto arrive = [&](uint32_t bar) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar);
    };
    // key and value tiles in the order they are used: K V K V ...
    auto stage_of = [](uint32_t at) { return at % S::kStages; };
    auto phase_of = [](uint32_t at) { return (at / S::kStages) & 1; };
    // the n-th item; its fields are read from shared memory where they are used
    auto item = [&](uint32_t n) -> const volatile PaItem & { return sh.ring[n % kRing]; };
    auto item_wait = [&](uint32_t n) { return all_wait(item_full + 8 * (n % kRing), (n / kRing) & 1, 0x500, a.walk_ns); };
    auto item_done = [&](uint32_t n) { arrive(item_empty + 8 * (n % kRing)); };

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 11) {
        // ------------------------------------------- the walk, query loads
        PaItem it;
        uint64_t total = 0, tiles = 0;               // the call's units, this lane's rows' key tiles
        // the rows' units before and with each, where key tiles will be (of
        // 32 rows and less a lane keeps its own)
        uint64_t *units_to = reinterpret_cast<uint64_t *>(kv_smem);
        const bool few = a.rows <= 32;
        PaReq q{0, 0, 0, 0};
        uint64_t own = 0, incl = 0;
#pragma unroll 1
        for (int r0 = 0; r0 < a.rows; r0 += 32) {
            if (r0 > 0) {
                raw.state = -1;
                if (r0 + lane < a.rows) raw = pa_load(a, r0 + lane);
            }
            q = pa_request(a, raw);
            const int pairs = pa_pairs(a, q);
            uint64_t x = 0, y = 0;
#pragma unroll 1
            for (int m = 0; m < pairs; ++m) {
                const uint2 units = pa_units(a, q, m);
                x += units.x;
                y += units.y;
            }
            own = incl = x * a.kv_heads;
            tiles += y * a.kv_heads;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            if (!few) units_to[r0 + lane] = total + incl;
            total += __shfl_sync(0xffffffffu, incl, 31);
        }
        __syncwarp();
        if (total >> 31) {                           // fewer key tiles than units
#pragma unroll 1
            for (int o = 16; o > 0; o >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
            if (tiles >> 31) {
                if (lane == 0 && !pending) set_status(a.status, 2u /* MARKOV_EUNSUPPORTED */, 0x600);
                total = 0;
            }
        }
        PaSplit split;
        split.cut(pending ? 0u : total, gridDim.x);
        uint64_t u = 0, u_end = 0;                   // the current item's first unit, the range's end
        uint32_t skip = 0;                           // units of the first item before the range
        int r = 0, h = 0, m = 0, pairs = 0;
        if (blockIdx.x < split.blocks) {
            const uint64_t u0 = split.first(blockIdx.x);
            u_end = split.first(blockIdx.x + 1);
            uint64_t before, units;                  // of the row that holds the first unit
            if (few) {
                r = __ffs(__ballot_sync(0xffffffffu, u0 < incl && u0 >= incl - own)) - 1;
                before = __shfl_sync(0xffffffffu, incl - own, r);
                units = __shfl_sync(0xffffffffu, own, r);
                q.np = __shfl_sync(0xffffffffu, q.np, r);
                q.qs = __shfl_sync(0xffffffffu, q.qs, r);
                q.pos0 = __shfl_sync(0xffffffffu, q.pos0, r);
                q.state = __shfl_sync(0xffffffffu, q.state, r);
            } else {
#pragma unroll 1
                for (int r0 = 0;; r0 += 32) {
                    const int x = r0 + lane;
                    const bool here = x < a.rows && u0 < units_to[x] && (x == 0 || u0 >= units_to[x - 1]);
                    const uint32_t found = __ballot_sync(0xffffffffu, here);
                    if (found) { r = r0 + __ffs(found) - 1; break; }
                }
                before = r ? units_to[r - 1] : 0;
                units = units_to[r] - before;
                q = pa_request(a, r);
            }
            pairs = pa_pairs(a, q);
            const uint64_t head = units / a.kv_heads;
            h = (int)((u0 - before) / head);
            u = before + h * head;
#pragma unroll 1
            for (;; ++m) {
                const uint32_t units = pa_units(a, q, m).x;
                if (u0 - u < units) break;
                u += units;
            }
            skip = (uint32_t)(u0 - u);
        }
        tc::fence_proxy_async_smem();                // units_to is read; TMA writes come
        uint32_t q_phase = 0;                        // a bit a slot
        PaJoin join{0, 0, 0, 0, 0};
        int q_token = 0, q_head = 0, q_tiles = 0;    // the queries of the item published last
        bool ok = true;
        uint64_t limit_ns = a.timeout_ns;            // with the time that the items published so far may take
        for (uint32_t n = 0; ok; ++n) {
            int token = q_token, head = q_head, tiles = q_tiles;
            ok = all_wait(item_empty + 8 * (n % kRing), (n / kRing & 1) ^ 1, 0x510, limit_ns);
            if (!ok) break;
            q_tiles = 0;
            bool more = false;
            while (!more && u < u_end) {
                pa_span(a, q, m, it);
                const uint32_t units = pa_weight(a, it), weight = pa_tile_weight(a, it);
                const int all = max(it.steps, 1);
                it.j0 = pa_tile_at(a, it, skip);
                const int j1 = u_end - u < units ? pa_tile_at(a, it, (uint32_t)(u_end - u)) : all;
                more = it.j0 < j1;                   // not a tile of it: another block's
                if (more) {
                    limit_ns += (uint64_t)(j1 - it.j0) * weight * kUnitNs;
                    it.qs = q.qs;
                    it.pos0 = q.pos0;
                    it.state = q.state;
                    it.h = h;
                    it.c0 = it.c1 = blockIdx.x;
                    if (it.j0 > 0 || j1 < all) {
                        it.c0 = split.block_of(u + pa_ends_weight(a, it) + weight - 1);
                        it.c1 = split.block_of(u + units - 1);
                    }
                    it.steps = min(j1, it.steps) - it.j0;    // 0 where nothing is seen
                    if (it.steps > 0) {
                        q_token = q.qs + it.t0;
                        q_head = h * a.group;
                        q_tiles = weight;
                    }
                }
                u += units;
                skip = 0;
                if (++m == pairs) {
                    m = 0;
                    if (++h == a.kv_heads) {
                        h = 0;
                        if (u < u_end) {
                            do {
                                q = pa_request(a, ++r);
                            } while (q.np <= 0);
                            pairs = pa_pairs(a, q);
                        }
                    }
                }
            }
            if (!more) it.tokens = 0;
            if (more && it.c0 != it.c1 && it.c0 == (int)blockIdx.x)
                join = PaJoin{it.c0, it.c1, it.qs + it.t0, it.tokens, it.h * a.group};
            if (lane == 0) sh.ring[n % kRing] = it;
            arrive(item_full + 8 * (n % kRing));
            // the queries of the item before (of the first at once), so that
            // the loads of keys know of an item ahead
            if (n == 0) {
                token = q_token;
                head = q_head;
                tiles = q_tiles;
                q_tiles = 0;
            }
#pragma unroll 1
            for (int s = 0; s < tiles; ++s, token += a.tile_tokens) {
                ok = all_wait(q_empty + 8 * s, (q_phase >> s & 1) ^ 1, 0x300 + s, limit_ns);
                if (!ok) break;
                q_phase ^= 1u << s;
                if (lane == 0) {
                    tc::mbar_expect_tx(q_full + 8 * s, a.tile_tokens * a.group * D * 2);
#pragma unroll 1
                    for (int half = 0; half < S::kHalves; ++half)
                        tma_load_3d(tc::smem_u32(q_smem) + s * S::kQBytes + half * S::kHalf, &qmap, half * 64, head,
                                    token, q_full + 8 * s);
                }
                __syncwarp();
            }
            if (!more) break;
        }
        if (lane == 0) reinterpret_cast<PaJoin *>(a.joins)[blockIdx.x] = join;
        if (lane == 0 && sh.abort) {
            // gave up: no load may be in flight when the block leaves
            const uint64_t until = tc::now_ns() + a.timeout_ns;
            for (int s = 0; s < 2; ++s)
                while (!tc::mbar_test(q_full + 8 * s, (q_phase >> s & 1) ^ 1) && tc::now_ns() < until) {}
        }
    } else if (warp == 9 || warp == 10) {
        // ------------------------------------------------ key / value loads
        const bool values = warp == 10;
        const CUtensorMap *map = values ? &vmap : &kmap;
        uint32_t filled = 0, fill_phase = 0;         // stages it filled, and their phases
        const int page = 1 << a.page_shift;
        const int box = min(page, kPaTile), boxes = kPaTile / box;     // boxes of a tile
        uint32_t at = values ? 1 : 0;
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            ok = item_wait(n);
            const volatile PaItem &it = item(n);
            if (!ok || it.tokens == 0) break;
            const int32_t *table = a.table + (int64_t)max(it.state, 0) * a.table_s0;
            const int j0 = it.j0, j1 = j0 + it.steps, sinks = it.sink_tiles, w0 = it.w0;
            const int end = it.end, first = it.first, kept = it.kept, h = it.h;
            item_done(n);
            auto page_of = [&](int j) {
                const int key = (j < sinks ? j : w0 + j - sinks) * kPaTile + lane * box;
                return lane < boxes && key < end && (key + box > first || key < kept)
                           ? __ldg(table + (key >> a.page_shift)) : -1;
            };
            int next = j0 < j1 ? page_of(j0) : -1;
            for (int j = j0; j < j1; ++j, at += 2) {
                const int pid = next;
                if (j + 1 < j1) next = page_of(j + 1);
                const int slot0 = (j < sinks ? j : w0 + j - sinks) * kPaTile & (page - 1);
                const uint32_t stage = stage_of(at), phase = phase_of(at), full = kv_full + 8 * stage;
                ok = step_wait(kv_empty + 8 * stage, phase ^ 1, 0x100 + stage);
                if (!ok) break;
                if (lane == 0) tc::mbar_expect_tx(full, S::kKvBytes);
                __syncwarp();
                // the whole warp goes through the boxes, an elected lane issues
                uint32_t dst = tc::smem_u32(kv_smem + stage * S::kKvBytes);
#pragma unroll 2
                for (int b = 0; b < boxes; ++b, dst += box * 128) {
                    const int id = __shfl_sync(0xffffffffu, pid, b);
#pragma unroll
                    for (int half = 0; half < S::kHalves; ++half)
                        tma_load_4d_elect(dst + half * S::kHalf, map, half * 64, slot0, h, id, full);
                }
                filled |= 1u << stage;
                fill_phase = (fill_phase & ~(1u << stage)) | (phase << stage);
            }
        }
        if (lane == 0 && sh.abort) {
            // gave up: no load may be in flight when the block leaves
            const uint64_t until = tc::now_ns() + a.timeout_ns;
            for (int i = 0; i < S::kStages; ++i)
                if (filled >> i & 1)
                    while (!tc::mbar_test(kv_full + 8 * i, fill_phase >> i & 1) && tc::now_ns() < until) {}
        }
    } else if (warp == 8) {
        // ---------------------------------------------------- MMA issue
        // the whole warp, so that control flow and descriptors stay uniform;
        // an elected lane issues
        uint32_t q_phase = 0, p_phase = 0;           // a bit a slot
        bool ok = true;
        constexpr uint32_t kIdescS = pa_idesc<F16>(kPaTile, false), kIdescO = pa_idesc<F16>(D, true);
        constexpr uint32_t kStep = S::kKvBytes / 16;
        const uint64_t q_desc = tc::sw128_desc(tc::smem_u32(q_smem)), k_desc = tc::sw128_desc(tc::smem_u32(kv_smem)),
                       v_desc = sw128_mn_desc(tc::smem_u32(kv_smem), S::kHalf);
        const uint32_t t_o = tmem + 2 * kPaTile;
        // a place in the ring of key and value tiles
        struct Place {
            uint32_t stage, phase;
            __device__ __forceinline__ Place after(int n) const {
                Place p{stage + n, phase};
                if (p.stage >= S::kStages) { p.stage -= S::kStages; p.phase ^= 1; }
                return p;
            }
        };
        auto loaded = [&](Place k) { return step_wait(kv_full + 8 * k.stage, k.phase, 0x200); };
        auto scores = [&](int slot, int q_tile, Place k) {
            mma_scores<D>(tmem + slot * kPaTile, q_desc + q_tile * (S::kQBytes / 16), k_desc + k.stage * kStep, kIdescS);
            tc::commit_elect(s_full + 8 * slot);
        };
        // O += P V, once the slot's P is there
        auto values = [&](int slot, Place v, bool accumulate) {
            if (!step_wait(p_full + 8 * slot, p_phase >> slot & 1, 0x220 + slot)) return false;
            p_phase ^= 1u << slot;
            tc::fence_after_sync();
            mma_values(t_o + slot * D, tmem + slot * kPaTile, v_desc + v.stage * kStep, kIdescO, accumulate);
            return true;
        };
        auto release = [&](Place k) { tc::commit_elect(kv_empty + 8 * k.stage); };
        auto queries = [&](int tile) {
            const bool r = step_wait(q_full + 8 * tile, q_phase >> tile & 1, 0x210 + tile);
            q_phase ^= 1u << tile;
            return r;
        };
        Place k{0, 0};                               // the next key tile for scores
        for (uint32_t n = 0; ok; ++n) {
            ok = item_wait(n);
            const int tokens = item(n).tokens, steps = item(n).steps;
            if (!ok || tokens == 0) break;
            item_done(n);
            if (steps <= 0) continue;                // nothing seen: the output is written without MMAs
            // Either way a slot's turn is: its P comes, O += P V, the next
            // scores over P's place (MMAs run in the order of their issue).
            Place v = k.after(1);
            if (tokens > a.tile_tokens) {
                // two row tiles, a slot each, every key tile for both
                ok = queries(0) && loaded(k);
                if (!ok) break;
                tc::fence_after_sync();
                scores(0, 0, k);
                ok = queries(1);
                if (!ok) break;
                tc::fence_after_sync();
                scores(1, 1, k);
                release(k);
                k = k.after(2);
#pragma unroll 1
                for (int j = 1; j < steps; ++j) {
                    ok = loaded(v) && values(0, v, j > 1) && loaded(k);
                    if (!ok) break;
                    scores(0, 0, k);
                    ok = values(1, v, j > 1);
                    if (!ok) break;
                    release(v);
                    scores(1, 1, k);
                    release(k);
                    v = v.after(2);
                    k = k.after(2);
                }
                if (!ok) break;
                tc::commit_elect(q_empty);
                tc::commit_elect(q_empty + 8);
                ok = loaded(v);
#pragma unroll 1
                for (int s = 0; ok && s < 2; ++s) {
                    ok = values(s, v, steps > 1);
                    if (ok) tc::commit_elect(pv_done + 8 * s);
                }
                release(v);
            } else {
                // one: the key tiles in turn
                ok = queries(0);
#pragma unroll 1
                for (int j = 0; ok && j < steps && j < 2; ++j) {
                    ok = loaded(k);
                    if (!ok) break;
                    tc::fence_after_sync();
                    scores(j, 0, k);
                    release(k);
                    k = k.after(2);
                }
                if (steps <= 2) tc::commit_elect(q_empty);
#pragma unroll 1
                for (int j = 0; ok && j < steps; ++j) {
                    ok = loaded(v) && values(j & 1, v, j > 1);
                    if (!ok) break;
                    release(v);                      // before the wait for keys: the loads may need the place
                    v = v.after(2);
                    if (j + 2 < steps) {
                        ok = loaded(k);
                        if (!ok) break;
                        scores(j & 1, 0, k);
                        release(k);
                        if (j + 3 == steps) tc::commit_elect(q_empty);
                        k = k.after(2);
                    } else {
                        tc::commit_elect(pv_done + 8 * (j & 1));
                    }
                }
            }
        }
        if (sh.abort) {
            // gave up: no MMA may be in flight when the block leaves
            tc::commit_elect(leave);
            tc::mbar_wait_for(leave, 0, a.timeout_ns);
        }
    } else {
        // -------------------------------------------- softmax and output
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int slot = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;    // TMEM lane of the warp
        const uint32_t t_s = tmem + slot * kPaTile + lanes, t_o = tmem + 2 * kPaTile + slot * D + lanes;
        const float c = a.scale2;
        constexpr float kShift = pa_shift<F16>();     // fp16 weights: up to 2^15, small ones stay normal
        uint32_t s_phase = 0, pv_phase = 0, merge_phase = 0, at = 0;
        bool ok = true, owed = false;                 // owed: slot 0 may not have read what slot 1 left
        for (uint32_t n = 0; ok; ++n) {
            ok = item_wait(n);
            const volatile PaItem &it = item(n);
            if (!ok || it.tokens == 0) break;
            const bool two = it.tokens > a.tile_tokens;
            const int t0 = it.t0 + (two ? slot * a.tile_tokens : 0);
            const int tokens = min(it.tokens + it.t0 - t0, a.tile_tokens), rows = tokens * a.group;
            const int steps = it.steps, ahead = two ? 1 : 2;
            // rows past the tokens take the last one's position: theirs may not fit
            const int tok = row * a.group_inv >> 16, pos = it.pos0 + t0 + min(tok, tokens - 1);
            const bool busy = (warp & 3) * 32 < rows;
            // a tile is seen whole by the warp's rows when its last key is
            // not past the first one's and its first within the last one's window
            const int whole_end = min(__shfl_sync(0xffffffffu, pos, 0) + 1, a.room);
            const int whole_first = pa_window(a, __shfl_sync(0xffffffffu, pos, 31));
            const int end = it.end, first = it.first, kept = it.kept;
            const float lazy = two ? kLazy : 0.0f;
            float m = -INFINITY, l = 0.0f;
            bool any = false;                         // a key tile of this slot's went by
            for (int i = two ? 0 : slot; i < steps; i += ahead) {
                int key0 = it.j0 + i;
                {
                    const int sink_tiles = it.sink_tiles;
                    key0 = (key0 < sink_tiles ? key0 : it.w0 + key0 - sink_tiles) * kPaTile;
                }
                ok = step_wait(s_full + 8 * slot, s_phase, 0x400 + slot);
                if (!ok) break;
                s_phase ^= 1;
                tc::fence_after_sync();
                // value rows that nobody sees: zeros
                if (key0 + kPaTile > end || (key0 < first && key0 + kPaTile > kept)) {
                    const uint32_t v = at + 2 * i + 1;
                    ok = step_wait(kv_full + 8 * stage_of(v), phase_of(v), 0x420 + slot);
                    if (!ok) break;
                    const int key = key0 + row;
                    if (key >= end || (key < first && key >= kept)) {
                        const uint32_t dst = tc::smem_u32(kv_smem) + stage_of(v) * S::kKvBytes + row * 128;
#pragma unroll 2
                        for (int k = 0; k < 8 * S::kHalves; ++k)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             dst + (k >> 3) * S::kHalf + 16 * (k & 7)),
                                         "r"(0)
                                         : "memory");
                    }
                    tc::fence_proxy_async_smem();
                }
                if (owed) {                           // before this slot's O is written again
                    ok = step_wait(merge_free, merge_phase, 0x460);
                    if (!ok) break;
                    merge_phase ^= 1;
                    owed = false;
                }
                if (busy) {
                    float s[kPaTile];
                    float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 4; ++k) ld_32x32b_x32(t_s + 32 * k, s + 32 * k);
                    tc::wait_ld();
                    if (a.negate) {
#pragma unroll
                        for (int k = 0; k < kPaTile; ++k) s[k] = -s[k];
                    }
                    if (key0 + kPaTile > whole_end || (key0 < whole_first && key0 + kPaTile > a.sinks)) {
                        const int hi = min(pos + 1, a.room) - key0, sk = min(a.sinks - key0, hi);
                        const int lo = pa_window(a, pos) - key0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t seen = (ones(hi - 32 * k) & ~ones(lo - 32 * k)) | ones(sk - 32 * k);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                s[32 * k + e] = seen & (1u << e) ? s[32 * k + e] : -INFINITY;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kPaTile; k += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e) top4[e] = fmaxf(fmaxf(top4[e], s[k + 2 * e]), s[k + 2 * e + 1]);
                    const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                    // (top - m) c > lazy; m = -inf until the row has seen a key
                    const bool grow = top > m && (m == -INFINITY || (top - m) * c > lazy);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float mn = fmaxf(m, top);
                        const float f = m == -INFINITY ? 0.0f : ex2((m - mn) * c);
                        m = mn;
                        if (any) {
                            // the last PV is done: S's commit came after it
                            l *= f;
#pragma unroll 1
                            for (int k = 0; k < D / 16; ++k) {
                                uint32_t o[16];
                                tc::ld_32x32b_x16(t_o + 16 * k, o);
                                tc::wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tc::st_32x32b_x16(t_o + 16 * k, o);
                            }
                        }
                    }
                    const float mc = m == -INFINITY ? 0.0f : kShift - m * c;
                    const uint64_t c2 = f32x2(c, c), mc2 = f32x2(mc, mc);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int k = 0; k < kPaTile / 32; ++k) {
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float x0, x1;
                            split2(fma2(f32x2(s[32 * k + 2 * e], s[32 * k + 2 * e + 1]), c2, mc2), x0, x1);
                            const float p0 = ex2(x0), p1 = ex2(x1);
                            sum[e & 1] = add2(sum[e & 1], f32x2(p0, p1));
                            p[e] = pack2<F16>(p0, p1);
                        }
                        tc::st_32x32b_x16(t_s + 16 * k, p);
                    }
                    float s0, s1;
                    split2(add2(sum[0], sum[1]), s0, s1);
                    l += s0 + s1;
                    tc::wait_st();
                }
                any = true;
                tc::fence_before_sync();
                arrive(p_full + 8 * slot);
            }
            if (!ok) break;
            at += 2 * steps;
            if (any) {
                ok = step_wait(pv_done + 8 * slot, pv_phase, 0x430 + slot);
                pv_phase ^= 1;
                if (!ok) break;
                tc::fence_after_sync();
            }
            if (!two && slot == 1) {
                // an odd slot leaves m and l; its O lies beside slot 0's
                if (any) {
                    exchange[row] = m;
                    exchange[kPaTile + row] = l;
                    tc::fence_before_sync();
                    arrive(merge_full);
                    owed = true;
                }
                item_done(n);
                continue;
            }
            // O = f0 O_0 + f1 O_1
            float f0 = any ? 1.0f : 0.0f, f1 = 0.0f;
            const bool merge = !two && steps > 1;
            if (merge) {
                ok = step_wait(merge_full, merge_phase, 0x470);
                if (!ok) break;
                merge_phase ^= 1;
                tc::fence_after_sync();
                const float m1 = exchange[row], l1 = exchange[kPaTile + row];
                const float mn = fmaxf(m, m1);
                f0 = m == -INFINITY ? 0.0f : ex2((m - mn) * c);
                f1 = m1 == -INFINITY ? 0.0f : ex2((m1 - mn) * c);
                m = mn;
                l = l * f0 + l1 * f1;
            }
            const int c0 = it.c0, c1 = it.c1, h = it.h, token0 = it.qs + t0;
            item_done(n);
            const bool live = row < rows;
            const bool split = c0 != c1;
            float *part = pa_part<D>(a, blockIdx.x, (int)blockIdx.x == c0, slot);
            if (!split) {                             // the whole item: the output
                const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
                f0 *= inv;
                f1 *= inv;
            }
            const int64_t token = token0 + tok;
            const int head = h * a.group + row - tok * a.group;
            uint16_t *out = a.out + token * a.out_s0 + head * a.out_s1;
            if (busy) {
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    float o[32];
                    if (any) {
                        ld_32x32b_x32(t_o + k, o);
                        tc::wait_ld();
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = any ? o[e] * f0 : 0.0f;
                    if (merge) {
                        float x[32];
                        ld_32x32b_x32(t_o + D + k, x);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] += x[e] * f1;
                    }
                    if (split) {
                        float *dst = part + (k / 4 * kPaTile + row) * 4;
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<float4 *>(dst + e * kPaTile * 4) =
                                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        }
                        continue;
                    }
                    // 4 x 4 transposition of 16-byte pieces over four lanes: a
                    // lane then has the same piece of four rows, and a store
                    // writes 64 bytes of each of eight rows (a row a lane, 16
                    // bytes each, measured 11 us an item)
                    uint32_t w[4][4];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[e / 4][e % 4] = l == 0.0f ? 0u : pack2<F16>(o[2 * e], o[2 * e + 1]);
#pragma unroll
                    for (int b = 1; b < 4; b <<= 1) {
                        const bool upper = lane & b;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (e & b) continue;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t send = upper ? w[e][i] : w[e | b][i];
                                const uint32_t got = __shfl_xor_sync(0xffffffffu, send, b);
                                if (upper) w[e][i] = got; else w[e | b][i] = got;
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint64_t to = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(out), (lane & 28) + e);
                        if ((row & 124) + e < rows)
                            *reinterpret_cast<uint4 *>(to + (k + (lane & 3) * 8) * 2) =
                                make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
                    }
                }
            }
            // O is read: the next item's values may come (its P arrives after this)
            tc::fence_before_sync();
            if (merge) arrive(merge_free);
            if (!split) {
                if (live && a.lse) a.lse[token * a.q_heads + head] = pa_lse<F16>(m, l, c);
                continue;
            }
            // unnormalised, for the second launch
            if (live) {
                float *dst = part + kPaTile * D + row;
                dst[0] = m;
                dst[kPaTile] = l;
            }
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && sh.abort) set_status(a.status, 4u /* MARKOV_ETIMEOUT */, sh.abort);
    if (warp == 8) tc::tmem_dealloc(tmem, 512);
}

// ----------------------------------------------------------------- joining

constexpr int kJoinThreads = 256;

// Block (b, g): 32 rows of the item that begins in block b and is cut, g =
// slot * 4 + their quarter of the tile.  A thread has a row and some vectors of
// four columns; four parts' loads are in flight together.  4 to 5 us of a call:
// latency, of the launch, the parts and their sums (512 threads: no faster).
template <int D, bool F16>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ AttnArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PaJoin j = reinterpret_cast<const PaJoin *>(a.joins)[blockIdx.x];
    const int slot = blockIdx.y >> 2, r = (blockIdx.y & 3) * 32 + (threadIdx.x & 31);
    const int tokens = min(j.tokens - slot * a.tile_tokens, a.tile_tokens);
    if (j.c0 == j.c1 || r >= tokens * a.group || __ldcg(a.status) != 0u) return;
    constexpr int kVec = D / 4 / (kJoinThreads / 32);
    const int k0 = (threadIdx.x >> 5) * kVec;
    const float c = a.scale2;
    float M = -INFINITY, L = 0.0f, o[4 * kVec];
#pragma unroll
    for (int k = 0; k < 4 * kVec; ++k) o[k] = 0.0f;
    for (int b0 = j.c0; b0 <= j.c1; b0 += 4) {
        float pm[4], pl[4], mn = M;
        float4 y[4][kVec];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            pm[e] = -INFINITY;
            pl[e] = 0.0f;
            if (b0 + e > j.c1) continue;
            const float *p = pa_part<D>(a, b0 + e, b0 + e == j.c0, slot);
            pm[e] = __ldcg(p + kPaTile * D + r);
            pl[e] = __ldcg(p + kPaTile * D + kPaTile + r);
#pragma unroll
            for (int k = 0; k < kVec; ++k)
                y[e][k] = __ldcg(reinterpret_cast<const float4 *>(p + ((k0 + k) * kPaTile + r) * 4));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) mn = fmaxf(mn, pm[e]);
        const float f = M == -INFINITY ? 0.0f : ex2((M - mn) * c);
        M = mn;
        L *= f;
#pragma unroll
        for (int k = 0; k < 4 * kVec; ++k) o[k] *= f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (b0 + e > j.c1) continue;
            const float g = pm[e] == -INFINITY ? 0.0f : ex2((pm[e] - M) * c);
            L += pl[e] * g;
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                o[4 * k] += y[e][k].x * g;
                o[4 * k + 1] += y[e][k].y * g;
                o[4 * k + 2] += y[e][k].z * g;
                o[4 * k + 3] += y[e][k].w * g;
            }
        }
    }
    const float inv = L == 0.0f ? 0.0f : __fdiv_rn(1.0f, L);
    const int tok = r * a.group_inv >> 16, head = j.head + r - tok * a.group;
    const int64_t token = j.token + slot * a.tile_tokens + tok;
    uint16_t *out = a.out + token * a.out_s0 + head * a.out_s1 + 4 * k0;
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
        uint2 v = make_uint2(pack2<F16>(o[4 * k] * inv, o[4 * k + 1] * inv), pack2<F16>(o[4 * k + 2] * inv, o[4 * k + 3] * inv));
        if (L == 0.0f) v = make_uint2(0u, 0u);
        *reinterpret_cast<uint2 *>(out + 4 * k) = v;
    }
    if (k0 == 0 && a.lse) a.lse[token * a.q_heads + head] = pa_lse<F16>(M, L, c);
}

template <int D, bool F16>
static cudaError_t launch_typed(const AttnArgs &a, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                                int blocks, cudaStream_t s) {
    paged_attention_kernel<D, F16><<<blocks, kPaThreads, PaShape<D>::kSmem, s>>>(a, q, k, v);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, 8);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, F16>, a);
}

cudaError_t launch_paged_attention(const AttnArgs &a, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                                   int head_dim, bool f16, int blocks, cudaStream_t s) {
    if (head_dim == 64)
        return f16 ? launch_typed<64, true>(a, q, k, v, blocks, s) : launch_typed<64, false>(a, q, k, v, blocks, s);
    return f16 ? launch_typed<128, true>(a, q, k, v, blocks, s) : launch_typed<128, false>(a, q, k, v, blocks, s);
}

cudaError_t paged_attention_prepare() {
    const auto set = [](const void *fn, int bytes) {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    };
    cudaError_t e = set((const void *)paged_attention_kernel<64, false>, PaShape<64>::kSmem);
    if (e == cudaSuccess) e = set((const void *)paged_attention_kernel<64, true>, PaShape<64>::kSmem);
    if (e == cudaSuccess) e = set((const void *)paged_attention_kernel<128, false>, PaShape<128>::kSmem);
    if (e == cudaSuccess) e = set((const void *)paged_attention_kernel<128, true>, PaShape<128>::kSmem);
    return e;
}

// Floats of the parts that `blocks` blocks may leave.
size_t paged_attention_parts(int head_dim, int blocks) {
    return (size_t)blocks * 4 * kPaTile * (head_dim + 2);
}

size_t paged_attention_joins(int blocks) { return blocks * sizeof(PaJoin); }

}  // namespace dtm
