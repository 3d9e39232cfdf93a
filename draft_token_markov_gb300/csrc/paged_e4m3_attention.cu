// paged_e4m3_attention.cu -- attention of chunks of new tokens over a paged e4m3
// cache on tcgen05: drafts of many query rows, prompt chunks, mixed batches.
//
// Rows, items, the two slots that take turns on the tensor core and the cut of the
// call's work into ranges are those of the attention over a 16-bit cache: an item
// is (request, key head, up to two tiles of 128 stacked query rows, or one where a
// request has no more on average), its keys go by in tiles of 128.  Between the loads and the MMAs stands a warpgroup of its own:
// it reads a tile as TMA brought it (bytes, a row a thread) and writes it as fp16
// in the operand's swizzled layout, exactly; values that nobody sees become zeros
// there.  BF16 queries become fp16 ones in place, each row times a power of two
// that its scores are freed of again.
//   S = Q K^T,  y = S c ks + log2 vs,  p = 2^(y - m),  l += 2^(-log2 vs) sum p,
//   O += P V    (p rounded to fp16, in TMEM over S)
// ks and vs of 16 keys come from a ring in shared memory: the scales cost the
// softmax a product for each maximum of 16 scores and two additions for each 16
// weights.  m is the maximum of y and moves when a row's has grown by 2^8 or more.
//
// Roles.  Warps 0-3 and 4-7: softmax and output of the two slots, a thread a row;
// 8-11: conversion; 12: MMAs; 13 and 14: loads of keys and values, the former with
// the scales of both; 15: walks the block's items and loads queries.
//
// Bounds.  4096 tokens over 16384 keys (32 / 8 heads of 128) take 722 us, 1332 TFLOP/s
// (68% of the GEMM rate; 660 us over a cache of BF16): a turn of two row tiles over 128
// keys takes some 3600 cycles, of which the MMAs are 2048; a slot's softmax and its
// hand-overs are most of the rest, and shared memory is busy with operands, conversion
// and loads (about 2900 cycles of 128 bytes).  Without conversion and scales it took
// 729 us of what were then 840.  Instructions to fetch counted most: with the conversion
// loops rolled, one body for keys and values, and negative scales put into the queries,
// 840 us became 722, and 32 rows of 9 tokens over 500 to 16000 keys 117 us 90.  8 rows of
// 9 tokens over 1000 to 16000 keys take 36 us in a graph (74 MB, 11 us at the copy
// rate; 38.7 us with pairs of row tiles): some 17 us for start, ends and the join, the
// rest conversion of every tile by one warpgroup (some 1300 cycles for keys and values).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention_tc.cuh"
#include "common.cuh"
#include "e4m3.cuh"
#include "f32x2.cuh"
#include "paged.h"
#include "paged_rows.cuh"
#include "tc.cuh"

namespace dtm {

namespace {

constexpr int kManyThreads = 512;
constexpr int kRing = 4;                     // items that are known ahead
constexpr int kTileRows = 128, kTileShift = 7;   // keys of a tile, and rows
constexpr int kGrains = kTileRows / 16;          // groups of 16 keys of a tile, a scale each
constexpr int kScaleRing = 8;                // tiles whose scales are kept; eight at most are in use (five with D = 128)
// an item's start and end, in tiles of one and of two row tiles.  In us, for 16 rows of
// 1-500 tokens (7 query heads a key head), 24 rows of 1-300 (8) and 32 rows of 9 tokens:
// 3 and 10 109, 123, 90; 3 and 7 108, 131, 90; 4 and 9 105, 127, 93; 6 and 12 112, 124, 97
constexpr int kWeightOne = 3, kWeightTwo = 10;
constexpr uint64_t kUnitNs = 20000;          // what a unit of work may take at most
constexpr uint32_t kReaders = 15;            // warps that read an item

// ONE: items are of one row tile, whose queries take the place of one tile; the other's
// is an operand's.
template <int D, bool ONE>
struct Shape {
    static constexpr int kQueries = ONE ? 1 : 2;                 // tiles of queries
    static constexpr int kHalf = kTileRows * 128;                // 64 elements of every row
    static constexpr int kHalves = D / 64;
    static constexpr int kOperand = kTileRows * D * 2;           // a tile of queries, or of keys or values in fp16
    static constexpr int kRaw = kTileRows * D;                   // one of keys or values in e4m3
    static constexpr int kOperands = (D == 128 ? 5 : 7) - kQueries, kRaws = D == 128 ? 4 : 8;
    static constexpr int kOperandAt = kQueries * kOperand;
    static constexpr int kRawAt = kOperandAt + kOperands * kOperand;
    static constexpr int kExchange = kRawAt + kRaws * kRaw;
    static constexpr int kScales = kExchange + 2 * kTileRows * 4;
    static constexpr int kRowExp = kScales + kScaleRing * 3 * kGrains * 4;
    static constexpr int kBars = kRowExp + 4 * kTileRows;
    static constexpr int kMisc = kBars + 8 * (2 * kOperands + 2 * kRaws + 15 + 2 * kRing);
    static constexpr int kSmem = kMisc + 256;
};
static_assert(Shape<128, false>::kSmem <= 232448 && Shape<64, false>::kSmem <= 232448, "shared memory");
static_assert(Shape<128, true>::kSmem <= 232448 && Shape<64, true>::kSmem <= 232448, "shared memory");

struct Item {
    int tokens, t0;            // tokens of the item (0: no more items), the first within the request
    int qs, pos0, state;       // the request's first token, its position; its table row, -1 for none
    int h;                     // key head
    int end, first, kept;      // some row sees keys [first, end) and [0, kept)
    int sink_tiles, w0;        // key tiles: [0, sink_tiles), then from w0 on
    int j0, steps;             // the block's share: key tiles from the j0-th on
    int c0, c1;                // blocks that share the item
};

struct Shared {
    uint32_t abort, tmem;
    Item ring[kRing];
};
static_assert(sizeof(Shared) <= 256, "kMisc");

// What the joining launch has to know of the item that begins in a block and goes
// on in the next (c0 == c1: none).
struct Join {
    int c0, c1;
    int token, tokens, head;   // its first token, its tokens, its first query head
};

// The m-th item of a request's key head: a pair of row tiles, or one.
template <bool ONE>
__device__ __forceinline__ void span(const AttnE4m3Args &a, const RowOfCall &q, int m, Item &it) {
    const int most = ONE ? a.tile_tokens : 2 * a.tile_tokens;
    it.t0 = m * most;
    it.tokens = min(q.np - it.t0, most);
    const int p0 = q.pos0 + it.t0;
    const KeySpan s = key_span<kTileShift>(a.r, a.window, a.sinks, q.state, p0, p0 + it.tokens - 1);
    it.end = s.end;
    it.first = s.first;
    it.kept = s.kept;
    it.sink_tiles = s.sinks;
    it.w0 = s.w0;
    it.steps = s.steps;
}

// An item's weight: its start and end, its key tiles (twice where it has two row
// tiles).
__device__ __forceinline__ int tile_weight(const AttnE4m3Args &a, const Item &it) { return it.tokens > a.tile_tokens ? 2 : 1; }
__device__ __forceinline__ int ends_weight(const AttnE4m3Args &a, const Item &it) {
    return it.tokens > a.tile_tokens ? kWeightTwo : kWeightOne;
}
__device__ __forceinline__ uint32_t weight(const AttnE4m3Args &a, const Item &it) {
    return ends_weight(a, it) + max(it.steps, 1) * tile_weight(a, it);
}
// How many of its key tiles end before an offset.
__device__ __forceinline__ int tile_at(const AttnE4m3Args &a, const Item &it, uint32_t off) {
    const int past = (int)off - ends_weight(a, it);
    return past <= 0 ? 0 : min(past / tile_weight(a, it), max(it.steps, 1));
}
// The weight of an item and its key tiles.
template <bool ONE>
__device__ __noinline__ uint2 units_of(const AttnE4m3Args &a, RowOfCall q, int m) {
    Item it;
    span<ONE>(a, q, m, it);
    return make_uint2(weight(a, it), it.steps);
}
template <bool ONE>
__device__ __forceinline__ int items_of(const AttnE4m3Args &a, const RowOfCall &q) {
    const int most = ONE ? a.tile_tokens : 2 * a.tile_tokens;
    return (q.np + most - 1) / most;
}

// An item's part from a block, for one slot: [D / 4][128 rows] vectors of four
// columns, then m and l.
template <int D>
__device__ __forceinline__ float *part_of(const AttnE4m3Args &a, int block, bool begins, int slot) {
    return a.parts + ((int64_t)(block * 2 + (begins ? 1 : 0)) * 2 + slot) * kTileRows * (D + 2);
}

// m + log2 l, less the weights' shift, as a natural logarithm.
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : (m - kShiftE4 + __log2f(l)) * 0.69314718055994531f;
}

__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// A row of a tile of bytes as fp16 in the operand's layout, or zeros.  The TMA's
// swizzle of the bytes (128 bytes a row, or 64) and the operand's (128) let eight
// neighbouring rows' vectors fall to different banks.
template <int D>
__device__ __forceinline__ void convert_row(uint32_t raw, uint32_t operand, int row, bool zero) {
    constexpr int kVec = D / 16;
    const int x = row & 7;
    const uint32_t from = raw + row * D, to = operand + row * 128;
#pragma unroll 1
    for (int v0 = 0; v0 < kVec; v0 += 2) {
        uint4 w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] = lds128(from + (((v0 + i) ^ (D == 128 ? x : x >> 1)) << 4));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t h[8];
            if (zero) w[i] = make_uint4(0, 0, 0, 0);
            f16x4_of_e4m3(w[i].x, h[0], h[1]);
            f16x4_of_e4m3(w[i].y, h[2], h[3]);
            f16x4_of_e4m3(w[i].z, h[4], h[5]);
            f16x4_of_e4m3(w[i].w, h[6], h[7]);
            const uint32_t half = to + (v0 >> 2) * (kTileRows * 128);
            sts128(half + (((2 * (v0 + i) & 7) ^ x) << 4), h[0], h[1], h[2], h[3]);
            sts128(half + (((2 * (v0 + i) + 1 & 7) ^ x) << 4), h[4], h[5], h[6], h[7]);
        }
    }
}

// A row of BF16 queries times 2^k as fp16, in place, with `sign` (of a negative scale)
// in each half's sign bit; returns k.  fp16 queries get the sign alone.
template <int D, bool F16>
__device__ __forceinline__ int convert_query(uint32_t tile, int row, uint32_t sign) {
    constexpr int kVec = D / 8;
    const uint32_t at = tile + row * 128;
    const auto place = [&](int v) { return at + (v >> 3) * (kTileRows * 128) + (((v & 7) ^ (row & 7)) << 4); };
    if (F16) {
#pragma unroll 2
        for (int v = 0; v < kVec; ++v) {
            const uint4 w = lds128(place(v));
            sts128(place(v), w.x ^ sign, w.y ^ sign, w.z ^ sign, w.w ^ sign);
        }
        return 0;
    }
    uint32_t top = 0;
#pragma unroll 2
    for (int v = 0; v < kVec; ++v) {
        const uint4 w = lds128(place(v));
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(a[i] << 16 & 0x7fffffffu, a[i] & 0x7fff0000u));
    }
    // NaN counts as the largest
    const int k = row_exponent(__uint_as_float(min(top, 0x7f800000u)));
    const float power = power_of_two(k);
#pragma unroll 2
    for (int v = 0; v < kVec; ++v) {
        const uint4 w = lds128(place(v));
        uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            a[i] = pack2<true>(__uint_as_float(a[i] << 16) * power, __uint_as_float(a[i] & 0xffff0000u) * power);
        sts128(place(v), a[0] ^ sign, a[1] ^ sign, a[2] ^ sign, a[3] ^ sign);
    }
    return k;
}

// ------------------------------------------------------------------ kernel

template <int D, bool F16, bool ONE>
__global__ void __launch_bounds__(kManyThreads, 1)
attention_e4m3_kernel(const __grid_constant__ AttnE4m3Args a, const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using S = Shape<D, ONE>;
    constexpr uint32_t kQs = S::kQueries;
    extern __shared__ __align__(1024) uint8_t base[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t smem = tc::smem_u32(base), operands = smem + S::kOperandAt, raws = smem + S::kRawAt;
    float *exchange = reinterpret_cast<float *>(base + S::kExchange);
    float *scales = reinterpret_cast<float *>(base + S::kScales);
    uint8_t *row_exp = base + S::kRowExp;
    Shared &sh = *reinterpret_cast<Shared *>(base + S::kMisc);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t raw_full = smem + S::kBars, raw_empty = raw_full + 8 * S::kRaws, op_full = raw_empty + 8 * S::kRaws,
                   op_empty = op_full + 8 * S::kOperands, q_full = op_empty + 8 * S::kOperands, q_empty = q_full + 16,
                   q_ready = q_full + 32, s_full = q_full + 48, p_full = q_full + 64, pv_done = q_full + 80,
                   merge_full = q_full + 96, merge_free = q_full + 104, leave = q_full + 112,
                   item_full = q_full + 120, item_empty = item_full + 8 * kRing;
    if (tid == 0) {
        sh.abort = 0;
        for (int i = 0; i < S::kRaws; ++i) {
            tc::mbar_init(raw_full + 8 * i, 1);
            tc::mbar_init(raw_empty + 8 * i, 4);     // the converting warps
        }
        for (int i = 0; i < S::kOperands; ++i) {
            tc::mbar_init(op_full + 8 * i, 4);
            tc::mbar_init(op_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(q_full + 8 * i, 1);
            tc::mbar_init(q_empty + 8 * i, 1);
            tc::mbar_init(q_ready + 8 * i, 4);
            tc::mbar_init(s_full + 8 * i, 1);
            tc::mbar_init(p_full + 8 * i, 4);        // the slot's warps
            tc::mbar_init(pv_done + 8 * i, 1);
        }
        tc::mbar_init(merge_full, 4);                // slot 1's warps
        tc::mbar_init(merge_free, 4);                // slot 0's
        tc::mbar_init(leave, 1);
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(item_full + 8 * i, 1);
            tc::mbar_init(item_empty + 8 * i, kReaders);
        }
        tc::mbar_init_fence();
    }
    if (warp >= 13 && lane == 0) {
        const CUtensorMap *map = warp == 13 ? &kmap : warp == 14 ? &vmap : &qmap;
        asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    }
    if (warp == 12) tc::tmem_alloc(tc::smem_u32(&sh.tmem), 512);
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
    // the n-th item; its fields are read from shared memory where they are used
    auto item = [&](uint32_t n) -> const volatile Item & { return sh.ring[n % kRing]; };
    auto item_wait = [&](uint32_t n) { return all_wait(item_full + 8 * (n % kRing), (n / kRing) & 1, 0x500, a.walk_ns); };
    auto item_done = [&](uint32_t n) { arrive(item_empty + 8 * (n % kRing)); };
    // the stage and the phase of the at-th use of a ring of N
    struct Place {
        uint32_t stage, phase;
    };

    // 256 x 192 + 256 x 64 registers of the 512 x 128 at launch
    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 15) {
        // ------------------------------------------- the walk, query loads
        Item it;
        const uint32_t pending = __ldcg(a.status);   // a pending status: nothing is done
        uint64_t total = 0, tiles_seen = 0;          // the call's units, this lane's rows' key tiles
        // the rows' units before and with each, where operands will be
        uint64_t *units_to = reinterpret_cast<uint64_t *>(base + S::kOperandAt);
#pragma unroll 1
        for (int r0 = 0; r0 < a.r.rows; r0 += 32) {
            uint64_t x = 0, y = 0;
            if (r0 + lane < a.r.rows) {
                const RowOfCall q = row_of_call(a.r, r0 + lane);
                const int pairs = items_of<ONE>(a, q);
#pragma unroll 1
                for (int m = 0; m < pairs; ++m) {
                    const uint2 units = units_of<ONE>(a, q, m);
                    x += units.x;
                    y += units.y;
                }
            }
            uint64_t incl = x * a.kv_heads;
            tiles_seen += y * a.kv_heads;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t z = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += z;
            }
            units_to[r0 + lane] = total + incl;
            total += __shfl_sync(0xffffffffu, incl, 31);
        }
        __syncwarp();
        if (total >> 31) {                           // fewer key tiles than units
#pragma unroll 1
            for (int o = 16; o > 0; o >>= 1) tiles_seen += __shfl_xor_sync(0xffffffffu, tiles_seen, o);
            if (tiles_seen >> 31) {
                if (lane == 0 && !pending) set_status(a.status, 2u /* MARKOV_EUNSUPPORTED */, 0x600);
                total = 0;
            }
        }
        UnitSplit split;
        split.cut(pending ? 0u : total, gridDim.x, 2);       // a range holds a tile of either weight
        uint64_t u = 0, u_end = 0;                   // the current item's first unit, the range's end
        uint32_t skip = 0;                           // units of the first item before the range
        RowOfCall q{0, 0, 0, -1};
        int r = 0, h = 0, m = 0, pairs = 0;
        if (blockIdx.x < split.ranges) {
            const uint64_t u0 = split.first(blockIdx.x);
            u_end = split.first(blockIdx.x + 1);
#pragma unroll 1
            for (int r0 = 0;; r0 += 32) {
                const int x = r0 + lane;
                const bool here = x < a.r.rows && u0 < units_to[x] && (x == 0 || u0 >= units_to[x - 1]);
                const uint32_t found = __ballot_sync(0xffffffffu, here);
                if (found) { r = r0 + __ffs(found) - 1; break; }
            }
            const uint64_t before = r ? units_to[r - 1] : 0, units = units_to[r] - before;
            q = row_of_call(a.r, r);
            pairs = items_of<ONE>(a, q);
            const uint64_t head = units / a.kv_heads;
            h = (int)((u0 - before) / head);
            u = before + h * head;
#pragma unroll 1
            for (;; ++m) {
                const uint32_t w = units_of<ONE>(a, q, m).x;
                if (u0 - u < w) break;
                u += w;
            }
            skip = (uint32_t)(u0 - u);
        }
        __syncwarp();                                // units_to is read; operands come
        uint32_t qt = 0;                             // query tiles loaded
        Join join{0, 0, 0, 0, 0};
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
                span<ONE>(a, q, m, it);
                const uint32_t units = weight(a, it), w = tile_weight(a, it);
                const int all = max(it.steps, 1);
                it.j0 = tile_at(a, it, skip);
                const int j1 = u_end - u < units ? tile_at(a, it, (uint32_t)(u_end - u)) : all;
                more = it.j0 < j1;                   // not a tile of it: another block's
                if (more) {
                    limit_ns += (uint64_t)(j1 - it.j0) * w * kUnitNs;
                    it.qs = q.qs;
                    it.pos0 = q.pos0;
                    it.state = q.state;
                    it.h = h;
                    it.c0 = it.c1 = blockIdx.x;
                    if (it.j0 > 0 || j1 < all) {
                        it.c0 = split.range_of(u + ends_weight(a, it) + w - 1);
                        it.c1 = split.range_of(u + units - 1);
                    }
                    it.steps = min(j1, it.steps) - it.j0;    // 0 where nothing is seen
                    if (it.steps > 0) {
                        q_token = q.qs + it.t0;
                        q_head = h * a.group;
                        q_tiles = w;
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
                                q = row_of_call(a.r, ++r);
                            } while (q.np <= 0);
                            pairs = items_of<ONE>(a, q);
                        }
                    }
                }
            }
            if (!more) it.tokens = 0;
            if (more && it.c0 != it.c1 && it.c0 == (int)blockIdx.x)
                join = Join{it.c0, it.c1, it.qs + it.t0, it.tokens, it.h * a.group};
            if (lane == 0) sh.ring[n % kRing] = it;
            arrive(item_full + 8 * (n % kRing));
            // the queries of the item before (of the first at once), so that the
            // loads of keys know of an item ahead
            if (n == 0) {
                token = q_token;
                head = q_head;
                tiles = q_tiles;
                q_tiles = 0;
            }
#pragma unroll 1
            for (int s = 0; s < tiles; ++s, token += a.tile_tokens) {
                const uint32_t buf = qt % kQs, full = q_full + 8 * buf;
                ok = all_wait(q_empty + 8 * buf, (qt / kQs & 1) ^ 1, 0x300 + buf, limit_ns);
                if (!ok) break;
                ++qt;
                if (lane == 0) {
                    tc::mbar_expect_tx(full, a.tile_tokens * a.group * D * 2);
#pragma unroll 1
                    for (int half = 0; half < S::kHalves; ++half)
                        tma_load_3d(smem + buf * S::kOperand + half * S::kHalf, &qmap, half * 64, head, token, full);
                }
                __syncwarp();
            }
            if (!more) break;
        }
        if (lane == 0) reinterpret_cast<Join *>(a.joins)[blockIdx.x] = join;
        if (lane == 0 && sh.abort) {
            // gave up: no load may be in flight when the block leaves
            const uint64_t until = tc::now_ns() + a.timeout_ns;
            for (uint32_t t = qt > kQs ? qt - kQs : 0; t < qt; ++t)
                while (!tc::mbar_test(q_full + 8 * (t % kQs), t / kQs & 1) && tc::now_ns() < until) {}
        }
    } else if (warp == 13 || warp == 14) {
        // ------------------------------------------------ key / value loads
        const bool values = warp == 14;
        const CUtensorMap *map = values ? &vmap : &kmap;
        const int page = 1 << a.r.page_shift;
        const int box = min(page, kTileRows), boxes = kTileRows / box;       // boxes of a tile
        uint32_t at = values ? 1 : 0;                // in the ring: K V K V ...
        bool ok = true;
        for (uint32_t n = 0; ok; ++n) {
            ok = item_wait(n);
            const volatile Item &it = item(n);
            if (!ok || it.tokens == 0) break;
            const int32_t *table = a.r.table + (int64_t)max(it.state, 0) * a.r.table_s0;
            const int j0 = it.j0, j1 = j0 + it.steps, sinks = it.sink_tiles, w0 = it.w0;
            const int end = it.end, first = it.first, kept = it.kept, h = it.h;
            item_done(n);
            auto key_of = [&](int j) { return (j < sinks ? j : w0 + j - sinks) * kTileRows; };
            auto seen = [&](int key, int n) { return key < end && (key + n > first || key < kept); };
            auto page_of = [&](int j) {
                const int key = key_of(j) + lane * box;
                if (j >= j1 || lane >= boxes || !seen(key, box)) return -1;
                const int id = __ldg(table + (key >> a.r.page_shift));
                return id >= 0 && id < a.r.num_pages ? id : -1;
            };
            // lane g: the scale of the tile's g-th 16 keys, lane kGrains + g: of their
            // values, 1 where nobody sees one.  Both are the keys' warp's: the softmax reads
            // them once a tile's scores are done, which wait for its keys, not for its values
            auto scale_of = [&](int j, int pids) {
                const int g = lane & (kGrains - 1), id = __shfl_sync(0xffffffffu, pids, g * 16 / box);
                if (values || j >= j1 || lane >= 2 * kGrains) return 1.0f;
                const int key = key_of(j) + g * 16;
                if (id < 0 || !seen(key, 16)) return 1.0f;
                const E4m3Scales &sc = lane < kGrains ? a.ks : a.vs;
                return __ldg(sc.p + id * sc.s_page + ((key & (page - 1)) >> sc.block_shift) * sc.s_block + h * sc.s_head);
            };
            int pid = page_of(j0), pid_next = page_of(j0 + 1);
            float scale = scale_of(j0, pid);
            for (int j = j0; j < j1; ++j, at += 2) {
                const int slot0 = key_of(j) & (page - 1);
                const uint32_t stage = at % S::kRaws, phase = at / S::kRaws & 1, full = raw_full + 8 * stage;
                ok = step_wait(raw_empty + 8 * stage, phase ^ 1, 0x100 + stage);
                if (!ok) break;
                if (!values && lane < 2 * kGrains) {
                    float *to = scales + (at / 2 % kScaleRing) * 3 * kGrains + lane;
                    if (lane < kGrains) {
                        to[0] = fmaxf(scale, 1e-30f);        // positive: a masked score stays -inf
                    } else {
                        const float lv = scale_log2(scale);
                        to[0] = lv;
                        to[kGrains] = ex2(-lv);
                    }
                }
                __syncwarp();                                // before the arrival that the scores wait for
                if (lane == 0) tc::mbar_expect_tx(full, S::kRaw);
                __syncwarp();
                // the whole warp goes through the boxes, an elected lane issues
                uint32_t dst = raws + stage * S::kRaw;
#pragma unroll 1
                for (int b = 0; b < boxes; ++b, dst += box * D)
                    tma_load_4d_elect(dst, map, 0, slot0, h, __shfl_sync(0xffffffffu, pid, b), full);
                pid = pid_next;
                scale = scale_of(j + 1, pid);
                pid_next = page_of(j + 2);
            }
        }
        if (lane == 0 && sh.abort) {
            // gave up: no load may be in flight when the block leaves; this warp's
            // uses of the ring end before `at`
            const uint64_t until = tc::now_ns() + a.timeout_ns;
            for (int i = 1; i <= S::kRaws / 2; ++i) {
                if (at < 2u * i) break;
                const uint32_t t = at - 2 * i;
                while (!tc::mbar_test(raw_full + 8 * (t % S::kRaws), t / S::kRaws & 1) && tc::now_ns() < until) {}
            }
        }
    } else if (warp == 12) {
        // ---------------------------------------------------- MMA issue
        // the whole warp, so that control flow and descriptors stay uniform;
        // an elected lane issues
        uint32_t qt = 0, p_phase = 0;                // p_phase: a bit a slot
        bool ok = true;
        constexpr uint32_t kIdescS = pa_idesc<true>(kTileRows, false), kIdescO = pa_idesc<true>(D, true);
        constexpr uint32_t kStep = S::kOperand / 16;
        const uint64_t q_desc = tc::sw128_desc(smem), k_desc = tc::sw128_desc(operands), v_desc = sw128_mn_desc(operands, S::kHalf);
        const uint32_t t_o = tmem + 2 * kTileRows;
        auto after = [](Place p, int n) {
            p.stage += n;
            if (p.stage >= S::kOperands) { p.stage -= S::kOperands; p.phase ^= 1; }
            return p;
        };
        auto loaded = [&](Place k) { return step_wait(op_full + 8 * k.stage, k.phase, 0x200); };
        auto scores = [&](int slot, uint32_t tile, Place k) {
            mma_scores<D>(tmem + slot * kTileRows, q_desc + tile % kQs * kStep, k_desc + k.stage * kStep, kIdescS);
            tc::commit_elect(s_full + 8 * slot);
        };
        // O += P V, once the slot's P is there
        auto values = [&](int slot, Place v, bool accumulate) {
            if (!step_wait(p_full + 8 * slot, p_phase >> slot & 1, 0x220 + slot)) return false;
            p_phase ^= 1u << slot;
            tc::fence_after_sync();
            mma_values(t_o + slot * D, tmem + slot * kTileRows, v_desc + v.stage * kStep, kIdescO, accumulate);
            return true;
        };
        auto release = [&](Place k) { tc::commit_elect(op_empty + 8 * k.stage); };
        auto queries = [&](uint32_t tile) {
            return step_wait((F16 && a.scale2 >= 0.0f ? q_full : q_ready) + 8 * (tile % kQs), tile / kQs & 1, 0x210 + tile % kQs);
        };
        Place k{0, 0};                               // the next key tile for scores
        for (uint32_t n = 0; ok; ++n) {
            ok = item_wait(n);
            const int tokens = item(n).tokens, steps = item(n).steps;
            if (!ok || tokens == 0) break;
            item_done(n);
            if (steps <= 0) continue;                // nothing seen: the output is written without MMAs
            // Either way a slot's turn is: its P comes, O += P V, the next scores
            // over P's place (MMAs run in the order of their issue).
            Place v = after(k, 1);
            if (!ONE && tokens > a.tile_tokens) {
                // two row tiles, a slot each, every key tile for both
                ok = queries(qt) && loaded(k);
                if (!ok) break;
                tc::fence_after_sync();
                scores(0, qt, k);
                ok = queries(qt + 1);
                if (!ok) break;
                tc::fence_after_sync();
                scores(1, qt + 1, k);
                release(k);
                k = after(k, 2);
#pragma unroll 1
                for (int j = 1; j < steps; ++j) {
                    ok = loaded(v) && values(0, v, j > 1) && loaded(k);
                    if (!ok) break;
                    tc::fence_after_sync();
                    scores(0, qt, k);
                    ok = values(1, v, j > 1);
                    if (!ok) break;
                    release(v);
                    scores(1, qt + 1, k);
                    release(k);
                    v = after(v, 2);
                    k = after(k, 2);
                }
                if (!ok) break;
                tc::commit_elect(q_empty + 8 * (qt % kQs));
                tc::commit_elect(q_empty + 8 * ((qt + 1) % kQs));
                qt += 2;
                ok = loaded(v);
#pragma unroll 1
                for (int s = 0; ok && s < 2; ++s) {
                    ok = values(s, v, steps > 1);
                    if (ok) tc::commit_elect(pv_done + 8 * s);
                }
                release(v);
            } else {
                // one: the key tiles in turn
                ok = queries(qt);
#pragma unroll 1
                for (int j = 0; ok && j < steps && j < 2; ++j) {
                    ok = loaded(k);
                    if (!ok) break;
                    tc::fence_after_sync();
                    scores(j, qt, k);
                    release(k);
                    k = after(k, 2);
                }
                if (steps <= 2) tc::commit_elect(q_empty + 8 * (qt % kQs));
#pragma unroll 1
                for (int j = 0; ok && j < steps; ++j) {
                    ok = loaded(v) && values(j & 1, v, j > 1);
                    if (!ok) break;
                    release(v);                      // before the wait for keys: the loads may need the place
                    v = after(v, 2);
                    if (j + 2 < steps) {
                        ok = loaded(k);
                        if (!ok) break;
                        tc::fence_after_sync();
                        scores(j & 1, qt, k);
                        release(k);
                        if (j + 3 == steps) tc::commit_elect(q_empty + 8 * (qt % kQs));
                        k = after(k, 2);
                    } else {
                        tc::commit_elect(pv_done + 8 * (j & 1));
                    }
                }
                ++qt;
            }
        }
        if (sh.abort) {
            // gave up: no MMA may be in flight when the block leaves
            tc::commit_elect(leave);
            tc::mbar_wait_for(leave, 0, a.timeout_ns);
        }
    } else if (warp >= 8) {
        // -------------------------------------------------------- conversion
        const int row = tid & 127;
        uint32_t qt = 0, raw = 0, op = 0;            // query tiles, tiles of bytes and operands so far
        bool ok = true;
        // the next tile of the ring
        auto convert = [&](bool zero) {
            const uint32_t rs = raw % S::kRaws, os = op % S::kOperands;
            ok = step_wait(raw_full + 8 * rs, raw / S::kRaws & 1, 0x800 + rs) &&
                 step_wait(op_empty + 8 * os, (op / S::kOperands & 1) ^ 1, 0x820 + os);
            if (!ok) return;
            convert_row<D>(raws + rs * S::kRaw, operands + os * S::kOperand, row, zero);
            tc::fence_proxy_async_smem();
            arrive(raw_empty + 8 * rs);
            arrive(op_full + 8 * os);
            ++raw;
            ++op;
        };
        for (uint32_t n = 0; ok; ++n) {
            ok = item_wait(n);
            const volatile Item &it = item(n);
            if (!ok || it.tokens == 0) break;
            const int tiles = !ONE && it.tokens > a.tile_tokens ? 2 : 1, steps = it.steps;
            const int j0 = it.j0, sinks = it.sink_tiles, w0 = it.w0, end = it.end, first = it.first, kept = it.kept;
            item_done(n);
            if (steps <= 0) continue;
            if (!F16 || a.scale2 < 0.0f) {
#pragma unroll 1
                for (int s = 0; s < tiles; ++s, ++qt) {
                    ok = step_wait(q_full + 8 * (qt % kQs), qt / kQs & 1, 0x840);
                    if (!ok) break;
                    const int k = convert_query<D, F16>(smem + qt % kQs * S::kOperand, row, a.scale2 < 0.0f ? 0x80008000u : 0u);
                    row_exp[(qt & 3) * kTileRows + row] = (uint8_t)(k + 127);
                    tc::fence_proxy_async_smem();
                    arrive(q_ready + 8 * (qt % kQs));
                }
            }
            // keys and values in turn, by the same code
            const int tiles2 = 2 * steps;
#pragma unroll 1
            for (int i = 0; ok && i < tiles2; ++i) {
                const int j = j0 + (i >> 1), key = (j < sinks ? j : w0 + j - sinks) * kTileRows + row;
                convert((i & 1) && (key >= end || (key < first && key >= kept)));
            }
        }
    } else {
        // -------------------------------------------- softmax and output
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        const int slot = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;    // TMEM lane of the warp
        const uint32_t t_s = tmem + slot * kTileRows + lanes, t_o = tmem + 2 * kTileRows + slot * D + lanes;
        uint32_t s_phase = 0, pv_phase = 0, merge_phase = 0, qt = 0, tile = 0;
        bool ok = true, owed = false;                 // owed: slot 0 may not have read what slot 1 left
        for (uint32_t n = 0; ok; ++n) {
            ok = item_wait(n);
            const volatile Item &it = item(n);
            if (!ok || it.tokens == 0) break;
            const bool two = !ONE && it.tokens > a.tile_tokens;
            const int t0 = it.t0 + (two ? slot * a.tile_tokens : 0);
            const int tokens = min(it.tokens + it.t0 - t0, a.tile_tokens), rows = tokens * a.group;
            const int steps = it.steps, ahead = two ? 1 : 2;
            // rows past the tokens take the last one's position: theirs may not fit
            const int tok = row * a.group_inv >> 16, pos = it.pos0 + t0 + min(tok, tokens - 1);
            const bool busy = (warp & 3) * 32 < rows;
            // a tile is seen whole by the warp's rows when its last key is not past
            // the first one's and its first within the last one's window
            const int whole_end = min(__shfl_sync(0xffffffffu, pos, 0) + 1, a.r.room);
            const int whole_first = window_start(a.window, __shfl_sync(0xffffffffu, pos, 31));
            float m = -INFINITY, l = 0.0f, c = 0.0f;
            bool any = false;                         // a key tile of this slot's went by
            for (int i = two ? 0 : slot; i < steps; i += ahead) {
                int key0 = it.j0 + i;
                {
                    const int sink_tiles = it.sink_tiles;
                    key0 = (key0 < sink_tiles ? key0 : it.w0 + key0 - sink_tiles) * kTileRows;
                }
                ok = step_wait(s_full + 8 * slot, s_phase, 0x400 + slot);
                if (!ok) break;
                s_phase ^= 1;
                tc::fence_after_sync();
                if (owed) {                           // before this slot's O is written again
                    ok = step_wait(merge_free, merge_phase, 0x460);
                    if (!ok) break;
                    merge_phase ^= 1;
                    owed = false;
                }
                if (!any) {
                    // the factor on the row's scores, never 0
                    c = fmaxf(fabsf(a.scale2), 1e-30f);
                    if (!F16) c *= power_of_two(127 - row_exp[((qt + (two ? slot : 0)) & 3) * kTileRows + row]);
                }
                if (busy) {
                    const float *sc = scales + ((tile + i) % kScaleRing) * 3 * kGrains;
                    float s[kTileRows];
#pragma unroll
                    for (int k = 0; k < 4; ++k) ld_32x32b_x32(t_s + 32 * k, s + 32 * k);
                    tc::wait_ld();
                    if (key0 + kTileRows > whole_end || (key0 < whole_first && key0 + kTileRows > a.sinks)) {
                        const int hi = min(pos + 1, a.r.room) - key0, sk = min(a.sinks - key0, hi);
                        const int lo = window_start(a.window, pos) - key0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t seen = (ones(hi - 32 * k) & ~ones(lo - 32 * k)) | ones(sk - 32 * k);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                s[32 * k + e] = seen & (1u << e) ? s[32 * k + e] : -INFINITY;
                        }
                    }
                    // the factors of 16 keys each; not below the least normal, as -inf * 0 is NaN
                    auto factor = [&](int g) { return fmaxf(sc[g] * c, 1.2e-38f); };
                    float top = -INFINITY;
#pragma unroll
                    for (int g = 0; g < kGrains; ++g) {
                        float t = fmaxf(s[16 * g], s[16 * g + 1]), t2 = fmaxf(s[16 * g + 2], s[16 * g + 3]);
#pragma unroll
                        for (int e = 4; e < 16; e += 4) {
                            t = fmaxf(fmaxf(t, s[16 * g + e]), s[16 * g + e + 1]);
                            t2 = fmaxf(fmaxf(t2, s[16 * g + e + 2]), s[16 * g + e + 3]);
                        }
                        top = fmaxf(top, fmaf(fmaxf(t, t2), factor(g), sc[kGrains + g]));
                    }
                    // m = -inf until the row has seen a key
                    const bool grow = top > m && (m == -INFINITY || top - m > kLazyE4);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float mn = fmaxf(m, top);
                        const float f = m == -INFINITY ? 0.0f : ex2(m - mn);
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
                    const float mc = m == -INFINITY ? 0.0f : kShiftE4 - m;
                    uint64_t sum = 0;
#pragma unroll
                    for (int k = 0; k < kTileRows / 32; ++k) {
                        uint32_t p[16];
#pragma unroll
                        for (int g = 2 * k; g < 2 * k + 2; ++g) {
                            const float cg = factor(g), bg = sc[kGrains + g] + mc, iv = sc[2 * kGrains + g];
                            const uint64_t c2 = f32x2(cg, cg), b2 = f32x2(bg, bg);
                            uint64_t part[2] = {0, 0};
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float x0, x1;
                                split2(fma2(f32x2(s[16 * g + 2 * e], s[16 * g + 2 * e + 1]), c2, b2), x0, x1);
                                const float p0 = ex2(x0), p1 = ex2(x1);
                                part[e & 1] = e < 2 ? f32x2(p0, p1) : add2(part[e & 1], f32x2(p0, p1));
                                p[8 * (g & 1) + e] = pack2<true>(p0, p1);
                            }
                            sum = fma2(add2(part[0], part[1]), f32x2(iv, iv), sum);
                        }
                        tc::st_32x32b_x16(t_s + 16 * k, p);
                    }
                    float s0, s1;
                    split2(sum, s0, s1);
                    l += s0 + s1;
                    tc::wait_st();
                }
                any = true;
                tc::fence_before_sync();
                arrive(p_full + 8 * slot);
            }
            if (!ok) break;
            tile += steps;
            if (steps > 0) qt += two ? 2 : 1;
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
                    exchange[kTileRows + row] = l;
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
                const float m1 = exchange[row], l1 = exchange[kTileRows + row];
                const float mn = fmaxf(m, m1);
                f0 = m == -INFINITY ? 0.0f : ex2(m - mn);
                f1 = m1 == -INFINITY ? 0.0f : ex2(m1 - mn);
                m = mn;
                l = l * f0 + l1 * f1;
            }
            const int c0 = it.c0, c1 = it.c1, h = it.h, token0 = it.qs + t0;
            item_done(n);
            const bool live = row < rows;
            const bool split = c0 != c1;
            float *part = part_of<D>(a, blockIdx.x, (int)blockIdx.x == c0, slot);
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
                        float *dst = part + (k / 4 * kTileRows + row) * 4;
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<float4 *>(dst + e * kTileRows * 4) =
                                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        }
                        continue;
                    }
                    // 4 x 4 transposition of 16-byte pieces over four lanes: a store
                    // then writes 64 bytes of each of eight rows
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
                if (live && a.lse) a.lse[token * a.q_heads + head] = lse_of(m, l);
                continue;
            }
            // unnormalised, for the second launch
            if (live) {
                float *dst = part + kTileRows * D + row;
                dst[0] = m;
                dst[kTileRows] = l;
            }
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && sh.abort) set_status(a.status, 4u /* MARKOV_ETIMEOUT */, sh.abort);
    if (warp == 12) tc::tmem_dealloc(tmem, 512);
}

// ----------------------------------------------------------------- joining

constexpr int kJoinThreads = 256;

// Block (b, g): 32 rows of the item that begins in block b and is cut, g = slot * 4
// + their quarter of the tile.  A thread has a row and some vectors of four columns;
// four parts' loads are in flight together.
template <int D, bool F16>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttnE4m3Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Join j = reinterpret_cast<const Join *>(a.joins)[blockIdx.x];
    const int slot = blockIdx.y >> 2, r = (blockIdx.y & 3) * 32 + (threadIdx.x & 31);
    const int tokens = min(j.tokens - slot * a.tile_tokens, a.tile_tokens);
    if (j.c0 == j.c1 || r >= tokens * a.group || __ldcg(a.status) != 0u) return;
    constexpr int kVec = D / 4 / (kJoinThreads / 32);
    const int k0 = (threadIdx.x >> 5) * kVec;
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
            const float *p = part_of<D>(a, b0 + e, b0 + e == j.c0, slot);
            pm[e] = __ldcg(p + kTileRows * D + r);
            pl[e] = __ldcg(p + kTileRows * D + kTileRows + r);
#pragma unroll
            for (int k = 0; k < kVec; ++k)
                y[e][k] = __ldcg(reinterpret_cast<const float4 *>(p + ((k0 + k) * kTileRows + r) * 4));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) mn = fmaxf(mn, pm[e]);
        const float f = M == -INFINITY ? 0.0f : ex2(M - mn);
        M = mn;
        L *= f;
#pragma unroll
        for (int k = 0; k < 4 * kVec; ++k) o[k] *= f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (b0 + e > j.c1) continue;
            const float g = pm[e] == -INFINITY ? 0.0f : ex2(pm[e] - M);
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
    if (k0 == 0 && a.lse) a.lse[token * a.q_heads + head] = lse_of(M, L);
}

template <int D, bool F16, bool ONE>
cudaError_t launch_typed(const AttnE4m3Args &a, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, int blocks,
                         cudaStream_t s) {
    attention_e4m3_kernel<D, F16, ONE><<<blocks, kManyThreads, Shape<D, ONE>::kSmem, s>>>(a, q, k, v);
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
    return cudaLaunchKernelEx(&cfg, join_kernel<D, F16>, a);
}

}  // namespace

cudaError_t launch_attention_e4m3_many(const AttnE4m3Args &a, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                                       int head_dim, bool f16, bool one, int blocks, cudaStream_t s) {
    const auto launch = head_dim == 64 ? f16 ? one ? launch_typed<64, true, true> : launch_typed<64, true, false>
                                             : one ? launch_typed<64, false, true> : launch_typed<64, false, false>
                                       : f16 ? one ? launch_typed<128, true, true> : launch_typed<128, true, false>
                                             : one ? launch_typed<128, false, true> : launch_typed<128, false, false>;
    return launch(a, q, k, v, blocks, s);
}

namespace {

template <int D, bool ONE>
cudaError_t prepare() {
    for (const void *fn : {(const void *)attention_e4m3_kernel<D, false, ONE>, (const void *)attention_e4m3_kernel<D, true, ONE>}) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D, ONE>::kSmem);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t attention_e4m3_many_prepare() {
    for (const cudaError_t e : {prepare<64, false>(), prepare<64, true>(), prepare<128, false>(), prepare<128, true>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

// Floats of the parts that `blocks` blocks may leave, bytes of their joins.
size_t attention_e4m3_many_parts(int head_dim, int blocks) { return (size_t)blocks * 4 * kTileRows * (head_dim + 2); }
size_t attention_e4m3_many_joins(int blocks) { return (size_t)blocks * sizeof(Join); }

}  // namespace dtm
