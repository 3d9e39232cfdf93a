// paged_e4m3_few.cu -- attention of few query rows a request (single tokens of a
// batch, short drafts) over a paged e4m3 cache: bound by the cache's bytes.
//
// A warp is a worker of its own: it has a range of the call's work, a ring of
// shared memory that TMA fills with 32 keys and values at a time, and the running
// softmax of the item it is at.  An item is (request, key head, 16 stacked query
// rows: row = token * group + head, or 8 where a request has no more).
//   S = Q K^T    m16n8k16 on fp16: four tiles of 8 keys, dims in any order as Q's
//   m, p = 2^(y - m), y = S ks c + log2 vs, l += 2^(-log2 vs) sum p
//   O += P V     the scores' registers are P's fragment
// The scale of a value enters its weight, as an addition in the exponent, and is
// taken out of the sum again; m is the maximum of y, which is what bounds p.  So a
// block's scales cost a few instructions for half a step's 16 keys.  Keys and values go
// from shared memory to registers once and become fp16 there (exact: e4m3 is a
// subset); values in pairs of keys by byte permutes.  (Through tcgen05 they would be
// written to shared memory as fp16 and read from there: 7 bytes of its traffic for each
// of the cache, more than it has to give at the memory's rate; 64 requests with 16 rows
// take 87 us that way and 72 here.)
//
// The maximum that p is taken against moves when a row's grows by more than 2^8
// (kLazyE4), so that most steps need no exchange between lanes; weights are at most
// 2^(kShiftE4 + kLazyE4) = 2^15.
//
// Work.  An item weighs one for each of its steps of 32 keys and kEnds for its
// start and end.  Neighbouring warps have neighbouring key heads (as many as the
// largest power of two up to 8 that divides their number) of the same keys, whose
// bytes lie side by side in a cache with the heads inside a slot: such a lane of
// heads has the items of the call end to end, in order of request, group of heads and
// rows, cut into ranges of equal weight, one a warp.  A cut item leaves its parts in
// the plan's scratch, which a second launch joins.
//
// Bounds.  64 single tokens over 500 to 32000 keys (64 / 8 heads of 128, 0.91 GB) take
// 150 us, 90% of the copy rate; 163 us with a head's warps on keys of their own, 231 us
// with lines of 256 bytes, which fetch a neighbouring head's too.  One row's token over
// 1000 keys takes 11.4 us in a graph: the start, four steps, the join; over 16000 31 us.  With 16 rows the
// arithmetic counts: 32 requests of two tokens with 8 heads each 68 us for 37 us of
// bytes.  8 warps of 250 registers and steps of 32 keys; 12 warps of 168 and steps of 16
// took 186 us where these took 166.
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

constexpr int kFewWarps = 8;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kStep = 32;                    // keys of a step, in two halves of 16
constexpr int kStepShift = 5;
// an item's start and end, in steps, and the least units of a range.  One row's token and
// the 64 of above in us: 2 and 2 12.2 and 150.3; 3 and 3 14.5 and 151.1; 3 and 1 12.6 and
// 150.9; 1 and 1 12.9 and 155.2
constexpr int kEnds = 2;
constexpr int kLeast = 2;
// What a part costs the join, in a warp's steps: a range has sqrt(kPartCost * an item's
// units) or more, where steps and joins cost the same.  0 and 0.25: a row's token over
// 16000 keys (8 key heads) 39 and 31 us, 32 requests of 500-8000 keys with 16 rows (one
// key head) 31 and 23 us, calls whose ranges are longer anyway the same.
constexpr float kPartCost = 0.25f;

template <int D>
struct FewShape {
    static constexpr int kSide = kStep * D;                  // bytes of a step's keys or values
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kRing = 2 * kSide * kStages;        // of a warp
    static constexpr int kBars = kFewWarps * kRing;
    static constexpr int kAborts = kBars + 8 * kFewWarps * kStages;
    static constexpr int kSmem = kAborts + 4 * kFewWarps;
};

struct FewItem {
    int qs, head0;             // the request's first token, the group's first query head
    int row0, rows;            // its stacked rows
    int pos0, state, h;
    KeySpan keys;
};

struct FewJoin {
    int c0, c1;                // workers that share the item, every `step`-th (c0 == c1: none)
    int step;
    int qs, head0, row0, rows;
};

// A warp's part of an item: 16 rows of D columns, then m and l of each.
template <int D>
__device__ __forceinline__ float *few_part(const AttnE4m3Args &a, int worker, bool begins) {
    return a.parts + (int64_t)(worker * 2 + (begins ? 1 : 0)) * 16 * (D + 2);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// The scores of dim steps: Q's fragments of rows g and g + 8, and each row's
// factor on its scores.
template <int D, bool F16, bool HALF>
struct FewQueries {
    uint32_t lo[D / 16][2], hi[HALF ? 1 : D / 16][2];
    float c[2];

    __device__ __forceinline__ void load_row(const AttnE4m3Args &a, const FewItem &it, int r, uint32_t (*to)[2], float &c) {
        const int lane = threadIdx.x & 31, q = lane & 3;
        uint4 v[D / 32];
        const bool there = r < it.rows;
        if (there) {
            const int row = it.row0 + r, tok = row / a.group, head = it.head0 + row - tok * a.group;
            const uint16_t *p = a.q + (int64_t)(it.qs + tok) * a.q_s0 + head * a.q_s1 + q * (D / 4);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
        } else {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) v[i] = make_uint4(0, 0, 0, 0);
        }
        const uint32_t *w = reinterpret_cast<const uint32_t *>(v);
        if (F16) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) to[i / 2][i % 2] = w[i];
            c = a.scale2;
        } else {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int k = row_exponent(top);
            const float power = power_of_two(k);
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                to[i / 2][i % 2] = pack2<true>(__uint_as_float(w[i] << 16) * power, __uint_as_float(w[i] & 0xffff0000u) * power);
            c = a.scale2 * power_of_two(-k);
        }
    }
    __device__ __forceinline__ void load(const AttnE4m3Args &a, const FewItem &it) {
        const int g = (threadIdx.x & 31) >> 2;
        load_row(a, it, g, lo, c[0]);
        if (!HALF) load_row(a, it, g + 8, hi, c[1]);
    }
};

template <int D, bool F16, bool HALF>
__global__ void __launch_bounds__(kFewThreads, 1)
attention_e4m3_few_kernel(const __grid_constant__ AttnE4m3Args a, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap) {
    using S = FewShape<D>;
    constexpr int kRows = HALF ? 8 : 16, kHalves = HALF ? 1 : 2, kSteps = D / 16, kTiles = D / 8;
    extern __shared__ __align__(1024) uint8_t base[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint32_t *abort_s = reinterpret_cast<uint32_t *>(base + S::kAborts);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    const uint32_t ring = tc::smem_u32(base) + warp * S::kRing, bars = tc::smem_u32(base + S::kBars) + 8 * warp * S::kStages;
    if (lane == 0) {
        abort_s[warp] = 0;
        for (int i = 0; i < S::kStages; ++i) tc::mbar_init(bars + 8 * i, 1);
        tc::mbar_init_fence();
    }
    __syncwarp();
    const uint32_t pending = __ldcg(a.status);
    const int lanes = min(a.kv_heads & -a.kv_heads, kFewWarps), head_groups = a.kv_heads / lanes;
    // ranges go round the blocks, so that a small call is spread
    const int range = warp / lanes * gridDim.x + blockIdx.x, head_lane = warp % lanes;
    const int worker = range * lanes + head_lane, ranges = gridDim.x * (kFewWarps / lanes);

    // ---------------------------------------------------------- the range
    const auto span = [&](const RowOfCall &r, int m) {
        const int last = min((int64_t)(m + 1) * kRows, (int64_t)r.np * a.group) - 1;
        return key_span<kStepShift>(a.r, a.window, a.sinks, r.state, r.pos0 + m * kRows / a.group, r.pos0 + last / a.group);
    };
    const auto tiles_of = [&](const RowOfCall &r) { return (r.np * a.group + kRows - 1) / kRows; };
    const auto units_of = [&](const RowOfCall &r) {          // of one key head
        uint64_t x = 0;
        const int n = tiles_of(r);
#pragma unroll 1
        for (int m = 0; m < n; ++m) x += kEnds + max(span(r, m).steps, 1);
        return x;
    };
    FewJoin join{0, 0, 0, 0, 0, 0, 0};
    uint64_t total = 0;
    uint32_t items = 0;                                      // of one key head
#pragma unroll 1
    for (int r0 = 0; r0 < a.r.rows; r0 += 32) {
        uint64_t x = 0;
        uint32_t n = 0;
        if (r0 + lane < a.r.rows) {
            const RowOfCall mine = row_of_call(a.r, r0 + lane);
            x = units_of(mine);
            n = tiles_of(mine);
        }
        items += __reduce_add_sync(0xffffffffu, n);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        total += x;
    }
    if (total * a.kv_heads >> 33) {                          // 2^31 tiles of 128 keys
        if (tid == 0 && !pending) set_status(a.status, 2u /* MARKOV_EUNSUPPORTED */, 0x700);
        total = 0;
    }
    // the parts of an item are joined one after the other: few of them where it is long
    const float mean = (float)total / (float)max(items, 1u);
    const uint32_t least = max(kLeast, (int)sqrtf(mean * kPartCost));
    UnitSplit split;
    split.cut(pending ? 0 : total * head_groups, ranges, least);
    if (range >= split.ranges) {
        if (lane == 0) reinterpret_cast<FewJoin *>(a.joins)[worker] = join;
        return;
    }
    const uint64_t u0 = split.first(range), u_end = split.first(range + 1);
    uint64_t u = 0;                                          // the current item's first unit
    int r = 0;
    RowOfCall row;
#pragma unroll 1
    for (int r0 = 0;; r0 += 32) {
        RowOfCall mine{0, 0, 0, -1};
        if (r0 + lane < a.r.rows) mine = row_of_call(a.r, r0 + lane);
        const uint64_t own = units_of(mine) * head_groups;
        uint64_t incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        incl += u;
        const uint32_t found = __ballot_sync(0xffffffffu, u0 < incl && u0 >= incl - own);
        if (found) {
            const int at = __ffs(found) - 1;
            r = r0 + at;
            u = __shfl_sync(0xffffffffu, incl - own, at);
            row.np = __shfl_sync(0xffffffffu, mine.np, at);
            row.qs = __shfl_sync(0xffffffffu, mine.qs, at);
            row.pos0 = __shfl_sync(0xffffffffu, mine.pos0, at);
            row.state = __shfl_sync(0xffffffffu, mine.state, at);
            break;
        }
        u = __shfl_sync(0xffffffffu, incl, 31);
    }
    int tiles = tiles_of(row), m = 0, hg;                    // hg: group of key heads
    {
        const uint64_t head = units_of(row);
        hg = (int)((u0 - u) / head);
        u += hg * head;
#pragma unroll 1
        for (;; ++m) {
            const uint32_t units = kEnds + max(span(row, m).steps, 1);
            if (u0 - u < units) break;
            u += units;
        }
    }

    // -------------------------------------------------------------- items
    // the next stages to load and to use, the latter's phase, and how many so far
    uint32_t fill = 0, use = 0, use_phase = 0, loaded = 0, used = 0;
    bool ok = true;
    // the step of an offset within an item's units
    const auto step_at = [&](uint64_t off, int all) { return off <= kEnds ? 0 : (int)min(off - kEnds, (uint64_t)all); };
#pragma unroll 1
    while (ok && u < u_end) {
        const int h = hg * lanes + head_lane;
        FewItem it;
        it.qs = row.qs;
        it.head0 = h * a.group;
        it.row0 = m * kRows;
        it.rows = min(row.np * a.group - it.row0, kRows);
        it.pos0 = row.pos0;
        it.state = row.state;
        it.h = h;
        it.keys = span(row, m);
        const int all = max(it.keys.steps, 1);
        const uint32_t units = kEnds + all;
        const int j0 = u0 > u ? step_at(u0 - u, all) : 0, j1 = u_end - u < units ? step_at(u_end - u, all) : all;
        if (j0 < j1) {
            const int steps = min(j1, it.keys.steps);        // its share: steps [j0, steps)
            int c0 = range, c1 = range;
            if (j0 > 0 || j1 < all) {
                c0 = split.range_of(u + kEnds);              // the range that has the first step's unit
                c1 = split.range_of(u + units - 1);
            }
            // page and scales of 16 steps, a lane a half, and of the next 16
            int pid = -1, pid_next = -1;
            float ks = 1.0f, lv = 0.0f, ks_next = 1.0f, lv_next = 0.0f;
            const bool pairs = a.r.page_shift >= kStepShift;         // a step's keys lie in one page
            const auto seen = [&](int key, int n) {
                return key < it.keys.end && (key + n > it.keys.first || key < it.keys.kept);
            };
            const auto look = [&](int j, int &pid, float &ks, float &lv) {
                pid = -1;
                ks = 1.0f;
                lv = 0.0f;
                j += lane >> 1;
                if (j >= steps) return;
                const int key0 = it.keys.key<kStepShift>(j), key = key0 + 16 * (lane & 1);
                if (!(pairs || seen(key, 16))) return;
                const int id = __ldg(a.r.table + it.state * a.r.table_s0 + (key0 + (pairs ? 0 : 16 * (lane & 1)) >> a.r.page_shift));
                if (id < 0 || id >= a.r.num_pages) return;
                pid = id;
                if (!seen(key, 16)) return;
                const int slot = key & ((1 << a.r.page_shift) - 1);
                ks = __ldg(a.ks.p + id * a.ks.s_page + (slot >> a.ks.block_shift) * a.ks.s_block + h * a.ks.s_head);
                lv = scale_log2(__ldg(a.vs.p + id * a.vs.s_page + (slot >> a.vs.block_shift) * a.vs.s_block + h * a.vs.s_head));
            };
            look(j0, pid, ks, lv);
            look(j0 + 16, pid_next, ks_next, lv_next);
            int jb = j0;                                     // the step of lane 0
            int issued = j0;
            const auto issue = [&]() {
                const int off = 2 * (issued - jb);
                const int ids = off < 32 ? pid : pid_next;
                const int id0 = __shfl_sync(0xffffffffu, ids, off & 31), id1 = __shfl_sync(0xffffffffu, ids, off + 1 & 31);
                if (lane == 0) {
                    const uint32_t bar = bars + 8 * fill, dst = ring + fill * 2 * S::kSide;
                    const int slot = it.keys.key<kStepShift>(issued) & ((1 << a.r.page_shift) - 1);
                    tc::mbar_expect_tx(bar, 2 * S::kSide);
                    tma_load_4d(dst, &kmap, 0, slot, h, id0, bar);
                    tma_load_4d(dst + S::kSide, &vmap, 0, slot, h, id0, bar);
                    if (!pairs) {
                        tma_load_4d(dst + S::kSide / 2, &kmap, 0, slot, h, id1, bar);
                        tma_load_4d(dst + S::kSide + S::kSide / 2, &vmap, 0, slot, h, id1, bar);
                    }
                }
                if (++fill == S::kStages) fill = 0;
                ++loaded;
                ++issued;
                __syncwarp();
            };
#pragma unroll 1
            for (int i = 0; i < S::kStages && issued < steps; ++i) issue();
            FewQueries<D, F16, HALF> qf;
            qf.load(a, it);
            float o[kTiles][4], M[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < kTiles; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
            // positions of the lane's rows; rows that are not there take the last one's
            int pos[kHalves];
#pragma unroll
            for (int x = 0; x < kHalves; ++x)
                pos[x] = it.pos0 + (it.row0 + min(g + 8 * x, it.rows - 1)) / a.group;
            // a step is seen whole by every row before whole_end and from whole_first on
            const int whole_end = min(it.pos0 + it.row0 / a.group + 1, a.r.room);
            const int whole_first = window_start(a.window, it.pos0 + (it.row0 + it.rows - 1) / a.group);
#pragma unroll 1
            for (int j = j0; j < steps; ++j) {
                if (j - jb == 16) {
                    jb = j;
                    pid = pid_next;
                    ks = ks_next;
                    lv = lv_next;
                    look(j + 16, pid_next, ks_next, lv_next);
                }
                float ks_j[2], lv_j[2];
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    ks_j[f] = __shfl_sync(0xffffffffu, ks, 2 * (j - jb) + f);
                    lv_j[f] = __shfl_sync(0xffffffffu, lv, 2 * (j - jb) + f);
                }
                const uint32_t bar = bars + 8 * use;
                if (!__all_sync(0xffffffffu, tc::mbar_test(bar, use_phase)))
                    ok = __all_sync(0xffffffffu, tc::mbar_wait_or_abort(bar, use_phase, 0x710, a.timeout_ns, abort_s + warp));
                if (!ok) break;
                const uint32_t kst = ring + use * 2 * S::kSide, vst = kst + S::kSide;
                if (++use == S::kStages) {
                    use = 0;
                    use_phase ^= 1;
                }
                ++used;
                const int key0 = it.keys.key<kStepShift>(j);
                // ------------------------------------------------ S = Q K^T
                float sc[4][4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
                    uint4 w[D / 64];
#pragma unroll
                    for (int i = 0; i < D / 64; ++i)
                        w[i] = D == 128 ? lds128(kst + n * 1024 + g * 128 + (((2 * q + i) ^ g) << 4))
                                        : lds128(kst + n * 512 + g * 64 + ((q ^ (g >> 1)) << 4));
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        const uint4 &x = w[s / 4];
                        uint32_t b0, b1;
                        f16x4_of_e4m3((s & 3) == 0 ? x.x : (s & 3) == 1 ? x.y : (s & 3) == 2 ? x.z : x.w, b0, b1);
                        mma_f16(sc[n], qf.lo[s][0], HALF ? 0u : qf.hi[HALF ? 0 : s][0], qf.lo[s][1],
                                HALF ? 0u : qf.hi[HALF ? 0 : s][1], b0, b1);
                    }
                }
                // ---------------------------------------------------- values
                // of each half, word w of four keys' dims: keys 2 q, 2 q + 1, 2 q + 8, 2 q + 9
                uint32_t v[2][4][kTiles / 4];
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const uint32_t at = vst + f * (S::kSide / 2);
                    if (D == 128) {
                        const uint32_t even = at + q * 256 + ((g ^ (2 * q)) << 4), odd = at + q * 256 + 128 + ((g ^ (2 * q + 1)) << 4);
                        *reinterpret_cast<uint4 *>(v[f][0]) = lds128(even);
                        *reinterpret_cast<uint4 *>(v[f][1]) = lds128(odd);
                        *reinterpret_cast<uint4 *>(v[f][2]) = lds128(even + 1024);
                        *reinterpret_cast<uint4 *>(v[f][3]) = lds128(odd + 1024);
                    } else {
                        const uint32_t even = at + q * 128 + (((g >> 1) ^ q) << 4) + (g & 1) * 8;
                        *reinterpret_cast<uint2 *>(v[f][0]) = lds64(even);
                        *reinterpret_cast<uint2 *>(v[f][1]) = lds64(even + 64);
                        *reinterpret_cast<uint2 *>(v[f][2]) = lds64(even + 512);
                        *reinterpret_cast<uint2 *>(v[f][3]) = lds64(even + 576);
                    }
                }
                __syncwarp();                                // the stage is read
                if (issued < steps) issue();
                // --------------------------------------------------- softmax
                float y[kHalves][8];
#pragma unroll
                for (int x = 0; x < kHalves; ++x)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const float c = qf.c[x] * ks_j[f];
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[x][4 * f + e] = fmaf(sc[2 * f + (e >> 1)][2 * x + (e & 1)], c, lv_j[f]);
                    }
                if (key0 + kStep > whole_end || (key0 < whole_first && key0 + kStep > a.sinks)) {
                    // values that nobody sees can be anything: zeros
                    const int end = it.keys.end, first = it.keys.first, kept = it.keys.kept;
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = key0 + 16 * f + (e >> 1) * 8 + 2 * q + (e & 1);
                            if (k >= end || (k < first && k >= kept)) {
#pragma unroll
                                for (int i = 0; i < kTiles / 4; ++i) v[f][e][i] = 0;
                            }
#pragma unroll
                            for (int x = 0; x < kHalves; ++x) {
                                const bool sees = k <= pos[x] && k < a.r.room && (k >= window_start(a.window, pos[x]) || k < a.sinks);
                                if (!sees) y[x][4 * f + e] = -INFINITY;
                            }
                        }
                }
                bool grow = false;
                float top[kHalves];
#pragma unroll
                for (int x = 0; x < kHalves; ++x) {
                    top[x] = fmaxf(fmaxf(fmaxf(y[x][0], y[x][1]), fmaxf(y[x][2], y[x][3])),
                                   fmaxf(fmaxf(y[x][4], y[x][5]), fmaxf(y[x][6], y[x][7])));
                    grow |= top[x] > M[x] + kLazyE4;
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int x = 0; x < kHalves; ++x) {
                        float most = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
                        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                        if (most > M[x]) {
                            const float f = M[x] == -INFINITY ? 0.0f : ex2(M[x] - most);
                            M[x] = most;
                            l[x] *= f;
#pragma unroll
                            for (int i = 0; i < kTiles; ++i) {
                                o[i][2 * x] *= f;
                                o[i][2 * x + 1] *= f;
                            }
                        }
                    }
                }
                uint32_t p[2][4];
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const float iv = ex2(-lv_j[f]);
                    p[f][1] = p[f][3] = 0;
#pragma unroll
                    for (int x = 0; x < kHalves; ++x) {
                        const float b = M[x] == -INFINITY ? 0.0f : kShiftE4 - M[x];
                        const float p0 = ex2(y[x][4 * f] + b), p1 = ex2(y[x][4 * f + 1] + b), p2 = ex2(y[x][4 * f + 2] + b),
                                    p3 = ex2(y[x][4 * f + 3] + b);
                        l[x] = fmaf((p0 + p1) + (p2 + p3), iv, l[x]);
                        p[f][x] = pack2<true>(p0, p1);
                        p[f][2 + x] = pack2<true>(p2, p3);
                    }
                }
                // ------------------------------------------------ O += P V
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int i = 0; i < kTiles / 4; ++i) {
                        uint32_t b[4], d[4];
                        f16x4_of_e4m3(__byte_perm(v[f][0][i], v[f][1][i], 0x5140), b[0], b[1]);
                        f16x4_of_e4m3(__byte_perm(v[f][0][i], v[f][1][i], 0x7362), b[2], b[3]);
                        f16x4_of_e4m3(__byte_perm(v[f][2][i], v[f][3][i], 0x5140), d[0], d[1]);
                        f16x4_of_e4m3(__byte_perm(v[f][2][i], v[f][3][i], 0x7362), d[2], d[3]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) mma_f16(o[4 * i + e], p[f][0], p[f][1], p[f][2], p[f][3], b[e], d[e]);
                    }
            }
            if (!ok) break;
            // ------------------------------------------------------- the end
            const bool split_item = c0 != c1;
            if (split_item && c0 == range)
                join = FewJoin{worker, c1 * lanes + head_lane, lanes, it.qs, it.head0, it.row0, it.rows};
#pragma unroll
            for (int x = 0; x < kHalves; ++x) {
                float sum = l[x];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                const int rr = g + 8 * x;
                if (rr >= it.rows) continue;
                // the lane's columns: D / 4 from q D / 4 on, the tiles' even columns first
                if (split_item) {
                    float *part = few_part<D>(a, worker, c0 == range);
                    float4 *to = reinterpret_cast<float4 *>(part + rr * D + q * (D / 4));
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const int t = i * 4 % kTiles, e = 2 * x + i * 4 / kTiles;
                        to[i] = make_float4(o[t][e], o[t + 1][e], o[t + 2][e], o[t + 3][e]);
                    }
                    if (q == 0) {
                        part[16 * D + rr] = M[x];
                        part[16 * D + 16 + rr] = sum;
                    }
                    continue;
                }
                const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
                const int sr = it.row0 + rr, tok = sr / a.group, head = it.head0 + sr - tok * a.group;
                const int64_t token = it.qs + tok;
                uint4 *to = reinterpret_cast<uint4 *>(a.out + token * a.out_s0 + head * a.out_s1 + q * (D / 4));
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int col = 8 * i + 2 * k, t = col % kTiles, e = 2 * x + col / kTiles;
                        w[k] = sum == 0.0f ? 0u : pack2<F16>(o[t][e] * inv, o[t + 1][e] * inv);
                    }
                    to[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (q == 0 && a.lse)
                    a.lse[token * a.q_heads + head] = sum == 0.0f ? -INFINITY : (M[x] - kShiftE4 + __log2f(sum)) * 0.69314718055994531f;
            }
        }
        u += units;
        if (++m == tiles) {
            m = 0;
            if (++hg == head_groups) {
                hg = 0;
                if (u < u_end) {
                    do {
                        row = row_of_call(a.r, ++r);
                    } while (row.np <= 0);
                    tiles = tiles_of(row);
                }
            }
        }
    }
    if (lane == 0) reinterpret_cast<FewJoin *>(a.joins)[worker] = join;
    if (!ok && lane == 0) {
        // gave up: no load may be in flight when the block leaves
        set_status(a.status, 4u /* MARKOV_ETIMEOUT */, abort_s[warp]);
        const uint64_t until = tc::now_ns() + a.timeout_ns;
        for (; used != loaded; ++used) {
            while (!tc::mbar_test(bars + 8 * use, use_phase) && tc::now_ns() < until) {}
            if (++use == S::kStages) {
                use = 0;
                use_phase ^= 1;
            }
        }
    }
}

// ----------------------------------------------------------------- joining

constexpr int kFewJoinParts = 8;             // loads in flight

// Block w: the item that begins in worker w's range and is cut; a thread has four
// columns of a row.  Latency, of its loads kFewJoinParts at a time: a request of 16000
// keys may have 50 parts (sixteen at a time take one row's token over them in 29.4 us for
// 30.8, but 32 rows' in 57.7 for 56.5; four at a time and 128 threads took 40 us of a call
// of 8 requests).  Blocks for 32 columns each cost one row's token 2 us: most have nothing
// to do.
template <int D, bool F16, int ROWS>
__global__ void __launch_bounds__(ROWS * D / 4) few_join_kernel(const __grid_constant__ AttnE4m3Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const FewJoin j = reinterpret_cast<const FewJoin *>(a.joins)[blockIdx.x];
    if (j.c0 == j.c1 || __ldcg(a.status) != 0u) return;
    const int r = threadIdx.x / (D / 4), k = threadIdx.x % (D / 4);
    if (r >= j.rows) return;
    float M = -INFINITY, L = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int b0 = j.c0; b0 <= j.c1; b0 += kFewJoinParts * j.step) {
        float pm[kFewJoinParts], pl[kFewJoinParts], mn = M;
        float4 y[kFewJoinParts];
#pragma unroll
        for (int e = 0; e < kFewJoinParts; ++e) {
            pm[e] = -INFINITY;
            pl[e] = 0.0f;
            const int b = b0 + e * j.step;
            if (b > j.c1) continue;
            const float *p = few_part<D>(a, b, b == j.c0);
            pm[e] = __ldcg(p + 16 * D + r);
            pl[e] = __ldcg(p + 16 * D + 16 + r);
            y[e] = __ldcg(reinterpret_cast<const float4 *>(p + r * D) + k);
        }
#pragma unroll
        for (int e = 0; e < kFewJoinParts; ++e) mn = fmaxf(mn, pm[e]);
        const float f = M == -INFINITY ? 0.0f : ex2(M - mn);
        M = mn;
        L *= f;
        o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
        for (int e = 0; e < kFewJoinParts; ++e) {
            if (pm[e] == -INFINITY) continue;
            const float w = ex2(pm[e] - M);
            L = fmaf(pl[e], w, L);
            o = make_float4(fmaf(y[e].x, w, o.x), fmaf(y[e].y, w, o.y), fmaf(y[e].z, w, o.z), fmaf(y[e].w, w, o.w));
        }
    }
    const float inv = L == 0.0f ? 0.0f : __fdiv_rn(1.0f, L);
    const int sr = j.row0 + r, tok = sr / a.group, head = j.head0 + sr - tok * a.group;
    const int64_t token = j.qs + tok;
    uint2 v = make_uint2(pack2<F16>(o.x * inv, o.y * inv), pack2<F16>(o.z * inv, o.w * inv));
    if (L == 0.0f) v = make_uint2(0u, 0u);
    *reinterpret_cast<uint2 *>(a.out + token * a.out_s0 + head * a.out_s1 + 4 * k) = v;
    if (k == 0 && a.lse)
        a.lse[token * a.q_heads + head] = L == 0.0f ? -INFINITY : (M - kShiftE4 + __log2f(L)) * 0.69314718055994531f;
}

template <int D, bool F16, bool HALF>
static cudaError_t launch_few_typed(const AttnE4m3Args &a, const CUtensorMap &k, const CUtensorMap &v, int blocks, cudaStream_t s) {
    attention_e4m3_few_kernel<D, F16, HALF><<<blocks, kFewThreads, FewShape<D>::kSmem, s>>>(a, k, v);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks * kFewWarps);
    constexpr int kRows = HALF ? 8 : 16;
    cfg.blockDim = dim3(kRows * D / 4);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, few_join_kernel<D, F16, kRows>, a);
}

template <int D>
static cudaError_t launch_few(const AttnE4m3Args &a, const CUtensorMap &k, const CUtensorMap &v, bool f16, bool half, int blocks,
                              cudaStream_t s) {
    if (f16)
        return half ? launch_few_typed<D, true, true>(a, k, v, blocks, s) : launch_few_typed<D, true, false>(a, k, v, blocks, s);
    return half ? launch_few_typed<D, false, true>(a, k, v, blocks, s) : launch_few_typed<D, false, false>(a, k, v, blocks, s);
}

cudaError_t launch_attention_e4m3_few(const AttnE4m3Args &a, const CUtensorMap &k, const CUtensorMap &v, int head_dim, bool f16,
                                      bool half, int blocks, cudaStream_t s) {
    return head_dim == 64 ? launch_few<64>(a, k, v, f16, half, blocks, s) : launch_few<128>(a, k, v, f16, half, blocks, s);
}

template <int D>
static cudaError_t prepare_few() {
    for (const void *fn : {(const void *)attention_e4m3_few_kernel<D, false, false>, (const void *)attention_e4m3_few_kernel<D, false, true>,
                           (const void *)attention_e4m3_few_kernel<D, true, false>, (const void *)attention_e4m3_few_kernel<D, true, true>}) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, FewShape<D>::kSmem);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t attention_e4m3_few_prepare() {
    const cudaError_t e = prepare_few<64>();
    return e == cudaSuccess ? prepare_few<128>() : e;
}

// Floats of the parts that `blocks` blocks may leave, bytes of their joins.
size_t attention_e4m3_few_parts(int head_dim, int blocks) { return (size_t)blocks * kFewWarps * 2 * 16 * (head_dim + 2); }
size_t attention_e4m3_few_joins(int blocks) { return (size_t)blocks * kFewWarps * sizeof(FewJoin); }

}  // namespace dtm
