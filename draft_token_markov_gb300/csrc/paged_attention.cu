// paged_attention.cu -- attention of a chunk of new tokens over a paged
// cache on tcgen05: one persistent launch for single tokens, draft chunks
// and prompt chunks alike.
//
// Rows.  The queries of a row's tokens that share a key head are stacked,
// row = token * group + head in group, so an MMA tile of 128 rows holds
// 128 / group tokens whatever the group, and keys and values are read once
// for all of them.  An item is (request, key head, up to two such tiles); its
// keys go by in tiles of 128:
//   S = Q K^T           128 x 128, fp32 in TMEM (both operands in shared memory)
//   m, p = 2^(S c - m c), l += sum p     a thread a row, in registers
//   O += P V            P rounded to the type into S's columns of TMEM, the
//                       A operand; V as it lies in the cache (MN-major B)
// with c = scale log2 e.  Two tiles take turns on the tensor core, one in its
// MMAs while the other is in its softmax.  The maximum that p is taken
// against moves only when a row's has grown by more than 2^8 (kLazy): then O
// is rescaled in TMEM, else the sums go on, exact all the same.
//
// Work.  A unit is one key tile of an item.  The units of the call, in order
// of request, key head, tile of rows and keys, are cut into one contiguous
// range a block, whatever the lengths, so every block streams the same number
// of tiles; every block finds its range from the lengths by itself (a scan
// over the rows).  An item cut between blocks leaves its parts, O, m and l in
// fp32, in the plan's scratch, and the block that finishes last joins them in
// the order of the keys.
//
// Roles.  Warps 0-3 and 4-7: softmax and output of the two tiles; warp 8
// issues MMAs; warp 9 loads key and value tiles by TMA, a page a box (a box
// of a page that nobody sees is read out of range, as zeros); warps 10-11
// load queries.  Value rows that no row of the item sees can hold anything:
// they are zeroed in shared memory before the MMA (0 * NaN).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "paged.h"
#include "tc.cuh"

namespace dtm {

constexpr int kPaThreads = 384;
constexpr int kPaTile = 128;                 // keys of a tile, and rows
constexpr float kLazy = 8.0f;

template <int D>
struct PaShape {
    static constexpr int kQBytes = kPaTile * D * 2;          // one tile of queries
    static constexpr int kKvBytes = kPaTile * D * 2;         // one tile of keys or values
    static constexpr int kStages = D == 128 ? 5 : 12;
    static constexpr int kHalf = kPaTile * 128;              // 64 elements of every row
    static constexpr int kHalves = D / 64;
    static constexpr int kData = 2 * kQBytes + kStages * kKvBytes;
    static constexpr int kSmem = 1024 + kData + 512;
};

// ------------------------------------------------------------------- items

struct PaItem {
    int r, h, m;               // request, key head, pair of row tiles
    int rows, row0;            // rows of the item, the first within the request
    int end, first, kept;      // some row sees keys [first, end) and [0, kept)
    int sink_tiles, w0, tiles; // key tiles: [0, sink_tiles), then from w0 on
};

struct PaReq {
    int np, qs;                // tokens that there are queries for, the first
    int pos0;                  // position of its token 0
    int state;                 // its table row, -1 for none
};

__device__ __forceinline__ PaReq pa_request(const AttnArgs &a, int r) {
    PaReq q;
    const int64_t s = __ldg(a.idx + r);
    q.qs = __ldg(a.query_start + r);
    const int n = __ldg(a.query_start + r + 1) - q.qs;
    int len = __ldg(a.seq_lens + r);
    if (len < 0) len = 0;
    q.np = s < 0 || q.qs < 0 || q.qs >= a.T || n < 0 ? 0 : min(n, a.T - q.qs);
    q.pos0 = len - n;
    q.state = s < a.num_states ? (int)s : -1;
    return q;
}

// The key tiles of pair m of a request; at least one unit.
__device__ __forceinline__ int pa_tiles(const AttnArgs &a, const PaReq &q, int m, PaItem &it) {
    it.row0 = m * 2 * kPaTile;
    it.rows = min(q.np * a.group - it.row0, 2 * kPaTile);
    const int p0 = q.pos0 + it.row0 / a.group, p1 = q.pos0 + (it.row0 + it.rows - 1) / a.group;
    it.end = q.state < 0 ? 0 : max(0, min(p1 + 1, a.room));
    it.first = a.window > 0 ? max(0, p0 - a.window + 1) : 0;
    it.kept = min(min(a.sinks, it.first), it.end);
    it.w0 = it.first / kPaTile;
    const int nw = it.first < it.end ? (it.end + kPaTile - 1) / kPaTile - it.w0 : 0;
    it.sink_tiles = (it.kept + kPaTile - 1) / kPaTile;
    if (nw > 0 && it.sink_tiles > it.w0) it.sink_tiles = it.w0;
    it.tiles = it.sink_tiles + nw;
    return it.tiles > 0 ? it.tiles : 1;
}

__device__ __forceinline__ int pa_pairs(const AttnArgs &a, const PaReq &q) {
    return (q.np * a.group + 2 * kPaTile - 1) / (2 * kPaTile);
}

// Where a block's range starts, in shared memory.
struct PaStart {
    int r, h, m, j;            // first unit: request, key head, pair, key tile
    int blocks;                // blocks that have work
    int64_t u0, u1, total;     // its units, all units
};

// A block's items one after the other; every role walks them by itself.
struct PaWalk {
    PaItem it;
    PaReq q;
    int64_t u;                 // the current item's first unit
    int j0, j1;                // the range of it that is this block's
    int units, pairs;
    int64_t u_end;

    __device__ __forceinline__ void start(const AttnArgs &a, const PaStart &s) {
        it.r = s.r;
        it.h = s.h;
        it.m = s.m;
        q = pa_request(a, s.r);
        pairs = pa_pairs(a, q);
        u_end = s.u1;
        u = s.u0 - s.j;
        set(a, s.j);
    }
    __device__ __forceinline__ void set(const AttnArgs &a, int j) {
        units = pa_tiles(a, q, it.m, it);
        j0 = j;
        j1 = (int)min((int64_t)units, u_end - u);
    }
    __device__ __forceinline__ bool next(const AttnArgs &a) {
        u += units;
        if (u >= u_end) return false;
        if (++it.m == pairs) {
            it.m = 0;
            if (++it.h == a.kv_heads) {
                it.h = 0;
                do {
                    ++it.r;
                    q = pa_request(a, it.r);
                } while (q.np <= 0);
                pairs = pa_pairs(a, q);
            }
        }
        set(a, 0);
        return true;
    }
};

__device__ __forceinline__ int64_t pa_first_unit(int64_t total, int blocks, int c) {
    return total * c / blocks;
}

__device__ __forceinline__ int pa_block_of(int64_t total, int blocks, int64_t u) {
    int c = (int)(u * blocks / total);
    while (pa_first_unit(total, blocks, c + 1) <= u) ++c;
    return c;
}

// Every thread: this block's range.  scratch: 16 int64.
__device__ void pa_schedule(const AttnArgs &a, PaStart *out, int64_t *scratch) {
    constexpr int kPer = (kPagedMaxRows + kPaThreads - 1) / kPaThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t mine[kPer], sum = 0;
    PaItem it;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int r = tid * kPer + k;
        mine[k] = 0;
        if (r < a.rows) {
            const PaReq q = pa_request(a, r);
            const int pairs = pa_pairs(a, q);
            int64_t units = 0;
            for (int m = 0; m < pairs; ++m) units += pa_tiles(a, q, m, it);
            mine[k] = units * a.kv_heads;
        }
        sum += mine[k];
    }
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < kPaThreads / 32; ++w) {
        if (w < warp) incl += scratch[w];
        total += scratch[w];
    }
    const int blocks = (int)min((int64_t)gridDim.x, total);
    if (tid == 0) {
        out->total = total;
        out->blocks = blocks;
    }
    if ((int)blockIdx.x >= blocks) return;
    const int64_t u0 = pa_first_unit(total, blocks, blockIdx.x);
    int64_t before = incl - sum;
    if (u0 < before || u0 >= incl) return;
    // the thread whose rows hold the first unit
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (u0 >= before && u0 < before + mine[k]) {
            const int r = tid * kPer + k;
            const PaReq q = pa_request(a, r);
            const int64_t head = mine[k] / a.kv_heads;
            int64_t rem = u0 - before;
            const int h = (int)(rem / head);
            rem -= h * head;
            int m = 0;
            for (;; ++m) {
                const int units = pa_tiles(a, q, m, it);
                if (rem < units) break;
                rem -= units;
            }
            out->r = r;
            out->h = h;
            out->m = m;
            out->j = (int)rem;
            out->u0 = u0;
            out->u1 = pa_first_unit(total, blocks, blockIdx.x + 1);
        }
        before += mine[k];
    }
}

// ----------------------------------------------------------------- helpers

// Bounded waits: a wait that gives up records the status and raises the
// block's abort flag, and every role leaves at its next wait.
struct PaWait {
    uint64_t timeout_ns;
    uint32_t *status;
    volatile uint32_t *abort;

    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, uint32_t where) const {
        if (tc::mbar_test(bar, parity)) return true;
        return slow(bar, parity, where);
    }
    __device__ __forceinline__ bool slow(uint32_t bar, uint32_t parity, uint32_t where) const {
        const uint64_t deadline = tc::now_ns() + timeout_ns;
        while (!tc::mbar_test_sleep(bar, parity)) {
            if (*abort) return false;
            if (tc::now_ns() > deadline) {
                set_status(status, 4u /* MARKOV_ETIMEOUT */, where);
                *abort = 1u;
                return false;
            }
        }
        return true;
    }
};

// B operand, MN-major, 128-byte swizzle: 64 elements of N contiguous, the
// next 64 `lbo` bytes on; 8 rows of K 128 bytes apart, the next 8 1024 on.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t lbo) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

template <bool F16>
__host__ __device__ constexpr uint32_t pa_idesc(uint32_t N, bool mn_major_b) {
    return (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | (mn_major_b ? 1u << 16 : 0u) |
           ((N >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, int x, int y, int z,
                                            int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4, %5}], [%6];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void ld_32x32b_x32(uint32_t taddr, float *r) {
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
          "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
          "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void st_32x32b_x32(uint32_t taddr, const uint32_t *u) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]),
        "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]),
        "r"(u[17]), "r"(u[18]), "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]),
        "r"(u[25]), "r"(u[26]), "r"(u[27]), "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
        : "memory");
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (F16) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    return bf16x2_rn(lo, hi);
}

// Two fp32 values in one register pair, and the packed arithmetic on them.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split2(uint64_t x, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float pa_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------------ kernel

template <int D, bool F16>
__global__ void __launch_bounds__(kPaThreads, 1)
paged_attention_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
    using S = PaShape<D>;
    extern __shared__ uint8_t raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *q_smem = base, *kv_smem = base + 2 * S::kQBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + S::kData);
    __shared__ PaStart start_s;
    __shared__ int64_t scratch_s[16];
    __shared__ uint32_t tmem_s, abort_s, last_s[2];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t bar0 = tc::smem_u32(bars);
    const uint32_t kv_full = bar0, kv_empty = bar0 + 8 * S::kStages;
    const uint32_t q_full = bar0 + 16 * S::kStages, q_empty = q_full + 16, s_full = q_full + 32,
                   p_full = q_full + 48, pv_done = q_full + 64, group = q_full + 80, leave = q_full + 96;
    if (tid == 0) {
        abort_s = ld_acquire_u32(a.status);          // a pending status: nothing is done
        for (int i = 0; i < S::kStages; ++i) {
            tc::mbar_init(kv_full + 8 * i, 1);
            tc::mbar_init(kv_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(q_full + 8 * i, 2);       // the two loading warps
            tc::mbar_init(q_empty + 8 * i, 1);
            tc::mbar_init(s_full + 8 * i, 1);
            tc::mbar_init(p_full + 8 * i, 4);       // the tile's four warps
            tc::mbar_init(pv_done + 8 * i, 1);
            tc::mbar_init(group + 8 * i, 128);
        }
        tc::mbar_init(leave, 1);
        tc::mbar_init_fence();
    }
    if (warp == 8) tc::tmem_alloc(tc::smem_u32(&tmem_s), 512);
    pa_schedule(a, &start_s, scratch_s);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_s;
    const bool work = !abort_s && (int)blockIdx.x < start_s.blocks;
    const PaWait wait{a.timeout_ns, a.status, &abort_s};
    uint32_t filled = 0, fill_phase = 0;             // loader: stages it filled, and their phases
    // registers: 8 x 32 x 200 + 4 x 32 x 104 are the launch's 384 x 168
    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (work && warp == 9) {
        // ------------------------------------------------ key / value loads
        PaWalk w;
        w.start(a, start_s);
        const int page = 1 << a.page_shift;
        const int box = min(page, kPaTile), boxes = kPaTile / box;     // boxes of a tile
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        do {
            const PaItem &it = w.it;
            const int32_t *table = a.table + (int64_t)max(w.q.state, 0) * a.table_s0;
            const int j1 = min(w.j1, it.tiles);
            for (int j = w.j0; ok && j < j1; ++j) {
                const int key0 = (j < it.sink_tiles ? j : it.w0 + j - it.sink_tiles) * kPaTile;
                int pid = -1;
                const int key = key0 + lane * box;
                if (lane < boxes && key < it.end && (key + box > it.first || key < it.kept))
                    pid = __ldg(table + (key >> a.page_shift));
                for (int kv = 0; ok && kv < 2; ++kv) {
                    if (lane == 0) ok = wait(kv_empty + 8 * stage, phase ^ 1, 0x100 + stage);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    const uint32_t full = kv_full + 8 * stage;
                    if (lane == 0) tc::mbar_expect_tx(full, S::kKvBytes);
                    __syncwarp();
                    if (lane < boxes) {
                        const uint32_t dst = tc::smem_u32(kv_smem + stage * S::kKvBytes) + lane * box * 128;
#pragma unroll
                        for (int half = 0; half < S::kHalves; ++half)
                            tma_load_4d(dst + half * S::kHalf, kv ? &vmap : &kmap, half * 64,
                                        key & (page - 1), it.h, pid, full);
                    }
                    filled |= 1u << stage;
                    fill_phase = (fill_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == S::kStages) { stage = 0; phase ^= 1; }
                }
            }
        } while (ok && w.next(a));
    } else if (work && warp == 8) {
        // ---------------------------------------------------- MMA issue
        if (lane == 0) {
            PaWalk w;
            w.start(a, start_s);
            int stage = 0;
            uint32_t phase = 0, q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
            bool ok = true;
            const uint32_t q_addr = tc::smem_u32(q_smem), kv_addr = tc::smem_u32(kv_smem);
            constexpr uint32_t kIdescS = pa_idesc<F16>(kPaTile, false), kIdescO = pa_idesc<F16>(D, true);
            auto scores = [&](int slot, int st) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k / 4) * S::kHalf + (k % 4) * 32;
                    tc::mma_smemA(tmem + slot * kPaTile, tc::sw128_desc(q_addr + slot * S::kQBytes + off),
                                  tc::sw128_desc(kv_addr + st * S::kKvBytes + off), kIdescS, k > 0);
                }
                tc::commit(s_full + 8 * slot);
            };
            auto values = [&](int slot, int st, bool accumulate) {
#pragma unroll
                for (int k = 0; k < kPaTile / 16; ++k)
                    tc::mma_tmemA(tmem + 2 * kPaTile + slot * D, tmem + slot * kPaTile + k * 8,
                                  sw128_mn_desc(kv_addr + st * S::kKvBytes + k * 2048, S::kHalf), kIdescO,
                                  accumulate || k > 0);
                tc::commit(pv_done + 8 * slot);
            };
            do {
                const int slots = w.it.rows > kPaTile ? 2 : 1;
                const int j1 = min(w.j1, w.it.tiles);
                if (w.j0 >= j1) continue;            // nothing seen: the output is written without MMAs
                ok = wait(kv_full + 8 * stage, phase, 0x200);
                for (int s = 0; ok && s < slots; ++s) {
                    ok = wait(q_full + 8 * s, q_phase[s], 0x210 + s);
                    if (!ok) break;
                    q_phase[s] ^= 1;
                    tc::fence_after_sync();
                    scores(s, stage);
                    if (w.j0 + 1 == j1) tc::commit(q_empty + 8 * s);
                }
                if (!ok) break;
                tc::commit(kv_empty + 8 * stage);
                if (++stage == S::kStages) { stage = 0; phase ^= 1; }
                for (int j = w.j0; ok && j < j1; ++j) {
                    const int v_stage = stage;
                    const uint32_t v_phase = phase;
                    if (++stage == S::kStages) { stage = 0; phase ^= 1; }
                    const bool more = j + 1 < j1;
                    for (int s = 0; ok && s < slots; ++s) {
                        ok = wait(p_full + 8 * s, p_phase[s], 0x220 + s) &&
                             wait(kv_full + 8 * v_stage, v_phase, 0x230);
                        if (!ok) break;
                        p_phase[s] ^= 1;
                        tc::fence_after_sync();
                        values(s, v_stage, j > w.j0);
                        if (s == slots - 1) tc::commit(kv_empty + 8 * v_stage);
                        if (more) {
                            ok = wait(kv_full + 8 * stage, phase, 0x240);
                            if (!ok) break;
                            tc::fence_after_sync();
                            scores(s, stage);
                            if (j + 2 == j1) tc::commit(q_empty + 8 * s);
                        }
                    }
                    if (ok && more) {
                        tc::commit(kv_empty + 8 * stage);
                        if (++stage == S::kStages) { stage = 0; phase ^= 1; }
                    }
                }
            } while (ok && w.next(a));
        }
        __syncwarp();
    } else if (work && warp >= 10) {
        // ------------------------------------------------- query loads
        PaWalk w;
        w.start(a, start_s);
        uint32_t phase[2] = {0, 0};
        const int t = tid - 320;
        constexpr int V = D / 8;                     // 16-byte pieces of a row
        bool ok = true;
        do {
            const PaItem &it = w.it;
            if (w.j0 >= min(w.j1, it.tiles)) continue;
            for (int s = 0; ok && s * kPaTile < it.rows; ++s) {
                const int rows = min(it.rows - s * kPaTile, kPaTile);
                if (lane == 0) ok = wait(q_empty + 8 * s, phase[s] ^ 1, 0x300 + s);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                phase[s] ^= 1;
                uint8_t *dst = q_smem + s * S::kQBytes;
#pragma unroll 4
                for (int e = t; e < rows * V; e += 64) {
                    const int row = e / V, c = e % V, x = it.row0 + s * kPaTile + row;
                    const int tok = x / a.group, head = it.h * a.group + x - tok * a.group;
                    uint4 v = __ldg(reinterpret_cast<const uint4 *>(a.q + (w.q.qs + tok) * a.q_s0 +
                                                                    head * a.q_s1 + c * 8));
                    v.x ^= a.q_sign;
                    v.y ^= a.q_sign;
                    v.z ^= a.q_sign;
                    v.w ^= a.q_sign;
                    *reinterpret_cast<uint4 *>(dst + (c >> 3) * S::kHalf + row * 128 +
                                               (((c & 7) ^ (row & 7)) << 4)) = v;
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(q_full + 8 * s);
            }
        } while (ok && w.next(a));
    } else if (work) {
        // -------------------------------------------- softmax and output
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int slot = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;             // TMEM lane of the warp
        const uint32_t t_s = tmem + slot * kPaTile + lanes, t_o = tmem + 2 * kPaTile + slot * D + lanes;
        const float c = a.scale2;
        constexpr float kShift = F16 ? 7.0f : 0.0f;   // fp16 weights: up to 2^15, small ones stay normal
        PaWalk w;
        w.start(a, start_s);
        uint32_t s_phase = 0, pv_phase = 0, v_stage = 0, v_phase = 0;  // v_*: this block's next value tile
        const uint32_t kv_addr = tc::smem_u32(kv_smem);
        bool ok = true;
        // a wait that some lane gives up is given up by the warp
        auto all_wait = [&](uint32_t bar, uint32_t parity, uint32_t where) {
            return (bool)__all_sync(0xffffffffu, wait(bar, parity, where));
        };
        uint32_t group_phase = 0;
        auto group_sync = [&]() {
            tc::mbar_arrive(group + 8 * slot);
            const bool r = all_wait(group + 8 * slot, group_phase, 0x440 + slot);
            group_phase ^= 1;
            return r;
        };
        do {
            const PaItem &it = w.it;
            const int j1 = min(w.j1, it.tiles), rows = it.rows - slot * kPaTile;
            const int steps = max(0, j1 - w.j0);
            if (rows <= 0) {                          // one tile: this group has none
                const uint32_t x = v_stage + 2 * steps;
                v_phase ^= (x / S::kStages) & 1;
                v_stage = x % S::kStages;
                continue;
            }
            const int x = it.row0 + slot * kPaTile + row, tok = x / a.group;
            const int head = it.h * a.group + x - tok * a.group;
            const int pos = w.q.pos0 + tok;
            // the warp's rows: positions of the first and the last that there is
            const int wrow = slot * kPaTile + (warp & 3) * 32;
            const bool busy = wrow < it.rows;
            const int lo_pos = w.q.pos0 + (it.row0 + wrow) / a.group;
            const int hi_pos = w.q.pos0 + (it.row0 + min(wrow + 31, it.rows - 1)) / a.group;
            const int limit = min(pos + 1, a.room);
            float m = -INFINITY, l = 0.0f;
            for (int j = w.j0; j < j1; ++j) {
                const int key0 = (j < it.sink_tiles ? j : it.w0 + j - it.sink_tiles) * kPaTile;
                if (++v_stage == S::kStages) { v_stage = 0; v_phase ^= 1; }    // past the key tile
                ok = all_wait(s_full + 8 * slot, s_phase, 0x400 + slot);
                if (!ok) break;
                s_phase ^= 1;
                tc::fence_after_sync();
                if (busy) {
                    const bool whole = key0 + kPaTile <= min(lo_pos + 1, a.room) &&
                                       (a.window <= 0 || key0 > hi_pos - a.window || key0 + kPaTile <= a.sinks);
                    const int hi = limit - key0, sk = min(a.sinks - key0, hi);
                    const int lo = a.window > 0 ? pos - a.window + 1 - key0 : 0;
                    auto hide = [&](float (&s)[kPaTile]) {
#pragma unroll
                        for (int i = 0; i < kPaTile; ++i)
                            s[i] = (i < hi && i >= lo) || i < sk ? s[i] : -INFINITY;
                    };
                    float s[kPaTile], top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 4; ++k) ld_32x32b_x32(t_s + 32 * k, s + 32 * k);
                    tc::wait_ld();
                    if (!whole) hide(s);
#pragma unroll
                    for (int i = 0; i < kPaTile; i += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k) top4[k] = fmaxf(fmaxf(top4[k], s[i + 2 * k]), s[i + 2 * k + 1]);
                    const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                    // (top - m) c > kLazy; m = -inf until the row has seen a key
                    const bool grow = top > m && (m == -INFINITY || (top - m) * c > kLazy);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float mn = fmaxf(m, top);
                        const float f = m == -INFINITY ? 0.0f : pa_ex2((m - mn) * c);
                        m = mn;
                        if (j > w.j0) {
                            // the last PV is done: S's commit came after it
                            l *= f;
#pragma unroll
                            for (int k = 0; k < D / 32; ++k) {
                                float o[32];
                                ld_32x32b_x32(t_o + 32 * k, o);
                                tc::wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] *= f;
                                st_32x32b_x32(t_o + 32 * k, reinterpret_cast<const uint32_t *>(o));
                            }
                        }
                    }
                    const float mc = m == -INFINITY ? 0.0f : kShift - m * c;
                    const uint64_t c2 = f32x2(c, c), mc2 = f32x2(mc, mc);
                    uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x0, x1;
                            split2(fma2(f32x2(s[32 * k + 2 * i], s[32 * k + 2 * i + 1]), c2, mc2), x0, x1);
                            const float p0 = pa_ex2(x0), p1 = pa_ex2(x1);
                            sum[i & 3] = add2(sum[i & 3], f32x2(p0, p1));
                            p[i] = pack2<F16>(p0, p1);
                        }
                        tc::st_32x32b_x16(t_s + 16 * k, p);
                    }
                    float s0, s1;
                    split2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
                    l += s0 + s1;
                }
                // value rows that nobody sees: zeros
                const int key = key0 + row;
                if (key0 + kPaTile > it.end || (key0 < it.first && key0 + kPaTile > it.kept)) {
                    ok = all_wait(kv_full + 8 * v_stage, v_phase, 0x420 + slot);
                    if (!ok) break;
                    if (key >= it.end || (key < it.first && key >= it.kept)) {
                        const uint32_t at = kv_addr + v_stage * S::kKvBytes + row * 128;
#pragma unroll
                        for (int half = 0; half < S::kHalves; ++half)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + half * S::kHalf + 16 * i),
                                             "r"(0)
                                             : "memory");
                    }
                    tc::fence_proxy_async_smem();
                }
                if (++v_stage == S::kStages) { v_stage = 0; v_phase ^= 1; }
                if (busy) tc::wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(p_full + 8 * slot);
                pv_phase ^= 1;                        // P is on its way: one more PV to come
            }
            if (!ok) break;
            if (steps > 0) {
                ok = all_wait(pv_done + 8 * slot, pv_phase ^ 1, 0x430 + slot);
                if (!ok) break;
                tc::fence_after_sync();
            }
            const bool live = row < rows;
            const int64_t token = w.q.qs + tok;
            if (w.j0 == 0 && w.j1 == w.units) {
                // the whole item: the output
                const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
                if (live && a.lse)
                    a.lse[token * a.q_heads + head] = l == 0.0f ? -INFINITY : (m * c - kShift + __log2f(l)) * 0.69314718055994531f;
                uint16_t *out = a.out + token * a.out_s0 + head * a.out_s1;
                if (steps > 0 && busy) {
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        float o[32];
                        ld_32x32b_x32(t_o + 32 * k, o);
                        tc::wait_ld();
                        if (live) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint4 v;
                                uint32_t *u = &v.x;
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    u[e] = l == 0.0f ? 0u : pack2<F16>(o[8 * i + 2 * e] * inv, o[8 * i + 2 * e + 1] * inv);
                                *reinterpret_cast<uint4 *>(out + 32 * k + 8 * i) = v;
                            }
                        }
                    }
                } else if (live) {
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) *reinterpret_cast<uint4 *>(out + 8 * i) = make_uint4(0, 0, 0, 0);
                }
            } else {
                // a part of it: unnormalised, for the block that comes last
                const int64_t total = start_s.total;
                const int blocks = start_s.blocks;
                const int c0 = pa_block_of(total, blocks, w.u), c1 = pa_block_of(total, blocks, w.u + w.units - 1);
                auto part = [&](int block) {          // the item's first block has it as its last
                    return a.parts + ((int64_t)(block * 2 + (block == c0 ? 1 : 0)) * 2 + slot) * kPaTile * (D + 2);
                };
                float *mine = part(blockIdx.x);
                if (busy) {
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        float o[32];
                        ld_32x32b_x32(t_o + 32 * k, o);
                        tc::wait_ld();
                        if (live) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<float4 *>(mine + row * D + 32 * k + 4 * i) =
                                    make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        }
                    }
                    if (live) {
                        mine[kPaTile * D + row] = m;
                        mine[kPaTile * D + kPaTile + row] = l;
                    }
                }
                __threadfence();
                if (!(ok = group_sync())) break;
                if (row == 0) {
                    const uint32_t before = atomicAdd(a.arrivals + c0 * 2 + slot, 1u);
                    last_s[slot] = before == (uint32_t)(c1 - c0);
                    if (before == (uint32_t)(c1 - c0)) a.arrivals[c0 * 2 + slot] = 0u;
                }
                if (!(ok = group_sync())) break;
                if (last_s[slot]) {
                    __threadfence();
                    constexpr int V = D / 8;
                    const int n = min(rows, kPaTile) * V;
                    for (int e = row; e < n; e += 128) {
                        const int rr = e / V, cc = e % V;
                        float M = -INFINITY, L = 0.0f, o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = 0.0f;
#pragma unroll 4
                        for (int b = c0; b <= c1; ++b) {
                            const float *p = part(b);
                            const float pm = __ldcg(p + kPaTile * D + rr), pl = __ldcg(p + kPaTile * D + kPaTile + rr);
                            const float4 u = __ldcg(reinterpret_cast<const float4 *>(p + rr * D + cc * 8));
                            const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + rr * D + cc * 8) + 1);
                            const float mn = fmaxf(M, pm);
                            const float f = M == -INFINITY ? 0.0f : pa_ex2((M - mn) * c);
                            const float g = pm == -INFINITY ? 0.0f : pa_ex2((pm - mn) * c);
                            M = mn;
                            L = L * f + pl * g;
                            const float y[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] = o[i] * f + y[i] * g;
                        }
                        const float inv = L == 0.0f ? 0.0f : __fdiv_rn(1.0f, L);
                        const int xx = it.row0 + slot * kPaTile + rr, tt = xx / a.group;
                        const int hh = it.h * a.group + xx - tt * a.group;
                        uint4 v;
                        uint32_t *u = &v.x;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            u[i] = L == 0.0f ? 0u : pack2<F16>(o[2 * i] * inv, o[2 * i + 1] * inv);
                        *reinterpret_cast<uint4 *>(a.out + (w.q.qs + tt) * a.out_s0 + hh * a.out_s1 + cc * 8) = v;
                        if (cc == 0 && a.lse)
                            a.lse[(int64_t)(w.q.qs + tt) * a.q_heads + hh] =
                                L == 0.0f ? -INFINITY : (M * c - kShift + __log2f(L)) * 0.69314718055994531f;
                    }
                }
            }
            // O is read: the next item's values may come (its P arrives after this)
            tc::fence_before_sync();
        } while (ok && w.next(a));
    }
    __syncwarp();
    if (work && warp == 9 && lane == 0 && abort_s) {
        // gave up: no load may be in flight when the block leaves
        const uint64_t until = tc::now_ns() + a.timeout_ns;
        for (int i = 0; i < S::kStages; ++i)
            if (filled >> i & 1)
                while (!tc::mbar_test(kv_full + 8 * i, fill_phase >> i & 1) && tc::now_ns() < until) {}
    }
    if (work && warp == 8 && lane == 0 && abort_s) {
        // nor an MMA
        tc::commit(leave);
        tc::mbar_wait_for(leave, 0, a.timeout_ns);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 8) tc::tmem_dealloc(tmem, 512);
}

template <int D, bool F16>
static cudaError_t launch_typed(const AttnArgs &a, const CUtensorMap &k, const CUtensorMap &v, int blocks,
                                cudaStream_t s) {
    paged_attention_kernel<D, F16><<<blocks, kPaThreads, PaShape<D>::kSmem, s>>>(a, k, v);
    return cudaGetLastError();
}

cudaError_t launch_paged_attention(const AttnArgs &a, const CUtensorMap &k, const CUtensorMap &v,
                                   int head_dim, bool f16, int blocks, cudaStream_t s) {
    if (head_dim == 64)
        return f16 ? launch_typed<64, true>(a, k, v, blocks, s) : launch_typed<64, false>(a, k, v, blocks, s);
    return f16 ? launch_typed<128, true>(a, k, v, blocks, s) : launch_typed<128, false>(a, k, v, blocks, s);
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

}  // namespace dtm
