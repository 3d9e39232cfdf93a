// paged_layout.cu -- room for new tokens in a paged key/value cache (page
// tables, slots, positions from request lengths) and the store of their keys
// and values.
#include "paged.h"
#include "common.cuh"

namespace dtm {

// ------------------------------------------------------------------ layout
//
// Row b needs n_b = ceil((c_b + q_b) / page) pages and holds h_b.  With
// G_b, S_b, Q_b the prefix sums over rows of max(n - h, 0), max(h - n, 0) and
// q, the e-th page taken in the call is ring[head + e] and belongs to the row
// with G_b <= e < G_{b+1}, the e-th page returned goes to ring[head + count +
// e], and token t belongs to the row with Q_b <= t < Q_{b+1}.  So every block
// scans the rows for itself (at most one row a thread: a few loads and
// shuffles), and then pages and tokens are independent: each is found by a
// binary search over a prefix sum in shared memory, strided over the grid, so
// one long prompt among many short rows costs no more than its share.
//
// In place: positions of the ring and the tables that a call writes are
// disjoint from those it reads.  The held counts and the ring's state are
// read by every block, so the block that arrives last writes them: no block
// waits for another.
//
// Bound by latency (the scan, a search, two dependent loads): 3.3 us for 8 rows
// of 9 tokens, 6.2 us for 256 rows of which one has 8192 tokens, in a graph.

template <int THREADS>
__device__ __forceinline__ void block_scan3(int64_t (&x)[3], int64_t *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x[k], o);
            if (lane >= o) x[k] += y;
        }
        if (lane == 31) warp_sums[k * 32 + warp] = x[k];
    }
    __syncthreads();
    if (warp < 3) {
        int64_t w = lane < THREADS / 32 ? warp_sums[warp * 32 + lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        warp_sums[warp * 32 + lane] = w;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (warp > 0) x[k] += warp_sums[k * 32 + warp - 1];
}

// The first of n rows whose inclusive prefix sum exceeds e.
__device__ __forceinline__ int row_of(const int64_t *incl, int n, int64_t e) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (incl[mid] > e) hi = mid; else lo = mid + 1;
    }
    return lo;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) paged_layout_kernel(LayoutArgs a) {
    __shared__ int64_t grown[THREADS], shrunk[THREADS], queried[THREADS], warp_sums[96];
    __shared__ int32_t ctx[THREADS], held[THREADS], need[THREADS], state[THREADS];
    __shared__ int taken_s;
    __shared__ uint32_t last_s;
    const int tid = threadIdx.x;
    if (__ldcg(a.status) != 0u) return;
    if (tid == 0) taken_s = 0;

    const int64_t C = a.ring_size;
    int64_t head = a.free_in[0], count = a.free_in[1];
    if (head < 0 || head >= C) head = 0;
    count = count < 0 ? 0 : count > C ? C : count;

    int64_t x[3] = {0, 0, 0};
    int c = 0, n = 0, h = 0, s = -1, q = 0;
    if (tid < a.rows) {
        c = a.context[tid];
        q = a.query[tid];
        const int64_t si = a.idx[tid];
        if (si >= 0 && si < a.num_states && c >= 0 && q >= 0 && (int64_t)c + q <= a.room) {
            h = a.held[si];
            n = (int)(((int64_t)c + q + (1 << a.page_shift) - 1) >> a.page_shift);
            if (h >= 0 && h <= a.width) {
                s = (int)si;
                x[0] = n > h ? n - h : 0;
                x[1] = h > n ? h - n : 0;
            }
        }
        x[2] = q > 0 ? q : 0;
    }
    block_scan3<THREADS>(x, warp_sums);
    // short of pages: this row and every later one that needs some
    if (s >= 0 && n > h) {
        if (x[0] <= count) atomicMax(&taken_s, (int)x[0]); else s = -1;
    }
    grown[tid] = x[0];
    shrunk[tid] = x[1];
    queried[tid] = x[2];
    ctx[tid] = c;
    held[tid] = h;
    need[tid] = n;
    state[tid] = s;
    __syncthreads();
    const int64_t taken = taken_s, returned = shrunk[a.rows - 1];

    if (blockIdx.x == 0 && tid < a.rows) {
        const int64_t qs = x[2] > INT32_MAX ? INT32_MAX : x[2];
        if (tid == 0) a.query_start[0] = 0;
        a.query_start[tid + 1] = (int32_t)qs;
        a.seq_lens[tid] = s >= 0 ? c + q : 0;
    }
    const int64_t first = (int64_t)blockIdx.x * THREADS + tid, step = (int64_t)gridDim.x * THREADS;
    for (int64_t e = first; e < taken; e += step) {
        const int b = row_of(grown, a.rows, e);
        int64_t at = head + e;
        if (at >= C) at -= C;
        const int64_t k = e - (grown[b] - (need[b] - held[b])) + held[b];
        a.table[state[b] * a.table_s0 + k] = a.ring[at];
    }
    for (int64_t e = first; e < returned; e += step) {
        const int b = row_of(shrunk, a.rows, e);
        int64_t at = head + count + e;
        while (at >= C) at -= C;
        const int64_t k = e - (shrunk[b] - (held[b] - need[b])) + need[b];
        a.ring[at] = a.table[state[b] * a.table_s0 + k];
    }
    const int64_t total = queried[a.rows - 1];
    for (int64_t t = first; t < a.T; t += step) {
        int pos = 0;
        int64_t slot = -1;
        if (t < total) {
            const int b = row_of(queried, a.rows, t);
            if (state[b] >= 0) {
                pos = ctx[b] + (int)(t - (b > 0 ? queried[b - 1] : 0));
                const int k = pos >> a.page_shift;
                int page;
                if (k < held[b]) {
                    page = a.table[state[b] * a.table_s0 + k];
                } else {
                    int64_t at = head + grown[b] - (need[b] - held[b]) + (k - held[b]);
                    if (at >= C) at -= C;
                    page = a.ring[at];
                }
                slot = ((int64_t)page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
            }
        }
        a.positions[t] = pos;
        a.slots[t] = slot;
    }

    if (gridDim.x > 1) {
        __syncthreads();       // every read of the held counts is done
        if (tid == 0) {
            __threadfence();
            const uint32_t before = atomicAdd(a.arrivals, 1u);
            last_s = before == gridDim.x - 1;
            if (last_s) *a.arrivals = 0u;
        }
        __syncthreads();
        if (!last_s) return;
    }
    if (tid < a.rows && s >= 0) a.held_out[s] = n;
    if (tid == 0) {
        int64_t nh = head + taken;
        if (nh >= C) nh -= C;
        int64_t nc = count - taken + returned;
        a.free_out[0] = nh;
        a.free_out[1] = nc > C ? C : nc;
    }
}

cudaError_t launch_paged_layout(const LayoutArgs &a, cudaStream_t s) {
    const int threads = a.rows <= 256 ? 256 : 1024;
    // a block per two tokens a thread: the scan that each block repeats is a
    // few microseconds, the tokens' two loads overlap within a thread
    int64_t blocks = ((int64_t)a.T + 2 * threads - 1) / (2 * threads);
    if (blocks < 1) blocks = 1;
    if (blocks > 128) blocks = 128;
    if (threads == 256)
        paged_layout_kernel<256><<<(int)blocks, 256, 0, s>>>(a);
    else
        paged_layout_kernel<1024><<<(int)blocks, 1024, 0, s>>>(a);
    return cudaGetLastError();
}

// ------------------------------------------------------------------- write
//
// A copy of 16-byte vectors; bound by memory (or, for a draft step's tokens,
// by the launch).  A thread moves two vectors of the keys and the same two of
// the values, a grid's width apart: four loads are in flight from it.  8192
// tokens of 8 heads of 128 (67 MB moved) take 14.4 us, 16.4 us with one vector
// of each; 72 tokens 1.9 us in a graph.  At 52 registers a thread four blocks
// fit a multiprocessor, so that those 2048 blocks are 3.4 rounds.

constexpr int kWriteThreads = 256;

__global__ void __launch_bounds__(kWriteThreads) paged_write_kernel(WriteArgs a) {
    if (__ldcg(a.status) != 0u) return;
    const int64_t total = ((int64_t)a.T * a.heads) << a.vec_shift;
    const int64_t step = (int64_t)gridDim.x * kWriteThreads;
    for (int64_t i0 = (int64_t)blockIdx.x * kWriteThreads + threadIdx.x; i0 < total; i0 += 2 * step) {
        uint4 k[2], v[2];
        int64_t slot[2] = {-1, -1};
        uint32_t h[2];
        int d[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int64_t i = i0 + e * step;
            if (i >= total) break;
            const uint32_t th = (uint32_t)(i >> a.vec_shift), t = th / (uint32_t)a.heads;
            d[e] = (int)(i & ((1 << a.vec_shift) - 1));
            h[e] = th - t * (uint32_t)a.heads;
            slot[e] = __ldg(a.slots + t);
            k[e] = __ldcs(a.k.src + t * a.k.src_s0 + h[e] * a.k.src_s1 + d[e]);
            v[e] = __ldcs(a.v.src + t * a.v.src_s0 + h[e] * a.v.src_s1 + d[e]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (slot[e] < 0 || slot[e] >= a.num_slots) continue;
            const int64_t page = slot[e] >> a.page_shift, at = slot[e] & ((1 << a.page_shift) - 1);
            a.k.dst[page * a.k.s_page + at * a.k.s_slot + h[e] * a.k.s_head + d[e]] = k[e];
            a.v.dst[page * a.v.s_page + at * a.v.s_slot + h[e] * a.v.s_head + d[e]] = v[e];
        }
    }
}

cudaError_t launch_paged_write(const WriteArgs &a, cudaStream_t s) {
    const int64_t total = ((int64_t)a.T * a.heads) << a.vec_shift;
    int64_t blocks = (total + 2 * kWriteThreads - 1) / (2 * kWriteThreads);
    if (blocks > 65535) blocks = 65535;
    paged_write_kernel<<<(int)blocks, kWriteThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace dtm
