// paged_e4m3.cu -- the store of keys and values into a paged cache of e4m3 with a
// scale for each block of tokens and head, and reading it back.
#include <cuda_bf16.h>

#include "common.cuh"
#include "e4m3.cuh"
#include "paged.h"

namespace dtm {

// 8 elements of the plan's type as fp32.
template <bool F16>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (F16) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        } else {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

// ------------------------------------------------------------------- store
//
// A block's scale needs the largest of the call's values for it before the first
// of them is rounded, and a block that was begun by earlier calls may have to be
// rescaled: a thread block (chunk of tokens, head, side) takes the cache blocks
// whose first token of the call lies in its chunk, one after the other, with all
// of their tokens, also those past the chunk.  Where the runs of a cache block's
// tokens begin and end is found once, from the slots: a bit a token.  Where many begin
// in a chunk (single tokens of a batch) its warps take one each.
// Up to kHeld * 128 vectors of a run stay in registers between the maximum and the
// rounding, the rest is read again.  Rescaling comes before the new values, so that
// it need not know which entries they replace.  Bound by latency: slots, scale, values and
// maximum come one after the other.  8192 tokens of 8 heads of 128 (50 MB, scales of 64
// tokens) take 15 us, 50% of the copy rate and 2.2 of 4 instructions a cycle, neither at
// its limit, in two rounds of blocks; 72 tokens 3.7 us in a graph; 1000 single tokens 14.7
// us for 1 us of bytes, as a warp takes its runs in turn.  With the maximum in fp32 and
// divisions in the loop the first took 27 us.  With given scales, where every token is on
// its own, the three take 15, 1.9 and 3.4 us.
constexpr int kStoreThreads = 128;
constexpr int kHeld = 8;
constexpr int kMostChunk = 256;              // tokens of a chunk: a cache block at most

// x / s, rounded.
__device__ __noinline__ uint2 divide8(float x0, float x1, float x2, float x3, float x4, float x5, float x6, float x7, float s) {
    return make_uint2(e4m3_of_f32(__fdiv_rn(x0, s), __fdiv_rn(x1, s), __fdiv_rn(x2, s), __fdiv_rn(x3, s)),
                      e4m3_of_f32(__fdiv_rn(x4, s), __fdiv_rn(x5, s), __fdiv_rn(x6, s), __fdiv_rn(x7, s)));
}
// By its reciprocal where that is exact (s a power of two; inv is 0 elsewhere).
__device__ __forceinline__ uint2 round8(const float (&x)[8], float s, float inv) {
    if (inv == 0.0f) return divide8(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], s);
    return make_uint2(e4m3_of_f32(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                      e4m3_of_f32(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}

// 1 / s where it is exact and normal, else 0.
__device__ __forceinline__ float exact_inverse(float s) {
    const uint32_t b = __float_as_uint(s), e = b >> 23;
    return (b & 0x7fffffu) == 0u && e >= 1u && e <= 252u ? __uint_as_float((254u - e) << 23) : 0.0f;
}

// The larger magnitudes of two pairs of 16-bit floats, as their bits.
__device__ __forceinline__ uint32_t larger_magnitudes(uint32_t a, uint32_t b) {
    return __vmaxu2(a, b & 0x7fff7fffu);
}

// The run [t0, t1) of one cache block's tokens, by a block or a warp (TEAM threads).
// slot_at, place: a token's slot and its place in its cache block; begins_anew: whether
// the cache block's first place is among tokens.
template <int D, bool F16, int TEAM, class SlotAt, class Place, class Anew>
__device__ __forceinline__ void store_run(const StoreArgs &a, const StoreSide &side, int head, int t0, int t1, const SlotAt &slot_at,
                                          const Place &place, const Anew &begins_anew, uint32_t *top_s) {
    constexpr int kLanes = D / 8, kTokens = TEAM / kLanes;              // threads of a token, tokens of a turn
    const E4m3Side &c = side.cache;
    const int tid = threadIdx.x % TEAM, sub = tid / kLanes, vec = tid % kLanes;
    const auto sync = [] {
        if (TEAM == 32) __syncwarp(); else __syncthreads();
    };
    const uint4 *src = side.src + head * side.src_s1 + vec;
    const auto load = [&](int t) { return __ldcs(src + t * side.src_s0); };
    uint4 held[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        const int t = t0 + k * kTokens + sub;
        held[k] = t < t1 ? load(t) : make_uint4(0, 0, 0, 0);
    }
    const int64_t slot0 = slot_at(t0), in_page = slot0 & ((1 << a.page_shift) - 1);
    float *scale = c.scales + (slot0 >> a.page_shift) * c.ss_page + (in_page >> c.block_shift) * c.ss_block + head * c.ss_head;
    const float old = __ldcg(scale);
    const bool anew = begins_anew(t0, t1);
    // magnitudes as bits; infinities and NaN, which are the largest, do not count
    constexpr uint32_t kInfinity = F16 ? 0x7c00u : 0x7f80u;
    uint32_t top2 = 0;
    const auto look = [&](const uint4 &v) {
        top2 = larger_magnitudes(larger_magnitudes(larger_magnitudes(larger_magnitudes(top2, v.x), v.y), v.z), v.w);
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k) look(held[k]);
    for (int t = t0 + kHeld * kTokens + sub; t < t1; t += kTokens) look(load(t));
    uint32_t top = __reduce_max_sync(0xffffffffu, max(top2 & 0xffffu, top2 >> 16));
    if (top >= kInfinity) {
        top = 0;
#pragma unroll 1
        for (int t = t0 + sub; t < t1; t += kTokens) {
            const uint4 v = load(t);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = w[i] & 0x7fffu, hi = w[i] >> 16 & 0x7fffu;
                top = max(top, max(lo < kInfinity ? lo : 0u, hi < kInfinity ? hi : 0u));
            }
        }
        __syncwarp();
        top = __reduce_max_sync(0xffffffffu, top);
    }
    if (TEAM > 32) {
        if ((tid & 31) == 0) top_s[tid >> 5] = top;
        __syncthreads();                              // every thread has read the old scale
        top = top_s[0];
#pragma unroll
        for (int w = 1; w < TEAM / 32; ++w) top = max(top, top_s[w]);
    } else {
        __syncwarp();                                 // likewise: a reduction orders no memory
    }
    float s = scale_of(F16 ? __half2float(__ushort_as_half((unsigned short)top)) : __uint_as_float(top << 16));
    // the block's first entry of the head
    uint8_t *at = c.data + (slot0 >> a.page_shift) * c.s_page + head * c.s_head + (in_page >> c.block_shift << c.block_shift) * c.s_slot;
    if (!anew && usable_scale(old)) {
        if (s > old) {
            // the block's entries so far, 16 bytes a thread
            const float ratio = __fdiv_rn(old, s);
            constexpr int kVec = D / 16;
            for (int i = tid; i < kVec << c.block_shift; i += TEAM) {
                uint4 *p = reinterpret_cast<uint4 *>(at + (i / kVec) * c.s_slot + i % kVec * 16);
                uint4 v = *p;
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 lo = f32x2_of_e4m3(w[j]), hi = f32x2_of_e4m3(w[j] >> 16);
                    w[j] = e4m3_of_f32(lo.x * ratio, lo.y * ratio, hi.x * ratio, hi.y * ratio);
                }
                *p = make_uint4(w[0], w[1], w[2], w[3]);
            }
            sync();
        } else {
            s = old;
        }
    }
    const float inv = exact_inverse(s);
    at += 8 * vec;
    const auto store = [&](int t, const uint4 &v) {
        float x[8];
        unpack8<F16>(v, x);
        *reinterpret_cast<uint2 *>(at + place(t) * c.s_slot) = round8(x, s, inv);
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        const int t = t0 + k * kTokens + sub;
        if (t < t1) store(t, held[k]);
    }
    for (int t = t0 + kHeld * kTokens + sub; t < t1; t += kTokens) store(t, load(t));
    if (tid == 0) *scale = s;
    sync();                                           // top_s is free
}

// MANY: a chunk may have several runs (in us, without and with: 72 tokens, a token a
// chunk, 4.0 and 4.5; 1000 single tokens, 16 a chunk, 38 and 14).
template <int D, bool F16, bool KEEP, bool MANY>
__global__ void __launch_bounds__(kStoreThreads, 7) store_e4m3_kernel(const __grid_constant__ StoreArgs a) {
    constexpr int kLanes = D / 8, kTokens = kStoreThreads / kLanes;     // threads of a token, tokens of a turn
    const uint32_t pending = __ldcg(a.status);                          // nothing is written then
    const int tid = threadIdx.x, lane = tid & 31, sub = tid / kLanes, vec = tid % kLanes;
    const StoreSide &side = a.side[blockIdx.z];
    const E4m3Side &c = side.cache;
    const int head = blockIdx.y, t_first = blockIdx.x * a.chunk, t_last = min(t_first + a.chunk, a.T);
    const int in_block = (1 << c.block_shift) - 1;
    const int64_t in_page = (1 << a.page_shift) - 1;
    const auto slot_at = [&](int t) {
        const int64_t s = t >= 0 && t < a.T ? __ldg(a.slots + t) : -1;
        return s >= 0 && s < a.num_slots ? s : (int64_t)-1;
    };
    const auto scale_at = [&](int64_t slot) {
        return c.scales + (slot >> a.page_shift) * c.ss_page + ((slot & in_page) >> c.block_shift) * c.ss_block +
               head * c.ss_head;
    };
    if (KEEP) {
        for (int t = t_first + sub; t < t_last; t += kTokens) {
            const int64_t slot = slot_at(t);
            if (slot < 0 || pending) continue;
            const float s = __ldg(scale_at(slot));
            float x[8];
            unpack8<F16>(__ldcs(side.src + t * side.src_s0 + head * side.src_s1 + vec), x);
            uint8_t *to = c.data + (slot >> a.page_shift) * c.s_page + (slot & in_page) * c.s_slot + head * c.s_head + 8 * vec;
            *reinterpret_cast<uint2 *>(to) = round8(x, s, exact_inverse(s));
        }
        return;
    }
    // of token t_first + i: its place in its cache block, and bits: whether its block is
    // another than the token's before, whether (of the chunk) it is one of the cache's
    // with that, whether its place is the block's first
    __shared__ uint8_t place_s[2 * kMostChunk];
    __shared__ uint32_t breaks_s[kMostChunk / 16], begins_s[kMostChunk / 32], first_s[kMostChunk / 16];
    __shared__ uint32_t top_s[kStoreThreads / 32];
    // a run is a cache block's tokens at most, as a rule
    const int window = (a.chunk + in_block + 1 + 31) & ~31;
    for (int i = tid; i < window; i += kStoreThreads) {
        const int64_t s = slot_at(t_first + i);
        int64_t before = __shfl_up_sync(0xffffffffu, s, 1);
        if (lane == 0) before = slot_at(t_first + i - 1);
        const bool breaks = s < 0 || before < 0 || s >> c.block_shift != before >> c.block_shift;
        const uint32_t b = __ballot_sync(0xffffffffu, breaks), n = __ballot_sync(0xffffffffu, breaks && s >= 0),
                       f = __ballot_sync(0xffffffffu, s >= 0 && (s & in_block) == 0);
        place_s[i] = (uint8_t)(s & in_block);
        if (lane == 0) {
            breaks_s[i >> 5] = b;
            first_s[i >> 5] = f;
            if (i < a.chunk) begins_s[i >> 5] = n;
        }
    }
    __syncthreads();
    if (pending) return;
    // the first break from token i of the window on; past the window the slots are looked at
    const auto run_end = [&](int i) {
        for (; i < window; i = (i | 31) + 1) {
            const uint32_t b = breaks_s[i >> 5] >> (i & 31);
            if (b) return t_first + i + __ffs(b) - 1;
        }
        int t = t_first + window;
        const int64_t block = slot_at(t - 1) >> c.block_shift;
        for (int64_t s; t < a.T && (s = slot_at(t)) >= 0 && s >> c.block_shift == block; ++t) {}
        return t;
    };
    const auto place = [&](int t) {
        return t - t_first < window ? (int)place_s[t - t_first] : (int)(slot_at(t) & in_block);
    };
    // whether a place 0 is among tokens [t0, t1)
    const auto begins_anew = [&](int t0, int t1) {
        bool anew = false;
        for (int i = t0 - t_first; i < t1 - t_first;) {
            if (i >= window) {
                anew |= place(t_first + i++) == 0;
                continue;
            }
            const int next = min((i | 31) + 1, t1 - t_first);
            uint32_t f = first_s[i >> 5] >> (i & 31);
            if (next - i < 32) f &= (1u << (next - i)) - 1u;
            anew |= f != 0;
            i = next;
        }
        return anew;
    };
    // short runs: a warp each; long ones: the block together
    const int tokens = t_last - t_first;
    int runs = 0;
    for (int i = 0; i < tokens; i += 32) runs += __popc(begins_s[i >> 5] & (tokens - i < 32 ? (1u << (tokens - i)) - 1u : ~0u));
    const bool by_warp = MANY && runs > 1 && tokens <= 16 * runs;
    int n = 0;
    for (int i = 0; i < tokens; i = (i | 31) + 1) {
        for (uint32_t b = begins_s[i >> 5] & (tokens - i < 32 ? (1u << (tokens - i)) - 1u : ~0u); b; b &= b - 1, ++n) {
            if (by_warp && n % (kStoreThreads / 32) != tid >> 5) continue;
            const int i0 = i + __ffs(b) - 1, t0 = t_first + i0, t1 = run_end(i0 + 1);
            if (MANY && by_warp)
                store_run<D, F16, 32>(a, side, head, t0, t1, slot_at, place, begins_anew, top_s);
            else
                store_run<D, F16, kStoreThreads>(a, side, head, t0, t1, slot_at, place, begins_anew, top_s);
        }
    }
}

template <int D, bool F16>
static cudaError_t launch_store_typed(const StoreArgs &a, bool keep, cudaStream_t s) {
    const dim3 grid((a.T + a.chunk - 1) / a.chunk, a.heads, 2);
    if (keep)
        store_e4m3_kernel<D, F16, true, false><<<grid, kStoreThreads, 0, s>>>(a);
    else if (a.chunk == 1)
        store_e4m3_kernel<D, F16, false, false><<<grid, kStoreThreads, 0, s>>>(a);
    else
        store_e4m3_kernel<D, F16, false, true><<<grid, kStoreThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_store_e4m3(const StoreArgs &a, int head_dim, bool f16, bool keep, cudaStream_t s) {
    if (head_dim == 64)
        return f16 ? launch_store_typed<64, true>(a, keep, s) : launch_store_typed<64, false>(a, keep, s);
    return f16 ? launch_store_typed<128, true>(a, keep, s) : launch_store_typed<128, false>(a, keep, s);
}

// ------------------------------------------------------------------- fetch
//
// A thread block finds the slots of its tokens (a binary search over the rows, a
// thread a token), then copies their vectors of 16 bytes, each to 32.  Bound by
// memory: 16 requests of up to 8000 tokens (429 MB moved) take 74 us, 86% of the copy
// rate (77 us without the streaming hint on its stores), one of 500 tokens 3.7 us in a
// graph.
constexpr int kFetchThreads = 256;
constexpr int kFetchTokens = 32;

template <int D, bool F16>
__global__ void __launch_bounds__(kFetchThreads) fetch_e4m3_kernel(const __grid_constant__ FetchArgs a) {
    if (__ldcg(a.status) != 0u) return;
    // page * 2^32 + slot in it; kNone: zeros, kSkip: not a row's
    constexpr int64_t kNone = -1, kSkip = -2;
    __shared__ int64_t where[kFetchTokens];
    const int tid = threadIdx.x, t0 = blockIdx.x * a.tile, tokens = min(a.tile, a.r.T - t0);
    if (tid < tokens) {
        const int t = t0 + tid;
        // the last row that begins at or before t: of those with the same start the last
        // is the one that is not empty, or none is
        int lo = 0, hi = a.r.rows;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.r.query_start + mid) <= t) lo = mid; else hi = mid;
        }
        const int qs = __ldg(a.r.query_start + lo), qe = __ldg(a.r.query_start + lo + 1);
        const int64_t state = __ldg(a.r.idx + lo);
        int64_t at = kSkip;
        if (t >= qs && t < qe && state >= 0) {
            const int64_t pos = (int64_t)max(__ldg(a.r.seq_lens + lo), 0) - (qe - qs) + (t - qs);
            at = kNone;
            if (pos >= 0 && pos < a.r.room && state < a.r.num_states) {
                const int page = __ldg(a.r.table + state * a.r.table_s0 + (pos >> a.r.page_shift));
                if (page >= 0 && page < a.r.num_pages) at = (int64_t)page << 32 | (pos & ((1 << a.r.page_shift) - 1));
            }
        }
        where[tid] = at;
    }
    __syncthreads();
    constexpr int kVec = D / 16;
    const int n = tokens * a.heads * kVec;
#pragma unroll 2
    for (int i = tid; i < n; i += kFetchThreads) {
        const int th = i / kVec, v = i % kVec, t = th / a.heads, h = th - t * a.heads;
        const int64_t at = where[t];
        if (at == kSkip) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const E4m3Side &c = a.side[k];
            uint4 x = make_uint4(0, 0, 0, 0);
            float s = 0.0f;
            if (at != kNone) {
                const int64_t page = at >> 32, slot = at & 0xffffffff;
                x = __ldcs(reinterpret_cast<const uint4 *>(c.data + page * c.s_page + slot * c.s_slot + h * c.s_head + 16 * v));
                s = __ldg(c.scales + page * c.ss_page + (slot >> c.block_shift) * c.ss_block + h * c.ss_head);
            }
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            uint32_t y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = f32x2_of_e4m3(j & 1 ? w[j >> 1] >> 16 : w[j >> 1]);
                if (F16)
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y[j]) : "f"(f.y * s), "f"(f.x * s));
                else
                    y[j] = bf16x2_rn(f.x * s, f.y * s);
            }
            uint4 *to = a.dst[k] + (int64_t)(t0 + t) * a.dst_s0[k] + h * a.dst_s1[k] + 2 * v;
            __stcs(to, make_uint4(y[0], y[1], y[2], y[3]));
            __stcs(to + 1, make_uint4(y[4], y[5], y[6], y[7]));
        }
    }
}

template <int D, bool F16>
static cudaError_t launch_fetch_typed(const FetchArgs &a, cudaStream_t s) {
    fetch_e4m3_kernel<D, F16><<<(a.r.T + a.tile - 1) / a.tile, kFetchThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_fetch_e4m3(const FetchArgs &a, int head_dim, bool f16, cudaStream_t s) {
    if (head_dim == 64) return f16 ? launch_fetch_typed<64, true>(a, s) : launch_fetch_typed<64, false>(a, s);
    return f16 ? launch_fetch_typed<128, true>(a, s) : launch_fetch_typed<128, false>(a, s);
}

}  // namespace dtm
