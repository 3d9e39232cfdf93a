// verify.cu -- acceptance of drafts against the target's logits.
//
// Two launches.  The first reads every logit once: its warps take segments of
// a position's row (target or draft) and leave each one's maximum m and
// z = sum exp((l - m) / T).  The second, a programmatic dependent of the first,
// joins a request's partials in every one of its blocks (at most 33 rows of
// 32), walks the drafts, and takes the argmax of the residual's key over its
// ids of one position: one target row, one draft row, much of them still in
// L2, and the request's noise.  That, the drafts and their logits do not wait
// for the first launch.  (Joined in the first launch instead, by the warp that
// came last, the fences at each segment's end took longer than its loads: 129
// against 46 us for 64 requests of 8 drafts.)
//
// exp((l - m) / T) is ex2((l - m) * c) with c = log2(e) / T: l - m is exact
// or rounded once, and an overflow of l / T cannot make it NaN.
#include <climits>

#include "common.cuh"
#include "f32x2.cuh"
#include "paged.h"
#include "tc.cuh"

namespace dtm {

constexpr int kVerifyThreads = 256;
constexpr int kSegment = 1024;             // ids; a multiple of a warp's turn

// log2(e) / T, finite (a T so small that it overflows is the limit T -> 0) and
// not 0 (T = inf: any difference of two finite logits times the least subnormal
// is 0 in 2^x, and -inf, of masked ids and of those past the end, stays -inf
// where 0 * -inf would be NaN).
__device__ __forceinline__ float inv_temperature(float T) {
    return fmaxf(fminf(__fdiv_rn(1.4426950408889634f, T), 3.0e38f), 1.401298464e-45f);
}

// 8 consecutive logits as fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void *row, int64_t at, float (&x)[8]) {
    if (F32) {
        const float4 u = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(row) + at));
        const float4 w = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(row) + at) + 1);
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
    } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + at));
        const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(r[j] << 16);
            x[2 * j + 1] = __uint_as_float(r[j] & 0xffff0000u);
        }
    }
}

template <bool F32>
__device__ __forceinline__ float load1(const void *row, int64_t at) {
    if (F32) return __ldg(static_cast<const float *>(row) + at);
    return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(row) + at) << 16);
}

// A block's maximum key; every thread gets it.
__device__ __forceinline__ uint64_t block_max(uint64_t x, uint64_t *shared) {
    x = tc::warp_max_u64(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = x;
    __syncthreads();
    x = shared[threadIdx.x & (kVerifyThreads / 32 - 1)];
    return tc::warp_max_u64(x);
}

// The segment's best (logit, id) in the argmax order, whatever it holds; by
// one warp.
template <bool F32>
__device__ __noinline__ uint64_t segment_key(const void *row, int64_t base, int lo, int hi) {
    uint64_t best = 0;
    for (int v = lo + (threadIdx.x & 31) * 8; v < hi; v += 256) {
        float x[8];
        load8<F32>(row, base + v, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint64_t k = pack_key(x[j], (uint32_t)(v + j));
            best = k > best ? k : best;
        }
    }
    return tc::warp_max_u64(best);
}

// 8 consecutive logits as they lie, and their maximum (NaN if one is).
template <bool F32>
struct Raw8 {
    uint4 v[F32 ? 2 : 1];

    // -inf where there are none
    __device__ __forceinline__ void load(const void *row, int64_t at, bool there) {
        constexpr uint32_t kNone = F32 ? 0xff800000u : 0xff80ff80u;
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(row) + at * (F32 ? 4 : 2));
#pragma unroll
        for (int k = 0; k < (F32 ? 2 : 1); ++k) v[k] = there ? __ldg(p + k) : make_uint4(kNone, kNone, kNone, kNone);
    }
    // word j: ids 2 j and 2 j + 1 of BF16 logits, id j of fp32 ones
    __device__ __forceinline__ uint32_t word(int j) const {
        const uint4 &u = v[j >> 2];
        return (j & 3) == 0 ? u.x : (j & 3) == 1 ? u.y : (j & 3) == 2 ? u.z : u.w;
    }
    __device__ __forceinline__ void pair(int j, float &lo, float &hi) const {
        if (F32) {
            lo = __uint_as_float(word(2 * j));
            hi = __uint_as_float(word(2 * j + 1));
        } else {
            lo = __uint_as_float(word(j) << 16);
            hi = __uint_as_float(word(j) & 0xffff0000u);
        }
    }
};

// Running maximum of words (two BF16 values or an fp32 one); NaN wins.
template <bool F32>
__device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t b) {
    uint32_t r;
    if (F32)
        asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A thread's part of a segment: the maximum, the sum against it and, for a
// greedy row, the turn in which the maximum came.
struct Running {
    float m, z;
    int at;
};

// vectors of 8 ids that a lane takes a turn: 64 bytes, the next 64 meanwhile
template <bool F32>
constexpr int kTurnVectors = F32 ? 2 : 4;

// One turn's vectors, the first from id v on.  Some four instructions an id
// for a sampled row; a greedy one needs the maxima alone.  A NaN stays in z.
template <bool F32>
__device__ __forceinline__ void take_turn(const Raw8<F32> (&x)[kTurnVectors<F32>], int v, bool sampled, float c, Running &s) {
    constexpr int kWords = F32 ? 8 : 4;
    uint32_t w = x[0].word(0);
#pragma unroll
    for (int k = 0; k < kTurnVectors<F32>; ++k)
#pragma unroll
        for (int j = 0; j < kWords; ++j) w = word_max<F32>(w, x[k].word(j));
    float top = __uint_as_float(F32 ? w : w << 16);
    if (!F32) top = __uint_as_float(word_max<true>(__float_as_uint(top), w & 0xffff0000u));
    if (top != top) s.z = NAN;
    if (top > s.m) {
        if (s.m != -INFINITY) s.z *= ex2((s.m - top) * c);
        s.m = top;
        s.at = v;
    }
    if (!sampled) return;
    const float ref = s.m == -INFINITY ? 0.0f : s.m;
    const uint64_t neg = f32x2(-ref, -ref), c2 = f32x2(c, c);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < kTurnVectors<F32>; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float e0, e1;
            x[k].pair(j, e0, e1);
            split2(mul2(add2(f32x2(e0, e1), neg), c2), e0, e1);
            sum[j & 1] = add2(sum[j & 1], f32x2(ex2(e0), ex2(e1)));
        }
    float s0, s1;
    split2(add2(sum[0], sum[1]), s0, s1);
    s.z += s0 + s1;
}

// A segment's partial from its lanes': m, z and the key.  For a sampled row the
// key says only whether the maximum is finite, and where it is if it is not.
template <bool F32>
__device__ void end_segment(const void *row, int64_t base, int lo, int hi, bool sampled, float c, const Running &s,
                            uint4 *out) {
    float m = s.m, z = s.z;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (s.m != -INFINITY) z *= ex2((s.m - m) * c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    uint64_t key = pack_key(m, (uint32_t)lo);
    if (z != z || m == INFINITY || z == INFINITY) {
        key = segment_key<F32>(row, base, lo, hi);
    } else if (!sampled && m != -INFINITY) {
        // the lowest id of the maximum, among the ids of its turn
        Raw8<F32> x[kTurnVectors<F32>];
#pragma unroll
        for (int k = 0; k < kTurnVectors<F32>; ++k) x[k].load(row, base + s.at + k * 256, s.at + k * 256 < hi);
        int id = INT_MAX;
#pragma unroll
        for (int k = kTurnVectors<F32> - 1; k >= 0; --k)
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                float e0, e1;
                x[k].pair(j, e0, e1);
                if (e1 == m) id = s.at + k * 256 + 2 * j + 1;
                if (e0 == m) id = s.at + k * 256 + 2 * j;
            }
        key = tc::warp_max_u64(s.m == m ? pack_key(m, (uint32_t)id) : 0ull);
    }
    if ((threadIdx.x & 31) == 0)
        __stcg(out, make_uint4(__float_as_uint(m), __float_as_uint(z), (uint32_t)key, (uint32_t)(key >> 32)));
}

// A position's distribution: exp((l - m) / T) * inv_z, or one-hot at `id`.
struct Dist {
    float m, inv_z;
    int id;                    // -1: not one-hot
};

__device__ __forceinline__ float prob(const Dist &d, float l, int v, float c) {
    if (d.id >= 0) return v == d.id ? 1.0f : 0.0f;
    // rounded: p - q is 0 where the two are equal, not a fused product's rest
    return __fmul_rn(ex2((l - d.m) * c), d.inv_z);
}

// One segment: ids [lo, hi) of a row that starts at element `base`.
template <bool F32>
__device__ __forceinline__ void take_segment(const void *row, int64_t base, int lo, int hi, bool sampled, float c,
                                             uint4 *out) {
    const int lane8 = (threadIdx.x & 31) * 8;
    Running s{-INFINITY, 0.0f, lo + lane8};
    constexpr int kV = kTurnVectors<F32>, kTurn = kV * 256;
    Raw8<F32> x[kV], y[kV];
    auto load = [&](int v, Raw8<F32> (&x)[kV]) {
#pragma unroll
        for (int k = 0; k < kV; ++k) x[k].load(row, base + v + k * 256, v + k * 256 < hi);
    };
    // two turns a round, each loaded while the other is taken
    load(lo + lane8, x);
#pragma unroll 1
    for (int v = lo + lane8; v - lane8 < hi; v += 2 * kTurn) {
        const bool second = v - lane8 + kTurn < hi;
        if (second) load(v + kTurn, y);
        take_turn<F32>(x, v, sampled, c, s);
        if (!second) break;
        if (v - lane8 + 2 * kTurn < hi) load(v + 2 * kTurn, x);
        take_turn<F32>(y, v + kTurn, sampled, c, s);
    }
    end_segment<F32>(row, base, lo, hi, sampled, c, s, out);
}

// The segments of the call, row = request * (2 N + 1) + position, are dealt to
// the warps in turn; a warp's loads pause only between two of them, and the
// 32 warps of a multiprocessor do so at different times.  Bound by memory: 246
// MB (64 requests of 8 drafts, V = 129280, an eighth of them padding) in 44.6 us
// (5.5 TB/s); the warps' ends lie 16 us apart, as they have five to eight
// segments, those of padding rows, which cost nothing, among them.  fp32 logits
// and caches: 492 MB in 77.6 us (6.3 TB/s).  With one of each type both forms are in
// the loop and spill some registers: 76.5 us for the 362 MB of a BF16 target and
// an fp32 cache.  (Taken from a counter instead, asked for a segment
// ahead, the whole call took 66.7 us against 61.7 us.)
template <bool TF32, bool CF32>
__global__ void __launch_bounds__(kVerifyThreads, 4) verify_stats_kernel(VerifyArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (__ldcg(a.status) != 0u) return;
    const int per = 2 * a.N + 1;
    const int tasks = a.rows * per * a.segs, warps = gridDim.x * (kVerifyThreads / 32);
#pragma unroll 1
    for (int task = blockIdx.x * (kVerifyThreads / 32) + (threadIdx.x >> 5); task < tasks; task += warps) {
        const int row = task / a.segs, b = row / per, i = row - b * per;
        if (a.idx[b] < 0) continue;
        const int lo = (task - row * a.segs) * a.seg_len, hi = min(a.V, lo + a.seg_len);
        const float T = a.temperature[b];
        const bool sampled = samples(T);
        const float c = sampled ? inv_temperature(T) : 0.0f;
        const bool draft = i > a.N;
        const void *from = draft ? a.cache : a.target;
        const int64_t base = draft ? b * a.cache_s0 + (i - a.N - 1) * a.cache_s1 : b * a.target_s0 + i * a.target_s1;
        if (TF32 == CF32)
            take_segment<TF32>(from, base, lo, hi, sampled, c, a.part + task);
        else if (draft)
            take_segment<CF32>(from, base, lo, hi, sampled, c, a.part + task);
        else
            take_segment<TF32>(from, base, lo, hi, sampled, c, a.part + task);
    }
}

// What the pick has to know of a request: its distributions at the position it
// draws, and that position.
struct Verdict {
    Dist p, q;
    int n;
};

// The drafts and their probabilities, kept for the outputs.
struct Drafts {
    int64_t x[kMaxSteps];
    float p[kMaxSteps], q[kMaxSteps];
};

// A thread's draft, and its logits; what does not wait for the first launch.
struct Draft {
    int64_t x;
    float lp, lq, u;
};

template <bool TF32, bool CF32>
__device__ __forceinline__ Draft load_draft(const VerifyArgs &a, int b) {
    Draft d{-1, 0.0f, 0.0f, 0.0f};
    const int i = threadIdx.x;
    if (i < a.N) {
        d.x = a.draft[b * a.draft_s0 + i];
        d.u = a.uniforms[b * a.uni_s0 + i];
        if (d.x >= 0 && d.x < a.V) {
            d.lp = load1<TF32>(a.target, b * a.target_s0 + i * a.target_s1 + d.x);
            d.lq = load1<CF32>(a.cache, b * a.cache_s0 + i * a.cache_s1 + d.x);
        }
    }
    return d;
}

// By a whole block: the request's distributions from their partials, the walk
// over its drafts.
__device__ __forceinline__ Verdict walk(const VerifyArgs &a, int b, float T, const Draft &d, Drafts &drafts) {
    constexpr int kWarps = kVerifyThreads / 32, kTurns = (2 * kMaxSteps + 1 + kWarps - 1) / kWarps;
    __shared__ Dist dist[2 * kMaxSteps + 1];
    __shared__ uint32_t accepted_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.N, per = 2 * N + 1;
    const float c = samples(T) ? inv_temperature(T) : 0.0f;
    // a warp a position in turn, a lane a segment
    uint4 part[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        part[k] = make_uint4(0xff800000u, 0u, 0u, 0u);
        if (warp + k * kWarps < per && lane < a.segs)
            part[k] = __ldcg(a.part + ((int64_t)b * per + warp + k * kWarps) * a.segs + lane);
    }
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        if (warp + k * kWarps >= per) break;
        const float m = __uint_as_float(part[k].x);
        float M = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float Z = m == -INFINITY ? 0.0f : __uint_as_float(part[k].y) * ex2((m - M) * c);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) Z += __shfl_xor_sync(0xffffffffu, Z, o);
        const uint64_t key = tc::warp_max_u64(((uint64_t)part[k].w << 32) | part[k].z);
        if (lane == 0) {
            const uint32_t o = packed_ordered(key);
            const bool finite = o != 0xffffffffu && isfinite(key_from_ordered(o));
            dist[warp + k * kWarps] = Dist{M, 1.0f / Z, samples(T) && finite ? -1 : (int)packed_id(key)};
        }
    }
    __syncthreads();
    if (warp == 0) {
        float p = 0.0f, q = 0.0f;
        if (d.x >= 0 && d.x < a.V) {
            p = prob(dist[lane], d.lp, (int)d.x, c);
            q = prob(dist[N + 1 + lane], d.lq, (int)d.x, c);
        }
        // the drafts before the first refusal
        const uint32_t refused = __ballot_sync(0xffffffffu, !(lane < N && d.u * q < p));
        if (lane == 0) accepted_s = __ffs(refused) - 1;
        if (lane < N) {
            drafts.x[lane] = d.x;
            drafts.p[lane] = p;
            drafts.q[lane] = q;
        }
    }
    __syncthreads();
    const int n = (int)accepted_s;
    return Verdict{dist[n], dist[n < N ? N + 1 + n : n], n};
}

// Block (g, b): ids [g pick_len, (g + 1) pick_len) of request b.  At the size
// above, 17 us of the call: some 3 us until it starts, 2.4 us for the joined
// partials and the walk, 8 us for its ids (43 MB of logits and noise, in part
// from L2); the rest is not attributed.  The block that ends last writes all
// outputs, so that tokens may lie where the drafts do: every block has read
// those by then.
template <bool TF32, bool CF32>
__global__ void __launch_bounds__(kVerifyThreads) verify_pick_kernel(VerifyArgs a) {
    __shared__ uint64_t key_s[kVerifyThreads / 32];
    __shared__ uint32_t last_s;
    __shared__ Drafts drafts;
    const int b = blockIdx.y, N = a.N, tid = threadIdx.x;
    const bool padding = a.idx[b] < 0;
    const float T = a.temperature[b];
    const float c = samples(T) ? inv_temperature(T) : 0.0f;
    const float *noise = a.noise + b * a.noise_s0;
    const int lo = blockIdx.x * a.pick_len, hi = min(a.V, lo + a.pick_len);
    Raw8<true> first;
    first.load(noise, lo + tid * 8, !padding && samples(T) && lo + tid * 8 < hi);
    Draft d{-1, 0.0f, 0.0f, 0.0f};
    if (!padding) d = load_draft<TF32, CF32>(a, b);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (padding || __ldcg(a.status) != 0u) return;
    const Verdict verdict = walk(a, b, T, d, drafts);
    const int n = verdict.n;
    const Dist P = verdict.p, Q = verdict.q;
    const int64_t t_base = b * a.target_s0 + n * a.target_s1, c_base = b * a.cache_s0 + n * a.cache_s1;

    // The best key over [lo, hi): of ln(p - q) + g, or of ln p + g with whole.
    // The fast logarithm (within 1e-4 here) tells which few ids, near the
    // warp's best, need the exact one.
    auto best_of = [&](int lo, int hi, bool whole, bool again) {
        constexpr int kStep = kVerifyThreads * 8;
        uint64_t best = 0;
        float near = -INFINITY;
        Raw8<TF32> x;
        Raw8<CF32> y;
        Raw8<true> g;
        auto load = [&](int v, bool noise_too) {
            x.load(a.target, t_base + v, v < hi);
            y.load(a.cache, c_base + v, !whole && v < hi);
            if (noise_too) g.load(noise, v, v < hi);
        };
        g = first;
        load(lo + tid * 8, again);
#pragma unroll 1
        for (int v0 = lo; v0 < hi; v0 += kStep) {
            const int v = v0 + tid * 8;
            float key[8], r[8], z[8], top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float p0, p1, q0, q1;
                x.pair(j, p0, p1);
                y.pair(j, q0, q1);
                g.pair(j, z[2 * j], z[2 * j + 1]);
                r[2 * j] = prob(P, p0, v + 2 * j, c);
                r[2 * j + 1] = prob(P, p1, v + 2 * j + 1, c);
                if (!whole) {
                    r[2 * j] -= prob(Q, q0, v + 2 * j, c);
                    r[2 * j + 1] -= prob(Q, q1, v + 2 * j + 1, c);
                }
            }
            if (v0 + kStep < hi) load(v + kStep, true);        // the next ones on their way
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                r[j] = v < hi ? fmaxf(r[j], 0.0f) : 0.0f;
                key[j] = __logf(r[j]) + z[j];
                top = fmaxf(top, key[j]);
            }
            const uint32_t warp_top = __reduce_max_sync(0xffffffffu, ordered_key(top));
            near = fmaxf(near, key_from_ordered(warp_top) - 1e-3f);
            if (top >= near) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (r[j] > 0.0f && key[j] >= near) {
                        const uint64_t k = pack_key(logf(r[j]) + z[j], (uint32_t)(v + j));
                        best = k > best ? k : best;
                    }
            }
        }
        return block_max(best, key_s);
    };
    // where p is one-hot there is nothing to draw
    const uint64_t best = P.id < 0 ? best_of(lo, hi, n == N, false) : 0;
    __shared__ uint64_t win_s;
    if (tid == 0) {
        if (best) atomicMax(reinterpret_cast<unsigned long long *>(a.win + b), (unsigned long long)best);
        __threadfence();
        const bool last = atomicAdd(a.arrivals + b, 1u) == gridDim.x - 1;
        last_s = last;
        if (last) {
            __threadfence();
            win_s = ld_cg_u64(a.win + b);
            a.win[b] = 0;
            a.arrivals[b] = 0;
        }
    }
    __syncthreads();
    if (!last_s) return;
    int token = P.id;
    if (token < 0) {
        uint64_t win = win_s;
        if (win == 0) win = best_of(0, a.V, true, true);   // p <= q everywhere
        token = win ? packed_id(win) : 0;
    }
    if (tid < N && a.p) {
        a.p[(int64_t)b * N + tid] = drafts.p[tid];
        a.q[(int64_t)b * N + tid] = drafts.q[tid];
    }
    if (tid == 0) a.accepted[b] = n;
    if (tid <= N) a.tokens[b * a.tok_s0 + tid] = tid < n ? drafts.x[tid] : tid == n ? token : -1;
}

template <bool TF32, bool CF32>
static cudaError_t launch_verify_typed(const VerifyArgs &a, cudaStream_t s) {
    verify_stats_kernel<TF32, CF32><<<a.stat_blocks, kVerifyThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(a.pick_segs, a.rows);
    return cudaLaunchKernelEx(&cfg, verify_pick_kernel<TF32, CF32>, a);
}

cudaError_t launch_verify(VerifyArgs a, bool target_f32, bool cache_f32, int sms, cudaStream_t s) {
    // segments of whole turns, at most kVerifyMaxSegs segments a row; as many blocks as
    // there is room for
    const int turns = (a.V + kSegment - 1) / kSegment;
    a.seg_len = (turns + kVerifyMaxSegs - 1) / kVerifyMaxSegs * kSegment;
    a.segs = (a.V + a.seg_len - 1) / a.seg_len;
    const int64_t tasks = (int64_t)a.rows * (2 * a.N + 1) * a.segs, warps = kVerifyThreads / 32;
    a.stat_blocks = (int)((tasks + warps - 1) / warps < 4 * sms ? (tasks + warps - 1) / warps : 4 * sms);
    // the pick: blocks for one wave, a vector of 8 ids a thread at least
    const int round = kVerifyThreads * 8, most = (a.V + round - 1) / round;
    int n = 4 * sms / a.rows;
    if (n < 1) n = 1;
    if (n > most) n = most;
    a.pick_len = ((a.V + n - 1) / n + 7) / 8 * 8;
    a.pick_segs = (a.V + a.pick_len - 1) / a.pick_len;
    if (target_f32)
        return cache_f32 ? launch_verify_typed<true, true>(a, s) : launch_verify_typed<true, false>(a, s);
    return cache_f32 ? launch_verify_typed<false, true>(a, s) : launch_verify_typed<false, false>(a, s);
}

}  // namespace dtm
