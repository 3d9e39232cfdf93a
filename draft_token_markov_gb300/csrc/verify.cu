// verify.cu -- acceptance of drafts against the target's logits.
//
// Two launches.  The first reads every logit once: a block takes a segment
// of one position's row (target or draft) and leaves its maximum m and
// z = sum exp((l - m) / T); the block that finishes a request's last segment
// joins them and walks the drafts.  The second, a programmatic dependent of
// the first, takes the argmax of the residual's key over one position of each
// request: one target row, one draft row, much of them still in L2, and the
// request's noise, which does not wait for the first launch.
//
// exp((l - m) / T) is ex2((l - m) * c) with c = log2(e) / T: l - m is exact
// or rounded once, and an overflow of l / T cannot make it NaN.
#include "paged.h"
#include "common.cuh"

namespace dtm {

constexpr int kVerifyThreads = 256;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2(e) / T, finite (a T so small that it overflows is the limit T -> 0).
__device__ __forceinline__ float inv_temperature(float T) {
    return fminf(__fdiv_rn(1.4426950408889634f, T), 3.0e38f);
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

__device__ __forceinline__ uint64_t warp_max(uint64_t x) {
    const uint32_t hi = (uint32_t)(x >> 32), lo = (uint32_t)x;
    const uint32_t hm = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t lm = __reduce_max_sync(0xffffffffu, hi == hm ? lo : 0u);
    return ((uint64_t)hm << 32) | lm;
}

// A block's maximum key; every thread gets it.
__device__ __forceinline__ uint64_t block_max(uint64_t x, uint64_t *shared) {
    x = warp_max(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = x;
    __syncthreads();
    x = shared[threadIdx.x & (kVerifyThreads / 32 - 1)];
    return warp_max(x);
}

// The segment's best (logit, id) in the argmax order, whatever it holds.
template <bool F32>
__device__ __noinline__ uint64_t segment_key(const void *row, int64_t base, int lo, int hi, uint64_t *shared) {
    uint64_t best = 0;
    for (int v = lo + threadIdx.x * 8; v < hi; v += kVerifyThreads * 8) {
        float x[8];
        load8<F32>(row, base + v, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint64_t k = pack_key(x[j], (uint32_t)(v + j));
            best = k > best ? k : best;
        }
    }
    return block_max(best, shared);
}

// Two fp32 values in one register pair, and the packed arithmetic on them.
__device__ __forceinline__ uint64_t pack_f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split_f2(uint64_t x, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A row's partial: m, z and the key.  For a row that is sampled the key says
// only whether the maximum is finite, and where it is if it is not.  Both
// kinds of row take kVectors vectors of 8 ids a turn, their loads in flight
// together, and compare the running maximum once a turn; a NaN shows in a
// sum, and then the segment is looked through again.
template <bool F32>
__device__ void segment_stats(const VerifyArgs &a, const void *row, int64_t base, float T, uint4 *out) {
    constexpr int kVectors = F32 ? 2 : 4, kStep = kVerifyThreads * 8;
    __shared__ uint64_t key_s[kVerifyThreads / 32];
    __shared__ float m_s[kVerifyThreads / 32], z_s[kVerifyThreads / 32];
    const int lo = blockIdx.x * a.seg_len, hi = min(a.V, lo + a.seg_len);
    const bool sampled = samples(T);
    const float c = sampled ? inv_temperature(T) : 0.0f;
    float m = -INFINITY, z = 0.0f;
    int at = lo;                                     // greedy: the turn of the maximum
    for (int v = lo + threadIdx.x * 8; v < hi; v += kVectors * kStep) {
        float x[kVectors][8], top = -INFINITY;
#pragma unroll
        for (int k = 0; k < kVectors; ++k) {
            if (v + k * kStep < hi) {
                load8<F32>(row, base + v + k * kStep, x[k]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[k][j] = -INFINITY;
            }
        }
#pragma unroll
        for (int k = 0; k < kVectors; ++k)
#pragma unroll
            for (int j = 0; j < 8; j += 2) top = fmaxf(fmaxf(top, x[k][j]), x[k][j + 1]);
        if (top > m) {
            z = m == -INFINITY ? z : z * ex2((m - top) * c);
            m = top;
            at = v;
        }
        uint64_t sum[2] = {0, 0};
        if (sampled) {
            const float ref = m == -INFINITY ? 0.0f : m;
            const uint64_t neg = pack_f2(-ref, -ref), c2 = pack_f2(c, c);
#pragma unroll
            for (int k = 0; k < kVectors; ++k)
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    float e0, e1;
                    split_f2(mul_f2(add_f2(pack_f2(x[k][j], x[k][j + 1]), neg), c2), e0, e1);
                    sum[j / 2 & 1] = add_f2(sum[j / 2 & 1], pack_f2(ex2(e0), ex2(e1)));
                }
        } else {
            // only for its NaNs (that of inf - inf costs a second look)
#pragma unroll
            for (int k = 0; k < kVectors; ++k)
                if (v + k * kStep < hi)
#pragma unroll
                    for (int j = 0; j < 8; j += 2)
                        sum[j / 2 & 1] = add_f2(sum[j / 2 & 1], pack_f2(x[k][j], x[k][j + 1]));
        }
        float s0, s1;
        split_f2(add_f2(sum[0], sum[1]), s0, s1);
        z += s0 + s1;
    }
    // join the warp, then the block
    const float own = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (own != -INFINITY) z *= ex2((own - m) * c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if ((threadIdx.x & 31) == 0) {
        m_s[threadIdx.x >> 5] = m;
        z_s[threadIdx.x >> 5] = z;
    }
    __syncthreads();
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kVerifyThreads / 32; ++w) m = fmaxf(m, m_s[w]);
    z = 0.0f;
#pragma unroll
    for (int w = 0; w < kVerifyThreads / 32; ++w) z += m_s[w] == -INFINITY ? z_s[w] : z_s[w] * ex2((m_s[w] - m) * c);
    uint64_t key = pack_key(m, (uint32_t)lo);
    if (z != z || m == INFINITY || (sampled && z == INFINITY)) {
        key = segment_key<F32>(row, base, lo, hi, key_s);
    } else if (!sampled && m != -INFINITY) {
        // the lowest id of the maximum, among the ids of its turn
        uint64_t best = 0;
        if (own == m) {
#pragma unroll 1
            for (int k = kVectors - 1; k >= 0; --k)
#pragma unroll 1
                for (int j = 7; j >= 0; --j)
                    if (at + k * kStep < hi && load1<F32>(row, base + at + k * kStep + j) == m)
                        best = pack_key(m, (uint32_t)(at + k * kStep + j));
        }
        key = block_max(best, key_s);
    }
    if (threadIdx.x == 0)
        __stcg(out, make_uint4(__float_as_uint(m), __float_as_uint(z), (uint32_t)key, (uint32_t)(key >> 32)));
}

// A position's distribution: exp((l - m) / T) * inv_z, or one-hot at `id`.
struct Dist {
    float m, inv_z;
    int id;                    // -1: not one-hot
};

__device__ __forceinline__ float prob(const Dist &d, float l, int v, float c) {
    if (d.id >= 0) return v == d.id ? 1.0f : 0.0f;
    return ex2((l - d.m) * c) * d.inv_z;
}

// What the second launch has to know of a request: its distributions at the
// position it draws, and that position; the row's winner word is cleared.
struct Verdict {
    Dist p, q;
    int n;
    int pad;
};
static_assert(sizeof(Verdict) == kVerdictBytes, "plan scratch");

// By the block that finished the last of the request's segments: its 2 N + 1
// distributions, the walk over the drafts and what is known by now of the
// outputs.
template <bool TF32, bool CF32>
__device__ void decide(const VerifyArgs &a, int b, float T) {
    constexpr int kWarps = kVerifyThreads / 32, kTurns = (2 * kMaxSteps + 1 + kWarps - 1) / kWarps;
    __shared__ Dist dist[2 * kMaxSteps + 1];
    __shared__ float p_s[kMaxSteps], q_s[kMaxSteps], u_s[kMaxSteps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.N, per = 2 * N + 1;
    const float c = samples(T) ? inv_temperature(T) : 0.0f;
    // every load of the block first: partials, drafts and their logits
    uint4 part[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        part[k] = make_uint4(0xff800000u, 0u, 0u, 0u);
        if (warp + k * kWarps < per && lane < a.segs)
            part[k] = __ldcg(a.part + ((int64_t)b * per + warp + k * kWarps) * a.segs + lane);
    }
    int64_t x = -1;
    float lp = 0.0f, lq = 0.0f;
    if (tid < N) {
        x = a.draft[b * a.draft_s0 + tid];
        u_s[tid] = a.uniforms[b * a.uni_s0 + tid];
        if (x >= 0 && x < a.V) {
            lp = load1<TF32>(a.target, b * a.target_s0 + tid * a.target_s1 + x);
            lq = load1<CF32>(a.cache, b * a.cache_s0 + tid * a.cache_s1 + x);
        }
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
        const uint64_t key = warp_max(((uint64_t)part[k].w << 32) | part[k].z);
        if (lane == 0) {
            const uint32_t o = packed_ordered(key);
            const bool finite = o != 0xffffffffu && isfinite(key_from_ordered(o));
            dist[warp + k * kWarps] = Dist{M, 1.0f / Z, samples(T) && finite ? -1 : (int)packed_id(key)};
        }
    }
    __syncthreads();
    if (tid < N) {
        const bool in = x >= 0 && x < a.V;
        p_s[tid] = in ? prob(dist[tid], lp, (int)x, c) : 0.0f;
        q_s[tid] = in ? prob(dist[N + 1 + tid], lq, (int)x, c) : 0.0f;
    }
    __syncthreads();
    int n = 0;
    while (n < N && u_s[n] * q_s[n] < p_s[n]) ++n;
    if (tid < N && a.p) {
        a.p[(int64_t)b * N + tid] = p_s[tid];
        a.q[(int64_t)b * N + tid] = q_s[tid];
    }
    const Dist P = dist[n];
    if (tid <= N) {
        // where p is one-hot there is nothing to draw
        int64_t *token = a.tokens + b * a.tok_s0 + tid;
        if (tid < n) *token = x;
        else if (tid > n) *token = -1;
        else if (P.id >= 0) *token = P.id;
    }
    if (tid == 0) {
        a.accepted[b] = n;
        Verdict v{P, n < N ? dist[N + 1 + n] : P, n, 0};
        reinterpret_cast<Verdict *>(a.verdicts)[b] = v;
        a.win[b] = 0;
    }
}

template <bool TF32, bool CF32>
__global__ void __launch_bounds__(kVerifyThreads) verify_stats_kernel(VerifyArgs a) {
    __shared__ uint32_t last_s;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int per = 2 * a.N + 1, row = blockIdx.y, b = row / per, i = row - b * per;
    if (a.idx[b] < 0 || __ldcg(a.status) != 0u) return;
    uint4 *out = a.part + (int64_t)row * a.segs + blockIdx.x;
    const float T = a.temperature[b];
    if (i <= a.N)
        segment_stats<TF32>(a, a.target, b * a.target_s0 + i * a.target_s1, T, out);
    else
        segment_stats<CF32>(a, a.cache, b * a.cache_s0 + (i - a.N - 1) * a.cache_s1, T, out);
    if (threadIdx.x == 0) {
        __threadfence();
        const uint32_t blocks = (uint32_t)(per * a.segs);
        last_s = atomicAdd(a.arrivals + b, 1u) == blocks - 1;
        if (last_s) a.arrivals[b] = 0;               // the second launch counts from here
        __threadfence();
    }
    __syncthreads();
    if (last_s) decide<TF32, CF32>(a, b, T);
}

template <bool TF32, bool CF32>
__global__ void __launch_bounds__(kVerifyThreads) verify_pick_kernel(VerifyArgs a) {
    __shared__ uint64_t key_s[kVerifyThreads / 32];
    __shared__ uint32_t last_s;
    const int b = blockIdx.y, N = a.N, tid = threadIdx.x;
    const float *noise = a.noise + b * a.noise_s0;
    const int lo = blockIdx.x * a.pick_len, hi = min(a.V, lo + a.pick_len);
    const bool padding = a.idx[b] < 0;
    const float T = a.temperature[b];
    const float c = samples(T) ? inv_temperature(T) : 0.0f;
    // an input, and the largest: on its way before the first launch is done
    float first[8];
    if (!padding && samples(T) && lo + tid * 8 < hi) load8<true>(noise, lo + tid * 8, first);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (padding || __ldcg(a.status) != 0u) return;
    const uint4 *said = reinterpret_cast<const uint4 *>(reinterpret_cast<const Verdict *>(a.verdicts) + b);
    const uint4 v0 = __ldcg(said), v1 = __ldcg(said + 1);
    const Dist P{__uint_as_float(v0.x), __uint_as_float(v0.y), (int)v0.z};
    const Dist Q{__uint_as_float(v0.w), __uint_as_float(v1.x), (int)v1.y};
    const int n = (int)v1.z;
    if (P.id >= 0) return;                           // its token is out
    const int64_t t_base = b * a.target_s0 + n * a.target_s1, c_base = b * a.cache_s0 + n * a.cache_s1;

    // the best key over [lo, hi): of ln(p - q) + g, or of ln p + g with whole
    auto best_of = [&](int lo, int hi, bool whole, bool again) {
        uint64_t best = 0;
        float mine = -INFINITY;
        for (int v = lo + tid * 8; v < hi; v += kVerifyThreads * 8) {
            float x[8], y[8], g[8];
            load8<TF32>(a.target, t_base + v, x);
            if (!whole) load8<CF32>(a.cache, c_base + v, y);
            if (!again && v < lo + kVerifyThreads * 8) {
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = first[j];
            } else {
                load8<true>(noise, v, g);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float r = prob(P, x[j], v + j, c);
                if (!whole) r -= prob(Q, y[j], v + j, c);
                // the fast logarithm (within 1e-5 here) tells which few ids
                // need the exact one
                if (r > 0.0f && __logf(r) + g[j] >= mine - 1e-3f) {
                    const float key = logf(r) + g[j];
                    if (key > mine || best == 0) {
                        mine = key;
                        best = pack_key(key, (uint32_t)(v + j));
                    }
                }
            }
        }
        return block_max(best, key_s);
    };
    const uint64_t best = best_of(lo, hi, n == N, false);
    if (tid == 0) {
        if (best) atomicMax(reinterpret_cast<unsigned long long *>(a.win + b), (unsigned long long)best);
        __threadfence();
        last_s = atomicAdd(a.arrivals + b, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last_s) return;
    __threadfence();
    uint64_t win = ld_cg_u64(a.win + b);
    if (win == 0) win = best_of(0, a.V, true, true);   // p <= q everywhere
    if (tid == 0) {
        a.tokens[b * a.tok_s0 + n] = win ? packed_id(win) : 0;
        a.arrivals[b] = 0;
    }
}

template <bool TF32, bool CF32>
static cudaError_t launch_verify_typed(const VerifyArgs &a, cudaStream_t s) {
    verify_stats_kernel<TF32, CF32><<<dim3(a.segs, a.rows * (2 * a.N + 1)), kVerifyThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.pick_segs, a.rows);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_pick_kernel<TF32, CF32>, a);
}

// Segments of V ids for `rows` rows: about `blocks` blocks, at least one
// vector of 8 ids a thread.
static void segments(int V, int rows, int blocks, int *segs, int *len) {
    const int round = kVerifyThreads * 8;
    int n = (blocks + rows - 1) / rows;
    const int most = (V + round - 1) / round;
    if (n > most) n = most;
    if (n > kVerifyMaxSegs) n = kVerifyMaxSegs;
    if (n < 1) n = 1;
    *len = ((V + n - 1) / n + 7) / 8 * 8;
    *segs = (V + *len - 1) / *len;
}

cudaError_t launch_verify(VerifyArgs a, bool target_f32, bool cache_f32, int sms, cudaStream_t s) {
    segments(a.V, a.rows * (2 * a.N + 1), 24 * sms, &a.segs, &a.seg_len);
    segments(a.V, a.rows, 12 * sms, &a.pick_segs, &a.pick_len);
    if (target_f32)
        return cache_f32 ? launch_verify_typed<true, true>(a, s) : launch_verify_typed<true, false>(a, s);
    return cache_f32 ? launch_verify_typed<false, true>(a, s) : launch_verify_typed<false, false>(a, s);
}

}  // namespace dtm
