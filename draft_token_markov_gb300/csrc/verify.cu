// verify.cu -- acceptance of drafts against the target's logits.
//
// Two launches.  The first reads every logit once: a block takes a segment
// of one position's row (target or draft) and leaves its maximum m and
// z = sum exp((l - m) / T).  The second, a programmatic dependent of the
// first, joins a request's partials in every one of its blocks (at most 33
// rows of 64), walks the drafts, and takes the argmax of the residual's key
// over the block's ids; the block that arrives last writes the token.  The
// second look touches one target and one draft row of a request, most of it
// still in L2, and its row of noise.
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

// The segment's best (logit, id) in the argmax order.
template <bool F32>
__device__ uint64_t segment_key(const void *row, int64_t base, int lo, int hi, uint64_t *shared) {
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

// A row's partial: m, z and the key.  For a row that is sampled the key says
// only whether the maximum is finite, and where it is if it is not.
template <bool F32>
__device__ void segment_stats(const VerifyArgs &a, const void *row, int64_t base, float T, uint4 *out) {
    __shared__ uint64_t key_s[kVerifyThreads / 32];
    __shared__ float m_s[kVerifyThreads / 32], z_s[kVerifyThreads / 32];
    const int lo = blockIdx.x * a.seg_len, hi = min(a.V, lo + a.seg_len);
    float m = -INFINITY, z = 0.0f;
    uint64_t key = 0;
    if (samples(T)) {
        const float c = inv_temperature(T);
        // two loads in flight; the running maximum is compared once per 8
        for (int v = lo + threadIdx.x * 8; v < hi; v += kVerifyThreads * 8) {
            float x[8];
            load8<F32>(row, base + v, x);
            float top = x[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) top = fmaxf(top, x[j]);
            if (top > m) {
                z = m == -INFINITY ? 0.0f : z * ex2((m - top) * c);
                m = top;
            }
            const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int j = 0; j < 8; ++j) z += ex2((x[j] - ref) * c);
        }
        // join the warp, then the block
        float M = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        z = m == -INFINITY ? z : z * ex2((m - M) * c);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if ((threadIdx.x & 31) == 0) {
            m_s[threadIdx.x >> 5] = M;
            z_s[threadIdx.x >> 5] = z;
        }
        __syncthreads();
        m = -INFINITY;
        for (int w = 0; w < kVerifyThreads / 32; ++w) m = fmaxf(m, m_s[w]);
        z = 0.0f;
        for (int w = 0; w < kVerifyThreads / 32; ++w)
            z += m_s[w] == -INFINITY ? z_s[w] : z_s[w] * ex2((m_s[w] - m) * c);
        key = pack_key(m, (uint32_t)lo);
        // a NaN or an infinity: the id decides
        if (!(z < INFINITY) || m == INFINITY) key = segment_key<F32>(row, base, lo, hi, key_s);
    } else {
        key = segment_key<F32>(row, base, lo, hi, key_s);
    }
    if (threadIdx.x == 0)
        *out = make_uint4(__float_as_uint(m), __float_as_uint(z), (uint32_t)key, (uint32_t)(key >> 32));
}

template <bool TF32, bool CF32>
__global__ void __launch_bounds__(kVerifyThreads) verify_stats_kernel(VerifyArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int per = 2 * a.N + 1, row = blockIdx.y, b = row / per, i = row - b * per;
    if (a.idx[b] < 0 || ld_acquire_u32(a.status) != 0u) return;
    uint4 *out = a.part + (int64_t)row * a.segs + blockIdx.x;
    const float T = a.temperature[b];
    if (i <= a.N)
        segment_stats<TF32>(a, a.target, b * a.target_s0 + i * a.target_s1, T, out);
    else
        segment_stats<CF32>(a, a.cache, b * a.cache_s0 + (i - a.N - 1) * a.cache_s1, T, out);
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

template <bool TF32, bool CF32>
__global__ void __launch_bounds__(kVerifyThreads) verify_pick_kernel(VerifyArgs a) {
    __shared__ Dist dist[2 * kMaxSteps + 1];
    __shared__ float p_s[kMaxSteps], q_s[kMaxSteps];
    __shared__ uint64_t key_s[kVerifyThreads / 32];
    __shared__ uint32_t last_s;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.y, N = a.N, per = 2 * N + 1;
    if (a.idx[b] < 0 || ld_acquire_u32(a.status) != 0u) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float T = a.temperature[b];
    const float c = samples(T) ? inv_temperature(T) : 0.0f;

    // the row's 2 N + 1 distributions, a warp each in turn
    for (int i = warp; i < per; i += kVerifyThreads / 32) {
        const uint4 *part = a.part + ((int64_t)b * per + i) * a.segs;
        float m[kVerifyMaxSegs / 32], z[kVerifyMaxSegs / 32], M = -INFINITY;
        uint64_t key = 0;
#pragma unroll
        for (int k = 0; k < kVerifyMaxSegs / 32; ++k) {
            m[k] = -INFINITY;
            z[k] = 0.0f;
            if (lane + 32 * k < a.segs) {
                const uint4 x = __ldcg(part + lane + 32 * k);
                m[k] = __uint_as_float(x.x);
                z[k] = __uint_as_float(x.y);
                const uint64_t y = ((uint64_t)x.w << 32) | x.z;
                key = y > key ? y : key;
            }
            M = fmaxf(M, m[k]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float Z = 0.0f;
#pragma unroll
        for (int k = 0; k < kVerifyMaxSegs / 32; ++k)
            if (m[k] != -INFINITY) Z += z[k] * ex2((m[k] - M) * c);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) Z += __shfl_xor_sync(0xffffffffu, Z, o);
        key = warp_max(key);
        if (lane == 0) {
            const uint32_t o = packed_ordered(key);
            const bool finite = o != 0xffffffffu && isfinite(key_from_ordered(o));
            dist[i].m = M;
            dist[i].inv_z = 1.0f / Z;
            dist[i].id = samples(T) && finite ? -1 : (int)packed_id(key);
        }
    }
    __syncthreads();
    if (tid < N) {
        const int64_t x = a.draft[b * a.draft_s0 + tid];
        float p = 0.0f, q = 0.0f;
        if (x >= 0 && x < a.V) {
            p = prob(dist[tid], load1<TF32>(a.target, b * a.target_s0 + tid * a.target_s1 + x), (int)x, c);
            q = prob(dist[N + 1 + tid], load1<CF32>(a.cache, b * a.cache_s0 + tid * a.cache_s1 + x), (int)x, c);
        }
        p_s[tid] = p;
        q_s[tid] = q;
    }
    __syncthreads();
    int n = 0;
    while (n < N && a.uniforms[b * a.uni_s0 + n] * q_s[n] < p_s[n]) ++n;

    if (blockIdx.x == 0) {
        if (tid < N && a.p) {
            a.p[(int64_t)b * N + tid] = p_s[tid];
            a.q[(int64_t)b * N + tid] = q_s[tid];
        }
        if (tid == 0) a.accepted[b] = n;
        if (tid <= N && tid != n)
            a.tokens[b * a.tok_s0 + tid] = tid < n ? a.draft[b * a.draft_s0 + tid] : -1;
    }
    const Dist P = dist[n];
    if (P.id >= 0) {           // nothing to draw
        if (blockIdx.x == 0 && tid == 0) a.tokens[b * a.tok_s0 + n] = P.id;
        return;
    }
    Dist Q = n < N ? dist[N + 1 + n] : P;
    const int64_t t_base = b * a.target_s0 + n * a.target_s1, c_base = b * a.cache_s0 + n * a.cache_s1;
    const float *noise = a.noise + b * a.noise_s0;

    // the best key over [lo, hi): of ln(p - q) + g, or of ln p + g with whole
    auto best_of = [&](int lo, int hi, bool whole) {
        uint64_t best = 0;
        float mine = -INFINITY;
        for (int v = lo + tid * 8; v < hi; v += kVerifyThreads * 8) {
            float x[8], y[8], g[8];
            load8<TF32>(a.target, t_base + v, x);
            if (!whole) load8<CF32>(a.cache, c_base + v, y);
            load8<true>(noise, v, g);
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
    const int lo = blockIdx.x * a.pick_len, hi = min(a.V, lo + a.pick_len);
    const uint64_t best = best_of(lo, hi, n == N);
    if (tid == 0) {
        if (best) atomicMax(reinterpret_cast<unsigned long long *>(a.win + b), (unsigned long long)best);
        __threadfence();
        last_s = atomicAdd(a.arrivals + b, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last_s) return;
    __threadfence();
    uint64_t win = ld_cg_u64(a.win + b);
    if (win == 0) win = best_of(0, a.V, true);     // p <= q everywhere
    if (tid == 0) {
        a.tokens[b * a.tok_s0 + n] = win ? packed_id(win) : 0;
        a.win[b] = 0;
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

// Segments of V ids for `rows` rows: about eight blocks an SM, at least one
// round of loads a block.
static void segments(int V, int rows, int sms, int *segs, int *len) {
    const int round = kVerifyThreads * 8;
    int n = (8 * sms + rows - 1) / rows;
    const int most = (V + round - 1) / round;
    if (n > most) n = most;
    if (n > kVerifyMaxSegs) n = kVerifyMaxSegs;
    if (n < 1) n = 1;
    *len = ((V + n - 1) / n + 7) / 8 * 8;
    *segs = (V + *len - 1) / *len;
}

cudaError_t launch_verify(VerifyArgs a, bool target_f32, bool cache_f32, int sms, cudaStream_t s) {
    segments(a.V, a.rows * (2 * a.N + 1), sms, &a.segs, &a.seg_len);
    segments(a.V, a.rows, sms, &a.pick_segs, &a.pick_len);
    if (target_f32)
        return cache_f32 ? launch_verify_typed<true, true>(a, s) : launch_verify_typed<true, false>(a, s);
    return cache_f32 ? launch_verify_typed<false, true>(a, s) : launch_verify_typed<false, false>(a, s);
}

}  // namespace dtm
