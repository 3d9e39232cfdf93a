// logprobs.cu -- log probabilities of given tokens, rank, entropy and the most
// probable alternatives: one launch, a cluster of thread blocks a row of logits,
// and its C ABI.
//
// Each block of the cluster takes a slice of the row to shared memory (at most
// 32 KB where 8 blocks do, so that several slices are in flight on a
// multiprocessor) and reads it there three times: for the largest logit, for the
// sums
//   Z = sum 2^d,  S = sum 2^d d,  d = (l - m) log2(e) / T
// against the slice's own maximum m, and for the few logits that may be among
// the `top` largest.  For these, the slice is cut into 64 groups (four
// neighbouring lanes each): the top-th largest group maximum is a bound that at
// least `top` logits reach and that fewer than `top` groups exceed; what exceeds
// it is collected, what equals it too (lowest ids first), and put in order by
// counting.  The first block joins the cluster's sums and sorted lists, which the
// others write to its shared memory.
//
// ln p = (l - m) / T - ln Z, entropy = (log2 Z - S / Z) ln 2.  Every logit is read
// once from memory.
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "../../include/markov.h"
#include "common.cuh"
#include "f32x2.cuh"
#include "host_util.h"

using namespace dtm;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = kThreads / 4;
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr int kSliceBytes = 32768;        // of a block, unless eight of them are not enough
constexpr int kTies = 256;
constexpr int kMostShared = 200 << 10;    // 262144 fp32 logits need 164 KB

struct LogprobArgs {
    const uint8_t *logits;
    int64_t s0;                           // bytes
    int vocab, top;
    const int64_t *tokens;
    const float *temperature;
    float *logprobs, *entropy, *top_logprobs;
    int32_t *ranks, *top_ids;
    int slice;                            // bytes of a block, a multiple of 16
    int list;                             // entries of the list of candidates
};

// What a block knows of its slice, in the first block's shared memory.
struct Part {
    float m, z, s;
    int before;                           // ids that come before the token
    uint64_t best;                        // the argmax's key where m is not finite
    uint64_t top[kMaxTop];                // keys, falling
};

template <bool F32>
__device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t b) {
    uint32_t r;
    if (F32)
        asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 16 bytes as logits.
template <bool F32>
struct Logits {
    static constexpr int kN = F32 ? 4 : 8;
    float x[kN];
    __device__ __forceinline__ explicit Logits(const uint4 &v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (F32) {
                x[i] = __uint_as_float(w[i]);
            } else {
                x[(2 * i) % kN] = __uint_as_float(w[i] << 16);
                x[(2 * i + 1) % kN] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
};

template <bool F32>
__device__ __forceinline__ float vector_max(const uint4 &v) {
    const uint32_t w = word_max<F32>(word_max<F32>(v.x, v.y), word_max<F32>(v.z, v.w));
    if (F32) return __uint_as_float(w);
    return __uint_as_float(word_max<true>(w << 16, w & 0xffff0000u));
}

__device__ __forceinline__ float nan_max(float a, float b) {
    return __uint_as_float(word_max<true>(__float_as_uint(a), __float_as_uint(b)));
}

__device__ __forceinline__ uint64_t warp_max_key(uint64_t x) {
    const uint32_t hi = (uint32_t)(x >> 32), hm = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t lm = __reduce_max_sync(0xffffffffu, hi == hm ? (uint32_t)x : 0u);
    return (uint64_t)hm << 32 | lm;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address of the same variable in the cluster's first block.
__device__ __forceinline__ uint32_t first_block(const void *p) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)));
    return r;
}
__device__ __forceinline__ void st_cluster(uint32_t to, uint32_t x) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(x) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t to, uint64_t x) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(x) : "memory");
}

constexpr float kLn2 = 0.69314718055994531f;

template <bool F32>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const __grid_constant__ LogprobArgs a) {
    constexpr int kSize = F32 ? 4 : 2, kN = 16 / kSize;
    extern __shared__ __align__(16) uint8_t smem[];
    uint4 *slice = reinterpret_cast<uint4 *>(smem);
    uint16_t *list = reinterpret_cast<uint16_t *>(smem + a.slice);     // elements of the slice
    __shared__ Part parts[kMaxCluster];
    __shared__ float warp_f[3][kWarps];
    __shared__ int warp_i[kWarps];
    __shared__ uint64_t warp_k[kWarps];
    __shared__ float group_max[kGroups];
    __shared__ uint16_t ties[kTies];
    __shared__ int listed_s, ties_s;
    __shared__ float bound_s;
    __shared__ uint64_t sorted[kMaxTop];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), blocks = gridDim.x;
    const int64_t row = blockIdx.y;
    const int64_t token = a.tokens ? __ldg(a.tokens + row) : -1;
    if (a.tokens && (token < 0 || token >= a.vocab)) return;           // the whole cluster
    if (blocks > 1) cluster_arrive();                                  // every block runs

    // the slice: whole vectors from the row's first on, whose first `lead` elements
    // lie before the row
    const uint8_t *from = a.logits + row * a.s0;
    const int lead_bytes = (int)(reinterpret_cast<uintptr_t>(from) & 15u);
    const int64_t bytes = (int64_t)a.vocab * kSize + lead_bytes;       // from the first vector's start
    const int64_t begin = (int64_t)rank * a.slice;
    const int vectors = (int)(min(max(bytes - begin, (int64_t)0), (int64_t)a.slice) + 15) / 16;
    const uint8_t *first = from - lead_bytes + begin;
    const int id0 = (int)((begin - lead_bytes) / kSize);               // of the slice's first element
    for (int v = tid; v < vectors; v += kThreads) {
        const int id = id0 + v * kN;
        if (id >= 0 && id + kN <= a.vocab) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(slice + v)),
                         "l"(first + 16 * (int64_t)v)
                         : "memory");
        } else {
            // -inf where the row does not reach
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                const bool there = id + e >= 0 && id + e < a.vocab;
                if (F32) {
                    w[e % 4] = there ? __ldg(reinterpret_cast<const uint32_t *>(from) + id + e) : 0xff800000u;
                } else {
                    const uint32_t x = there ? __ldg(reinterpret_cast<const uint16_t *>(from) + id + e) : 0xff80u;
                    w[e / 2 % 4] = e & 1 ? w[e / 2 % 4] | x << 16 : x;
                }
            }
            slice[v] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    float T = a.temperature ? __ldg(a.temperature + row) : 1.0f;
    if (!samples(T)) T = 1.0f;
    // finite, and not 0: with T = inf the difference of finite logits vanishes, -inf stays
    const float c = fmaxf(fminf(__fdiv_rn(1.4426950408889634f, T), 3.0e38f), 1.401298464e-45f);
    float own = 0.0f;
    if (a.tokens)
        own = F32 ? __ldg(reinterpret_cast<const float *>(from) + token)
                  : __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(from) + token) << 16);
    if (tid == 0) listed_s = ties_s = 0;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();

    // ------------------------------------------------------------- maximum
    const auto element = [&](int e) {
        return F32 ? reinterpret_cast<const float *>(smem)[e]
                   : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(smem)[e] << 16);
    };
    const auto inside = [&](int e) { return id0 + e >= 0 && id0 + e < a.vocab; };
    float top = -INFINITY;
    for (int v = tid; v < vectors; v += kThreads) top = nan_max(top, vector_max<F32>(slice[v]));
    float group = nan_max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    group = nan_max(group, __shfl_xor_sync(0xffffffffu, group, 2));
    if ((lane & 3) == 0) group_max[tid >> 2] = group;
    float m = group;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) m = nan_max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) warp_f[0][warp] = m;
    __syncthreads();
    m = warp_f[0][0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = nan_max(m, warp_f[0][w]);
    const bool odd = !(fabsf(m) < INFINITY);                           // NaN, an infinity, nothing

    // ------------------------------------------- sums, ids before the token
    float z = 0.0f, s = 0.0f;
    int before = 0;
    uint64_t best = 0;
    const bool by_key = a.tokens && (odd || !(own > -INFINITY));       // NaN or -inf in the comparison
    if (!odd) {
        const uint64_t neg = f32x2(-m, -m), c2 = f32x2(c, c);
        uint64_t z2[2] = {0, 0}, s2[2] = {0, 0};
        for (int v = tid; v < vectors; v += kThreads) {
            const Logits<F32> l(slice[v]);
#pragma unroll
            for (int e = 0; e < kN; e += 2) {
                float d0, d1;
                split2(mul2(add2(f32x2(l.x[e], l.x[e + 1]), neg), c2), d0, d1);
                const uint64_t p = f32x2(ex2(d0), ex2(d1));
                z2[e / 2 & 1] = add2(z2[e / 2 & 1], p);
                // a masked logit's 0 times -inf is 0
                s2[e / 2 & 1] = fma2(p, f32x2(fmaxf(d0, -1024.0f), fmaxf(d1, -1024.0f)), s2[e / 2 & 1]);
            }
            if (a.tokens && !by_key) {
                const int64_t id = id0 + (int64_t)v * kN;
                if (id + kN <= token) {
#pragma unroll
                    for (int e = 0; e < kN; ++e) before += l.x[e] >= own;
                } else if (id > token) {
#pragma unroll
                    for (int e = 0; e < kN; ++e) before += l.x[e] > own;
                } else {
#pragma unroll
                    for (int e = 0; e < kN; ++e) before += id + e < token ? l.x[e] >= own : l.x[e] > own;
                }
            }
        }
        float x0, x1, y0, y1;
        split2(add2(z2[0], z2[1]), x0, x1);
        split2(add2(s2[0], s2[1]), y0, y1);
        z = x0 + x1;
        s = y0 + y1;
    }
    if (odd || by_key) {
        const uint64_t own_key = a.tokens ? pack_key(own, (uint32_t)token) : 0;
        for (int e = tid; e < vectors * kN; e += kThreads) {
            if (!inside(e)) continue;
            const uint64_t k = pack_key(element(e), (uint32_t)(id0 + e));
            if (by_key) before += k > own_key;
            if (odd) best = k > best ? k : best;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, o);
        s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    before = __reduce_add_sync(0xffffffffu, before);
    best = warp_max_key(best);
    if (lane == 0) {
        warp_f[1][warp] = z;
        warp_f[2][warp] = s;
        warp_i[warp] = before;
        warp_k[warp] = best;
    }

    // --------------------------------------------------------- alternatives
    if (a.top > 0) {
        if (warp == 0) {
            // the top-th largest group maximum
            uint32_t g0 = ordered_key(group_max[lane]), g1 = ordered_key(group_max[32 + lane]), g = 0;
            for (int k = 0; k < a.top; ++k) {
                const uint32_t mine = max(g0, g1);
                g = __reduce_max_sync(0xffffffffu, mine);
                const uint32_t who = __ballot_sync(0xffffffffu, mine == g);
                if (lane == __ffs(who) - 1) {
                    if (g0 == g) g0 = 0; else g1 = 0;
                }
            }
            if (lane == 0) bound_s = key_from_ordered(g);              // NaN for NaN: 0x7fffffff
        }
        __syncthreads();
        const float bound = bound_s;
        const uint32_t bound_key = ordered_key(bound);
        if (ordered_key(group) >= bound_key) {
            for (int v = tid; v < vectors; v += kThreads) {
                const uint4 w = slice[v];
                if (ordered_key(vector_max<F32>(w)) < bound_key) continue;
                const Logits<F32> l(w);
#pragma unroll
                for (int e = 0; e < kN; ++e) {
                    const uint32_t k = ordered_key(l.x[e]);
                    const int at = v * kN + e;
                    if (k > bound_key) {
                        list[atomicAdd(&listed_s, 1)] = (uint16_t)at;
                    } else if (k == bound_key && inside(at)) {
                        const int n = atomicAdd(&ties_s, 1);
                        if (n < kTies) ties[n] = (uint16_t)at;
                    }
                }
            }
        }
        __syncthreads();
        const int listed = listed_s;
        int tied = ties_s;
        if (tied > kTies) {
            // many: the lowest ids of them, in order
            if (warp == 0) {
                int n = 0;
                for (int e0 = 0; n < a.top && e0 < vectors * kN; e0 += 32) {
                    const int e = e0 + lane;
                    const bool is = e < vectors * kN && inside(e) && ordered_key(element(e)) == bound_key;
                    const uint32_t who = __ballot_sync(0xffffffffu, is);
                    const int at = n + __popc(who & ((1u << lane) - 1u));
                    if (is && at < a.top) ties[at] = (uint16_t)e;
                    n += __popc(who);
                }
            }
            tied = a.top;
            __syncthreads();
        }
        if (tid < kMaxTop) sorted[tid] = 0;
        __syncthreads();
        // in order, by counting
        const auto key = [&](int i) {
            const int e = i < listed ? list[i] : ties[i - listed];
            return pack_key(element(e), (uint32_t)(id0 + e));
        };
        for (int i = tid; i < listed + tied; i += kThreads) {
            const uint64_t k = key(i);
            int n = 0;
            for (int j = 0; j < listed + tied && n < a.top; ++j) n += key(j) > k;
            if (n < a.top) sorted[n] = k;
        }
    }
    __syncthreads();

    // ------------------------------------------------------------ the parts
    Part &mine = parts[rank];
    if (blocks > 1) cluster_wait();                                    // the first block runs
    if (warp == 0) {
        z = s = 0.0f;
        before = 0;
        best = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            z += warp_f[1][w];
            s += warp_f[2][w];
            before += warp_i[w];
            best = warp_k[w] > best ? warp_k[w] : best;
        }
        const uint32_t to = first_block(&mine);
        if (lane == 0) {
            st_cluster(to + offsetof(Part, m), __float_as_uint(m));
            st_cluster(to + offsetof(Part, z), __float_as_uint(z));
            st_cluster(to + offsetof(Part, s), __float_as_uint(s));
            st_cluster(to + offsetof(Part, before), (uint32_t)before);
            st_cluster(to + offsetof(Part, best), best);
        }
        if (lane < a.top) st_cluster(to + offsetof(Part, top) + 8 * lane, sorted[lane]);
    }
    if (blocks > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (rank != 0) return;

    // ------------------------------------------------------------- the join
    float all = parts[0].m;
    for (uint32_t b = 1; b < blocks; ++b) all = nan_max(all, parts[b].m);
    const bool one_hot = !(fabsf(all) < INFINITY);
    z = s = 0.0f;
    before = 0;
    best = 0;
    for (uint32_t b = 0; b < blocks; ++b) {
        const Part &p = parts[b];
        before += p.before;
        best = p.best > best ? p.best : best;
        if (one_hot || p.m == -INFINITY) continue;
        const float d = (p.m - all) * c, f = ex2(d);
        z += p.z * f;
        s += f > 0.0f ? f * (p.s + d * p.z) : 0.0f;
    }
    const float log_z = one_hot ? 0.0f : log2f(z);
    const auto log_p = [&](float l, int id) {
        if (one_hot) return id == (int)packed_id(best) ? 0.0f : -INFINITY;
        // in nats: a logit of the type's lowest value would leave the range of d
        return l == -INFINITY ? l : __fdiv_rn(l - all, T) - log_z * kLn2;
    };
    if (tid == 0) {
        if (a.logprobs && a.tokens) a.logprobs[row] = log_p(own, (int)token);
        if (a.ranks && a.tokens) a.ranks[row] = before;
        if (a.entropy) a.entropy[row] = one_hot ? 0.0f : fmaxf((log_z - __fdiv_rn(s, z)) * kLn2, 0.0f);
    }
    if (a.top > 0 && a.top_ids) {
        // a key's place: its own in its list, and the larger ones of the other lists
        for (int i = tid; i < (int)blocks * a.top; i += kThreads) {
            const int b = i / a.top;
            const uint64_t k = parts[b].top[i - b * a.top];
            if (k == 0) continue;
            int n = i - b * a.top;
            for (int o = 0; o < (int)blocks && n < a.top; ++o) {
                if (o == b) continue;
                int lo = 0, hi = a.top;                                // the first that is not larger
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (parts[o].top[mid] > k) lo = mid + 1; else hi = mid;
                }
                n += lo;
            }
            if (n < a.top) {
                const int id = (int)packed_id(k);
                a.top_ids[row * a.top + n] = id;
                a.top_logprobs[row * a.top + n] = log_p(key_from_ordered(packed_ordered(k)), id);
            }
        }
    }
}

// The blocks of a row's cluster and the bytes of a slice.
void cut_row(int64_t bytes, int &blocks, int &slice) {
    blocks = 1;
    while (blocks < kMaxCluster && (bytes + blocks - 1) / blocks > kSliceBytes) blocks *= 2;
    slice = (int)((bytes + blocks - 1) / blocks + 15) / 16 * 16;
}

// Lets the kernels take what a call may need, once a device.
bool allow_shared_memory(int device) {
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = device < 64 ? 1ull << device : 0ull;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    for (const void *fn : {(const void *)logprobs_kernel<false>, (const void *)logprobs_kernel<true>})
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

}  // namespace

extern "C" markov_status markov_logprobs(const void *logits, markov_dtype dtype, int64_t logits_s0,
                                         int32_t rows, int32_t vocab, const int64_t *tokens,
                                         const float *temperature, int32_t top, float *logprobs,
                                         int32_t *ranks, float *entropy, int32_t *top_ids,
                                         float *top_logprobs, void *stream) {
    if (dtype != MARKOV_BF16 && dtype != MARKOV_F32) return MARKOV_EINVAL;
    const bool f32 = dtype == MARKOV_F32;
    const int size = f32 ? 4 : 2;
    if (rows < 0 || vocab < 1 || vocab > kMaxVocab || top < 0 || top > kMaxTop || top > vocab) return MARKOV_EINVAL;
    if (rows > 1 && logits_s0 < vocab) return MARKOV_EINVAL;
    if (!tokens && (logprobs || ranks)) return MARKOV_EINVAL;
    if ((top_ids == nullptr) != (top_logprobs == nullptr)) return MARKOV_EINVAL;
    if (rows == 0) return MARKOV_OK;
    if (!logits || reinterpret_cast<uintptr_t>(logits) % size != 0) return MARKOV_EINVAL;
    if (!top_ids) top = 0;
    if (!logprobs && !ranks && !entropy && top == 0) return MARKOV_OK;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, logits) != cudaSuccess ||
        (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)) {
        cudaGetLastError();
        return MARKOV_EDEVICE;
    }
    DeviceGuard guard(at.device);
    if (!guard.ok) return MARKOV_EDEVICE;
    LogprobArgs a{};
    a.logits = static_cast<const uint8_t *>(logits);
    a.s0 = rows > 1 ? logits_s0 * size : 0;
    a.vocab = vocab;
    a.top = top;
    a.tokens = tokens;
    a.temperature = temperature;
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.top_logprobs = top_logprobs;
    a.ranks = ranks;
    a.top_ids = top_ids;
    int blocks;
    cut_row((int64_t)vocab * size + 16, blocks, a.slice);
    // fewer than `top` groups have logits above the bound
    const int in_group = 4 * ((a.slice / 16 + kThreads - 1) / kThreads) * (16 / size);
    a.list = (top > 0 ? top - 1 : 0) * in_group;
    const int smem = a.slice + (a.list * 2 + 15) / 16 * 16;
    if (!allow_shared_memory(at.device)) return MARKOV_ECUDA;
    for (int32_t r0 = 0; r0 < rows; r0 += 65535) {
        LogprobArgs b = a;
        b.logits += r0 * a.s0;
        if (tokens) b.tokens += r0;
        if (temperature) b.temperature += r0;
        if (logprobs) b.logprobs += r0;
        if (ranks) b.ranks += r0;
        if (entropy) b.entropy += r0;
        if (top_ids) { b.top_ids += (int64_t)r0 * top; b.top_logprobs += (int64_t)r0 * top; }
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = blocks;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(blocks, rows - r0 < 65535 ? rows - r0 : 65535);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = (cudaStream_t)stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = f32 ? cudaLaunchKernelEx(&cfg, logprobs_kernel<true>, b)
                                  : cudaLaunchKernelEx(&cfg, logprobs_kernel<false>, b);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return MARKOV_ECUDA;
        }
    }
    return MARKOV_OK;
}
