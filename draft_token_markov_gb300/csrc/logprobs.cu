// logprobs.cu -- log probabilities of given tokens, rank, entropy and the most
// probable alternatives: one launch and its C ABI.
//
// A block has a row of logits, or a cluster of blocks a slice each where there are
// few rows.  Its threads stream the slice once, four vectors of 16 bytes a turn and
// the next four on their way, without a stop for the block: a thread keeps its own
// maximum m and
//   Z = sum 2^d,  S = sum 2^d d,  d = x c - M,  c = log2(e) / T,  M = m c rounded
// (one fused operation a logit; what the rounding of M is worth is put right at the
// end), the ids before the token, and each turn's maximum in shared memory.  The
// top-th largest of the threads' maxima bounds the alternatives from below; turns
// that reach it are read again (from L2; some 20 of 4000 for 20 alternatives of a row
// of 129280), and what reaches it in them goes to a list, which is put in order by
// counting.  Where the list is too short (many equal logits), the block takes its
// maximum `top` times instead, and a row whose maximum is too large for the fused form
// (kFused) is read again for its sums.  The cluster's first block joins sums and sorted
// lists, which the others write to its shared memory.
//
// ln p = (d - log2 Z) ln 2, entropy = (log2 Z - S / Z) ln 2.
//
// At no unit's limit.  576 rows of 129280 BF16 logits with 20 alternatives (149 MB) take
// 47 us, 47% of the copy rate, as long with every eighth left out; fp32 ones 65 us (298
// MB, 69%); 9 rows in clusters of 8 blocks 11.2 and 13.1 us in a graph.  A multiprocessor that has
// blocks issues 2.2 instructions of 4 a cycle (92 for 256 BF16 logits, all told), its
// warps waiting for loads a third of the time and at the blocks' barriers a fifth; and
// they have blocks 72% of the time, as rows are whole and some take four where others take
// three.  The token is looked at before the first load, which costs 1.6 us of the 47.  (On
// another card, with the load ahead of it, 44 us; there slices in shared memory and read
// three times took 111 us, slices in registers with a bound for the cluster 86, 9 rows
// 9.0; the stream without the next turn on its way 45.4, one logit an instruction 44.8 to
// 45.9; against the maximum of the turn before it takes no less.)
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>

#include "../../include/markov.h"
#include "common.cuh"
#include "f32x2.cuh"
#include "host_util.h"

using namespace dtm;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTurn = 4;                  // vectors of a thread's turn
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr int kList = 512;                // logits that may be among the largest

struct LogprobArgs {
    const uint8_t *logits;
    int64_t s0;                           // bytes
    int vocab, top;
    const int64_t *tokens;
    const float *temperature;
    float *logprobs, *entropy, *top_logprobs;
    int32_t *ranks, *top_ids;
    int slice;                            // vectors of 16 bytes of a block
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
    return F32 ? __uint_as_float(w) : __uint_as_float(word_max<true>(w << 16, w & 0xffff0000u));
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
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of the same variable in a block of the cluster.
__device__ __forceinline__ uint32_t of_block(const void *p, uint32_t block) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(block));
    return r;
}
__device__ __forceinline__ void st_cluster(uint32_t to, uint32_t x) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(x) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t to, uint64_t x) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(x) : "memory");
}

constexpr float kLn2 = 0.69314718055994531f;

// Counts logits above a bound, two at a time where they are BF16 (a count of up to
// 256 in each half is exact).
template <bool F32>
struct Above;
template <>
struct Above<false> {
    __nv_bfloat162 n = __float2bfloat162_rn(0.0f);
    // the bound in both halves
    static __device__ __forceinline__ uint32_t spread(uint32_t bound) { return bound >> 16 | (bound & 0xffff0000u); }
    __device__ __forceinline__ void take(const uint4 &v, uint32_t bound) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162 *>(&bound);
#pragma unroll
        for (int i = 0; i < 4; ++i) n = __hadd2(n, __hgt2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]), b));
    }
    __device__ __forceinline__ int count() const { return (int)(__low2float(n) + __high2float(n)); }
};
template <>
struct Above<true> {
    int n = 0;
    static __device__ __forceinline__ uint32_t spread(uint32_t bound) { return bound; }
    __device__ __forceinline__ void take(const uint4 &v, uint32_t bound) {
        const float b = __uint_as_float(bound);
        n += (__uint_as_float(v.x) > b) + (__uint_as_float(v.y) > b) + (__uint_as_float(v.z) > b) + (__uint_as_float(v.w) > b);
    }
    __device__ __forceinline__ int count() const { return n; }
};

// The bits of the next lower logit of a finite one (fp32 bits; a BF16 one's are the
// upper half).
template <bool F32>
__device__ __forceinline__ uint32_t next_below(float x) {
    const uint32_t one = F32 ? 1u : 0x10000u, b = __float_as_uint(x);
    if ((b & 0x7fffffffu) == 0u) return 0x80000000u | one;
    return b >> 31 ? b + one : b - one;
}

// A vector at a row's end, -inf where the row does not reach; id: of its first logit.
template <bool F32>
__device__ __noinline__ uint4 edge_vector(const uint8_t *from, int id, int vocab) {
    constexpr int kN = F32 ? 4 : 8;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < kN; ++e) {
        const bool there = id + e >= 0 && id + e < vocab;
        if (F32) {
            w[e % 4] = there ? __ldg(reinterpret_cast<const uint32_t *>(from) + id + e) : 0xff800000u;
        } else {
            const uint32_t y = there ? __ldg(reinterpret_cast<const uint16_t *>(from) + id + e) : 0xff80u;
            w[e / 2 % 4] = e & 1 ? w[e / 2 % 4] | y << 16 : y;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// (l - m) c.  The difference of a very negative logit to a large maximum may leave the
// range of fp32 where its product with c does not; the products' signs differ then.
__device__ __forceinline__ float scaled(float l, float m, float c) {
    const float x = l - m;
    return x > -INFINITY || l == -INFINITY ? x * c : __fmul_rn(l, c) - __fmul_rn(m, c);
}

// Rows whose largest |m c| is below this are summed in the fused form.  A thread's d of
// its own maximum is what M's rounding left out, half a unit of M in its last place: 4
// at most there, but 128 from |M| = 2^31 on, as for masked logits of -1e10, and then Z is
// infinite.  M only moves by whole units, so from 2^31 - 128 on every step towards 0
// has the factor 2^-128 or less, that is 0, and what was summed so far is dropped, not
// multiplied: no such sum comes back below 2^31, or into a row's where the maximum is
// below 2^27.
constexpr float kFused = 134217728.0f;

// A thread's logits so far.
template <bool F32>
struct Running {
    float m = -INFINITY, M = 0.0f, z = 0.0f, s = 0.0f;

    // One turn; returns its maximum.
    __device__ __forceinline__ float take(const uint4 (&x)[kTurn], float c) {
        constexpr int kN = F32 ? 4 : 8;
        uint32_t w = word_max<F32>(word_max<F32>(x[0].x, x[0].y), word_max<F32>(x[0].z, x[0].w));
#pragma unroll
        for (int k = 1; k < kTurn; ++k)
            w = word_max<F32>(w, word_max<F32>(word_max<F32>(x[k].x, x[k].y), word_max<F32>(x[k].z, x[k].w)));
        const float top = F32 ? __uint_as_float(w) : __uint_as_float(word_max<true>(w << 16, w & 0xffff0000u));
        if (!(top <= m) && m == m) {                  // larger, or NaN, which stays
            const float next = top * c, back = M - next;
            if (m != -INFINITY) {
                // not a product where the weight is 0: see kFused
                const float f = ex2(back);
                s = f > 0.0f ? f * fmaf(back, z, s) : 0.0f;
                z = f > 0.0f ? f * z : 0.0f;
            }
            m = top;
            M = next;
        }
        if (m == -INFINITY) return top;
        const uint64_t neg = f32x2(-M, -M), c2 = f32x2(c, c);
        uint64_t z2[2] = {0, 0}, s2[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < kTurn; ++k) {
            // a masked logit's 0 times -inf would be NaN: -1e30 times c weighs 0 too where
            // the row's maximum is below kFused / c, and other rows are summed again
            constexpr uint32_t kLow = F32 ? 0xf149f2cau : 0xf149f149u;
            const Logits<F32> l(make_uint4(word_max<F32>(x[k].x, kLow), word_max<F32>(x[k].y, kLow), word_max<F32>(x[k].z, kLow),
                                           word_max<F32>(x[k].w, kLow)));
#pragma unroll
            for (int e = 0; e < kN; e += 2) {
                const uint64_t d = fma2(f32x2(l.x[e], l.x[e + 1]), c2, neg);
                float d0, d1;
                split2(d, d0, d1);
                const uint64_t p = f32x2(ex2(d0), ex2(d1));
                z2[e / 2 & 1] = add2(z2[e / 2 & 1], p);
                s2[e / 2 & 1] = fma2(p, d, s2[e / 2 & 1]);
            }
        }
        float x0, x1, y0, y1;
        split2(add2(z2[0], z2[1]), x0, x1);
        split2(add2(s2[0], s2[1]), y0, y1);
        z += x0 + x1;
        s += y0 + y1;
        return top;
    }
};

template <bool F32>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const __grid_constant__ LogprobArgs a) {
    constexpr int kSize = F32 ? 4 : 2, kN = 16 / kSize, kTurnVectors = kTurn * kThreads;
    extern __shared__ float turn_max[];                                // [turns][kThreads]
    __shared__ Part parts[kMaxCluster];
    __shared__ float warp_f[3][kWarps];
    __shared__ int warp_i[kWarps];
    __shared__ uint64_t warp_k[kWarps];
    __shared__ uint32_t thread_key[kThreads];
    __shared__ uint64_t list[kList];
    __shared__ int listed_s;
    __shared__ uint32_t bound_s;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), blocks = gridDim.x;
    const int64_t row = blockIdx.y;
    const int64_t token64 = a.tokens ? __ldg(a.tokens + row) : 0;

    // the slice: whole vectors from the row's first on, whose first elements may lie
    // before the row
    const uint8_t *from = a.logits + row * a.s0;
    const int lead = (int)(reinterpret_cast<uintptr_t>(from) & 15u) / kSize;
    const int slice0 = (int)rank * a.slice;                            // its first vector
    const int vectors = max(min(a.slice, (a.vocab + lead + kN - 1) / kN - slice0), 0);
    const int whole0 = slice0 == 0 && lead > 0 ? 1 : 0;                // vectors that lie in the row, whole
    const int whole = min(vectors, (a.vocab + lead) / kN - slice0) - whole0;
    const int first_id = slice0 * kN - lead;                           // of the slice's first vector
    const uint8_t *at0 = from + (int64_t)first_id * kSize;
    constexpr uint32_t kNone = F32 ? 0xff800000u : 0xff80ff80u;
    const auto load1 = [&](int v) {
        if ((uint32_t)(v - whole0) < (uint32_t)whole && whole > 0) return __ldg(reinterpret_cast<const uint4 *>(at0) + v);
        if (v < vectors) return edge_vector<F32>(from, first_id + v * kN, a.vocab);
        return make_uint4(kNone, kNone, kNone, kNone);
    };
    const uint4 *mine = reinterpret_cast<const uint4 *>(at0) + tid;
    const auto load = [&](uint4 (&x)[kTurn], int turn) {
        const int v0 = turn * kTurnVectors;
        if (v0 >= whole0 && v0 + kTurnVectors <= whole0 + whole) {
#pragma unroll
            for (int k = 0; k < kTurn; ++k) x[k] = __ldg(mine + v0 + k * kThreads);
        } else {
#pragma unroll
            for (int k = 0; k < kTurn; ++k) x[k] = load1(v0 + k * kThreads + tid);
        }
    };
    // f(logit, id) of the slice's logits, read again: for what is rare
    const auto each = [&](const auto &f) {
        const int id1 = min(first_id + vectors * kN, a.vocab);
#pragma unroll 1
        for (int id = max(first_id, 0) + tid; id < id1; id += kThreads)
            f(F32 ? __ldg(reinterpret_cast<const float *>(from) + id)
                  : __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(from) + id) << 16),
              id);
    };
    uint4 x[kTurn], y[kTurn];
    const int turns = (vectors + kTurnVectors - 1) / kTurnVectors;
    // the whole cluster, before the first load: a row that is left out is not read
    if (token64 < 0 || token64 >= a.vocab) return;
    if (turns > 0) load(x, 0);
    if (blocks > 1) cluster_arrive();                                  // every block runs
    const int token = (int)token64;
    float T = a.temperature ? __ldg(a.temperature + row) : 1.0f;
    if (!samples(T)) T = 1.0f;
    float own = 0.0f;
    if (a.tokens)
        own = F32 ? __ldg(reinterpret_cast<const float *>(from) + token)
                  : __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(from) + token) << 16);
    // finite, and not 0: with T = inf the difference of finite logits vanishes, -inf stays
    const float c = fmaxf(fminf(__fdiv_rn(1.4426950408889634f, T), 3.0e38f), 1.401298464e-45f);
    if (tid == 0) listed_s = 0;

    // ------------------------------------------------------------- the stream
    // equal logits come before the token where their ids are lower
    const bool ranked = a.tokens && fabsf(own) < INFINITY;
    const uint32_t equal = Above<F32>::spread(__float_as_uint(own)), below = Above<F32>::spread(next_below<F32>(own));
    Running<F32> r;
    Above<F32> above;
    int before = 0;
    const auto take = [&](const uint4 (&x)[kTurn], int turn) {
        turn_max[turn * kThreads + tid] = r.take(x, c);
        if (!ranked) return;
        // the turn lies before the token, behind it or around it
        const int id = first_id + turn * kTurnVectors * kN;
        if (token < id || token >= id + kTurnVectors * kN) {
            const uint32_t bound = token < id ? equal : below;
#pragma unroll
            for (int k = 0; k < kTurn; ++k) above.take(x[k], bound);
        } else {
#pragma unroll
            for (int k = 0; k < kTurn; ++k) {
                const int at = id + (k * kThreads + tid) * kN;
                const Logits<F32> l(x[k]);
#pragma unroll
                for (int e = 0; e < kN; ++e) before += at + e < token ? l.x[e] >= own : l.x[e] > own;
            }
        }
        // BF16 counts are exact up to 256 in each half
        if ((turn & 7) == 7) {
            before += above.count();
            above = Above<F32>();
        }
    };
#pragma unroll 1
    for (int turn = 0; turn < turns; turn += 2) {
        if (turn + 1 < turns) load(y, turn + 1);
        take(x, turn);
        if (turn + 1 == turns) break;
        if (turn + 2 < turns) load(x, turn + 2);
        take(y, turn + 1);
    }
    before += above.count();
    thread_key[tid] = ordered_key(r.m);
    float m = r.m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = nan_max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) warp_f[0][warp] = m;
    __syncthreads();
    m = warp_f[0][0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = nan_max(m, warp_f[0][w]);
    const bool odd = !(fabsf(m) < INFINITY);                           // NaN, an infinity, nothing
    // what the fused form cannot do: scales and logits that leave its range
    const bool plain = !(fabsf(m * c) < kFused) || c < 1e-20f || c > 1e7f;
    float z = 0.0f, s = 0.0f;
    uint64_t best = 0;
    if (!odd && !plain) {
        if (r.m != -INFINITY) {
            // relative to the slice's maximum, and to m c instead of M
            const float off = fmaf(r.m, c, -r.M), d = fmaf(r.m - m, c, -off), f = ex2(d);
            s = f > 0.0f ? f * fmaf(d, r.z, r.s) : 0.0f;
            z = f > 0.0f ? f * r.z : 0.0f;
        }
    } else if (!odd) {
        // a thread's terms one after the other, often equal ones: what a sum's rounding
        // leaves out is kept and goes into the next
        float z_off = 0.0f, s_off = 0.0f;
        const auto add = [](float &sum, float &off, float x) {
            const float y = __fadd_rn(x, -off), t = __fadd_rn(sum, y);
            off = __fadd_rn(__fadd_rn(t, -sum), -y);
            sum = t;
        };
        each([&](float l, int) {
            const float d = scaled(l, m, c), p = ex2(d);
            add(z, z_off, p);
            add(s, s_off, d > -1024.0f ? p * d : 0.0f);
        });
    }
    const bool by_key = a.tokens && (odd || !ranked);                  // NaN or an infinity in the comparison
    if (odd || by_key) {
        if (by_key) before = 0;
        const uint64_t own_key = a.tokens ? pack_key(own, (uint32_t)token) : 0;
        each([&](float l, int id) {
            const uint64_t k = pack_key(l, (uint32_t)id);
            if (by_key) before += k > own_key;
            if (odd) best = k > best ? k : best;
        });
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, o);
        s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    before = __reduce_add_sync(0xffffffffu, before);
    if (odd) best = warp_max_key(best);
    if (lane == 0) {
        warp_f[1][warp] = z;
        warp_f[2][warp] = s;
        warp_i[warp] = before;
        warp_k[warp] = best;
    }
    if (a.top > 0 && warp == 0) {
        // the top-th largest of the threads' maxima, eight a lane
        static_assert(kWarps == 8, "the network");
        uint32_t g[kWarps], key = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) g[w] = thread_key[w * 32 + lane];
        // a lane's in falling order (a network of 19 exchanges), then the first of all
        constexpr uint8_t kNetwork[19][2] = {{0, 2}, {1, 3}, {4, 6}, {5, 7}, {0, 4}, {1, 5}, {2, 6}, {3, 7}, {0, 1}, {2, 3},
                                             {4, 5}, {6, 7}, {2, 4}, {3, 5}, {1, 4}, {3, 6}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
        for (int e = 0; e < 19; ++e) {
            const uint32_t hi = max(g[kNetwork[e][0]], g[kNetwork[e][1]]), lo = min(g[kNetwork[e][0]], g[kNetwork[e][1]]);
            g[kNetwork[e][0]] = hi;
            g[kNetwork[e][1]] = lo;
        }
        for (int i = 0; i < a.top; ++i) {
            key = __reduce_max_sync(0xffffffffu, g[0]);
            const uint32_t who = __ballot_sync(0xffffffffu, g[0] == key);
            if (lane == __ffs(who) - 1) {
#pragma unroll
                for (int w = 0; w + 1 < kWarps; ++w) g[w] = g[w + 1];
                g[kWarps - 1] = 0;
            }
        }
        if (lane == 0) bound_s = key;
    }
    if (blocks > 1) cluster_wait();                                    // the first block runs
    __syncthreads();

    // --------------------------------------------------------- alternatives
    const uint32_t part_at = of_block(parts + rank, 0);
    const auto put = [&](int n, uint64_t k) { st_cluster(part_at + (uint32_t)offsetof(Part, top) + 8 * n, k); };
    if (a.top > 0) {
        const float bound = key_from_ordered(bound_s);
        bool slow = m != m || m == INFINITY;                           // NaN and infinities: by their keys
        int listed = 0;
        if (!slow) {
            const float least = fmaxf(bound, -3.402823466e38f);        // masked logits are not listed
            if (r.m >= least) {
#pragma unroll 1
                for (int turn = 0; turn < turns; ++turn) {
                    if (!(turn_max[turn * kThreads + tid] >= least)) continue;
#pragma unroll 1
                    for (int k = 0; k < kTurn; ++k) {
                        const uint4 v = load1(turn * kTurnVectors + k * kThreads + tid);
                        if (!(vector_max<F32>(v) >= least)) continue;
                        const int id = first_id + (turn * kTurnVectors + k * kThreads + tid) * kN;
                        const Logits<F32> l(v);
#pragma unroll
                        for (int e = 0; e < kN; ++e)
                            if (l.x[e] >= least) {
                                const int at = atomicAdd(&listed_s, 1);
                                if (at < kList) list[at] = pack_key(l.x[e], (uint32_t)(id + e));
                            }
                    }
                }
            }
            __syncthreads();
            listed = listed_s;
            slow = listed > kList;
        }
        if (!slow && listed < a.top && bound == -INFINITY) {
            // masked ids follow by their number: those of the first 32 vectors are enough, or the slow way
            __syncthreads();                                           // listed_s is read
            if (warp == 0) {
                uint32_t masked = 0;
                const Logits<F32> l(load1(lane));
                const int id = first_id + lane * kN;
#pragma unroll
                for (int e = 0; e < kN; ++e)
                    if (lane < vectors && l.x[e] == -INFINITY && id + e >= 0 && id + e < a.vocab) masked |= 1u << e;
                int at = __popc(masked);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int n = __shfl_up_sync(0xffffffffu, at, o);
                    if (lane >= o) at += n;
                }
                const int all = __shfl_sync(0xffffffffu, at, 31);
                at -= __popc(masked);
#pragma unroll
                for (int e = 0; e < kN; ++e)
                    if (masked >> e & 1) {
                        if (at < a.top) list[listed + at] = pack_key(-INFINITY, (uint32_t)(id + e));
                        ++at;
                    }
                if (lane == 0) listed_s = all >= a.top || vectors <= 32 ? listed + min(all, a.top) : kList + 1;
            }
            __syncthreads();
            listed = listed_s;
            slow = listed > kList;
        }
        if (!slow) {
            // in order, by counting; by one warp where the others would not help
            const int step = listed > 64 ? kThreads : 32;
            for (int i = tid; i < listed && tid < step; i += step) {
                const uint64_t k = list[i];
                int n = 0;
                for (int j = 0; j < listed; ++j) n += list[j] > k;
                if (n < a.top) put(n, k);
            }
            if (tid < a.top && tid >= listed) put(tid, 0);
        } else {
            __syncthreads();                                           // the list is read
            uint64_t last = 1;
            for (int n = 0; n < a.top; ++n) {
                uint64_t most = 0;
                if (last != 0)
                    each([&](float l, int id) {
                        const uint64_t k = pack_key(l, (uint32_t)id);
                        if (n == 0 || k < last) most = k > most ? k : most;
                    });
                most = warp_max_key(most);
                if (lane == 0) list[warp] = most;
                __syncthreads();
                last = 0;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) last = list[w] > last ? list[w] : last;
                if (tid == 0) put(n, last);
                __syncthreads();
            }
        }
    }

    // ------------------------------------------------------------ the parts
    if (warp == kWarps - 1) {
        z = lane < kWarps ? warp_f[1][lane] : 0.0f;
        s = lane < kWarps ? warp_f[2][lane] : 0.0f;
        before = lane < kWarps ? warp_i[lane] : 0;
        best = lane < kWarps ? warp_k[lane] : 0;
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) {
            z += __shfl_xor_sync(0xffffffffu, z, o);
            s += __shfl_xor_sync(0xffffffffu, s, o);
        }
        before = __reduce_add_sync(0xffffffffu, before);
        if (odd) best = warp_max_key(best);
        if (lane == 0) {
            st_cluster(part_at + offsetof(Part, m), __float_as_uint(m));
            st_cluster(part_at + offsetof(Part, z), __float_as_uint(z));
            st_cluster(part_at + offsetof(Part, s), __float_as_uint(s));
            st_cluster(part_at + offsetof(Part, before), (uint32_t)before);
            st_cluster(part_at + offsetof(Part, best), best);
        }
    }
    if (blocks > 1) {
        cluster_arrive();
        if (rank != 0) return;
        cluster_wait();
    } else {
        __syncthreads();
    }

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
        const float d = scaled(p.m, all, c), f = ex2(d);
        z += p.z * f;
        s += f > 0.0f ? f * (p.s + d * p.z) : 0.0f;
    }
    const float log_z = one_hot ? 0.0f : log2f(z);
    const auto log_p = [&](float l, int id) {
        if (one_hot) return id == (int)packed_id(best) ? 0.0f : -INFINITY;
        if (l == -INFINITY) return l;
        const float x = l - all, d = scaled(l, all, c);
        if (d > -INFINITY) return (d - log_z) * kLn2;
        // a logit of the type's lowest value leaves the range of d (and of x: see scaled)
        return x > -INFINITY ? __fdiv_rn(x, T) : __fdiv_rn(l, T) - __fdiv_rn(all, T);
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

// Lets the kernels take what a call may need, once a device.
constexpr int kMostShared = 80 << 10;     // 262144 fp32 logits: 65 turns of 1 KB

bool allow_shared_memory(int device, int &multiprocessors) {
    static std::atomic<int> known[64];
    const bool kept = device < 64;
    if (kept && (multiprocessors = known[device].load(std::memory_order_relaxed)) > 0) return true;
    for (const void *fn : {(const void *)logprobs_kernel<false>, (const void *)logprobs_kernel<true>})
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared) != cudaSuccess) return false;
    if (cudaDeviceGetAttribute(&multiprocessors, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return false;
    if (kept) known[device].store(multiprocessors, std::memory_order_relaxed);
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
    int multiprocessors = 0;
    if (!allow_shared_memory(at.device, multiprocessors)) {
        cudaGetLastError();
        return MARKOV_ECUDA;
    }
    // whole vectors, the first of which may begin before the row; a cluster a row while
    // its blocks find a place, four to a multiprocessor, and have a turn to do
    const int vectors = (int)(((int64_t)vocab * size + 15) / 16) + 1;
    int blocks = 1;
    while (blocks < kMaxCluster && (int64_t)rows * blocks * 2 <= 4 * multiprocessors && vectors > 2 * blocks * kTurn * kThreads)
        blocks *= 2;
    a.slice = (vectors + blocks - 1) / blocks;
    const int turns = (a.slice + kTurn * kThreads - 1) / (kTurn * kThreads);
    const void *fn = f32 ? (const void *)logprobs_kernel<true> : (const void *)logprobs_kernel<false>;
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
        cfg.dynamicSmemBytes = turns * kThreads * sizeof(float);
        cfg.stream = (cudaStream_t)stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        void *params[1] = {&b};
        if (cudaLaunchKernelExC(&cfg, fn, params) != cudaSuccess) {
            cudaGetLastError();
            return MARKOV_ECUDA;
        }
    }
    return MARKOV_OK;
}
