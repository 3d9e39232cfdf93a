// rotary.cu -- rotary positions of queries and keys: the plan's frequencies
// (host), one launch that turns both (device), and their C ABI.
//
// The angle of pair i at position p is p f_i.  Frequencies are kept as turns
// per position in units of 2^-64, as integers: the product with the position
// wraps at whole turns, so its upper 32 bits are the angle within a turn
// whatever the position (an fp32 angle of position 10^6 would be off by 0.03
// radians; fp64 ones run at a fraction of the rate here).
//
// A block takes the sines and cosines of its tokens to shared memory, amplitude
// included, then walks their heads in 16-byte vectors (half layout: the vector
// and its partner rot_dim / 2 further on).  Bound by memory: each element is
// read and written once; 8191 tokens of 40 heads of 128 (168 MB) take 30 us, 84% of the
// copy rate, with 8 tokens a block and 4 vectors in flight a thread (31 us with 4
// tokens, 33 with 2; 35 with 2 vectors); 72 tokens 2.9 us in a graph.  The same 40 heads
// in fp32 (335 MB) take 58 us, 86%, and 72 tokens 3.3 to 3.6 us.
#include <cmath>
#include <cstdint>
#include <new>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/markov.h"
#include "host_util.h"

using namespace dtm;

struct markov_rotary_plan {
    markov_rotary_desc d;
    float amplitude = 1.0f;
    uint64_t *turns = nullptr;    // [rot_dim / 2]
};

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;     // tokens of a block
constexpr int kUnroll = 4;        // vectors that a thread has in flight

// n / d for 32-bit n by a multiplication (d >= 1): exact for n < 2^31.
struct Div {
    uint32_t d, mul, shift;
    __host__ static Div of(uint32_t d) {
        uint32_t s = 0;
        while ((1u << s) < d) ++s;
        return Div{d, (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - d)) / d + 1), s};
    }
    __device__ __forceinline__ uint32_t quotient(uint32_t n) const {
        return (__umulhi(n, mul) + n) >> shift;
    }
};

struct Side {
    const char *src;
    char *dst;
    int64_t src_s0, src_s1, dst_s0, dst_s1;   // bytes
};

struct RotaryArgs {
    Side q, k;
    int q_heads, tokens, tile;    // tile: tokens of a block
    const int32_t *positions;
    const uint64_t *turns;
    float amplitude;
    int pairs, turned;            // rot_dim / 2; vectors that turn (the rest is copied)
    Div heads, vectors;           // of all heads together; of a head
};

template <typename T>
struct Vec;                       // 8 elements
template <>
struct Vec<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const char *p) { v = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void store(char *p) const { __stcs(reinterpret_cast<uint4 *>(p), v); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec<__half> {
    uint4 v;
    __device__ __forceinline__ void load(const char *p) { v = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void store(char *p) const { __stcs(reinterpret_cast<uint4 *>(p), v); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const char *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void store(char *p) const {
        *reinterpret_cast<float4 *>(p) = a;
        *(reinterpret_cast<float4 *>(p) + 1) = b;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
};

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
    extern __shared__ __align__(16) float2 turn[];    // [tile][pairs] cosine and sine
    const int t0 = blockIdx.x * a.tile, tokens = min(a.tile, a.tokens - t0);
    for (int i = threadIdx.x; i < tokens * a.pairs; i += kThreads) {
        const int t = i / a.pairs;
        const int64_t p = a.positions[t0 + t];
        const uint64_t phase = (uint64_t)p * a.turns[i - t * a.pairs];
        float s, c;
        // the angle in half turns
        sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &s, &c);
        turn[i] = make_float2(c * a.amplitude, s * a.amplitude);
    }
    __syncthreads();
    const uint32_t n = (uint32_t)tokens * a.heads.d * a.vectors.d;
    constexpr int kPartner = INTERLEAVED ? 0 : 1;
    for (uint32_t i0 = threadIdx.x; i0 < n; i0 += kThreads * kUnroll) {
        Vec<T> x[kUnroll][1 + kPartner];
        char *dst[kUnroll];
        int vec[kUnroll], tok[kUnroll];
#pragma unroll
        for (int e = 0; e < kUnroll; ++e) {
            const uint32_t i = i0 + e * kThreads;
            if (i >= n) break;
            const uint32_t th = a.vectors.quotient(i), t = a.heads.quotient(th);
            const int v = (int)(i - th * a.vectors.d), h = (int)(th - t * a.heads.d);
            const Side &s = h < a.q_heads ? a.q : a.k;
            const int head = h < a.q_heads ? h : h - a.q_heads;
            const bool turns = v < a.turned;
            // the first element of the vector; what is copied lies behind the pairs
            const int64_t at = (turns ? v * 8 : 2 * a.pairs + (v - a.turned) * 8) * (int)sizeof(T);
            const char *src = s.src + (int64_t)(t0 + t) * s.src_s0 + head * s.src_s1 + at;
            dst[e] = s.dst + (int64_t)(t0 + t) * s.dst_s0 + head * s.dst_s1 + at;
            vec[e] = turns ? v : -1;
            tok[e] = t;
            x[e][0].load(src);
            if (!INTERLEAVED && turns) x[e][kPartner].load(src + a.pairs * (int)sizeof(T));
        }
#pragma unroll
        for (int e = 0; e < kUnroll; ++e) {
            if (i0 + e * kThreads >= n) break;
            if (vec[e] < 0) {
                x[e][0].store(dst[e]);
                continue;
            }
            // two pairs' cosines and sines in each
            const float4 *cs = reinterpret_cast<const float4 *>(turn + tok[e] * a.pairs + vec[e] * (INTERLEAVED ? 4 : 8));
            if (INTERLEAVED) {
                float y[8], z[8];
                x[e][0].get(y);
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const float4 w = cs[j / 2];
                    z[2 * j] = y[2 * j] * w.x - y[2 * j + 1] * w.y;
                    z[2 * j + 1] = y[2 * j + 1] * w.x + y[2 * j] * w.y;
                    z[2 * j + 2] = y[2 * j + 2] * w.z - y[2 * j + 3] * w.w;
                    z[2 * j + 3] = y[2 * j + 3] * w.z + y[2 * j + 2] * w.w;
                }
                x[e][0].put(z);
                x[e][0].store(dst[e]);
            } else {
                float y[8], z[8], u[8], w[8];
                x[e][0].get(y);
                x[e][kPartner].get(z);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float4 r = cs[j / 2];
                    u[j] = y[j] * r.x - z[j] * r.y;
                    w[j] = z[j] * r.x + y[j] * r.y;
                    u[j + 1] = y[j + 1] * r.z - z[j + 1] * r.w;
                    w[j + 1] = z[j + 1] * r.z + y[j + 1] * r.w;
                }
                x[e][0].put(u);
                x[e][kPartner].put(w);
                x[e][0].store(dst[e]);
                x[e][kPartner].store(dst[e] + a.pairs * (int)sizeof(T));
            }
        }
    }
}

// A frequency in radians as turns in units of 2^-64: f / (2 pi) in two doubles,
// f h + (its rounding error + f l).
uint64_t turns_of(double f) {
    const double h = 0.15915494309189535, l = -9.839338337591243e-18;
    const double p = f * h, e = std::fma(f, h, -p) + f * l;
    const double top = std::floor(p * 4294967296.0);
    const double rest = p * 4294967296.0 - top;             // exact: p has 53 bits
    const double low = std::nearbyint((rest + e * 4294967296.0) * 4294967296.0);
    return ((uint64_t)(int64_t)top << 32) + (uint64_t)(int64_t)low;
}

bool positive(double x) { return std::isfinite(x) && x > 0.0; }

// The angle per position of pair i; the desc is valid.
double frequency(const markov_rotary_desc &d, int i) {
    if (d.scaling == MARKOV_ROTARY_GIVEN) return d.frequencies[i];
    const double pi = 3.14159265358979323846, rot = d.rot_dim;
    const double theta = d.scaling == MARKOV_ROTARY_BASE ? d.theta * std::pow(d.factor, rot / (rot - 2.0)) : d.theta;
    const double f = std::pow(theta, -2.0 * i / rot);
    if (d.scaling == MARKOV_ROTARY_LINEAR) return f / d.factor;
    if (d.scaling == MARKOV_ROTARY_PARTS) {
        auto dim = [&](double r) { return rot * std::log(d.original_len / (2.0 * pi * r)) / (2.0 * std::log(d.theta)); };
        const double a = std::fmax(std::floor(dim(d.high)), 0.0), b = std::fmin(std::ceil(dim(d.low)), rot - 1.0);
        const double t = std::fmin(std::fmax((i - a) / std::fmax(b - a, 0.001), 0.0), 1.0);
        return f / d.factor * t + f * (1.0 - t);
    }
    if (d.scaling == MARKOV_ROTARY_WAVELENGTH) {
        const double t = std::fmin(std::fmax((d.original_len * f / (2.0 * pi) - d.low) / (d.high - d.low), 0.0), 1.0);
        return f * t + f / d.factor * (1.0 - t);
    }
    return f;
}

bool valid_desc(const markov_rotary_desc &d) {
    if (d.head_dim < 16 || d.head_dim > 512 || d.head_dim % 16 != 0) return false;
    if (d.rot_dim < 16 || d.rot_dim > d.head_dim || d.rot_dim % 16 != 0) return false;
    if (d.interleaved != 0 && d.interleaved != 1) return false;
    if (!std::isfinite(d.amplitude) || d.amplitude < 0.0) return false;
    if (d.scaling == MARKOV_ROTARY_GIVEN) {
        if (!d.frequencies) return false;
        for (int i = 0; i < d.rot_dim / 2; ++i)
            if (!(std::fabs(d.frequencies[i]) <= 6.2831853071795865)) return false;
        return true;
    }
    if (d.scaling < MARKOV_ROTARY_NONE || d.scaling > MARKOV_ROTARY_WAVELENGTH) return false;
    if (!positive(d.theta) || d.theta <= 1.0) return false;
    if (d.scaling == MARKOV_ROTARY_NONE) return true;
    if (!positive(d.factor)) return false;
    if (d.scaling == MARKOV_ROTARY_PARTS || d.scaling == MARKOV_ROTARY_WAVELENGTH)
        if (!positive(d.original_len) || !positive(d.low) || !positive(d.high) || d.low >= d.high) return false;
    // stretched the other way, a pair may turn more than once a position
    for (int i = 0; i < d.rot_dim / 2; ++i)
        if (!(std::fabs(frequency(d, i)) <= 6.2831853071795865)) return false;
    return true;
}

template <typename T>
cudaError_t launch(const RotaryArgs &a, bool interleaved, int grid, size_t smem, cudaStream_t s) {
    if (interleaved)
        rotary_kernel<T, true><<<grid, kThreads, smem, s>>>(a);
    else
        rotary_kernel<T, false><<<grid, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

extern "C" {

markov_status markov_rotary_plan_create(const markov_rotary_desc *desc, markov_rotary_plan **out) {
    if (!out) return MARKOV_EINVAL;
    *out = nullptr;
    if (!desc || !valid_desc(*desc)) return MARKOV_EINVAL;
    const markov_rotary_desc d = *desc;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || d.device < 0 || d.device >= ndev) {
        cudaGetLastError();
        return MARKOV_EDEVICE;
    }
    DeviceGuard guard(d.device);
    if (!guard.ok) return MARKOV_EDEVICE;
    markov_rotary_plan *p = new (std::nothrow) markov_rotary_plan();
    if (!p) return MARKOV_ECUDA;
    p->d = d;
    p->d.frequencies = nullptr;                   // the caller's, not kept
    if (d.amplitude > 0.0)
        p->amplitude = (float)d.amplitude;
    else if (d.scaling == MARKOV_ROTARY_PARTS && d.factor > 1.0)
        p->amplitude = (float)(0.1 * std::log(d.factor) + 1.0);
    uint64_t turns[256];
    const int pairs = d.rot_dim / 2;
    for (int i = 0; i < pairs; ++i) turns[i] = turns_of(frequency(d, i));
    // a copy from pageable memory may return before it has arrived, and the plan's calls run
    // on streams that do not wait for the default one
    if (cudaMalloc(&p->turns, pairs * sizeof(uint64_t)) != cudaSuccess ||
        cudaMemcpy(p->turns, turns, pairs * sizeof(uint64_t), cudaMemcpyHostToDevice) != cudaSuccess ||
        cudaStreamSynchronize(nullptr) != cudaSuccess) {
        cudaGetLastError();
        if (p->turns) cudaFree(p->turns);
        delete p;
        return MARKOV_ECUDA;
    }
    *out = p;
    return MARKOV_OK;
}

void markov_rotary_plan_destroy(markov_rotary_plan *p) {
    if (!p) return;
    DeviceGuard guard(p->d.device);
    cudaDeviceSynchronize();
    cudaFree(p->turns);
    delete p;
}

markov_status markov_rotary(markov_rotary_plan *p, const void *q, int64_t q_s0, int64_t q_s1,
                            int32_t q_heads, const void *k, int64_t k_s0, int64_t k_s1,
                            int32_t k_heads, markov_dtype dtype, const int32_t *positions,
                            int32_t num_tokens, void *q_out, int64_t qo_s0, int64_t qo_s1,
                            void *k_out, int64_t ko_s0, int64_t ko_s1, void *stream) {
    if (!p || num_tokens < 0 || q_heads < 0 || k_heads < 0 || (int64_t)q_heads + k_heads < 1) return MARKOV_EINVAL;
    if (dtype != MARKOV_BF16 && dtype != MARKOV_F16 && dtype != MARKOV_F32) return MARKOV_EINVAL;
    if ((int64_t)q_heads + k_heads > 4096) return MARKOV_EINVAL;
    const int heads = q_heads + k_heads;
    if ((int64_t)num_tokens * heads > INT32_MAX) return MARKOV_EINVAL;
    if (num_tokens == 0) return MARKOV_OK;
    if (!positions) return MARKOV_EINVAL;
    const int size = dtype == MARKOV_F32 ? 4 : 2, per16 = 16 / size;
    auto valid = [&](const void *x, int64_t s0, int64_t s1, int n) {
        return x && aligned16(x) && s0 >= 0 && (n == 1 || s1 >= p->d.head_dim) && s1 >= 0 && s0 % per16 == 0 &&
               s1 % per16 == 0;
    };
    if (q_heads && (!valid(q, q_s0, q_s1, q_heads) || !valid(q_out, qo_s0, qo_s1, q_heads))) return MARKOV_EINVAL;
    if (k_heads && (!valid(k, k_s0, k_s1, k_heads) || !valid(k_out, ko_s0, ko_s1, k_heads))) return MARKOV_EINVAL;
    const bool q_here = q == q_out || !q_heads, k_here = k == k_out || !k_heads;
    if ((q_heads && q_here && (q_s0 != qo_s0 || q_s1 != qo_s1)) || (k_heads && k_here && (k_s0 != ko_s0 || k_s1 != ko_s1)))
        return MARKOV_EINVAL;
    DeviceGuard guard(p->d.device);
    if (!guard.ok) return MARKOV_EDEVICE;
    RotaryArgs a{};
    auto side = [&](const void *x, int64_t s0, int64_t s1, void *y, int64_t o0, int64_t o1) {
        return Side{static_cast<const char *>(x), static_cast<char *>(y), s0 * size, s1 * size, o0 * size, o1 * size};
    };
    a.q = side(q, q_s0, q_s1, q_out, qo_s0, qo_s1);
    a.k = side(k, k_s0, k_s1, k_out, ko_s0, ko_s1);
    a.q_heads = q_heads;
    a.tokens = num_tokens;
    a.positions = positions;
    a.turns = p->turns;
    a.amplitude = p->amplitude;
    a.pairs = p->d.rot_dim / 2;
    a.turned = p->d.interleaved ? p->d.rot_dim / 8 : p->d.rot_dim / 16;
    a.heads = Div::of(heads);
    // nothing is copied in place
    a.vectors = Div::of(a.turned + (q_here && k_here ? 0 : (p->d.head_dim - p->d.rot_dim) / 8));
    // a token a block spreads short calls; in us, with 8 + 1 heads of 128 in BF16: 4096 tokens
    // by eight a block 7.3, 4095 by one 12.7, and 2048 by one 6.2
    a.tile = num_tokens >= 4096 ? kMaxTokens : 1;
    const int grid = (num_tokens + a.tile - 1) / a.tile;
    const size_t smem = (size_t)a.tile * a.pairs * sizeof(float2);
    const cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == MARKOV_F32 ? launch<float>(a, p->d.interleaved, grid, smem, s)
                          : dtype == MARKOV_F16 ? launch<__half>(a, p->d.interleaved, grid, smem, s)
                                                : launch<__nv_bfloat16>(a, p->d.interleaved, grid, smem, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return MARKOV_ECUDA;
    }
    return MARKOV_OK;
}

}  // extern "C"
