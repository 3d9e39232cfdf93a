// paged_attention.cu -- attention of a chunk of new tokens over a paged
// cache: the simple form, one block per token and query head.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.h"
#include "common.cuh"

namespace dtm {

constexpr int kAttnWarps = 4;

template <bool F16>
__device__ __forceinline__ float elem(uint16_t x) {
    if (F16) return __half2float(__ushort_as_half(x));
    return __uint_as_float((uint32_t)x << 16);
}

template <bool F16>
__device__ __forceinline__ uint16_t rounded(float x) {
    if (F16) return __half_as_ushort(__float2half_rn(x));
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// Each warp takes every fourth visible key with a running maximum, sum and
// weighted value of its own (a lane holds D / 32 elements); the four are
// joined at the end.
template <int D, bool F16>
__global__ void __launch_bounds__(32 * kAttnWarps) paged_attention_kernel(AttnArgs a) {
    constexpr int E = D / 32;
    __shared__ float m_s[kAttnWarps], l_s[kAttnWarps], o_s[kAttnWarps][D];
    if (ld_acquire_u32(a.status) != 0u) return;
    const int t = blockIdx.x, hq = blockIdx.y, hk = hq / a.group;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (t >= a.query_start[a.rows] || t < a.query_start[0]) return;
    int lo = 0, hi = a.rows - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.query_start[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    const int b = lo;
    const int64_t s = a.idx[b];
    if (s < 0) return;
    const int len = a.seq_lens[b], n = a.query_start[b + 1] - a.query_start[b];
    const int pos = len - n + (t - a.query_start[b]);
    const int64_t room = (int64_t)a.width << a.page_shift;
    const int end = s < a.num_states ? (int)(pos + 1 < room ? pos + 1 : room) : 0;
    int first = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
    const int kept = a.sinks < first ? a.sinks : first;
    const int seen = kept + (end > first ? end - first : 0);

    float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = elem<F16>(a.q[t * a.q_s0 + hq * a.q_s1 + lane * E + e]);
        o[e] = 0.0f;
    }
    for (int i = warp; i < seen; i += kAttnWarps) {
        const int key = i < kept ? i : first + i - kept;
        if (key >= end) break;
        const int64_t page = a.table[s * a.table_s0 + (key >> a.page_shift)];
        const int at = key & ((1 << a.page_shift) - 1);
        const bool there = page >= 0 && page < a.num_pages;
        float x = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (there)
                x += q[e] * elem<F16>(a.k[page * a.k_page + at * a.k_slot + hk * a.k_head + lane * E + e]);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        x *= a.scale;
        const float mn = fmaxf(m, x);
        const float keep = mn == -INFINITY ? 1.0f : expf(m - mn);
        const float p = mn == -INFINITY ? 0.0f : expf(x - mn);
        l = l * keep + p;
        m = mn;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float v = there ? elem<F16>(a.v[page * a.v_page + at * a.v_slot + hk * a.v_head + lane * E + e]) : 0.0f;
            o[e] = o[e] * keep + p * v;
        }
    }
    if (lane == 0) { m_s[warp] = m; l_s[warp] = l; }
#pragma unroll
    for (int e = 0; e < E; ++e) o_s[warp][lane * E + e] = o[e];
    __syncthreads();
    float M = -INFINITY, L = 0.0f;
    for (int w = 0; w < kAttnWarps; ++w) M = fmaxf(M, m_s[w]);
    float f[kAttnWarps];
    for (int w = 0; w < kAttnWarps; ++w) {
        f[w] = m_s[w] == -INFINITY ? 0.0f : expf(m_s[w] - M);
        L += f[w] * l_s[w];
    }
    for (int d = threadIdx.x; d < D; d += 32 * kAttnWarps) {
        float x = 0.0f;
        for (int w = 0; w < kAttnWarps; ++w) x += f[w] * o_s[w][d];
        a.out[t * a.out_s0 + hq * a.out_s1 + d] = rounded<F16>(L > 0.0f ? x / L : L == 0.0f ? 0.0f : L);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[(int64_t)t * a.q_heads + hq] = L == 0.0f ? -INFINITY : M + logf(L);
}

cudaError_t launch_paged_attention(const AttnArgs &a, int head_dim, bool f16, cudaStream_t s) {
    const dim3 grid(a.T, a.q_heads);
    if (head_dim == 64 && f16)
        paged_attention_kernel<64, true><<<grid, 32 * kAttnWarps, 0, s>>>(a);
    else if (head_dim == 64)
        paged_attention_kernel<64, false><<<grid, 32 * kAttnWarps, 0, s>>>(a);
    else if (f16)
        paged_attention_kernel<128, true><<<grid, 32 * kAttnWarps, 0, s>>>(a);
    else
        paged_attention_kernel<128, false><<<grid, 32 * kAttnWarps, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace dtm
