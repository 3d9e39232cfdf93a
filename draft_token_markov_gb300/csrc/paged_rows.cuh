// paged_rows.cuh -- the rows of a call over a paged cache as the e4m3 attention
// kernels see them, and the cut of its work into ranges.
#pragma once
#include <cstdint>

#include "paged.h"

namespace dtm {

struct RowOfCall {
    int np, qs;                // tokens that there are queries for, the first
    int pos0;                  // position of its token 0
    int state;                 // its table row, -1 for none
};

__device__ __forceinline__ RowOfCall row_of_call(const PagedRows &a, int r) {
    const int64_t state = __ldg(a.idx + r);
    const int qe = __ldg(a.query_start + r + 1), len = __ldg(a.seq_lens + r);
    RowOfCall q;
    q.qs = __ldg(a.query_start + r);
    const int n = qe - q.qs;
    q.np = state < 0 || q.qs < 0 || q.qs >= a.T || n < 0 ? 0 : min(n, a.T - q.qs);
    q.pos0 = max(len, 0) - n;
    q.state = state < a.num_states ? (int)state : -1;
    return q;
}

// The keys that the tokens at positions [p0, p1] see, in pieces of 2^SHIFT keys:
// the window's and, before it, those of the first tokens that are kept.
struct KeySpan {
    int end, first, kept;      // some token sees keys [first, end) and [0, kept)
    int sinks, w0;             // pieces: [0, sinks), then from w0 on
    int steps;                 // pieces together

    // The first key of the j-th piece.
    template <int SHIFT>
    __device__ __forceinline__ int key(int j) const {
        return (j < sinks ? j : w0 + j - sinks) << SHIFT;
    }
};

__device__ __forceinline__ int window_start(int window, int pos) {
    return window > 0 && pos >= window ? pos - window + 1 : 0;
}

template <int SHIFT>
__device__ __forceinline__ KeySpan key_span(const PagedRows &a, int window, int sinks, int state, int p0, int p1) {
    constexpr int kPiece = 1 << SHIFT;
    KeySpan s;
    s.end = state < 0 ? 0 : max(0, p1 >= a.room ? a.room : p1 + 1);
    s.first = window_start(window, p0);
    s.kept = min(min(sinks, s.first), s.end);
    s.w0 = s.first >> SHIFT;
    const int nw = s.first < s.end ? ((s.end + kPiece - 1) >> SHIFT) - s.w0 : 0;
    s.sinks = (s.kept + kPiece - 1) >> SHIFT;
    if (nw > 0 && s.sinks > s.w0) s.sinks = s.w0;
    s.steps = s.sinks + nw;
    return s;
}

// The call's units cut into ranges of equal length, the first `rem` one longer.
struct UnitSplit {
    uint64_t base;
    uint32_t ranges, rem;

    // at most `most` ranges, of `least` units each or more
    __device__ __forceinline__ void cut(uint64_t total, uint32_t most, uint32_t least) {
        ranges = total == 0 ? 0u : (uint32_t)max((uint64_t)1, min((uint64_t)most, total / least));
        base = ranges ? total / ranges : 0;
        rem = (uint32_t)(total - base * ranges);
    }
    __device__ __forceinline__ uint64_t first(uint32_t c) const { return c * base + min(c, rem); }
    __device__ __forceinline__ int range_of(uint64_t u) const {
        const uint64_t longer = rem * (base + 1);
        return (int)(u < longer ? u / (base + 1) : rem + (u - longer) / base);
    }
};

}  // namespace dtm
