// paged.h -- structures shared by the verify step's host code and kernels
// (paged layout, paged writes, attention over the paged cache, acceptance).
#pragma once
#include <cstdint>

#include <cuda_runtime.h>

#include "internal.h"

namespace dtm {

constexpr int kPagedMaxRows = 1024;    // request rows of a paged call

struct LayoutArgs {
    const int32_t *context, *query;
    const int64_t *idx;
    int rows;
    int32_t *table;
    int64_t table_s0;
    int num_states, width, page_shift;
    int64_t room;              // tokens that a row may have: positions are 32 bits
    const int32_t *held;
    int32_t *ring;
    int64_t ring_size;
    const int64_t *free_in;
    int32_t *held_out;
    int64_t *free_out;
    int32_t *query_start, *seq_lens, *positions;
    int64_t *slots;
    int T;
    const uint32_t *status;
    uint32_t *arrivals;        // blocks done; zero between calls
};

// One side of a paged write: [T, heads, D] into a paged cache.
struct WriteSide {
    const uint4 *src;
    int64_t src_s0, src_s1;    // in 16-byte units, as all strides here
    uint4 *dst;
    int64_t s_page, s_slot, s_head;
};

struct WriteArgs {
    WriteSide k, v;
    const int64_t *slots;
    int64_t num_slots;
    int T, heads, vec_shift, page_shift;
    const uint32_t *status;
};

struct AttnArgs {
    int negate;                // the scale is negative
    const int32_t *table;
    int64_t table_s0;
    int num_states, room, page_shift;      // room: keys that a table row has pages for
    const int64_t *idx;
    const int32_t *query_start, *seq_lens;
    int rows, T, q_heads, kv_heads, group;
    int tile_tokens;           // tokens of a row tile: 128 / group
    int group_inv;             // ceil(2^16 / group): row * group_inv >> 16 is row / group below 128
    float scale2;              // |scale| log2(e), not zero
    int window, sinks;
    uint16_t *out;
    int64_t out_s0, out_s1;
    float *lse;
    float *parts;              // split items' parts: [blocks][2][2 tiles][128 (D + 2)]
    void *joins;               // [blocks]: the item that begins in a block and goes on
    uint32_t *status;
    uint64_t timeout_ns;
    uint64_t walk_ns;          // the same with the time that the walk to the first item may take
};

struct VerifyArgs {
    const void *target;
    int64_t target_s0, target_s1;
    const int64_t *draft;
    int64_t draft_s0;
    const void *cache;
    int64_t cache_s0, cache_s1;
    const float *temperature, *uniforms;
    int64_t uni_s0;
    const float *noise;
    int64_t noise_s0;
    const int64_t *idx;
    int rows, N, V;
    int64_t *tokens;
    int64_t tok_s0;
    int32_t *accepted;
    float *p, *q;
    uint4 *part;               // [rows * (2N + 1)][segs] softmax partials
    uint64_t *win;             // [rows] best key; zero between calls
    uint32_t *arrivals;        // [rows] blocks done; zero between calls
    const uint32_t *status;
    int segs, seg_len, stat_blocks;   // of the statistics kernel
    int pick_segs, pick_len;   // of the pick kernel
};

constexpr int kVerifyMaxSegs = 32;         // a lane each

cudaError_t launch_paged_layout(const LayoutArgs &a, cudaStream_t s);
cudaError_t launch_paged_write(const WriteArgs &a, cudaStream_t s);
cudaError_t paged_attention_prepare();
size_t paged_attention_parts(int head_dim, int blocks);
size_t paged_attention_joins(int blocks);
cudaError_t launch_paged_attention(const AttnArgs &a, const CUtensorMap &q, const CUtensorMap &k,
                                   const CUtensorMap &v,
                                   int head_dim, bool f16, int blocks, cudaStream_t s);
cudaError_t launch_verify(VerifyArgs a, bool target_f32, bool cache_f32, int sms, cudaStream_t s);

}  // namespace dtm
