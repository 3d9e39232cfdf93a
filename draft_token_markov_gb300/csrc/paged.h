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

// One side of an e4m3 cache; data strides in bytes, scale strides in floats.
struct E4m3Side {
    uint8_t *data;
    int64_t s_page, s_slot, s_head;
    float *scales;
    int64_t ss_page, ss_block, ss_head;
    int block_shift;           // log2 of the tokens of a scale
};

// One side of a store into an e4m3 cache: [T, heads, D] of 16-bit elements.
struct StoreSide {
    const uint4 *src;
    int64_t src_s0, src_s1;    // in 16-byte units
    E4m3Side cache;
};

struct StoreArgs {
    StoreSide side[2];         // keys, values
    const int64_t *slots;
    int64_t num_slots;
    int T, heads, page_shift;
    int chunk;                 // tokens whose blocks a thread block looks after
    const uint32_t *status;
};

// The rows of a call over a paged cache.
struct PagedRows {
    const int32_t *table;
    int64_t table_s0;
    int num_states, room, page_shift;
    int64_t num_pages;
    const int64_t *idx;
    const int32_t *query_start, *seq_lens;
    int rows, T;
};

struct FetchArgs {
    PagedRows r;
    E4m3Side side[2];
    uint4 *dst[2];
    int64_t dst_s0[2], dst_s1[2];          // in 16-byte units
    int heads, tile;           // tile: tokens of a block
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

// The scales of one side of an e4m3 cache, as attention reads them.
struct E4m3Scales {
    const float *p;
    int64_t s_page, s_block, s_head;
    int block_shift;
};

struct AttnE4m3Args {
    PagedRows r;
    E4m3Scales ks, vs;
    int q_heads, kv_heads, group;
    int tile_tokens, group_inv;            // as in AttnArgs
    float scale2;              // scale log2(e)
    int window, sinks;
    const uint16_t *q;
    int64_t q_s0, q_s1;
    uint16_t *out;
    int64_t out_s0, out_s1;
    float *lse;
    float *parts;              // split items' parts
    void *joins;               // the item that begins in a worker's range and goes on
    uint32_t *status;
    uint64_t timeout_ns;
    uint64_t walk_ns;          // as in AttnArgs
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
cudaError_t launch_store_e4m3(const StoreArgs &a, int head_dim, bool f16, bool keep, cudaStream_t s);
cudaError_t launch_fetch_e4m3(const FetchArgs &a, int head_dim, bool f16, cudaStream_t s);
cudaError_t attention_e4m3_few_prepare();
size_t attention_e4m3_few_parts(int head_dim, int blocks);
size_t attention_e4m3_few_joins(int blocks);
// Calls of few query rows a request: k and v are maps of up to 32 slots by head_dim.
cudaError_t launch_attention_e4m3_few(const AttnE4m3Args &a, const CUtensorMap &k, const CUtensorMap &v, int head_dim,
                                      bool f16, bool half, int blocks, cudaStream_t s);
cudaError_t attention_e4m3_many_prepare();
size_t attention_e4m3_many_parts(int head_dim, int blocks);
size_t attention_e4m3_many_joins(int blocks);
// Other calls: k and v are maps of up to 128 slots, q one of 64 elements by a row tile's tokens.
cudaError_t launch_attention_e4m3_many(const AttnE4m3Args &a, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                                       int head_dim, bool f16, bool one, int blocks, cudaStream_t s);
cudaError_t paged_attention_prepare();
size_t paged_attention_parts(int head_dim, int blocks);
size_t paged_attention_joins(int blocks);
cudaError_t launch_paged_attention(const AttnArgs &a, const CUtensorMap &q, const CUtensorMap &k,
                                   const CUtensorMap &v,
                                   int head_dim, bool f16, int blocks, cudaStream_t s);
cudaError_t launch_verify(VerifyArgs a, bool target_f32, bool cache_f32, int sms, cudaStream_t s);

}  // namespace dtm
