// paged_abi.cu -- host side of the paged calls declared in include/markov.h:
// plan creation (all scratch allocated once), argument checks, launches and
// the sticky device status.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "../../include/markov.h"
#include "host_util.h"
#include "paged.h"

using namespace dtm;

struct markov_paged_plan {
    markov_paged_desc d;
    int sm_count = 0;
    int page_shift = 0;
    int blocks = 0;               // of an attention launch: one a multiprocessor
    uint32_t *ctrl = nullptr;     // [0..1] status, where; [2] the layout's arrivals
    float *parts = nullptr;       // split attention rows
    void *joins = nullptr;        // which they are
};

namespace {

constexpr size_t kCtrlWords = 8;

void free_plan(markov_paged_plan *p) {
    if (!p) return;
    if (p->ctrl) cudaFree(p->ctrl);
    if (p->parts) cudaFree(p->parts);
    if (p->joins) cudaFree(p->joins);
    delete p;
}

// A cache view whose every element can be read in 16-byte pieces.
bool valid_view(const markov_cache_view *v, const markov_paged_desc &d) {
    if (!v || !v->data || !aligned16(v->data)) return false;
    if (v->num_pages < 1 || v->num_pages > INT32_MAX) return false;
    if (v->s_page < 0 || v->s_slot < d.head_dim || v->s_head < d.head_dim) return false;
    return v->s_page % 8 == 0 && v->s_slot % 8 == 0 && v->s_head % 8 == 0;
}

constexpr int64_t kMaxRoom = 1 << 30;     // keys of a table row

// A cache as [pages, heads, slots, head_dim] tiles of 64 elements by a page's
// slots (at most 128), 128-byte swizzle; pages out of range read as zero.
bool encode_cache_map(CUtensorMap *m, const markov_cache_view &v, const markov_paged_plan &p) {
    const EncodeTiledFn fn = tensor_map_encoder();
    if (!fn) return false;
    const int page = p.d.page_size;
    const cuuint64_t dims[4] = {(cuuint64_t)p.d.head_dim, (cuuint64_t)page, (cuuint64_t)p.d.kv_heads,
                                (cuuint64_t)v.num_pages};
    // a lone page's stride is never used, but has to be one
    const int64_t s_page = v.num_pages > 1 ? v.s_page : v.s_slot * page;
    const cuuint64_t strides[3] = {(cuuint64_t)v.s_slot * 2, (cuuint64_t)v.s_head * 2, (cuuint64_t)s_page * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(page < 128 ? page : 128), 1, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, p.d.dtype == MARKOV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
              v.data, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries [tokens, heads, head_dim] as tiles of 64 elements by a group of
// heads by the tokens that 128 rows hold.
bool encode_query_map(CUtensorMap *m, const void *q, int64_t s0, int64_t s1, int tokens,
                      const markov_paged_plan &p) {
    const EncodeTiledFn fn = tensor_map_encoder();
    if (!fn) return false;
    const int group = p.d.q_heads / p.d.kv_heads;
    const cuuint64_t dims[3] = {(cuuint64_t)p.d.head_dim, (cuuint64_t)p.d.q_heads, (cuuint64_t)tokens};
    // a lone token's stride is never used, but has to be one
    const cuuint64_t strides[2] = {(cuuint64_t)s1 * 2, (cuuint64_t)(tokens > 1 ? s0 : s1 * p.d.q_heads) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)(128 / group)};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, p.d.dtype == MARKOV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
              const_cast<void *>(q), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An e4m3 cache view of the plan's pages; scales that are written must be the
// blocks' own.
bool valid_view(const markov_e4m3_view *v, const markov_paged_desc &d, bool scales_written) {
    if (!v || !v->data || !aligned16(v->data) || !v->scales || (reinterpret_cast<uintptr_t>(v->scales) & 3u)) return false;
    if (v->num_pages < 1 || v->num_pages > INT32_MAX) return false;
    if (v->s_page < 0 || v->s_slot < d.head_dim || v->s_head < d.head_dim) return false;
    if (v->s_page % 16 || v->s_slot % 16 || v->s_head % 16) return false;
    if (v->block < 16 || v->block > d.page_size || (v->block & (v->block - 1)) != 0) return false;
    if (v->ss_page < 0 || v->ss_block < 0 || v->ss_head < 0) return false;
    if (scales_written)
        return (v->num_pages == 1 || v->ss_page > 0) && (v->block == d.page_size || v->ss_block > 0) &&
               (d.kv_heads == 1 || v->ss_head > 0);
    return true;
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

E4m3Side side_of(const markov_e4m3_view &v) {
    return E4m3Side{static_cast<uint8_t *>(v.data), v.s_page, v.s_slot, v.s_head, v.scales, v.ss_page, v.ss_block, v.ss_head,
                    log2_of(v.block)};
}

E4m3Scales scales_of(const markov_e4m3_view &v) {
    return E4m3Scales{v.scales, v.ss_page, v.ss_block, v.ss_head, log2_of(v.block)};
}

// An e4m3 cache as [pages, heads, slots, head_dim] tiles of `slots` slots; the
// swizzle spans a slot's bytes of a head.
bool encode_e4m3_map(CUtensorMap *m, const markov_e4m3_view &v, const markov_paged_plan &p, int slots) {
    const EncodeTiledFn fn = tensor_map_encoder();
    if (!fn) return false;
    const int page = p.d.page_size;
    const cuuint64_t dims[4] = {(cuuint64_t)p.d.head_dim, (cuuint64_t)page, (cuuint64_t)p.d.kv_heads,
                                (cuuint64_t)v.num_pages};
    // a lone page's stride is never used, but has to be one
    const int64_t s_page = v.num_pages > 1 ? v.s_page : v.s_slot * page;
    const cuuint64_t strides[3] = {(cuuint64_t)v.s_slot, (cuuint64_t)v.s_head, (cuuint64_t)s_page};
    const cuuint32_t box[4] = {(cuuint32_t)p.d.head_dim, (cuuint32_t)(page < slots ? page : slots), 1, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    // where a head's slots lie apart, what lies between them is another head's: promoted
    // to 256 bytes, 64 single tokens read 1.32 GB for 0.91 and took 231 us
    const CUtensorMapL2promotion lines = v.s_slot == p.d.head_dim ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                         : p.d.head_dim == 128    ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                                  : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, v.data, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              p.d.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              lines, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What a call over a paged cache says of its rows.
bool valid_table(const void *page_table, int64_t table_s0, int32_t num_states, int32_t table_width, const void *idx,
                 const void *query_start, const void *seq_lens, const markov_paged_plan &p) {
    return page_table && idx && query_start && seq_lens && num_states >= 1 && table_width >= 1 &&
           table_s0 >= table_width && ((int64_t)table_width << p.page_shift) <= kMaxRoom;
}

// Token rows [T, heads, head_dim].
bool valid_rows(const void *p, int64_t s0, int64_t s1, const markov_paged_desc &d) {
    return p && aligned16(p) && s0 >= 0 && s1 >= d.head_dim && s0 % 8 == 0 && s1 % 8 == 0;
}

PagedRows rows_of(const markov_paged_plan &p, const int32_t *page_table, int64_t table_s0, int32_t num_states,
                  int32_t table_width, int64_t num_pages, const int64_t *idx, const int32_t *query_start,
                  const int32_t *seq_lens, int32_t rows, int32_t num_tokens) {
    return PagedRows{page_table, table_s0, num_states, (int)((int64_t)table_width << p.page_shift), p.page_shift, num_pages, idx,
                     query_start, seq_lens, rows, num_tokens};
}

}  // namespace

extern "C" {

markov_status markov_paged_plan_create(const markov_paged_desc *desc, markov_paged_plan **out) {
    if (!out) return MARKOV_EINVAL;
    *out = nullptr;
    if (!desc) return MARKOV_EINVAL;
    const markov_paged_desc d = *desc;
    if (d.kv_heads < 1 || d.q_heads < d.kv_heads || d.q_heads > 256 || d.q_heads % d.kv_heads != 0 ||
        d.q_heads / d.kv_heads > 128)
        return MARKOV_EINVAL;
    if (d.head_dim != 64 && d.head_dim != 128) return MARKOV_EINVAL;
    if (d.page_size < 8 || d.page_size > 256 || (d.page_size & (d.page_size - 1)) != 0)
        return MARKOV_EINVAL;
    if (d.max_rows < 1 || d.max_rows > kPagedMaxRows) return MARKOV_EINVAL;
    if (d.dtype != MARKOV_BF16 && d.dtype != MARKOV_F16) return MARKOV_EINVAL;
    if (d.timeout_ms < 0) return MARKOV_EINVAL;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || d.device < 0 || d.device >= ndev) {
        cudaGetLastError();
        return MARKOV_EDEVICE;
    }
    DeviceGuard guard(d.device);
    if (!guard.ok) return MARKOV_EDEVICE;
    cudaDeviceProp prop;
    if (cudaGetDeviceProperties(&prop, d.device) != cudaSuccess) return MARKOV_EDEVICE;
    if (prop.major < 10) return MARKOV_EUNSUPPORTED;    // the kernels are built for sm_103a

    markov_paged_plan *p = new (std::nothrow) markov_paged_plan();
    if (!p) return MARKOV_ECUDA;
    p->d = d;
    if (p->d.timeout_ms == 0) p->d.timeout_ms = 1000;
    p->sm_count = prop.multiProcessorCount;
    while ((1 << p->page_shift) < d.page_size) ++p->page_shift;
    p->blocks = p->sm_count;
    // the scratch serves the calls over either kind of cache
    const size_t parts = std::max({paged_attention_parts(d.head_dim, p->blocks), attention_e4m3_few_parts(d.head_dim, p->blocks),
                                   attention_e4m3_many_parts(d.head_dim, p->blocks)});
    const size_t joins = std::max({paged_attention_joins(p->blocks), attention_e4m3_few_joins(p->blocks),
                                   attention_e4m3_many_joins(p->blocks)});
    if (paged_attention_prepare() != cudaSuccess || attention_e4m3_few_prepare() != cudaSuccess ||
        attention_e4m3_many_prepare() != cudaSuccess ||
        cudaMalloc(&p->ctrl, kCtrlWords * sizeof(uint32_t)) != cudaSuccess ||
        cudaMalloc(&p->parts, parts * sizeof(float)) != cudaSuccess ||
        cudaMalloc(&p->joins, joins) != cudaSuccess ||
        cudaMemset(p->ctrl, 0, kCtrlWords * sizeof(uint32_t)) != cudaSuccess ||
        cudaDeviceSynchronize() != cudaSuccess) {
        cudaGetLastError();
        free_plan(p);
        return MARKOV_ECUDA;
    }
    *out = p;
    return MARKOV_OK;
}

void markov_paged_plan_destroy(markov_paged_plan *p) {
    if (!p) return;
    DeviceGuard guard(p->d.device);
    cudaDeviceSynchronize();
    free_plan(p);
}

markov_status markov_paged_plan_status(markov_paged_plan *p) {
    if (!p) return MARKOV_EINVAL;
    DeviceGuard guard(p->d.device);
    if (!guard.ok) return MARKOV_EDEVICE;
    uint32_t ctrl[2];
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpy(ctrl, p->ctrl, sizeof(ctrl), cudaMemcpyDeviceToHost) != cudaSuccess) {
        cudaGetLastError();
        return MARKOV_ECUDA;
    }
    if (ctrl[0] == 0u) return MARKOV_OK;
    // a kernel gave up: clear the status and every counter it may have left
    if (cudaMemset(p->ctrl, 0, kCtrlWords * sizeof(uint32_t)) != cudaSuccess ||
        cudaDeviceSynchronize() != cudaSuccess) {
        cudaGetLastError();
        return MARKOV_ECUDA;
    }
    return (markov_status)ctrl[0];
}

markov_status markov_paged_plan_inject_status(markov_paged_plan *p, markov_status code,
                                              uint32_t where) {
    if (!p || code == MARKOV_OK) return MARKOV_EINVAL;
    DeviceGuard guard(p->d.device);
    if (!guard.ok) return MARKOV_EDEVICE;
    const uint32_t w[2] = {(uint32_t)code, where};
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpy(p->ctrl, w, sizeof(w), cudaMemcpyHostToDevice) != cudaSuccess) {
        cudaGetLastError();
        return MARKOV_ECUDA;
    }
    return MARKOV_OK;
}

markov_status markov_paged_layout(markov_paged_plan *p, const int32_t *context_lens,
                                  const int32_t *query_lens, const int64_t *row_state_idx,
                                  int32_t rows, int32_t *page_table, int64_t table_s0,
                                  int32_t num_states, int32_t table_width,
                                  const int32_t *pages_held, int32_t *free_pages,
                                  int64_t ring_size, const int64_t *free_state,
                                  int32_t *pages_held_out, int64_t *free_state_out,
                                  int32_t *query_start, int32_t *seq_lens, int32_t *positions,
                                  int64_t *slots, int32_t num_tokens, void *stream) {
    if (!p || !context_lens || !query_lens || !row_state_idx || !page_table || !pages_held ||
        !free_pages || !free_state || !pages_held_out || !free_state_out || !query_start ||
        !seq_lens)
        return MARKOV_EINVAL;
    if (rows < 1 || rows > p->d.max_rows) return MARKOV_EINVAL;
    if (num_states < 1 || table_width < 1 || table_s0 < table_width) return MARKOV_EINVAL;
    if (ring_size < 1 || ring_size > INT32_MAX) return MARKOV_EINVAL;
    if (num_tokens < 0 || (num_tokens > 0 && (!positions || !slots))) return MARKOV_EINVAL;
    DeviceGuard guard(p->d.device);
    if (!guard.ok) return MARKOV_EDEVICE;
    LayoutArgs a{};
    a.context = context_lens;
    a.query = query_lens;
    a.idx = row_state_idx;
    a.rows = rows;
    a.table = page_table;
    a.table_s0 = table_s0;
    a.num_states = num_states;
    a.width = table_width;
    a.page_shift = p->page_shift;
    a.room = (int64_t)table_width << p->page_shift;
    if (a.room > INT32_MAX) a.room = INT32_MAX;
    a.held = pages_held;
    a.ring = free_pages;
    a.ring_size = ring_size;
    a.free_in = free_state;
    a.held_out = pages_held_out;
    a.free_out = free_state_out;
    a.query_start = query_start;
    a.seq_lens = seq_lens;
    a.positions = positions;
    a.slots = slots;
    a.T = num_tokens;
    a.status = p->ctrl;
    a.arrivals = p->ctrl + 2;
    if (launch_paged_layout(a, (cudaStream_t)stream) != cudaSuccess) {
        cudaGetLastError();
        return MARKOV_ECUDA;
    }
    return MARKOV_OK;
}

markov_status markov_paged_write(markov_paged_plan *p, const void *key, int64_t key_s0,
                                 int64_t key_s1, const void *value, int64_t value_s0,
                                 int64_t value_s1, const markov_cache_view *k_cache,
                                 const markov_cache_view *v_cache, const int64_t *slots,
                                 int32_t num_tokens, void *stream) {
    if (!p || num_tokens < 0 || (int64_t)num_tokens * p->d.kv_heads > INT32_MAX) return MARKOV_EINVAL;
    if (num_tokens == 0) return MARKOV_OK;
    if (!valid_rows(key, key_s0, key_s1, p->d) || !valid_rows(value, value_s0, value_s1, p->d) ||
        !valid_view(k_cache, p->d) || !valid_view(v_cache, p->d) || !slots ||
        k_cache->num_pages != v_cache->num_pages)
        return MARKOV_EINVAL;
    DeviceGuard guard(p->d.device);
    if (!guard.ok) return MARKOV_EDEVICE;
    auto side = [](const void *src, int64_t s0, int64_t s1, const markov_cache_view *c) {
        return WriteSide{static_cast<const uint4 *>(src), s0 / 8, s1 / 8,
                         static_cast<uint4 *>(c->data), c->s_page / 8, c->s_slot / 8, c->s_head / 8};
    };
    WriteArgs a{};
    a.k = side(key, key_s0, key_s1, k_cache);
    a.v = side(value, value_s0, value_s1, v_cache);
    a.slots = slots;
    a.num_slots = k_cache->num_pages << p->page_shift;
    a.T = num_tokens;
    a.heads = p->d.kv_heads;
    a.vec_shift = p->d.head_dim == 64 ? 3 : 4;
    a.page_shift = p->page_shift;
    a.status = p->ctrl;
    if (launch_paged_write(a, (cudaStream_t)stream) != cudaSuccess) {
        cudaGetLastError();
        return MARKOV_ECUDA;
    }
    return MARKOV_OK;
}

markov_status markov_paged_attention(markov_paged_plan *p, const void *q, int64_t q_s0,
                                     int64_t q_s1, const markov_cache_view *k_cache,
                                     const markov_cache_view *v_cache, const int32_t *page_table,
                                     int64_t table_s0, int32_t num_states, int32_t table_width,
                                     const int64_t *row_state_idx, const int32_t *query_start,
                                     const int32_t *seq_lens, int32_t rows, int32_t num_tokens,
                                     float scale, int32_t window, int32_t sinks, void *out,
                                     int64_t out_s0, int64_t out_s1, float *lse, void *stream) {
    if (!p || num_tokens < 0 || rows < 1 || rows > p->d.max_rows) return MARKOV_EINVAL;
    if (!std::isfinite(scale) || window < 0 || sinks < 0) return MARKOV_EINVAL;
    if (!page_table || !row_state_idx || !query_start || !seq_lens || num_states < 1 ||
        table_width < 1 || table_s0 < table_width)
        return MARKOV_EINVAL;
    if (!valid_view(k_cache, p->d) || !valid_view(v_cache, p->d) ||
        k_cache->num_pages != v_cache->num_pages)
        return MARKOV_EINVAL;
    const int64_t room = (int64_t)table_width << p->page_shift;
    if (room > kMaxRoom || (int64_t)num_tokens * (p->d.q_heads / p->d.kv_heads) > INT32_MAX / 2)
        return MARKOV_EINVAL;
    if (num_tokens == 0) return MARKOV_OK;
    if (!valid_rows(q, q_s0, q_s1, p->d) || !valid_rows(out, out_s0, out_s1, p->d) || q == out)
        return MARKOV_EINVAL;
    DeviceGuard guard(p->d.device);
    if (!guard.ok) return MARKOV_EDEVICE;
    CUtensorMap qmap, kmap, vmap;
    if (!encode_query_map(&qmap, q, q_s0, q_s1, num_tokens, *p) ||
        !encode_cache_map(&kmap, *k_cache, *p) || !encode_cache_map(&vmap, *v_cache, *p))
        return MARKOV_EINVAL;
    AttnArgs a{};
    a.negate = scale < 0.0f;
    a.table = page_table;
    a.table_s0 = table_s0;
    a.num_states = num_states;
    a.room = (int)room;
    a.page_shift = p->page_shift;
    a.idx = row_state_idx;
    a.query_start = query_start;
    a.seq_lens = seq_lens;
    a.rows = rows;
    a.T = num_tokens;
    a.q_heads = p->d.q_heads;
    a.kv_heads = p->d.kv_heads;
    a.group = p->d.q_heads / p->d.kv_heads;
    a.tile_tokens = 128 / a.group;
    a.group_inv = (65536 + a.group - 1) / a.group;
    a.scale2 = std::fmax(std::fabs(scale) * 1.4426950408889634f, 1e-30f);
    a.window = window;
    // a row has no more keys than kMaxRoom
    a.sinks = sinks < kMaxRoom ? sinks : (int)kMaxRoom;
    a.out = static_cast<uint16_t *>(out);
    a.out_s0 = out_s0;
    a.out_s1 = out_s1;
    a.lse = lse;
    a.parts = p->parts;
    a.joins = p->joins;
    a.status = p->ctrl;
    a.timeout_ns = (uint64_t)p->d.timeout_ms * 1000000ull;
    // a pair of row tiles takes the walk a fraction of a microsecond, twice
    a.walk_ns = a.timeout_ns + (uint64_t)((int64_t)num_tokens * a.group / 256 + rows + 1) * 1000ull;
    if (launch_paged_attention(a, qmap, kmap, vmap, p->d.head_dim, p->d.dtype == MARKOV_F16, p->blocks,
                               (cudaStream_t)stream) != cudaSuccess) {
        cudaGetLastError();
        return MARKOV_ECUDA;
    }
    return MARKOV_OK;
}

markov_status markov_paged_write_e4m3(markov_paged_plan *p, const void *key, int64_t key_s0,
                                      int64_t key_s1, const void *value, int64_t value_s0,
                                      int64_t value_s1, const markov_e4m3_view *k_cache,
                                      const markov_e4m3_view *v_cache, const int64_t *slots,
                                      int32_t num_tokens, int32_t keep_scales, void *stream) {
    if (!p || num_tokens < 0 || (int64_t)num_tokens * p->d.kv_heads > INT32_MAX) return MARKOV_EINVAL;
    if (keep_scales != 0 && keep_scales != 1) return MARKOV_EINVAL;
    if (num_tokens == 0) return MARKOV_OK;
    if (!valid_rows(key, key_s0, key_s1, p->d) || !valid_rows(value, value_s0, value_s1, p->d) ||
        !valid_view(k_cache, p->d, !keep_scales) || !valid_view(v_cache, p->d, !keep_scales) || !slots ||
        k_cache->num_pages != v_cache->num_pages)
        return MARKOV_EINVAL;
    DeviceGuard guard(p->d.device);
    if (!guard.ok) return MARKOV_EDEVICE;
    StoreArgs a{};
    a.side[0] = StoreSide{static_cast<const uint4 *>(key), key_s0 / 8, key_s1 / 8, side_of(*k_cache)};
    a.side[1] = StoreSide{static_cast<const uint4 *>(value), value_s0 / 8, value_s1 / 8, side_of(*v_cache)};
    a.slots = slots;
    a.num_slots = k_cache->num_pages << p->page_shift;
    a.T = num_tokens;
    a.heads = p->d.kv_heads;
    a.page_shift = p->page_shift;
    // a token a block while those find a place at once, then more: of single tokens of a
    // batch a warp takes one after the other, of a prompt a block a cache block
    a.chunk = 1;
    while (a.chunk < 64 && (int64_t)(num_tokens + a.chunk - 1) / a.chunk * p->d.kv_heads * 2 > 16 * p->sm_count) a.chunk *= 4;
    if (a.chunk == 64) a.chunk = std::max({64, (int)k_cache->block, (int)v_cache->block});
    a.status = p->ctrl;
    if (launch_store_e4m3(a, p->d.head_dim, p->d.dtype == MARKOV_F16, keep_scales != 0, (cudaStream_t)stream) != cudaSuccess) {
        cudaGetLastError();
        return MARKOV_ECUDA;
    }
    return MARKOV_OK;
}

markov_status markov_paged_read_e4m3(markov_paged_plan *p, const markov_e4m3_view *k_cache,
                                     const markov_e4m3_view *v_cache, const int32_t *page_table,
                                     int64_t table_s0, int32_t num_states, int32_t table_width,
                                     const int64_t *row_state_idx, const int32_t *query_start,
                                     const int32_t *seq_lens, int32_t rows, int32_t num_tokens,
                                     void *key, int64_t key_s0, int64_t key_s1, void *value,
                                     int64_t value_s0, int64_t value_s1, void *stream) {
    if (!p || num_tokens < 0 || rows < 1 || rows > p->d.max_rows) return MARKOV_EINVAL;
    if (!valid_table(page_table, table_s0, num_states, table_width, row_state_idx, query_start, seq_lens, *p) ||
        !valid_view(k_cache, p->d, false) || !valid_view(v_cache, p->d, false) ||
        k_cache->num_pages != v_cache->num_pages)
        return MARKOV_EINVAL;
    if (num_tokens == 0) return MARKOV_OK;
    if (!valid_rows(key, key_s0, key_s1, p->d) || !valid_rows(value, value_s0, value_s1, p->d) || key == value)
        return MARKOV_EINVAL;
    DeviceGuard guard(p->d.device);
    if (!guard.ok) return MARKOV_EDEVICE;
    FetchArgs a{};
    a.r = rows_of(*p, page_table, table_s0, num_states, table_width, k_cache->num_pages, row_state_idx, query_start, seq_lens,
                  rows, num_tokens);
    a.side[0] = side_of(*k_cache);
    a.side[1] = side_of(*v_cache);
    a.dst[0] = static_cast<uint4 *>(key);
    a.dst[1] = static_cast<uint4 *>(value);
    a.dst_s0[0] = key_s0 / 8;
    a.dst_s1[0] = key_s1 / 8;
    a.dst_s0[1] = value_s0 / 8;
    a.dst_s1[1] = value_s1 / 8;
    a.heads = p->d.kv_heads;
    // two blocks a multiprocessor before a block takes more tokens
    a.tile = 1;
    while (a.tile < 32 && num_tokens / (2 * a.tile) >= 2 * p->sm_count) a.tile *= 2;
    a.status = p->ctrl;
    if (launch_fetch_e4m3(a, p->d.head_dim, p->d.dtype == MARKOV_F16, (cudaStream_t)stream) != cudaSuccess) {
        cudaGetLastError();
        return MARKOV_ECUDA;
    }
    return MARKOV_OK;
}

markov_status markov_paged_attention_e4m3(
    markov_paged_plan *p, const void *q, int64_t q_s0, int64_t q_s1,
    const markov_e4m3_view *k_cache, const markov_e4m3_view *v_cache, const int32_t *page_table,
    int64_t table_s0, int32_t num_states, int32_t table_width, const int64_t *row_state_idx,
    const int32_t *query_start, const int32_t *seq_lens, int32_t rows, int32_t num_tokens,
    float scale, int32_t window, int32_t sinks, void *out, int64_t out_s0, int64_t out_s1,
    float *lse, void *stream) {
    if (!p || num_tokens < 0 || rows < 1 || rows > p->d.max_rows) return MARKOV_EINVAL;
    if (!std::isfinite(scale) || window < 0 || sinks < 0) return MARKOV_EINVAL;
    if (!valid_table(page_table, table_s0, num_states, table_width, row_state_idx, query_start, seq_lens, *p) ||
        !valid_view(k_cache, p->d, false) || !valid_view(v_cache, p->d, false) ||
        k_cache->num_pages != v_cache->num_pages)
        return MARKOV_EINVAL;
    const int group = p->d.q_heads / p->d.kv_heads;
    if ((int64_t)num_tokens * group > INT32_MAX / 2) return MARKOV_EINVAL;
    if (num_tokens == 0) return MARKOV_OK;
    if (!valid_rows(q, q_s0, q_s1, p->d) || !valid_rows(out, out_s0, out_s1, p->d) || q == out)
        return MARKOV_EINVAL;
    DeviceGuard guard(p->d.device);
    if (!guard.ok) return MARKOV_EDEVICE;
    AttnE4m3Args a{};
    a.r = rows_of(*p, page_table, table_s0, num_states, table_width, k_cache->num_pages, row_state_idx, query_start, seq_lens,
                  rows, num_tokens);
    a.ks = scales_of(*k_cache);
    a.vs = scales_of(*v_cache);
    a.q_heads = p->d.q_heads;
    a.kv_heads = p->d.kv_heads;
    a.group = group;
    a.tile_tokens = 128 / group;
    a.group_inv = (65536 + group - 1) / group;
    a.scale2 = scale * 1.4426950408889634f;
    a.window = window;
    // a row has no more keys than kMaxRoom
    a.sinks = sinks < kMaxRoom ? sinks : (int)kMaxRoom;
    a.q = static_cast<const uint16_t *>(q);
    a.q_s0 = q_s0;
    a.q_s1 = q_s1;
    a.out = static_cast<uint16_t *>(out);
    a.out_s0 = out_s0;
    a.out_s1 = out_s1;
    a.lse = lse;
    a.parts = p->parts;
    a.joins = p->joins;
    a.status = p->ctrl;
    a.timeout_ns = (uint64_t)p->d.timeout_ms * 1000000ull;
    a.walk_ns = a.timeout_ns + (uint64_t)((int64_t)num_tokens * group / 256 + rows + 1) * 1000ull;
    const bool f16 = p->d.dtype == MARKOV_F16;
    const cudaStream_t s = (cudaStream_t)stream;
    // Few rows of query heads a request on average: bound by the cache's bytes.  In us,
    // few against many: 64 requests of 500-16000 keys with 16 rows for each of 4 key heads
    // 72 and 87; 32 of them with 16 rows for each of 8 key heads 69 and 80, 24 rows 92 and
    // 81; 8 of 1000-16000 keys with 16 rows 38 and 34, of 32000 keys 106 and 141, 32 rows of
    // 1000-16000 44 and 35.  These are of requests that are alike: of mixed ones one form
    // takes all, and padding rows count.  64 single tokens and a chunk together and apart
    // (8 key heads, 2000 keys and 500-8000): with 1 query head each and a chunk of 900 166
    // and 98 + 32, of 2000 197 and 98 + 46 (430 with 400 padding rows), with 4 and 900 223 and
    // 100 + 68 (382 with padding rows)
    const int64_t query_rows = (int64_t)num_tokens * group;
    const bool few = query_rows <= 16 * (int64_t)rows;
    // and of many, items of one row tile while a request has no more on average: a place for
    // another operand, work that spreads.  In us, a pair of row tiles an item and one: 8
    // rows of 9 tokens (72 query rows a key head) 38.7 and 36.4; 64 of 8 tokens (32) 175 and
    // 161; 16 of 16 tokens (128) 63 and 59; 24 of 1-40 tokens (164 on average) 98 and 88,
    // but 16 of 24 tokens (192) 86 and 97, a prompt's 4096 tokens 726 and 955
    const bool one = query_rows <= 128 * (int64_t)rows;
    CUtensorMap qmap, kmap, vmap;
    const int slots = few ? 32 : 128;
    if (!encode_e4m3_map(&kmap, *k_cache, *p, slots) || !encode_e4m3_map(&vmap, *v_cache, *p, slots) ||
        (!few && !encode_query_map(&qmap, q, q_s0, q_s1, num_tokens, *p)))
        return MARKOV_EINVAL;
    const cudaError_t e =
        few ? launch_attention_e4m3_few(a, kmap, vmap, p->d.head_dim, f16, query_rows <= 8 * (int64_t)rows, p->blocks, s)
            : launch_attention_e4m3_many(a, qmap, kmap, vmap, p->d.head_dim, f16, one, p->blocks, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return MARKOV_ECUDA;
    }
    return MARKOV_OK;
}

}  // extern "C"
