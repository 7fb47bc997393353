// sq_serve_api.hip -- host side of the operators around the state pool: block
// tables, cache append, paged attention, prompt form.  Argument checks and
// dispatch only; see include/sq.h for the contract of every entry point.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/sq.h"
#include "sq_paged.h"
#include "sq_prefill.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// log2 of a page size in [16, 256], or -1
int page_shift(int32_t page)
{
    for (int s = 4; s <= 8; s++)
        if (page == 1 << s) return s;
    return -1;
}

int cache_ok(const sq_kv_cache *c)
{
    if (!c || !c->k || !c->v || c->n_pages < 1 || c->n_kv_heads < 1) return SQ_ERR_INVALID;
    if (c->dtype != SQ_F32 && c->dtype != SQ_BF16) return SQ_ERR_INVALID;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return SQ_ERR_INVALID;
    if (page_shift(c->page_size) < 0 || !sqk::attend_head_dim(c->head_dim)) return SQ_ERR_UNSUPPORTED;
    return SQ_OK;
}

sqk::CacheArgs cache_args(const sq_kv_cache *c)
{
    sqk::CacheArgs a;
    a.k = c->k;
    a.v = c->v;
    a.n_pages = c->n_pages;
    a.page_shift = page_shift(c->page_size);
    a.heads = c->n_kv_heads;
    a.d = c->head_dim;
    return a;
}

int elem_bytes(int32_t dtype) { return dtype == SQ_BF16 ? 2 : 4; }

// a token stride: at least a token's elements, and rows that stay 16-byte aligned
bool stride_ok(int64_t stride, int64_t row, int32_t dtype)
{
    return stride >= row && stride * elem_bytes(dtype) % 16 == 0;
}

// the launchers refuse a grid that does not fit one launch before they make any HIP call
int status(hipError_t e)
{
    return e == hipSuccess ? SQ_OK : e == hipErrorInvalidConfiguration ? SQ_ERR_UNSUPPORTED : SQ_ERR_HIP;
}

constexpr int64_t kMaxGrid = 0x7fffffff;
constexpr int32_t kMaxReach = 1 << 30;
constexpr int32_t kMaxTokens = 0x7fffffff - 64;  // the kernels step up to 64 tokens past the last in 32 bits

bool prefill_shape(int32_t dk, int32_t dv)
{
    return dk >= 4 && dv >= 4 && dk <= 256 && dv <= 256 && dk % 4 == 0 && dv % 4 == 0;
}

struct Split {
    int32_t q_tiles, chunk, splits;
};

Split split_of(const sq_kv_cache *c, int32_t n_req, int32_t n_heads, int32_t max_len)
{
    Split s;
    s.q_tiles = (n_heads / c->n_kv_heads + 15) / 16;
    sqk::attend_split(n_req, c->n_kv_heads, s.q_tiles, max_len, &s.chunk, &s.splits);
    return s;
}

uint64_t part_bytes(const sq_kv_cache *c, uint64_t rows) { return rows * (uint64_t)(c->head_dim + 2) * 4; }

}  // namespace

extern "C" {

int sq_block_tables(const int32_t *ctx_lens, const int32_t *new_lens, int32_t n_req,
                    int32_t page_size, const int32_t *free_pages, int32_t n_free,
                    int32_t *block_table, int64_t table_stride, int32_t *seq_lens, int32_t *cu_new,
                    int32_t *cu_pages, int64_t *slot_map, int64_t n_slots, int32_t *result,
                    void *stream)
{
    if (n_req < 0 || n_free < 0 || n_slots < 0 || n_slots > 0x7fffffff || table_stride < 0)
        return SQ_ERR_INVALID;
    if (!cu_new || !cu_pages || !result) return SQ_ERR_INVALID;
    if (n_req > 0 && (!ctx_lens || !new_lens || !seq_lens || (table_stride > 0 && !block_table)))
        return SQ_ERR_INVALID;
    if ((n_free > 0 && !free_pages) || (n_slots > 0 && !slot_map)) return SQ_ERR_INVALID;
    if (!aligned(slot_map, 8) || !aligned(ctx_lens, 4) || !aligned(new_lens, 4) ||
        !aligned(free_pages, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(cu_new, 4) || !aligned(cu_pages, 4) || !aligned(result, 4))
        return SQ_ERR_INVALID;
    const int shift = page_shift(page_size);
    if (shift < 0) return SQ_ERR_UNSUPPORTED;
    sqk::TableArgs a;
    a.ctx = ctx_lens;
    a.fresh = new_lens;
    a.free_pages = free_pages;
    a.n = n_req;
    a.n_free = n_free;
    a.page_shift = shift;
    a.table = block_table;
    a.stride = table_stride;
    a.seq = seq_lens;
    a.cu_new = cu_new;
    a.cu_pages = cu_pages;
    a.slots = slot_map;
    a.capacity = n_slots;
    a.result = result;
    return status(sqk::launch_tables(a, (hipStream_t)stream));
}

int sq_kv_append(const sq_kv_cache *cache, const void *k, const void *v, int64_t k_stride,
                 int64_t v_stride, const int64_t *slot_map, int32_t n_tok, void *stream)
{
    if (int st = cache_ok(cache)) return st;
    if (n_tok < 0) return SQ_ERR_INVALID;
    if (n_tok == 0) return SQ_OK;
    if (!k || !v || !slot_map || !aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 8))
        return SQ_ERR_INVALID;
    const int64_t row = (int64_t)cache->n_kv_heads * cache->head_dim;
    if (!stride_ok(k_stride, row, cache->dtype) || !stride_ok(v_stride, row, cache->dtype))
        return SQ_ERR_INVALID;
    if ((int64_t)n_tok * cache->n_kv_heads > kMaxGrid) return SQ_ERR_UNSUPPORTED;
    sqk::AppendArgs a;
    a.c = cache_args(cache);
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.slots = slot_map;
    a.n = n_tok;
    return status(sqk::launch_append(a, cache->dtype == SQ_BF16, (hipStream_t)stream));
}

uint64_t sq_paged_attention_workspace(const sq_kv_cache *cache, int32_t n_req, int32_t n_heads,
                                      int32_t max_len)
{
    if (cache_ok(cache) != SQ_OK || n_req < 1 || n_heads < 1 || max_len < 0 ||
        n_heads % cache->n_kv_heads != 0 || (int64_t)n_req * n_heads > kMaxGrid)
        return 0;
    return part_bytes(cache, sqk::attend_rows_bound(n_req, cache->n_kv_heads, n_heads, max_len));
}

int sq_paged_attention(const sq_kv_cache *cache, const void *q, int64_t q_stride, int32_t n_req,
                       int32_t n_heads, const int32_t *block_table, int64_t table_stride,
                       const int32_t *seq_lens, int32_t max_len, float scale, int32_t window,
                       void *o, float *lse, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (int st = cache_ok(cache)) return st;
    if (n_req < 0 || n_heads < 1 || max_len < 0 || window < 0 || table_stride < 0 ||
        n_heads % cache->n_kv_heads != 0 || !isfinite(scale))
        return SQ_ERR_INVALID;
    if (n_req == 0) return SQ_OK;
    if (!q || !o || !seq_lens || (table_stride > 0 && !block_table)) return SQ_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
        !aligned(seq_lens, 4))
        return SQ_ERR_INVALID;
    if (!stride_ok(q_stride, (int64_t)n_heads * cache->head_dim, cache->dtype)) return SQ_ERR_INVALID;
    // no request is longer than its table row; token positions are 32 bits in the
    // kernels, with room for a split's length past the last
    const int shift = page_shift(cache->page_size);
    const int32_t reach = table_stride <= (max_len >> shift) ? (int32_t)(table_stride << shift) : max_len;
    if (reach > kMaxReach || (int64_t)n_req * n_heads > kMaxGrid) return SQ_ERR_UNSUPPORTED;
    const int32_t most = window > 0 && window < reach ? window : reach;
    const Split s = split_of(cache, n_req, n_heads, most);
    const uint64_t need =
        s.splits > 1 ? part_bytes(cache, (uint64_t)n_req * (uint64_t)n_heads * (uint64_t)s.splits) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return SQ_ERR_INVALID;
    if ((int64_t)n_req * cache->n_kv_heads * s.q_tiles > kMaxGrid / s.splits) return SQ_ERR_UNSUPPORTED;
    sqk::AttendArgs a;
    a.c = cache_args(cache);
    a.q = q;
    a.q_stride = q_stride;
    a.table = block_table;
    a.table_stride = table_stride;
    a.lens = seq_lens;
    a.n = n_req;
    a.q_heads = n_heads;
    a.group = n_heads / cache->n_kv_heads;
    a.q_tiles = s.q_tiles;
    a.max_len = reach;
    a.window = window;
    a.chunk = s.chunk;
    a.splits = s.splits;
    a.scale_log2 = scale * 1.44269504088896341f;
    a.o = o;
    a.lse = lse;
    a.part = static_cast<float *>(workspace);
    return status(sqk::launch_attend(a, cache->dtype == SQ_BF16, (hipStream_t)stream));
}

static bool prefill_sizes(int32_t n_seq, int32_t n_tokens, int32_t n_heads, int32_t dtype, int32_t rule)
{
    return n_seq >= 0 && n_tokens >= 0 && n_heads >= 1 && (dtype == SQ_F32 || dtype == SQ_BF16) &&
           (rule == SQ_RULE_DELTA || rule == SQ_RULE_LINEAR);
}

uint64_t sq_prefill_workspace(int32_t n_seq, int32_t n_tokens, int32_t n_heads, int32_t d_k,
                              int32_t d_v, int32_t dtype, int32_t rule)
{
    if (!prefill_sizes(n_seq, n_tokens, n_heads, dtype, rule) || !prefill_shape(d_k, d_v)) return 0;
    return sqk::prefill_workspace(n_seq, n_tokens, n_heads, d_k, d_v, dtype == SQ_BF16,
                                  rule == SQ_RULE_DELTA);
}

int sq_prefill(const sq_prefill_desc *desc, void *stream)
{
    if (!desc) return SQ_ERR_INVALID;
    const sq_prefill_desc &d = *desc;
    if (!prefill_sizes(d.n_seq, d.n_tokens, d.n_heads, d.dtype, d.rule) || d.n_k_heads < 1 ||
        d.n_heads % d.n_k_heads != 0)
        return SQ_ERR_INVALID;
    if (!prefill_shape(d.d_k, d.d_v) || d.n_tokens > kMaxTokens) return SQ_ERR_UNSUPPORTED;
    if (d.n_seq == 0) return SQ_OK;
    if (!d.cu_seqlens || !aligned(d.cu_seqlens, 4)) return SQ_ERR_INVALID;
    if (d.n_tokens > 0) {
        if (!d.q || !d.k || !d.v || !d.alpha || !d.beta || !d.o) return SQ_ERR_INVALID;
        const uintptr_t es = (uintptr_t)elem_bytes(d.dtype);
        if (!aligned(d.q, es) || !aligned(d.k, es) || !aligned(d.v, es) || !aligned(d.o, es) ||
            !aligned(d.alpha, 4) || !aligned(d.beta, 4))
            return SQ_ERR_INVALID;
        if (d.q_stride < (int64_t)d.n_k_heads * d.d_k || d.k_stride < (int64_t)d.n_k_heads * d.d_k ||
            d.v_stride < (int64_t)d.n_heads * d.d_v)
            return SQ_ERR_INVALID;
    }
    if (!aligned(d.S0, 16) || !aligned(d.S, 16)) return SQ_ERR_INVALID;
    if ((int64_t)d.n_seq * d.n_heads > kMaxGrid / 64 ||
        ((int64_t)d.n_tokens / 16 + d.n_seq) > kMaxGrid / d.n_heads)
        return SQ_ERR_UNSUPPORTED;
    sqk::PrefillArgs a;
    a.q = d.q;
    a.k = d.k;
    a.v = d.v;
    a.q_stride = d.q_stride;
    a.k_stride = d.k_stride;
    a.v_stride = d.v_stride;
    a.alpha = d.alpha;
    a.beta = d.beta;
    a.cu = d.cu_seqlens;
    a.n_seq = d.n_seq;
    a.n_tokens = d.n_tokens;
    a.heads = d.n_heads;
    a.per_k = d.n_heads / d.n_k_heads;
    a.dk = d.d_k;
    a.dv = d.d_v;
    a.S0 = d.S0;
    a.o = d.o;
    a.S = d.S;
    a.ws = static_cast<uint8_t *>(d.workspace);
    const uint64_t need = sqk::prefill_needs(a, d.dtype == SQ_BF16, d.rule == SQ_RULE_DELTA);
    if (need > 0 && (!d.workspace || d.workspace_bytes < need || !aligned(d.workspace, 256)))
        return SQ_ERR_INVALID;
    return status(sqk::launch_prefill(a, d.dtype == SQ_BF16, d.rule == SQ_RULE_DELTA,
                                      (hipStream_t)stream));
}

}  // extern "C"
