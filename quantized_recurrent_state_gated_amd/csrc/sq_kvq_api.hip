// sq_kvq_api.hip -- host side of the 8-bit paged key-value cache: argument
// checks and dispatch only; see include/sq.h for the contract of every entry point.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/sq.h"
#include "sq_checks.h"
#include "sq_kvq.h"
#include "sq_paged.h"

using namespace sqk;

namespace {

int cache_ok(const sq_kvq_cache *c)
{
    if (!c || !c->k || !c->v || !c->scales || c->n_pages < 1 || c->n_kv_heads < 1) return SQ_ERR_INVALID;
    if (c->format != SQ_KVQ_INT8 && c->format != SQ_KVQ_E4M3) return SQ_ERR_INVALID;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->scales, 16)) return SQ_ERR_INVALID;
    if (page_shift(c->page_size) < 0 || !attend_head_dim(c->head_dim)) return SQ_ERR_UNSUPPORTED;
    return SQ_OK;
}

KvqCache cache_args(const sq_kvq_cache *c)
{
    KvqCache a;
    a.k = static_cast<uint8_t *>(c->k);
    a.v = static_cast<uint8_t *>(c->v);
    a.scales = c->scales;
    a.n_pages = c->n_pages;
    a.page_shift = page_shift(c->page_size);
    a.heads = c->n_kv_heads;
    a.d = c->head_dim;
    a.e4m3 = c->format == SQ_KVQ_E4M3;
    return a;
}

bool dtype_ok(int32_t dtype) { return dtype == SQ_F32 || dtype == SQ_BF16; }

// what append and load check alike, and their arguments
int rows_args(const sq_kvq_cache *cache, const void *k, const void *v, int64_t k_stride, int64_t v_stride,
              int32_t dtype, int32_t n_tok, const int32_t *start, const int32_t *cu, int32_t n_req,
              const int32_t *table, int64_t table_stride, KvqRowsArgs *a)
{
    if (n_tok < 0 || n_req < 0 || table_stride < 0 || !dtype_ok(dtype)) return SQ_ERR_INVALID;
    if (n_tok == 0 || n_req == 0) return SQ_OK;
    if (!cu || (table_stride > 0 && !table)) return SQ_ERR_INVALID;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(start, 4) || !aligned(cu, 4) || !aligned(table, 4))
        return SQ_ERR_INVALID;
    const int64_t row = (int64_t)cache->n_kv_heads * cache->head_dim;
    if ((k && !stride_ok(k_stride, row, dtype)) || (v && !stride_ok(v_stride, row, dtype))) return SQ_ERR_INVALID;
    a->c = cache_args(cache);
    a->k = const_cast<void *>(k);
    a->v = const_cast<void *>(v);
    a->k_stride = k_stride;
    a->v_stride = v_stride;
    a->start = start;
    a->cu = cu;
    a->n = n_tok;
    a->n_req = n_req;
    a->table = table;
    a->table_stride = table_stride;
    return SQ_OK;
}

}  // namespace

extern "C" {

int sq_kvq_append(const sq_kvq_cache *cache, const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                  int32_t dtype, int32_t n_tok, const int32_t *ctx_lens, const int32_t *cu_new, int32_t n_req,
                  const int32_t *block_table, int64_t table_stride, void *stream)
{
    if (int st = cache_ok(cache)) return st;
    KvqRowsArgs a;
    if (int st = rows_args(cache, k, v, k_stride, v_stride, dtype, n_tok, ctx_lens, cu_new, n_req, block_table,
                           table_stride, &a))
        return st;
    if (n_tok == 0 || n_req == 0) return SQ_OK;
    if (!k || !v || !ctx_lens) return SQ_ERR_INVALID;
    return status(launch_kvq_append(a, dtype == SQ_BF16, (hipStream_t)stream));
}

int sq_kvq_load(const sq_kvq_cache *cache, const int32_t *first, const int32_t *cu, int32_t n_req,
                const int32_t *block_table, int64_t table_stride, void *k, void *v, int64_t k_stride,
                int64_t v_stride, int32_t dtype, int32_t n_tok, void *stream)
{
    if (int st = cache_ok(cache)) return st;
    KvqRowsArgs a;
    if (int st = rows_args(cache, k, v, k_stride, v_stride, dtype, n_tok, first, cu, n_req, block_table,
                           table_stride, &a))
        return st;
    if (n_tok == 0 || n_req == 0) return SQ_OK;
    if (!k && !v) return SQ_ERR_INVALID;
    return status(launch_kvq_load(a, dtype == SQ_BF16, (hipStream_t)stream));
}

uint64_t sq_kvq_attention_workspace(const sq_kvq_cache *cache, int32_t n_req, int32_t n_q, int32_t n_heads,
                                    int32_t max_len)
{
    if (cache_ok(cache) != SQ_OK || n_req < 1 || n_q < 1 || n_heads < 1 || max_len < 0 || max_len > kMaxReach ||
        n_heads % cache->n_kv_heads != 0 || (int64_t)n_req * n_heads > kMaxGrid / 2 ||
        (int64_t)n_q * n_heads > kMaxGrid / 2)
        return 0;
    return kvq_plan_bound(n_req, n_q, cache->n_kv_heads, n_heads, cache->head_dim, max_len);
}

int sq_kvq_attention(const sq_kvq_cache *cache, const void *q, int64_t q_stride, int32_t dtype, int32_t n_q,
                     int32_t n_heads, const int32_t *cu_q, int32_t n_req, const int32_t *block_table,
                     int64_t table_stride, const int32_t *seq_lens, int32_t max_len, float scale, int32_t window,
                     void *o, float *lse, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (int st = cache_ok(cache)) return st;
    if (!dtype_ok(dtype) || n_q < 0 || n_req < 0 || n_heads < 1 || max_len < 0 || window < 0 || table_stride < 0 ||
        n_heads % cache->n_kv_heads != 0 || !isfinite(scale) || (!cu_q && n_q != n_req))
        return SQ_ERR_INVALID;
    if (n_req == 0 || n_q == 0) return SQ_OK;
    if (!q || !o || !seq_lens || (table_stride > 0 && !block_table)) return SQ_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(cu_q, 4))
        return SQ_ERR_INVALID;
    if (!stride_ok(q_stride, (int64_t)n_heads * cache->head_dim, dtype)) return SQ_ERR_INVALID;
    // no request is longer than its table row; token positions are 32 bits in the
    // kernels, with room for a split's length past the last
    const int shift = page_shift(cache->page_size);
    const int32_t reach = table_stride <= (max_len >> shift) ? (int32_t)(table_stride << shift) : max_len;
    if (reach > kMaxReach || (int64_t)n_req * n_heads > kMaxGrid / 2 || (int64_t)n_q * n_heads > kMaxGrid / 2)
        return SQ_ERR_UNSUPPORTED;
    KvqAttendArgs a;
    a.c = cache_args(cache);
    a.q = q;
    a.q_stride = q_stride;
    a.cu = cu_q;
    a.table = block_table;
    a.table_stride = table_stride;
    a.lens = seq_lens;
    a.n = n_req;
    a.n_q = n_q;
    a.q_heads = n_heads;
    a.group = n_heads / cache->n_kv_heads;
    a.max_len = reach;
    a.window = window;
    // the kernels multiply scores by a positive factor: the sign goes to the queries
    a.scale_log2 = scale == 0.0f ? 1.0f : fabsf(scale) * 1.44269504088896341f;
    a.sign = scale > 0.0f ? 1.0f : scale < 0.0f ? -1.0f : 0.0f;
    a.o = o;
    a.lse = lse;
    const uint64_t need = kvq_plan(a, dtype == SQ_BF16);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return SQ_ERR_INVALID;
    a.part = static_cast<float *>(workspace);
    return status(launch_kvq_attend(a, dtype == SQ_BF16, (hipStream_t)stream));
}

}  // extern "C"
