// sq_kvq.h -- internal interface between the host code (sq_kvq_api.hip) and the
// kernels of the 8-bit paged key-value cache (sq_kvq.hip: write and read back,
// sq_kvq_few.hip, sq_kvq_tiles.hip: attention).  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sqk {

constexpr int kKvqBlock = 16;  // token positions that share a scale

// Codes of keys [page][head][token][d], of values [page][head][block][d][16],
// scales [page][head][block][2].
struct KvqCache {
    uint8_t *k, *v;
    float *scales;
    int32_t n_pages, page_shift, heads, d;
    int32_t e4m3;                // 0: integer codes + 128
};

// Tokens cu[r] .. cu[r + 1] - 1 of request r and its positions from start[r] on.
struct KvqRowsArgs {
    KvqCache c;
    void *k, *v;                 // [n][heads][d]; load: either may be null
    int64_t k_stride, v_stride;  // elements between tokens
    const int32_t *start;        // [n_req], or null for zeros
    const int32_t *cu;           // [n_req + 1]
    int32_t n, n_req;
    const int32_t *table;        // [n_req][table_stride]
    int64_t table_stride;
};

hipError_t launch_kvq_append(const KvqRowsArgs &a, bool bf16, hipStream_t st);
hipError_t launch_kvq_load(const KvqRowsArgs &a, bool bf16, hipStream_t st);

struct KvqAttendArgs {
    KvqCache c;
    const void *q;               // [n_q][q_heads][d], queries q_stride elements apart
    int64_t q_stride;
    const int32_t *cu;           // [n + 1], or null: one query a request
    const int32_t *table;        // [n][table_stride]
    int64_t table_stride;
    const int32_t *lens;         // [n]
    int32_t n, n_q, q_heads, group;
    int32_t max_len, window;
    float scale_log2;            // |scale| * log2(e), or 1 for a scale of zero
    float sign;                  // of the scale, or 0
    void *o;                     // [n_q][q_heads][d]
    float *lse;                  // [n_q][q_heads] or null
    float *part;                 // partial results: few-query form, then tile form
    // few queries (one token, or at most 16 rows of queries x group)
    int32_t few_on;              // 0: every request goes to the tile form
    int32_t q_tiles, rows;       // 16-row tiles and rows of partial results per (request, head)
    int32_t chunk, splits;       // tokens per split, splits of the longest request
    // many queries: tiles of 256 or 128 rows
    int32_t tile_rows;
    int32_t tiles;               // tile slots over all requests, 0: none can need them
    int32_t t_chunk, t_splits;
};

// Whether the tile kernel's registers leave room for two waves on a SIMD.
constexpr bool two_a_simd(bool bf16, int d) { return d <= 96 || (bf16 && d <= 128); }
// Whether tiles of 256 rows pay anywhere (kvq_plan says where).
constexpr bool tiles_of_256(bool bf16, int d) { return bf16 && d == 128; }

// Fills the split fields from the sizes; returns the bytes of partial results.
uint64_t kvq_plan(KvqAttendArgs &a, bool bf16);
// Upper bound of those bytes over every call with at most these sizes.
uint64_t kvq_plan_bound(int32_t n, int32_t n_q, int32_t kv_heads, int32_t q_heads, int32_t d, int32_t max_len);
hipError_t launch_kvq_tiles(const KvqAttendArgs &a, bool bf16, hipStream_t st);
hipError_t launch_kvq_attend(const KvqAttendArgs &a, bool bf16, hipStream_t st);

}  // namespace sqk
