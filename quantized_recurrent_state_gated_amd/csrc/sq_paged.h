// sq_paged.h -- internal interface between the host code (sq_serve_api.hip)
// and the kernels of the paged key-value cache (sq_paged.hip): block tables,
// append, decode attention.  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sqk {

struct TableArgs {
    const int32_t *ctx, *fresh;  // [n] cached tokens, new tokens
    const int32_t *free_pages;   // [n_free]
    int32_t n, n_free;
    int32_t page_shift;          // log2(page size)
    int32_t *table;              // [n][stride]
    int64_t stride;
    int32_t *seq;                // [n]
    int32_t *cu_new, *cu_pages;  // [n + 1]
    int64_t *slots;              // [capacity]
    int64_t capacity;
    int32_t *result;
};

hipError_t launch_tables(const TableArgs &a, hipStream_t st);

// The cache both kernels address: keys [page][head][token][d], values
// [page][head][d][token].
struct CacheArgs {
    void *k, *v;
    int32_t n_pages, page_shift, heads, d;
};

struct AppendArgs {
    CacheArgs c;
    const void *k, *v;           // [n][heads][d], tokens k_stride / v_stride elements apart
    int64_t k_stride, v_stride;
    const int64_t *slots;        // [n]
    int32_t n;
};

hipError_t launch_append(const AppendArgs &a, bool bf16, hipStream_t st);

struct AttendArgs {
    CacheArgs c;
    const void *q;               // [n][q_heads][d], requests q_stride elements apart
    int64_t q_stride;
    const int32_t *table;        // [n][table_stride]
    int64_t table_stride;
    const int32_t *lens;         // [n]
    int32_t n, q_heads, group;   // group = q_heads / c.heads
    int32_t q_tiles;             // ceil(group / 16)
    int32_t max_len, window;
    int32_t chunk, splits;       // tokens per split, splits of the longest request
    float scale_log2;            // scale * log2(e)
    void *o;                     // [n][q_heads][d]
    float *lse;                  // [n][q_heads] or null
    float *part;                 // [n][q_heads][splits][d], then [n][q_heads][splits][2] (max, sum)
};

// Tokens per split and number of splits for n requests of up to max_len tokens.
void attend_split(int32_t n, int32_t heads, int32_t q_tiles, int32_t max_len, int32_t *chunk,
                  int32_t *splits);
// Upper bound of rows x splits over every call with at most n requests and
// max_len tokens (each of the partial results is one such row).
uint64_t attend_rows_bound(int32_t n, int32_t kv_heads, int32_t q_heads, int32_t max_len);
bool attend_head_dim(int32_t d);
hipError_t launch_attend(const AttendArgs &a, bool bf16, hipStream_t st);

}  // namespace sqk
