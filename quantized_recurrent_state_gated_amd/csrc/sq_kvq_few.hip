// sq_kvq_few.hip -- gfx950 kernels of attention over the 8-bit paged cache, one or a
// few queries a request, the join of both forms' splits, and how a call is cut;
// sq_kvq_attend.h has how codes and scales are multiplied.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sq_grid.h"
#include "sq_kvq.h"
#include "sq_kvq_attend.h"

namespace sqk {

namespace {

using namespace kvq;

// ---------------------------------------------------------------- few queries
//
// Every code is used by the rows (queries x heads) of its key-value head and by
// nothing else: at most 16 rows, so HBM bounds it.
//
// A workgroup takes one (request, head, tile of 16 rows, split); its four waves
// take every fourth tile of 64 tokens, four blocks.  With the 16 x 16 result of an
// instruction held as rows 4 (lane / 16) + e, column lane % 16:
//     S^T = K Q^T    [tokens x rows]   four products u = 0 .. 3
//     O^T += V^T P^T [d x rows]        two steps of 32 tokens
// Row m of product u is token 16 (m / 4) + 4 u + m % 4, so lane group g holds the
// 16 scores of block g, in order: one key scale, one value scale a lane and tile, its
// 16 bytes of a value column are one load, and the probabilities go from the first product
// to the second in the lane's own registers.  Codes come from HBM in 16-byte
// pieces (the order of d inside a product is free as long as q has the same).
//
// 70 requests to 16,384 tokens, 32 query and 8 key-value heads, d = 128: 223 us for 1.2 GB
// of codes and scales, 5.4 TB/s (a copy of 2 GiB reaches 5.0), and 7 us for the join.  Three
// contexts to 30,001, 20 and 4 heads, d = 64, fp32 queries: 14 and 4 us.  One request of
// 201 tokens: 7.2 us, its loads one behind the other.

constexpr int kMaxChunk = 8192;  // tokens per split at most (page ids kept in shared memory)
constexpr int kPageIds = kMaxChunk / 16 + 4;

template <typename T, bool E4M3, int D>
__global__ __launch_bounds__(256) void k_kvq_few(KvqAttendArgs a)
{
    constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
    constexpr int NW = D / 64, TAIL = D % 64 / 32, NS = D / 32, ND = D / 16;
    __shared__ int32_t ids[kPageIds];
    __shared__ int any_bad;
    __shared__ float sm_m[4][16], sm_l[4][16];
    __shared__ f32x4 sm_o[3][ND][64];

    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
    const unsigned heads = (unsigned)a.c.heads, units = (unsigned)a.n * heads;
    const unsigned unit = blockIdx.x % units, rest = blockIdx.x / units;
    const int r = (int)(unit / heads), h = (int)(unit % heads);
    const int qt = (int)(rest % (unsigned)a.q_tiles), sp = (int)(rest / (unsigned)a.q_tiles);

    // One query a request: the query and, without a window, the split's first page ids are
    // asked for together with the length; none waits for another.
    const int ps = a.c.page_shift, bs = ps - 4;
    const int32_t *pages_of = a.table + (int64_t)r * a.table_stride;
    const int32_t len = a.lens[r];
    const int64_t early_at = ((int64_t)sp * a.chunk >> ps) + threadIdx.x;
    int32_t early = 0;
    if (a.window == 0 && early_at << ps < a.max_len) early = pages_of[early_at];

    const Req q = req_of(a, r, len);
    if (q.m < 1 || !few(a, q.m)) return;
    const int rows = q.m * a.group, row = qt * 16 + c;  // this lane's row
    if (qt * 16 >= rows) return;
    const bool row_in = row < rows;
    const int ti = row / a.group, hd = h * a.group + row % a.group;
    const int64_t out = (int64_t)(q.q0 + ti) * a.q_heads + hd;

    // queries: product step i takes d = 64 (i / 2) + 16 g + 8 (i % 2) + e, the last
    // 32 of an odd number of steps 64 NW + 8 g + e
    f32x8 qx[NS];
    {
        const T *qp = reinterpret_cast<const T *>(a.q) + (int64_t)(q.q0 + ti) * a.q_stride + (int64_t)hd * D;
#pragma unroll
        for (int i = 0; i < NS; i++) {
            qx[i] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
            if (row_in) qx[i] = row8(qp + (TAIL && i == NS - 1 ? 64 * NW + 8 * g : 64 * (i / 2) + 16 * g + 8 * (i % 2)));
        }
    }

    const Span s = span_of(a, q.len - q.m + 1, q.len, a.chunk);
    const int32_t begin = s.from + sp * a.chunk;
    const int32_t end = begin + a.chunk < s.end ? begin + a.chunk : s.end;
    if (begin >= s.end && sp > 0) return;
    if (s.splits == 0) {  // no tokens: zeros, and the logarithm of an empty sum
        if (wv == 0 && row_in) {
            T *dst = reinterpret_cast<T *>(a.o) + out * D;
#pragma unroll
            for (int i = 0; i < ND; i++) store4(dst + 16 * i + 4 * g, f32x4{0, 0, 0, 0});
            if (a.lse && g == 0) a.lse[out] = -kInf;
        }
        return;
    }

    // the split's page ids; an id outside the cache is kept as -1, its keys are masked
    const int32_t p0 = begin >> ps, np = ((end - 1) >> ps) - p0 + 1;
    if (threadIdx.x == 0) any_bad = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < np; i += 256) {
        int32_t id = a.window == 0 && i < 256 ? early : pages_of[p0 + i];  // without a window p0 is early_at's first
        if ((uint32_t)id >= (uint32_t)a.c.n_pages) {
            id = -1;
            any_bad = 1;
        }
        ids[i] = id;
    }

    h8 qf[NS][PARTS];
    float qscale;
    {
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < NS; i++)
#pragma unroll
            for (int e = 0; e < 8; e++) most = fmaxf(most, __builtin_fabsf(qx[i][e]));
        most = fmaxf(most, __shfl_xor(most, 16));
        most = fmaxf(most, __shfl_xor(most, 32));
        float up, down;
        unit_of(most, up, down);
#pragma unroll
        for (int i = 0; i < NS; i++) split8<PARTS>(qx[i] * (up * a.sign), qf[i]);
        qscale = down * a.scale_log2;
    }
    __syncthreads();
    const bool bad = any_bad != 0;

    const int32_t limit = q.len - q.m + 1 + ti;  // this lane's row sees [lowest, limit)
    const int32_t lowest = a.window > 0 && limit > a.window ? limit - a.window : 0;
    // tiles inside [low_all, high_all) are seen whole by every row
    const int32_t high_all = q.len - q.m + 1 < end ? q.len - q.m + 1 : end;
    const int32_t low_all = a.window > 0 && q.len > a.window ? q.len - a.window : 0;

    // block index (page, head, block) of position x; pages that do not exist and
    // positions past the split read some block that does, and are masked
    auto block_of = [&](int32_t x) -> int64_t {
        const int32_t id = ids[((x < end ? x : end - 1) >> ps) - p0];
        return ((((int64_t)(id < 0 ? 0 : id) * heads + h) << bs)) + ((x >> 4) & ((1 << bs) - 1));
    };

    f32x4 acc[ND];
#pragma unroll
    for (int i = 0; i < ND; i++) acc[i] = f32x4{0, 0, 0, 0};
    float m = -kInf, l = 0.0f;
    float ref = 0.0f;  // the row's largest weight, times 2^m

    u32x4_t kf[4][NW > 0 ? NW : 1];
    u32x2_t kt[4];
    f32x2 sc;
    auto load_k = [&](int32_t base) {
        const uint8_t *kp = a.c.k + block_of(base + 16 * (c >> 2)) * (16 * D) + (c & 3) * D;
#pragma unroll
        for (int u = 0; u < 4; u++) {
#pragma unroll
            for (int i = 0; i < NW; i++) kf[u][i] = *reinterpret_cast<const u32x4_t *>(kp + 4 * u * D + 64 * i + 16 * g);
            if (TAIL) kt[u] = *reinterpret_cast<const u32x2_t *>(kp + 4 * u * D + 64 * NW + 8 * g);
        }
    };

    int32_t base = begin + wv * 64;
    if (base < end) load_k(base);
    for (; base < end; base += 256) {
        u32x4_t vf[ND];
        {
            const int64_t b = block_of(base + 16 * g);
            sc = *reinterpret_cast<const f32x2 *>(a.c.scales + 2 * b);
            const uint8_t *vp = a.c.v + b * (16 * D) + c * 16;
#pragma unroll
            for (int i = 0; i < ND; i++) vf[i] = *reinterpret_cast<const u32x4_t *>(vp + 256 * i);
        }
        f32x4 x[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
            x[u] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < NS; i++) {
                const h8 k = TAIL && i == NS - 1 ? halves8<E4M3>(kt[u][0], kt[u][1])
                                                 : halves8<E4M3>(kf[u][i / 2][2 * (i % 2)], kf[u][i / 2][2 * (i % 2) + 1]);
#pragma unroll
                for (int k2 = 0; k2 < PARTS; k2++)
                    x[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, qf[i][k2], x[u], 0, 0, 0);
            }
        }
        if (base + 256 < end) load_k(base + 256);

        const bool edge = base + 64 > high_all || base < low_all || bad;
        uint32_t in = 0xffffu;  // the tokens of this lane's block that its row sees
        float sk = sc[0], sv = sc[1];
        if (edge) {
            const int32_t x0 = base + 16 * g;
            const bool gone = x0 >= end || ids[(x0 >> ps) - p0] < 0;
            in = 0;
            uint32_t held = 0;  // the tokens whose values are used by some row
#pragma unroll
            for (int e = 0; e < 16; e++) {
                in |= (uint32_t)(!gone && x0 + e < (limit < end ? limit : end) && x0 + e >= lowest) << e;
                held |= (uint32_t)(!gone && x0 + e < end && x0 + e >= s.first) << e;
            }
            if (!held) sk = 1.0f, sv = 0.0f;  // what lies there need not be a scale
            // nor must a NaN there meet a zero
#pragma unroll
            for (int w = 0; w < 4; w++) {
                const uint32_t n = held >> 4 * w & 0xf;
                const uint32_t keep = (n & 1 ? 0xffu : 0) | (n & 2 ? 0xff00u : 0) | (n & 4 ? 0xff0000u : 0) | (n & 8 ? 0xff000000u : 0);
#pragma unroll
                for (int i = 0; i < ND; i++) vf[i][w] &= keep;
            }
        }
        const float fk = fmaxf(sk * qscale, kTiny);
        float mb = -kInf;  // of the block
        float t[16];
#pragma unroll
        for (int e = 0; e < 16; e++) {
            t[e] = rounded(x[e / 4][e % 4], fk);
            if (edge && !(in >> e & 1)) t[e] = -kInf;
            mb = fmaxf(mb, t[e]);
        }
        float mx = fmaxf(in ? -kFloatMax : -kInf, mb);
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        if (__ballot(mx > m || top_weight(mb, m, sv) > ref)) {  // rows that need neither keep their bits
            const float mn = fmaxf(m, mx);
            const float f = mn == -kInf ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
            float top = top_weight(mb, mn, sv);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float r2 = fmaxf(fmaxf(ref * f, top), kLeastRef);
            const float fv = f * (ref / r2);
            ref = r2;
#pragma unroll
            for (int i = 0; i < ND; i++) acc[i] *= fv;
        }
        const float mu = m == -kInf ? 0.0f : m;
        const float wv_ = factor_of(sv, kProbUp / ref);
#pragma unroll
        for (int e = 0; e < 16; e++) {
            t[e] = __builtin_amdgcn_exp2f(t[e] - mu);
            l += t[e];
            t[e] *= wv_;
        }
#pragma unroll
        for (int k = 0; k < 2; k++) {
            h8 p[PARTS];
            split8<PARTS>(f32x8{t[8 * k], t[8 * k + 1], t[8 * k + 2], t[8 * k + 3], t[8 * k + 4], t[8 * k + 5],
                                t[8 * k + 6], t[8 * k + 7]}, p);
#pragma unroll
            for (int i = 0; i < ND; i++) {
                const h8 v = halves8<E4M3>(vf[i][2 * k], vf[i][2 * k + 1]);
#pragma unroll
                for (int k2 = 0; k2 < PARTS; k2++) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p[k2], acc[i], 0, 0, 0);
            }
        }
    }

    // join the four waves: a common maximum, then the sums
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
        sm_m[wv][c] = m;
        sm_l[wv][c] = l;
    }
    __syncthreads();
    float M = sm_m[0][c];
#pragma unroll
    for (int w = 1; w < 4; w++) M = fmaxf(M, sm_m[w][c]);
    float L = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; w++) {
        const float mw = sm_m[w][c];
        L += mw == -kInf ? 0.0f : sm_l[w][c] * __builtin_amdgcn_exp2f(mw - M);
    }
    const float f = m == -kInf ? 0.0f : __builtin_amdgcn_exp2f(m - M) * (ref * kProbDown);
#pragma unroll
    for (int i = 0; i < ND; i++) acc[i] *= f;
    if (wv > 0) {
#pragma unroll
        for (int i = 0; i < ND; i++) sm_o[wv - 1][i][lane] = acc[i];
    }
    __syncthreads();
    if (wv > 0 || !row_in) return;
#pragma unroll
    for (int i = 0; i < ND; i++) acc[i] += sm_o[0][i][lane] + sm_o[1][i][lane] + sm_o[2][i][lane];
    if (s.splits == 1) {
        const float inv = inverse_sum(M, L);
        T *dst = reinterpret_cast<T *>(a.o) + out * D;
#pragma unroll
        for (int i = 0; i < ND; i++) store4(dst + 16 * i + 4 * g, acc[i] * inv);
        if (a.lse && g == 0) a.lse[out] = log_sum(M, L);
    } else {
        const int64_t at = ((int64_t)unit * a.rows + row) * a.splits + sp;
        float *dst = a.part + at * D;
#pragma unroll
        for (int i = 0; i < ND; i++) store4(dst + 16 * i + 4 * g, acc[i]);
        if (g == 0) {
            float *ml = a.part + (int64_t)units * a.rows * a.splits * D + at * 2;
            ml[0] = M;
            ml[1] = L;
        }
    }
}

// ---------------------------------------------------------------- join of splits

constexpr int kWaveSplits = 8;  // up to so many splits of a tile a wave joins a row

// A workgroup joins one row: its four waves take every fourth split, four in flight.
template <typename T, int D>
__device__ __forceinline__ void join_row(const KvqAttendArgs &a, const float *src, const float *ml, int splits, int64_t out)
{
    constexpr int PER = (D + 63) / 64, IN = 4;
    __shared__ float sm_o[4][PER * 64], sm_l[4], sm_m[4];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    float M = -kInf;
    for (int i = threadIdx.x; i < splits; i += 256) M = fmaxf(M, ml[2 * i]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) M = fmaxf(M, __shfl_xor(M, d));
    if (lane == 0) sm_m[wv] = M;
    __syncthreads();
    M = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
    float o[PER], L = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; j++) o[j] = 0.0f;
    for (int i0 = wv; i0 < splits; i0 += 4 * IN) {
        float m[IN], l[IN], x[IN][PER];
#pragma unroll
        for (int u = 0; u < IN; u++) {
            const int i = i0 + 4 * u;
            const bool in = i < splits;
            m[u] = in ? ml[2 * i] : -kInf;
            l[u] = in ? ml[2 * i + 1] : 0.0f;
#pragma unroll
            for (int j = 0; j < PER; j++) {
                const int d = j * 64 + lane;
                x[u][j] = in && d < D ? src[(int64_t)i * D + d] : 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < IN; u++) {
            const float f = m[u] == -kInf ? 0.0f : __builtin_amdgcn_exp2f(m[u] - M);
            L = fmaf(l[u], f, L);
#pragma unroll
            for (int j = 0; j < PER; j++) o[j] = fmaf(x[u][j], f, o[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < PER; j++) sm_o[wv][j * 64 + lane] = o[j];
    if (lane == 0) sm_l[wv] = L;
    __syncthreads();
    L = sm_l[0] + sm_l[1] + sm_l[2] + sm_l[3];
    const float inv = inverse_sum(M, L);
    T *dst = reinterpret_cast<T *>(a.o) + out * D;
    for (int d = threadIdx.x; d < D; d += 256) {
        const float y = (sm_o[0][d] + sm_o[1][d] + sm_o[2][d] + sm_o[3][d]) * inv;
        if constexpr (sizeof(T) == 4) dst[d] = y;
        else dst[d] = __builtin_bit_cast(uint16_t, (__bf16)y);
    }
    if (a.lse && threadIdx.x == 0) a.lse[out] = log_sum(M, L);
}

// The same by one wave, for few splits.
template <typename T, int D>
__device__ __forceinline__ void join_row_wave(const KvqAttendArgs &a, const float *src, const float *ml, int splits, int64_t out)
{
    constexpr int PER = (D + 63) / 64;
    const int lane = threadIdx.x & 63;
    float M = -kInf;
    for (int i = 0; i < splits; i++) M = fmaxf(M, ml[2 * i]);
    float o[PER], L = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; j++) o[j] = 0.0f;
    for (int i = 0; i < splits; i++) {
        const float m = ml[2 * i], f = m == -kInf ? 0.0f : __builtin_amdgcn_exp2f(m - M);
        L = fmaf(ml[2 * i + 1], f, L);
#pragma unroll
        for (int j = 0; j < PER; j++) {
            const int d = j * 64 + lane;
            if (D % 64 == 0 || d < D) o[j] = fmaf(src[(int64_t)i * D + d], f, o[j]);
        }
    }
    const float inv = inverse_sum(M, L);
    T *dst = reinterpret_cast<T *>(a.o) + out * D;
#pragma unroll
    for (int j = 0; j < PER; j++) {
        const int d = j * 64 + lane;
        if (D % 64 != 0 && d >= D) continue;
        if constexpr (sizeof(T) == 4) dst[d] = o[j] * inv;
        else dst[d] = __builtin_bit_cast(uint16_t, (__bf16)(o[j] * inv));
    }
    if (a.lse && lane == 0) a.lse[out] = log_sum(M, L);
}

// row `id` of the few-query form's partial results
template <typename T, int D>
__device__ __forceinline__ void join_few(const KvqAttendArgs &a, unsigned id)
{
    const unsigned heads = (unsigned)a.c.heads, rows = (unsigned)a.rows;
    const unsigned unit = id / rows, row = id % rows;
    const int r = (int)(unit / heads), h = (int)(unit % heads);
    const Req q = req_of(a, r);
    if (q.m < 1 || !few(a, q.m) || (int)row >= q.m * a.group) return;
    const Span s = span_of(a, q.len - q.m + 1, q.len, a.chunk);
    if (s.splits <= 1) return;  // written already
    const int64_t out = (int64_t)(q.q0 + (int)row / a.group) * a.q_heads + h * a.group + (int)row % a.group;
    const int64_t at = (int64_t)id * a.splits;
    const float *ml = a.part + (int64_t)a.n * heads * rows * a.splits * D;
    join_row<T, D>(a, a.part + at * D, ml + at * 2, s.splits, out);
}

// row `out` of the outputs, of the tile form's
template <typename T, int D>
__device__ __forceinline__ void join_tiles(const KvqAttendArgs &a, int64_t out)
{
    const int32_t qi = (int32_t)(out / a.q_heads);
    const int r = wave_count(a.n, [&](int i) { return clamp_to(a.cu[i], a.n_q) <= qi; }) - 1;
    if (r < 0) return;
    const Req q = req_of(a, r);
    if (qi < q.q0 || qi >= q.q0 + q.m || few(a, q.m)) return;  // padding; offsets that fall
    // the row's tile, as the tiles were cut
    const int64_t rows = (int64_t)q.m * a.group;
    const int64_t tile = a.tile_rows;
    const int64_t row0 = ((int64_t)(qi - q.q0) * a.group + (int)(out % a.q_heads) % a.group) / tile * tile;
    const int32_t t_first = (int32_t)(row0 / a.group);
    const int32_t t_last = (int32_t)((row0 + tile < rows ? row0 + tile - 1 : rows - 1) / a.group);
    const int32_t before = q.len - q.m + 1;
    const Span s = span_of(a, before + t_first, before + t_last, a.t_chunk);
    if (s.splits <= 1) return;  // written already
    const float *part = a.part + (int64_t)a.n * a.c.heads * a.rows * (a.splits > 1 ? a.splits : 0) * (D + 2);
    const int64_t at = out * a.t_splits;
    const float *ml = part + (int64_t)a.n_q * a.q_heads * a.t_splits * D + at * 2;
    if (a.t_splits <= kWaveSplits) join_row_wave<T, D>(a, part + at * D, ml, s.splits, out);
    else join_row<T, D>(a, part + at * D, ml, s.splits, out);
}

// Both forms' rows in one launch, those of the tiles first: a workgroup each, or a wave
// each where there are few splits.
template <typename T, int D>
__global__ __launch_bounds__(256) void k_kvq_join(KvqAttendArgs a, unsigned tile_wgs)
{
    if (blockIdx.x >= tile_wgs) {
        join_few<T, D>(a, blockIdx.x - tile_wgs);
    } else if (a.t_splits <= kWaveSplits) {
        const int64_t out = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
        if (out < (int64_t)a.n_q * a.q_heads) join_tiles<T, D>(a, out);
    } else {
        join_tiles<T, D>(a, blockIdx.x);
    }
}

// ---------------------------------------------------------------- launches

template <typename T, bool E4M3, int D>
hipError_t attend_tfd(const KvqAttendArgs &a, hipStream_t st)
{
    const int64_t units = (int64_t)a.n * a.c.heads;
    const int64_t few_grid = units * a.q_tiles * a.splits, tile_grid = (int64_t)a.tiles * a.c.heads * a.t_splits;
    const int64_t few_rows = a.splits > 1 ? units * a.rows : 0, rows = a.t_splits > 1 ? (int64_t)a.n_q * a.q_heads : 0;
    const int64_t tile_wgs = a.t_splits <= kWaveSplits ? (rows + 3) / 4 : rows;
    if (!grid_fits(few_grid, 256) || !grid_fits(tile_grid, 2 * a.tile_rows) || !grid_fits(few_rows + tile_wgs, 256))
        return hipErrorInvalidConfiguration;
    if (a.tiles > 0)
        if (hipError_t e = launch_kvq_tiles(a, sizeof(T) == 2, st)) return e;
    if (a.q_tiles > 0) {
        hipLaunchKernelGGL((k_kvq_few<T, E4M3, D>), dim3((unsigned)few_grid), dim3(256), 0, st, a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    if (few_rows + tile_wgs > 0)
        hipLaunchKernelGGL((k_kvq_join<T, D>), dim3((unsigned)(few_rows + tile_wgs)), dim3(256), 0, st, a, (unsigned)tile_wgs);
    return hipGetLastError();
}

template <typename T, bool E4M3>
hipError_t attend_tf(const KvqAttendArgs &a, hipStream_t st)
{
    switch (a.c.d) {
    case 32: return attend_tfd<T, E4M3, 32>(a, st);
    case 64: return attend_tfd<T, E4M3, 64>(a, st);
    case 96: return attend_tfd<T, E4M3, 96>(a, st);
    case 128: return attend_tfd<T, E4M3, 128>(a, st);
    case 192: return attend_tfd<T, E4M3, 192>(a, st);
    case 256: return attend_tfd<T, E4M3, 256>(a, st);
    default: return hipErrorInvalidValue;
    }
}

template <typename T>
hipError_t attend_t(const KvqAttendArgs &a, hipStream_t st)
{
    return a.c.e4m3 ? attend_tf<T, true>(a, st) : attend_tf<T, false>(a, st);
}

// Few queries: as the 16-bit cache's single-token form, workgroups of even size
// that fill the card several times over where there is work for it.
constexpr int64_t kMost = 4096, kFew = 512, kLongSplit = 2048, kMinChunk = 256;

// Many queries: splits only where the tiles alone leave the card idle.
constexpr int64_t kCus = 256, kMinTileChunk = 1024;

uint64_t part_bytes(int64_t rows, int32_t d) { return (uint64_t)rows * (uint64_t)(d + 2) * 4; }

// rows of a (request, head), in fours where the tile form's partial results come behind them
int64_t rows_few(bool one, int64_t group) { return one ? group : group > 16 ? (group + 3) / 4 * 4 : 16; }

}  // namespace

uint64_t kvq_plan(KvqAttendArgs &a, bool bf16)
{
    const bool one = a.cu == nullptr, tiled = !one && a.n_q > 1 && (int64_t)a.n_q * a.group > 16;
    const int64_t heads = a.c.heads, most = a.window > 0 && a.window < a.max_len ? a.window : a.max_len;
    // positions between the first that a request's (tile's) rows see, from a multiple of
    // 64, and the last: a window's rows lie up to 15 (a tile's rows) tokens apart
    auto span = [&](int64_t apart) { return most == a.max_len || most + apart + 63 > a.max_len ? (int64_t)a.max_len : most + apart + 63; };
    uint64_t bytes = 0;

    // The tile form takes any number of queries.  The other one is worth its launches where
    // requests of few queries are likely (the mean says so) or have long contexts: single
    // tokens among prompts, 8 heads of 4: 31 beside a prompt of 512 over 500, 1,000, 2,000 and 8,000
    // tokens 57, 78, 95 and 271 us with it, 42, 55, 102 and 295 without; 12 beside 4 of 200 42, 58, 90 and
    // 202, and 30, 45, 76 and 270.
    a.few_on = !tiled || (a.n > 1 && (most > 2048 || (int64_t)a.n_q * a.group <= 16 * (int64_t)a.n));
    a.rows = (int32_t)rows_few(one, a.group);
    a.q_tiles = a.few_on ? (a.rows + 15) / 16 : 0;
    a.chunk = 256;
    a.splits = 1;
    if (a.few_on) {
        const int64_t all = most * a.n * heads * a.q_tiles;
        int64_t c = (all + kFew - 1) / kFew;
        if (c > kLongSplit) c = kLongSplit;
        if (c < (all + kMost - 1) / kMost) c = (all + kMost - 1) / kMost;
        if (c < kMinChunk) c = kMinChunk;
        c = (c + 255) / 256 * 256;  // whole rounds of four waves' tiles
        if (c > kMaxChunk) c = kMaxChunk;
        const int64_t s = (span(15) + c - 1) / c;
        a.chunk = (int32_t)c;
        a.splits = (int32_t)(s < 1 ? 1 : s);
        if (a.splits > 1) bytes += part_bytes(a.n * heads * a.rows * a.splits, a.c.d);
    }

    a.tiles = 0;
    a.t_chunk = 64;
    a.t_splits = 1;
    a.tile_rows = 128;
    if (tiled) {
        auto cut = [&](int32_t rows) {
            a.tile_rows = rows;
            a.tiles = (int32_t)((int64_t)a.n_q * a.group / rows + a.n);
            // what is likely of them: every request may end in a part of a tile, or have none
            const int64_t all = (int64_t)a.n_q * a.group, likely = a.n == 1 ? (all + rows - 1) / rows : all / rows + a.n / 4;
            const int64_t wgs = (likely < 1 ? 1 : likely) * heads;
            const int64_t at_once = rows == 128 && two_a_simd(bf16, a.c.d) ? 2 * kCus : kCus;
            const int64_t n = wgs > at_once / 2 ? 1 : at_once / wgs;
            int64_t c = ((span(rows - 1) + n - 1) / n + 63) / 64 * 64;
            if (c < kMinTileChunk) c = kMinTileChunk;
            int64_t s = (span(rows - 1) + c - 1) / c;
            // a split saves turns (of 64 tokens, 2.2 us) and costs a launch, and partial
            // results written and read: 26,000 rows x 2 splits some 25 us
            const int64_t out = (int64_t)a.n_q * a.q_heads, turns = span(rows - 1) / 64;
            if (s > 1 && turns - turns / s <= 4 + out / 2500 + out * s * a.c.d / 1100000) {
                s = 1;
                c = (span(rows - 1) + 63) / 64 * 64;
            }
            a.t_chunk = (int32_t)(c < 64 ? 64 : c);
            a.t_splits = (int32_t)(s < 1 ? 1 : s);
        };
        // Tiles of 256 rows stage a token half as often, and their waves take turns; of 128
        // rows there are two workgroups a unit, each of which ends beside the other's work.
        // Measured (8 heads of 4, us with 256 and 128):
        //   long contexts, many rounds of tiles: one prompt of 8,192 595 and 614
        //   fewer rounds, the last one decides: one of 6,000 350 and 341, 8 x 512 behind 4,000
        //   325 and 333, 6 ragged behind 6,000 289 and 277
        //   short ones: 20 x 800 239 and 217, 8,192 tokens in a window of 1,024 205 and 195
        //   few rows, 256 hold them as well as 2 x 128: 33 behind 60,000 73 and 82, 30 x 40
        //   behind 8,000 267 and 298; not so: 20 behind 60,000 70 and 54, 80 behind 30,000
        //   81 and 74
        // and where d is not 128, or two float16 stand for a query, 128 everywhere (d = 64, one
        // prompt of 8,192: 504 and 420, 20 x 800 197 and 155).
        const int64_t mean = ((int64_t)a.n_q * a.group + a.n - 1) / a.n;
        const bool even = (mean + 255) / 256 * 256 <= (mean + 127) / 128 * 128;
        if (tiles_of_256(bf16, a.c.d) && most >= 4096 && even) cut(256);
        if (a.tile_rows == 128 || (mean > 256 && (int64_t)a.tiles * heads < 3 * kCus)) cut(128);
        if (a.t_splits > 1) bytes += part_bytes((int64_t)a.n_q * a.q_heads * a.t_splits, a.c.d);
    }
    return bytes;
}

uint64_t kvq_plan_bound(int32_t n, int32_t n_q, int32_t kv_heads, int32_t q_heads, int32_t d, int32_t max_len)
{
    // Few queries: R rows in units of at most 16 rows.  Splits are at least 256 tokens:
    // R ceil(len / 256).  They are cut for kMost workgroups: with splits of c tokens,
    // c >= most units / kMost and at most (most + 78) / c + 1 of them, where most > 178 if
    // there are two: R splits <= 1.44 x 16 kMost + R; or c is kMaxChunk.
    const int64_t group = q_heads / kv_heads, len = max_len;
    const int64_t R = (int64_t)n * kv_heads * rows_few(false, group);
    const int64_t fine = (len + kMinChunk - 1) / kMinChunk, coarse = (len + kMaxChunk - 1) / kMaxChunk;
    const int64_t cut = 24 * kMost + R > R * coarse ? 24 * kMost + R : R * coarse;
    const int64_t few = R * fine < cut ? R * fine : cut;
    // Tiles of 256 rows: rows <= 512 x the tiles they are taken for, which are split only
    // if their workgroups are at most kCus / 2, into kCus over their number; or of 128
    // rows, and twice as many workgroups
    const int64_t whole = (int64_t)n_q * q_heads * ((len + kMinTileChunk - 1) / kMinTileChunk);
    const int64_t tiled = whole < kCus * 512 ? whole : kCus * 512;
    return part_bytes(few, d) + part_bytes(tiled, d);
}

hipError_t launch_kvq_attend(const KvqAttendArgs &a, bool bf16, hipStream_t st)
{
    return bf16 ? attend_t<uint16_t>(a, st) : attend_t<float>(a, st);
}

}  // namespace sqk
