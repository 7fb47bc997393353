// sq_kvq_attend.hip -- gfx950 kernels of attention over the 8-bit paged cache.
//
//     o = sum_x p_x v_x,  p = softmax_x(scale q.k_x),  x at or before the query
//
// A code is at most 8 bits of a number, so float16 holds it exactly: the codes
// become float16 operands (an integer byte u as 1024 + u, put together by one
// byte permutation for two, less 1152; e4m3 by the conversion instruction) and
// the matrix instructions multiply them without a rounding.  The scales stay
// outside, in fp32:
//   - queries are float16 after a power of two that puts the largest of a row
//     at 2^14 (bfloat16 queries are then exact down to 2^-31 of it, fp32 ones
//     are two float16, 22 bits);
//   - a score is (q.code) times its block's key scale, query scale and `scale`;
//   - a probability is multiplied by its block's value scale over a power of
//     two near the largest one seen (kept like the running maximum: when it grows,
//     the sums so far are scaled down), and rounded to one float16 (11 bits, three
//     more than the bfloat16 output; fp32 outputs take two).
// Scores, maxima, sums of probabilities and outputs are fp32.
//
// A row's maximum starts at -inf and is at least the lowest float once a key
// is seen, so it says by itself whether any was: a row without keys has -inf
// (zeros, log sum -inf), one whose scores are all -inf a sum of zero under a
// finite maximum (NaN, like any score that is NaN or +inf).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sq_grid.h"
#include "sq_kvq.h"
#include "sq_kvq_dev.h"

namespace sqk {

namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr float kInf = __builtin_inff();
constexpr float kFloatMax = 3.402823466e+38f;
constexpr float kTiny = 1.17549435e-38f;
constexpr float kLn2 = 0.69314718055994531f;
// probabilities are kept as float16 times 32: the largest, 2^8 (the tile form lets a
// row's maximum stand until weights pass 2^8) x 2 (value scale) x 32, stays below
// float16's top, and its last place is 2^-29 of a probability of one
constexpr float kProbUp = 32.0f, kProbDown = 1.0f / 32.0f;
constexpr float kGrown = 256.0f;

template <bool E4M3>
__device__ __forceinline__ h4 halves4(uint32_t w)
{
    if constexpr (E4M3) {
        const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
        const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
        return h4{a[0], a[1], b[0], b[1]};
    } else {
        const h2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
        const h2 a = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) - bias;
        const h2 b = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) - bias;
        return h4{a[0], a[1], b[0], b[1]};
    }
}
template <bool E4M3>
__device__ __forceinline__ h8 halves8(uint32_t lo, uint32_t hi)
{
    return __builtin_shufflevector(halves4<E4M3>(lo), halves4<E4M3>(hi), 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ f32x8 row8(const uint16_t *p)
{
    const u32x4_t w = *reinterpret_cast<const u32x4_t *>(p);
    f32x8 x;
#pragma unroll
    for (int i = 0; i < 4; i++) x[2 * i] = bits_f(w[i] << 16), x[2 * i + 1] = bits_f(w[i] & 0xffff0000u);
    return x;
}
__device__ __forceinline__ f32x8 row8(const float *p)
{
    const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ void store4(float *p, f32x4 x) { *reinterpret_cast<f32x4 *>(p) = x; }
__device__ __forceinline__ void store4(uint16_t *p, f32x4 x)
{
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<u32x2_t *>(p) = __builtin_bit_cast(u32x2_t, __builtin_convertvector(x, bf16x4));
}

// x as PARTS float16 whose sum it is to 11 bits each
template <int PARTS>
__device__ __forceinline__ void split8(f32x8 x, h8 (&out)[PARTS])
{
#pragma unroll
    for (int k = 0; k < PARTS; k++) {
        out[k] = __builtin_convertvector(x, h8);
        if (k + 1 < PARTS) x -= __builtin_convertvector(out[k], f32x8);
    }
}

// the power of two that puts `most` at 2^14 .. 2^15 and its inverse
__device__ __forceinline__ void unit_of(float most, float &up, float &down)
{
    uint32_t e = f_bits(most) >> 23;
    e = e < 15 ? 15 : e > 254 ? 254 : e;
    up = bits_f((268 - e) << 23);
    down = bits_f((e - 14) << 23);
}

// 1 / L and log sum exp of a row with maximum M and sum L (base 2): no keys at
// all give 0 and -inf, a sum that is zero or NaN under keys gives NaN
__device__ __forceinline__ float inverse_sum(float M, float L)
{
    return M == -kInf ? 0.0f : L > 0.0f ? 1.0f / L : __builtin_nanf("");
}
__device__ __forceinline__ float log_sum(float M, float L)
{
    if (M == -kInf) return M;
    return L > 0.0f ? (M + __builtin_log2f(L)) * kLn2 : __builtin_nanf("");
}

// Rows of the many-query form's tiles, 32 a wave: two waves on every SIMD where the
// registers allow it.
constexpr int tile_rows(bool bf16, int d) { return d <= 96 || (bf16 && d <= 128) ? 256 : 128; }

// ---------------------------------------------------------------- requests, spans

struct Req {
    int32_t q0, m, len;  // first query, queries, tokens
};

constexpr int32_t kMostTokens = 0x7fffffff - 64;  // rows past a request's last count on by up to 16

__device__ __forceinline__ Req req_of(const KvqAttendArgs &a, int r)
{
    Req q;
    q.q0 = a.cu ? clamp_to(a.cu[r], a.n_q) : r;
    q.m = a.cu ? clamp_to(a.cu[r + 1], a.n_q) - q.q0 : 1;
    q.len = clamp_to(a.lens[r], kMostTokens);
    return q;
}

// the few-query form's requests: one query, or 16 rows at most
__device__ __forceinline__ bool few(const KvqAttendArgs &a, int32_t m)
{
    return a.few_on && (m == 1 || (int64_t)m * a.group <= 16);
}

// Positions that rows with limits in [first_limit, last_limit] see: a row with
// limit L (its position + 1) sees [L - window, L), up to max_len.  Cut from `from` on.
struct Span {
    int32_t first, end, from, splits;
};

__device__ __forceinline__ Span span_of(const KvqAttendArgs &a, int32_t first_limit, int32_t last_limit, int32_t chunk)
{
    Span s;
    s.first = a.window > 0 && first_limit > a.window ? first_limit - a.window : 0;
    s.end = clamp_to(last_limit, a.max_len);
    s.from = s.first & ~63;
    s.splits = s.end > s.from ? (s.end - s.from + chunk - 1) / chunk : 0;
    return s;
}

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

    const Req q = req_of(a, r);
    if (q.m < 1 || !few(a, q.m)) return;
    const int rows = q.m * a.group, row = qt * 16 + c;  // this lane's row
    if (qt * 16 >= rows) return;
    const bool row_in = row < rows;
    const int ti = row / a.group, hd = h * a.group + row % a.group;
    const int64_t out = (int64_t)(q.q0 + ti) * a.q_heads + hd;

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
    const int ps = a.c.page_shift, bs = ps - 4;
    const int32_t *pages_of = a.table + (int64_t)r * a.table_stride;
    const int32_t p0 = begin >> ps, np = ((end - 1) >> ps) - p0 + 1;
    if (threadIdx.x == 0) any_bad = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < np; i += 256) {
        int32_t id = pages_of[p0 + i];
        if ((uint32_t)id >= (uint32_t)a.c.n_pages) {
            id = -1;
            any_bad = 1;
        }
        ids[i] = id;
    }

    // queries: product step i takes d = 64 (i / 2) + 16 g + 8 (i % 2) + e, the last
    // 32 of an odd number of steps 64 NW + 8 g + e
    h8 qf[NS][PARTS];
    float qscale;
    {
        const T *qp = reinterpret_cast<const T *>(a.q) + (int64_t)(q.q0 + ti) * a.q_stride + (int64_t)hd * D;
        f32x8 x[NS];
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < NS; i++) {
            x[i] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
            if (row_in) x[i] = row8(qp + (TAIL && i == NS - 1 ? 64 * NW + 8 * g : 64 * (i / 2) + 16 * g + 8 * (i % 2)));
#pragma unroll
            for (int e = 0; e < 8; e++) most = fmaxf(most, __builtin_fabsf(x[i][e]));
        }
        most = fmaxf(most, __shfl_xor(most, 16));
        most = fmaxf(most, __shfl_xor(most, 32));
        float up, down;
        unit_of(most, up, down);
#pragma unroll
        for (int i = 0; i < NS; i++) split8<PARTS>(x[i] * (up * a.sign), qf[i]);
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
    float vref = 0x1p-111f;  // power of two under the value scales: at most twice it

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
        float mx = in ? -kFloatMax : -kInf;
        float t[16];
#pragma unroll
        for (int e = 0; e < 16; e++) {
            t[e] = x[e / 4][e % 4] * fk;
            if (edge && !(in >> e & 1)) t[e] = -kInf;
            mx = fmaxf(mx, t[e]);
        }
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        if (__ballot(mx > m || sv > 2.0f * vref)) {
            float most = sv;
            most = fmaxf(most, __shfl_xor(most, 16));
            most = fmaxf(most, __shfl_xor(most, 32));
            const float v2 = fmaxf(vref, bits_f(f_bits(most) & 0x7f800000u));
            const float mn = fmaxf(m, mx);
            const float f = mn == -kInf ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
            const float fv = f * (vref / v2);
            vref = v2;
#pragma unroll
            for (int i = 0; i < ND; i++) acc[i] *= fv;
        }
        const float mu = m == -kInf ? 0.0f : m;
        const float wv_ = sv * (kProbUp / vref);
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
    const float f = m == -kInf ? 0.0f : __builtin_amdgcn_exp2f(m - M) * (vref * kProbDown);
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

template <typename T, int D>
__global__ __launch_bounds__(256) void k_kvq_join_few(KvqAttendArgs a)
{
    const unsigned heads = (unsigned)a.c.heads, rows = (unsigned)a.rows;
    const unsigned unit = blockIdx.x / rows, row = blockIdx.x % rows;
    const int r = (int)(unit / heads), h = (int)(unit % heads);
    const Req q = req_of(a, r);
    if (q.m < 1 || !few(a, q.m) || (int)row >= q.m * a.group) return;
    const Span s = span_of(a, q.len - q.m + 1, q.len, a.chunk);
    if (s.splits <= 1) return;  // written already
    const int64_t out = (int64_t)(q.q0 + (int)row / a.group) * a.q_heads + h * a.group + (int)row % a.group;
    const int64_t at = (int64_t)blockIdx.x * a.splits;
    const float *ml = a.part + (int64_t)a.n * heads * rows * a.splits * D;
    join_row<T, D>(a, a.part + at * D, ml + at * 2, s.splits, out);
}

// ---------------------------------------------------------------- many queries
//
// Rows (queries x heads of a group) in tiles of 128, 32 a wave; tokens 64 at a
// time.  A key is used by 128 rows and more, so the matrix instructions and
// the softmax between them bound it, and the codes become float16 once a workgroup,
// on their way into shared memory.  With the 32 x 32 result of an instruction held
// as rows 8 (e / 4) + 4 (lane / 32) + e % 4, column lane % 32:
//     S^T = K Q^T    [64 tokens x 32 rows]
//     O^T += V^T P^T [d x 32 rows]         a step is a block of 16 tokens
// Row m = 8 j + 4 i + e of a product is token 16 (j / 2) + 8 i + 4 (j % 2) + e of 32, so a
// lane's 8 scores of a block are the second product's operand in its own registers.
// One running maximum a row, left standing until a tile passes it by 2^8.

template <typename T, bool E4M3, int D>
__global__ __launch_bounds__(2 * tile_rows(sizeof(T) == 2, D), tile_rows(sizeof(T) == 2, D) / 128) void k_kvq_tiles(KvqAttendArgs a)
{
    constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
    constexpr int ROWS = tile_rows(sizeof(T) == 2, D), WAVES = ROWS / 32, TPB = 64 * WAVES;
    constexpr int NS = D / 16, ND = D / 32;
    constexpr int KP = D + 8, VP = 64 + 8;     // halves from row to row: 16 bytes off a multiple of the banks
    constexpr int PIECES = 4 * D, NP = (PIECES + TPB - 1) / TPB;  // 16-byte pieces of 64 tokens
    __shared__ __align__(16) _Float16 sm_k[2][64 * KP], sm_v[2][D * VP];
    __shared__ f32x4 sm_s[4][4];               // of the four blocks: key scales; value scales, their log2 and inverse

    const int lane = threadIdx.x & 63, hh = lane >> 5, c = lane & 31;
    const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int grp = WAVES == 8 ? wv >> 2 : 0;                       // which half of the waves: the two take turns
    const int part = WAVES == 8 ? (wv & 3) * 2 + grp : wv;          // which 32 rows: few rows spread over both halves
    const unsigned heads = (unsigned)a.c.heads, tiles = (unsigned)a.tiles;
    const int h = (int)(blockIdx.x % heads);
    const int64_t slot = tiles - 1 - blockIdx.x / heads % tiles;  // late tiles see the most: first
    const int sp = (int)(blockIdx.x / heads / tiles);

    const int r = wave_count(a.n, [&](int i) { return (int64_t)clamp_to(a.cu[i], a.n_q) * a.group / ROWS + i <= slot; }) - 1;
    if (r < 0) return;
    const Req q = req_of(a, r);
    if (q.m < 1 || few(a, q.m)) return;
    const int64_t rows = (int64_t)q.m * a.group;
    const int64_t row0 = (slot - ((int64_t)q.q0 * a.group / ROWS + r)) * ROWS;
    if (row0 >= rows) return;
    const bool active = row0 + part * 32 < rows;  // the wave has rows (it stages tokens in any case)
    const int64_t row = row0 + part * 32 + c;
    const bool row_in = row < rows;
    const int32_t ti = (int32_t)((row_in ? row : rows - 1) / a.group);
    const int hd = h * a.group + (int)((row_in ? row : rows - 1) % a.group);
    const int64_t out = (int64_t)(q.q0 + ti) * a.q_heads + hd;

    const int32_t t_first = (int32_t)(row0 / a.group);
    const int32_t t_last = (int32_t)((row0 + ROWS < rows ? row0 + ROWS - 1 : rows - 1) / a.group);
    const int32_t before = q.len - q.m + 1;  // limit of the request's first query
    const Span s = span_of(a, before + t_first, before + t_last, a.t_chunk);
    const int32_t begin = s.from + sp * a.t_chunk;
    const int32_t end = begin + a.t_chunk < s.end ? begin + a.t_chunk : s.end;
    if (begin >= s.end && sp > 0) return;

    // queries: product step i takes d = 16 i + 8 hh + e
    h8 qf[NS][PARTS];
    float qscale;
    {
        const T *qp = reinterpret_cast<const T *>(a.q) + (int64_t)(q.q0 + ti) * a.q_stride + (int64_t)hd * D + 8 * hh;
        f32x8 x[NS];
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < NS; i++) {
            x[i] = row8(qp + 16 * i);
#pragma unroll
            for (int e = 0; e < 8; e++) most = fmaxf(most, __builtin_fabsf(x[i][e]));
        }
        most = fmaxf(most, __shfl_xor(most, 32));
        float up, down;
        unit_of(most, up, down);
#pragma unroll
        for (int i = 0; i < NS; i++) split8<PARTS>(x[i] * (up * a.sign), qf[i]);
        qscale = down * a.scale_log2;
    }

    const int32_t limit = before + ti;  // this lane's row sees [lowest, limit)
    const int32_t lowest = a.window > 0 && limit > a.window ? limit - a.window : 0;
    // tiles inside [low_all, high_all) are seen whole by every row
    const int32_t high_all = before + t_first < end ? before + t_first : end;
    const int32_t low_all = a.window > 0 && before + t_last > a.window ? before + t_last - a.window : 0;

    const int ps = a.c.page_shift, bs = ps - 4;
    const int32_t *pages_of = a.table + (int64_t)r * a.table_stride;
    // A tile's pages: lane b of every four holds block b's, -1 where there is none.  They are
    // asked for two turns before they are used, as one load of a wave.
    auto page_ids = [&](int32_t base) -> int32_t {
        const int32_t x = base + 16 * (lane & 3);
        return x < end ? pages_of[x >> ps] : -1;
    };
    auto gone_of = [&](int32_t id) { return (uint32_t)__ballot((uint32_t)id >= (uint32_t)a.c.n_pages) & 0xfu; };
    // block index (page, head, block) of a tile's block; page 0 stands in for pages that do not exist
    auto block_of = [&](int32_t base, int32_t page, int blk) -> int64_t {
        return (((int64_t)((uint32_t)page < (uint32_t)a.c.n_pages ? page : 0) * heads + h) << bs) +
               (((base >> 4) + blk) & ((1 << bs) - 1));
    };
    // pieces p = thread + TPB j, of keys and of values: piece p % D of block p / D, which is
    // one for the wave, and its address a scalar, where 64 divides D
    const int wave0 = D % 64 ? (int)threadIdx.x : 64 * wv;
    struct Piece {
        u32x4_t w[NP];
    };
    auto fetch = [&](const uint8_t *codes, int32_t base, int32_t id, Piece &p) {
#pragma unroll
        for (int j = 0; j < NP; j++) {
            if (PIECES % TPB != 0 && wave0 + TPB * j >= PIECES) continue;
            const int blk = (wave0 + TPB * j) / D;
            const int64_t b = block_of(base, D % 64 ? __shfl(id, blk) : __builtin_amdgcn_readlane(id, blk), blk);
            p.w[j] = *reinterpret_cast<const u32x4_t *>(codes + b * (16 * D) + (threadIdx.x + TPB * j) % D * 16);
        }
    };
    // a tile's keys, values and scales into shared memory, codes as float16
    auto stage_keys = [&](int buf, const Piece &pc) {
#pragma unroll
        for (int j = 0; j < NP; j++) {
            const int p = threadIdx.x + TPB * j;
            if (PIECES % TPB != 0 && p >= PIECES) continue;
            _Float16 *kd = sm_k[buf] + p / (D / 16) * KP + p % (D / 16) * 16;
            *reinterpret_cast<h8 *>(kd) = halves8<E4M3>(pc.w[j][0], pc.w[j][1]);
            *reinterpret_cast<h8 *>(kd + 8) = halves8<E4M3>(pc.w[j][2], pc.w[j][3]);
        }
    };
    auto stage_values = [&](int buf, int32_t base, uint32_t gone, Piece &pc) {
        // positions outside the span, pages that do not exist: values that no row uses must not be a NaN
        if (base < s.first || base + 64 > end || gone) {
#pragma unroll
            for (int j = 0; j < NP; j++) {
                const int blk = (int)(threadIdx.x + TPB * j) / D;
                const int lo = s.first - (base + 16 * blk), hi = gone >> blk & 1 ? 0 : end - (base + 16 * blk);
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    const int l4 = lo - 4 * w, h4_ = hi - 4 * w;
                    const uint32_t below_hi = h4_ <= 0 ? 0u : h4_ >= 4 ? ~0u : (1u << 8 * h4_) - 1;
                    const uint32_t below_lo = l4 <= 0 ? 0u : l4 >= 4 ? ~0u : (1u << 8 * l4) - 1;
                    pc.w[j][w] &= below_hi & ~below_lo;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NP; j++) {
            const int p = threadIdx.x + TPB * j;
            if (PIECES % TPB != 0 && p >= PIECES) continue;
            _Float16 *vd = sm_v[buf] + p % D * VP + p / D * 16;
            *reinterpret_cast<h8 *>(vd) = halves8<E4M3>(pc.w[j][0], pc.w[j][1]);
            *reinterpret_cast<h8 *>(vd + 8) = halves8<E4M3>(pc.w[j][2], pc.w[j][3]);
        }
    };
    // scales by the first lanes of one wave, block by block: a lane's block of a tile
    const bool scaler = wv == WAVES - 1 && lane < 4;
    auto fetch_scales = [&](int32_t base, int32_t id) {
        f32x2 sc = {1.0f, 0.0f};
        // where no row sees a position of the block, what lies there need not be a scale
        if (scaler) {
            const int32_t x = base + 16 * lane;
            if (x < end && x + 16 > s.first && (uint32_t)id < (uint32_t)a.c.n_pages)
                sc = *reinterpret_cast<const f32x2 *>(a.c.scales + 2 * block_of(base, id, lane));
        }
        return sc;
    };
    auto stage_scales = [&](int ring, f32x2 sc) {
        if (!scaler) return;
        float *to = reinterpret_cast<float *>(sm_s[ring]) + lane;
        to[0] = sc[0], to[4] = sc[1];
        if constexpr (PARTS == 1) to[8] = __builtin_amdgcn_logf(sc[1]), to[12] = sc[1] > 0.0f ? 1.0f / sc[1] : 0.0f;
    };

    f32x16 acc[ND], x[2];
#pragma unroll
    for (int i = 0; i < ND; i++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[i][e] = 0.0f;
    h8 p[4][PARTS];
    float m = -kInf, l = 0.0f;
    float vref = 0x1p-111f;  // power of two under the value scales, and with it what p is kept times
    float up = kProbUp / vref, down = vref * kProbDown, up_log = 116.0f;

    // element 8 (b % 2) + e of x[b / 2] is token 16 b + 8 hh + e of the tile
    const int krow = 16 * (c >> 4) + 8 * ((c >> 2) & 1) + 4 * ((c >> 3) & 1) + (c & 3);  // token of product row c
    auto scores = [&](int buf) {
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
            for (int e = 0; e < 16; e++) x[u][e] = 0.0f;
        const _Float16 *kp = sm_k[buf] + krow * KP + 8 * hh;
#pragma unroll
        for (int i = 0; i < NS; i++)
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const h8 k = *reinterpret_cast<const h8 *>(kp + 32 * u * KP + 16 * i);
#pragma unroll
                for (int k2 = 0; k2 < PARTS; k2++) x[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, qf[i][k2], x[u], 0, 0, 0);
            }
    };
    auto outputs = [&](int buf) {
        const _Float16 *vp = sm_v[buf] + c * VP + 8 * hh;
#pragma unroll
        for (int b = 0; b < 4; b++)
#pragma unroll
            for (int i = 0; i < ND; i++) {
                const h8 v = *reinterpret_cast<const h8 *>(vp + 32 * i * VP + 16 * b);
#pragma unroll
                for (int k2 = 0; k2 < PARTS; k2++) acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, p[b][k2], acc[i], 0, 0, 0);
            }
    };
    // p and the sum of it from x, by the maximum so far
    auto weigh = [&](const f32x4 (&sc)[4], const float (&fk)[4]) {
        const float mu = m == -kInf ? 0.0f : m, c1 = up_log - mu;
        float sum = 0.0f;
#pragma unroll
        for (int b = 0; b < 4; b++) {
            f32x8 t;
            if constexpr (PARTS == 1) {
                // 2^(score - mu) times the value scale in one exponential; the sum takes it out again
                const float c0 = sc[2][b] + c1;
#pragma unroll
                for (int e = 0; e < 8; e++) t[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[b >> 1][8 * (b & 1) + e], fk[b], c0));
                sum = __builtin_fmaf(((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7])), sc[3][b], sum);
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++) t[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[b >> 1][8 * (b & 1) + e], fk[b], -mu));
                sum += ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
                t *= sc[1][b] * up;
            }
            split8<PARTS>(t, p[b]);
        }
        return PARTS == 1 ? sum * down : sum;
    };
    auto weights = [&](int ring, int32_t base, uint32_t gone) {
        const f32x4 sc[4] = {sm_s[ring][0], sm_s[ring][1], sm_s[ring][2], sm_s[ring][3]};
        float fk[4];
#pragma unroll
        for (int b = 0; b < 4; b++) fk[b] = sc[0][b] * qscale;
        bool in = true;
        if (base + 64 > high_all || base < low_all || gone) {
            in = false;
            const int32_t high = limit < end ? limit : end;
#pragma unroll
            for (int b = 0; b < 4; b++) {
                fk[b] = fmaxf(fk[b], kTiny);  // it may be zero, and x is -inf
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int32_t at = base + 16 * b + 8 * hh + e;
                    const bool ok = at < high && at >= lowest && !(gone >> b & 1);
                    in = in || ok;
                    if (!ok) x[b >> 1][8 * (b & 1) + e] = -kInf;
                }
            }
        }
        float sum = weigh(sc, fk);
        // A tile whose weights pass 2^kGrow (their sum says so at the latest), the first of a
        // row, or value scales past their reference: the maximum is found and the weights
        // are made again.  Few tiles do.
        const float most = fmaxf(fmaxf(sc[1][0], sc[1][1]), fmaxf(sc[1][2], sc[1][3]));
        const bool grown = !(sum <= kGrown) || m == -kInf;
        if (__ballot(grown || most > 2.0f * vref)) {
            float mx = in ? -kFloatMax : -kInf;
#pragma unroll
            for (int b = 0; b < 4; b++)
#pragma unroll
                for (int e = 0; e < 8; e++) mx = fmaxf(mx, x[b >> 1][8 * (b & 1) + e] * fk[b]);
            // of the rows that need it alone: what another one holds (a NaN) must not show in a row
            const int other_grown = __shfl_xor((int)grown, 32);
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float mn = grown || other_grown ? fmaxf(m, mx) : m;
            const float f = mn == -kInf ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            const float v2 = fmaxf(vref, bits_f(f_bits(most) & 0x7f800000u)), fv = f * (vref / v2);
            m = mn;
            l *= f;
            vref = v2;
            up = kProbUp / v2, down = v2 * kProbDown, up_log = __builtin_log2f(up);
#pragma unroll
            for (int i = 0; i < ND; i++) acc[i] *= fv;
            sum = weigh(sc, fk);
        }
        l += sum;
    };
    auto turn = [&] {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    };

    // Turns.  A wave's work on tile j is a product turn (the outputs of tile j - 1, the
    // scores of tile j) and a vector turn (the weights of tile j; tokens to come into shared
    // memory).  The second half of eight waves is one turn behind the first, so that on every
    // SIMD one wave multiplies while the other one's vector units work; a barrier ends every
    // turn.  In its vector turn j, half g stages its pieces of keys of tile j + 1 + g and of
    // values of tile j + g: the first half reads both in the next turn, and what they
    // overwrite was read two turns ago and more.  Scales are kept for four tiles: a
    // vector turn reads them while another wave writes later ones.
    if (begin < end) {
        uint32_t gone[3];  // of tiles j + g - 1, j + g, j + g + 1
        Piece kp, vp;
        int32_t idv = page_ids(begin), idk = page_ids(begin + 64);
        fetch(a.c.k, begin, idv, kp);
        f32x2 sc = fetch_scales(begin, idv);
        stage_keys(0, kp);
        stage_scales(0, sc);
        // the first stage in the loop: keys of tile 1 (half 1: tile 1 before the loop, then tile 2), values of tile 0
        int32_t at = begin;  // first position of tile j + g
        gone[0] = 0, gone[1] = gone_of(idv), gone[2] = gone_of(idk);
        fetch(a.c.k, begin + 64, idk, kp);
        fetch(a.c.v, begin, idv, vp);
        sc = fetch_scales(begin + 64, idk);
        idv = idk;
        idk = page_ids(begin + 128);
        turn();
        // stage tile (j + g)'s values and the next one's keys and scales, and ask for those after them
        int n = 0;  // j + g
        auto stage = [&] {
            stage_keys((n + 1) & 1, kp);
            stage_values(n & 1, at, gone[1], vp);
            stage_scales((n + 1) & 3, sc);
            n++;
            at += 64;
            gone[0] = gone[1], gone[1] = gone[2], gone[2] = gone_of(idk);
            if (at < end) fetch(a.c.v, at, idv, vp);
            if (at + 64 < end) {
                fetch(a.c.k, at + 64, idk, kp);
                sc = fetch_scales(at + 64, idk);
            }
            idv = idk;
            idk = page_ids(at + 128);
        };
        if (grp == 1) {
            stage();
            turn();
        }
        int j = 0;
        for (int32_t base = begin; base < end; base += 64, j++) {
            if (active) {
                __builtin_amdgcn_s_setprio(1);
                if (j > 0) outputs((j + 1) & 1);
                scores(j & 1);
                __builtin_amdgcn_s_setprio(0);
            }
            turn();
            if (active) weights(j & 3, base, gone[1 - grp]);
            stage();
            turn();
        }
        if (active) outputs((j + 1) & 1);
        if (WAVES == 8 && grp == 0) turn();
    }

    l += __shfl_xor(l, 32);
    if (!row_in) return;
    if (s.splits <= 1) {
        const float inv = inverse_sum(m, l) * down;
        T *dst = reinterpret_cast<T *>(a.o) + out * D + 4 * hh;
#pragma unroll
        for (int i = 0; i < ND; i++)
#pragma unroll
            for (int j = 0; j < 4; j++)
                store4(dst + 32 * i + 8 * j, f32x4{acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]} * inv);
        if (a.lse && hh == 0) a.lse[out] = log_sum(m, l);
    } else {
        const int64_t at = out * a.t_splits + sp;
        float *part_o = a.part + (int64_t)a.n * heads * a.rows * (a.splits > 1 ? a.splits : 0) * (D + 2);
        float *dst = part_o + at * D + 4 * hh;
#pragma unroll
        for (int i = 0; i < ND; i++)
#pragma unroll
            for (int j = 0; j < 4; j++)
                store4(dst + 32 * i + 8 * j, f32x4{acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]} * down);
        if (hh == 0) {
            float *ml = part_o + (int64_t)a.n_q * a.q_heads * a.t_splits * D + at * 2;
            ml[0] = m;
            ml[1] = l;
        }
    }
}

template <typename T, int D>
__global__ __launch_bounds__(256) void k_kvq_join_tiles(KvqAttendArgs a)
{
    const int64_t out = blockIdx.x;
    const int32_t qi = (int32_t)(out / a.q_heads);
    const int r = wave_count(a.n, [&](int i) { return clamp_to(a.cu[i], a.n_q) <= qi; }) - 1;
    if (r < 0) return;
    const Req q = req_of(a, r);
    if (qi >= q.q0 + q.m || few(a, q.m)) return;
    // the row's tile, as the tiles were cut
    const int64_t rows = (int64_t)q.m * a.group;
    constexpr int ROWS = tile_rows(sizeof(T) == 2, D);
    const int64_t row0 = ((int64_t)(qi - q.q0) * a.group + (int)(out % a.q_heads) % a.group) / ROWS * ROWS;
    const int32_t t_first = (int32_t)(row0 / a.group);
    const int32_t t_last = (int32_t)((row0 + ROWS < rows ? row0 + ROWS - 1 : rows - 1) / a.group);
    const int32_t before = q.len - q.m + 1;
    const Span s = span_of(a, before + t_first, before + t_last, a.t_chunk);
    if (s.splits <= 1) return;  // written already
    const float *part = a.part + (int64_t)a.n * a.c.heads * a.rows * (a.splits > 1 ? a.splits : 0) * (D + 2);
    const int64_t at = out * a.t_splits;
    join_row<T, D>(a, part + at * D, part + (int64_t)a.n_q * a.q_heads * a.t_splits * D + at * 2, s.splits, out);
}

// ---------------------------------------------------------------- launches

template <typename T, bool E4M3, int D>
hipError_t attend_tfd(const KvqAttendArgs &a, hipStream_t st)
{
    const int64_t units = (int64_t)a.n * a.c.heads;
    const int64_t few_grid = units * a.q_tiles * a.splits, few_rows = units * a.rows;
    constexpr int tile_threads = 2 * tile_rows(sizeof(T) == 2, D);
    const int64_t tile_grid = (int64_t)a.tiles * a.c.heads * a.t_splits, tile_rows = (int64_t)a.n_q * a.q_heads;
    if (!grid_fits(few_grid, 256) || (a.splits > 1 && !grid_fits(few_rows, 256)) || !grid_fits(tile_grid, tile_threads) ||
        (a.t_splits > 1 && !grid_fits(tile_rows, 256)))
        return hipErrorInvalidConfiguration;
    if (a.tiles > 0) {
        hipLaunchKernelGGL((k_kvq_tiles<T, E4M3, D>), dim3((unsigned)tile_grid), dim3(tile_threads), 0, st, a);
        if (hipError_t e = hipGetLastError()) return e;
        if (a.t_splits > 1) {
            hipLaunchKernelGGL((k_kvq_join_tiles<T, D>), dim3((unsigned)tile_rows), dim3(256), 0, st, a);
            if (hipError_t e = hipGetLastError()) return e;
        }
    }
    if (a.q_tiles > 0) {
        hipLaunchKernelGGL((k_kvq_few<T, E4M3, D>), dim3((unsigned)few_grid), dim3(256), 0, st, a);
        if (hipError_t e = hipGetLastError()) return e;
        if (a.splits > 1) hipLaunchKernelGGL((k_kvq_join_few<T, D>), dim3((unsigned)few_rows), dim3(256), 0, st, a);
    }
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
constexpr int64_t kTileWgs = 256, kMinTileChunk = 1024;

uint64_t part_bytes(int64_t rows, int32_t d) { return (uint64_t)rows * (uint64_t)(d + 2) * 4; }

int64_t rows_few(bool one, int64_t group) { return one || group > 16 ? group : 16; }

}  // namespace

uint64_t kvq_plan(KvqAttendArgs &a, bool bf16)
{
    const int64_t tile = tile_rows(bf16, a.c.d);
    const bool one = a.cu == nullptr, tiled = !one && a.n_q > 1 && (int64_t)a.n_q * a.group > 16;
    const int64_t heads = a.c.heads, most = a.window > 0 && a.window < a.max_len ? a.window : a.max_len;
    // positions between the first that a request's (tile's) rows see, from a multiple of
    // 64, and the last: a window's rows lie up to 15 (a tile's rows) tokens apart
    auto span = [&](int64_t apart) { return most == a.max_len || most + apart + 63 > a.max_len ? (int64_t)a.max_len : most + apart + 63; };
    uint64_t bytes = 0;

    // one request that may have many queries is left to the tile form, which takes
    // any number; of several, each goes to the form of its own size
    a.few_on = !tiled || a.n > 1;
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
    if (tiled) {
        a.tiles = (int32_t)((int64_t)a.n_q * a.group / tile + a.n);
        const int64_t wgs = (int64_t)a.tiles * heads, n = wgs > kTileWgs / 2 ? 1 : kTileWgs / wgs;
        int64_t c = ((span(tile - 1) + n - 1) / n + 63) / 64 * 64;
        if (c < kMinTileChunk) c = kMinTileChunk;
        const int64_t s = (span(tile - 1) + c - 1) / c;
        a.t_chunk = (int32_t)c;
        a.t_splits = (int32_t)(s < 1 ? 1 : s);
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
    // Tiles: split only where they are at most kTileWgs / 2, into kTileWgs / tiles
    const int64_t whole = (int64_t)n_q * q_heads * ((len + kMinTileChunk - 1) / kMinTileChunk);
    const int64_t tiled = whole < kTileWgs * 256 ? whole : kTileWgs * 256;
    return part_bytes(few, d) + part_bytes(tiled, d);
}

hipError_t launch_kvq_attend(const KvqAttendArgs &a, bool bf16, hipStream_t st)
{
    return bf16 ? attend_t<uint16_t>(a, st) : attend_t<float>(a, st);
}

}  // namespace sqk
