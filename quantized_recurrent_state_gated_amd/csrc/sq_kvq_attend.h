// sq_kvq_attend.h -- what the kernels of attention over the 8-bit paged cache share
// (sq_kvq_few.hip, sq_kvq_tiles.hip).  Not installed, not part of the ABI.
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
//   - a probability is multiplied by its block's value scale over the largest such
//     product that its row has seen (kept like the running maximum: when it grows, the sums
//     so far are scaled down), and rounded to one float16 (11 bits, three more than
//     the bfloat16 output; fp32 outputs take two).  That reference is the row's own: tokens
//     that it does not see, or whose weight is small, do not move it.
// Scores, maxima, sums of probabilities and outputs are fp32.  Differences to the maximum
// are taken of the products that it was found among, rounded as they were there:
// past 2^24 a fused product and sum can lie a power of two and more above it.
//
// A row's maximum starts at -inf and is at least the lowest float once a key
// is seen, so it says by itself whether any was: a row without keys has -inf
// (zeros, log sum -inf), one whose scores are all -inf a sum of zero under a
// finite maximum (NaN, like any score that is NaN or +inf).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sq_kvq.h"
#include "sq_kvq_dev.h"

namespace sqk {

namespace kvq {

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
// Weights (probabilities times value scales over the reference) are kept as float16 times 32:
// its last place is 2^-29 of a weight of one.  The tile form lets maximum and reference stand
// until a lane's probabilities of a tile pass 2^8, or its weights float16's top.
constexpr float kProbUp = 32.0f, kProbDown = 1.0f / 32.0f;
constexpr float kGrown = 256.0f, kMostWeight = 32768.0f;
// Probabilities of 2^-120 and less may lose their bits, or count as zero: they do not enter the reference,
// and the factor that makes weights of them ends at 2^126.  References end at 2^-111,
// under the smallest scale.
constexpr float kLeastProb = -120.0f, kMostFactor = 0x1p126f, kLeastRef = 0x1p-111f;

// a product that is not fused with what it is added to
__device__ __forceinline__ float rounded(float a, float b)
{
#pragma clang fp contract(off)
    return a * b;
}
// weight (before it is divided by the reference) of a block's largest score
__device__ __forceinline__ float top_weight(float score, float m, float scale)
{
    const float d = score - m;
    return d >= kLeastProb ? __builtin_amdgcn_exp2f(d) * scale : 0.0f;
}
// what turns a block's probabilities into weights
__device__ __forceinline__ float factor_of(float scale, float up) { return fminf(scale * up, kMostFactor); }

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

// ---------------------------------------------------------------- requests, spans

struct Req {
    int32_t q0, m, len;  // first query, queries, tokens
};

constexpr int32_t kMostTokens = 0x7fffffff - 64;  // rows past a request's last count on by up to 16

__device__ __forceinline__ Req req_of(const KvqAttendArgs &a, int r, int32_t len)
{
    Req q;
    q.q0 = a.cu ? clamp_to(a.cu[r], a.n_q) : r;
    q.m = a.cu ? clamp_to(a.cu[r + 1], a.n_q) - q.q0 : 1;
    q.len = clamp_to(len, kMostTokens);
    return q;
}
__device__ __forceinline__ Req req_of(const KvqAttendArgs &a, int r) { return req_of(a, r, a.lens[r]); }

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

}  // namespace kvq

}  // namespace sqk
