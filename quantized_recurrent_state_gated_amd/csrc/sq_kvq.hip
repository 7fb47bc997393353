// sq_kvq.hip -- gfx950 kernels that write the 8-bit paged key-value cache and
// read it back.
//
// A block is 16 positions of one page and head.  Its keys share one scale, its
// values another: the largest magnitude over 127 (integer codes) or 448 (e4m3
// codes), so that
//     code = round(x / s),  x ~ code s,  |x - code s| <= s / 2 (integer codes).
// Tokens arrive in pieces.  The first ones of a block set its scale (what a
// page held before does not count); later ones raise it if they have to, and
// then the codes before them are read back and written anew.
//
// A wave takes the keys or the values of one block and head: 16 tokens x d are
// 4 KB in and 2 KB out for d = 128 in bfloat16, so the maximum is one
// reduction over the wave, nothing passes through shared memory and no two
// waves write one block.  Keys: a lane takes 8 consecutive values of a token.
// Values are kept transposed, [d][16]: a lane takes two columns of all 16
// tokens, and writes 32 consecutive bytes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sq_grid.h"
#include "sq_kvq.h"
#include "sq_kvq_dev.h"

namespace sqk {

namespace {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kFloatMax = 3.402823466e+38f;
constexpr float kLeastScale = 7.888609052210118e-31f;  // 2^-100: quotients by a scale stay normal numbers

// ---------------------------------------------------------------- codes
//
// The code is the one nearest to the exact quotient x / s, the even one of two.
// x (1 / s) in fp32 is off by 127 x 2^-24 at most, so it finds that code or, next to a
// border, its neighbour.  There r = x - v s, in one rounding, is exact (a multiple of
// s's last place, at most about half a step: it fits 24 bits), and comparing
// it with half a step decides: a tie goes on where the code found is odd, which is a
// comparison with the float below.  All of it without a branch: borders are no
// rarity, bfloat16 values over a bfloat16 maximum meet one in most blocks
// (4 x 8,191 tokens x 8 heads, d = 128: 42 us; quotients alone, made again by a form
// with branches where one was near, took 65, that form for all 71).

constexpr float kRound = 12582912.0f;  // 1.5 x 2^23: what is added to it is rounded to an integer, its last bit the parity

// four codes of finite x, lowest byte first
template <bool E4M3>
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float s, float inv)
{
    if constexpr (!E4M3) {
        const uint32_t half = f_bits(0.5f * s);
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float f = __builtin_fmaf(x[i], inv, kRound + 128.0f);
            const float r = __builtin_fmaf(kRound + 128.0f - f, s, x[i]);
            y[i] = f_bits(f);
            const float h = bits_f(half - (y[i] & 1));
            y[i] += r > h;
            y[i] -= r < -h;
        }
        return __builtin_amdgcn_perm(y[1], y[0], 0x0c0c0400u) | __builtin_amdgcn_perm(y[3], y[2], 0x04000c0cu);
    } else {
        float v[4];
        const float half = 0.5f * s;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float q = x[i] * inv;
            uint32_t e = f_bits(q) & 0x7f800000u;  // neighbours are 2^-3 of this apart, 2^-9 below 2^-6
            e = e < 121u << 23 ? 121u << 23 : e;
            const float step = bits_f(e - (3u << 23));
            const float f = __builtin_fmaf(q, bits_f((257u << 23) - e), kRound);
            v[i] = (f - kRound) * step;
            const float r = __builtin_fmaf(-v[i], s, x[i]);
            const float h = bits_f(f_bits(half * step) - (f_bits(f) & 1));
            v[i] = __builtin_copysignf(v[i] + (r > h ? step : r < -h ? -step : 0.0f), x[i]);
        }
        const int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
    }
}

template <bool E4M3>
__device__ __forceinline__ void unpack4(uint32_t w, float (&x)[4])
{
    if constexpr (!E4M3) {
#pragma unroll
        for (int i = 0; i < 4; i++) x[i] = (float)((w >> 8 * i) & 0xff) - 128.0f;
    } else {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
        x[0] = lo[0], x[1] = lo[1], x[2] = hi[0], x[3] = hi[1];
    }
}

// values that are not finite do not enter the scale; NaN counts as 0, infinities as the
// largest value that the block can hold
__device__ __forceinline__ float finite(float x)
{
    const float a = __builtin_fabsf(x);
    return a <= kFloatMax ? a : 0.0f;
}
template <bool E4M3>
__device__ __forceinline__ float largest(float s) { return fminf((E4M3 ? 448.0f : 127.0f) * s, kFloatMax); }
__device__ __forceinline__ float tame(float x, float most)
{
    return x == x ? __builtin_amdgcn_fmed3f(x, -most, most) : 0.0f;
}

// four codes read back and written anew
template <bool E4M3>
__device__ __forceinline__ uint32_t again4(uint32_t w, float old, float s, float inv)
{
    float x[4];
    unpack4<E4M3>(w, x);
#pragma unroll
    for (int i = 0; i < 4; i++) x[i] = tame(x[i] * old, largest<E4M3>(s));  // whatever byte was there
    return codes4<E4M3>(x, s, inv);
}

// ---------------------------------------------------------------- rows in memory

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Eight values of a row and two columns of one, as they lie in memory, and the
// largest magnitude as bits: of NaN and infinities above all numbers'.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
    using Eight = u32x4_t;
    using Two = uint32_t;
    static __device__ __forceinline__ float at(const Eight &w, int i) { return bits_f(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16); }
    static __device__ __forceinline__ float at(Two w, int i) { return bits_f(i ? w & 0xffff0000u : w << 16); }
    static __device__ __forceinline__ uint32_t top(uint32_t acc, Two w)  // both halves apart
    {
        const u16x2 a = __builtin_bit_cast(u16x2, acc), b = __builtin_bit_cast(u16x2, w & 0x7fff7fffu);
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
    }
    static __device__ __forceinline__ uint32_t top(uint32_t acc, const Eight &w)
    {
        return top(top(top(top(acc, w[0]), w[1]), w[2]), w[3]);
    }
    static __device__ __forceinline__ uint32_t bits(uint32_t acc)
    {
        const uint32_t hi = acc & 0xffff0000u, lo = acc << 16;
        return hi > lo ? hi : lo;
    }
};
template <>
struct Raw<float> {
    typedef float Eight __attribute__((ext_vector_type(8)));
    using Two = f32x2;
    template <typename W>
    static __device__ __forceinline__ float at(const W &w, int i) { return w[i]; }
    template <typename W>
    static __device__ __forceinline__ uint32_t top(uint32_t acc, const W &w)
    {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(W) / 4); i++) {
            const uint32_t b = f_bits(w[i]) & 0x7fffffffu;
            acc = b > acc ? b : acc;
        }
        return acc;
    }
    static __device__ __forceinline__ uint32_t bits(uint32_t acc) { return acc; }
};

__device__ __forceinline__ uint32_t pair(float a, float b)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ void store8(uint16_t *p, const float (&x)[8])
{
    *reinterpret_cast<u32x4_t *>(p) = u32x4_t{pair(x[0], x[1]), pair(x[2], x[3]), pair(x[4], x[5]), pair(x[6], x[7])};
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8])
{
    *reinterpret_cast<f32x4 *>(p) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4 *>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
}
__device__ __forceinline__ void store2(uint16_t *p, float a, float b) { *reinterpret_cast<uint32_t *>(p) = pair(a, b); }
__device__ __forceinline__ void store2(float *p, float a, float b) { *reinterpret_cast<f32x2 *>(p) = f32x2{a, b}; }

// ---------------------------------------------------------------- which block
//
// Request r's tokens lie at start_r + 0 .. m_r - 1 and touch at most
// floor(m_r / 16) + 2 blocks.  Block slots are numbered so that the host can
// count them without the lengths: those of request r begin at
//     floor(cu_r / 16) + 2 r,
// which leaves floor(m_r / 16) + 2 of them at least.

struct Place {
    int64_t tok;     // packed token at the block's first position (it may be another request's, or none)
    int64_t at;      // the block within its request
    int r;           // the request
    int lo, hi;      // places of the tokens, lo < hi; hi == 0: nothing to do
};

// The request of a slot, its tokens and their first position.  Up to 256 requests a
// wave reads all offsets and positions at once and picks (one round of loads:
// single tokens are bound by the chain of loads), more are searched.
__device__ __forceinline__ int request_of(const KvqRowsArgs &a, int64_t slot, int32_t &t0, int32_t &t1, int32_t &start)
{
    constexpr int PER = 4;
    const int lane = threadIdx.x & 63;
    if (a.n_req <= 64 * PER) {
        int32_t lo[PER], hi[PER], st[PER];
#pragma unroll
        for (int k = 0; k < PER; k++) {
            const int i = lane + 64 * k;
            lo[k] = hi[k] = st[k] = 0;
            if (i < a.n_req) {
                lo[k] = a.cu[i];
                hi[k] = a.cu[i + 1];
                if (a.start) st[k] = a.start[i];
            }
        }
        int r = -1;
#pragma unroll
        for (int k = 0; k < PER; k++) {
            const int i = lane + 64 * k;
            r += __popcll(__ballot(i < a.n_req && (clamp_to(lo[k], a.n) >> 4) + 2 * (int64_t)i <= slot));
        }
        t0 = t1 = start = 0;
#pragma unroll
        for (int k = 0; k < PER; k++)
            if (r >> 6 == k) {  // r is the wave's
                t0 = __builtin_amdgcn_readlane(lo[k], r & 63);
                t1 = __builtin_amdgcn_readlane(hi[k], r & 63);
                start = __builtin_amdgcn_readlane(st[k], r & 63);
            }
        t0 = clamp_to(t0, a.n);
        t1 = clamp_to(t1, a.n);
        return r;
    }
    const int r = wave_count(a.n_req, [&](int i) { return (clamp_to(a.cu[i], a.n) >> 4) + 2 * (int64_t)i <= slot; }) - 1;
    if (r < 0) return r;
    t0 = clamp_to(a.cu[r], a.n);
    t1 = clamp_to(a.cu[r + 1], a.n);
    start = a.start ? a.start[r] : 0;
    return r;
}

__device__ __forceinline__ Place place_of(const KvqRowsArgs &a, int64_t slot)
{
    int32_t t0, t1, start;
    const int r = request_of(a, slot, t0, t1, start);
    Place p{0, 0, r, 0, 0};
    if (r < 0) return p;
    const int64_t nth = slot - ((t0 >> 4) + 2 * (int64_t)r);  // of the request's slots; negative where offsets fall
    if (start < 0 || t1 <= t0 || nth < 0) return p;
    const int64_t end = (int64_t)start + (t1 - t0);
    const int64_t b = (start >> 4) + nth;  // block of the request
    const int64_t pos = b << 4;
    if (pos >= end) return p;
    p.tok = t0 + pos - start;
    p.lo = pos < start ? (int)(start - pos) : 0;
    p.hi = end - pos < 16 ? (int)(end - pos) : 16;
    p.at = b;
    return p;
}

// (page, head, block) as an index into the scales, -1: the page does not exist
__device__ __forceinline__ int64_t block_of(const KvqRowsArgs &a, const Place &p, int h)
{
    const int per = a.c.page_shift - 4;
    const int64_t pg = p.at >> per;
    if (pg >= a.table_stride) return -1;
    const int32_t id = a.table[(int64_t)p.r * a.table_stride + pg];
    if ((uint32_t)id >= (uint32_t)a.c.n_pages) return -1;
    return (((int64_t)id * a.c.heads + h) << per) + (p.at & ((1 << per) - 1));
}

// wave-uniform numbering: keys and values of a head next to each other, heads, slots
// (a launch has fewer than 2^26 waves)
__device__ __forceinline__ uint32_t wave_id()
{
    return blockIdx.x * 4 + (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
}

// the scale of a block: of its new values alone, or raised by them
__device__ __forceinline__ float scale_of(float most, float top, bool held, float old)
{
    const float s = fmaxf(most / top, kLeastScale);
    return held && !(s > old) ? old : s;
}

__device__ __forceinline__ uint32_t wave_top(uint32_t x)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t y = __shfl_xor((int)x, d);
        x = y > x ? y : x;
    }
    return x;
}

// ---------------------------------------------------------------- write
//
// Bound by HBM for prompts: 4 x 8,191 tokens x 8 heads, d = 128 in bfloat16, 42 us (201 MB,
// 4.8 TB/s).  Single tokens are bound by the chain of loads: offsets, then the page id
// and the new values together, then the scale and the codes that are there (70 requests
// x 8 heads 5.8 us).

template <typename T, int D, bool E4M3>
__device__ __forceinline__ void append_keys(const KvqRowsArgs &a, const Place &p, int h)
{
    using R = Raw<T>;
    constexpr int NU = D / 32, ROW = D / 8;  // 8-value units per lane, per token
    constexpr float TOP = E4M3 ? 448.0f : 127.0f;
    const int lane = threadIdx.x & 63;
    const T *src = reinterpret_cast<const T *>(a.k) + (int64_t)h * D;
    typename R::Eight x[NU];
    uint32_t acc = 0;
#pragma unroll
    for (int j = 0; j < NU; j++) {
        const int u = lane + 64 * j, t = u / ROW, c = u % ROW * 8;
        x[j] = typename R::Eight{};
        if (t >= p.lo && t < p.hi) x[j] = *reinterpret_cast<const typename R::Eight *>(src + (p.tok + t) * a.k_stride + c);
    }
    const int64_t block = block_of(a, p, h);
    if (block < 0) return;
    uint8_t *dst = a.c.k + block * (16 * D);
    float *scale = a.c.scales + 2 * block;
    u32x2_t was[NU];
    float old = 0.0f;
    if (p.lo > 0) {
        old = *scale;
#pragma unroll
        for (int j = 0; j < NU; j++)
            if ((lane + 64 * j) / ROW < p.lo) was[j] = *reinterpret_cast<const u32x2_t *>(dst + (lane + 64 * j) * 8);
    }
#pragma unroll
    for (int j = 0; j < NU; j++) acc = R::top(acc, x[j]);
    uint32_t most = wave_top(R::bits(acc));
    const bool odd = most >= 0x7f800000u;
    if (odd) {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < NU; j++)
#pragma unroll
            for (int i = 0; i < 8; i++) m = fmaxf(m, finite(R::at(x[j], i)));
        most = wave_top(f_bits(m));
    }
    const float s = scale_of(bits_f(most), TOP, p.lo > 0, old), inv = 1.0f / s;
    const bool raised = p.lo > 0 && s != old;
    u32x2_t w[NU];
    auto encode = [&](auto value) {
#pragma unroll
        for (int j = 0; j < NU; j++)
#pragma unroll
            for (int g = 0; g < 2; g++) {
                const float y[4] = {value(R::at(x[j], 4 * g)), value(R::at(x[j], 4 * g + 1)), value(R::at(x[j], 4 * g + 2)),
                                    value(R::at(x[j], 4 * g + 3))};
                w[j][g] = codes4<E4M3>(y, s, inv);
            }
    };
    if (odd) encode([&](float v) { return tame(v, largest<E4M3>(s)); });
    else encode([](float v) { return v; });
#pragma unroll
    for (int j = 0; j < NU; j++) {
        const int u = lane + 64 * j, t = u / ROW;
        u32x2_t *to = reinterpret_cast<u32x2_t *>(dst + u * 8);
        if (t >= p.lo && t < p.hi) *to = w[j];
        else if (raised && t < p.lo) *to = u32x2_t{again4<E4M3>(was[j][0], old, s, inv), again4<E4M3>(was[j][1], old, s, inv)};
    }
    if (lane == 0) *scale = s;
}

template <typename T, int D, bool E4M3>
__device__ __forceinline__ void append_values(const KvqRowsArgs &a, const Place &p, int h)
{
    using R = Raw<T>;
    constexpr int NP = (D + 127) / 128;  // column pairs per lane
    constexpr float TOP = E4M3 ? 448.0f : 127.0f;
    const int lane = threadIdx.x & 63;
    const T *src = reinterpret_cast<const T *>(a.v) + (int64_t)h * D;
    typename R::Two x[NP][16];
    uint32_t acc = 0;
#pragma unroll
    for (int j = 0; j < NP; j++) {
        const int c = 2 * (lane + 64 * j);
#pragma unroll
        for (int t = 0; t < 16; t++) {
            x[j][t] = typename R::Two{};
            if ((D % 128 == 0 || c < D) && t >= p.lo && t < p.hi)
                x[j][t] = *reinterpret_cast<const typename R::Two *>(src + (p.tok + t) * a.v_stride + c);
        }
    }
    const int64_t block = block_of(a, p, h);
    if (block < 0) return;
    uint8_t *dst = a.c.v + block * (16 * D);
    float *scale = a.c.scales + 2 * block + 1;
    u32x4_t was[NP][2];
    float old = 0.0f;
    if (p.lo > 0) {
        old = *scale;
#pragma unroll
        for (int j = 0; j < NP; j++) {
            const int c = 2 * (lane + 64 * j);
            if (D % 128 != 0 && c >= D) continue;
#pragma unroll
            for (int i = 0; i < 2; i++) was[j][i] = *reinterpret_cast<const u32x4_t *>(dst + (c + i) * 16);
        }
    }
#pragma unroll
    for (int j = 0; j < NP; j++)
#pragma unroll
        for (int t = 0; t < 16; t++) acc = R::top(acc, x[j][t]);
    uint32_t most = wave_top(R::bits(acc));
    const bool odd = most >= 0x7f800000u;
    if (odd) {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < NP; j++)
#pragma unroll
            for (int t = 0; t < 16; t++) m = fmaxf(m, fmaxf(finite(R::at(x[j][t], 0)), finite(R::at(x[j][t], 1))));
        most = wave_top(f_bits(m));
    }
    const float s = scale_of(bits_f(most), TOP, p.lo > 0, old), inv = 1.0f / s;
    const bool raised = p.lo > 0 && s != old;
    u32x4_t w[NP][2];
    auto encode = [&](auto value) {
#pragma unroll
        for (int j = 0; j < NP; j++)
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    w[j][i][g] = 0;
                    if (4 * g >= p.hi || 4 * g + 4 <= p.lo) continue;  // no new token in this word
                    const float y[4] = {value(R::at(x[j][4 * g], i)), value(R::at(x[j][4 * g + 1], i)),
                                        value(R::at(x[j][4 * g + 2], i)), value(R::at(x[j][4 * g + 3], i))};
                    w[j][i][g] = codes4<E4M3>(y, s, inv);
                }
    };
    if (odd) encode([&](float v) { return tame(v, largest<E4M3>(s)); });
    else encode([](float v) { return v; });
#pragma unroll
    for (int j = 0; j < NP; j++) {
        const int c = 2 * (lane + 64 * j);
        if (D % 128 != 0 && c >= D) continue;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (p.lo > 0) {
#pragma unroll
                for (int g = 0; g < 4; g++) {  // places of the new tokens in this word take its bytes, the others stay
                    const uint32_t before = raised ? again4<E4M3>(was[j][i][g], old, s, inv) : was[j][i][g];
                    const int lo = p.lo - 4 * g, hi = p.hi - 4 * g;
                    const uint32_t below_hi = hi <= 0 ? 0u : hi >= 4 ? ~0u : (1u << 8 * hi) - 1;
                    const uint32_t below_lo = lo <= 0 ? 0u : lo >= 4 ? ~0u : (1u << 8 * lo) - 1;
                    const uint32_t fresh = below_hi & ~below_lo;
                    w[j][i][g] = (w[j][i][g] & fresh) | (before & ~fresh);
                }
            }
            *reinterpret_cast<u32x4_t *>(dst + (c + i) * 16) = w[j][i];
        }
    }
    if (lane == 0) *scale = s;
}

template <typename T, int D, bool E4M3>
__global__ __launch_bounds__(256) void k_kvq_append(KvqRowsArgs a, uint32_t waves)
{
    const uint32_t w = wave_id();
    if (w >= waves) return;
    const uint32_t heads = (uint32_t)a.c.heads;
    const int h = (int)((w >> 1) % heads);
    const Place p = place_of(a, (w >> 1) / heads);
    if (p.hi == 0) return;
    if (w & 1) append_values<T, D, E4M3>(a, p, h);
    else append_keys<T, D, E4M3>(a, p, h);
}

// ---------------------------------------------------------------- read back
//
// Bound by HBM: 8 requests to 8,192 tokens x 8 heads, d = 128 into bfloat16 (231 MB): 55 us for a call on
// a cache that it finds in HBM, 4.2 TB/s; 37 us of kernel where part of it lies in the last-level cache.

template <typename T, int D, bool E4M3>
__device__ __forceinline__ void load_keys(const KvqRowsArgs &a, const Place &p, int h)
{
    constexpr int NU = D / 32, ROW = D / 8;
    const int lane = threadIdx.x & 63;
    T *dst = reinterpret_cast<T *>(a.k) + (int64_t)h * D;
    const int64_t block = block_of(a, p, h);
    const uint8_t *src = a.c.k + block * (16 * D);
    const bool there = block >= 0;
    const float s = there ? a.c.scales[2 * block] : 0.0f;
    u32x2_t w[NU];
#pragma unroll
    for (int j = 0; j < NU; j++) {
        const int u = lane + 64 * j, t = u / ROW;
        if (there && t >= p.lo && t < p.hi) w[j] = *reinterpret_cast<const u32x2_t *>(src + u * 8);
    }
#pragma unroll
    for (int j = 0; j < NU; j++) {
        const int u = lane + 64 * j, t = u / ROW, c = u % ROW * 8;
        if (t < p.lo || t >= p.hi) continue;
        float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (there) {
            float lo[4], hi[4];
            unpack4<E4M3>(w[j][0], lo);
            unpack4<E4M3>(w[j][1], hi);
#pragma unroll
            for (int i = 0; i < 4; i++) x[i] = lo[i] * s, x[4 + i] = hi[i] * s;
        }
        store8(dst + (p.tok + t) * a.k_stride + c, x);
    }
}

template <typename T, int D, bool E4M3>
__device__ __forceinline__ void load_values(const KvqRowsArgs &a, const Place &p, int h)
{
    constexpr int NP = (D + 127) / 128;
    const int lane = threadIdx.x & 63;
    T *dst = reinterpret_cast<T *>(a.v) + (int64_t)h * D;
    const int64_t block = block_of(a, p, h);
    const uint8_t *src = a.c.v + block * (16 * D);
    const bool there = block >= 0;
    const float s = there ? a.c.scales[2 * block + 1] : 0.0f;
    u32x4_t w[NP][2];
#pragma unroll
    for (int j = 0; j < NP; j++) {
        const int c = 2 * (lane + 64 * j);
        if (D % 128 != 0 && c >= D) continue;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            w[j][i] = u32x4_t{0, 0, 0, 0};
            if (there) w[j][i] = *reinterpret_cast<const u32x4_t *>(src + (c + i) * 16);
        }
    }
#pragma unroll
    for (int j = 0; j < NP; j++) {
        const int c = 2 * (lane + 64 * j);
        if (D % 128 != 0 && c >= D) continue;
#pragma unroll
        for (int g = 0; g < 4; g++) {
            float x[2][4];
            unpack4<E4M3>(w[j][0][g], x[0]);
            unpack4<E4M3>(w[j][1][g], x[1]);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int t = 4 * g + e;
                if (t < p.lo || t >= p.hi) continue;
                store2(dst + (p.tok + t) * a.v_stride + c, there ? x[0][e] * s : 0.0f, there ? x[1][e] * s : 0.0f);
            }
        }
    }
}

template <typename T, int D, bool E4M3>
__global__ __launch_bounds__(256) void k_kvq_load(KvqRowsArgs a, uint32_t waves)
{
    const uint32_t w = wave_id();
    if (w >= waves) return;
    if ((w & 1) ? !a.v : !a.k) return;
    const uint32_t heads = (uint32_t)a.c.heads;
    const int h = (int)((w >> 1) % heads);
    const Place p = place_of(a, (w >> 1) / heads);
    if (p.hi == 0) return;
    if (w & 1) load_values<T, D, E4M3>(a, p, h);
    else load_keys<T, D, E4M3>(a, p, h);
}

enum Rows { APPEND, LOAD };

template <Rows R, typename T, int D>
hipError_t rows_td(const KvqRowsArgs &a, hipStream_t st)
{
    const int64_t waves = (((int64_t)a.n >> 4) + 2 * (int64_t)a.n_req) * a.c.heads * 2;
    const int64_t grid = (waves + 3) / 4;
    if (!grid_fits(grid, 256)) return hipErrorInvalidConfiguration;
    const dim3 g((unsigned)grid), b(256);
    if constexpr (R == APPEND) {
        if (a.c.e4m3) hipLaunchKernelGGL((k_kvq_append<T, D, true>), g, b, 0, st, a, (uint32_t)waves);
        else hipLaunchKernelGGL((k_kvq_append<T, D, false>), g, b, 0, st, a, (uint32_t)waves);
    } else {
        if (a.c.e4m3) hipLaunchKernelGGL((k_kvq_load<T, D, true>), g, b, 0, st, a, (uint32_t)waves);
        else hipLaunchKernelGGL((k_kvq_load<T, D, false>), g, b, 0, st, a, (uint32_t)waves);
    }
    return hipGetLastError();
}

template <Rows R, typename T>
hipError_t rows_t(const KvqRowsArgs &a, hipStream_t st)
{
    switch (a.c.d) {
    case 32: return rows_td<R, T, 32>(a, st);
    case 64: return rows_td<R, T, 64>(a, st);
    case 96: return rows_td<R, T, 96>(a, st);
    case 128: return rows_td<R, T, 128>(a, st);
    case 192: return rows_td<R, T, 192>(a, st);
    case 256: return rows_td<R, T, 256>(a, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_kvq_append(const KvqRowsArgs &a, bool bf16, hipStream_t st)
{
    return bf16 ? rows_t<APPEND, uint16_t>(a, st) : rows_t<APPEND, float>(a, st);
}

hipError_t launch_kvq_load(const KvqRowsArgs &a, bool bf16, hipStream_t st)
{
    return bf16 ? rows_t<LOAD, uint16_t>(a, st) : rows_t<LOAD, float>(a, st);
}

}  // namespace sqk
