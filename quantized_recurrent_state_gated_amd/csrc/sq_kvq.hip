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
// The code is the one nearest to the exact quotient x / s, the even one of
// two.  x (1 / s) in fp32 finds it but for quotients next to a border; there
// r = x - v s, in one rounding, is exact (a multiple of s's last place, at most
// about half a step: it fits 24 bits), and comparing it with half a step decides.

// value (a code before its scale) nearest to x / s
template <bool E4M3>
__device__ __forceinline__ float nearest(float x, float s, float inv)
{
    if constexpr (!E4M3) {
        float n = __builtin_rintf(__builtin_amdgcn_fmed3f(x * inv, -127.0f, 127.0f));
        const float r = __builtin_fmaf(-n, s, x), a = __builtin_fabsf(r), h = 0.5f * s;
        if (a > h || (a == h && ((int)n & 1))) n += __builtin_copysignf(1.0f, r);
        return __builtin_amdgcn_fmed3f(n, -127.0f, 127.0f);
    } else {
        const float y = __builtin_amdgcn_fmed3f(x * inv, -448.0f, 448.0f);
        uint32_t e = (f_bits(y) >> 23) & 0xff;  // neighbours are 2^(e - 3) apart, 2^-9 below 2^-6
        e = e < 121 ? 121 : e;
        const float step = bits_f((e - 3) << 23);
        float n = __builtin_rintf(y * bits_f((257 - e) << 23)), v = n * step;
        const float r = __builtin_fmaf(-v, s, x), a = __builtin_fabsf(r), h = 0.5f * step * s;
        if (a > h || (a == h && ((int)n & 1))) v += __builtin_copysignf(step, r);
        return __builtin_amdgcn_fmed3f(v, -448.0f, 448.0f);
    }
}

// four such values as bytes, lowest first
template <bool E4M3>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    if constexpr (!E4M3) {
        return (uint32_t)(int)(a + 128.0f) | (uint32_t)(int)(b + 128.0f) << 8 | (uint32_t)(int)(c + 128.0f) << 16 |
               (uint32_t)(int)(d + 128.0f) << 24;
    } else {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
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

// four codes read back and written anew
template <bool E4M3>
__device__ __forceinline__ uint32_t again4(uint32_t w, float old, float s, float inv)
{
    float x[4];
    unpack4<E4M3>(w, x);
#pragma unroll
    for (int i = 0; i < 4; i++) x[i] = nearest<E4M3>(x[i] * old, s, inv);
    return pack4<E4M3>(x[0], x[1], x[2], x[3]);
}

// ---------------------------------------------------------------- rows in memory

__device__ __forceinline__ float bf(uint32_t x) { return bits_f(x << 16); }

__device__ __forceinline__ void load8(const uint16_t *p, float (&x)[8])
{
    const u32x4_t w = *reinterpret_cast<const u32x4_t *>(p);
#pragma unroll
    for (int i = 0; i < 4; i++) x[2 * i] = bf(w[i] & 0xffff), x[2 * i + 1] = bf(w[i] >> 16);
}
__device__ __forceinline__ void load8(const float *p, float (&x)[8])
{
    const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; i++) x[i] = a[i], x[4 + i] = b[i];
}
__device__ __forceinline__ f32x2 load2(const uint16_t *p)
{
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    return f32x2{bf(w & 0xffff), bf(w >> 16)};
}
__device__ __forceinline__ f32x2 load2(const float *p) { return *reinterpret_cast<const f32x2 *>(p); }

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
    int64_t block;   // (page, head, block) as an index into the scales, -1: the page does not exist
    int lo, hi;      // places of the tokens, lo < hi; hi == 0: nothing to do
};

__device__ __forceinline__ Place place_of(const KvqRowsArgs &a, int64_t slot, int h)
{
    const int r = wave_count(a.n_req, [&](int i) { return (clamp_to(a.cu[i], a.n) >> 4) + 2 * (int64_t)i <= slot; }) - 1;
    Place p{0, -1, 0, 0};
    if (r < 0) return p;
    const int32_t t0 = clamp_to(a.cu[r], a.n), t1 = clamp_to(a.cu[r + 1], a.n);
    const int32_t start = a.start ? a.start[r] : 0;
    if (start < 0 || t1 <= t0) return p;
    const int64_t end = (int64_t)start + (t1 - t0);
    const int64_t b = (start >> 4) + slot - ((t0 >> 4) + 2 * (int64_t)r);  // block of the request
    const int64_t pos = b << 4;
    if (pos >= end) return p;
    p.tok = t0 + pos - start;
    p.lo = pos < start ? (int)(start - pos) : 0;
    p.hi = end - pos < 16 ? (int)(end - pos) : 16;
    const int64_t pg = pos >> a.c.page_shift;
    if (pg >= a.table_stride) return p;
    const int32_t id = a.table[(int64_t)r * a.table_stride + pg];
    if ((uint32_t)id >= (uint32_t)a.c.n_pages) return p;
    const int per = a.c.page_shift - 4;
    p.block = ((((int64_t)id * a.c.heads + h) << per)) + (b & ((1 << per) - 1));
    return p;
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
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) most = fmaxf(most, __shfl_xor(most, d));
    const float s = fmaxf(most / top, kLeastScale);
    return held && !(s > old) ? old : s;
}

// not finite: NaN counts as 0, infinities saturate and do not enter the scale
__device__ __forceinline__ float clean(float x, float &most)
{
    const float a = __builtin_fabsf(x);
    most = a <= kFloatMax ? fmaxf(most, a) : most;
    return x == x ? x : 0.0f;
}

// ---------------------------------------------------------------- write
//
// Bound by HBM for prompts: x bytes are read and half (bfloat16) or a quarter
// (fp32) as many written.

template <typename T, int D, bool E4M3>
__device__ __forceinline__ void append_keys(const KvqRowsArgs &a, const Place &p, int h)
{
    constexpr int NU = D / 32, ROW = D / 8;  // 8-value units per lane, per token
    const int lane = threadIdx.x & 63;
    const T *src = reinterpret_cast<const T *>(a.k) + (int64_t)h * D;
    uint8_t *dst = a.c.k + p.block * (16 * D);
    float *scale = a.c.scales + 2 * p.block;
    float x[NU][8], most = 0.0f;
#pragma unroll
    for (int j = 0; j < NU; j++) {
        const int u = lane + 64 * j, t = u / ROW, c = u % ROW * 8;
        if (t >= p.lo && t < p.hi) load8(src + (p.tok + t) * a.k_stride + c, x[j]);
    }
    u32x2_t was[NU];
    float old = 0.0f;
    if (p.lo > 0) {
        old = *scale;
#pragma unroll
        for (int j = 0; j < NU; j++)
            if ((lane + 64 * j) / ROW < p.lo) was[j] = *reinterpret_cast<const u32x2_t *>(dst + (lane + 64 * j) * 8);
    }
#pragma unroll
    for (int j = 0; j < NU; j++) {
        const int t = (lane + 64 * j) / ROW;
        if (t >= p.lo && t < p.hi) {
#pragma unroll
            for (int i = 0; i < 8; i++) x[j][i] = clean(x[j][i], most);
        }
    }
    const float s = scale_of(most, E4M3 ? 448.0f : 127.0f, p.lo > 0, old), inv = 1.0f / s;
    const bool raised = p.lo > 0 && s != old;
#pragma unroll
    for (int j = 0; j < NU; j++) {
        const int u = lane + 64 * j, t = u / ROW;
        u32x2_t *to = reinterpret_cast<u32x2_t *>(dst + u * 8);
        if (t >= p.lo && t < p.hi) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = nearest<E4M3>(x[j][i], s, inv);
            *to = u32x2_t{pack4<E4M3>(v[0], v[1], v[2], v[3]), pack4<E4M3>(v[4], v[5], v[6], v[7])};
        } else if (raised && t < p.lo) {
            *to = u32x2_t{again4<E4M3>(was[j][0], old, s, inv), again4<E4M3>(was[j][1], old, s, inv)};
        }
    }
    if (lane == 0) *scale = s;
}

template <typename T, int D, bool E4M3>
__device__ __forceinline__ void append_values(const KvqRowsArgs &a, const Place &p, int h)
{
    constexpr int NP = (D + 127) / 128;  // column pairs per lane
    const int lane = threadIdx.x & 63;
    const T *src = reinterpret_cast<const T *>(a.v) + (int64_t)h * D;
    uint8_t *dst = a.c.v + p.block * (16 * D);
    float *scale = a.c.scales + 2 * p.block + 1;
    f32x2 x[NP][16];
    u32x4_t was[NP][2];
    float most = 0.0f, old = 0.0f;
#pragma unroll
    for (int j = 0; j < NP; j++) {
        const int c = 2 * (lane + 64 * j);
        if (D % 128 != 0 && c >= D) continue;
#pragma unroll
        for (int t = 0; t < 16; t++) {
            x[j][t] = f32x2{0.0f, 0.0f};
            if (t >= p.lo && t < p.hi) x[j][t] = load2(src + (p.tok + t) * a.v_stride + c);
        }
    }
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
    for (int j = 0; j < NP; j++) {
        if (D % 128 != 0 && 2 * (lane + 64 * j) >= D) continue;
#pragma unroll
        for (int t = 0; t < 16; t++) {
            x[j][t][0] = clean(x[j][t][0], most);
            x[j][t][1] = clean(x[j][t][1], most);
        }
    }
    const float s = scale_of(most, E4M3 ? 448.0f : 127.0f, p.lo > 0, old), inv = 1.0f / s;
    const bool raised = p.lo > 0 && s != old;
#pragma unroll
    for (int j = 0; j < NP; j++) {
        const int c = 2 * (lane + 64 * j);
        if (D % 128 != 0 && c >= D) continue;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            u32x4_t w;
#pragma unroll
            for (int g = 0; g < 4; g++) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; e++) v[e] = nearest<E4M3>(x[j][4 * g + e][i], s, inv);
                w[g] = pack4<E4M3>(v[0], v[1], v[2], v[3]);
                if (p.lo > 0) {  // places of the new tokens in this word take its bytes, the others stay
                    const uint32_t before = raised ? again4<E4M3>(was[j][i][g], old, s, inv) : was[j][i][g];
                    const int lo = p.lo - 4 * g, hi = p.hi - 4 * g;
                    const uint32_t below_hi = hi <= 0 ? 0u : hi >= 4 ? ~0u : (1u << 8 * hi) - 1;
                    const uint32_t below_lo = lo <= 0 ? 0u : lo >= 4 ? ~0u : (1u << 8 * lo) - 1;
                    const uint32_t fresh = below_hi & ~below_lo;
                    w[g] = (w[g] & fresh) | (before & ~fresh);
                }
            }
            *reinterpret_cast<u32x4_t *>(dst + (c + i) * 16) = w;
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
    const Place p = place_of(a, (w >> 1) / heads, h);
    if (p.hi == 0 || p.block < 0) return;
    if (w & 1) append_values<T, D, E4M3>(a, p, h);
    else append_keys<T, D, E4M3>(a, p, h);
}

// ---------------------------------------------------------------- read back

template <typename T, int D, bool E4M3>
__device__ __forceinline__ void load_keys(const KvqRowsArgs &a, const Place &p, int h)
{
    constexpr int NU = D / 32, ROW = D / 8;
    const int lane = threadIdx.x & 63;
    T *dst = reinterpret_cast<T *>(a.k) + (int64_t)h * D;
    const uint8_t *src = a.c.k + p.block * (16 * D);
    const bool there = p.block >= 0;
    const float s = there ? a.c.scales[2 * p.block] : 0.0f;
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
    const uint8_t *src = a.c.v + p.block * (16 * D);
    const bool there = p.block >= 0;
    const float s = there ? a.c.scales[2 * p.block + 1] : 0.0f;
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
    const Place p = place_of(a, (w >> 1) / heads, h);
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
