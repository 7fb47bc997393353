// sq_prefill.hip -- gfx950 kernels of the prompt form of the recurrent
// layers: a whole sequence of tokens through
//     S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T   (delta)
//     S_t = alpha_t S_{t-1} + beta_t k_t v_t^T                          (plain decay)
//     o_t = S_t^T q_t
// from the state S_0 (or zero) to the state that the decode steps go on from.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "sq_grid.h"
#include "sq_prefill.h"

namespace sqk {

namespace {

template <typename T>
__device__ __forceinline__ float up(T x);
template <>
__device__ __forceinline__ float up<float>(float x) { return x; }
template <>
__device__ __forceinline__ float up<uint16_t>(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

template <typename T>
__device__ __forceinline__ T down(float x);
template <>
__device__ __forceinline__ float down<float>(float x) { return x; }
template <>
__device__ __forceinline__ uint16_t down<uint16_t>(float x)
{
    return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// Tokens [first, last) of sequence s, 0 <= first <= last <= n_tokens whatever cu says.
struct Seq {
    int32_t first, last;
};

__device__ __forceinline__ Seq seq_of(const PrefillArgs &a, int s)
{
    Seq r{a.cu[s], a.cu[s + 1]};
    if (r.first < 0) r.first = 0;
    if (r.first > a.n_tokens) r.first = a.n_tokens;
    if (r.last > a.n_tokens) r.last = a.n_tokens;
    if (r.last < r.first) r.last = r.first;
    return r;
}

// the shared-memory barrier alone: loads and stores in flight to global memory
// (the next chunk's inputs, this chunk's outputs) are not waited for
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------- token by token
//
// Any d_k, d_v (multiples of 4, at most 256) and both element types.  The
// columns of S are independent of each other: LPC lanes hold a column, RPL rows
// each, in registers.  Per token a lane does three fused multiply-adds a row for
//     u = k^T S, y = q^T S, and the update S = alpha S + k w,
//     w = beta (v - alpha u), o = alpha y + (q.k) w,
// and the column's lanes join their sums by DPP exchanges.  Tokens, with their
// q.k, are staged through shared memory TB at a time.  A token takes as long as
// its chain of instructions: 16 lanes a column where workgroups are few
// (36 heads x 77 tokens of fp32, d = 128: 30 us against 46 with 4; 48 heads x 400
// tokens 127 against 214), 4 where there are enough of them and the exchanges only
// cost (384 heads x 200 tokens 176 us against 250).

constexpr int kTB = 16;  // tokens staged at a time

template <int CTRL>
__device__ __forceinline__ float dpp_sum(float x)
{
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, false));
}

// sum over LPC neighbouring lanes, in all of them
template <int LPC>
__device__ __forceinline__ float lanes_sum(float x)
{
    x = dpp_sum<0xb1>(x);                        // quad_perm [1,0,3,2]
    x = dpp_sum<0x4e>(x);                        // quad_perm [2,3,0,1]
    if constexpr (LPC >= 8) x = dpp_sum<0x141>(x);   // row_half_mirror: sums of 8
    if constexpr (LPC >= 16) x = dpp_sum<0x140>(x);  // row_mirror: sums of 16
    return x;
}

template <typename T, bool DELTA, int LPC, int RPL>
__global__ __launch_bounds__(256) void k_prefill_tokens(PrefillArgs a)
{
    constexpr int ROWS = LPC * RPL, COLS = 256 / LPC;
    __shared__ __align__(16) float sq[kTB][ROWS], sk[kTB][ROWS];
    __shared__ float sv[kTB][COLS];
    __shared__ float4 sg[kTB];  // alpha, beta, q.k
    const int t = threadIdx.x, part = t % LPC, col = t / LPC;
    const int tiles = (a.dv + COLS - 1) / COLS;
    const int j0 = (int)(blockIdx.x % (unsigned)tiles) * COLS;
    const int sh = (int)(blockIdx.x / (unsigned)tiles);
    const int h = sh % a.heads, s = sh / a.heads;
    const Seq sr = seq_of(a, s);
    const int j = j0 + col;
    const bool in = j < a.dv;
    const int64_t tile = (int64_t)sh * a.dk * a.dv;

    // row 4 (LPC i + part) + e
    float S[RPL];
#pragma unroll
    for (int i = 0; i < RPL; i++) {
        const int row = 4 * (LPC * (i >> 2) + part) + (i & 3);
        S[i] = a.S0 && in && row < a.dk ? a.S0[tile + (int64_t)row * a.dv + j] : 0.0f;
    }
    const T *q = reinterpret_cast<const T *>(a.q) + (int64_t)(h / a.per_k) * a.dk;
    const T *k = reinterpret_cast<const T *>(a.k) + (int64_t)(h / a.per_k) * a.dk;
    const T *v = reinterpret_cast<const T *>(a.v) + (int64_t)h * a.dv;
    T *o = reinterpret_cast<T *>(a.o) + (int64_t)h * a.dv;

    // 16 lanes a token bring it, 16 tokens at once, a block ahead of its use
    constexpr int NQ = ROWS / 16, NV = COLS / 16;
    const int bx = t >> 4, bl = t & 15;
    float nq[NQ], nk[NQ], nv[NV], na = 0.0f, nb = 0.0f;
    auto bring = [&](int32_t t0) {
        const int64_t tok = t0 + bx;  // (the host keeps n_tokens 64 below the top of 32 bits)
        if (tok >= sr.last) return;
#pragma unroll
        for (int i = 0; i < NQ; i++) {
            const int d = 16 * i + bl;
            nq[i] = d < a.dk ? up<T>(q[tok * a.q_stride + d]) : 0.0f;
            nk[i] = d < a.dk ? up<T>(k[tok * a.k_stride + d]) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int d = 16 * i + bl;
            nv[i] = j0 + d < a.dv ? up<T>(v[tok * a.v_stride + j0 + d]) : 0.0f;
        }
        if (bl == 0) {
            na = a.alpha[tok * a.heads + h];
            nb = a.beta[tok * a.heads + h];
        }
    };
#pragma unroll
    for (int i = 0; i < NQ; i++) nq[i] = nk[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; i++) nv[i] = 0.0f;
    bring(sr.first);
    for (int32_t t0 = sr.first; t0 < sr.last; t0 += kTB) {
        // at least one; in a scalar register (a vector compare a token costs 36 heads x
        // 77 tokens 1.4 us of 30)
        const int nt = __builtin_amdgcn_readfirstlane(sr.last - t0 < kTB ? sr.last - t0 : kTB);
        {
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NQ; i++) {
                sq[bx][16 * i + bl] = nq[i];
                sk[bx][16 * i + bl] = nk[i];
                dot = fmaf(nq[i], nk[i], dot);
            }
#pragma unroll
            for (int i = 0; i < NV; i++) sv[bx][16 * i + bl] = nv[i];
            dot = lanes_sum<16>(dot);
            if (bl == 0) sg[bx] = make_float4(na, nb, dot, 0.0f);
        }
        if (t0 + kTB < sr.last) bring(t0 + kTB);
        lds_barrier();
        int x = 0;
        do {
            float u = 0.0f, y = 0.0f, kr[RPL];
#pragma unroll
            for (int i = 0; i < RPL; i += 4) {
                const float4 k4 = *reinterpret_cast<const float4 *>(&sk[x][LPC * i + 4 * part]);
                const float4 q4 = *reinterpret_cast<const float4 *>(&sq[x][LPC * i + 4 * part]);
                const float qe[4] = {q4.x, q4.y, q4.z, q4.w};
                kr[i] = k4.x; kr[i + 1] = k4.y; kr[i + 2] = k4.z; kr[i + 3] = k4.w;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    if (DELTA) u = fmaf(kr[i + e], S[i + e], u);
                    y = fmaf(qe[e], S[i + e], y);
                }
            }
            if (DELTA) u = lanes_sum<LPC>(u);
            y = lanes_sum<LPC>(y);
            const float4 gt = sg[x];
            const float vj = sv[x][col];
            const float w = gt.y * (DELTA ? vj - gt.x * u : vj);
#pragma unroll
            for (int i = 0; i < RPL; i++) S[i] = fmaf(gt.x, S[i], kr[i] * w);
            if (part == 0 && in) o[(int64_t)(t0 + x) * a.heads * a.dv + j] = down<T>(fmaf(gt.x, y, gt.z * w));
        } while (++x < nt);
        lds_barrier();
    }
    if (!a.S || !in) return;
#pragma unroll
    for (int i = 0; i < RPL; i++) {
        const int row = 4 * (LPC * (i >> 2) + part) + (i & 3);
        if (row < a.dk) a.S[tile + (int64_t)row * a.dv + j] = S[i];
    }
}

template <typename T, bool DELTA, int LPC>
hipError_t tokens_l(const PrefillArgs &a, hipStream_t st)
{
    constexpr int COLS = 256 / LPC;
    const int64_t groups = (int64_t)a.n_seq * a.heads * ((a.dv + COLS - 1) / COLS);
    if (!grid_fits(groups, 256)) return hipErrorInvalidConfiguration;
    const unsigned grid = (unsigned)groups;
    if (a.dk <= 64)
        hipLaunchKernelGGL((k_prefill_tokens<T, DELTA, LPC, 64 / LPC>), dim3(grid), dim3(256), 0, st, a);
    else if (a.dk <= 128)
        hipLaunchKernelGGL((k_prefill_tokens<T, DELTA, LPC, 128 / LPC>), dim3(grid), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((k_prefill_tokens<T, DELTA, LPC, 256 / LPC>), dim3(grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <typename T, bool DELTA>
hipError_t tokens_t(const PrefillArgs &a, hipStream_t st)
{
    if ((int64_t)a.n_seq * a.heads * a.dv <= 12288) return tokens_l<T, DELTA, 16>(a, st);
    return tokens_l<T, DELTA, 4>(a, st);
}

// ---------------------------------------------------------------- chunked form, d = 128, bfloat16
//
// C = 64 tokens at a time.  With G_i the running sum of log2 alpha in the
// chunk, D_ij = 2^(G_i - G_j) and S the state before it,
//     (I + tril(beta_i D_ij k_i.k_j, -1)) W = beta (V - 2^G (K S))
//     O = 2^G (Q S) + tril(D_ij q_i.k_j) W
//     S' = 2^G_C S + K^T (2^(G_C - G) W)
// (plain decay: W = beta V).  Everything is a product of 64- and 128-wide
// matrices, on the 16 x 16 x 32 bfloat16 matrix instructions.  The triangular
// system is solved by halves of 32 tokens: T_a, T_b are the inverses of its
// diagonal blocks (times beta), N the block D_ij k_i.k_j below, and
//     W_a = T_a X_a,   W_b = T_b (X_b - N W_a),   X = V - 2^G (K S).
// (Inverting all 64 rows at once costs four times the products of the two
// halves, on the slow fp32 matrix instructions.)
//
// Precision.  q, k and v are bfloat16, exact operands.  What is fp32 (S, T, W)
// enters a product as the sum of bfloat16 planes cut from its own mantissa:
// three planes of 8 bits are the fp32 value to the last bit, two are 16 bits
// of it.  Whatever feeds the state takes three planes (the state stays an
// fp32 computation over any length); what only reaches O, which is rounded to
// bfloat16, takes two: 2^-16 of the terms that O sums, where the 8 bits of the
// queries, keys and values themselves leave 2^-9 of them open.
//
// Operand order.  A 16 x 16 result holds rows 4 (lane / 16) + r of column
// lane % 16; an operand wants, per lane, 8 consecutive indexes 8 (lane / 16) + i
// of the 32 that an instruction sums over.  So result m holds, for the axis it
// shares with a later product, row x = index 32 (m / 2) + 8 (x / 4) + 4 (m % 2)
// + x % 4 (perm below): results 2 n and 2 n + 1 are then together, in the
// lane's own registers, the operand of indexes 32 n .. 32 n + 31.  No product's
// result passes through memory.  O is made transposed (the same registers as
// the other operand), so that a lane ends with four neighbouring columns.

constexpr int kC = 64, kD = 128;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ constexpr int perm(int m, int x)
{
    return 32 * (m >> 1) + 8 * (x >> 2) + 4 * (m & 1) + (x & 3);
}

// 2^x for running sums that may be long: the fraction is taken in double
__device__ __forceinline__ float pow2(double x)
{
    x = x < -160.0 ? -160.0 : x;
    const double n = __builtin_rint(x);
    return __builtin_ldexpf(__builtin_amdgcn_exp2f((float)(x - n)), (int)n);
}

// NP planes of 8 fp32 values as operands: each takes the top 16 bits of what
// the planes before it left.
template <int NP>
__device__ __forceinline__ void planes(const f32x4 &a, const f32x4 &b, bf16x8 (&p)[NP])
{
    float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int n = 0; n < NP; n++) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; i++)
            w[i] = __builtin_amdgcn_perm(__float_as_uint(x[2 * i + 1]), __float_as_uint(x[2 * i]), 0x07060302u);
        p[n] = __builtin_bit_cast(bf16x8, w);
        if (n + 1 < NP) {
#pragma unroll
            for (int i = 0; i < 8; i++) x[i] -= __uint_as_float(__float_as_uint(x[i]) & 0xffff0000u);
        }
    }
}

// Fragment f of a lower-triangular 64 x 64 operand: rows perm(mt, 0 .. 15),
// columns 32 ks .. + 31 (ks <= mt / 2; the rest is zero).
__device__ __forceinline__ constexpr int frag_of(int mt, int ks) { return mt + 2 * ks; }

// Keys and queries lie in shared memory row by row, the 16-byte pieces of row
// x exchanged by swz(x): the 16 rows that an operand's lanes read at once fall
// on 16 different bank groups.  Transposed keys (for the state's update) are
// read from the same rows by the transposing LDS read.
__device__ __forceinline__ constexpr int swz(int x) { return ((x >> 3) & 3) << 2 | (x & 3); }

constexpr int kH = 32, kLD = kH + 4;  // halves of the triangular system; rows stay 16-byte aligned

struct Side {
    double G[kC];                            // running sums of log2 alpha
    float gam[kC], dec[kC], be[kC];          // 2^G, 2^(G_C - G), beta
    float gh[kC], gl[kC];                    // G as the sum of two floats
};
struct SmemChunk {
    alignas(16) unsigned char K[2][kC * 256];
    alignas(16) unsigned char Q[2][kC * 256];
    alignas(16) unsigned char P[2][2][6 * 1024];  // planes of tril(D q.k), fragments
    alignas(16) Side side[4];
};
struct SmemChunkDelta : SmemChunk {
    alignas(16) unsigned char T[2][3][6 * 1024];  // planes of T_a, -N, T_b, fragments
    alignas(16) float A[2][2][kH * kLD];          // the inverses, of two chunks
};

__device__ __forceinline__ bf16x8 lds16(const unsigned char *p)
{
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(p));
}

// order of one wave's own shared-memory accesses across its lanes (the
// hardware keeps it; this keeps the compiler to it)
__device__ __forceinline__ void wave_order() { asm volatile("" ::: "memory"); }

// Rows of global memory, `n` of `row` bytes, `stride` bytes apart: reads past
// the last are zero, writes past it are dropped (the buffer instructions' own
// range check), so a chunk that ends inside the 64 tokens takes the same
// instructions as a whole one.  Offsets go into the lane's part: a scalar offset
// is not covered by the check in every case.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void *p, int n, int32_t stride, int32_t row)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (n - 1) * stride + row, 0x00027000);
}

// x, in a way that keeps sums with it from being made ahead of a loop (they
// would hold a register each through all of it)
__device__ __forceinline__ int32_t here(int32_t x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// log2 of x > 0 to the last bits of an fp32 result, also next to 1 where the
// result is small: exponent and log2 of the mantissa m in [0.7, 1.4) as
// 2 / ln 2 (y + y^3 / 3 + ...), y = (m - 1) / (m + 1), |y| < 0.172.
__device__ __forceinline__ double log2_exact(float x)
{
    int e;
    float m = frexpf(x, &e);  // [0.5, 1)
    if (m < 0.70710678f) {
        m *= 2.0f;
        e -= 1;
    }
    const float y = (m - 1.0f) / (m + 1.0f), z = y * y;
    float p = 1.0f / 11.0f;
    p = fmaf(p, z, 1.0f / 9.0f);
    p = fmaf(p, z, 1.0f / 7.0f);
    p = fmaf(p, z, 1.0f / 5.0f);
    p = fmaf(p, z, 1.0f / 3.0f);
    p = fmaf(p * z, y, y);
    return (double)e + (double)p * 2.8853900817779268;
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, true);
    return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Gates of one chunk, a lane per token.  The running sums are double: at
// half-lives of a few tokens they reach hundreds, and their differences have to
// keep their last bits.  A gate of zero counts as 2^-200: nothing before it is
// left.
__device__ __forceinline__ void make_side(Side &sd, int lane, float al, float bt)
{
    double x = al > 0.0f ? log2_exact(al) : al == 0.0f ? -200.0 : __builtin_nan("");
    x = dpp_add<0x111, 0xf>(x);  // row_shr 1, 2, 4, 8: sums within 16 lanes
    x = dpp_add<0x112, 0xf>(x);
    x = dpp_add<0x114, 0xf>(x);
    x = dpp_add<0x118, 0xf>(x);
    x = dpp_add<0x142, 0xa>(x);  // last lane of a row into the next: rows 1 and 3
    x = dpp_add<0x143, 0xc>(x);  // lane 31 into rows 2 and 3
    const double last = __shfl(x, 63);
    sd.G[lane] = x;
    sd.gam[lane] = pow2(x);
    sd.dec[lane] = pow2(last - x);
    sd.gh[lane] = (float)x;
    sd.gl[lane] = (float)(x - (double)(float)x);
    sd.be[lane] = bt;
}

// The products of one 16-row fragment: rows perm(mt, .) of q (or k) with the 32
// keys of kf, transposed (a lane gets one row's 8 weights: the operand's order).
struct Pair {
    f32x4 p[2];
};
__device__ __forceinline__ Pair products(const bf16x8 (&kf)[2][4], const bf16x8 (&rf)[4])
{
    Pair y{{f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}}};
#pragma unroll
    for (int x = 0; x < 4; x++)
#pragma unroll
        for (int u = 0; u < 2; u++) y.p[u] = mma(kf[u][x], rf[x], y.p[u]);
    return y;
}

// A fragment of tril(D_ij q_i.k_j), two planes.  D from G as two floats: gates of
// zero count 200 each, so a G rounded to one float would be off by up to 2^-11.
__device__ __forceinline__ void put_P(unsigned char (&P)[2][6 * 1024], const Side &sd, int mt, int ks, Pair y, int lane,
                                      int g, int c)
{
    const int i = perm(mt, c);
    const float Gi = sd.gh[i], gi = sd.gl[i];
#pragma unroll
    for (int u = 0; u < 2; u++) {
        const int j0 = perm(2 * ks + u, 4 * g);
        const f32x4 Gj = *reinterpret_cast<const f32x4 *>(&sd.gh[j0]);
        const f32x4 gj = *reinterpret_cast<const f32x4 *>(&sd.gl[j0]);
#pragma unroll
        for (int r = 0; r < 4; r++)
            y.p[u][r] = j0 + r <= i ? y.p[u][r] * __builtin_amdgcn_exp2f((Gi - Gj[r]) + (gi - gj[r])) : 0.0f;
    }
    bf16x8 pl[2];
    planes<2>(y.p[0], y.p[1], pl);
#pragma unroll
    for (int n = 0; n < 2; n++)
        *reinterpret_cast<u32x4 *>(&P[0][0] + lane * 16 + (6 * n + frag_of(mt, ks)) * 1024) =
            __builtin_bit_cast(u32x4, pl[n]);
}

// A fragment of -N (N_ij = D_ij k_i.k_j, i in the second half, j in the first),
// three planes: it reaches the state, so D is taken from the double sums.
__device__ __forceinline__ void put_N(unsigned char (&T)[3][6 * 1024], const Side &sd, int mt, Pair y, int lane, int g,
                                      int c)
{
    const double Gi = sd.G[perm(mt, c)];
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
        for (int r = 0; r < 4; r++)
            y.p[u][r] *= -__builtin_amdgcn_exp2f((float)(Gi - sd.G[perm(u, 4 * g) + r]));
    bf16x8 pl[3];
    planes<3>(y.p[0], y.p[1], pl);
#pragma unroll
    for (int n = 0; n < 3; n++)
        *reinterpret_cast<u32x4 *>(&T[0][0] + lane * 16 + (6 * n + frag_of(mt, 0)) * 1024) =
            __builtin_bit_cast(u32x4, pl[n]);
}

// The inverses of one chunk's two diagonal halves, by one wave.  kf[j][x]: keys
// 16 j + c, d = 32 x + 8 g ...  The four 16 x 16 diagonal blocks are inverted at
// once by forward substitution (a lane per column; stable whatever the keys,
// where a product of powers of the matrix is not), the block below each pair is
// -T_11 M_10 T_00 on the fp32 matrix instructions.
struct Gram {
    f32x4 kk[2][3];  // per half: blocks (0, 0), (1, 0), (1, 1) of K K^T
};
__device__ __forceinline__ Gram gram(const bf16x8 (&kf)[4][4])
{
    Gram y;
#pragma unroll
    for (int b = 0; b < 2; b++)
#pragma unroll
        for (int u = 0; u < 3; u++) y.kk[b][u] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int x = 0; x < 4; x++)
#pragma unroll
        for (int u = 0; u < 3; u++)
#pragma unroll
            for (int b = 0; b < 2; b++)
                y.kk[b][u] = mma(kf[2 * b + (u > 0)][x], kf[2 * b + (u > 1)][x], y.kk[b][u]);
    return y;
}

// The block above the diagonal of each half, which nothing else writes.
__device__ __forceinline__ void zero_A(float (&A)[2][kH * kLD], int lane)
{
#pragma unroll
    for (int b = 0; b < 2; b++)
        *reinterpret_cast<f32x4 *>(&A[b][(lane >> 2) * kLD + 16 + 4 * (lane & 3)]) = f32x4{0, 0, 0, 0};
}

// x_i = [i == c] + sum_{l < i} m_l(lane i) x_l, i = I .. 15
template <int I>
__device__ __forceinline__ void forward(const float (&m)[16], float (&x)[16], int c)
{
    float v = I == c ? 1.0f : 0.0f, w = 0.0f;
#pragma unroll
    for (int l = 0; l < I; l++) {
        const float b = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(m[l]), 0x150 + I, 0xf, 0xf, true));
        if (l & 1) w = fmaf(b, x[l], w);
        else v = fmaf(b, x[l], v);
    }
    x[I] = v + w;
    if constexpr (I < 15) forward<I + 1>(m, x, c);
}

__device__ __forceinline__ void invert(float (&A)[2][kH * kLD], const Side &sd, Gram y, int g, int c)
{
    float *Ag = &A[0][0] + 4 * g * kLD + c;
#pragma unroll
    for (int b = 0; b < 2; b++)
#pragma unroll
        for (int u = 0; u < 3; u++) {
            const int i0 = 16 * (u > 0) + 4 * g, j = 16 * (u > 1) + c;
            const double Gj = sd.G[32 * b + j];
            const f32x4 bi = *reinterpret_cast<const f32x4 *>(&sd.be[32 * b + i0]);
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const float m = bi[r] * __builtin_amdgcn_exp2f((float)(sd.G[32 * b + i0 + r] - Gj)) * y.kk[b][u][r];
                Ag[b * kH * kLD + (16 * (u > 0) + r) * kLD + 16 * (u > 1)] = i0 + r > j ? m : 0.0f;
            }
        }
    wave_order();
    {
        // block g: lane c brings row c of the matrix and leaves with column c of the
        // inverse; element (i, l) comes from lane i by a broadcast within the 16 lanes
        float *Ab = A[g >> 1] + 16 * (g & 1) * (kLD + 1);
        float m[16], x[16];
#pragma unroll
        for (int l = 0; l < 16; l += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(Ab + c * kLD + l);
#pragma unroll
            for (int e = 0; e < 4; e++) m[l + e] = -v[e];
        }
        forward<0>(m, x, c);
        wave_order();
#pragma unroll
        for (int i = 0; i < 16; i++) Ab[i * kLD + c] = x[i];
    }
    wave_order();
    {
        f32x4 R[2], X[2];
#pragma unroll
        for (int b = 0; b < 2; b++) {
            R[b] = X[b] = f32x4{0, 0, 0, 0};
            const f32x4 m = *reinterpret_cast<const f32x4 *>(A[b] + (16 + c) * kLD + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; e++)
                R[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(m[e], A[b][(4 * g + e) * kLD + c], R[b], 0, 0, 0);
        }
#pragma unroll
        for (int b = 0; b < 2; b++) {
            const f32x4 ti = *reinterpret_cast<const f32x4 *>(A[b] + (16 + c) * kLD + 16 + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; e++) X[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(ti[e], R[b][e], X[b], 0, 0, 0);
        }
        wave_order();
#pragma unroll
        for (int b = 0; b < 2; b++)
#pragma unroll
            for (int r = 0; r < 4; r++) A[b][(16 + 4 * g + r) * kLD + c] = -X[b][r];
    }
}

// The inverses times beta, as three planes.
__device__ __forceinline__ void put_T(unsigned char (&T)[3][6 * 1024], const float (&A)[2][kH * kLD], const Side &sd,
                                      int lane, int g, int c)
{
#pragma unroll
    for (int mt = 0; mt < 4; mt++) {
        const int b = mt >> 1, row = perm(mt & 1, c), col = 8 * g;
        f32x4 v[2];  // (zero above the diagonal: the inverses' own zeros, and the block that zero_A cleared)
#pragma unroll
        for (int u = 0; u < 2; u++) {
            v[u] = *reinterpret_cast<const f32x4 *>(A[b] + row * kLD + col + 4 * u);
            const f32x4 bb = *reinterpret_cast<const f32x4 *>(&sd.be[32 * b + col + 4 * u]);
            v[u] *= bb;
        }
        bf16x8 pl[3];
        planes<3>(v[0], v[1], pl);
#pragma unroll
        for (int p = 0; p < 3; p++)
            *reinterpret_cast<u32x4 *>(&T[0][0] + lane * 16 + (6 * p + frag_of(mt, b)) * 1024) =
                __builtin_bit_cast(u32x4, pl[p]);
    }
}

// The n-th longest of up to 64 sequences (in order of index where lengths are
// equal; above 64 sequences, simply the n-th).
__device__ __forceinline__ int nth_longest(const PrefillArgs &a, int n, int lane)
{
    if (a.n_seq > 64) return n;
    int len = -1;
    if (lane < a.n_seq) {
        const Seq r = seq_of(a, lane);
        len = r.last - r.first;
    }
    int rank = 0;
    for (int i = 0; i < a.n_seq; i++) {
        const int other = __builtin_amdgcn_readlane(len, i);
        rank += other > len || (other == len && i < lane);
    }
    return __builtin_ctzll(__ballot(lane < a.n_seq && rank == n));
}

// A workgroup walks one (sequence, head, 16 NW columns) chunk by chunk.  NW
// waves hold 16 columns of the state each and do nothing but chunk n; four more
// run ahead of them and make what is the same for all columns: they bring keys
// and queries to shared memory and compute P, T and N of chunk n + 1, the
// inverses of chunk n + 2 and the gates of chunk n + 3.  One barrier a chunk.
// Inputs are read once, and no intermediate leaves the CU.
//
// What bounds it.  8 ragged sequences x 48 heads up to 4,096 tokens take 465 to 478 us,
// 2.2 times what the bytes take at the card's copy rate.  The longest sequence's 64
// steps and the three before them, 12,800 cycles each, are 451 us of it at 1.9 GHz,
// the rest is the launch and the state's way in and out.  (Launched without a pause the
// clock falls: 500 to 630 us from the fourth launch on.)  Per step (cycles, whole heads,
// delta) the state's waves work 7,700 to 10,800, of which the matrix instructions
// are 5,800, keys with N and T 10,800, queries with gates and scores 9,500, the
// other scores 9,700 and the inverses' chain of dependent instructions 12,000.
//
// STEP.  kWhole: a workgroup takes a whole sequence.  With a plain decay the
// state after a segment is a sum, decay x (state before) + (what the segment
// writes), so long sequences of few heads are cut into segments of a.seg chunks:
// kWrites leaves what each segment writes from zero, and its decay, in the
// workspace, and kSegment then starts each segment from the sum of those before
// it.  The first pass needs neither queries nor outputs: two fifths of the work.
enum Step { kWhole, kWrites, kSegment };

template <bool DELTA, int NW, int STEP>
__global__ __launch_bounds__(64 * (NW + 4)) void k_prefill_chunks(PrefillArgs a)
{
    static_assert(STEP == kWhole || !DELTA, "the delta rule's segments do not add up");
    using SM = typename std::conditional<DELTA, SmemChunkDelta, SmemChunk>::type;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SM &sm = *reinterpret_cast<SM *>(smem_raw);

    const int t = threadIdx.x, lane = t & 63, g = lane >> 4, c = lane & 15;
    const int wv = __builtin_amdgcn_readfirstlane(t >> 6);
    // workgroups of long sequences first (the rest fills in behind them); the
    // column splits of a head next to each other
    const int split = (int)(blockIdx.x % (unsigned)(8 / NW));
    const unsigned rest = blockIdx.x / (unsigned)(8 / NW);
    const int h = (int)(rest % (unsigned)a.heads);
    int s, segment = 0, more = 0;  // the segment's number, and how many follow it
    Seq sr;
    if constexpr (STEP == kWhole) {
        s = nth_longest(a, (int)(rest / (unsigned)a.heads), lane);
        sr = seq_of(a, s);
    } else {
        // segment i of sequence s is record first / length + s + i: records of
        // different sequences are disjoint
        const int rec = (int)(rest / (unsigned)a.heads), length = a.seg * kC;
        for (s = 0; s + 1 < a.n_seq && seq_of(a, s + 1).first / length + s + 1 <= rec;) s++;
        sr = seq_of(a, s);
        segment = rec - (sr.first / length + s);
        const int64_t from = sr.first + (int64_t)segment * length;
        if (segment < 0 || (from >= sr.last && segment > 0)) return;
        // the last segment's writes are not asked for
        if (STEP == kWrites && from + length >= sr.last) return;
        sr.first = (int32_t)from;
        more = (sr.last - sr.first - 1) / length;
    }
    if (more > 0) sr.last = sr.first + a.seg * kC;
    const int64_t sh = (int64_t)s * a.heads + h;
    const int chunks = (sr.last - sr.first + kC - 1) / kC;
    // row strides in bytes (the host has checked that 64 rows are below 2^31)
    const int32_t ks2 = (int32_t)a.k_stride * 2, qs2 = (int32_t)a.q_stride * 2, vs2 = (int32_t)a.v_stride * 2;
    const int32_t os2 = a.heads * kD * 2;
    const uint16_t *q = reinterpret_cast<const uint16_t *>(a.q) + (int64_t)(h / a.per_k) * kD;
    const uint16_t *k = reinterpret_cast<const uint16_t *>(a.k) + (int64_t)(h / a.per_k) * kD;

    auto first_of = [&](int n) { return (int64_t)sr.first + (int64_t)n * kC; };
    auto tokens_of = [&](int n) {
        const int64_t left = sr.last - first_of(n);
        return left < kC ? (int)left : kC;
    };
    auto key_window = [&](int n) { return rows_of(k + first_of(n) * a.k_stride, tokens_of(n), ks2, 256); };
    auto query_window = [&](int n) { return rows_of(q + first_of(n) * a.q_stride, tokens_of(n), qs2, 256); };
    const int32_t rho = 8 * (c >> 2) + (c & 3);  // perm(m, c) = perm(m, 0) + rho

    if (wv >= NW) {
        if (chunks == 0) return;
        const int role = wv - NW;
        if (STEP == kWrites && role >= 2) return;
        // an operand's pieces straight from global memory: rows perm(m, c)
        auto rows = [&](__amdgpu_buffer_rsrc_t w, int32_t st, int m, bf16x8 (&f)[4]) {
            const int32_t b = here(rho * st + 16 * g) + perm(m, 0) * st;
#pragma unroll
            for (int x = 0; x < 4; x++)
                f[x] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(w, b + 64 * x, 0, 0));
        };
        // In step n the state's waves are at chunk n (or have not begun); chunk n + 1
        // is made ready, the inverses of chunk n + 2 and the gates of chunk n + 3.
        // 64 rows from global to shared memory: row 4 u + g, 16-byte piece c, at
        // exchanged piece c ^ swz(4 u + g) = c ^ (4 (u / 2 mod 4) + g)
        int at_w[4], at_own[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            at_w[i] = g * 256 + ((c ^ (4 * i + g)) * 16);
            at_own[i] = rho * 256 + (((4 * i + g) ^ c) * 16);  // piece 4 i + g of row perm(0, c)
        }
        auto load_rows = [&](__amdgpu_buffer_rsrc_t w, int32_t st, u32x4 (&x)[16]) {
            const int32_t b = here(g * st + c * 16);
#pragma unroll
            for (int u = 0; u < 16; u++) x[u] = __builtin_amdgcn_raw_buffer_load_b128(w, b + 4 * u * st, 0, 0);
        };
        auto put_rows = [&](unsigned char *dst, const u32x4 (&x)[16]) {
#pragma unroll
            for (int u = 0; u < 16; u++) *reinterpret_cast<u32x4 *>(dst + at_w[(u >> 1) & 3] + u * 1024) = x[u];
            wave_order();
        };
        // an operand from rows that this wave has put itself
        auto own = [&](const unsigned char *dst, int m, bf16x8 (&o)[4]) {
#pragma unroll
            for (int x = 0; x < 4; x++) o[x] = lds16(dst + at_own[x] + perm(m, 0) * 256);
        };
        if (role == 0) {
            // keys; N and T of the delta rule, half of P with a plain decay.  The rows are
            // loaded a step ahead, which also brings them to the L2 cache for the waves
            // that load operands from global memory.
            u32x4 x[16];
            load_rows(key_window(0), ks2, x);
            for (int n = -3; n < chunks; n++) {
                lds_barrier();
                if (n + 1 < 0 || n + 1 >= chunks) continue;
                unsigned char *dst = sm.K[(n + 1) & 1];
                const Side &sd = sm.side[(n + 1) & 3];
                put_rows(dst, x);
                if (n + 2 < chunks) load_rows(key_window(n + 2), ks2, x);
                if constexpr (DELTA) {
                    Pair y[2];
#pragma unroll
                    for (int m = 0; m < 2; m++) y[m].p[0] = y[m].p[1] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int x = 0; x < 4; x++) {
                        bf16x8 e[4];
#pragma unroll
                        for (int m = 0; m < 4; m++) e[m] = lds16(dst + at_own[x] + perm(m, 0) * 256);
#pragma unroll
                        for (int m = 0; m < 2; m++)
#pragma unroll
                            for (int u = 0; u < 2; u++) y[m].p[u] = mma(e[u], e[2 + m], y[m].p[u]);
                    }
#pragma unroll
                    for (int m = 0; m < 2; m++) put_N(sm.T[(n + 1) & 1], sd, 2 + m, y[m], here(lane), here(g), here(c));
                    put_T(sm.T[(n + 1) & 1], sm.A[(n + 1) & 1], sd, here(lane), here(g), here(c));
                } else if constexpr (STEP != kWrites) {
                    bf16x8 e[2][4], i[4];
                    own(dst, 0, e[0]);
                    own(dst, 1, e[1]);
#pragma unroll
                    for (int m = 0; m < 2; m++) {
                        rows(query_window(n + 1), qs2, m, i);
                        put_P(sm.P[(n + 1) & 1], sd, m, 0, products(e, i), lane, g, c);
                    }
                }
            }
        } else if (role == 1) {
            // queries and gates; half of P for the delta rule
            u32x4 x[16];
            float al = 1.0f, bt = 0.0f;
            auto gates = [&](int n) {
                const bool in = lane < tokens_of(n);
                const int64_t i = (first_of(n) + lane) * a.heads + h;
                al = in ? a.alpha[i] : 1.0f;
                bt = in ? a.beta[i] : 0.0f;
            };
            gates(0);
            if constexpr (STEP != kWrites) load_rows(query_window(0), qs2, x);
            for (int n = -3; n < chunks; n++) {
                lds_barrier();
                if (n + 3 < chunks) {
                    make_side(sm.side[(n + 3) & 3], lane, al, bt);
                    if (n + 4 < chunks) gates(n + 4);
                }
                if (STEP == kWrites || n + 1 < 0 || n + 1 >= chunks) continue;
                unsigned char *dst = sm.Q[(n + 1) & 1];
                put_rows(dst, x);
                if (n + 2 < chunks) load_rows(query_window(n + 2), qs2, x);
                if constexpr (DELTA) {
                    const auto kw = key_window(n + 1);
                    bf16x8 f[2][4], e[4];
                    rows(kw, ks2, 0, f[0]);
                    rows(kw, ks2, 1, f[1]);
#pragma unroll
                    for (int m = 0; m < 2; m++) {
                        own(dst, m, e);
                        put_P(sm.P[(n + 1) & 1], sm.side[(n + 1) & 3], m, 0, products(f, e), lane, g, c);
                    }
                }
            }
        } else if (!DELTA || role == 2) {
            // P's other half (plain decay: shared with the fourth wave)
            constexpr int N = DELTA ? 2 : 1;
            bf16x8 kf[N][2][4], qf[2][4];
            const int ks0 = DELTA ? 0 : role - 2;
            for (int n = -3; n < chunks; n++) {
                lds_barrier();
                if (n + 1 < 0 || n + 1 >= chunks) continue;
                const auto kw = key_window(n + 1), qw = query_window(n + 1);
#pragma unroll
                for (int m = 0; m < 2; m++) {
                    rows(qw, qs2, 2 + m, qf[m]);
#pragma unroll
                    for (int z = 0; z < N; z++) rows(kw, ks2, 2 * (ks0 + z) + m, kf[z][m]);
                }
#pragma unroll
                for (int z = 0; z < N; z++)
#pragma unroll
                    for (int m = 0; m < 2; m++)
                        put_P(sm.P[(n + 1) & 1], sm.side[(n + 1) & 3], 2 + m, ks0 + z, products(kf[z], qf[m]), lane, g, c);
            }
        } else if constexpr (DELTA) {
            // The inverses take longest: they are made a chunk earlier than the rest, their
            // keys loaded a step before that.  (No raised priority: the two state waves of
            // the same SIMD then fall behind, 490 us against 435 for the longest sequence
            // of prompts of 384 heads.)
            bf16x8 kf[4][4];
            zero_A(sm.A[0], lane);
            zero_A(sm.A[1], lane);
            for (int n = -3; n < chunks; n++) {
                lds_barrier();
                const bool now = n + 2 >= 0 && n + 2 < chunks;
                Gram y;
                if (now) y = gram(kf);
                if (n + 3 < chunks) {
                    const auto kw = key_window(n + 3);
                    const int32_t b = here(c * ks2 + 16 * g);
#pragma unroll
                    for (int m = 0; m < 4; m++)
#pragma unroll
                        for (int x = 0; x < 4; x++)
                            kf[m][x] = __builtin_bit_cast(
                                bf16x8, __builtin_amdgcn_raw_buffer_load_b128(kw, b + 16 * m * ks2 + 64 * x, 0, 0));
                }
                if (now) invert(sm.A[n & 1], sm.side[(n + 2) & 3], y, here(g), here(c));
            }
        }
        return;
    }

    // the state: result m, row perm(m, 4 g + r), column col0 + c
    const int col0 = (split * NW + wv) * 16;
    const int64_t tile = sh * kD * kD + col0 + c;
    f32x4 S[8];
#pragma unroll
    for (int m = 0; m < 8; m++)
#pragma unroll
        for (int r = 0; r < 4; r++)
            S[m][r] = a.S0 && (STEP == kWhole || segment == 0) ? a.S0[tile + (int64_t)perm(m, 4 * g + r) * kD] : 0.0f;
    float decay = 1.0f;  // of the whole segment
    float *ws_decay = reinterpret_cast<float *>(a.ws);
    float *ws_state = ws_decay + a.seg_pad;
    const int64_t rec = (int64_t)(rest / (unsigned)a.heads) * a.heads + h;
    auto slot = [&](int64_t record) { return ws_state + record * kD * kD + col0 + c; };
    if constexpr (STEP != kWhole) {
        // S may be S0, and the last segment may end before the first begins: the
        // first pass keeps S0 in the last segment's record, which it leaves unused
        if (segment == 0 && more > 0 && a.S0 && a.S) {
            float *kept = slot(rec + (int64_t)more * a.heads);
#pragma unroll
            for (int m = 0; m < 8; m++)
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    float *p = kept + (int64_t)perm(m, 4 * g + r) * kD;
                    if (STEP == kWrites) *p = S[m][r];
                    else S[m][r] = *p;
                }
        }
    }
    if constexpr (STEP == kSegment) {
        // (segment 0 started from S0, so its writes hold the state itself)
        for (int i = segment; i > 0; i--) {
            const float *src = slot(rec - (int64_t)i * a.heads);
            const float f = ws_decay[rec - (int64_t)i * a.heads];
#pragma unroll
            for (int m = 0; m < 8; m++)
#pragma unroll
                for (int r = 0; r < 4; r++) S[m][r] = fmaf(f, S[m][r], src[(int64_t)perm(m, 4 * g + r) * kD]);
        }
    }

    const uint16_t *v = reinterpret_cast<const uint16_t *>(a.v) + (int64_t)h * kD + col0;
    uint16_t *o = reinterpret_cast<uint16_t *>(a.o) + (int64_t)h * kD + col0;
    const int32_t at_v = 8 * g * vs2 + 2 * c, at_o = rho * os2 + 8 * g;
    uint16_t vr[4][4];  // the next chunk's values
    auto load_v = [&](int n) {
        const auto w = rows_of(v + first_of(n) * a.v_stride, tokens_of(n), vs2, 32);
        const int32_t b = here(at_v);
#pragma unroll
        for (int m = 0; m < 4; m++)
#pragma unroll
            for (int r = 0; r < 4; r++)
                vr[m][r] = __builtin_amdgcn_raw_buffer_load_b16(w, b + perm(m, r) * vs2, 0, 0);
    };
    // swz(perm(m, c)) = c: piece 4 x + g of row perm(m, c) lies here, perm(m, 0) rows on
    int at_row[4], at_kt[4];
#pragma unroll
    for (int x = 0; x < 4; x++) {
        at_row[x] = rho * 256 + (((4 * x + g) ^ c) * 16);
        // transposing read: lanes 4 i + z of 16 read token 8 g + i (+ 32 ks + 4 u, which
        // leaves swz alone), d 32 x + 8 z (+ 4); each gets four tokens of one d
        at_kt[x] = (8 * g + (c >> 2)) * 256 + (((4 * x + (c & 3)) ^ swz(8 * g + (c >> 2))) * 16);
    }
    auto rows = [&](const unsigned char *base, int m, int x) { return lds16(base + at_row[x] + perm(m, 0) * 256); };

    if (chunks > 0) {
        load_v(0);
        lds_barrier();
        lds_barrier();
        lds_barrier();
    }
    for (int n = 0; n < chunks; n++) {
        lds_barrier();
        const unsigned char *K = sm.K[n & 1], *Q = sm.Q[n & 1];
        const Side &sd = sm.side[n & 3];
        f32x4 W[4];  // V, then V - 2^G K S, then W
#pragma unroll
        for (int m = 0; m < 4; m++)
#pragma unroll
            for (int r = 0; r < 4; r++) W[m][r] = __uint_as_float((uint32_t)vr[m][r] << 16);
        if (n + 1 < chunks) load_v(n + 1);

        // K S, and S^T Q^T
        f32x4 O[4];
        if constexpr (STEP == kWrites) {
#pragma unroll
            for (int m = 0; m < 4; m++) W[m] *= *reinterpret_cast<const f32x4 *>(&sd.be[perm(m, 4 * g)]);
        } else {
            f32x4 KS[4];
#pragma unroll
            for (int m = 0; m < 4; m++) O[m] = KS[m] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int x = 0; x < 4; x++) {
                bf16x8 sp[3];
                planes<3>(S[2 * x], S[2 * x + 1], sp);
#pragma unroll
                for (int mh = 0; mh < 4; mh += 2) {
                    bf16x8 qf[2], kf[2];
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        qf[i] = rows(Q, mh + i, x);
                        if constexpr (DELTA) kf[i] = rows(K, mh + i, x);
                    }
#pragma unroll
                    for (int p = 0; p < 3; p++)
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            if (p < 2) O[mh + i] = mma(sp[p], qf[i], O[mh + i]);
                            if constexpr (DELTA) KS[mh + i] = mma(kf[i], sp[p], KS[mh + i]);
                        }
                }
            }
#pragma unroll
            for (int m = 0; m < 4; m++) {
                O[m] *= sd.gam[perm(m, c)];
                if constexpr (DELTA) W[m] -= *reinterpret_cast<const f32x4 *>(&sd.gam[perm(m, 4 * g)]) * KS[m];
                else W[m] *= *reinterpret_cast<const f32x4 *>(&sd.be[perm(m, 4 * g)]);
            }
        }
        const float gC = sd.gam[kC - 1];
        if constexpr (STEP == kWrites) decay *= gC;
#pragma unroll
        for (int m = 0; m < 8; m++) S[m] *= gC;
#pragma unroll
        for (int ks = 0; ks < 2; ks++) {
            const int m0 = 2 * ks;
            bf16x8 wp[3];
            if constexpr (DELTA) {
                // W = T X, half by half; the first half's W then leaves X of the second
                const auto &T = sm.T[n & 1];
                planes<3>(W[m0], W[m0 + 1], wp);
                f32x4 Y[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
                for (int p = 0; p < 3; p++) {
                    const bf16x8 t0 = lds16(T[p] + frag_of(m0, ks) * 1024 + lane * 16);
                    const bf16x8 t1 = lds16(T[p] + frag_of(m0 + 1, ks) * 1024 + lane * 16);
#pragma unroll
                    for (int z = 0; z < 3 - p; z++) {
                        Y[0] = mma(t0, wp[z], Y[0]);
                        Y[1] = mma(t1, wp[z], Y[1]);
                    }
                }
                W[m0] = Y[0];
                W[m0 + 1] = Y[1];
                planes<3>(W[m0], W[m0 + 1], wp);
                if (ks == 0) {
#pragma unroll
                    for (int p = 0; p < 3; p++) {
                        const bf16x8 t0 = lds16(T[p] + frag_of(2, 0) * 1024 + lane * 16);
                        const bf16x8 t1 = lds16(T[p] + frag_of(3, 0) * 1024 + lane * 16);
#pragma unroll
                        for (int z = 0; z < 3 - p; z++) {
                            W[2] = mma(t0, wp[z], W[2]);
                            W[3] = mma(t1, wp[z], W[3]);
                        }
                    }
                }
            } else if constexpr (STEP != kWrites) {
                planes<3>(W[m0], W[m0 + 1], wp);
            }
            if constexpr (STEP != kWrites) {
            // O^T = 2^G (S^T Q^T) + W^T P^T
            bf16x8 p0[4], p1[4];
#pragma unroll
            for (int m = m0; m < 4; m++) {
                p0[m] = lds16(sm.P[n & 1][0] + frag_of(m, ks) * 1024 + lane * 16);
                p1[m] = lds16(sm.P[n & 1][1] + frag_of(m, ks) * 1024 + lane * 16);
            }
#pragma unroll
            for (int m = m0; m < 4; m++) O[m] = mma(wp[0], p0[m], O[m]);
#pragma unroll
            for (int m = m0; m < 4; m++) O[m] = mma(wp[1], p0[m], O[m]);
#pragma unroll
            for (int m = m0; m < 4; m++) O[m] = mma(wp[0], p1[m], O[m]);
            }
            // S' = 2^G_C S + K^T (2^(G_C - G) W)
            const f32x4 d0 = *reinterpret_cast<const f32x4 *>(&sd.dec[32 * ks + 8 * g]);
            const f32x4 d1 = *reinterpret_cast<const f32x4 *>(&sd.dec[32 * ks + 8 * g + 4]);
            planes<3>(W[m0] * d0, W[m0 + 1] * d1, wp);
#pragma unroll
            for (int mh = 0; mh < 8; mh += 4) {
                bf16x8 kt[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int m = mh + i;
                    s16x4 part[2];
#pragma unroll
                    for (int u = 0; u < 2; u++)
                        part[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (__attribute__((address_space(3))) s16x4 *)(K + at_kt[m >> 1] + (32 * ks + 4 * u) * 256 +
                                                                       (m & 1) * 8));
                    kt[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7));
                }
#pragma unroll
                for (int p = 0; p < 3; p++)
#pragma unroll
                    for (int i = 0; i < 4; i++) S[mh + i] = mma(kt[i], wp[p], S[mh + i]);
            }
        }
        if constexpr (STEP != kWrites) {
        // a lane's four neighbouring columns of token perm(m, c)
        const auto ow = rows_of(o + first_of(n) * a.heads * kD, tokens_of(n), os2, 32);
#pragma unroll
        for (int m = 0; m < 4; m++) {
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, __builtin_convertvector(O[m], bf16x4)),
                                                  ow, here(at_o) + perm(m, 0) * os2, 0, 0);
        }
        }
    }
    if constexpr (STEP == kWrites) {
        float *dst = slot(rec);
#pragma unroll
        for (int m = 0; m < 8; m++)
#pragma unroll
            for (int r = 0; r < 4; r++) dst[(int64_t)perm(m, 4 * g + r) * kD] = S[m][r];
        // (every wave writes the same decay)
        if (lane == 0) ws_decay[rec] = decay;
        return;
    }
    if (!a.S || more > 0) return;
#pragma unroll
    for (int m = 0; m < 8; m++)
#pragma unroll
        for (int r = 0; r < 4; r++) a.S[tile + (int64_t)perm(m, 4 * g + r) * kD] = S[m][r];
}

template <bool DELTA, int NW, int STEP>
hipError_t chunks_t(const PrefillArgs &a, int64_t units, hipStream_t st)
{
    const int64_t grid = units * a.heads * (8 / NW);
    if (!grid_fits(grid, 64 * (NW + 4))) return hipErrorInvalidConfiguration;
    const size_t lds = DELTA ? sizeof(SmemChunkDelta) : sizeof(SmemChunk);
    auto kern = k_prefill_chunks<DELTA, NW, STEP>;
    if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds))
        return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(64 * (NW + 4)), lds, st, a);
    return hipGetLastError();
}

// How a plain decay's sequences are cut: chunks per segment (0: not), and the
// number of segment records.  Worth it while the heads of all sequences leave
// CUs idle and the sequences are long, 40 chunks on average; the segments then
// fill the 256 CUs once (48 heads x 16 Ki tokens from a state 429 us against 779 uncut, 64 heads x
// 4,096 tokens 135 against 167, 96 heads 232 against 218; 64 heads x 2,048 tokens 94
// against 83).
struct Cut {
    int32_t seg;
    int64_t records;
};
constexpr int32_t kCutHeads = 64, kCutMin = 40, kSegMin = 16;

Cut cut_of(int32_t n_seq, int32_t n_tokens, int32_t heads)
{
    const int64_t sh = (int64_t)n_seq * heads, chunks = ((int64_t)n_tokens + kC - 1) / kC;
    if (sh > kCutHeads || chunks < (int64_t)kCutMin * n_seq) return Cut{0, 0};
    int64_t seg = (chunks * heads + 255 - sh) / (256 - sh);
    if (seg < kSegMin) seg = kSegMin;
    return Cut{(int32_t)seg, (int64_t)n_tokens / (seg * kC) + n_seq + 1};
}

// decays, padded to whole lines, then states
int64_t cut_pad(int64_t rows) { return (rows + 63) / 64 * 64; }
uint64_t cut_bytes(int64_t rows) { return 4 * ((uint64_t)cut_pad(rows) + (uint64_t)rows * kD * kD); }

template <bool DELTA>
hipError_t chunked(const PrefillArgs &a, hipStream_t st)
{
    if constexpr (!DELTA) {
        const Cut cut = cut_of(a.n_seq, a.n_tokens, a.heads);
        if (cut.seg > 0) {
            PrefillArgs b = a;
            b.seg = cut.seg;
            b.seg_pad = cut_pad(cut.records * a.heads);
            if (hipError_t e = chunks_t<false, 8, kWrites>(b, cut.records, st)) return e;
            return chunks_t<false, 8, kSegment>(b, cut.records, st);
        }
    }
    // One workgroup fits a CU.  While the halves of all heads fit the 256 CUs
    // together, two workgroups a head are faster (a step of fewer columns: delta,
    // 96 heads x 4,096 tokens 321 us against 360, 48 heads 272 against 335); above
    // that, whole heads, whose common work is done once (144 heads 356 us against
    // 562, 192 heads 387 against 578).
    return (int64_t)a.n_seq * a.heads <= 128 ? chunks_t<DELTA, 4, kWhole>(a, a.n_seq, st)
                                             : chunks_t<DELTA, 8, kWhole>(a, a.n_seq, st);
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// bfloat16 tiles of 128 x 128 with rows that 16-byte loads can take
bool chunk_shape(int32_t dk, int32_t dv, bool bf16) { return bf16 && dk == kD && dv == kD; }

bool chunk_aligned(const PrefillArgs &a)
{
    constexpr int64_t kMost = 1 << 23;  // elements between tokens: 64 rows stay below 2^31 bytes
    return aligned16(a.q) && aligned16(a.k) && aligned16(a.v) && aligned16(a.o) && a.q_stride % 8 == 0 &&
           a.k_stride % 8 == 0 && a.v_stride % 8 == 0 && a.q_stride <= kMost && a.k_stride <= kMost &&
           a.v_stride <= kMost && (int64_t)a.heads * kD <= kMost;
}

bool takes_chunks(const PrefillArgs &a, bool bf16)
{
    // A few tokens a sequence go faster one by one than as a padded chunk (delta, 768
    // heads: 8 tokens each 36 us against 43, 12 tokens 41 against 43, 16 tokens 46
    // against 43; 48 heads: 12 tokens 10.7 against 11.6, 16 tokens 11.1 against 11.5).
    // A plain decay would have it lower (768 heads: 8 tokens 34 against 30, 12 tokens 39
    // against 30).  The average is all that the host knows: 400 single tokens with
    // one sequence of 4,096 take 2,730 us, the long one by itself 285.
    const bool few = a.n_tokens <= 12 * (int64_t)a.n_seq;
    return chunk_shape(a.dk, a.dv, bf16) && chunk_aligned(a) && !few;
}

}  // namespace

uint64_t prefill_workspace(int32_t n_seq, int32_t n_tokens, int32_t heads, int32_t dk, int32_t dv, bool bf16,
                           bool delta)
{
    // for every call with at most these sizes: records x heads <= min(n_tokens /
    // (64 kSegMin) heads, 256) + n_seq heads + heads, n_seq heads <= kCutHeads
    if (!chunk_shape(dk, dv, bf16) || delta || ((int64_t)n_tokens + kC - 1) / kC < kCutMin || n_seq < 1) return 0;
    const int64_t by_tokens = (int64_t)n_tokens / (kSegMin * kC) * heads, sh = (int64_t)n_seq * heads;
    return cut_bytes((by_tokens < 256 ? by_tokens : 256) + (sh < kCutHeads ? sh : kCutHeads) +
                     (heads < kCutHeads ? heads : kCutHeads));
}

uint64_t prefill_needs(const PrefillArgs &a, bool bf16, bool delta)
{
    if (!takes_chunks(a, bf16) || delta) return 0;
    const Cut cut = cut_of(a.n_seq, a.n_tokens, a.heads);
    return cut.seg > 0 ? cut_bytes(cut.records * a.heads) : 0;
}

hipError_t launch_prefill(const PrefillArgs &a, bool bf16, bool delta, hipStream_t st)
{
    if (takes_chunks(a, bf16)) return delta ? chunked<true>(a, st) : chunked<false>(a, st);
    if (bf16) return delta ? tokens_t<uint16_t, true>(a, st) : tokens_t<uint16_t, false>(a, st);
    return delta ? tokens_t<float, true>(a, st) : tokens_t<float, false>(a, st);
}

}  // namespace sqk
