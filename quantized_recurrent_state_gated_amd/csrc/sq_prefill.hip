// sq_prefill.hip -- gfx950 kernels of the prompt form of the recurrent
// layers: a whole sequence of tokens through
//     S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T   (delta)
//     S_t = alpha_t S_{t-1} + beta_t k_t v_t^T                          (plain decay)
//     o_t = S_t^T q_t
// from the state S_0 (or zero) to the state that the decode steps go on from.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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

// Tokens [first, last) of sequence s, held inside [0, n_tokens) whatever cu says.
struct Seq {
    int32_t first, last;
};

__device__ __forceinline__ Seq seq_of(const PrefillArgs &a, int s)
{
    Seq r{a.cu[s], a.cu[s + 1]};
    if (r.first < 0) r.first = 0;
    if (r.last > a.n_tokens) r.last = a.n_tokens;
    if (r.last < r.first) r.last = r.first;
    return r;
}

// ---------------------------------------------------------------- token by token
//
// Any d_k, d_v (multiples of 4, at most 256) and both element types: one
// workgroup per (sequence, head, 64 columns), four lanes per column, each
// holding RPL rows of it in registers.  The columns of S are independent of
// each other; per token a lane does three fused multiply-adds a row for
//     u = k^T S, y = q^T S, and the update S = alpha S + k w,
//     w = beta (v - alpha u), o = alpha y + (q.k) w,
// and the four lanes join their sums with two exchanges.  Tokens are staged
// through shared memory TB at a time.

constexpr int kTB = 16;  // tokens staged at a time

__device__ __forceinline__ float quad_sum(float x)
{
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0xb1, 0xf, 0xf, false));
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x4e, 0xf, 0xf, false));
    return x;
}

template <typename T, bool DELTA, int RPL>
__global__ __launch_bounds__(256) void k_prefill_tokens(PrefillArgs a)
{
    constexpr int ROWS = 4 * RPL;
    __shared__ __align__(16) float sq[kTB][ROWS], sk[kTB][ROWS];
    __shared__ float sv[kTB][64], sg[kTB][2];
    const int t = threadIdx.x, part = t & 3, col = t >> 2;
    const int tiles = (a.dv + 63) / 64;
    const int j0 = (int)(blockIdx.x % (unsigned)tiles) * 64;
    const int sh = (int)(blockIdx.x / (unsigned)tiles);
    const int h = sh % a.heads, s = sh / a.heads;
    const Seq sr = seq_of(a, s);
    const int j = j0 + col;
    const bool in = j < a.dv;
    const int64_t tile = (int64_t)sh * a.dk * a.dv;

    // row 16 i + 4 part + e
    float S[RPL];
#pragma unroll
    for (int i = 0; i < RPL; i++) {
        const int row = 16 * (i >> 2) + 4 * part + (i & 3);
        S[i] = a.S0 && in && row < a.dk ? a.S0[tile + (int64_t)row * a.dv + j] : 0.0f;
    }
    const T *q = reinterpret_cast<const T *>(a.q) + (int64_t)(h / a.per_k) * a.dk;
    const T *k = reinterpret_cast<const T *>(a.k) + (int64_t)(h / a.per_k) * a.dk;
    const T *v = reinterpret_cast<const T *>(a.v) + (int64_t)h * a.dv;
    T *o = reinterpret_cast<T *>(a.o) + (int64_t)h * a.dv;

    for (int32_t t0 = sr.first; t0 < sr.last; t0 += kTB) {
        const int nt = sr.last - t0 < kTB ? sr.last - t0 : kTB;
        __syncthreads();
        for (int i = t; i < nt * ROWS; i += 256) {
            const int x = i / ROWS, d = i % ROWS;
            const int64_t tok = t0 + x;
            sq[x][d] = d < a.dk ? up<T>(q[tok * a.q_stride + d]) : 0.0f;
            sk[x][d] = d < a.dk ? up<T>(k[tok * a.k_stride + d]) : 0.0f;
        }
        for (int i = t; i < nt * 64; i += 256) {
            const int x = i >> 6, d = i & 63;
            sv[x][d] = j0 + d < a.dv ? up<T>(v[(int64_t)(t0 + x) * a.v_stride + j0 + d]) : 0.0f;
        }
        if (t < nt) {
            sg[t][0] = a.alpha[(int64_t)(t0 + t) * a.heads + h];
            sg[t][1] = a.beta[(int64_t)(t0 + t) * a.heads + h];
        }
        __syncthreads();
        for (int x = 0; x < nt; x++) {
            float u = 0.0f, y = 0.0f, qk = 0.0f, kr[RPL];
#pragma unroll
            for (int i = 0; i < RPL; i += 4) {
                const float4 k4 = *reinterpret_cast<const float4 *>(&sk[x][4 * i + 4 * part]);
                const float4 q4 = *reinterpret_cast<const float4 *>(&sq[x][4 * i + 4 * part]);
                const float qe[4] = {q4.x, q4.y, q4.z, q4.w};
                kr[i] = k4.x; kr[i + 1] = k4.y; kr[i + 2] = k4.z; kr[i + 3] = k4.w;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    if (DELTA) u = fmaf(kr[i + e], S[i + e], u);
                    y = fmaf(qe[e], S[i + e], y);
                    qk = fmaf(qe[e], kr[i + e], qk);
                }
            }
            if (DELTA) u = quad_sum(u);
            y = quad_sum(y);
            qk = quad_sum(qk);
            const float al = sg[x][0], vj = sv[x][col];
            const float w = sg[x][1] * (DELTA ? vj - al * u : vj);
#pragma unroll
            for (int i = 0; i < RPL; i++) S[i] = fmaf(al, S[i], kr[i] * w);
            if (part == 0 && in)
                o[(int64_t)(t0 + x) * a.heads * a.dv + j] = down<T>(fmaf(al, y, qk * w));
        }
    }
    if (!a.S || !in) return;
#pragma unroll
    for (int i = 0; i < RPL; i++) {
        const int row = 16 * (i >> 2) + 4 * part + (i & 3);
        if (row < a.dk) a.S[tile + (int64_t)row * a.dv + j] = S[i];
    }
}

template <typename T, bool DELTA>
hipError_t tokens_t(const PrefillArgs &a, hipStream_t st)
{
    const unsigned grid = (unsigned)((int64_t)a.n_seq * a.heads * ((a.dv + 63) / 64));
    if (a.dk <= 64)
        hipLaunchKernelGGL((k_prefill_tokens<T, DELTA, 16>), dim3(grid), dim3(256), 0, st, a);
    else if (a.dk <= 128)
        hipLaunchKernelGGL((k_prefill_tokens<T, DELTA, 32>), dim3(grid), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((k_prefill_tokens<T, DELTA, 64>), dim3(grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

// ---------------------------------------------------------------- chunked form, d = 128, bfloat16
//
// C = 64 tokens at a time.  With G_i the running sum of log2 alpha in the
// chunk, D_ij = 2^(G_i - G_j) and S the state before it,
//     W = T (V - 2^G (K S)),   T = (I + tril(beta_i D_ij k_i.k_j, -1))^-1 diag(beta)
//     O = 2^G (Q S) + tril(D_ij q_i.k_j) W
//     S' = 2^G_C S + K^T (2^(G_C - G) W)
// (plain decay: W = beta V).  Everything is a product of 64- and 128-wide
// matrices, on the 16 x 16 x 32 bfloat16 matrix instructions.  T depends on
// the keys and gates only: k_prefill_prepare makes it for all chunks at once;
// k_prefill_chunks then walks a sequence chunk by chunk, a wave holding
// 16 NT columns of the state in its accumulators (columns of S, V, W and O
// go together and never meet others).
//
// Precision.  q, k and v are bfloat16, exact operands.  What is fp32 (S, T, W)
// enters a product as the sum of bfloat16 planes cut from its own mantissa:
// three planes of 8 bits are the fp32 value to the last bit, two are 16 bits
// of it.  Whatever feeds the state takes three planes (the state stays an
// fp32 computation over any length); what only reaches O, which is rounded to
// bfloat16, takes two.
//
// Operand order.  A 16 x 16 result holds rows 4 (lane / 16) + r of column
// lane % 16; an operand wants, per lane, 8 of 32 consecutive indexes of the
// summed axis.  Two results on top of each other are taken as that operand
// directly by counting the axis in the order the results hold it: slot (g, i)
// is index 4 g + i of the first for i < 4, of the second for i >= 4.  The
// other operand is stored in shared memory in the same order ("fragments" of
// 64 lanes x 16 bytes), so no product's result passes through memory.

constexpr int kC = 64, kD = 128;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// 2^x for a difference of running sums (held in double: at half-lives of a
// few tokens they reach hundreds, and their difference has to keep its last bits)
__device__ __forceinline__ float pow2(double x)
{
    x = x < -160.0 ? -160.0 : x;
    const double n = __builtin_rint(x);
    return __builtin_ldexpf(__builtin_amdgcn_exp2f((float)(x - n)), (int)n);
}

// One record of the workspace per (chunk, head).
struct Prep {
    double G[kC];
    float T[6][64][8];  // fragments of T's lower triangle, see frag_of
};

// Fragment f of a lower-triangular 64 x 64 operand: rows 16 mt .. + 15,
// columns 32 ks .. + 31.  The order spreads the work of making them over the waves.
__device__ __forceinline__ constexpr int frag_mt(int f) { return f == 0 || f == 1 ? 3 : f == 2 || f == 4 ? 2 : f == 3 ? 1 : 0; }
__device__ __forceinline__ constexpr int frag_ks(int f) { return f == 1 || f == 4 ? 1 : 0; }
__device__ __forceinline__ constexpr int frag_of(int mt, int ks)
{
    return mt == 3 ? ks : mt == 2 ? (ks ? 4 : 2) : mt == 1 ? 3 : 5;
}

// Chunk c of sequence s is record first / 64 + s + c: records of different
// sequences are disjoint, and none reaches n_tokens / 64 + n_seq + 1.
__host__ __device__ __forceinline__ int64_t prep_chunks(int32_t n_seq, int32_t n_tokens)
{
    return (int64_t)n_tokens / kC + n_seq + 1;
}

template <bool DELTA>
__global__ __launch_bounds__(256) void k_prefill_prepare(PrefillArgs a)
{
    constexpr int LD = kC + 1;
    __shared__ float M[DELTA ? kC * LD : 1], T[DELTA ? kC * LD : 1];
    __shared__ double G[kC];
    __shared__ float be[kC];
    const int t = threadIdx.x, lane = t & 63, wv = t >> 6, g = lane >> 4, c = lane & 15;
    const int h = (int)(blockIdx.x % (unsigned)a.heads);
    const int64_t rec = blockIdx.x / (unsigned)a.heads;

    // the sequence: the last s with cu[s] / 64 + s <= rec
    int lo = 0, hi = a.n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)(seq_of(a, mid).first / kC) + mid <= rec) lo = mid;
        else hi = mid;
    }
    const Seq sr = seq_of(a, lo);
    const int64_t t0 = sr.first + (rec - (sr.first / kC) - lo) * kC;
    if (t0 < sr.first || t0 >= sr.last) return;
    const int nt = sr.last - t0 < kC ? (int)(sr.last - t0) : kC;
    Prep &out = reinterpret_cast<Prep *>(a.ws)[rec * a.heads + h];

    if (wv == 0) {
        // running sums of log2 alpha; a gate of zero counts as 2^-2000
        const float al = lane < nt ? a.alpha[(t0 + lane) * a.heads + h] : 1.0f;
        double x = al > 0.0f ? log2((double)al) : -2000.0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double y = __shfl_up(x, d);
            if (lane >= d) x += y;
        }
        out.G[lane] = x;
        if (DELTA) {
            G[lane] = x;
            be[lane] = lane < nt ? a.beta[(t0 + lane) * a.heads + h] : 0.0f;
        }
    }
    if constexpr (!DELTA) return;
    // wave w: tiles (w, 0 .. w) of K K^T, straight from global memory
    const uint16_t *k = reinterpret_cast<const uint16_t *>(a.k) + t0 * a.k_stride + (int64_t)(h / a.per_k) * kD;
    bf16x8 ki[4];
#pragma unroll
    for (int s = 0; s < 4; s++) {
        const int row = 16 * wv + c;
        u32x4 x = {0, 0, 0, 0};
        if (row < nt) x = *reinterpret_cast<const u32x4 *>(k + row * a.k_stride + 32 * s + 8 * g);
        ki[s] = __builtin_bit_cast(bf16x8, x);
    }
    f32x4 kk[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        kk[j] = f32x4{0, 0, 0, 0};
        if (j > wv) continue;
#pragma unroll
        for (int s = 0; s < 4; s++) {
            const int row = 16 * j + c;
            u32x4 x = {0, 0, 0, 0};
            if (row < nt) x = *reinterpret_cast<const u32x4 *>(k + row * a.k_stride + 32 * s + 8 * g);
            kk[j] = mma(ki[s], __builtin_bit_cast(bf16x8, x), kk[j]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; j++) {
        if (j > wv) continue;
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const int i = 16 * wv + 4 * g + r, jj = 16 * j + c;
            M[i * LD + jj] = i > jj ? be[i] * pow2(G[i] - G[jj]) * kk[j][r] : 0.0f;
        }
    }
    __syncthreads();
    // wave w: inverse of its own 16 x 16 diagonal block, lane = column, by
    // forward substitution
    {
        float x[16];
        const int b = 16 * wv;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            float v = i == c ? 1.0f : 0.0f;
#pragma unroll
            for (int l = 0; l < i; l++) v = fmaf(-M[(b + i) * LD + b + l], x[l], v);
            x[i] = v;
        }
        if (g == 0) {
#pragma unroll
            for (int i = 0; i < 16; i++) T[(b + i) * LD + b + c] = x[i];
        }
    }
    __syncthreads();
    // the blocks below, one diagonal after the other:
    // T_ij = -T_ii sum_{l=j}^{i-1} M_il T_lj (fp32 matrix instructions)
#pragma unroll
    for (int d = 1; d < 4; d++) {
        if (wv < 4 - d) {
            const int j = wv, i = wv + d;
            f32x4 R = {0, 0, 0, 0}, X = {0, 0, 0, 0};
            for (int l = j; l < i; l++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    R = __builtin_amdgcn_mfma_f32_16x16x4f32(M[(16 * i + c) * LD + 16 * l + 4 * g + e],
                                                             T[(16 * l + 4 * g + e) * LD + 16 * j + c], R, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; e++)
                X = __builtin_amdgcn_mfma_f32_16x16x4f32(T[(16 * i + c) * LD + 16 * i + 4 * g + e], R[e], X, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; r++) T[(16 * i + 4 * g + r) * LD + 16 * j + c] = -X[r];
        }
        __syncthreads();
    }
    // fragments of T diag(beta)
    for (int f = wv; f < 6; f += 4) {
        const int mt = frag_mt(f), ks = frag_ks(f);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int row = 16 * mt + c, col = 32 * ks + (i >> 2) * 16 + 4 * g + (i & 3);
            v[i] = row >= col ? T[row * LD + col] * be[col] : 0.0f;
        }
        f32x4 *dst = reinterpret_cast<f32x4 *>(&out.T[f][lane][0]);
        dst[0] = f32x4{v[0], v[1], v[2], v[3]};
        dst[1] = f32x4{v[4], v[5], v[6], v[7]};
    }
}

// The first NP planes of 8 fp32 values (two results a, b) as operands.
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

constexpr int kFragBytes = 1024 + 16;  // 64 lanes x 16 bytes; the pad spreads transposed writes over the banks

struct SmemChunk {
    alignas(16) unsigned char K[16 * kFragBytes];      // [mt 4][ks 4]: rows tokens, axis d_k
    alignas(16) unsigned char Q[16 * kFragBytes];
    alignas(16) unsigned char KT[16 * kFragBytes];     // [mt 8][ks 2]: rows d_k, axis tokens
    alignas(16) unsigned char P[2][6 * kFragBytes];    // planes of tril(D q.k)
    alignas(16) float gam[kC], dec[kC];                // 2^G, 2^(G_C - G)
    alignas(16) double G[kC];
    alignas(16) float be[kC];
};
struct SmemChunkT : SmemChunk {
    alignas(16) unsigned char T[3][6 * kFragBytes];    // planes of T
};

__device__ __forceinline__ bf16x8 frag(const unsigned char *base, int f, int lane)
{
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(base + f * kFragBytes + lane * 16));
}

template <bool DELTA, int NT, int NW>
__global__ __launch_bounds__(64 * NW) void k_prefill_chunks(PrefillArgs a)
{
    constexpr int TH = 64 * NW, U = 256 / TH, COLS = 16 * NT * NW, NTV = 768 / TH;
    using SM = typename std::conditional<DELTA, SmemChunkT, SmemChunk>::type;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SM &sm = *reinterpret_cast<SM *>(smem_raw);

    const int t = threadIdx.x, lane = t & 63, wv = t >> 6, g = lane >> 4, c = lane & 15;
    const unsigned sh = blockIdx.x % (unsigned)(a.n_seq * a.heads);
    const int split = (int)(blockIdx.x / (unsigned)(a.n_seq * a.heads));
    const int h = (int)(sh % (unsigned)a.heads), s = (int)(sh / (unsigned)a.heads);
    const Seq sr = seq_of(a, s);
    const int col = split * COLS + wv * 16 * NT + NT * c;  // this lane's NT columns
    const int64_t tile = (int64_t)sh * kD * kD;

    // the state: rows 16 m + 4 g + r
    f32x4 S[8][NT];
#pragma unroll
    for (int m = 0; m < 8; m++)
#pragma unroll
        for (int r = 0; r < 4; r++)
#pragma unroll
            for (int n = 0; n < NT; n++)
                S[m][n][r] = a.S0 ? a.S0[tile + (int64_t)(16 * m + 4 * g + r) * kD + col + n] : 0.0f;

    const uint16_t *q = reinterpret_cast<const uint16_t *>(a.q) + (int64_t)(h / a.per_k) * kD;
    const uint16_t *k = reinterpret_cast<const uint16_t *>(a.k) + (int64_t)(h / a.per_k) * kD;
    const uint16_t *v = reinterpret_cast<const uint16_t *>(a.v) + (int64_t)h * kD + col;
    uint16_t *o = reinterpret_cast<uint16_t *>(a.o) + (int64_t)h * kD + col;
    const Prep *prep = reinterpret_cast<const Prep *>(a.ws);
    const int64_t rec0 = sr.first / kC + s, recs = prep_chunks(a.n_seq, a.n_tokens);

    // one chunk's inputs, loaded a chunk ahead: unit u of a thread is tokens
    // 4 tg .. + 3 and d = 8 dg .. + 7
    u32x4 kr[U][4], qr[U][4];
    f32x4 tr[DELTA ? NTV : 1];
    uint32_t vr[4][4];
    double Gr = 0.0, Gc = 0.0;
    float br = 0.0f;
    auto load = [&](int32_t t0) {
        const int nt = sr.last - t0 < kC ? sr.last - t0 : kC;
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int id = t + TH * u, dg = id & 15, tg = id >> 4;
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int64_t tok = t0 + 4 * tg + r;
                kr[u][r] = qr[u][r] = u32x4{0, 0, 0, 0};
                if (4 * tg + r < nt) {
                    kr[u][r] = *reinterpret_cast<const u32x4 *>(k + tok * a.k_stride + 8 * dg);
                    qr[u][r] = *reinterpret_cast<const u32x4 *>(q + tok * a.q_stride + 8 * dg);
                }
            }
        }
        int64_t rec = rec0 + (t0 - sr.first) / kC;
        rec = (rec < recs ? rec : recs - 1) * a.heads + h;
        if constexpr (DELTA) {
            const f32x4 *src = reinterpret_cast<const f32x4 *>(&prep[rec].T[0][0][0]);
#pragma unroll
            for (int i = 0; i < NTV; i++) tr[i] = src[t + TH * i];
        }
        if (t < kC) {
            Gr = prep[rec].G[t];
            Gc = prep[rec].G[kC - 1];
            br = t < nt ? a.beta[(int64_t)(t0 + t) * a.heads + h] : 0.0f;
        }
#pragma unroll
        for (int m = 0; m < 4; m++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int x = 16 * m + 4 * g + r;
                vr[m][r] = 0;
                if (x < nt) {
                    const uint16_t *p = v + (int64_t)(t0 + x) * a.v_stride;
                    if constexpr (NT == 2) vr[m][r] = *reinterpret_cast<const uint32_t *>(p);
                    else vr[m][r] = *p;
                }
            }
    };

    if (sr.first < sr.last) load(sr.first);
    for (int32_t t0 = sr.first; t0 < sr.last; t0 += kC) {
        // registers -> fragments in shared memory
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int id = t + TH * u, dg = id & 15, tg = id >> 4;
            const int ks = dg >> 2, half = (dg >> 1) & 1, g0 = (dg & 1) * 2;
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int x = 4 * tg + r;
                const int at = ((x >> 4) * 4 + ks) * kFragBytes + (g0 * 16 + (x & 15)) * 16 + half * 8;
                *reinterpret_cast<u32x2 *>(sm.K + at) = u32x2{kr[u][r][0], kr[u][r][1]};
                *reinterpret_cast<u32x2 *>(sm.K + at + 256) = u32x2{kr[u][r][2], kr[u][r][3]};
                *reinterpret_cast<u32x2 *>(sm.Q + at) = u32x2{qr[u][r][0], qr[u][r][1]};
                *reinterpret_cast<u32x2 *>(sm.Q + at + 256) = u32x2{qr[u][r][2], qr[u][r][3]};
            }
            const int tk = tg >> 3, tgg = tg & 3, th = (tg >> 2) & 1;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const int d = 8 * dg + e;
                const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
                const uint32_t lo = __builtin_amdgcn_perm(kr[u][1][e >> 1], kr[u][0][e >> 1], sel);
                const uint32_t hi = __builtin_amdgcn_perm(kr[u][3][e >> 1], kr[u][2][e >> 1], sel);
                *reinterpret_cast<u32x2 *>(sm.KT + ((d >> 4) * 2 + tk) * kFragBytes + (tgg * 16 + (d & 15)) * 16 +
                                           th * 8) = u32x2{lo, hi};
            }
        }
        if constexpr (DELTA) {
#pragma unroll
            for (int i = 0; i < NTV; i++) {
                // four values: half a lane's 16 bytes of each plane
                const int id = t + TH * i;
                float x[4] = {tr[i][0], tr[i][1], tr[i][2], tr[i][3]};
#pragma unroll
                for (int p = 0; p < 3; p++) {
                    u32x2 w;
                    w[0] = __builtin_amdgcn_perm(__float_as_uint(x[1]), __float_as_uint(x[0]), 0x07060302u);
                    w[1] = __builtin_amdgcn_perm(__float_as_uint(x[3]), __float_as_uint(x[2]), 0x07060302u);
                    *reinterpret_cast<u32x2 *>(sm.T[p] + (id >> 7) * kFragBytes + (id & 127) * 8) = w;
#pragma unroll
                    for (int e = 0; e < 4; e++) x[e] -= __uint_as_float(__float_as_uint(x[e]) & 0xffff0000u);
                }
            }
        }
        if (t < kC) {
            sm.G[t] = Gr;
            sm.gam[t] = pow2(Gr);
            sm.dec[t] = pow2(Gc - Gr);
            sm.be[t] = br;
        }
        f32x4 X[4][NT];  // V, then V - 2^G K S
#pragma unroll
        for (int m = 0; m < 4; m++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
                X[m][0][r] = __uint_as_float(vr[m][r] << 16);
                if constexpr (NT == 2) X[m][1][r] = __uint_as_float(vr[m][r] & 0xffff0000u);
            }
        __syncthreads();
        const int nt = sr.last - t0 < kC ? sr.last - t0 : kC;
        if (t0 + kC < sr.last) load(t0 + kC);

        // tril(D_ij q_i.k_j), two planes: the transposed products K Q^T leave
        // a lane one query's weights, which is the operand's order
        for (int f = wv; f < 6; f += NW) {
            const int mt = frag_mt(f), ks = frag_ks(f);
            f32x4 p[2];
            const double Gi = sm.G[16 * mt + c];
#pragma unroll
            for (int b = 0; b < 2; b++) {
                const int jt = 2 * ks + b;
                p[b] = f32x4{0, 0, 0, 0};
                if (jt > mt) continue;
#pragma unroll
                for (int x = 0; x < 4; x++) p[b] = mma(frag(sm.K, jt * 4 + x, lane), frag(sm.Q, mt * 4 + x, lane), p[b]);
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int j = 16 * jt + 4 * g + r;
                    p[b][r] = j <= 16 * mt + c ? p[b][r] * pow2(Gi - sm.G[j]) : 0.0f;
                }
            }
            bf16x8 pl[2];
            planes<2>(p[0], p[1], pl);
#pragma unroll
            for (int n = 0; n < 2; n++)
                *reinterpret_cast<u32x4 *>(sm.P[n] + f * kFragBytes + lane * 16) = __builtin_bit_cast(u32x4, pl[n]);
        }

        // K S and Q S
        f32x4 O[4][NT], KS[4][NT];
#pragma unroll
        for (int m = 0; m < 4; m++)
#pragma unroll
            for (int n = 0; n < NT; n++) O[m][n] = KS[m][n] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int x = 0; x < 4; x++) {
            bf16x8 sp[NT][3];
#pragma unroll
            for (int n = 0; n < NT; n++) planes<3>(S[2 * x][n], S[2 * x + 1][n], sp[n]);
#pragma unroll
            for (int m = 0; m < 4; m++) {
                const bf16x8 qf = frag(sm.Q, m * 4 + x, lane);
#pragma unroll
                for (int p = 0; p < 2; p++)
#pragma unroll
                    for (int n = 0; n < NT; n++) O[m][n] = mma(qf, sp[n][p], O[m][n]);
                if constexpr (DELTA) {
                    const bf16x8 kf = frag(sm.K, m * 4 + x, lane);
#pragma unroll
                    for (int p = 0; p < 3; p++)
#pragma unroll
                        for (int n = 0; n < NT; n++) KS[m][n] = mma(kf, sp[n][p], KS[m][n]);
                }
            }
        }
        // W
        f32x4 W[4][NT];
        if constexpr (DELTA) {
#pragma unroll
            for (int m = 0; m < 4; m++) {
                const f32x4 gm = *reinterpret_cast<const f32x4 *>(&sm.gam[16 * m + 4 * g]);
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    O[m][n] *= gm;
                    X[m][n] -= gm * KS[m][n];
                    W[m][n] = f32x4{0, 0, 0, 0};
                }
            }
#pragma unroll
            for (int ks = 0; ks < 2; ks++) {
                bf16x8 xp[NT][3];
#pragma unroll
                for (int n = 0; n < NT; n++) planes<3>(X[2 * ks][n], X[2 * ks + 1][n], xp[n]);
#pragma unroll
                for (int m = 2 * ks; m < 4; m++) {
                    const int f = frag_of(m, ks);
                    bf16x8 tf[3];
#pragma unroll
                    for (int p = 0; p < 3; p++) tf[p] = frag(sm.T[p], f, lane);
#pragma unroll
                    for (int p = 0; p < 3; p++)
#pragma unroll
                        for (int y = 0; y < 3 - p; y++)
#pragma unroll
                            for (int n = 0; n < NT; n++) W[m][n] = mma(tf[p], xp[n][y], W[m][n]);
                }
            }
        } else {
#pragma unroll
            for (int m = 0; m < 4; m++) {
                const f32x4 gm = *reinterpret_cast<const f32x4 *>(&sm.gam[16 * m + 4 * g]);
                const f32x4 bm = *reinterpret_cast<const f32x4 *>(&sm.be[16 * m + 4 * g]);
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    O[m][n] *= gm;
                    W[m][n] = X[m][n] * bm;
                }
            }
        }
        __syncthreads();  // P is whole
#pragma unroll
        for (int ks = 0; ks < 2; ks++) {
            bf16x8 wp[NT][2];
#pragma unroll
            for (int n = 0; n < NT; n++) planes<2>(W[2 * ks][n], W[2 * ks + 1][n], wp[n]);
#pragma unroll
            for (int m = 2 * ks; m < 4; m++) {
                const int f = frag_of(m, ks);
                const bf16x8 p0 = frag(sm.P[0], f, lane), p1 = frag(sm.P[1], f, lane);
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    O[m][n] = mma(p0, wp[n][0], O[m][n]);
                    O[m][n] = mma(p0, wp[n][1], O[m][n]);
                    O[m][n] = mma(p1, wp[n][0], O[m][n]);
                }
            }
        }
        // S' = 2^G_C S + K^T (2^(G_C - G) W)
        const float gC = sm.gam[kC - 1];
#pragma unroll
        for (int m = 0; m < 8; m++)
#pragma unroll
            for (int n = 0; n < NT; n++) S[m][n] *= gC;
#pragma unroll
        for (int ks = 0; ks < 2; ks++) {
            const f32x4 d0 = *reinterpret_cast<const f32x4 *>(&sm.dec[32 * ks + 4 * g]);
            const f32x4 d1 = *reinterpret_cast<const f32x4 *>(&sm.dec[32 * ks + 16 + 4 * g]);
            bf16x8 wp[NT][3];
#pragma unroll
            for (int n = 0; n < NT; n++) planes<3>(W[2 * ks][n] * d0, W[2 * ks + 1][n] * d1, wp[n]);
#pragma unroll
            for (int m = 0; m < 8; m++) {
                const bf16x8 kf = frag(sm.KT, m * 2 + ks, lane);
#pragma unroll
                for (int p = 0; p < 3; p++)
#pragma unroll
                    for (int n = 0; n < NT; n++) S[m][n] = mma(kf, wp[n][p], S[m][n]);
            }
        }
#pragma unroll
        for (int m = 0; m < 4; m++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int x = 16 * m + 4 * g + r;
                if (x >= nt) continue;
                uint16_t *p = o + (int64_t)(t0 + x) * a.heads * kD;
                if constexpr (NT == 2)
                    *reinterpret_cast<uint32_t *>(p) =
                        (uint32_t)down<uint16_t>(O[m][0][r]) | ((uint32_t)down<uint16_t>(O[m][1][r]) << 16);
                else
                    *p = down<uint16_t>(O[m][0][r]);
            }
        __syncthreads();
    }
    if (!a.S) return;
#pragma unroll
    for (int m = 0; m < 8; m++)
#pragma unroll
        for (int r = 0; r < 4; r++)
#pragma unroll
            for (int n = 0; n < NT; n++) a.S[tile + (int64_t)(16 * m + 4 * g + r) * kD + col + n] = S[m][n][r];
}

template <bool DELTA, int NT, int NW>
hipError_t chunks_t(const PrefillArgs &a, hipStream_t st)
{
    const unsigned grid = (unsigned)((int64_t)a.n_seq * a.heads * (kD / (16 * NT * NW)));
    const size_t lds = DELTA ? sizeof(SmemChunkT) : sizeof(SmemChunk);
    auto kern = k_prefill_chunks<DELTA, NT, NW>;
    if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds))
        return e;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(64 * NW), lds, st, a);
    return hipGetLastError();
}

template <bool DELTA>
hipError_t chunked(const PrefillArgs &a, hipStream_t st)
{
    const int64_t blocks = prep_chunks(a.n_seq, a.n_tokens) * a.heads;
    hipLaunchKernelGGL((k_prefill_prepare<DELTA>), dim3((unsigned)blocks), dim3(DELTA ? 256 : 64), 0, st, a);
    if (hipError_t e = hipGetLastError()) return e;
    const int64_t sh = (int64_t)a.n_seq * a.heads;
    if (sh >= 192) return chunks_t<DELTA, 2, 4>(a, st);
    return chunks_t<DELTA, 1, 2>(a, st);
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// bfloat16 tiles of 128 x 128 with rows that 16-byte loads can take
bool chunk_shape(int32_t dk, int32_t dv, bool bf16) { return bf16 && dk == kD && dv == kD; }

bool chunk_aligned(const PrefillArgs &a)
{
    return aligned16(a.q) && aligned16(a.k) && aligned16(a.v) && aligned16(a.o) && a.q_stride % 8 == 0 &&
           a.k_stride % 8 == 0 && a.v_stride % 8 == 0;
}

}  // namespace

uint64_t prefill_workspace(int32_t n_seq, int32_t n_tokens, int32_t heads, int32_t dk, int32_t dv, bool bf16,
                           bool)
{
    if (!chunk_shape(dk, dv, bf16)) return 0;
    return (uint64_t)prep_chunks(n_seq, n_tokens) * (uint64_t)heads * sizeof(Prep);
}

hipError_t launch_prefill(const PrefillArgs &a, bool bf16, bool delta, hipStream_t st)
{
    if (chunk_shape(a.dk, a.dv, bf16) && chunk_aligned(a)) return delta ? chunked<true>(a, st) : chunked<false>(a, st);
    if (bf16) return delta ? tokens_t<uint16_t, true>(a, st) : tokens_t<uint16_t, false>(a, st);
    return delta ? tokens_t<float, true>(a, st) : tokens_t<float, false>(a, st);
}

}  // namespace sqk
