// sq_prefill.hip -- gfx950 kernels of the prompt form of the recurrent
// layers: a whole sequence of tokens through
//     S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T   (delta)
//     S_t = alpha_t S_{t-1} + beta_t k_t v_t^T                          (plain decay)
//     o_t = S_t^T q_t
// from the state S_0 (or zero) to the state that the decode steps go on from.
#include <hip/hip_runtime.h>
#include <stdint.h>

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

}  // namespace

uint64_t prefill_workspace(int32_t, int32_t, int32_t, int32_t, int32_t, bool, bool) { return 0; }

hipError_t launch_prefill(const PrefillArgs &a, bool bf16, bool delta, hipStream_t st)
{
    if (bf16) return delta ? tokens_t<uint16_t, true>(a, st) : tokens_t<uint16_t, false>(a, st);
    return delta ? tokens_t<float, true>(a, st) : tokens_t<float, false>(a, st);
}

}  // namespace sqk
