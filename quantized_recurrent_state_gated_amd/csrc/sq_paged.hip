// sq_paged.hip -- gfx950 kernels of the paged key-value cache: the block
// tables and slot maps, the append of new keys and values, and the attention
// of one new token per request.
//
// The cache keeps keys as [page][head][token][d] and values transposed inside
// the page, [page][head][d][token].  Each is then the operand order of the
// matrix instructions that read it (a lane wants consecutive d of one key, and
// consecutive tokens of one value column), so attention feeds them from HBM
// with 16-byte loads and no pass through shared memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sq_grid.h"
#include "sq_paged.h"

namespace sqk {

namespace {

constexpr int64_t kInt32Max = 0x7fffffff;

// ---------------------------------------------------------------- block tables
//
// With c_i cached and m_i new tokens of request i and pages of P tokens:
//     held_i = ceil(c_i / P), need_i = ceil((c_i + m_i) / P) - held_i
//     N_i = sum_{j<i} m_j,    F_i = sum_{j<i} need_j
//     table[i][held_i + t] = free[F_i + t],  t < need_i
//     slot[N_i + t] = table[i][(c_i + t) / P] P + (c_i + t) mod P,  t < m_i
// A page of the new tokens is either held already (read from the table) or
// one of the fresh ones (read from the free list by its rank), so no thread
// reads a table entry that this launch writes, and one launch does it all.
// The prefix sums over the requests are cheap (8 bytes a request from L2), so
// up to kScanInBlock requests every workgroup computes them for itself in
// shared memory; above, one workgroup writes them first (they are outputs in
// any case) and a second launch reads them.  70 requests of one token take 3.7 us,
// 257 requests with 528 k new tokens 9 us (4.2 MB of slots): the launch and the
// chain of scan and search, not the bytes, set the time.

constexpr int kScanInBlock = 2048;
constexpr int kTokensPerBlock = 1024;

struct Need {
    int64_t ctx, fresh;  // clamped to >= 0
    int64_t held, need;
    bool bad;
};

__device__ __forceinline__ Need need_of(const TableArgs &a, int i)
{
    Need r;
    const int32_t c = a.ctx[i], m = a.fresh[i];
    r.bad = c < 0 || m < 0 || (int64_t)c + m > kInt32Max;
    r.ctx = r.bad ? 0 : c;
    r.fresh = r.bad ? 0 : m;
    const int64_t p = ((int64_t)1 << a.page_shift) - 1;
    r.held = (r.ctx + p) >> a.page_shift;
    r.need = ((r.ctx + r.fresh + p) >> a.page_shift) - r.held;
    return r;
}

__device__ __forceinline__ int32_t sat(int64_t x) { return (int32_t)(x > kInt32Max ? kInt32Max : x); }

// Exclusive prefix sums over the workgroup's TPB threads; the totals in `all`.
template <int TPB>
__device__ __forceinline__ void block_scan(int64_t &x, int64_t &y, int64_t (&all)[2], int64_t (*sm)[2])
{
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    int64_t a = x, b = y;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t ua = __shfl_up(a, d), ub = __shfl_up(b, d);
        if (lane >= d) {
            a += ua;
            b += ub;
        }
    }
    __syncthreads();  // sm may still be read from the scan before
    if (lane == 63) {
        sm[wv][0] = a;
        sm[wv][1] = b;
    }
    __syncthreads();
    int64_t ba = 0, bb = 0;
    all[0] = all[1] = 0;
#pragma unroll
    for (int w = 0; w < TPB / 64; w++) {
        if (w < wv) {
            ba += sm[w][0];
            bb += sm[w][1];
        }
        all[0] += sm[w][0];
        all[1] += sm[w][1];
    }
    x = ba + a - x;
    y = bb + b - y;
}

// Scan all requests into cn, cp (n + 1 entries each); `write` stores the
// outputs that are one per request as well.
template <int TPB>
__device__ void scan_requests(const TableArgs &a, int32_t *cn, int32_t *cp, bool write)
{
    __shared__ int64_t sm[TPB / 64][2];
    __shared__ int flags;
    if (threadIdx.x == 0) flags = 0;
    int64_t base_n = 0, base_p = 0;
    int bad = 0;
    for (int i0 = 0; i0 < a.n; i0 += TPB) {
        const int i = i0 + (int)threadIdx.x;
        Need r{};
        if (i < a.n) r = need_of(a, i);
        int64_t x = r.fresh, y = r.need, all[2];
        block_scan<TPB>(x, y, all, sm);
        if (i < a.n) {
            const int32_t en = sat(base_n + x), ep = sat(base_p + y);
            cn[i] = en;
            cp[i] = ep;
            if (write) {
                a.seq[i] = (int32_t)(r.ctx + r.fresh);
                if (a.cu_new != cn) a.cu_new[i] = en;
                if (a.cu_pages != cp) a.cu_pages[i] = ep;
                bad |= (r.bad ? 1 : 0) | (r.held + r.need > a.stride ? 4 : 0);
            }
        }
        base_n += all[0];
        base_p += all[1];
    }
    if (threadIdx.x == 0) {
        cn[a.n] = sat(base_n);
        cp[a.n] = sat(base_p);
        if (write) {
            a.cu_new[a.n] = sat(base_n);
            a.cu_pages[a.n] = sat(base_p);
            bad |= (base_p > a.n_free ? 2 : 0) | (base_n > a.capacity ? 8 : 0);
        }
    }
    if (write) {
        if (bad) atomicOr(&flags, bad);
        __syncthreads();
        if (threadIdx.x == 0) *a.result = flags;
    }
    __syncthreads();
}

// largest i < n with cu[i] <= x, for 0 <= x < cu[n]
__device__ __forceinline__ int find(const int32_t *cu, int n, int32_t x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ void fill_tables(const TableArgs &a, const int32_t *cn, const int32_t *cp)
{
    const int32_t tokens = cn[a.n], pages = cp[a.n];
    const int P = 1 << a.page_shift;
    // fresh pages into the rows; what a row has no room for (lengths past the table
    // may ask for 2^31 pages) is stepped over at once
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < pages; j += step) {
        const int i = find(cp, a.n, (int32_t)j);
        const Need r = need_of(a, i);
        const int64_t at = r.held + (j - cp[i]);
        if (at < a.stride) a.table[(int64_t)i * a.stride + at] = j < a.n_free ? a.free_pages[j] : -1;
        else j += (cp[i + 1] - 1 - j) / step * step;
    }
    // slots of the new tokens, and -1 after the last
    for (int64_t b = blockIdx.x; b * kTokensPerBlock < a.capacity; b += gridDim.x) {
        for (int u = 0; u < kTokensPerBlock / 256; u++) {
            const int64_t t = b * kTokensPerBlock + u * 256 + threadIdx.x;
            if (t >= a.capacity) break;
            int64_t slot = -1;
            if (t < tokens) {
                const int i = find(cn, a.n, (int32_t)t);
                const Need r = need_of(a, i);
                const int64_t pos = r.ctx + (t - cn[i]), pg = pos >> a.page_shift;
                int32_t id = -1;
                if (pg < r.held) {
                    if (pg < a.stride) id = a.table[(int64_t)i * a.stride + pg];
                } else {
                    const int64_t j = cp[i] + (pg - r.held);
                    if (pg < a.stride && j < a.n_free) id = a.free_pages[j];
                }
                if (id >= 0) slot = ((int64_t)id << a.page_shift) + (pos & (P - 1));
            }
            a.slots[t] = slot;
        }
    }
}

__global__ __launch_bounds__(256) void k_tables(TableArgs a)
{
    __shared__ int32_t cn[kScanInBlock + 1], cp[kScanInBlock + 1];
    scan_requests<256>(a, cn, cp, blockIdx.x == 0);
    fill_tables(a, cn, cp);
}

__global__ __launch_bounds__(1024) void k_tables_scan(TableArgs a)
{
    scan_requests<1024>(a, a.cu_new, a.cu_pages, true);
}

__global__ __launch_bounds__(256) void k_tables_fill(TableArgs a) { fill_tables(a, a.cu_new, a.cu_pages); }

}  // namespace

hipError_t launch_tables(const TableArgs &a, hipStream_t st)
{
    // the fill strides over whatever the grid does not cover at once
    const int64_t want = (a.capacity + kTokensPerBlock - 1) / kTokensPerBlock;
    const unsigned grid = (unsigned)(want < 1 ? 1 : want > 2048 ? 2048 : want);
    if (a.n <= kScanInBlock) {
        hipLaunchKernelGGL(k_tables, dim3(grid), dim3(256), 0, st, a);
    } else {
        hipLaunchKernelGGL(k_tables_scan, dim3(1), dim3(1024), 0, st, a);
        if (hipError_t e = hipGetLastError()) return e;
        hipLaunchKernelGGL(k_tables_fill, dim3(grid), dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------- append
//
// cache[slot_t] = (k_t, v_t) for one head and a tile of TT tokens a workgroup.
// Keys are copied row by row.  Values pass through shared memory: where TV
// tokens in a row fill a 16-byte piece of a page (consecutive slots from a
// multiple of TV), a lane writes that piece of its column at once; the other
// tokens are written element by element.  Slots outside the cache are skipped.
// Bound by HBM for prompts: four of 8,191 tokens x 8 heads, d = 128 in bfloat16 take
// 71 to 76 us (269 MB, 3.5 to 3.8 TB/s; 98 us when neighbouring lanes took
// neighbouring columns instead of neighbouring pieces); 70 single tokens take 3.9 us.

namespace {

template <typename T, int TT>
__global__ __launch_bounds__(256) void k_append(AppendArgs a)
{
    constexpr int TV = 16 / (int)sizeof(T);  // elements of 16 bytes
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int64_t slot[TT];
    __shared__ uint8_t single_at[TT], whole_at[TT];
    __shared__ int n_single, n_whole;
    static_assert(TT <= 64, "one wave sorts the tokens");
    const int d = a.c.d, heads = a.c.heads, P = 1 << a.c.page_shift;
    const int pitch = d + TV;     // rows stay 16-byte aligned
    T *vt = reinterpret_cast<T *>(smem);
    const int h = (int)(blockIdx.x % (unsigned)heads);
    const int64_t t0 = (int64_t)(blockIdx.x / (unsigned)heads) * TT;
    const int nt = (int)(a.n - t0 < TT ? a.n - t0 : TT);
    const int64_t limit = (int64_t)a.c.n_pages << a.c.page_shift;

    for (int t = threadIdx.x; t < TT; t += 256) {
        int64_t s = t < nt ? a.slots[t0 + t] : -1;
        if (s < 0 || s >= limit) s = -1;
        slot[t] = s;
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        const int t = threadIdx.x;
        const int64_t s = t < TT ? slot[t] : -1;
        int c = 0;  // 1: written by itself, 2: first token of a whole piece, 0: skipped, or in such a piece
        if (s >= 0) {
            const int e = (int)(s & (TV - 1));  // place in its piece, whose first token is t - e
            bool whole = t >= e && t - e + TV <= TT;
            for (int i = 0; i < TV && whole; i++) whole = slot[t - e + i] == s - e + i;
            c = !whole ? 1 : e == 0 ? 2 : 0;
        }
        const uint64_t m1 = __ballot(c == 1), m2 = __ballot(c == 2), below = (1ull << t) - 1;
        if (c == 1) single_at[__popcll(m1 & below)] = (uint8_t)t;
        if (c == 2) whole_at[__popcll(m2 & below)] = (uint8_t)t;
        if (t == 0) {
            n_single = __popcll(m1);
            n_whole = __popcll(m2);
        }
    }
    const int per = d / TV;  // 16-byte pieces of a row
    const T *ksrc = reinterpret_cast<const T *>(a.k), *vsrc = reinterpret_cast<const T *>(a.v);
    T *kc = reinterpret_cast<T *>(a.c.k), *vc = reinterpret_cast<T *>(a.c.v);
    for (int i = threadIdx.x; i < nt * per; i += 256) {
        const int t = i / per, x = (i - t * per) * TV;
        const uint4 vv = *reinterpret_cast<const uint4 *>(vsrc + (t0 + t) * a.v_stride + (int64_t)h * d + x);
        *reinterpret_cast<uint4 *>(vt + t * pitch + x) = vv;
        const int64_t s = slot[t];
        if (s < 0) continue;
        const uint4 kk = *reinterpret_cast<const uint4 *>(ksrc + (t0 + t) * a.k_stride + (int64_t)h * d + x);
        const int64_t row = ((s >> a.c.page_shift) * heads + h) * P + (s & (P - 1));
        *reinterpret_cast<uint4 *>(kc + row * d + x) = kk;
    }
    __syncthreads();
    // whole pieces: neighbouring lanes take neighbouring pieces of one column, so
    // that a tile's tokens leave as whole lines of the page
    for (int i = threadIdx.x; i < n_whole * d; i += 256) {
        const int x = i / n_whole, t = whole_at[i - x * n_whole];
        const int64_t s = slot[t];
        union {
            T e[TV];
            uint4 w;
        } u;
#pragma unroll
        for (int j = 0; j < TV; j++) u.e[j] = vt[(t + j) * pitch + x];
        *reinterpret_cast<uint4 *>(vc + (((s >> a.c.page_shift) * heads + h) * d + x) * P + (s & (P - 1))) = u.w;
    }
    for (int i = threadIdx.x; i < n_single * d; i += 256) {
        const int k = i / d, x = i - k * d, t = single_at[k];
        const int64_t s = slot[t];
        vc[(((s >> a.c.page_shift) * heads + h) * d + x) * P + (s & (P - 1))] = vt[t * pitch + x];
    }
}

template <typename T, int TT>
hipError_t append_t(const AppendArgs &a, hipStream_t st)
{
    const int64_t grid = ((int64_t)a.n + TT - 1) / TT * a.c.heads;
    if (!grid_fits(grid, 256)) return hipErrorInvalidConfiguration;
    const size_t lds = (size_t)TT * (size_t)(a.c.d + 16 / (int)sizeof(T)) * sizeof(T);
    hipLaunchKernelGGL((k_append<T, TT>), dim3((unsigned)grid), dim3(256), lds, st, a);
    return hipGetLastError();
}

template <typename T>
hipError_t append_any(const AppendArgs &a, hipStream_t st)
{
    // 64 tokens of bfloat16 fill the lines of a page's columns; few tokens: one
    // piece's worth per workgroup, for more workgroups.  Tokens x heads, us with
    // 8 tokens a workgroup against 64 (fp32: 32): 2,048 tokens x 2 heads 5.5 against 5.6
    // (5.4, 5.3), 512 x 8 5.0 against 5.5 (4.7, 5.2), 4,096 x 2 8.6 against 6.0 (7.8,
    // 6.1), 1,024 x 8 7.4 against 5.9 (6.7, 5.8), 64 x 8 3.2 against 5.3 (3.2, 4.6).
    if ((int64_t)a.n * a.c.heads >= 5120) return append_t<T, sizeof(T) == 2 ? 64 : 32>(a, st);
    return append_t<T, 8>(a, st);
}

}  // namespace

hipError_t launch_append(const AppendArgs &a, bool bf16, hipStream_t st)
{
    return bf16 ? append_any<uint16_t>(a, st) : append_any<float>(a, st);
}

// ---------------------------------------------------------------- decode attention
//
// o = sum_j softmax_j(scale q.k_j) v_j over a request's cached tokens.  Every
// key and value is used by the group of query heads that share its head and by
// nothing else: 4 group flops a byte pair, so the kernel is bound by HBM.
//
// A workgroup takes one (request, head, split of the context); its four waves
// take every fourth tile of keys.  Per tile, with the matrix instructions'
// 16 x 16 result held as rows 4 (lane / 16) + r, column lane % 16:
//     S^T = K Q^T   [keys x queries]   a lane holds keys of ONE query
//     O^T += V^T P^T [d x queries]     P^T wants, per lane, keys of one query
// so the probabilities go from the first product to the second in the lane's
// own registers.  The sixteen keys of a product's rows are chosen so that the
// orders agree: for bfloat16, row m of product t is key 8 (m / 4) + 4 t + m % 4
// of the 32, and lane group g then holds keys 8 g .. 8 g + 7.  The running
// maximum and sum are per query, that is per lane; the maximum joins the four
// lane groups with two exchanges per tile, the sum once at the end.
// The maximum starts at -inf and is at least the lowest float once a key is seen,
// so that it says by itself whether any was: a request without keys has a
// maximum of -inf (zeros, log sum -inf), one whose scores are all -inf a sum of
// zero under a finite maximum (NaN, like any score that is NaN or +inf).
// P is split into two bfloat16 (hi + lo): the second product costs nothing
// (the kernel waits for memory), and a single rounding would double the error
// that rounding the output makes anyway.
// 70 requests of up to 16 Ki tokens, 32 query and 8 key-value heads, d = 128 in
// bfloat16: 420 to 433 us, 5.6 to 5.8 TB/s of keys and values read once.

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

template <typename T>
struct Tile;

// 32 keys: two 16-row products, 8 elements a load
template <>
struct Tile<uint16_t> {
    static constexpr int KEYS = 32, SUB = 2, KSTEP = 32, EL = 8;
    using Reg = bf16x8;
};
// 16 keys: one product, 4 elements a load (four instructions of 4 each)
template <>
struct Tile<float> {
    static constexpr int KEYS = 16, SUB = 1, KSTEP = 16, EL = 4;
    using Reg = f32x4;
};

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(f32x4 a, f32x4 b, f32x4 c)
{
#pragma unroll
    for (int e = 0; e < 4; e++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

template <typename R, typename T>
__device__ __forceinline__ R load16(const T *p)
{
    return __builtin_bit_cast(R, *reinterpret_cast<const u32x4_t *>(p));
}

constexpr int kMaxChunk = 8192;  // tokens per split at most (page ids kept in shared memory)
constexpr int kPageIds = kMaxChunk / 16 + 2;

// How a request's context is cut: tokens [first, len), splits from `from`.
struct Span {
    int32_t len, first, from, splits;
};

__device__ __forceinline__ Span span_of(const AttendArgs &a, int r)
{
    Span s;
    int32_t len = a.lens[r];
    if (len > a.max_len) len = a.max_len;
    if (len < 0) len = 0;
    s.len = len;
    s.first = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
    s.from = s.first & ~31;  // tiles start on multiples of 32 tokens
    s.splits = (s.len - s.from + a.chunk - 1) / a.chunk;
    return s;
}

template <typename T>
__device__ __forceinline__ void store4(T *p, f32x4 x);
template <>
__device__ __forceinline__ void store4<float>(float *p, f32x4 x) { *reinterpret_cast<f32x4 *>(p) = x; }
template <>
__device__ __forceinline__ void store4<uint16_t>(uint16_t *p, f32x4 x)
{
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    const bf16x4 y = __builtin_convertvector(x, bf16x4);
    *reinterpret_cast<uint2 *>(p) = __builtin_bit_cast(uint2, y);
}

constexpr float kFloatMax = 3.402823466e+38f;

// 1 / L and log sum exp of a row with maximum M and sum L (base 2): no keys at
// all give 0 and -inf, a sum that is zero or NaN under keys gives NaN
__device__ __forceinline__ float inverse_sum(float M, float L)
{
    return M == -__builtin_inff() ? 0.0f : L > 0.0f ? 1.0f / L : __builtin_nanf("");
}
__device__ __forceinline__ float log_sum(float M, float L)
{
    if (M == -__builtin_inff()) return M;
    return L > 0.0f ? (M + __builtin_log2f(L)) * 0.69314718055994531f : __builtin_nanf("");
}

template <typename T, int D>
__global__ __launch_bounds__(256) void k_attend(AttendArgs a)
{
    using TL = Tile<T>;
    using R = typename TL::Reg;
    constexpr int NK = D / TL::KSTEP, ND = D / 16, KEYS = TL::KEYS, SUB = TL::SUB, EL = TL::EL;
    __shared__ int32_t ids[kPageIds];
    __shared__ int any_bad;
    __shared__ float sm_m[4][16], sm_l[4][16];
    __shared__ f32x4 sm_o[3][ND][64];

    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
    // Workgroups go to the eight XCDs in turn.  Splits are the slowest index: later
    // splits, which only long requests have, spread over all of them (as the
    // fastest of eight, each XCD had one split of every request, and the last ones
    // stood idle: 589 us against 431 at 70 requests x 8 heads up to 16 Ki tokens).
    const unsigned units = (unsigned)(a.n * a.c.heads);
    const unsigned unit = blockIdx.x % units, rest = blockIdx.x / units;
    const int r = (int)(unit / (unsigned)a.c.heads), h = (int)(unit % (unsigned)a.c.heads);
    const int qt = (int)(rest % (unsigned)a.q_tiles), sp = (int)(rest / (unsigned)a.q_tiles);

    // the queries, and without a window the split's first page ids, are asked for
    // together with the length: none of the three waits for another
    const int ps = a.c.page_shift, P = 1 << ps;
    const int qi = qt * 16 + c;  // this lane's query within the group
    const bool q_in = qi < a.group;
    const int64_t hq = (int64_t)h * a.group + qi;
    R qf[NK];
    {
        const T *qp = reinterpret_cast<const T *>(a.q) + (int64_t)r * a.q_stride + hq * D;
#pragma unroll
        for (int i = 0; i < NK; i++) {
            if (q_in) qf[i] = load16<R>(qp + i * TL::KSTEP + g * EL);
            else qf[i] = R{};
        }
    }
    const int32_t *pages_of = a.table + (int64_t)r * a.table_stride;
    const int64_t early_at = ((int64_t)sp * a.chunk >> ps) + threadIdx.x;
    int32_t early = 0;
    if (a.window == 0 && early_at << ps < a.max_len) early = pages_of[early_at];

    const Span s = span_of(a, r);
    const int32_t begin = s.from + sp * a.chunk;
    const int32_t end = begin + a.chunk < s.len ? begin + a.chunk : s.len;
    if (begin >= s.len && sp > 0) return;

    if (s.splits == 0) {  // no tokens: zeros, and the logarithm of an empty sum
        if (wv == 0 && q_in) {
            T *dst = reinterpret_cast<T *>(a.o) + ((int64_t)r * a.q_heads + hq) * D;
#pragma unroll
            for (int i = 0; i < ND; i++) store4<T>(dst + 16 * i + 4 * g, f32x4{0, 0, 0, 0});
            if (a.lse && g == 0) a.lse[(int64_t)r * a.q_heads + hq] = -__builtin_inff();
        }
        return;
    }

    // the split's page ids; an id outside the cache is kept as -1, its keys are masked
    const int32_t p0 = begin >> ps, np = ((end - 1) >> ps) - p0 + 1;
    if (threadIdx.x == 0) any_bad = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < np; i += 256) {
        int32_t id = a.window == 0 && i < 256 ? early : pages_of[p0 + i];
        if ((uint32_t)id >= (uint32_t)a.c.n_pages) {
            id = -1;
            any_bad = 1;
        }
        ids[i] = id;
    }

    __syncthreads();
    const bool bad = any_bad != 0;

    const T *kc = reinterpret_cast<const T *>(a.c.k), *vc = reinterpret_cast<const T *>(a.c.v);
    const int64_t page_el = (int64_t)a.c.heads << ps;  // rows of a page over all heads
    const int64_t head_row = (int64_t)h << ps;

    // this lane's key rows of tile t are base + kofs + 4 u (u < SUB), all in one page
    const int kofs = SUB == 2 ? 8 * (c >> 2) + (c & 3) : c;
    const int vofs = EL * g;

    auto page_of = [&](int32_t key) -> int32_t {
        const int32_t id = ids[((key < end ? key : end - 1) >> ps) - p0];
        return id < 0 ? 0 : id;  // masked below: any page will do
    };

    f32x4 acc[ND];
#pragma unroll
    for (int i = 0; i < ND; i++) acc[i] = f32x4{0, 0, 0, 0};
    float m = -__builtin_inff(), l = 0.0f;

    R kf[SUB][NK];
    auto load_k = [&](int32_t base) {
        const int32_t key = base + kofs;
        const T *kp = kc + ((int64_t)page_of(key) * page_el + head_row + (key & (P - 1))) * D + g * EL;
#pragma unroll
        for (int u = 0; u < SUB; u++)
#pragma unroll
            for (int i = 0; i < NK; i++) kf[u][i] = load16<R>(kp + u * 4 * D + i * TL::KSTEP);
    };

    int32_t base = begin + wv * KEYS;
    if (base < end) load_k(base);
    for (; base < end; base += 4 * KEYS) {
        R vf[ND];
        {
            const int32_t key = base + vofs;
            const T *vp = vc + ((int64_t)page_of(key) * page_el + head_row) * D + (key & (P - 1)) + (int64_t)c * P;
#pragma unroll
            for (int i = 0; i < ND; i++) vf[i] = load16<R>(vp + (int64_t)16 * i * P);
        }
        f32x4 x[SUB];
#pragma unroll
        for (int u = 0; u < SUB; u++) {
            x[u] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < NK; i++) x[u] = mma(kf[u][i], qf[i], x[u]);
        }
        if (base + 4 * KEYS < end) load_k(base + 4 * KEYS);

        // element (u, e) is key base + 8 g + 4 u + e (bfloat16) or base + 4 g + e
        float t[SUB * 4];
#pragma unroll
        for (int u = 0; u < SUB; u++)
#pragma unroll
            for (int e = 0; e < 4; e++) t[4 * u + e] = x[u][e] * a.scale_log2;
        const bool edge = base + KEYS > end || base < s.first || bad;
        uint32_t in = 0xffu;  // the keys that are there
        if (edge) {
            const int32_t key0 = base + vofs;
            const bool page_bad = bad && key0 < end && ids[(key0 >> ps) - p0] < 0;
            in = 0;
#pragma unroll
            for (int e = 0; e < SUB * 4; e++) {
                const bool ok = !page_bad && key0 + e < end && key0 + e >= s.first;
                in |= (ok ? 1u : 0u) << e;
                if (!ok) t[e] = -__builtin_inff();
            }
        }
        float mx = in ? -kFloatMax : -__builtin_inff();
#pragma unroll
        for (int e = 0; e < SUB * 4; e++) mx = fmaxf(mx, t[e]);
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        if (__ballot(mx > m)) {
            const float mn = fmaxf(m, mx);
            const float f = mn == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int i = 0; i < ND; i++) acc[i] *= f;
        }
        const float mu = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
        for (int e = 0; e < SUB * 4; e++) {
            t[e] = __builtin_amdgcn_exp2f(t[e] - mu);
            l += t[e];
        }
        if (edge) {
            // whatever lies in masked places (it may be NaN) must not meet a zero
#pragma unroll
            for (int i = 0; i < ND; i++)
#pragma unroll
                for (int e = 0; e < EL; e++)
                    if (!((in >> e) & 1)) vf[i][e] = R{}[e];
        }
        if constexpr (SUB == 2) {
            bf16x8 hi, lo;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                hi[e] = (__bf16)t[e];
                lo[e] = (__bf16)(t[e] - (float)hi[e]);
            }
#pragma unroll
            for (int i = 0; i < ND; i++) {
                acc[i] = mma(vf[i], hi, acc[i]);
                acc[i] = mma(vf[i], lo, acc[i]);
            }
        } else {
            const f32x4 p = {t[0], t[1], t[2], t[3]};
#pragma unroll
            for (int i = 0; i < ND; i++) acc[i] = mma(vf[i], p, acc[i]);
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
        L += mw == -__builtin_inff() ? 0.0f : sm_l[w][c] * __builtin_amdgcn_exp2f(mw - M);
    }
    const float f = m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m - M);
#pragma unroll
    for (int i = 0; i < ND; i++) acc[i] *= f;
    if (wv > 0) {
#pragma unroll
        for (int i = 0; i < ND; i++) sm_o[wv - 1][i][lane] = acc[i];
    }
    __syncthreads();
    if (wv > 0 || !q_in) return;
#pragma unroll
    for (int i = 0; i < ND; i++) acc[i] += sm_o[0][i][lane] + sm_o[1][i][lane] + sm_o[2][i][lane];
    const int64_t row = (int64_t)r * a.q_heads + hq;
    if (s.splits == 1) {
        const float inv = inverse_sum(M, L);
        T *dst = reinterpret_cast<T *>(a.o) + row * D;
#pragma unroll
        for (int i = 0; i < ND; i++) store4<T>(dst + 16 * i + 4 * g, acc[i] * inv);
        if (a.lse && g == 0) a.lse[row] = log_sum(M, L);
    } else {
        float *dst = a.part + (row * a.splits + sp) * D;
#pragma unroll
        for (int i = 0; i < ND; i++) *reinterpret_cast<f32x4 *>(dst + 16 * i + 4 * g) = acc[i];
        if (g == 0) {
            float *ml = a.part + (int64_t)a.n * a.q_heads * a.splits * D + (row * a.splits + sp) * 2;
            ml[0] = M;
            ml[1] = L;
        }
    }
}

// Join of the splits, a workgroup per (request, query head): the four waves take
// every fourth split, four of them in flight.
template <typename T, int D>
__global__ __launch_bounds__(256) void k_attend_join(AttendArgs a)
{
    constexpr int PER = (D + 63) / 64, IN = 4;
    __shared__ float sm_o[4][PER * 64], sm_l[4], sm_m[4];
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const Span s = span_of(a, (int)(row / a.q_heads));
    if (s.splits <= 1) return;  // written already
    const float *ml = a.part + (int64_t)a.n * a.q_heads * a.splits * D + row * a.splits * 2;
    float M = -__builtin_inff();
    for (int i = threadIdx.x; i < s.splits; i += 256) M = fmaxf(M, ml[2 * i]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) M = fmaxf(M, __shfl_xor(M, d));
    if (lane == 0) sm_m[wv] = M;
    __syncthreads();
    M = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
    float o[PER], L = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; j++) o[j] = 0.0f;
    const float *src = a.part + row * a.splits * D;
    for (int i0 = wv; i0 < s.splits; i0 += 4 * IN) {
        float m[IN], l[IN], x[IN][PER];
#pragma unroll
        for (int u = 0; u < IN; u++) {
            const int i = i0 + 4 * u;
            const bool in = i < s.splits;
            m[u] = in ? ml[2 * i] : -__builtin_inff();
            l[u] = in ? ml[2 * i + 1] : 0.0f;
#pragma unroll
            for (int j = 0; j < PER; j++) {
                const int d = j * 64 + lane;
                x[u][j] = in && d < D ? src[(int64_t)i * D + d] : 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < IN; u++) {
            const float f = m[u] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m[u] - M);
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
    T *dst = reinterpret_cast<T *>(a.o) + row * D;
    for (int d = threadIdx.x; d < D; d += 256) {
        const float y = (sm_o[0][d] + sm_o[1][d] + sm_o[2][d] + sm_o[3][d]) * inv;
        if constexpr (sizeof(T) == 4) dst[d] = y;
        else dst[d] = __builtin_bit_cast(uint16_t, (__bf16)y);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row] = log_sum(M, L);
}

template <typename T, int D>
hipError_t attend_td(const AttendArgs &a, hipStream_t st)
{
    const int64_t grid = (int64_t)a.n * a.c.heads * a.q_tiles * a.splits;
    const int64_t rows = (int64_t)a.n * a.q_heads;  // of the join
    if (!grid_fits(grid, 256) || (a.splits > 1 && !grid_fits(rows, 256))) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((k_attend<T, D>), dim3((unsigned)grid), dim3(256), 0, st, a);
    if (hipError_t e = hipGetLastError()) return e;
    if (a.splits > 1) hipLaunchKernelGGL((k_attend_join<T, D>), dim3((unsigned)rows), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <typename T>
hipError_t attend_t(const AttendArgs &a, hipStream_t st)
{
    switch (a.c.d) {
    case 32: return attend_td<T, 32>(a, st);
    case 64: return attend_td<T, 64>(a, st);
    case 96: return attend_td<T, 96>(a, st);
    case 128: return attend_td<T, 128>(a, st);
    case 192: return attend_td<T, 192>(a, st);
    case 256: return attend_td<T, 256>(a, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

bool attend_head_dim(int32_t d)
{
    return d == 32 || d == 64 || d == 96 || d == 128 || d == 192 || d == 256;
}

// Tokens per split.  Contexts of uneven length want many small workgroups to
// fill in behind each other (70 requests x 8 heads up to 16 Ki tokens: 430 us with
// 4096 workgroups, 445 with 1536, 478 with 1024), but every split pays for its
// start and its join: up to 2048 tokens a split, 512 workgroups do (one request,
// 8 heads x 100,000 tokens: 79 us with 512 workgroups, 84 with 1024, 103 with 4096; 128
// requests x 8 heads up to 1000 tokens: 59, 62, 69).  Below 256 tokens a split's
// start outweighs its work.
constexpr int64_t kMost = 4096, kFew = 512, kLongSplit = 2048, kMinChunk = 256;

uint64_t attend_rows_bound(int32_t n, int32_t kv_heads, int32_t q_heads, int32_t max_len)
{
    // splits <= (max_len + 31) / chunk + 1 with chunk >= max_len units / kMost,
    // kMinChunk <= chunk <= kMaxChunk; q_heads <= 16 x query tiles x kv_heads
    const uint64_t rows = (uint64_t)n * (uint64_t)q_heads;
    const uint64_t fine = ((uint64_t)max_len + 31 + kMinChunk - 1) / kMinChunk;
    const uint64_t coarse = ((uint64_t)max_len + 31 + kMaxChunk - 1) / kMaxChunk;
    const uint64_t group = (uint64_t)(q_heads / kv_heads), tile = group < 16 ? group : 16;
    const uint64_t a = rows * fine, b = kMost * tile + 2 * rows, c = rows * coarse;
    return a < (b > c ? b : c) ? a : (b > c ? b : c);
}

void attend_split(int32_t n, int32_t heads, int32_t q_tiles, int32_t max_len, int32_t *chunk,
                  int32_t *splits)
{
    const int64_t units = (int64_t)n * heads * q_tiles;
    const int64_t all = (int64_t)max_len * units;
    int64_t c = (all + kFew - 1) / kFew;
    if (c > kLongSplit) c = kLongSplit;
    if (c < (all + kMost - 1) / kMost) c = (all + kMost - 1) / kMost;
    if (c < kMinChunk) c = kMinChunk;
    c = (c + 127) / 128 * 128;  // whole rounds of four waves' tiles
    if (c > kMaxChunk) c = kMaxChunk;
    *chunk = (int32_t)c;
    // a window's first tile may start up to 31 tokens before it
    const int64_t s = ((int64_t)max_len + 31 + c - 1) / c;
    *splits = (int32_t)(s < 1 ? 1 : s);
}

hipError_t launch_attend(const AttendArgs &a, bool bf16, hipStream_t st)
{
    return bf16 ? attend_t<uint16_t>(a, st) : attend_t<float>(a, st);
}

}  // namespace sqk
