// sq_kvq_tiles.hip -- gfx950 kernel of attention over the 8-bit paged cache, many
// queries a request; sq_kvq_attend.h has how codes and scales are multiplied.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sq_grid.h"
#include "sq_kvq.h"
#include "sq_kvq_attend.h"

namespace sqk {

namespace {

using namespace kvq;

// Rows (queries x heads of a group) in tiles of 256 or 128, 32 a wave; tokens 64 at a
// time.  A key is used by all rows of a tile, so the matrix instructions and the
// weights between them bound it, and the codes become float16 once a workgroup, on
// their way into shared memory.  With the 32 x 32 result of an instruction held as rows
// 8 (e / 4) + 4 (lane / 32) + e % 4, column lane % 32:
//     S^T = K Q^T    [64 tokens x 32 rows]
//     O^T += V^T P^T [d x 32 rows]         a step is a block of 16 tokens
// Row m = 8 j + 4 i + e of a product is token 16 (j / 2) + 8 i + 4 (j % 2) + e of 32, so a
// lane's 8 scores of a block are the second product's operand in its own registers.
//
// What bounds it: a wave's tile is 32 products of 32 cycles, and 32 exponentials of 16
// cycles and some 180 other vector instructions a lane.  A product takes about 16 of its
// cycles from the other wave's vector instructions on the SIMD (measured), so turns of
// products beside turns of weights cannot do with less than about 1,800 cycles
// for two waves' halves; they take 2,400.  One causal prompt of 8,192 tokens, 32 query and 8
// key-value heads, d = 128 in integer codes: 590 to 615 us, 895 to 930 TFLOP/s, with other
// work or pauses between; 20 of them back to back 660 to 780, 704 on average, 780 TFLOP/s (a float16
// library product of 8192^3, back to back, reaches 1,092).  On the way: 1,046 us with one
// wave a SIMD, 660 with two that are not kept apart, 820 with turns but page ids waited for
// one by one, 631 with the maximum looked for in every tile.

template <typename T, bool E4M3, int D, int ROWS>
__global__ __launch_bounds__(2 * ROWS, two_a_simd(sizeof(T) == 2, D) ? 2 : 1) void k_kvq_tiles(KvqAttendArgs a)
{
    constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
    constexpr int WAVES = ROWS / 32, TPB = 64 * WAVES;
    constexpr int NS = D / 16, ND = D / 32;
    constexpr int KP = D + 8, VP = 64 + 8;     // halves from row to row: 16 bytes off a multiple of the banks
    constexpr int PIECES = 4 * D, NP = (PIECES + TPB - 1) / TPB;  // 16-byte pieces of 64 tokens
    __shared__ __align__(16) _Float16 sm_k[2][64 * KP], sm_v[2][D * VP];
    __shared__ f32x4 sm_s[4][4];               // of the four blocks: key scales; value scales, their log2 and inverse

    const int lane = threadIdx.x & 63, hh = lane >> 5, c = lane & 31;
    const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int grp = WAVES == 8 ? wv >> 2 : 0;                       // which half of the waves: the two take turns
    const int part = WAVES == 8 ? (wv & 3) * 2 + grp : wv;          // which 32 rows: few rows spread over both halves
    // A slot's splits lie side by side: slots that no tile takes come last.  (Between the
    // others they leave half of the card's engines without work, as workgroups go to these
    // in turn: 64 tokens behind 30,000, one slot of two taken: 96 us, 57 so.)
    const unsigned heads = (unsigned)a.c.heads, splits = (unsigned)a.t_splits;
    const int h = (int)(blockIdx.x % heads);
    const int sp = (int)(blockIdx.x / heads % splits);
    const int slot = (int)(blockIdx.x / heads / splits);

    // The slot's request and tile: longest requests first, so that short ones fill in
    // behind them (up to 64 requests; more go in their order), and of a request the late
    // tiles, which see the most.  (Six ragged
    // pieces of 1,024 tokens at most behind up to 6,000: 345 us as they come, 310 so.)
    int r;
    int64_t tile;
    if (a.n <= 64) {
        int32_t len = -1, count = 0;
        if (lane < a.n) {
            const Req q = req_of(a, lane);
            len = q.len;
            count = q.m < 1 || few(a, q.m) ? 0 : (int32_t)(((int64_t)q.m * a.group + ROWS - 1) / ROWS);
        }
        int32_t first = 0;
        for (int i = 0; i < a.n; i++) {
            const int32_t l = __builtin_amdgcn_readlane(len, i), k = __builtin_amdgcn_readlane(count, i);
            if (l > len || (l == len && i < lane)) first += k;
        }
        const uint64_t mine = __ballot(slot >= first && slot - first < count);
        if (!mine) return;
        r = __builtin_ctzll(mine);
        tile = __builtin_amdgcn_readlane(count, r) - 1 - (slot - __builtin_amdgcn_readlane(first, r));
    } else {
        const int back = a.tiles - 1 - slot;
        r = wave_count(a.n, [&](int i) { return (int64_t)clamp_to(a.cu[i], a.n_q) * a.group / ROWS + i <= back; }) - 1;
        if (r < 0) return;
        tile = back - ((int64_t)clamp_to(a.cu[r], a.n_q) * a.group / ROWS + r);
        if (tile < 0) return;  // where offsets fall
    }
    const Req q = req_of(a, r);
    if (q.m < 1 || few(a, q.m)) return;
    const int64_t rows = (int64_t)q.m * a.group, row0 = tile * ROWS;
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
        f32x2 sc = {1.0f, 1.0f};
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
        // weights are made with their value scale in the exponent: it has a logarithm
        const float v = fmaxf(sc[1], 0x1p-100f);
        float *to = reinterpret_cast<float *>(sm_s[ring]) + lane;
        to[0] = sc[0], to[4] = v;
        if constexpr (PARTS == 1) to[8] = __builtin_amdgcn_logf(v), to[12] = 1.0f / v;
    };

    f32x16 acc[ND], x[2];
#pragma unroll
    for (int i = 0; i < ND; i++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[i][e] = 0.0f;
    h8 p[4][PARTS];
    float m = -kInf, l = 0.0f;
    // the row's largest weight, times 2^m; what makes weights of probabilities, as a logarithm less m (where two float16
    // stand for a weight: as a factor); the least logarithm of a value scale that `weigh` is right for
    float ref = 0.0f, up = 0.0f, low = kInf;

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
        // four operands ahead of the products
        __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
        for (int i = 0; i < 2 * NS - 4; i++) {
            __builtin_amdgcn_sched_group_barrier(0x8, PARTS, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, PARTS * 4, 0);
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
        __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
        for (int i = 0; i < 4 * ND - 4; i++) {
            __builtin_amdgcn_sched_group_barrier(0x8, PARTS, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, PARTS * 4, 0);
    };
    // keeps a factor from the products made with it so far, which the compiler would hold on to for a
    // second pass over the scores, in registers that it has not got
    auto apart = [](float &f) { asm volatile("" : "+v"(f)); };
    // Weights p of a tile and the sum of its probabilities, by maximum and reference as they
    // stand; whether they could stand.
    auto weigh = [&](const f32x4 (&sc)[4], const float (&fk)[4], float &sum) {
        float most = 0.0f, least = PARTS == 1 ? sc[2][0] : 0.0f;
        sum = 0.0f;
#pragma unroll
        for (int b = 0; b < 4; b++) {
            // One float16: 2^(score - m) times the value scale over the reference in one exponential; the
            // sum takes the scale out again.  A scale 2^-60 under the reference could lose
            // probabilities so, and scores past 2^10 the exponent's last bits: `low` says so.
            const float c0 = PARTS == 1 ? sc[2][b] + up : -m;
            f32x8 t;
#pragma unroll
            for (int e = 0; e < 8; e++) t[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[b >> 1][8 * (b & 1) + e], fk[b], c0));
            const float s8 = ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
            if constexpr (PARTS == 1) {
                sum = __builtin_fmaf(s8, sc[3][b], sum);
                most += s8;
                least = fminf(least, sc[2][b]);
            } else {
                const float g = factor_of(sc[1][b], up);
                sum += s8;
                most = __builtin_fmaf(s8, g, most);
                t *= g;
            }
            split8<PARTS>(t, p[b]);
        }
        if constexpr (PARTS == 1) sum *= ref * kProbDown;
        return sum <= kGrown && most <= kMostWeight && least >= low;
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
        float sum;
        const bool grown = !weigh(sc, fk, sum);
        // Probabilities that pass 2^kGrown or weights that pass float16 (their sums say so at
        // the latest), the first tile of a row, scales or scores too far apart: maximum and
        // reference are found and the weights made again, probabilities first.  Few tiles do.
        if (__ballot(grown)) {
            // of the rows that need it alone: what another one holds must not show in a row's bits
            const int other = __shfl_xor((int)grown, 32);
            const bool need = grown || other;
            float mb[4], mx = in ? -kFloatMax : -kInf;
#pragma unroll
            for (int b = 0; b < 4; b++) {
                apart(fk[b]);
                mb[b] = -kInf;
#pragma unroll
                for (int e = 0; e < 8; e++) mb[b] = fmaxf(mb[b], rounded(x[b >> 1][8 * (b & 1) + e], fk[b]));
                mx = fmaxf(mx, mb[b]);
            }
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            const float mn = fmaxf(m, mx), mu = mn == -kInf ? 0.0f : mn;
            float top = 0.0f;
#pragma unroll
            for (int b = 0; b < 4; b++) top = fmaxf(top, top_weight(mb[b], mu, sc[1][b]));
            top = fmaxf(top, __shfl_xor(top, 32));
            float fv = 1.0f;
            if (need) {
                const float f = mn == -kInf ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
                const float r2 = fmaxf(fmaxf(ref * f, top), kLeastRef);
                fv = f * (ref / r2);
                m = mn;
                l *= f;
                ref = r2;
                up = kProbUp / r2;
                const bool near = __builtin_fabsf(m) <= 1024.0f;
                if constexpr (PARTS == 1) {
                    const float up_log = __builtin_log2f(up);
                    low = near ? -55.0f - up_log : kInf;
                    up = up_log - m;
                } else {
                    low = near ? 0.0f : kInf;
                }
            }
#pragma unroll
            for (int i = 0; i < ND; i++) acc[i] *= fv;
            // what `weigh` makes of the other rows, and of these probabilities first, which are 1 at
            // most: differences to the maximum are exact enough at any size of the scores
            const float factor = kProbUp / ref;
            sum = 0.0f;
#pragma unroll
            for (int b = 0; b < 4; b++) {
                apart(fk[b]);
                const float c0 = PARTS == 1 ? sc[2][b] + up : -m;
                f32x8 t;
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const float s1 = x[b >> 1][8 * (b & 1) + e];
                    t[e] = __builtin_amdgcn_exp2f(need ? rounded(s1, fk[b]) - mu : __builtin_fmaf(s1, fk[b], c0));
                }
                const float s8 = ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
                if constexpr (PARTS == 1) {
                    sum = __builtin_fmaf(s8, need ? 1.0f : sc[3][b], sum);
                    t *= need ? factor_of(sc[1][b], factor) : 1.0f;
                } else {
                    sum += s8;
                    t *= factor_of(sc[1][b], up);
                }
                split8<PARTS>(t, p[b]);
            }
            if (PARTS == 1 && !need) sum *= ref * kProbDown;
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
        const float inv = inverse_sum(m, l) * (ref * kProbDown);
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
                store4(dst + 32 * i + 8 * j, f32x4{acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]} * (ref * kProbDown));
        if (hh == 0) {
            float *ml = part_o + (int64_t)a.n_q * a.q_heads * a.t_splits * D + at * 2;
            ml[0] = m;
            ml[1] = l;
        }
    }
}

template <typename T, bool E4M3, int D>
hipError_t tiles_tfd(const KvqAttendArgs &a, hipStream_t st)
{
    const unsigned grid = (unsigned)((int64_t)a.tiles * a.c.heads * a.t_splits);
    if constexpr (tiles_of_256(sizeof(T) == 2, D)) {
        if (a.tile_rows == 256) {
            hipLaunchKernelGGL((k_kvq_tiles<T, E4M3, D, 256>), dim3(grid), dim3(512), 0, st, a);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((k_kvq_tiles<T, E4M3, D, 128>), dim3(grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <typename T, bool E4M3>
hipError_t tiles_tf(const KvqAttendArgs &a, hipStream_t st)
{
    switch (a.c.d) {
    case 32: return tiles_tfd<T, E4M3, 32>(a, st);
    case 64: return tiles_tfd<T, E4M3, 64>(a, st);
    case 96: return tiles_tfd<T, E4M3, 96>(a, st);
    case 128: return tiles_tfd<T, E4M3, 128>(a, st);
    case 192: return tiles_tfd<T, E4M3, 192>(a, st);
    case 256: return tiles_tfd<T, E4M3, 256>(a, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_kvq_tiles(const KvqAttendArgs &a, bool bf16, hipStream_t st)
{
    if (bf16) return a.c.e4m3 ? tiles_tf<uint16_t, true>(a, st) : tiles_tf<uint16_t, false>(a, st);
    return a.c.e4m3 ? tiles_tf<float, true>(a, st) : tiles_tf<float, false>(a, st);
}

}  // namespace sqk
