// Compares what sq_kvq_attention needs of its workspace with what sq_kvq_attention_workspace
// says for sizes at least as large, over random sizes.  Host code only.
//     kvq_plan_fuzz seed count
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <random>

#include "../quantized_recurrent_state_gated_amd/csrc/sq_kvq.h"

using namespace sqk;

int main(int argc, char **argv)
{
    std::mt19937_64 rng(argc > 1 ? atoll(argv[1]) : 1);
    const long count = argc > 2 ? atol(argv[2]) : 100000;
    auto upto = [&](int64_t top) {  // 1 .. top, their logarithms even
        const double x = std::uniform_real_distribution<double>(0.0, log((double)top + 0.5))(rng);
        return std::min<int64_t>(top, std::max<int64_t>(1, (int64_t)exp(x)));
    };
    const int widths[] = {32, 64, 96, 128, 192, 256};
    double most = 0.0;
    long some = 0;
    for (long i = 0; i < count; i++) {
        const int64_t kv = upto(64), group = upto(64), heads = kv * group, top = std::min<int64_t>((1 << 30) / heads, 1 << 22);
        const int64_t n = upto(top), n_q = rng() % 4 ? upto(top) : n, len = rng() % 8 ? upto(1 << 20) : upto(1 << 30);
        const int d = widths[rng() % 6];
        const uint64_t bound = kvq_plan_bound((int32_t)n, (int32_t)n_q, (int32_t)kv, (int32_t)heads, d, (int32_t)len);
        // that call itself, or one of fewer requests, queries and tokens
        const bool same = rng() % 2;
        const int32_t dummy = 0;
        KvqAttendArgs a{};
        a.c.heads = (int32_t)kv;
        a.c.d = d;
        a.n = (int32_t)(same ? n : upto(n));
        a.n_q = (int32_t)(same ? n_q : upto(n_q));
        a.cu = a.n == a.n_q && rng() % 2 ? nullptr : &dummy;
        a.q_heads = (int32_t)heads;
        a.group = (int32_t)group;
        a.max_len = (int32_t)(same ? len : rng() % 16 ? upto(len) : 0);
        a.window = rng() % 2 ? 0 : (int32_t)upto(1 << 30);
        const bool bf16 = rng() % 2;
        const uint64_t need = kvq_plan(a, bf16);
        some += need > 0;
        most = std::max(most, bound ? (double)need / (double)bound : need ? 1e9 : 0.0);
        // what the kernels index by
        const bool fits = a.splits >= 1 && a.t_splits >= 1 && a.chunk % 256 == 0 && a.chunk <= 8192 && a.t_chunk % 64 == 0 &&
                          (int64_t)a.t_splits * a.t_chunk < (int64_t(1) << 31) && (int64_t)a.splits * a.chunk < (int64_t(1) << 31);
        // a window's rows (of at most 16, of a tile) may see splits x chunk tokens, from a multiple of 64
        auto spans = [&](int64_t apart) {
            return a.window > 0 && a.window < a.max_len ? std::min<int64_t>(a.max_len, (int64_t)a.window + apart + 63) : a.max_len;
        };
        const bool reach = (!a.few_on || (int64_t)a.splits * a.chunk >= spans(15)) &&
                           (!a.tiles || (int64_t)a.t_splits * a.t_chunk >= spans(a.tile_rows - 1));
        if (need > bound || !fits || !reach) {
            printf("n %d n_q %d kv %lld group %lld d %d len %d window %d cu %d bf16 %d: need %llu of %llu, %d %d\n", a.n, a.n_q,
                   (long long)kv, (long long)group, d, a.max_len, a.window, a.cu != nullptr, bf16, (unsigned long long)need,
                   (unsigned long long)bound, fits, reach);
            return 1;
        }
    }
    printf("%ld calls, %ld with a workspace, at most %.4f of it used\n", count, some, most);
    return 0;
}
