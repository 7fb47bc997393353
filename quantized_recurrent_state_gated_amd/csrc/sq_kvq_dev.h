// sq_kvq_dev.h -- device helpers that the kernels of the 8-bit cache share.
// Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sq_kvq.h"

namespace sqk {

// How many of 0 .. n - 1 satisfy `pred`, where those that do come first: the 64
// lanes of a wave probe 64 places at a time.  Called by whole waves; ends for
// any `pred` (a round leaves less than a 64th of the range).
template <typename F>
__device__ __forceinline__ int wave_count(int n, F pred)
{
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = n;
    while (lo < hi) {
        const int step = (int)(((int64_t)hi - lo + 63) >> 6);
        const int64_t at = lo + (int64_t)lane * step;
        const int t = __popcll(__ballot(at < hi && pred((int)at)));
        if (t == 0) return lo;
        const int64_t next = lo + (int64_t)t * step;
        lo = lo + (t - 1) * step + 1;
        hi = next < hi ? (int)next : hi;
    }
    return lo;
}

__device__ __forceinline__ int32_t clamp_to(int32_t x, int32_t n) { return x < 0 ? 0 : x > n ? n : x; }

__device__ __forceinline__ float bits_f(uint32_t x) { return __builtin_bit_cast(float, x); }
__device__ __forceinline__ uint32_t f_bits(float x) { return __builtin_bit_cast(uint32_t, x); }

}  // namespace sqk
