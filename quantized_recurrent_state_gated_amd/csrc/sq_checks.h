// sq_checks.h -- argument checks that the host side of the serving operators
// shares (sq_serve_api.hip, sq_kvq_api.hip).  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/sq.h"

namespace sqk {

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// log2 of a page size in [16, 256], or -1
inline int page_shift(int32_t page)
{
    for (int s = 4; s <= 8; s++)
        if (page == 1 << s) return s;
    return -1;
}

inline int elem_bytes(int32_t dtype) { return dtype == SQ_BF16 ? 2 : 4; }

// a token stride: at least a token's elements, and rows that stay 16-byte aligned
inline bool stride_ok(int64_t stride, int64_t row, int32_t dtype)
{
    return stride >= row && stride * elem_bytes(dtype) % 16 == 0;
}

// the launchers refuse a grid that does not fit one launch before they make any HIP call
inline int status(hipError_t e)
{
    return e == hipSuccess ? SQ_OK : e == hipErrorInvalidConfiguration ? SQ_ERR_UNSUPPORTED : SQ_ERR_HIP;
}

constexpr int64_t kMaxGrid = 0x7fffffff;
constexpr int32_t kMaxReach = 1 << 30;

}  // namespace sqk
