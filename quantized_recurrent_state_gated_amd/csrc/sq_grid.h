// sq_grid.h -- the launch limit that the serving operators' launchers check.
// Not installed, not part of the ABI.
#pragma once

#include <stdint.h>

namespace sqk {

// A launch has fewer than 2^32 threads.  (At most 2^40 workgroups are asked for.)
inline bool grid_fits(int64_t workgroups, int threads) { return workgroups * threads < ((int64_t)1 << 32); }

}  // namespace sqk
