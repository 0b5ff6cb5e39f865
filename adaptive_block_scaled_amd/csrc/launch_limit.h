// How many workgroups one launch may have.  HIP counts the threads along a grid's dimension
// in 32 bits and launches what is left of a larger number, without an error: 2^32 + 512
// threads are 512.  So launchers look before, and answer hipErrorInvalidConfiguration, which
// callers of the C ABI get as IF4_ERR_SHAPE.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace if4 {

constexpr int64_t most_groups(int64_t threads) { return 0xFFFFFFFFll / threads; }

inline bool launchable(int64_t groups, int64_t threads) { return groups <= most_groups(threads); }

}  // namespace if4
