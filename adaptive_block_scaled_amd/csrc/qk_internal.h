// Launchers of qk.hip.  Not installed; callers use include/if4_qk.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/if4_qk.h"

namespace if4 {

hipError_t launch_norm_rotate(const if4_qk_args& a, hipStream_t stream);
hipError_t launch_norm_rotate_backward(const if4_qk_args& a, void* workspace, hipStream_t stream);
int64_t norm_rotate_backward_workspace(const if4_qk_args& a);

}  // namespace if4
