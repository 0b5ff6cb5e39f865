// Launchers of the KV-cache translation units and what they share.  Not
// installed; callers use include/if4_kv.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/if4_kv.h"

namespace if4 {

hipError_t launch_kv_append(const if4_kv_cache& c, const void* k, const void* v, int bf16,
                            int64_t tokens, const int64_t (&strides)[4], const int64_t* slots,
                            int mode, hipStream_t stream);

hipError_t launch_kv_read(const if4_kv_cache& c, const int64_t* slots, int64_t tokens, void* k,
                          void* v, int bf16, hipStream_t stream);

hipError_t launch_kv_attention(const if4_kv_cache& c, const if4_kv_attention_args& a,
                               void* workspace, hipStream_t stream);

int64_t kv_attention_workspace(const if4_kv_cache& c, const if4_kv_attention_args& a);

}  // namespace if4
