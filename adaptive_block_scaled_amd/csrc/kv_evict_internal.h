// Launchers of kv_evict.hip.  Not installed; callers use include/if4_kv_evict.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/if4_kv_evict.h"

namespace if4 {

hipError_t launch_kv_weights(const if4_kv_cache& c, const if4_kv_attention_args& a,
                             const if4_kv_mass& m, void* workspace, hipStream_t stream);
int64_t kv_weights_workspace(const if4_kv_cache& c, const if4_kv_attention_args& a);
int64_t kv_weights_workspace_most(const if4_kv_cache& c, const if4_kv_attention_args& a);

hipError_t launch_kv_select(const if4_kv_mass& m, const int32_t* seq_lens, int64_t batch,
                            int64_t kv_heads, int64_t keep, int64_t recent, int64_t sinks,
                            int32_t* kept, void* workspace, hipStream_t stream);
int64_t kv_select_workspace(const if4_kv_mass& m, int64_t batch, int64_t kv_heads, int64_t keep);

hipError_t launch_kv_compact(const if4_kv_cache& c, const int32_t* page_table,
                             int64_t table_stride, const int32_t* kept, int64_t batch,
                             int64_t keep, const int32_t* new_table, int64_t new_stride,
                             hipStream_t stream);

}  // namespace if4
