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

// 16-token tiles per page, and its reciprocal: n / d = n * magic >> shift for
// n < 2^31.  magic = ceil(2^shift / d) with shift = 31 + ceil(log2 d) exceeds
// 2^shift / d by less than 1 <= 2^(shift - 31) / d, which adds less than 1 / d to
// the quotient.
struct PageTiles {
    uint32_t n, magic;
    int shift;
    explicit PageTiles(int64_t page_size) {
        n = (uint32_t)(page_size / 16);
        int s = 0;
        while (((uint64_t)1 << s) < n) s++;
        shift = 31 + s;
        magic = (uint32_t)((((uint64_t)1 << shift) + n - 1) / n);
    }
    PageTiles() = default;
#ifdef __HIP__
    __device__ __forceinline__ uint32_t page_of(uint32_t tile) const {
        return (uint32_t)((uint64_t)tile * magic >> shift);
    }
#endif
};

}  // namespace if4
