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
int64_t kv_attention_workspace_most(const if4_kv_cache& c, const if4_kv_attention_args& a);

// A divisor fixed for a call: m / n = m * magic >> shift for m < 2^31.  magic =
// ceil(2^shift / n) with shift = 31 + ceil(log2 n) exceeds 2^shift / n by less than
// 1 <= 2^(shift - 31) / n, which adds less than 1 / n to the quotient.
struct Divisor {
    uint32_t n, magic;
    int shift;
    Divisor() = default;
    explicit Divisor(int64_t by) {
        n = (uint32_t)by;
        int s = 0;
        while (((uint64_t)1 << s) < n) s++;
        shift = 31 + s;
        magic = (uint32_t)((((uint64_t)1 << shift) + n - 1) / n);
    }
#ifdef __HIP__
    __device__ __forceinline__ uint32_t into(uint32_t m) const {
        return (uint32_t)((uint64_t)m * magic >> shift);
    }
#endif
};

}  // namespace if4
