// Launchers of the FP8 translation units.  Not installed; callers use
// include/if4_fp8.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/if4_fp8.h"

namespace if4 {

hipError_t launch_fp8_quantize(const void* x, int bf16, int64_t rows, int64_t cols, int64_t ld_x,
                               int square, uint8_t* codes, uint8_t* scales, hipStream_t stream);

hipError_t launch_fp8_quantize_t(const void* x, int bf16, int64_t rows, int64_t cols,
                                 int64_t ld_x, int square, uint8_t* codes, uint8_t* scales,
                                 hipStream_t stream);

struct Fp8Gemm {
    const uint8_t *a_codes, *a_scales, *w_codes, *w_scales;
    int w_square;
    int64_t M, N, K;
    void* c;
    int c_bf16;
    int64_t ldc;
    void* workspace;
};

hipError_t launch_fp8_gemm(const Fp8Gemm& g, hipStream_t stream);
int64_t fp8_gemm_workspace(int64_t M, int64_t N, int64_t K);

}  // namespace if4
