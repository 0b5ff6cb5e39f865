// IF4 dequantize for gfx950.
//
// Each group's scale byte selects the decode: FP4 nibbles decode to
// (+-) E2M1 * s', INT4 nibbles to (+-) |q| * s' descaled by 6/7
// ("Adaptive Block-Scaled Data Types", gist.science summary, section 2,
// "Metodo 6/7"), then times 2^E.  The INT4 value is the fp32 nearest to
// 6 |q| s' / 7 (times 2^E, which is exact: every result is fp32-normal).
//
// One lane per group (8 code bytes + 1 scale byte in, 16 values out), one
// wave (64 groups) per workgroup.
// The decode itself is in if4_decode.h.
// bf16 output rounds each fp32 value to nearest even (v_cvt_pk_bf16_f32).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "if4_decode.h"
#include "if4_internal.h"
#include "xcd_order.h"

namespace if4 {
namespace {

constexpr int kThreads = 64;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <bool kBf16, bool kContig>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                  int64_t rows, int64_t gpr, void* __restrict__ y, int64_t ld_y, float p_exp) {
    const int64_t ngroups = rows * gpr;
    auto store = [&](int64_t g, const float* out) {
        int64_t off;
        if constexpr (kContig) {
            off = g * 16;
        } else {
            const int64_t r = g / gpr;
            off = r * ld_y + (g - r * gpr) * 16;
        }
        if constexpr (kBf16) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                bf16x2 v;
                v[0] = (__bf16)out[2 * i];
                v[1] = (__bf16)out[2 * i + 1];
                w[i] = __builtin_bit_cast(uint32_t, v);
            }
            uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(y) + off);
            p[0] = make_uint4(w[0], w[1], w[2], w[3]);
            p[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
            float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(y) + off);
#pragma unroll
            for (int i = 0; i < 4; i++)
                p[i] = make_float4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
        }
    };

    // One group per thread, one wave per workgroup: the thread's loads go
    // out first (past the end they re-read the last group, whose store is
    // then skipped, so no load sits behind a branch) and the scale byte's
    // decode constants are computed by the thread itself -- no LDS table, no
    // barrier (a per-workgroup table of 256 entries cost the same VALU work
    // plus a barrier, and 12% more time at 256 x 256).  (Grid-stride loops
    // over fewer workgroups, with the next group prefetched, measured up to
    // 33% slower on a 470 MB output: they keep far fewer loads in flight.)
    const int64_t gid = xcd_paired_block(blockIdx.x, gridDim.x) * kThreads + threadIdx.x;
    const int64_t g = gid < ngroups - 1 ? gid : ngroups - 1;
    const uint2 cw = *reinterpret_cast<const uint2*>(codes + g * 8);
    const uint32_t b = scales[g];
    const Entry e = make_entry(b, p_exp);
    float out[16];
    decode_word(cw.x, e, out);
    decode_word(cw.y, e, out + 8);
    if (gid < ngroups) store(gid, out);
}

template <bool kBf16>
void launch(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t gpr, void* y,
            int64_t ld_y, float p_exp, unsigned blocks, hipStream_t stream) {
    if (ld_y == gpr * 16)
        hipLaunchKernelGGL((dequantize_kernel<kBf16, true>), dim3(blocks), dim3(kThreads), 0,
                           stream, codes, scales, rows, gpr, y, ld_y, p_exp);
    else
        hipLaunchKernelGGL((dequantize_kernel<kBf16, false>), dim3(blocks), dim3(kThreads), 0,
                           stream, codes, scales, rows, gpr, y, ld_y, p_exp);
}

}  // namespace

hipError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                             int64_t cols, int32_t scale_exp, void* y, int bf16, int64_t ld_y,
                             hipStream_t stream) {
    const int64_t gpr = cols / 16;
    const int64_t ngroups = rows * gpr;
    const int64_t blocks = (ngroups + kThreads - 1) / kThreads;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (bf16)
        launch<true>(codes, scales, rows, gpr, y, ld_y, pow2f(scale_exp), (unsigned)blocks, stream);
    else
        launch<false>(codes, scales, rows, gpr, y, ld_y, pow2f(scale_exp), (unsigned)blocks, stream);
    return hipGetLastError();
}

}  // namespace if4
