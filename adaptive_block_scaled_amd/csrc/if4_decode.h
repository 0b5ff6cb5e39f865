// Device helpers that decode IF4 groups to fp32 in a lane's registers (HIP
// translation units only).
//
// The decode is branch-free and identical for both formats:
//  * each nibble becomes an E4M3 byte -- FP4 s.e1e0.m -> s.00e1e0.m00 (the
//    value c * 2^-6), INT4 s.mmm -> s.0000.mmm (the subnormal |q| * 2^-9) --
//    and the hardware fp8 conversion yields m = +-c 2^-6 or +-|q| 2^-9
//    exactly, sign and zero included;
//  * y = fma(m, H, m * L) with a pair computed from the scale byte:
//    FP4: H = s' 2^(E+6), L = 0, so y = c s' 2^E exactly; INT4:
//    H = H' 2^(E+9) and L = fl32((6 s' - 7 H') * fl32(1/7)) 2^(E+9), where
//    H' is 6 s'/7 rounded toward zero: a two-term split of 6 s'/7 whose fma
//    gives the correctly rounded fl32(6 |q| s'/7) 2^E for every E4M3 s' and
//    |q| = 1..7 (checked exhaustively in exact arithmetic), with L >= 0 so
//    that a zero magnitude keeps its sign; NaN scales give H = NaN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace if4 {

__device__ __forceinline__ float e4m3_value_or_nan(uint32_t code7) {
    if (code7 == 0x7Fu) return __uint_as_float(0x7FC00000u);
    return code7 >= 8u ? __uint_as_float((code7 + 960u) << 20) : (float)code7 * 0.001953125f;
}

// Per-scale-byte decode constants: H, L, nibble shift (2 for FP4, 0 for INT4).
struct Entry {
    float h, l;
    uint32_t sh;
};

__device__ __forceinline__ Entry make_entry(uint32_t b, float p_exp) {
    const float sp = e4m3_value_or_nan(b & 0x7Fu);
    Entry e;
    if (b & 0x80u) {
        const float six = 6.0f * sp;  // exact
        // H = 6 s'/7 rounded toward zero, so the residual and L are >= 0 and
        // y keeps the sign of m for a zero magnitude (-0 stays -0)
        float h = six / 7.0f;
        if (__builtin_fmaf(-h, 7.0f, six) < 0.0f) h = __uint_as_float(__float_as_uint(h) - 1u);
        const float l = __builtin_fmaf(-h, 7.0f, six) * 0.142857149f;  // exact residual / 7
        const float k = p_exp * 512.0f;                       // 2^(E+9), exact
        e.h = h * k;
        e.l = l * k;
        e.sh = 0;
    } else {
        e.h = sp * (p_exp * 64.0f);                           // s' 2^(E+6)
        e.l = 0.0f;
        e.sh = 2;
    }
    return e;
}

// Decode the 8 nibbles of code word w (element 2j in the low nibble of byte
// j) into out[0..7] in element order.
__device__ __forceinline__ void decode_word(uint32_t w, const Entry& e, float* out) {
    const uint32_t mask = 0x07070707u << e.sh;
    // even nibbles (elements 0, 2, 4, 6) and odd ones (1, 3, 5, 7) as E4M3 bytes
    const uint32_t ev = ((w << 4) & 0x80808080u) | ((w << e.sh) & mask);
    const uint32_t od = (w & 0x80808080u) | ((w >> (4u - e.sh)) & mask);
    const auto e01 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(ev, 1.0f, false);  // elements 0, 2
    const auto e23 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(ev, 1.0f, true);   // 4, 6
    const auto o01 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(od, 1.0f, false);  // 1, 3
    const auto o23 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(od, 1.0f, true);   // 5, 7
    const float m[8] = {e01[0], o01[0], e01[1], o01[1], e23[0], o23[0], e23[1], o23[1]};
#pragma unroll
    for (int i = 0; i < 8; i++) out[i] = __builtin_fmaf(m[i], e.h, m[i] * e.l);
}

}  // namespace if4
