// Device helpers that encode one IF4 group in a lane's registers (HIP
// translation units only).  The rules are those of include/if4.h.
//
// Every rounding decision is taken exactly, for any fp32 input: each code
// is the count of grid midpoints the value passes, compared against exactly
// representable thresholds (s * midpoint for FP4; 7|x| - 3s(2k+1) by fma for
// INT4), with ties resolved to the even code by using >= or > per midpoint.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace if4 {

// E4M3 code (0..126) of RNE(a / 6), saturating at 448 (0x7E).  The fp32
// quotient is correctly rounded; rounding it again to 3 mantissa bits equals
// one rounding of the exact quotient because a/6 is never within half an
// fp32 ulp of an E4M3 midpoint M unless a = 6M exactly.
__device__ __forceinline__ uint32_t scale_code(float a_scaled) {
    float q = a_scaled / 6.0f;
    if (q < 0.015625f)  // below 2^-6: subnormal E4M3, spacing 2^-9
        return (uint32_t)__builtin_rintf(q * 512.0f);
    uint32_t b = __float_as_uint(q);
    b = b + 0x7FFFFu + ((b >> 20) & 1u);  // round the mantissa to 3 bits, ties even
    uint32_t code = (b >> 20) - 960u;     // (exponent + 120) << 3 | mantissa
    return code < 0x7Eu ? code : 0x7Eu;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
    return code >= 8u ? __uint_as_float((code + 960u) << 20) : (float)code * 0.001953125f;
}

// E2M1 index of |x| / s (ties to the even index, saturating at 6).
__device__ __forceinline__ uint32_t fp4_index(float ax, float s) {
    uint32_t i = 0;
    i += ax > 0.25f * s;
    i += ax >= 0.75f * s;
    i += ax > 1.25f * s;
    i += ax >= 1.75f * s;
    i += ax > 2.5f * s;
    i += ax >= 3.5f * s;
    i += ax > 5.0f * s;
    return i;
}

// min(RNE(7|x| / (6s)), 7): count the half-integers 7|x|/(6s) passes;
// t3 = 3s, midpoint k + 1/2 <=> 7|x| = 3s(2k+1).
__device__ __forceinline__ uint32_t int4_mag(float ax, float t3) {
    uint32_t q = 0;
#pragma unroll
    for (int k = 0; k < 7; k++) {
        float d = __builtin_fmaf(ax, 7.0f, -(float)(2 * k + 1) * t3);
        q += (k & 1) ? (d >= 0.0f) : (d > 0.0f);
    }
    return q;
}

__device__ __forceinline__ float e2m1_value(uint32_t idx) {
    // 0, .5, 1, 1.5, 2, 3, 4, 6
    float m = (idx & 1u) ? 1.5f : 1.0f;
    uint32_t e = idx >> 1;
    return e == 0 ? (idx ? 0.5f : 0.0f) : m * (float)(1u << (e - 1));
}

template <bool kBf16>
__device__ __forceinline__ void load_group(const void* __restrict__ x, int64_t off,
                                           float (&v)[16]) {
    if constexpr (kBf16) {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x) + off);
        uint4 a = *p;
        uint4 b = p[1];
        uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + off);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float4 t = p[i];
            v[4 * i] = t.x;
            v[4 * i + 1] = t.y;
            v[4 * i + 2] = t.z;
            v[4 * i + 3] = t.w;
        }
    }
}

// One group, exact rules for any fp32 values (x 2^-E): codes (element 2j in
// the low nibble of byte j of lo:hi) and the flagged scale byte.
template <int kMode>
__device__ __forceinline__ void exact_group(const float (&v)[16], float p_exp, float p_negexp,
                                            uint32_t& lo, uint32_t& hi, uint32_t& byte) {
    // group absmax; a NaN or infinity anywhere makes the group non-finite
    float a = 0.0f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        float ax = __builtin_fabsf(v[i]);
        finite &= ax <= 3.40282347e38f;
        a = __builtin_fmaxf(a, ax);
    }
    uint32_t sc = scale_code(a * p_negexp);
    lo = 0, hi = 0, byte = 0;
    if (!finite) {
        byte = 0x7Fu;
    } else if (sc != 0) {
        const float s = e4m3_value(sc) * p_exp;
        const float s7 = 7.0f * s, s6 = 6.0f * s, t3 = 3.0f * s;
        float ef = 0.0f, ei = 0.0f;
        uint32_t fl = 0, fh = 0, il = 0, ih = 0;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const float ax = __builtin_fabsf(v[i]);
            const uint32_t fi = fp4_index(ax, s);
            const uint32_t qi = int4_mag(ax, t3);
            const float df = __builtin_fmaf(ax, 7.0f, -(e2m1_value(fi) * s7));
            const float di = __builtin_fmaf(ax, 7.0f, -((float)qi * s6));
            ef = __builtin_fmaf(df, df, ef);
            ei = __builtin_fmaf(di, di, ei);
            const uint32_t sg = (__float_as_uint(v[i]) >> 28) & 8u;
            if (i < 8) {
                fl |= (sg | fi) << (4 * i);
                il |= (sg | qi) << (4 * i);
            } else {
                fh |= (sg | fi) << (4 * (i - 8));
                ih |= (sg | qi) << (4 * (i - 8));
            }
        }
        const bool use_int4 = kMode == 2 ? true : (kMode == 1 ? false : (ei < ef));
        lo = use_int4 ? il : fl;
        hi = use_int4 ? ih : fh;
        byte = sc | (use_int4 ? 0x80u : 0u);
    }
}

// Fast bf16 path.  Same results as the exact path for every bf16 input (the
// GPU tests sweep every (bf16 x, E4M3 s') pair), with cheaper arithmetic:
//
//  * scale: RNE_E4M3(a/6) from fl(a * fl(1/6)).  fl(1/6) is 1/6 (1 - e) with
//    e < 2^-25, so a tie a/6 = M (an E4M3 midpoint, 5 bits) rounds back to M
//    exactly, and a bf16 a (8 bits) is never within 2^-9 relative of any other
//    midpoint, far beyond the product's error.
//  * codes: u = |x|/s is approximated as |x| * r, r an approximation of 1/s
//    within 2.2 * 2^-24 relative, and snapped to a 2^-18 grid in the same fma
//    (adding 48 puts the sum in [32, 64), whose fp32 spacing is 2^-18); 7u/6
//    likewise with r7 ~ 7/(6s).  Every midpoint of either grid is a multiple
//    of 2^-18, and at the largest midpoint that matters (5 for u, 6.5 for
//    7u/6) the approximation error is below 6.5 * 2.2 * 2^-24 < 2^-20, well
//    inside half the grid spacing, so a value exactly on a midpoint snaps onto
//    it and every other value stays on its side (a bf16 x sits at least 2^-16
//    from any midpoint of u or 7u/6 that it does not hit).  r is v_rcp_f32 of
//    s' (within one ulp) refined by one Newton step (then within half an ulp
//    plus a 2^-46 relative term), r7 = r + r * fl(1/6) in one fma; the power
//    of two 2^-E is applied exactly after.  FP4: the snapped value carries x's
//    sign into the hardware E2M1
//    conversion (round to nearest even, saturating, signed zero kept), and
//    the same hardware decodes the codes back for the error.  INT4: adding
//    1.5 * 2^23 - 48 rounds the snapped 7|x|/(6s) to an integer (ties even),
//    min() clamps it to 7, and the low bits of the float are |q|.
//  * errors: for bf16 x every d = 7x - c*7s or 7|x| - |q|*6s is exact in
//    fp32, so fma(-c, 7s, 7x) equals the reference fma(|x|, 7, -|c|*7s).
//  * non-finite: a NaN reaches the FP4 error sum (NaN) and an infinity the
//    absmax; zero-scale groups use zero reciprocals so their sums stay finite.
// (An earlier version took r and r7 from a per-workgroup LDS table of
// correctly rounded reciprocals; computing them per group costs fewer
// instructions than filling the table, and drops its barrier.)

// One group of bf16-exact values, fast path (see above): codes and flagged
// scale byte, identical to exact_group for bf16 inputs.
template <int kMode, bool kElideClamp = false>
__device__ __forceinline__ void fast_group(const float (&v)[16],
                                           float p_exp, float p_negexp, uint32_t& lo,
                                           uint32_t& hi, uint32_t& byte) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i++) a = __builtin_fmaxf(a, __builtin_fabsf(v[i]));

    // scale code: RNE_E4M3(a * 2^-E / 6), saturating at 448
    const float q6 = (a * p_negexp) * 0.16666667f;
    uint32_t sc;
    if (q6 < 0.015625f) {
        sc = (uint32_t)__builtin_rintf(q6 * 512.0f);
    } else {
        uint32_t b = __float_as_uint(q6);
        b = b + 0x7FFFFu + ((b >> 20) & 1u);
        sc = (b >> 20) - 960u;
        sc = sc < 0x7Eu ? sc : 0x7Eu;
    }
    const float sp = e4m3_value(sc);
    const float s = sp * p_exp;
    float r = __builtin_amdgcn_rcpf(sp);
    r = __builtin_fmaf(r, __builtin_fmaf(-sp, r, 1.0f), r);
    float r7 = __builtin_fmaf(r, 0.16666667f, r);
    r = sc != 0 ? r : 0.0f;  // (rcp(0) is infinite)
    r7 = sc != 0 ? r7 : 0.0f;
    const float inv_s = r * p_negexp, k7 = r7 * p_negexp;
    const float s7 = 7.0f * s, s6 = 6.0f * s;

    // FP4 codes via the hardware E2M1 conversion of the snapped quotients
    float us[16];
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const float t = __builtin_fmaf(__builtin_fabsf(v[i]), inv_s, 48.0f) - 48.0f;
        us[i] = __builtin_copysignf(t, v[i]);
    }
    uint32_t f0 = 0, f1 = 0;
    f0 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(f0, us[0], us[1], 1.0f, 0);
    f0 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(f0, us[2], us[3], 1.0f, 1);
    f0 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(f0, us[4], us[5], 1.0f, 2);
    f0 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(f0, us[6], us[7], 1.0f, 3);
    f1 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(f1, us[8], us[9], 1.0f, 0);
    f1 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(f1, us[10], us[11], 1.0f, 1);
    f1 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(f1, us[12], us[13], 1.0f, 2);
    f1 = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(f1, us[14], us[15], 1.0f, 3);
    float c[16];
    {
        auto d0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(f0, 1.0f, 0);
        auto d1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(f0, 1.0f, 1);
        auto d2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(f0, 1.0f, 2);
        auto d3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(f0, 1.0f, 3);
        auto d4 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(f1, 1.0f, 0);
        auto d5 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(f1, 1.0f, 1);
        auto d6 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(f1, 1.0f, 2);
        auto d7 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(f1, 1.0f, 3);
        c[0] = d0[0]; c[1] = d0[1]; c[2] = d1[0]; c[3] = d1[1];
        c[4] = d2[0]; c[5] = d2[1]; c[6] = d3[0]; c[7] = d3[1];
        c[8] = d4[0]; c[9] = d4[1]; c[10] = d5[0]; c[11] = d5[1];
        c[12] = d6[0]; c[13] = d6[1]; c[14] = d7[0]; c[15] = d7[1];
    }

    // INT4 magnitudes and both error sums, index order 0..15.  The clamp
    // |q| <= 7 can only act when s' is an E4M3 subnormal (codes 1-7, spaced
    // 2^-9 apart, so s' may sit far below a'/6) or when a'/6 reaches 448 (the
    // scale saturates).  For every other scale s' >= (a'/6) / (1 + 2^-4) --
    // rounding to three mantissa bits moves a value down by at most 2^-4 of
    // its binade's base -- so 7|x|/(6s) <= 7 * 1.0625 = 7.4375 (plus the
    // snapped quotient's error, below 2^-20) rounds to at most 7 without it.
    // With kElideClamp the clamp is taken out of the loop when no lane of the
    // wave needs it, at the cost of a second copy of the loop: 16 fewer VALU
    // per group on the row kernel (3-5% faster on 86-470 MB tensors); the x^T
    // kernels gain nothing from it and the rotating kernel runs 1-2% slower.
    float ef = 0.0f, ei = 0.0f;
    uint32_t rq[16];
    auto int4_pass = [&](auto clamp_c) {
        constexpr bool kClamp = decltype(clamp_c)::value;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const float xa = __builtin_fabsf(v[i]);
            const float X = 7.0f * v[i];
            const float t = __builtin_fmaf(xa, k7, 48.0f);
            // 1.5*2^23 + |q|, clamped to |q| <= 7 (positive floats order as
            // their bits)
            uint32_t rb = __float_as_uint(t + 12582864.0f);
            if constexpr (kClamp) rb = __builtin_elementwise_min(rb, 0x4B400007u);
            rq[i] = rb;
            const float q = __uint_as_float(rb) - 12582912.0f;
            const float df = __builtin_fmaf(-c[i], s7, X);
            const float di = __builtin_fmaf(-q, s6, __builtin_fabsf(X));
            ef = __builtin_fmaf(df, df, ef);
            ei = __builtin_fmaf(di, di, ei);
        }
    };
    const bool need_clamp = (sc - 1u < 7u) || (q6 >= 448.0f);
    if (!kElideClamp || __builtin_amdgcn_ballot_w64(need_clamp) != 0)
        int4_pass(std::true_type{});
    else
        int4_pass(std::false_type{});
    // gather |q| (low byte of each float) into nibbles: even elements in
    // bits 0-2, odd elements in bits 4-6 of each byte
    uint32_t i0, i1;
    {
        const uint32_t e0 = __builtin_amdgcn_perm(rq[2], rq[0], 0x0C0C0400u) |
                            __builtin_amdgcn_perm(rq[6], rq[4], 0x04000C0Cu);
        const uint32_t o0 = __builtin_amdgcn_perm(rq[3], rq[1], 0x0C0C0400u) |
                            __builtin_amdgcn_perm(rq[7], rq[5], 0x04000C0Cu);
        const uint32_t e1 = __builtin_amdgcn_perm(rq[10], rq[8], 0x0C0C0400u) |
                            __builtin_amdgcn_perm(rq[14], rq[12], 0x04000C0Cu);
        const uint32_t o1 = __builtin_amdgcn_perm(rq[11], rq[9], 0x0C0C0400u) |
                            __builtin_amdgcn_perm(rq[15], rq[13], 0x04000C0Cu);
        // sign bits are those of the FP4 codes (both take x's sign bit)
        i0 = (e0 | (o0 << 4)) | (f0 & 0x88888888u);
        i1 = (e1 | (o1 << 4)) | (f1 & 0x88888888u);
    }

    const bool use_int4 = kMode == 2 ? true : (kMode == 1 ? false : (ei < ef));
    lo = use_int4 ? i0 : f0;
    hi = use_int4 ? i1 : f1;
    byte = sc | (use_int4 ? 0x80u : 0u);
    if (sc == 0) {
        lo = hi = 0;
        byte = 0;
    }
    if (!(a <= 3.40282347e38f) || ef != ef) {  // infinity or NaN in the group
        lo = hi = 0;
        byte = 0x7Fu;
    }
}

}  // namespace if4
