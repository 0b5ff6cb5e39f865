// IF3 and IF6 quantize / dequantize for gfx950.
//
// The pages extend the adaptive per-group choice to 3 and 6 bits per value
// ("Adaptive Block-Scaled Data Types for FP4 Training", podcast companion,
// "It Generalizes: IF3 and IF6"; gist.science summary, section 2,
// "Extensoes") without defining the formats.  The formats here keep IF4's
// construction (include/if4.h states them in full): sign-magnitude codes,
// one E4M3 scale per 16 values with the choice in its sign bit, the INT range
// pre-scaled so that its top value lands on the float grid's top value,
// scale = RNE_E4M3(amax / top), fp32 squared errors in a domain where the INT
// descale is exact.
//   IF6: FP6 E2M3 (top 7.5) or INT6 |q| <= 31 decoding to q * 15/62 * s;
//        errors x62.
//   IF3: FP3 E2M0 {0, 1, 2, 4} or INT3 |q| <= 3 decoding to q * 4/3 * s;
//        errors x3.
// Element i of a group occupies bits [bits*i, bits*(i+1)) of the group's
// little-endian 2*bits-byte code field.
//
// One group per thread (IF6 from bf16: two), one-wave workgroups for the
// quantizes and the IF3 dequantize and 256-thread ones for the IF6
// dequantize, the thread's loads issued first.  Every rounding is decided exactly (exact comparisons, or the
// exact sign of one fma), ties to the even index -- valid for any fp32 input
// -- in branch-free code.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "if4_internal.h"
#include "launch_limit.h"
#include "xcd_order.h"

namespace if4 {
namespace {

constexpr int kThreads = 256;  // IF6 dequantize: one workgroup builds its LDS tables for 256 groups
constexpr int kQThreads = 64;  // quantizes (no LDS): one-wave workgroups fill the chip sooner

template <int kBits>
struct Fmt;

template <>
struct Fmt<6> {
    static constexpr float kTop = 7.5f;     // 32 float magnitudes, INT 0..31
    static constexpr float kDn = 15.0f, kDd = 62.0f;  // top / qmax = dn / dd
    // E2M3 magnitude of index i: 2 exponent bits (bias 1), 3 mantissa bits
    __device__ static float fp(int i) {
        const int e = i >> 3, m = i & 7;
        return e == 0 ? (float)m * 0.125f : (float)(8 + m) * __builtin_ldexpf(1.0f, e - 4);
    }
};

template <>
struct Fmt<3> {
    static constexpr float kTop = 4.0f;     // E2M0: 0, 1, 2, 4; INT 0..3
    static constexpr float kDn = 4.0f, kDd = 3.0f;
    __device__ static float fp(int i) { return i == 0 ? 0.0f : __builtin_ldexpf(1.0f, i - 1); }
};

__device__ __forceinline__ float e4m3_value(uint32_t code) {
    return code >= 8u ? __uint_as_float((code + 960u) << 20) : (float)code * 0.001953125f;
}

// 1 if a magnitude ax (>= 0) rounds above the boundary t of index k (the
// midpoint between grid values k and k + 1): ax > t, or ax == t for odd k,
// so that ties go to the even index.  Non-negative floats order as their bit
// patterns; a negative t is always passed and t = +inf never.
__device__ __forceinline__ int passes(float ax, float t, int k) {
    return (int)__float_as_uint(ax) + (k & 1) > (int)__float_as_uint(t) ? 1 : 0;
}
// the same given the difference d = ax - t from one fma (its sign is exact and
// an exact zero is +0): d > 0, or d == +0 for odd k -- the low bit or'ed into
// d's bit pattern leaves a negative d negative
__device__ __forceinline__ int passes_d(float d, int k) {
    return ((int)__float_as_uint(d) | (k & 1)) > 0 ? 1 : 0;
}

// E2M3 on fp32 bits: the index k = 8e + m (2 exponent bits with bias 1, 3
// mantissa bits) placed at bit 20, k << 20, is the fp32 pattern with exponent
// field e and mantissa m / 8 -- read as a float it equals the E2M3 magnitude
// of k times 2^-126 for all 32 indices, E2M3's subnormals (e = 0) landing on
// fp32's.  Setting bit 19 as well gives the midpoint between k and k + 1.
// Multiplying by 2^126 makes either an exact normal float.
__device__ __forceinline__ float e2m3_value(int k) {
    return __uint_as_float((uint32_t)k << 20) * 0x1p126f;
}
__device__ __forceinline__ float e2m3_mid(int k) {
    return __uint_as_float(((uint32_t)k << 20) | (1u << 19)) * 0x1p126f;
}

// The scale code and IF6's indices are "guess, then one exact check".  A
// guess truncates an approximate quotient (at most a part in 2^21 off) to the
// grid below it, which gives the correctly rounded index or the one below
// (the grids are at least 2^-4 apart, relative); comparing with the exact
// boundary above the guess decides between them -- directly for the scale
// (an fp32 product of at most 9 significant bits), by the sign of one fma
// for the elements.  IF3 compares every element with its six boundaries.
template <int kBits, int kMode>
__device__ __forceinline__ void quantize_group(const float (&v)[16], float p_exp, float p_negexp,
                                               uint32_t (&out)[3], uint32_t& byte) {
    using F = Fmt<kBits>;
    constexpr float kInf = __builtin_inff();
    // amax on the magnitudes' bit patterns, which order as the values do and
    // put inf and NaN above every finite value
    uint32_t abits = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) abits = max(abits, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    out[0] = out[1] = out[2] = 0;
    if (abits >= 0x7F800000u) {
        byte = 0x7Fu;
        return;
    }
    const float a = __uint_as_float(abits);
    // scale code RNE_E4M3(a 2^-E / top) over the 127 finite codes; the
    // boundary above code k is top (v_k + v_{k+1}) / 2 (4 + 5 bits, exact)
    const float ap = a * p_negexp;
    const float qg = ap * (1.0f / F::kTop);
    int sc = qg < 0.015625f ? (int)(qg * 512.0f) : (int)(__float_as_uint(qg) >> 20) - 960;
    sc = sc < 126 ? sc : 126;
    sc += passes(ap, sc < 126 ? F::kTop * (0.5f * (e4m3_value(sc) + e4m3_value(sc + 1))) : kInf,
                 sc);
    if (sc == 0) {
        byte = 0;
        return;
    }
    const float s = e4m3_value((uint32_t)sc) * p_exp;
    const float sdd = F::kDd * s, sdn = F::kDn * s;
    constexpr int kFMax = (1 << (kBits - 1)) - 1, kQMax = kFMax;
    // IF6: reciprocals for the guesses.  IF3: its three boundaries of each
    // kind as fp32 values that ax is compared with directly.  The FP ones,
    // s (fp(k) + fp(k + 1)) / 2, are exact; the INT ones, dn s (k + 1/2) / dd,
    // are taken rounded down (exact when representable, as 2s is for k = 1):
    // a float passes the rounded-down value exactly when it passes the true
    // one, so "ax > t" decides an even k (ties stay down) and "ax >= t" the
    // odd k = 1, whose boundaries are exact.
    const float r = __builtin_amdgcn_rcpf(s);
    const float rq = r * (F::kDd / F::kDn);
    const float sdn_half = 0.5f * sdn;
    float tf[3], tq[3];
    if constexpr (kBits == 3) {
#pragma unroll
        for (int k = 0; k < 3; k++) {
            tf[k] = s * (0.5f * (F::fp(k) + F::fp(k + 1)));
            // within an ulp of sdn (k + 1/2) / dd; one step down if above it
            const float num = sdn * ((float)k + 0.5f);
            const float w = num * (1.0f / F::kDd);
            tq[k] = __builtin_fmaf(w, F::kDd, -num) > 0.0f ? __uint_as_float(__float_as_uint(w) - 1u) : w;
        }
    }
    float ef = 0.0f, ei = 0.0f;
    // magnitude fields of both candidates and the sign field, kBits per element
    uint32_t mf[3] = {0, 0, 0}, mq[3] = {0, 0, 0}, sg[3] = {0, 0, 0};
    auto put = [](uint32_t(&f)[3], uint32_t c, int bit) {
        f[bit >> 5] |= c << (bit & 31);
        if ((bit & 31) + kBits > 32) f[(bit >> 5) + 1] |= c >> (32 - (bit & 31));
    };
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const float ax = __builtin_fabsf(v[i]);
        int fi, q;
        // the candidates' values times dd s and dd s dn / dd = dn s, exact
        // (at most 14 significant bits)
        float fvs, qsdn;
        if constexpr (kBits == 6) {
            // guess: the approximate quotient u = ax / s times 2^-126 (an
            // fp32 subnormal below 1) truncated to the E2M3 bits above bit
            // 20, clamped to 30 so that the boundary above it exists; a
            // guess is never above the correctly rounded index.  The check
            // takes the sign of ax - mid s from one fma.
            const float u = ax * r;
            const int g = min((int)(__float_as_uint(__builtin_ldexpf(u, -126)) >> 20), kFMax - 1);
            fi = g + passes_d(__builtin_fmaf(e2m3_mid(g), -s, ax), g);
            fvs = e2m3_value(fi) * sdd;
            // INT: |q| > k  <=>  dd |x| > dn s (k + 1/2), the threshold
            // dn s k + dn s / 2 exact in one fma
            const int h = (int)__builtin_fminf(ax * rq, (float)(kQMax - 1));
            q = h + passes_d(__builtin_fmaf(ax, F::kDd, -__builtin_fmaf((float)h, sdn, sdn_half)), h);
            qsdn = (float)q * sdn;
        } else {
            const bool f0 = ax > tf[0], f1 = ax >= tf[1], f2 = ax > tf[2];
            const bool q0 = ax > tq[0], q1 = ax >= tq[1], q2 = ax > tq[2];
            fi = (int)f0 + (int)f1 + (int)f2;
            q = (int)q0 + (int)q1 + (int)q2;
            // E2M0 on fp32 bits: index k << 23 read as a float is 0, 1, 2, 4
            // times 2^-126 (exponent field k, k = 0 the zero)
            fvs = (__uint_as_float((uint32_t)fi << 23) * 0x1p126f) * sdd;
            qsdn = (float)q * sdn;
        }
        const float df = __builtin_fmaf(ax, F::kDd, -fvs);
        const float di = __builtin_fmaf(ax, F::kDd, -qsdn);
        ef = __builtin_fmaf(df, df, ef);
        ei = __builtin_fmaf(di, di, ei);
        put(mf, (uint32_t)fi, kBits * i);
        put(mq, (uint32_t)q, kBits * i);
        put(sg, (__float_as_uint(v[i]) >> 31) << (kBits - 1), kBits * i);
    }
    const bool use_int = kMode == 2 ? true : (kMode == 1 ? false : (ei < ef));
#pragma unroll
    for (int w = 0; w < 3; w++) out[w] = (use_int ? mq[w] : mf[w]) | sg[w];
    byte = (uint32_t)sc | (use_int ? 0x80u : 0u);
}

// ---------------------------------------------------------------------------
// bf16 fast path.  Same codes and scale bytes as quantize_group for every
// bf16 input (the GPU tests sweep every (bf16 x, E4M3 s') pair for both
// formats), with fewer instructions:
//
//  * quotients: u = |x|/s, and for INT the quotient on the INT grid, are
//    approximated with reciprocals of s' (v_rcp_f32 refined by one Newton
//    step: within 2^-24 (1 + 2^-22) relative) and snapped in the same fma to
//    a grid that holds every midpoint exactly: IF6's u onto 2^-18 (+48, sums
//    in [48, 64)); IF6's INT quotient 62|x|/(15 s) <= 34 onto 2^-17 (+64), as
//    62|x| (exact for bf16, and shared with both error terms) times the
//    reciprocal of 15 s; IF3's 3|x|/(4 s) onto 2^-19 (+16), as |x| * fl(0.75 r)
//    (one more rounding: within 2^-23 (1 + 2^-22) relative).  The
//    approximation error at the largest midpoint that matters (7.25, 30.5,
//    2.5) stays below half the snap grid, so a value on a midpoint snaps onto
//    it exactly, and a bf16 x that is not on a midpoint sits at least 2^-15
//    (in quotient units) from it, far beyond the error plus half a grid step.
//  * IF6 float codes: gfx950's E2M3 conversion (v_cvt_scalef32_2xpk16_fp6_f32,
//    round to nearest even, saturating at 7.5, signed zero kept; checked over
//    every multiple of 2^-18 in [-9, 9], infinities and huge values) encodes
//    the snapped signed quotients straight into the packed 6-bit layout (it
//    interleaves its two 16-value operands: slot 2j takes the first
//    operand's value j, slot 2j + 1 the second's), and the matching decode
//    (v_cvt_scalef32_pk32_f32_fp6) returns the grid values for the errors.
//  * IF3 float codes: the quotient against the three midpoints 0.5, 1.5 and 3
//    of {0, 1, 2, 4} (> for 0.5 and 3, >= for 1.5: ties to even), each moved
//    by less than the 2^-15 that separates a non-tie from it, toward the side
//    its tie belongs to: 0.5 by one clamped fma, 1.5 and 3 as the binades of
//    one affine function of u, whose exponent is the index.
//  * IF3 packing: the chosen magnitudes shifted into the 48-bit field (the
//    INT ones as whole magic-number floats, their constant part subtracted
//    once), the signs gathered from the bf16 words by v_perm's sign-fill
//    selectors.
//  * INT magnitudes: adding 1.5 * 2^23 minus the snap offset rounds the
//    snapped quotient to an integer (ties to even) in the float's low bits;
//    an integer min clamps it to qmax.
//  * errors: exactly the products and fmas of the reference (c dd s and
//    |q| dn s are exact), in index order; both formats subtract them from
//    dd |x| computed once (exact for bf16), which rounds the same difference
//    once (IF3's float product as 2c times dd s / 2, the same exact value).
//  * non-finite: an infinity makes the absmax infinite, a NaN the float
//    error sum NaN; zero scales get zero reciprocals so the sums stay finite.
__device__ __forceinline__ float refined_rcp(float d) {
    const float r = __builtin_amdgcn_rcpf(d);
    return __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.0f), r);
}

template <int kBits>
__device__ __forceinline__ int scale_code_of(float a, float p_negexp) {
    using F = Fmt<kBits>;
    const float ap = a * p_negexp;
    const float qg = ap * (1.0f / F::kTop);
    int sc = qg < 0.015625f ? (int)(qg * 512.0f) : (int)(__float_as_uint(qg) >> 20) - 960;
    sc = sc < 126 ? sc : 126;
    sc += passes(ap,
                 sc < 126 ? F::kTop * (0.5f * (e4m3_value(sc) + e4m3_value(sc + 1)))
                          : __builtin_inff(),
                 sc);
    return sc;
}

// the sign bit (bit 5 of each 6-bit field) positions in the three words of
// an IF6 group's code field
constexpr uint32_t kIf6Sign[3] = {0x20820820u, 0x08208208u, 0x82082082u};

// what the 1.5 * 2^23 of each INT3 element's rb adds to its code word when
// rb is shifted into place whole (mod 2^32; elements 0-10 in word 0, 11-15 in
// word 1)
constexpr uint32_t if3_int_bias(int w) {
    uint32_t k = 0;
    for (int i = 0; i < 16; i++)
        if ((i <= 10 ? 0 : 1) == w) k += 0x4B400000u << (3 * i - 32 * w);
    return k;
}
constexpr uint32_t kIf3IntBias[2] = {if3_int_bias(0), if3_int_bias(1)};

template <int kBits, int kMode>
__device__ __forceinline__ void fast_group_bf16(const float (&v)[16], const uint32_t (&xw)[8],
                                                float p_exp, float p_negexp, uint32_t (&out)[3],
                                                uint32_t& byte) {
    using F = Fmt<kBits>;
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i++) a = __builtin_fmaxf(a, __builtin_fabsf(v[i]));
    const int sc = scale_code_of<kBits>(a, p_negexp);
    const float sp = e4m3_value((uint32_t)sc);
    const float s = sp * p_exp;
    const float sdd = F::kDd * s, sdn = F::kDn * s;  // exact
    float r = refined_rcp(sp);
    r = sc != 0 ? r : 0.0f;  // (rcp(0) is infinite)
    const float rs = r * p_negexp;                // ~ 1/s
    const float rsk = rs * 0x1p18f;               // ~ 2^18 / s
    const float ra = rs * 1.33331811f;            // ~ (4/3 - 2^-16) / s
    const float rs34 = (0.75f * r) * p_negexp;    // ~ 3/(4s), one more rounding
    const float sdh = 0.5f * sdd;                 // exact
    float ef = 0.0f, ei = 0.0f;
    static_assert(kBits == 3, "IF6 takes two groups at a time: if6_pair_bf16");
    {
        uint32_t fiv[16], rbv[16];
        // The INT clamp |q| <= 3 can only act when s' is an E4M3 subnormal
        // (codes 1-7) or the 448 code (where a'/4 may lie far above it).  For
        // every other scale s' >= (a'/4) / (1 + 2^-4) -- rounding to three
        // mantissa bits moves a value down by at most 2^-4 of its binade's
        // base -- so 3|x|/(4s) <= 3 * 1.0625 = 3.1875 (plus the snapped
        // quotient's error) rounds to at most 3 without it; the loop runs
        // without the clamp when no lane of the wave needs it.
        auto pass = [&](auto clamp_c) {
        constexpr bool kClamp = decltype(clamp_c)::value;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const float ax = __builtin_fabsf(v[i]);
            // 3|x|, exact for bf16 (where it overflows, so does the reference's
            // fused 3|x| - c s dd, whose subtrahend is far below an ulp there)
            const float x3 = ax * F::kDd;
            // float index: u = |x|/s against the midpoints 0.5, 1.5 and 3 (ties
            // to 0, 2 and 2).  An exact tie is the only quotient closer than
            // 2^-15 to a midpoint, so each test may move its midpoint by less:
            //  u > 0.5:  h = 2^18 (u - 0.5 - 2^-17) clamped to [0, 1] is 0 or 1
            //            (the unclamped value is <= -1 or >= 1);
            //  u >= 1.5 and u > 3: f = (4/3 - 2^-16) u + 2^-15 has f(1.5) =
            //            2 + 2^-17 and f(3) = 4 - 2^-16; f raised to h and
            //            capped below 8 (an infinite product included) has the
            //            index as its exponent (frexp: [1, 2) -> 1, [2, 4) -> 2,
            //            [4, 8) -> 3; below 1 -> 0 or less, raised to 0).
            // The reciprocal's error moves f by under 2^-20 near the midpoints.
            const float h = __builtin_amdgcn_fmed3f(__builtin_fmaf(ax, rsk, -131074.0f), 0.0f, 1.0f);
            const float f = __builtin_amdgcn_fmed3f(__builtin_fmaf(ax, ra, 0x1p-15f), h, 7.99f);
            const int fi = __builtin_elementwise_max(__builtin_amdgcn_frexp_expf(f), 0);
            const float cv2 = __builtin_ldexpf(h, fi);  // twice the grid value: 0, 2, 4, 8
            const float df = __builtin_fmaf(-cv2, sdh, x3);
            ef = __builtin_fmaf(df, df, ef);
            // 3|x|/(4s) snapped to a multiple of 2^-19 (sums in [16, 32)); 1.5 *
            // 2^23 - 16 more rounds it to an integer (ties even) in the low bits
            const float t = __builtin_fmaf(ax, rs34, 16.0f);
            uint32_t rb = __float_as_uint(t + 12582896.0f);
            if constexpr (kClamp) rb = __builtin_elementwise_min(rb, 0x4B400003u);
            const float q = __uint_as_float(rb) - 12582912.0f;
            const float di = __builtin_fmaf(-q, sdn, x3);
            ei = __builtin_fmaf(di, di, ei);
            fiv[i] = (uint32_t)fi;
            rbv[i] = rb;
        }
        };
        const bool need_clamp = (uint32_t)(sc - 1) < 7u || sc >= 126;
        if (__builtin_amdgcn_ballot_w64(need_clamp) != 0)
            pass(std::true_type{});
        else
            pass(std::false_type{});
        const bool use_int = kMode == 2 ? true : (kMode == 1 ? false : (ei < ef));
        // the chosen magnitudes into the 48-bit field (element i at bits 3i,
        // 3i + 1; element 10 ends word 0).  An INT magnitude goes in as the
        // whole rb = 1.5 * 2^23 + |q|; what the constant adds is taken out after.
        uint32_t w0 = 0, w1 = 0;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const uint32_t c = use_int ? rbv[i] : fiv[i];
            if (i <= 10) w0 += c << (3 * i);
            else w1 += c << (3 * i - 32);
        }
        w0 -= use_int ? kIf3IntBias[0] : 0u;
        w1 -= use_int ? kIf3IntBias[1] : 0u;
        // sign bits (bit 3i + 2) from the bf16 words, whose bits 15 and 31 are
        // elements 2j and 2j + 1: v_perm's selectors 8-11 fill a byte with
        // bit 15 / 31 of its second source or bit 15 / 31 of its first, and 12
        // gives a zero byte; each perm places at most one element per byte.
        auto sgn = [](uint32_t hi, uint32_t lo, uint32_t sel, uint32_t mask) {
            return __builtin_amdgcn_perm(hi, lo, sel) & mask;
        };
        w0 |= sgn(xw[2], xw[0], 0x0C0B0A08u, 0x00024004u)    // el 0 (b0), 4 (b1), 5 (b2)
            | sgn(xw[3], xw[0], 0x0C0A0C09u, 0x00100020u)    // el 1 (b0), 6 (b2)
            | sgn(xw[4], xw[1], 0x0A0C080Cu, 0x04000100u)    // el 2 (b1), 8 (b3)
            | sgn(xw[4], xw[1], 0x0B0C090Cu, 0x20000800u)    // el 3 (b1), 9 (b3)
            | sgn(xw[3], xw[3], 0x0C090C0Cu, 0x00800000u);   // el 7 (b2)
        w1 |= sgn(xw[6], xw[5], 0x0C0C0B08u, 0x00000201u)    // el 10 (b0), 13 (b1)
            | sgn(xw[7], xw[6], 0x0C0C0A08u, 0x00001040u)    // el 12 (b0), 14 (b1)
            | sgn(xw[7], xw[5], 0x0C0C0B09u, 0x00008008u);   // el 11 (b0), 15 (b1)
        out[0] = w0;
        out[1] = w1;
        out[2] = 0;
        byte = (uint32_t)sc | (use_int ? 0x80u : 0u);
    }
    if (sc == 0) {
        out[0] = out[1] = out[2] = 0;
        byte = 0;
    }
    if (!(a <= 3.40282347e38f) || ef != ef) {  // infinity or NaN in the group
        out[0] = out[1] = out[2] = 0;
        byte = 0x7Fu;
    }
}

// what the 1.5 * 2^23 of each INT6 element's rb adds to the three code words
// when rb is shifted into its field whole (mod 2^32; a straddling field's
// upper part goes to the next word, where 1.5 * 2^23 >> (32 - bit) is exact:
// its low 22 bits are zero)
constexpr uint32_t if6_int_bias(int w) {
    uint32_t k = 0;
    for (int i = 0; i < 16; i++) {
        const int bit = 6 * i;
        if ((bit >> 5) == w) k += 0x4B400000u << (bit & 31);
        if ((bit & 31) + 6 > 32 && (bit >> 5) + 1 == w) k += 0x4B400000u >> (32 - (bit & 31));
    }
    return k;
}
constexpr uint32_t kIf6IntBias[3] = {if6_int_bias(0), if6_int_bias(1), if6_int_bias(2)};

// IF6, two groups at a time: the E2M3 conversion takes 32 values, slot 2j
// from its first operand's value j and slot 2j + 1 from the second's, so the
// even elements of groups 0 and 1 go to the first operand (positions 0-7 and
// 8-15) and the odd ones to the second, and the converted 192 bits hold group
// 0's field in words 0-2 and group 1's in words 3-5.
template <int kMode>
__device__ __forceinline__ void if6_pair_bf16(const float (&v)[2][16], float p_exp,
                                              float p_negexp, uint32_t (&out)[2][3],
                                              uint32_t (&byte)[2]) {
    using F = Fmt<6>;
    typedef float v16f __attribute__((ext_vector_type(16)));
    typedef float v32f __attribute__((ext_vector_type(32)));
    typedef uint32_t v6u __attribute__((ext_vector_type(6)));
    v16f ev, od;  // signed snapped quotients of the even / odd elements
    float x62[2][16];  // 62 |x|
    float a[2], ei[2] = {0.0f, 0.0f}, sdd[2];
    int sc[2];
    uint32_t mq[2][3] = {{0, 0, 0}, {0, 0, 0}};
#pragma unroll
    for (int h = 0; h < 2; h++) {
        a[h] = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i++) a[h] = __builtin_fmaxf(a[h], __builtin_fabsf(v[h][i]));
        sc[h] = scale_code_of<6>(a[h], p_negexp);
        const float sp = e4m3_value((uint32_t)sc[h]);
        const float s = sp * p_exp;
        sdd[h] = F::kDd * s;
        const float sdn = F::kDn * s;  // exact
        float r = refined_rcp(sp), rq = refined_rcp(15.0f * sp);  // 15 s' exact
        r = sc[h] != 0 ? r : 0.0f;  // (rcp(0) is infinite)
        rq = sc[h] != 0 ? rq : 0.0f;
        const float rs = r * p_negexp;          // ~ 1/s
        rq *= p_negexp;                         // ~ 1 / (15 s)
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const float ax = __builtin_fabsf(v[h][i]);
            // 62 |x|: exact for bf16 (5 + 8 significant bits).  Where it
            // overflows, the reference's fused 62|x| - c 62 s and 62|x| - |q| 15 s
            // overflow too: s <= 448 * 2^64 puts both subtrahends far below an
            // ulp there, and 62|x|, a multiple of 2^116 there, is never the
            // rounding midpoint to infinity.
            x62[h][i] = ax * F::kDd;
            const float u = __builtin_copysignf(__builtin_fmaf(ax, rs, 48.0f) - 48.0f, v[h][i]);
            if (i & 1)
                od[8 * h + (i >> 1)] = u;
            else
                ev[8 * h + (i >> 1)] = u;
            // INT: 1.5 * 2^23 + |q| in the float's bits, |q| clamped to 31;
            // 62|x| / (15 s) from the exact 62|x| and the reciprocal
            const float t = __builtin_fmaf(x62[h][i], rq, 64.0f);
            const uint32_t rb =
                __builtin_elementwise_min(__float_as_uint(t + 12582848.0f), 0x4B40001Fu);
            const float q = __uint_as_float(rb) - 12582912.0f;
            const float di = __builtin_fmaf(-q, sdn, x62[h][i]);  // |q| 15 s exact
            ei[h] = __builtin_fmaf(di, di, ei[h]);
            // rb = 1.5 * 2^23 + |q| shifted into the 6-bit field whole (its
            // constant part taken out once per word below); a field that
            // straddles two words puts its upper bits into the next one
            const int bit = 6 * i;
            mq[h][bit >> 5] += rb << (bit & 31);
            if ((bit & 31) + 6 > 32) mq[h][(bit >> 5) + 1] += rb >> (32 - (bit & 31));
        }
    }
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
        for (int w = 0; w < 3; w++) mq[h][w] -= kIf6IntBias[w];
    const auto fcv = __builtin_amdgcn_cvt_scalef32_2xpk16_fp6_f32(ev, od, 1.0f);
    const v6u fc = __builtin_bit_cast(v6u, fcv);
    const v32f c = __builtin_amdgcn_cvt_scalef32_pk32_f32_fp6(fcv, 1.0f);
#pragma unroll
    for (int h = 0; h < 2; h++) {
        float ef = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const float df = __builtin_fmaf(-__builtin_fabsf(c[16 * h + i]), sdd[h], x62[h][i]);
            ef = __builtin_fmaf(df, df, ef);
        }
        const bool use_int = kMode == 2 ? true : (kMode == 1 ? false : (ei[h] < ef));
#pragma unroll
        for (int w = 0; w < 3; w++)
            out[h][w] = use_int ? (mq[h][w] | (fc[3 * h + w] & kIf6Sign[w])) : fc[3 * h + w];
        byte[h] = (uint32_t)sc[h] | (use_int ? 0x80u : 0u);
        if (sc[h] == 0) {
            out[h][0] = out[h][1] = out[h][2] = 0;
            byte[h] = 0;
        }
        if (!(a[h] <= 3.40282347e38f) || ef != ef) {  // infinity or NaN in the group
            out[h][0] = out[h][1] = out[h][2] = 0;
            byte[h] = 0x7Fu;
        }
    }
}

// IF6 from bf16: two consecutive groups per thread (one 64-byte span of a
// row when the row holds both), both through if6_pair_bf16
template <int kMode, bool kContig>
__global__ void __launch_bounds__(kQThreads)
quantize_if6_bf16_kernel(const uint16_t* __restrict__ x, int64_t rows, int64_t gpr, int64_t ld_x,
                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, float p_exp,
                         float p_negexp) {
    const int64_t ngroups = rows * gpr;
    const int64_t g0 = 2 * ((int64_t)blockIdx.x * kQThreads + threadIdx.x);
    float v[2][16];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int64_t g = g0 + h < ngroups - 1 ? g0 + h : ngroups - 1;
        int64_t off;
        if constexpr (kContig) {
            off = g * 16;
        } else {
            const int64_t r = g / gpr;
            off = r * ld_x + (g - r * gpr) * 16;
        }
        const uint4* p = reinterpret_cast<const uint4*>(x + off);
        const uint4 a = p[0], b = p[1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; i++) {
            v[h][2 * i] = __uint_as_float(w[i] << 16);
            v[h][2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    uint32_t out[2][3], byte[2];
    if6_pair_bf16<kMode>(v, p_exp, p_negexp, out, byte);
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int64_t g = g0 + h;
        if (g < ngroups) {
            uint32_t* c = reinterpret_cast<uint32_t*>(codes + g * 12);
            c[0] = out[h][0];
            c[1] = out[h][1];
            c[2] = out[h][2];
            scales[g] = (uint8_t)byte[h];
        }
    }
}

// kContig: rows back to back (ld = cols), so a group's offset is 16 g with
// no division by the groups per row
template <int kBits, int kMode, bool kBf16, bool kContig>
__global__ void __launch_bounds__(kQThreads)
quantize_ifn_kernel(const void* __restrict__ x, int64_t rows, int64_t gpr, int64_t ld_x,
                    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, float p_exp,
                    float p_negexp) {
    const int64_t ngroups = rows * gpr;
    const int64_t gid = (int64_t)blockIdx.x * kQThreads + threadIdx.x;
    const int64_t g = gid < ngroups - 1 ? gid : ngroups - 1;
    int64_t off;
    if constexpr (kContig) {
        off = g * 16;
    } else {
        const int64_t r = g / gpr;
        off = r * ld_x + (g - r * gpr) * 16;
    }
    float v[16];
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if constexpr (kBf16) {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x) + off);
        const uint4 a = p[0], b = p[1];
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + off);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float4 t = p[i];
            v[4 * i] = t.x;
            v[4 * i + 1] = t.y;
            v[4 * i + 2] = t.z;
            v[4 * i + 3] = t.w;
        }
    }
    uint32_t out[3], byte;
    if constexpr (kBf16 && kBits == 3)
        fast_group_bf16<kBits, kMode>(v, w, p_exp, p_negexp, out, byte);
    else
        quantize_group<kBits, kMode>(v, p_exp, p_negexp, out, byte);
    if (gid >= ngroups) return;
    if constexpr (kBits == 6) {
        uint32_t* c = reinterpret_cast<uint32_t*>(codes + gid * 12);
        c[0] = out[0];
        c[1] = out[1];
        c[2] = out[2];
    } else {
        uint16_t* c = reinterpret_cast<uint16_t*>(codes + gid * 6);
        c[0] = (uint16_t)out[0];
        c[1] = (uint16_t)(out[0] >> 16);
        c[2] = (uint16_t)out[1];
    }
    scales[gid] = (uint8_t)byte;
}

// Dequantize: FP codes decode to fp(idx) * s' * 2^E (exact); INT codes to
// the fp32 nearest |q| dn s' / dd (times 2^E), as fma(q, h, q * l) with h =
// dn s'/dd rounded toward zero and l = fl32((dn s' - dd h) * fl32(1/dd)) --
// correctly rounded for every E4M3 s' and |q| (checked exhaustively in exact
// arithmetic), with l >= 0 so that a zero magnitude keeps its sign.
//
// Both forms are one fma: every element is fma(A, HE, A * LE) with A the
// code's signed integer on its grid and (HE, LE) a per-scale-byte pair --
// INT: A = +-|q|, (HE, LE) = (h, l) 2^E; FP: A = +-fp(idx) * kFpDen (an
// integer), (HE, LE) = (s' 2^E / kFpDen, 0), whose product is exact.  Each
// workgroup tabulates A for the 2 x 2^bits (flag, code) pairs and (HE, LE)
// for the 256 scale bytes in LDS while its loads are in flight, so an element
// costs one LDS read, a multiply and an fma.  (A NaN scale byte gives NaN.)
template <int kBits>
struct Fp {
    static constexpr float kDen = kBits == 6 ? 8.0f : 1.0f;  // fp(idx) * kDen is an integer
};

template <int kBits, bool kBf16, bool kContig>
__global__ void __launch_bounds__(kThreads)
dequantize_ifn_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      int64_t rows, int64_t gpr, void* __restrict__ y, int64_t ld_y, float p_exp) {
    using F = Fmt<kBits>;
    constexpr int kCodes = 1 << kBits;
    __shared__ float2 stab[256];
    __shared__ float ctab[2 * kCodes];
    const int64_t ngroups = rows * gpr;
    const int64_t gid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t g = gid < ngroups - 1 ? gid : ngroups - 1;
    uint32_t w[3];
    if constexpr (kBits == 6) {
        const uint32_t* c = reinterpret_cast<const uint32_t*>(codes + g * 12);
        w[0] = c[0];
        w[1] = c[1];
        w[2] = c[2];
    } else {
        const uint16_t* c = reinterpret_cast<const uint16_t*>(codes + g * 6);
        w[0] = (uint32_t)c[0] | ((uint32_t)c[1] << 16);
        w[1] = c[2];
        w[2] = 0;
    }
    const uint32_t b = scales[g];

    // the tables, while the loads are in flight
    {
        const uint32_t t = threadIdx.x;  // scale byte t
        const float sp =
            (t & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : e4m3_value(t & 0x7Fu);
        float2 e;
        if (t & 0x80u) {
            const float num = F::kDn * sp;  // exact
            float h = num / F::kDd;
            if (__builtin_fmaf(-h, F::kDd, num) < 0.0f) h = __uint_as_float(__float_as_uint(h) - 1u);
            const float l = __builtin_fmaf(-h, F::kDd, num) * (1.0f / F::kDd);
            e = make_float2(h * p_exp, l * p_exp);
        } else {
            e = make_float2(sp * p_exp * (1.0f / Fp<kBits>::kDen), 0.0f);
        }
        stab[t] = e;
        if (t < 2u * kCodes) {  // (flag, code) -> signed integer grid value
            const uint32_t c = t & (kCodes - 1u), mag = c & (kCodes / 2 - 1u);
            const float a = (t >= (uint32_t)kCodes) ? (float)mag : F::fp((int)mag) * Fp<kBits>::kDen;
            ctab[t] = (c >> (kBits - 1)) ? -a : a;
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");

    const float2 e = stab[b];
    const uint32_t fbase = (b >> 7) << kBits;  // INT codes in the table's upper half
    float out[16];
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int bit = kBits * i;
        uint32_t c = w[bit >> 5] >> (bit & 31);
        if ((bit & 31) + kBits > 32) c |= w[(bit >> 5) + 1] << (32 - (bit & 31));
        c &= (1u << kBits) - 1u;
        const float a = ctab[fbase + c];
        out[i] = __builtin_fmaf(a, e.x, a * e.y);
    }
    if (gid >= ngroups) return;
    int64_t off;
    if constexpr (kContig) {
        off = gid * 16;
    } else {
        const int64_t r = gid / gpr;
        off = r * ld_y + (gid - r * gpr) * 16;
    }
    if constexpr (kBf16) {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            bf16x2 t;
            t[0] = (__bf16)out[2 * i];
            t[1] = (__bf16)out[2 * i + 1];
            o[i] = __builtin_bit_cast(uint32_t, t);
        }
        uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(y) + off);
        p[0] = make_uint4(o[0], o[1], o[2], o[3]);
        p[1] = make_uint4(o[4], o[5], o[6], o[7]);
    } else {
        float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(y) + off);
#pragma unroll
        for (int i = 0; i < 4; i++)
            p[i] = make_float4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
    }
}

// IF3 dequantize in registers: each lane computes its scale byte's decode
// pair, turns its 16 three-bit codes into E4M3 bytes by one byte permute per
// four codes from an 8-byte table (FP3: s.0.0mm.000 = grid value 2^-6; INT3:
// s.0000.0mm = |q| 2^-9, the table picked by the flag), converts them with
// the hardware fp8 conversion and scales them by fma(m, H, m L) -- the same
// products as the table path, so the same results.  One wave per workgroup,
// and the workgroup order paired on the XCDs as in the IF4 dequantize (two
// neighbouring waves share a 128-byte line of scale bytes).
constexpr int kD3Threads = 64;
template <bool kBf16, bool kContig>
__global__ void __launch_bounds__(kD3Threads)
dequantize_if3_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      int64_t rows, int64_t gpr, void* __restrict__ y, int64_t ld_y, float p_exp) {
    using F = Fmt<3>;
    const int64_t ngroups = rows * gpr;
    const int64_t gid = xcd_paired_block(blockIdx.x, gridDim.x) * kD3Threads + threadIdx.x;
    const int64_t g = gid < ngroups - 1 ? gid : ngroups - 1;
    const uint16_t* c = reinterpret_cast<const uint16_t*>(codes + g * 6);
    const uint32_t w0 = (uint32_t)c[0] | ((uint32_t)c[1] << 16), w1 = c[2];
    const uint32_t b = scales[g];

    const float sp = (b & 0x7Fu) == 0x7Fu ? __uint_as_float(0x7FC00000u) : e4m3_value(b & 0x7Fu);
    const bool isint = (b & 0x80u) != 0;
    float hh, ll;
    {
        const float num = F::kDn * sp;  // exact
        float h = num / F::kDd;
        if (__builtin_fmaf(-h, F::kDd, num) < 0.0f) h = __uint_as_float(__float_as_uint(h) - 1u);
        const float l = __builtin_fmaf(-h, F::kDd, num) * (1.0f / F::kDd);
        hh = isint ? h * (p_exp * 512.0f) : sp * (p_exp * 64.0f);
        ll = isint ? l * (p_exp * 512.0f) : 0.0f;
    }
    const uint32_t tlo = isint ? 0x03020100u : 0x18100800u;
    const uint32_t thi = isint ? 0x83828180u : 0x98908880u;
    auto spread = [](uint32_t t) {  // four 3-bit codes into the low bits of four bytes
        return (t & 7u) | ((t << 5) & 0x700u) | ((t << 10) & 0x70000u) | ((t << 15) & 0x7000000u);
    };
    const uint32_t e[4] = {
        __builtin_amdgcn_perm(thi, tlo, spread(w0)),
        __builtin_amdgcn_perm(thi, tlo, spread(w0 >> 12)),
        __builtin_amdgcn_perm(thi, tlo, spread((w0 >> 24) | (w1 << 8))),
        __builtin_amdgcn_perm(thi, tlo, spread(w1 >> 4)),
    };
    float out[16];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(e[k], 1.0f, false);
        const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(e[k], 1.0f, true);
        const float m[4] = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
        for (int j = 0; j < 4; j++) out[4 * k + j] = __builtin_fmaf(m[j], hh, m[j] * ll);
    }
    if (gid >= ngroups) return;
    int64_t off;
    if constexpr (kContig) {
        off = gid * 16;
    } else {
        const int64_t r = gid / gpr;
        off = r * ld_y + (gid - r * gpr) * 16;
    }
    if constexpr (kBf16) {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            bf16x2 t;
            t[0] = (__bf16)out[2 * i];
            t[1] = (__bf16)out[2 * i + 1];
            o[i] = __builtin_bit_cast(uint32_t, t);
        }
        uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(y) + off);
        p[0] = make_uint4(o[0], o[1], o[2], o[3]);
        p[1] = make_uint4(o[4], o[5], o[6], o[7]);
    } else {
        float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(y) + off);
#pragma unroll
        for (int i = 0; i < 4; i++)
            p[i] = make_float4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
    }
}

template <int kBits, int kMode, bool kBf16>
hipError_t launch_q(const void* x, int64_t rows, int64_t cols, int64_t ld_x, uint8_t* codes,
                    uint8_t* scales, int32_t scale_exp, hipStream_t stream) {
    const int64_t gpr = cols / 16;
    if constexpr (kBits == 6 && kBf16) {
        const int64_t blocks = (rows * gpr + 2 * kQThreads - 1) / (2 * kQThreads);
        if (!launchable(blocks, kQThreads)) return hipErrorInvalidConfiguration;
        const uint16_t* xb = reinterpret_cast<const uint16_t*>(x);
        if (ld_x == cols)
            hipLaunchKernelGGL((quantize_if6_bf16_kernel<kMode, true>), dim3((unsigned)blocks),
                               dim3(kQThreads), 0, stream, xb, rows, gpr, ld_x, codes, scales,
                               pow2f(scale_exp), pow2f(-scale_exp));
        else
            hipLaunchKernelGGL((quantize_if6_bf16_kernel<kMode, false>), dim3((unsigned)blocks),
                               dim3(kQThreads), 0, stream, xb, rows, gpr, ld_x, codes, scales,
                               pow2f(scale_exp), pow2f(-scale_exp));
        return hipGetLastError();
    }
    const int64_t blocks = (rows * gpr + kQThreads - 1) / kQThreads;
    if (!launchable(blocks, kQThreads)) return hipErrorInvalidConfiguration;
    if (ld_x == cols)
        hipLaunchKernelGGL((quantize_ifn_kernel<kBits, kMode, kBf16, true>), dim3((unsigned)blocks),
                           dim3(kQThreads), 0, stream, x, rows, gpr, ld_x, codes, scales,
                           pow2f(scale_exp), pow2f(-scale_exp));
    else
        hipLaunchKernelGGL((quantize_ifn_kernel<kBits, kMode, kBf16, false>),
                           dim3((unsigned)blocks), dim3(kQThreads), 0, stream, x, rows, gpr, ld_x,
                           codes, scales, pow2f(scale_exp), pow2f(-scale_exp));
    return hipGetLastError();
}

template <int kBits>
hipError_t dispatch_q(const void* x, int bf16, int64_t rows, int64_t cols, int64_t ld_x,
                      uint8_t* codes, uint8_t* scales, int32_t scale_exp, int mode,
                      hipStream_t stream) {
#define IF4_QN(M, B) launch_q<kBits, M, B>(x, rows, cols, ld_x, codes, scales, scale_exp, stream)
    if (bf16) {
        if (mode == 1) return IF4_QN(1, true);
        if (mode == 2) return IF4_QN(2, true);
        return IF4_QN(0, true);
    }
    if (mode == 1) return IF4_QN(1, false);
    if (mode == 2) return IF4_QN(2, false);
    return IF4_QN(0, false);
#undef IF4_QN
}

template <int kBits>
hipError_t dispatch_dq(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                       int32_t scale_exp, void* y, int bf16, int64_t ld_y, hipStream_t stream) {
    const int64_t gpr = cols / 16;
    const bool contig = ld_y == cols;
    if constexpr (kBits == 3) {  // registers only
        const int64_t blocks = (rows * gpr + kD3Threads - 1) / kD3Threads;
        if (!launchable(blocks, kD3Threads)) return hipErrorInvalidConfiguration;
#define IF4_DQ3(B, C)                                                                          \
        hipLaunchKernelGGL((dequantize_if3_kernel<B, C>), dim3((unsigned)blocks),              \
                           dim3(kD3Threads), 0, stream, codes, scales, rows, gpr, y, ld_y,     \
                           pow2f(scale_exp))
        if (bf16) {
            if (contig) IF4_DQ3(true, true);
            else IF4_DQ3(true, false);
        } else {
            if (contig) IF4_DQ3(false, true);
            else IF4_DQ3(false, false);
        }
#undef IF4_DQ3
    } else {  // per-workgroup LDS tables
        const int64_t blocks = (rows * gpr + kThreads - 1) / kThreads;
        if (!launchable(blocks, kThreads)) return hipErrorInvalidConfiguration;
#define IF4_DQN(B, C)                                                                          \
        hipLaunchKernelGGL((dequantize_ifn_kernel<kBits, B, C>), dim3((unsigned)blocks),       \
                           dim3(kThreads), 0, stream, codes, scales, rows, gpr, y, ld_y,       \
                           pow2f(scale_exp))
        if (bf16) {
            if (contig) IF4_DQN(true, true);
            else IF4_DQN(true, false);
        } else {
            if (contig) IF4_DQN(false, true);
            else IF4_DQN(false, false);
        }
#undef IF4_DQN
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_ifn(int bits, const void* x, int bf16, int64_t rows, int64_t cols,
                               int64_t ld_x, uint8_t* codes, uint8_t* scales, int32_t scale_exp,
                               int mode, hipStream_t stream) {
    if (bits == 6)
        return dispatch_q<6>(x, bf16, rows, cols, ld_x, codes, scales, scale_exp, mode, stream);
    return dispatch_q<3>(x, bf16, rows, cols, ld_x, codes, scales, scale_exp, mode, stream);
}

hipError_t launch_dequantize_ifn(int bits, const uint8_t* codes, const uint8_t* scales,
                                 int64_t rows, int64_t cols, int32_t scale_exp, void* y, int bf16,
                                 int64_t ld_y, hipStream_t stream) {
    if (bits == 6)
        return dispatch_dq<6>(codes, scales, rows, cols, scale_exp, y, bf16, ld_y, stream);
    return dispatch_dq<3>(codes, scales, rows, cols, scale_exp, y, bf16, ld_y, stream);
}

}  // namespace if4
