// Device helpers that decode IF4 groups to fp16 MFMA operands (HIP translation
// units only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace if4 {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pk_mul(uint32_t a, uint32_t b) {
    half2v x = __builtin_bit_cast(half2v, a);
    half2v y = __builtin_bit_cast(half2v, b);
    return __builtin_bit_cast(uint32_t, x * y);
}

// Group multiplier (both fp16 halves) and nibble shift from a scale byte.
struct GroupScale {
    uint32_t sig2;
    uint32_t sh;
};

// s' comes from the hardware E4M3 conversion (exact; NaN for 0x7F, which
// then poisons the group's products).  FP4: s' * 2^5 (exact in fp16);
// INT4: fl16(fl32(s' * fl32(6/7))) * 2^7, computed as one fp32 product
// (power-of-two factors do not change the roundings).
__device__ __forceinline__ GroupScale group_scale(uint32_t b) {
    const float sp = __builtin_amdgcn_cvt_scalef32_f32_fp8(b & 0x7Fu, 1.0f, 0);
    const bool int4 = (b & 0x80u) != 0;
    const float sig = sp * (int4 ? 0.857142866f * 128.0f : 32.0f);
    const uint32_t h16 = __builtin_bit_cast(uint16_t, (_Float16)sig);
    GroupScale s;
    s.sig2 = h16 | (h16 << 16);
    s.sh = int4 ? 0u : 1u;
    return s;
}

// Decode the two code words of one group (w0: elements 0-7, w1: elements
// 8-15; element 2j in the low nibble of byte j) into 16 fp16 operands in K
// order.  Per word, two bytes hold the fp16 high bytes of its even and odd
// elements: he = [sign | magnitude << sh] of the low nibbles, ho the same
// for the high nibbles.  The magnitudes are shifted as one 64-bit word per
// group (the shift moves no bit across a nibble: bit 3 of every nibble is
// cleared first), and each byte is assembled by one bit-field insert under
// the mask 0x0F0F0F0F: the low half from the shifted magnitudes, the high
// half from the sign bits (moved up by 4 for the even elements; the bits a
// 64-bit shift carries across the word boundary land in masked-off
// positions).  27 VALU instructions per group.
// m ? a : b, bit by bit: one v_bitop3_b32 (truth table over (a, b, m)).
__device__ __forceinline__ uint32_t bit_select(uint32_t a, uint32_t b, uint32_t m) {
    return __builtin_amdgcn_bitop3_b32(a, b, m, 0xE4);
}
// 64-bit shifts by 4 as single instructions (full rate on gfx950).  The
// amount comes in as `four`, a value the compiler cannot fold: a constant
// amount makes it split each shift into two 32-bit operations, and writing the
// instruction as inline asm instead costs a hazard s_nop after every one.
__device__ __forceinline__ uint64_t shr64_by4(uint64_t x, uint32_t four) { return x >> four; }
__device__ __forceinline__ uint64_t shl64_by4(uint64_t x, uint32_t four) { return x << four; }
__device__ __forceinline__ void decode_group(uint32_t w0, uint32_t w1, GroupScale s, half8& o0,
                                             half8& o1, uint32_t four) {
    constexpr uint32_t kLo = 0x0F0F0F0Fu;  // low nibble of every byte
    const uint32_t m0 = w0 & 0x77777777u, m1 = w1 & 0x77777777u;
    const uint64_t ms = ((uint64_t)m1 << 32 | m0) << s.sh;
    const uint64_t mr = shr64_by4(ms, four);
    const uint32_t g0 = w0 ^ m0, g1 = w1 ^ m1;  // sign bits (bits 3 and 7 of each byte)
    const uint64_t g4 = shl64_by4((uint64_t)g1 << 32 | g0, four);
    const uint32_t he0 = bit_select((uint32_t)ms, (uint32_t)g4, kLo);
    const uint32_t he1 = bit_select((uint32_t)(ms >> 32), (uint32_t)(g4 >> 32), kLo);
    const uint32_t ho0 = bit_select((uint32_t)mr, g0, kLo);
    const uint32_t ho1 = bit_select((uint32_t)(mr >> 32), g1, kLo);
    // v_perm: byte j of he -> bits 15:8, byte j of ho -> bits 31:24, zeros below
    uint4 r0, r1;
    r0.x = pk_mul(__builtin_amdgcn_perm(ho0, he0, 0x040C000Cu), s.sig2);
    r0.y = pk_mul(__builtin_amdgcn_perm(ho0, he0, 0x050C010Cu), s.sig2);
    r0.z = pk_mul(__builtin_amdgcn_perm(ho0, he0, 0x060C020Cu), s.sig2);
    r0.w = pk_mul(__builtin_amdgcn_perm(ho0, he0, 0x070C030Cu), s.sig2);
    r1.x = pk_mul(__builtin_amdgcn_perm(ho1, he1, 0x040C000Cu), s.sig2);
    r1.y = pk_mul(__builtin_amdgcn_perm(ho1, he1, 0x050C010Cu), s.sig2);
    r1.z = pk_mul(__builtin_amdgcn_perm(ho1, he1, 0x060C020Cu), s.sig2);
    r1.w = pk_mul(__builtin_amdgcn_perm(ho1, he1, 0x070C030Cu), s.sig2);
    o0 = __builtin_bit_cast(half8, r0);
    o1 = __builtin_bit_cast(half8, r1);
}

}  // namespace if4
