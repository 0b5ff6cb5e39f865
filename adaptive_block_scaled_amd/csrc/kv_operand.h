// Device helpers that decode the KV cache's IF4 groups to fp16 MFMA operands
// (HIP translation units only).
//
// A code nibble becomes the high byte of an fp16 number by shifts and masks:
// FP4 s.e1e0.m -> s.000e1e0.m (the fp16 value c * 2^-14, exact, its e = 0
// codes being fp16 subnormals), INT4 s.mmm -> s.0000.mmm (|q| * 2^-16).
// v_perm_b32 puts two such bytes into a pair of fp16 numbers, and one packed
// multiply by the group's multiplier -- s' * 2^5 for FP4, fl16(6 s'/7 * 2^7)
// for INT4 -- leaves every operand as (decoded value) * 2^-9: FP4 exactly,
// INT4 with one fp16 rounding of |q| * fl16(6 s'/7).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace if4 {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pk_mul(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t,
                              __builtin_bit_cast(half2v, a) * __builtin_bit_cast(half2v, b));
}

// m ? a : b, bit by bit: one v_bitop3_b32 (truth table over (a, b, m)).
__device__ __forceinline__ uint32_t bit_select(uint32_t a, uint32_t b, uint32_t m) {
    return __builtin_amdgcn_bitop3_b32(a, b, m, 0xE4);
}

// Group multiplier (both fp16 halves) and nibble shift (both 16-bit halves)
// of a scale byte.
struct GroupScale {
    uint32_t sig2;
    uint32_t sh2;
};

// The tables that every workgroup keeps in LDS: a lookup is one ds_read_b64
// in place of about eight VALU instructions.  A NaN scale byte gives a NaN
// multiplier in K's table -- the key's scores are NaN and reach the rows that
// see it -- and zero in V's, where a product with a hidden key's zero
// probability would turn NaN; V's NaN are put in afterwards (poison_rows).
constexpr int kScaleTableBytes = 2 * 256 * 8;

__device__ __forceinline__ void fill_scale_tables(uint2* tables, int tid, int threads) {
    for (int b = tid; b < 256; b += threads) {
        const float sp = __builtin_amdgcn_cvt_scalef32_f32_fp8((uint32_t)b & 0x7Fu, 1.0f, 0);
        const bool int4 = (b & 0x80) != 0;
        const float sig = sp * (int4 ? 0.857142866f * 128.0f : 32.0f);
        const uint32_t h16 = __builtin_bit_cast(uint16_t, (_Float16)sig);
        const uint32_t sig2 = h16 | (h16 << 16), sh2 = int4 ? 0u : 0x00010001u;
        tables[b] = make_uint2(sig2, sh2);
        tables[256 + b] = make_uint2((b & 0x7F) == 0x7F ? 0u : sig2, sh2);
    }
}

__device__ __forceinline__ GroupScale k_scale(const uint2* tables, uint32_t byte) {
    const uint2 v = tables[byte];
    return {v.x, v.y};
}
__device__ __forceinline__ GroupScale v_scale(const uint2* tables, uint32_t byte) {
    const uint2 v = tables[256 + byte];
    return {v.x, v.y};
}

constexpr uint32_t kLoNibbles = 0x0F0F0F0Fu;

// fp16 high bytes of the even (he) and odd (ho) elements of 8 nibbles.
__device__ __forceinline__ void high_bytes(uint32_t w, uint32_t shifted, uint32_t masked,
                                           uint32_t& he, uint32_t& ho) {
    const uint32_t sign = w ^ masked;  // bits 3 and 7 of each byte
    he = bit_select(shifted, sign << 4, kLoNibbles);
    ho = bit_select(shifted >> 4, sign, kLoNibbles);
}

// byte i of lo and byte j of hi as the high bytes of a pair of fp16 numbers
template <int i, int j>
__device__ __forceinline__ uint32_t pair_of(uint32_t hi, uint32_t lo) {
    return __builtin_amdgcn_perm(hi, lo, 0x040C000Cu + ((uint32_t)j << 24) + ((uint32_t)i << 8));
}

// K: 8 consecutive elements of one group as one operand.
__device__ __forceinline__ half8 decode_k_word(uint32_t w, GroupScale s) {
    const uint32_t m = w & 0x77777777u;
    uint32_t he, ho;
    high_bytes(w, m << (s.sh2 & 31u), m, he, ho);
    uint4 r;
    r.x = pk_mul(pair_of<0, 0>(ho, he), s.sig2);
    r.y = pk_mul(pair_of<1, 1>(ho, he), s.sig2);
    r.z = pk_mul(pair_of<2, 2>(ho, he), s.sig2);
    r.w = pk_mul(pair_of<3, 3>(ho, he), s.sig2);
    return __builtin_bit_cast(half8, r);
}

// V: one piece (D/16 dims) of four consecutive tokens, words as they lie in
// the cache and the tokens' four scale bytes in one word.  out[d][0] holds dim
// d of tokens 0 and 1, out[d][1] of tokens 2 and 3: pairs of tokens come out
// of the same v_perm that K spends on pairs of dims, so V needs no transposition.
template <int D>
__device__ __forceinline__ void decode_v_piece(const uint32_t (&w)[D / 32], uint32_t scales,
                                               const uint2* tables, uint32_t (&out)[D / 16][2]) {
    GroupScale s[4];
#pragma unroll
    for (int t = 0; t < 4; t++) s[t] = v_scale(tables, (scales >> (8 * t)) & 0xFFu);
#pragma unroll
    for (int p = 0; p < 2; p++) {  // tokens 2p, 2p + 1
        const uint32_t sig = bit_select(s[2 * p].sig2, s[2 * p + 1].sig2, 0xFFFFu);
        if constexpr (D == 64) {
            // both tokens' 4 nibbles share a word
            typedef uint16_t us2 __attribute__((ext_vector_type(2)));
            const uint32_t sh = bit_select(s[2 * p].sh2, s[2 * p + 1].sh2, 0xFFFFu);
            const uint32_t m = w[p] & 0x77777777u;
            const uint32_t ms = __builtin_bit_cast(
                uint32_t, (us2)(__builtin_bit_cast(us2, m) << __builtin_bit_cast(us2, sh)));
            uint32_t he, ho;
            high_bytes(w[p], ms, m, he, ho);
            out[0][p] = pk_mul(__builtin_amdgcn_perm(he, he, 0x020C000Cu), sig);
            out[1][p] = pk_mul(__builtin_amdgcn_perm(ho, ho, 0x020C000Cu), sig);
            out[2][p] = pk_mul(__builtin_amdgcn_perm(he, he, 0x030C010Cu), sig);
            out[3][p] = pk_mul(__builtin_amdgcn_perm(ho, ho, 0x030C010Cu), sig);
        } else {
            constexpr int W = D / 128;  // words per token
#pragma unroll
            for (int k = 0; k < W; k++) {
                uint32_t he[2], ho[2];
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    const uint32_t x = w[(2 * p + t) * W + k], m = x & 0x77777777u;
                    high_bytes(x, m << (s[2 * p + t].sh2 & 31u), m, he[t], ho[t]);
                }
                out[8 * k + 0][p] = pk_mul(pair_of<0, 0>(he[1], he[0]), sig);
                out[8 * k + 1][p] = pk_mul(pair_of<0, 0>(ho[1], ho[0]), sig);
                out[8 * k + 2][p] = pk_mul(pair_of<1, 1>(he[1], he[0]), sig);
                out[8 * k + 3][p] = pk_mul(pair_of<1, 1>(ho[1], ho[0]), sig);
                out[8 * k + 4][p] = pk_mul(pair_of<2, 2>(he[1], he[0]), sig);
                out[8 * k + 5][p] = pk_mul(pair_of<2, 2>(ho[1], ho[0]), sig);
                out[8 * k + 6][p] = pk_mul(pair_of<3, 3>(he[1], he[0]), sig);
                out[8 * k + 7][p] = pk_mul(pair_of<3, 3>(ho[1], ho[0]), sig);
            }
        }
    }
}

// Whether any of four scale bytes is NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t scales) {
    return ((scales & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

}  // namespace if4
