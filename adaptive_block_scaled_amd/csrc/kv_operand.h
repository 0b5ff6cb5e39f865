// Device helpers that decode the KV cache's IF4 groups to fp16 MFMA operands
// (HIP translation units only).
//
// A code nibble becomes the high byte of an fp16 number by shifts and masks:
// FP4 s.e1e0.m -> s.000e1e0.m (the fp16 value c * 2^-14, exact, its e = 0
// codes being fp16 subnormals), INT4 s.mmm -> s.0000.mmm (|q| * 2^-16).
// v_perm_b32 puts two such bytes into a pair of fp16 numbers, and one packed
// multiply by the group's multiplier -- s' * 2^5 for FP4, fl16(6 s'/7 * 2^7)
// for INT4 -- leaves every operand as (decoded value) * 2^-9: FP4 exactly,
// INT4 with one fp16 rounding of |q| * fl16(6 s'/7): 2^-11 of the value, and not finer
// than 2^-15 2^E, where the operand is subnormal (values below 2^-5 2^E; E is set so that a
// tensor's largest reach some 2^11).  The matrix cores take fp16 and bf16 at the same
// rate, and bf16 would keep three bits less of the INT4 values.
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
// probability would turn NaN; V's NaN are put in afterwards (the kernels' `poison`).
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

constexpr uint32_t kLoNibbles = 0x0F0F0F0Fu, kMagnitudes = 0x77777777u;

// fp16 high bytes of the even (he) and odd (ho) elements of two words of 8
// nibbles, in three stages of four or five instructions each, so that a caller
// can put other work between them.  The shifts by 4 are 64-bit ones, single
// instructions on gfx950: what they carry from word to word lands in masked-off
// bits.  `four` is 4, kept opaque (a constant amount is split into 32-bit shifts).
struct HighBytes {
    uint64_t shifted, low, up;  // magnitudes at their places, down by 4; signs up by 4
    uint32_t g[2];              // bits 3 and 7 of each byte
    // (stage 0 makes `shifted` out of w & kMagnitudes, by scale)
    __device__ __forceinline__ void spread(const uint32_t (&w)[2], uint32_t four) {
        g[0] = w[0] & ~kMagnitudes;
        g[1] = w[1] & ~kMagnitudes;
        low = shifted >> four;
        up = ((uint64_t)g[1] << 32 | g[0]) << four;
    }
    __device__ __forceinline__ void merge(uint32_t& he0, uint32_t& he1, uint32_t& ho0,
                                          uint32_t& ho1) const {
        he0 = bit_select((uint32_t)shifted, (uint32_t)up, kLoNibbles);
        he1 = bit_select((uint32_t)(shifted >> 32), (uint32_t)(up >> 32), kLoNibbles);
        ho0 = bit_select((uint32_t)low, g[0], kLoNibbles);
        ho1 = bit_select((uint32_t)(low >> 32), g[1], kLoNibbles);
    }
};

// byte i of lo and byte j of hi as the high bytes of a pair of fp16 numbers
template <int i, int j>
__device__ __forceinline__ uint32_t pair_of(uint32_t hi, uint32_t lo) {
    return __builtin_amdgcn_perm(hi, lo, 0x040C000Cu + ((uint32_t)j << 24) + ((uint32_t)i << 8));
}

// K: one group (two words), unpacked to fp16 high bytes first, then either half
// as an operand of 8 consecutive elements.
struct KGroup {
    uint32_t he[2], ho[2], sig;
    HighBytes bytes;
    template <int stage>
    __device__ __forceinline__ void unpack_stage(uint32_t w0, uint32_t w1, GroupScale s,
                                                 uint32_t four) {
        if constexpr (stage == 0) {
            const uint64_t m = (uint64_t)(w1 & kMagnitudes) << 32 | (w0 & kMagnitudes);
            bytes.shifted = m << (s.sh2 & 63u);
        } else if constexpr (stage == 1) {
            const uint32_t w[2] = {w0, w1};
            bytes.spread(w, four);
        } else {
            bytes.merge(he[0], he[1], ho[0], ho[1]);
            sig = s.sig2;
        }
    }
    __device__ __forceinline__ void unpack(uint32_t w0, uint32_t w1, GroupScale s, uint32_t four) {
        unpack_stage<0>(w0, w1, s, four);
        unpack_stage<1>(w0, w1, s, four);
        unpack_stage<2>(w0, w1, s, four);
    }
    // elements 8 i + 2 j and 8 i + 2 j + 1
    template <int i, int j>
    __device__ __forceinline__ uint32_t pair() const {
        return pk_mul(pair_of<j, j>(ho[i], he[i]), sig);
    }
    template <int i>
    __device__ __forceinline__ half8 operand() const {
        return __builtin_bit_cast(half8,
                                  make_uint4(pair<i, 0>(), pair<i, 1>(), pair<i, 2>(), pair<i, 3>()));
    }
};

// V: one piece (D/16 dims) of four consecutive tokens.  Split in two, so that
// the codes' registers are free for the next loads before the operands exist:
// first the fp16 high bytes and the multipliers of token pairs, then any
// dim's operand half.  A pair of tokens comes out of the same v_perm that K
// spends on a pair of dims, so V needs no transposition.
template <int D>
struct VPiece {
    static constexpr int kWords = D / 32;   // even and odd bytes, one word each
    uint32_t he[kWords], ho[kWords];
    uint32_t sig[2];                        // tokens 0 and 1, tokens 2 and 3
    HighBytes bytes;

    // The four tokens' scales, from their four scale bytes.
    __device__ static __forceinline__ void look_up(const uint2* tables, uint32_t scales,
                                                   GroupScale (&s)[4]) {
#pragma unroll
        for (int t = 0; t < 4; t++) s[t] = v_scale(tables, (scales >> (8 * t)) & 0xFFu);
    }
    // w: words as they lie in the cache
    __device__ __forceinline__ void unpack(const uint32_t (&w)[D / 32], const GroupScale (&s)[4],
                                           uint32_t four) {
        each_word_pair<0>(w, s, four);
    }
    template <int i>
    __device__ __forceinline__ void each_word_pair(const uint32_t (&w)[D / 32],
                                                   const GroupScale (&s)[4], uint32_t four) {
        if constexpr (i < kWords / 2) {
            unpack_words<i>(w, s, four);
            each_word_pair<i + 1>(w, s, four);
        }
    }
    // words 2i and 2i + 1; the multipliers with the first
    template <int i>
    __device__ __forceinline__ void unpack_words(const uint32_t (&w)[D / 32],
                                                 const GroupScale (&s)[4], uint32_t four) {
        unpack_stage<i, 0>(w, s, four);
        unpack_stage<i, 1>(w, s, four);
        unpack_stage<i, 2>(w, s, four);
    }
    template <int i, int stage>
    __device__ __forceinline__ void unpack_stage(const uint32_t (&w)[D / 32],
                                                 const GroupScale (&s)[4], uint32_t four) {
        const uint32_t x[2] = {w[2 * i], w[2 * i + 1]};
        if constexpr (stage == 0) {
            if constexpr (i == 0) {
#pragma unroll
                for (int p = 0; p < 2; p++)
                    sig[p] = bit_select(s[2 * p].sig2, s[2 * p + 1].sig2, 0xFFFFu);
            }
            const uint32_t m[2] = {x[0] & kMagnitudes, x[1] & kMagnitudes};
            uint32_t sh[2];
            if constexpr (D == 64) {
                // a word holds two tokens' 4 nibbles: 16-bit shifts
                typedef uint16_t us2 __attribute__((ext_vector_type(2)));
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const uint32_t by = bit_select(s[2 * j].sh2, s[2 * j + 1].sh2, 0xFFFFu);
                    sh[j] = __builtin_bit_cast(uint32_t, (us2)(__builtin_bit_cast(us2, m[j])
                                                               << __builtin_bit_cast(us2, by)));
                }
            } else {
                constexpr int per = D / 128;  // words per token
                sh[0] = m[0] << (s[2 * i / per].sh2 & 31u);
                sh[1] = m[1] << (s[(2 * i + 1) / per].sh2 & 31u);
            }
            bytes.shifted = (uint64_t)sh[1] << 32 | sh[0];
        } else if constexpr (stage == 1) {
            bytes.spread(x, four);
        } else {
            bytes.merge(he[2 * i], he[2 * i + 1], ho[2 * i], ho[2 * i + 1]);
        }
    }
    // dim d of tokens 2p and 2p + 1
    template <int d, int p>
    __device__ __forceinline__ uint32_t pair() const {
        const uint32_t* const src = d & 1 ? ho : he;
        if constexpr (D == 64) {
            constexpr int b = d / 2;
            return pk_mul(__builtin_amdgcn_perm(src[p], src[p], 0x020C000Cu + b * 0x01000100u),
                          sig[p]);
        } else {
            constexpr int per = D / 128, k = d / 8, b = d % 8 / 2;
            return pk_mul(pair_of<b, b>(src[(2 * p + 1) * per + k], src[2 * p * per + k]), sig[p]);
        }
    }
};

// Whether any of four scale bytes is NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t scales) {
    return ((scales & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

}  // namespace if4
