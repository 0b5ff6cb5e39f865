// Writing the paged IF4 KV cache and reading it back, for gfx950.  The layouts
// are those of include/if4_kv.h.
//
// One lane owns one group of 16 values of one (token, head), of K or of V, so
// that encode and decode stay in its registers (if4_encode.h, if4_decode.h)
// and a wave's 64 groups are those of 64 / (D/16) consecutive tokens.
// Bound by memory: per value 2 or 4 bytes and 4.5 bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "if4_decode.h"
#include "if4_encode.h"
#include "if4_internal.h"
#include "kv_internal.h"

namespace if4 {
namespace {

constexpr int kThreads = 256;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Where a group (slot, head, group g) lives.  K: a row of D/2 code bytes and
// D/16 scale bytes per (page, head, offset).  V: the group's 16/(D/16)
// pieces lie 16 tokens apart, its scale bytes token-innermost.
template <int D>
struct Place {
    int64_t row;  // (page * kv_heads + head) * page_size + offset
    int64_t tile;
    int tok;
    // (all tiles of a cache, pages x kv heads x tiles of a page, fit 31 bits)
    __device__ __forceinline__ Place(int64_t slot, int head, int kv_heads, const Divisor& tiles) {
        const uint32_t t = (uint32_t)(slot >> 4), page = tiles.into(t);
        tile = (page * kv_heads + head) * tiles.n + (t - page * tiles.n);
        tok = (int)(slot & 15);
        row = tile * 16 + tok;
    }
    __device__ __forceinline__ int64_t k_code(int g) const { return row * (D / 2) + g * 8; }
    __device__ __forceinline__ int64_t k_scale(int g) const { return row * (D / 16) + g; }
    // code byte offset of piece p
    __device__ __forceinline__ int64_t v_code(int p) const {
        return tile * (8 * D) + (p * 16 + tok) * (D / 32);
    }
    __device__ __forceinline__ int64_t v_scale(int g) const { return tile * D + g * 16 + tok; }
};

template <int D>
__device__ __forceinline__ void store_v(uint8_t* codes, const Place<D>& at, int g, uint32_t lo,
                                        uint32_t hi) {
    if constexpr (D == 64) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t w = i < 2 ? lo : hi;
            *reinterpret_cast<uint16_t*>(codes + at.v_code(4 * g + i)) =
                (uint16_t)(w >> (16 * (i & 1)));
        }
    } else if constexpr (D == 128) {
        *reinterpret_cast<uint32_t*>(codes + at.v_code(2 * g)) = lo;
        *reinterpret_cast<uint32_t*>(codes + at.v_code(2 * g + 1)) = hi;
    } else {
        *reinterpret_cast<uint2*>(codes + at.v_code(g)) = make_uint2(lo, hi);
    }
}

template <int D>
__device__ __forceinline__ uint2 load_v(const uint8_t* codes, const Place<D>& at, int g) {
    if constexpr (D == 64) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            h[i] = *reinterpret_cast<const uint16_t*>(codes + at.v_code(4 * g + i));
        return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    } else if constexpr (D == 128) {
        return make_uint2(*reinterpret_cast<const uint32_t*>(codes + at.v_code(2 * g)),
                          *reinterpret_cast<const uint32_t*>(codes + at.v_code(2 * g + 1)));
    } else {
        return *reinterpret_cast<const uint2*>(codes + at.v_code(g));
    }
}

struct AppendArgs {
    const void* x[2];
    int64_t stride_token[2], stride_head[2];
    const int64_t* slots;
    uint8_t* codes[2];
    uint8_t* scales[2];
    float p_exp[2], p_negexp[2];
    int64_t tokens, nslots;
    Divisor tiles;  // of 16 tokens in a page
    int kv_heads;
};

// Quantize as written.  blockIdx.z: K or V; y: head; x: run of kThreads / (D/16)
// tokens.  Small calls are launch and latency (64 tokens of 8 heads of 128: 3.6 us,
// slot and values asked for together), large ones memory: 8192 tokens (43 MB moved)
// 12.5 us = 3.4 TB/s, the start and tail of a short kernel among them; one wave per
// workgroup 13.0, heads before tokens 13.2, loads past the caches 13.5.
template <int D, bool kBf16, int kMode>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs p) {
    constexpr int G = D / 16;
    const int part = blockIdx.z, head = blockIdx.y;
    const int g = threadIdx.x % G;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G;
    if (t >= p.tokens) return;
    const int64_t slot = p.slots[t];
    float v[16];
    load_group<kBf16>(p.x[part], t * p.stride_token[part] + head * p.stride_head[part] + g * 16,
                      v);
    if (slot < 0 || slot >= p.nslots) return;
    uint32_t lo, hi, byte;
    if constexpr (kBf16)
        fast_group<kMode>(v, p.p_exp[part], p.p_negexp[part], lo, hi, byte);
    else
        exact_group<kMode>(v, p.p_exp[part], p.p_negexp[part], lo, hi, byte);
    const Place<D> at(slot, head, p.kv_heads, p.tiles);
    if (part == 0) {
        *reinterpret_cast<uint2*>(p.codes[0] + at.k_code(g)) = make_uint2(lo, hi);
        p.scales[0][at.k_scale(g)] = (uint8_t)byte;
    } else {
        store_v<D>(p.codes[1], at, g, lo, hi);
        p.scales[1][at.v_scale(g)] = (uint8_t)byte;
    }
}

struct ReadArgs {
    const uint8_t* codes[2];
    const uint8_t* scales[2];
    void* y[2];
    const int64_t* slots;
    float p_exp[2];
    int64_t tokens, nslots;
    Divisor tiles;  // of 16 tokens in a page
    int kv_heads;
};

// Stores past the caches that follow one another at once: the compiler is told
// that all values are needed before the first.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void store_all(void* to, u32x4 a, u32x4 b) {
    asm volatile("" : "+v"(a), "+v"(b));
    u32x4* const q = reinterpret_cast<u32x4*>(to);
    __builtin_nontemporal_store(a, q);
    __builtin_nontemporal_store(b, q + 1);
}
__device__ __forceinline__ void store_all(void* to, u32x4 a, u32x4 b, u32x4 c, u32x4 d) {
    asm volatile("" : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
    u32x4* const q = reinterpret_cast<u32x4*>(to);
    __builtin_nontemporal_store(a, q);
    __builtin_nontemporal_store(b, q + 1);
    __builtin_nontemporal_store(c, q + 2);
    __builtin_nontemporal_store(d, q + 3);
}

// blockIdx.z: K or V; x: run of kThreads / (D/16) tokens, head fastest, so that
// neighbouring workgroups write neighbouring heads of the same tokens.  The stores
// leave nothing of the output in the caches, which would have to be written back
// from them before the next call's; a lane's follow one another at once, or half
// lines reach the memory.  A context of 32768 tokens of 8 heads of 128 (172 MB
// moved), 3000 calls in a row: 33.8 us = 5.1 TB/s, the rate of a large copy;
// ordinary stores 47.9 us, stores apart 49.0; two waves per workgroup 33.3, one 47
// (stores apart), eight 34.6; 8 values per lane, so that a wave stores 1 KB in one
// piece, 39 us (half as much in flight).
template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadArgs p) {
    constexpr int G = D / 16;
    const int part = blockIdx.z;
    const uint32_t run = blockIdx.x / p.kv_heads;
    const int head = blockIdx.x - run * p.kv_heads;
    const int g = threadIdx.x % G;
    const int64_t t = (int64_t)run * (kThreads / G) + threadIdx.x / G;
    if (t >= p.tokens) return;
    const int64_t slot = p.slots[t];
    uint2 w = make_uint2(0u, 0u);
    uint32_t byte = 0;
    if (slot >= 0 && slot < p.nslots) {
        const Place<D> at(slot, head, p.kv_heads, p.tiles);
        if (part == 0) {
            w = *reinterpret_cast<const uint2*>(p.codes[0] + at.k_code(g));
            byte = p.scales[0][at.k_scale(g)];
        } else {
            w = load_v<D>(p.codes[1], at, g);
            byte = p.scales[1][at.v_scale(g)];
        }
    }
    const Entry e = make_entry(byte, p.p_exp[part]);
    float out[16];
    decode_word(w.x, e, out);
    decode_word(w.y, e, out + 8);
    const int64_t off = (t * p.kv_heads + head) * D + g * 16;
    if constexpr (kBf16) {
        bf16x8 b[2];
#pragma unroll
        for (int i = 0; i < 16; i++) b[i >> 3][i & 7] = (__bf16)out[i];
        store_all(reinterpret_cast<uint16_t*>(p.y[part]) + off,
                  __builtin_bit_cast(u32x4, b[0]), __builtin_bit_cast(u32x4, b[1]));
    } else {
        f32x4 f[4];
#pragma unroll
        for (int i = 0; i < 16; i++) f[i >> 2][i & 3] = out[i];
        store_all(reinterpret_cast<float*>(p.y[part]) + off, __builtin_bit_cast(u32x4, f[0]),
                  __builtin_bit_cast(u32x4, f[1]), __builtin_bit_cast(u32x4, f[2]),
                  __builtin_bit_cast(u32x4, f[3]));
    }
}

template <int D, bool kBf16>
void append_mode(const AppendArgs& p, int mode, dim3 grid, hipStream_t stream) {
    if (mode == IF4_MODE_ADAPTIVE)
        hipLaunchKernelGGL((append_kernel<D, kBf16, 0>), grid, dim3(kThreads), 0, stream, p);
    else if (mode == IF4_MODE_FORCE_FP4)
        hipLaunchKernelGGL((append_kernel<D, kBf16, 1>), grid, dim3(kThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((append_kernel<D, kBf16, 2>), grid, dim3(kThreads), 0, stream, p);
}

template <int D>
hipError_t append(const if4_kv_cache& c, const AppendArgs& p, int bf16, int mode,
                  hipStream_t stream) {
    constexpr int per = kThreads / (D / 16);
    const int64_t runs = (p.tokens + per - 1) / per;
    if (runs > 0x7FFFFFFF) return hipErrorInvalidValue;
    const dim3 grid((unsigned)runs, (unsigned)c.kv_heads, 2);
    if (bf16)
        append_mode<D, true>(p, mode, grid, stream);
    else
        append_mode<D, false>(p, mode, grid, stream);
    return hipGetLastError();
}

template <int D>
hipError_t read(const if4_kv_cache& c, const ReadArgs& p, int bf16, hipStream_t stream) {
    constexpr int per = kThreads / (D / 16);
    const int64_t runs = (p.tokens + per - 1) / per;
    if (runs > 0x7FFFFFFF / c.kv_heads) return hipErrorInvalidValue;
    const dim3 grid((unsigned)(runs * c.kv_heads), 1, 2);
    if (bf16)
        hipLaunchKernelGGL((read_kernel<D, true>), grid, dim3(kThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((read_kernel<D, false>), grid, dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const if4_kv_cache& c, const void* k, const void* v, int bf16,
                            int64_t tokens, const int64_t (&strides)[4], const int64_t* slots,
                            int mode, hipStream_t stream) {
    AppendArgs p;
    p.x[0] = k;
    p.x[1] = v;
    for (int i = 0; i < 2; i++) {
        p.stride_token[i] = strides[2 * i];
        p.stride_head[i] = strides[2 * i + 1];
        const int e = i ? c.v_exp : c.k_exp;
        p.p_exp[i] = pow2f(e);
        p.p_negexp[i] = pow2f(-e);
    }
    p.slots = slots;
    p.codes[0] = c.k_codes;
    p.codes[1] = c.v_codes;
    p.scales[0] = c.k_scales;
    p.scales[1] = c.v_scales;
    p.tokens = tokens;
    p.tiles = Divisor(c.page_size / 16);
    p.nslots = c.pages * c.page_size;
    p.kv_heads = (int)c.kv_heads;
    if (c.head_dim == 64) return append<64>(c, p, bf16, mode, stream);
    if (c.head_dim == 128) return append<128>(c, p, bf16, mode, stream);
    return append<256>(c, p, bf16, mode, stream);
}

hipError_t launch_kv_read(const if4_kv_cache& c, const int64_t* slots, int64_t tokens, void* k,
                          void* v, int bf16, hipStream_t stream) {
    ReadArgs p;
    p.codes[0] = c.k_codes;
    p.codes[1] = c.v_codes;
    p.scales[0] = c.k_scales;
    p.scales[1] = c.v_scales;
    p.y[0] = k;
    p.y[1] = v;
    p.slots = slots;
    p.p_exp[0] = pow2f(c.k_exp);
    p.p_exp[1] = pow2f(c.v_exp);
    p.tokens = tokens;
    p.tiles = Divisor(c.page_size / 16);
    p.nslots = c.pages * c.page_size;
    p.kv_heads = (int)c.kv_heads;
    if (c.head_dim == 64) return read<64>(c, p, bf16, stream);
    if (c.head_dim == 128) return read<128>(c, p, bf16, stream);
    return read<256>(c, p, bf16, stream);
}

}  // namespace if4
