// FP8 quantize for gfx950: E4M3 codes and one power of two per block of 128 values
// or per square of 128 x 128.  The format is that of include/if4_fp8.h.
//
// Bound by memory: 2 or 4 bytes in and one out per value.  The exponent comes from
// the bits of the block's largest magnitude, the product x * 2^-e is exact (what
// underflows is far below half of the smallest code), and the hardware's conversion
// rounds it to E4M3, nearest even.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_internal.h"
#include "kv_internal.h"
#include "launch_limit.h"

namespace if4 {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = IF4_FP8_BLOCK;

// 16 consecutive values as fp32 bits.
template <bool kBf16>
__device__ __forceinline__ void load16(const void* x, int64_t at, uint32_t (&v)[16]) {
    if constexpr (kBf16) {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x) + at);
        const uint4 a = p[0], b = p[1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; i++) {
            v[2 * i] = w[i] << 16;
            v[2 * i + 1] = w[i] & 0xFFFF0000u;
        }
    } else {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(x) + at);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint4 a = p[i];
            v[4 * i] = a.x;
            v[4 * i + 1] = a.y;
            v[4 * i + 2] = a.z;
            v[4 * i + 3] = a.w;
        }
    }
}

__device__ __forceinline__ uint32_t magnitude(uint32_t bits) { return bits & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The largest of 8 consecutive lanes, in all of them.
__device__ __forceinline__ uint32_t max_of_8(uint32_t v) {
    v = larger(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // quad_perm 1,0,3,2
    v = larger(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));   // quad_perm 2,3,0,1
    return larger(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));  // half row mirrored
}

// A block's byte and the factor 2^-e, from the bits of its largest magnitude.  448 is
// 1.75 * 2^8: what has a larger fraction needs one more.
struct Scale {
    uint32_t byte;
    float inverse;
    bool bad;
    __device__ __forceinline__ explicit Scale(uint32_t amax) {
        bad = amax >= 0x7F800000u;
        const int e = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        byte = bad ? 255u : (uint32_t)(e < 0 ? 0 : e);
        inverse = __uint_as_float((254u - byte) << 23);
    }
};

// four codes, the first in the low byte
__device__ __forceinline__ uint32_t encode4(uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                            const Scale& s) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(__uint_as_float(a) * s.inverse,
                                            __uint_as_float(b) * s.inverse, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(__uint_as_float(c) * s.inverse,
                                        __uint_as_float(d) * s.inverse, w, true);
    return s.bad ? 0x7F7F7F7Fu : (uint32_t)w;
}

__device__ __forceinline__ uint4 encode16(const uint32_t (&v)[16], const Scale& s) {
    return make_uint4(encode4(v[0], v[1], v[2], v[3], s), encode4(v[4], v[5], v[6], v[7], s),
                      encode4(v[8], v[9], v[10], v[11], s),
                      encode4(v[12], v[13], v[14], v[15], s));
}

// Blocks of one row: 8 lanes of 16 values each, any lanes of a wave.  8192 x 8192 bf16 (202
// MB): 30.6 us, 6.6 TB/s (its codes stay in the caches for the product); 64 x 8192: 4 us.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads)
rows_kernel(const void* __restrict__ x, uint32_t blocks, Divisor per_row, int64_t cols,
            int64_t ld_x, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    const uint32_t block = blockIdx.x * (kThreads / 8) + threadIdx.x / 8;
    if (block >= blocks) return;  // all 8 lanes of a block together
    const uint32_t row = per_row.into(block), b = block - row * per_row.n;
    const int64_t col = (int64_t)b * kBlock + (threadIdx.x & 7) * 16;
    uint32_t v[16] = {};
    if (col < cols) load16<kBf16>(x, row * ld_x + col, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) m = larger(m, magnitude(v[i]));
    const Scale s(max_of_8(m));
    if (col < cols) *reinterpret_cast<uint4*>(codes + row * cols + col) = encode16(v, s);
    if ((threadIdx.x & 7) == 0) scales[block] = (uint8_t)s.byte;
}

// The largest magnitude of a workgroup.
__device__ __forceinline__ uint32_t workgroup_max(uint32_t m, uint32_t* shared) {
    m = max_of_8(m);
#pragma unroll
    for (int d = 8; d < 64; d *= 2) m = larger(m, (uint32_t)__shfl_xor((int)m, d));
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x / 64] = m;
    __syncthreads();
    return larger(larger(shared[0], shared[1]), larger(shared[2], shared[3]));
}

// A square per workgroup; thread t holds 16 values of rows t/8 + 32 i.  28672 x 8192 bf16:
// 5.6 TB/s.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads)
squares_kernel(const void* __restrict__ x, int64_t rows, int64_t cols, int64_t ld_x,
               Divisor across, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    __shared__ uint32_t shared[4];
    const uint32_t down = across.into(blockIdx.x), b = blockIdx.x - down * across.n;
    const int64_t col = (int64_t)b * kBlock + (threadIdx.x & 7) * 16;
    const int64_t row = (int64_t)down * kBlock + threadIdx.x / 8;
    uint32_t v[4][16] = {};
#pragma unroll
    for (int i = 0; i < 4; i++)
        if (row + 32 * i < rows && col < cols) load16<kBf16>(x, (row + 32 * i) * ld_x + col, v[i]);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 16; j++) m = larger(m, magnitude(v[i][j]));
    const Scale s(workgroup_max(m, shared));
#pragma unroll
    for (int i = 0; i < 4; i++)
        if (row + 32 * i < rows && col < cols)
            *reinterpret_cast<uint4*>(codes + (row + 32 * i) * cols + col) = encode16(v[i], s);
    if (threadIdx.x == 0) scales[blockIdx.x] = (uint8_t)s.byte;
}

// x^T: a tile of 128 rows by 128 columns of x per workgroup, the rows being the
// contraction dimension.  Thread t holds rows 4 (t/8) .. + 3 of columns 16 (t%8) ..
// + 15, so that four values of a column are four neighbouring codes, one word.  The
// words cross LDS (a column's 128 codes and 4 more words, which spreads the writes
// over the banks), and leave it 16 bytes per thread, a column's codes in one line.  4096 x 8192
// bf16 (101 MB): 20 us, 5.0 TB/s.
template <bool kBf16, bool kSquare>
__global__ void __launch_bounds__(kThreads)
transposed_kernel(const void* __restrict__ x, int64_t rows, int64_t cols, int64_t ld_x,
                  Divisor tiles_k, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    constexpr int kPitch = 36;  // words
    __shared__ __attribute__((aligned(16))) uint32_t tile[kBlock * kPitch];
    const uint32_t down = tiles_k.into(blockIdx.x), b = blockIdx.x - down * tiles_k.n;
    const int cg = threadIdx.x & 7, rg = threadIdx.x / 8;
    const int64_t col = (int64_t)down * kBlock + 16 * cg;  // first of this thread's columns
    const int64_t row = (int64_t)b * kBlock + 4 * rg;      // rows are a multiple of 16
    uint32_t v[4][16] = {};
    if (row < rows) {
        if (col + 16 <= cols) {
#pragma unroll
            for (int i = 0; i < 4; i++) load16<kBf16>(x, (row + i) * ld_x + col, v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 16; j++)
                    if (col + j < cols) {
                        const int64_t at = (row + i) * ld_x + col + j;
                        v[i][j] = kBf16 ? (uint32_t)reinterpret_cast<const uint16_t*>(x)[at] << 16
                                        : reinterpret_cast<const uint32_t*>(x)[at];
                    }
        }
    }
    uint32_t m[16];
#pragma unroll
    for (int j = 0; j < 16; j++)
        m[j] = larger(larger(magnitude(v[0][j]), magnitude(v[1][j])),
                      larger(magnitude(v[2][j]), magnitude(v[3][j])));
    const int64_t nb = tiles_k.n;
    if constexpr (kSquare) {
        uint32_t all = 0;
#pragma unroll
        for (int j = 0; j < 16; j++) all = larger(all, m[j]);
        const Scale s(workgroup_max(all, tile));
        if (threadIdx.x == 0) scales[down * nb + b] = (uint8_t)s.byte;
        __syncthreads();  // the maximum has been read
#pragma unroll
        for (int j = 0; j < 16; j++)
            tile[(16 * cg + j) * kPitch + rg] = encode4(v[0][j], v[1][j], v[2][j], v[3][j], s);
    } else {
        // partial maxima [row group][column], then a column's 32 by two threads
#pragma unroll
        for (int j = 0; j < 16; j++) tile[rg * kBlock + 16 * cg + j] = m[j];
        __syncthreads();
        const int c = threadIdx.x & (kBlock - 1), half = threadIdx.x / kBlock;
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 16; i++) most = larger(most, tile[(16 * half + i) * kBlock + c]);
        __syncthreads();
        tile[half * kBlock + c] = most;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 16; j++)
            m[j] = larger(tile[16 * cg + j], tile[kBlock + 16 * cg + j]);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 16; j++) {
            const Scale s(m[j]);
            tile[(16 * cg + j) * kPitch + rg] = encode4(v[0][j], v[1][j], v[2][j], v[3][j], s);
            if (rg == 0 && col + j < cols) scales[(col + j) * nb + b] = (uint8_t)s.byte;
        }
    }
    __syncthreads();
    const int64_t k = (int64_t)b * kBlock + 16 * cg;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int c = rg + 32 * i;
        const int64_t to = (int64_t)down * kBlock + c;
        if (to < cols && k < rows)
            *reinterpret_cast<uint4*>(codes + to * rows + k) =
                *reinterpret_cast<const uint4*>(tile + c * kPitch + 4 * cg);
    }
}

int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

}  // namespace

hipError_t launch_fp8_quantize(const void* x, int bf16, int64_t rows, int64_t cols, int64_t ld_x,
                               int square, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
    const int64_t across = blocks_of(cols);
    const int64_t count = (square ? blocks_of(rows) : rows) * across;
    const Divisor by(across);
    if (!launchable(square ? count : (count + kThreads / 8 - 1) / (kThreads / 8), kThreads))
        return hipErrorInvalidConfiguration;
    if (square) {
        const auto k = bf16 ? squares_kernel<true> : squares_kernel<false>;
        hipLaunchKernelGGL(k, dim3((unsigned)count), dim3(kThreads), 0, stream, x, rows, cols,
                           ld_x, by, codes, scales);
    } else {
        const auto k = bf16 ? rows_kernel<true> : rows_kernel<false>;
        hipLaunchKernelGGL(k, dim3((unsigned)((count + kThreads / 8 - 1) / (kThreads / 8))),
                           dim3(kThreads), 0, stream, x, (uint32_t)count, by, cols, ld_x, codes,
                           scales);
    }
    return hipGetLastError();
}

hipError_t launch_fp8_quantize_t(const void* x, int bf16, int64_t rows, int64_t cols,
                                 int64_t ld_x, int square, uint8_t* codes, uint8_t* scales,
                                 hipStream_t stream) {
    const int64_t count = blocks_of(rows) * blocks_of(cols);
    if (!launchable(count, kThreads)) return hipErrorInvalidConfiguration;
    const Divisor by(blocks_of(rows));
    const auto k = bf16 ? (square ? transposed_kernel<true, true> : transposed_kernel<true, false>)
                        : (square ? transposed_kernel<false, true> : transposed_kernel<false, false>);
    hipLaunchKernelGGL(k, dim3((unsigned)count), dim3(kThreads), 0, stream, x, rows, cols, ld_x,
                       by, codes, scales);
    return hipGetLastError();
}

}  // namespace if4
