// FP8 x FP8 product for gfx950: C[M,N] = A[M,K] * W[N,K]^T, E4M3 codes with a power
// of two per block of 128 along K (include/if4_fp8.h), fp32 sums.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp8_internal.h"

namespace if4 {
namespace {

typedef int int4v __attribute__((ext_vector_type(4)));
typedef int int8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float float16v __attribute__((ext_vector_type(16)));

constexpr int BK = IF4_FP8_BLOCK;  // one K step: a block, 128 bytes of each row
constexpr int kThreads = 256;
constexpr int kBandM = 4;  // M-tiles per band of the tile order
constexpr int kWindow = 4; // steps whose scale bytes one 32-bit register holds
constexpr int kRawBufferFlags = 0x00020000;

// Workgroup barrier that orders LDS only (the loads of the next steps stay in
// flight).
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Wait for all vector memory operations (vmcnt 0, the other counters free).
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// 16 bytes per lane from the buffer straight into LDS, lane l's at `lds` + 16 l.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff,
                                            uint32_t soff, uint8_t* lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc, (__attribute__((address_space(3))) void*)lds, 16, (int)voff, (int)soff, 0, 0);
}

// 32 codes to bf16, exactly, times the power of two in the low byte of `scale`.
__device__ __forceinline__ void widen(int8v codes, uint32_t scale, bf16x8 (&out)[4]) {
    const float s = __uint_as_float((scale & 0xFFu) << 23);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)codes[i], s, false);
        const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)codes[i], s, true);
        out[i / 2][4 * (i & 1)] = lo[0];
        out[i / 2][4 * (i & 1) + 1] = lo[1];
        out[i / 2][4 * (i & 1) + 2] = hi[0];
        out[i / 2][4 * (i & 1) + 3] = hi[1];
    }
}

// Scale bytes of one operand's rows: 32-bit offsets from the tile's first row.
// kBytes: an operand with fewer than four of them.
template <bool kBytes>
struct Scales {
    const uint8_t* base;
    int last;  // offset of the operand's last four bytes (its last one with kBytes)
    __device__ __forceinline__ Scales(const uint8_t* all, int64_t first_row, int64_t rows,
                                      int steps) {
        base = all + first_row * steps;
        const int64_t left = (rows - first_row) * steps - (kBytes ? 1 : 4);
        last = (int)(left < 0x7FFFFFFF ? left : 0x7FFFFFFF);
    }
    // The four bytes from `off` on, at any alignment; next to the operand's end the last
    // four, which take() moves into place.
    __device__ __forceinline__ uint32_t window(int off) const {
        uint32_t w = 0;
        if constexpr (kBytes) {
            for (int i = 0; i < kWindow; i++)
                w |= (uint32_t)base[off + i < last ? off + i : last] << (8 * i);
        } else {
            __builtin_memcpy(&w, base + (off < last ? off : last), 4);
        }
        return w;
    }
    __device__ __forceinline__ uint32_t take(uint32_t w, int off) const {
        return kBytes || off < last ? w : w >> ((8 * (off - last)) & 31);
    }
};

template <int BM, int BN, bool kBf16, bool kBytes>
__global__ void __launch_bounds__(kThreads)
tile_kernel(const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_scales,
            const uint8_t* __restrict__ w_codes, const uint8_t* __restrict__ w_scales,
            int w_square, int64_t M, int64_t N, int64_t K, void* __restrict__ c,
            int64_t ldc, int tiles_m, int tiles_n) {
    constexpr int TM = BM / 64, TN = BN / 64;  // 32 x 32 blocks of a wave
    constexpr int kBuffer = (BM + BN) * BK;    // bytes of one step
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;

    const int total = tiles_m * tiles_n;
    int bid = blockIdx.x;
    if (total % 8 == 0) bid = (bid % 8) * (total / 8) + bid / 8;
    const int band = bid / (kBandM * tiles_n), first_m = band * kBandM;
    const int band_m = tiles_m - first_m < kBandM ? tiles_m - first_m : kBandM;
    const int in_band = bid - band * kBandM * tiles_n;
    const int64_t m0 = (int64_t)(first_m + in_band % band_m) * BM;
    const int64_t n0 = (int64_t)(in_band / band_m) * BN;
    const int a_rows = (int)(M - m0 < BM ? M - m0 : BM), w_rows = (int)(N - n0 < BN ? N - n0 : BN);

    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(a_codes + m0 * K), 0, (int)(a_rows * K), kRawBufferFlags);
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(w_codes + n0 * K), 0, (int)(w_rows * K), kRawBufferFlags);
    const int steps = (int)((K + BK - 1) / BK);  // 1 at least

    // Loads: instruction i of a wave brings 8 rows (1 KB); lane l the piece that lies at
    // place l % 8 of row l / 8, which is piece (l % 8) ^ (row / 2 % 8) of the row.
    // Rows 8 (4 i + wave) ..: row / 2 % 8 = 4 (wave % 2) + l / 16.
    const int piece = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));
    const uint32_t voff = (uint32_t)(lane >> 3) * (uint32_t)K + 16 * piece;
    auto load_step = [&](int s) {
        // in a last step that is no whole block, pieces past K are outside
        const uint32_t v = (int64_t)s * BK + 16 * piece < K ? voff : 0x80000000u;  // (and steps past the last)
        uint8_t* const to = smem + (s & 1) * kBuffer;
#pragma unroll
        for (int i = 0; i < BM / 32; i++) {
            const int r = 8 * (4 * i + wave);
            load_to_lds(ra, v, (uint32_t)r * (uint32_t)K + (uint32_t)s * BK, to + r * BK);
        }
#pragma unroll
        for (int i = 0; i < BN / 32; i++) {
            const int r = 8 * (4 * i + wave);
            load_to_lds(rw, v, (uint32_t)r * (uint32_t)K + (uint32_t)s * BK, to + (BM + r) * BK);
        }
    };

    // Scale rows of this lane, clamped into the operand.
    const int64_t w_first = w_square ? n0 / BK : n0, w_count = w_square ? (N + BK - 1) / BK : N;
    const Scales<kBytes> scales_a(a_scales, m0, M, steps);
    const Scales<kBytes> scales_w(w_scales, w_first, w_count, steps);
    int off_a[TM], off_w[TN];
#pragma unroll
    for (int i = 0; i < TM; i++) {
        const int r = wm * (BM / 2) + 32 * i + (lane & 31);
        off_a[i] = (r < a_rows ? r : a_rows - 1) * steps;
    }
#pragma unroll
    for (int j = 0; j < TN; j++) {
        int r = wn * (BN / 2) + 32 * j + (lane & 31);
        r = r < w_rows ? r : w_rows - 1;
        off_w[j] = (w_square ? r / BK : r) * steps;
    }
    uint32_t ea[TM], ew[TN], next_a[TM], next_w[TN];
    auto load_scales = [&](int s) {
#pragma unroll
        for (int i = 0; i < TM; i++) next_a[i] = scales_a.window(off_a[i] + s);
#pragma unroll
        for (int j = 0; j < TN; j++) next_w[j] = scales_w.window(off_w[j] + s);
    };
    auto take_scales = [&](int s) {
#pragma unroll
        for (int i = 0; i < TM; i++) ea[i] = scales_a.take(next_a[i], off_a[i] + s);
#pragma unroll
        for (int j = 0; j < TN; j++) ew[j] = scales_w.take(next_w[j], off_w[j] + s);
    };

    float16v acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;

    // Fragment of row block R (32 rows), half h of a step's 128: lane l holds row l % 32,
    // pieces 4 h + 2 (l / 32) and the next.
    const int frow = lane & 31, fsw = (lane >> 1) & 7;
    const int fp[2] = {2 * (lane >> 5), 2 * (lane >> 5) + 1};
    auto fragment = [&](const uint8_t* block, int h) {
        const int4v x = *reinterpret_cast<const int4v*>(block + frow * BK + 16 * ((4 * h + fp[0]) ^ fsw));
        const int4v y = *reinterpret_cast<const int4v*>(block + frow * BK + 16 * ((4 * h + fp[1]) ^ fsw));
        return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    int8v fa[2][TM], fw[2][TN];
    auto read = [&](int s, int h) {
        const uint8_t* b = smem + (s & 1) * kBuffer;
#pragma unroll
        for (int i = 0; i < TM; i++) fa[h][i] = fragment(b + (wm * (BM / 2) + 32 * i) * BK, h);
#pragma unroll
        for (int j = 0; j < TN; j++) fw[h][j] = fragment(b + (BM + wn * (BN / 2) + 32 * j) * BK, h);
    };
    auto multiply = [&](int h, auto byte) {
        if constexpr (kBf16) {
#pragma unroll
            for (int i = 0; i < TM; i++)
#pragma unroll
                for (int j = 0; j < TN; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        fa[h][i], fw[h][j], acc[i][j], 0, 0, decltype(byte)::value, (int)ea[i],
                        decltype(byte)::value, (int)ew[j]);
        } else {
            constexpr int kShift = 8 * decltype(byte)::value;
            bf16x8 w[TN][4];
#pragma unroll
            for (int j = 0; j < TN; j++) widen(fw[h][j], ew[j] >> kShift, w[j]);
#pragma unroll
            for (int i = 0; i < TM; i++) {
                bf16x8 a[4];
                widen(fa[h][i], ea[i] >> kShift, a);
#pragma unroll
                for (int q = 0; q < 4; q++)
#pragma unroll
                    for (int j = 0; j < TN; j++)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[q], w[j][q], acc[i][j], 0, 0, 0);
            }
        }
    };
    constexpr int kProducts = kBf16 ? 1 : 4;
    constexpr int kLoads = ((BM + BN) / 32 + TM * TN - 1) / (TM * TN);
    constexpr int kReads = (2 * (TM + TN) + TM * TN - 1) / (TM * TN);
    // One step: the products of its two halves, each product beside reads of the half
    // after it.  The barrier in the middle says both that step s + 1 has arrived and that
    // all waves have read step s, so that its buffer takes step s + 2.  (No branch inside:
    // steps past the last load zeros.)
    auto step = [&](int s, auto byte) {
        read(s, 1);
        multiply(0, byte);
#pragma unroll
        for (int i = 0; i < TM * TN; i++) {
            __builtin_amdgcn_sched_group_barrier(0x008, kProducts, 0);       // MFMA
            __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);  // LDS read
        }
        __builtin_amdgcn_sched_barrier(0);
        wait_loads();
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        load_step(s + 2);
        read(s + 1, 0);
        multiply(1, byte);
#pragma unroll
        for (int i = 0; i < TM * TN; i++) {
            __builtin_amdgcn_sched_group_barrier(0x008, kProducts, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
            __builtin_amdgcn_sched_group_barrier(0x020, kLoads, 0);  // loads
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    load_scales(0);
    load_step(0);
    wait_loads();
    lds_barrier();
    take_scales(0);
    load_step(1);
    read(0, 0);
    for (int s = 0; s < steps; s += kWindow) {
        load_scales(s + kWindow);
        step(s, std::integral_constant<int, 0>{});
        if (s + 1 < steps) step(s + 1, std::integral_constant<int, 1>{});
        if (s + 2 < steps) step(s + 2, std::integral_constant<int, 2>{});
        if (s + 3 < steps) step(s + 3, std::integral_constant<int, 3>{});
        take_scales(s + kWindow);
    }
    wait_loads();  // (the last steps' zeros: LDS is not given back before they have arrived)

    // lane: column lane % 32 of a block, rows 8 (r / 4) + 4 (lane / 32) + r % 4.  The
    // stores go through a buffer resource over the tile's rows that exist: one
    // vector offset per lane, and a store past M is dropped.
    constexpr int kSize = kBf16 ? 2 : 4;
    if ((uint64_t)ldc * (kSize * BM) < (1ull << 31)) {
        const uint32_t ld = (uint32_t)ldc * kSize;
        const __amdgpu_buffer_rsrc_t rc = __builtin_amdgcn_make_buffer_rsrc(
            reinterpret_cast<uint8_t*>(c) + (m0 * ldc + n0) * kSize, 0, (int)((uint32_t)a_rows * ld),
            kRawBufferFlags);
        const uint32_t vo = (uint32_t)(lane & 31) * kSize + (uint32_t)(4 * (lane >> 5)) * ld;
#pragma unroll
        for (int j = 0; j < TN; j++) {
            const int col = wn * (BN / 2) + 32 * j;
            if (col + (lane & 31) >= w_rows) continue;
#pragma unroll
            for (int i = 0; i < TM; i++)
#pragma unroll
                for (int r = 0; r < 16; r++) {
                    const uint32_t so = (uint32_t)(wm * (BM / 2) + 32 * i + 8 * (r >> 2) + (r & 3)) * ld +
                                        col * kSize;
                    if constexpr (kBf16)
                        __builtin_amdgcn_raw_buffer_store_b16(
                            __builtin_bit_cast(short, (__bf16)acc[i][j][r]), rc, (int)vo, (int)so, 0);
                    else
                        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[i][j][r]), rc,
                                                              (int)vo, (int)so, 0);
                }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) {
            const int64_t col = n0 + wn * (BN / 2) + 32 * j + (lane & 31);
#pragma unroll
            for (int r = 0; r < 16; r++) {
                const int64_t row = m0 + wm * (BM / 2) + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                if (row < M && col < N) {
                    if constexpr (kBf16)
                        reinterpret_cast<__bf16*>(c)[row * ldc + col] = (__bf16)acc[i][j][r];
                    else
                        reinterpret_cast<float*>(c)[row * ldc + col] = acc[i][j][r];
                }
            }
        }
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads)
zero_kernel(void* __restrict__ c, int64_t M, int64_t N, int64_t ldc) {
    const int64_t total = M * N;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * kThreads) {
        const int64_t at = i / N * ldc + i % N;
        if constexpr (kBf16)
            reinterpret_cast<uint16_t*>(c)[at] = 0;
        else
            reinterpret_cast<uint32_t*>(c)[at] = 0;
    }
}

template <int BM, int BN, bool kBf16, bool kBytes>
hipError_t launch_tile(const Fp8Gemm& g, hipStream_t stream) {
    constexpr int kSmem = 2 * (BM + BN) * BK;
    const int64_t tiles_m = (g.M + BM - 1) / BM, tiles_n = (g.N + BN - 1) / BN;
    // dynamic LDS above 64 KB must be allowed per kernel (idempotent, any device)
    const hipError_t err = hipFuncSetAttribute((const void*)tile_kernel<BM, BN, kBf16, kBytes>,
                                               hipFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL((tile_kernel<BM, BN, kBf16, kBytes>), dim3((unsigned)(tiles_m * tiles_n)), dim3(kThreads),
                       kSmem, stream, g.a_codes, g.a_scales, g.w_codes, g.w_scales, g.w_square,
                       g.M, g.N, g.K, g.c, g.ldc, (int)tiles_m, (int)tiles_n);
    return hipGetLastError();
}

}  // namespace

int64_t fp8_gemm_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_fp8_gemm(const Fp8Gemm& g, hipStream_t stream) {
    if (g.K == 0) {
        const int64_t blocks = (g.M * g.N + kThreads - 1) / kThreads;
        const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
        const auto k = g.c_bf16 ? zero_kernel<true> : zero_kernel<false>;
        hipLaunchKernelGGL(k, grid, dim3(kThreads), 0, stream, g.c, g.M, g.N, g.ldc);
        return hipGetLastError();
    }
    const int64_t steps = (g.K + BK - 1) / BK;
    const int64_t w_scales = (g.w_square ? (g.N + BK - 1) / BK : g.N) * steps;
    const bool bytes = g.M * steps < 4 || w_scales < 4;
    const int64_t wide = ((g.M + 255) / 256) * ((g.N + 255) / 256);
    if (g.c_bf16)
        return bytes         ? launch_tile<128, 128, true, true>(g, stream)
               : wide >= 256 ? launch_tile<256, 256, true, false>(g, stream)
                             : launch_tile<128, 128, true, false>(g, stream);
    return bytes         ? launch_tile<128, 128, false, true>(g, stream)
           : wide >= 256 ? launch_tile<256, 256, false, false>(g, stream)
                         : launch_tile<128, 128, false, false>(g, stream);
}

}  // namespace if4
