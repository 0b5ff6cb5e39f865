// FP8 x FP8 product for gfx950: C[M,N] = A[M,K] * W[N,K]^T, E4M3 codes with a power
// of two per block of 128 along K (include/if4_fp8.h), fp32 sums.
//
// The block of 128 is a matrix instruction's K (or twice it), so that a block's byte goes into
// the instruction as its scale and costs nothing.  But the scaled FP8 instructions do not add
// products one by one: of 8 neighbouring k they bring the products to the largest one's
// exponent and cut them 13 bits below it, up to 2^-10 of the sum of the products' magnitudes.
// On operands of like magnitudes that is below what rounding a result to bf16 loses; where
// products cancel, or a few of K are far larger than the rest, it can be more.  Results in bf16
// take them for twice the rate all the same, and a caller who cannot has fp32 results.  These
// take the bf16 instructions, in which every product and every sum of fp32 is whole: E4M3
// times a power of two is exact in bf16 (for bytes 3 to 246; below, codes under bf16's least
// 2^-133 are rounded to a multiple of it, above, what reaches 2^128 overflows), and the
// conversion (v_cvt_scalef32) applies the byte too.  4096 x 8192 x 4096: 222 us in fp32 (1240
// TFLOP/s), 118 in bf16 (2330).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp8_internal.h"
#include "launch_limit.h"

namespace if4 {
namespace {

typedef int int4v __attribute__((ext_vector_type(4)));
typedef int int8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));
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

// Wait until no more than n vector memory operations are on their way (the other counters
// free).
template <int n>
__device__ __forceinline__ void wait_loads() {
    static_assert(n < 64, "vmcnt has six bits");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (n & 15) | (n >> 4) << 14);
}

// 16 bytes per lane from the buffer straight into LDS, lane l's at `lds` + 16 l.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff,
                                            uint32_t soff, uint8_t* lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc, (__attribute__((address_space(3))) void*)lds, 16, (int)voff, (int)soff, 0, 0);
}

// 32 codes to bf16, times the power of two in the low byte of `scale`: exactly for bytes 3 to
// 246 (the conversion takes a byte of 0, which is no fp32 power, as 2^-127).
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

// A tile of BM x BN results per workgroup, and (splits > 1) a share of K.
//
// A step is one block of K: BM + BN lines of 128 bytes, brought into LDS without a stop in
// registers, kStages steps ahead.  Its two halves of 64 are the operands of 32 x 32 x 64
// products, read one half ahead of the products that need them, a few reads beside each
// product.  In the loop nothing branches (a branch parts the reads from the products, which
// cost 8 to 15% wherever one was): what lies past K, M or N is outside the buffer resource and
// arrives as zeros, and a step's buffer is known when compiled.
//
// 256 x 256 with four waves of 128 x 128: 256 accumulators each, and the fewest LDS bytes a
// product (a wave reads 256 rows for 16 products a half; of 64 x 128 parts, 8 waves, 1.5 times
// as many, and slower).  One workgroup and one wave per SIMD fit, so that products wait
// wherever the wave waits: 8192 x 28672 x 8192 1470 us, 2620 TFLOP/s, with the matrix units busy
// 63% of the time (of no step but products 3830 are reached by one wave a SIMD and 4490 by
// two), 840 MB read and written once being 170 us.  Three stages or prefetch by half steps:
// slower.  Tiles of 128 (64 KB of LDS, two workgroups on a CU, each covering the other's
// waits) with two stages: 2048 x 4096 x 4096 44 us, four stages and one workgroup 60.  Tiles
// of 64 with four stages: 64 x 28672 x 8192, 239 MB, 64.6 us, 3.7 TB/s; two stages 66.5 (256 x
// 6144 x 4096: 23.9, 26.6).
//
// Tiles are gone through in bands of kBandM rows of tiles, and workgroups that follow one
// another on one XCD have tiles that follow one another, so that its L2 has their A and W
// (bands of 2, 8 and 16 were slower).
template <int BM, int BN, int kWavesM, int kWavesN, int kStages, bool kBf16, bool kBytes>
__global__ void __launch_bounds__(64 * kWavesM * kWavesN)
tile_kernel(const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_scales,
            const uint8_t* __restrict__ w_codes, const uint8_t* __restrict__ w_scales,
            int w_square, int64_t M, int64_t N, int64_t K, void* __restrict__ c,
            int64_t ldc, int tiles_m, int tiles_n, float* __restrict__ parts, int splits) {
    constexpr int WM = BM / kWavesM, WN = BN / kWavesN;  // a wave's part of the tile
    constexpr int TM = WM / 32, TN = WN / 32;            // its 32 x 32 blocks
    constexpr int kWaves = kWavesM * kWavesN;
    constexpr int kBuffer = (BM + BN) * BK;              // bytes of one step
    constexpr int kStepLoads = (BM + BN) / 8 / kWaves;   // of a wave, 1 KB each
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / kWavesN, wn = wave % kWavesN;

    const int total = tiles_m * tiles_n;
    int bid = blockIdx.x % total;
    const int split = blockIdx.x / total;
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
    // this split's steps, whole windows of scale bytes
    const int share = splits == 1 ? steps : ((steps + splits - 1) / splits + kWindow - 1) & ~(kWindow - 1);
    const int begin = split * share, end = begin + share < steps ? begin + share : steps;

    // Loads: one of a wave brings 8 rows (1 KB).  The piece of 16 bytes that lies at place l
    // of row r is piece l ^ (r / 2 % 8) of the row, so that the reads of 16 lanes, one piece of
    // 16 rows, cover all banks.  (Rows 8 (kWaves i + wave) ..: r / 2 % 8 = 4 (wave % 2) + lane / 16.)
    const int piece = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));
    const uint32_t voff = (uint32_t)(lane >> 3) * (uint32_t)K + 16 * piece;
    const int64_t limit = (int64_t)end * BK < K ? (int64_t)end * BK : K;
    // (A's first: W's first is 8% slower where tiles are many, 1490 and 1610 us)
    auto load_step = [&](int s, int buffer) {
        // in a last step that is no whole block, pieces past K are outside, and so are steps
        // past the last (one test, or a branch parts the reads from the products)
        const uint32_t v = (int64_t)s * BK + 16 * piece < limit ? voff : 0x80000000u;
        uint8_t* const to = smem + buffer * kBuffer;
#pragma unroll
        for (int i = 0; i < BM / 8 / kWaves; i++) {
            const int r = 8 * (kWaves * i + wave);
            load_to_lds(ra, v, (uint32_t)r * (uint32_t)K + (uint32_t)s * BK, to + r * BK);
        }
#pragma unroll
        for (int i = 0; i < BN / 8 / kWaves; i++) {
            const int r = 8 * (kWaves * i + wave);
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
        const int r = wm * WM + 32 * i + (lane & 31);
        off_a[i] = (r < a_rows ? r : a_rows - 1) * steps;
    }
#pragma unroll
    for (int j = 0; j < TN; j++) {
        int r = wn * WN + 32 * j + (lane & 31);
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
    auto fragment = [&](const uint8_t* block, int h) {
        const int at = 4 * h + 2 * (lane >> 5);
        const int4v x = *reinterpret_cast<const int4v*>(block + frow * BK + 16 * (at ^ fsw));
        const int4v y = *reinterpret_cast<const int4v*>(block + frow * BK + 16 * ((at + 1) ^ fsw));
        return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    int8v fa[2][TM], fw[2][TN];
    auto read = [&](int buffer, int h) {
        const uint8_t* b = smem + buffer * kBuffer;
#pragma unroll
        for (int i = 0; i < TM; i++) fa[h][i] = fragment(b + (wm * WM + 32 * i) * BK, h);
#pragma unroll
        for (int j = 0; j < TN; j++) fw[h][j] = fragment(b + (BM + wn * WN + 32 * j) * BK, h);
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
    // One step: the products of its two halves, each product beside reads of the half
    // after it.  The barrier in the middle says both that step s + 1 has arrived and that
    // all waves have read step s, so that its buffer takes step s + kStages.  (No branch
    // inside: steps past the last load zeros.)
    constexpr int kProducts = kBf16 ? 1 : 4;  // matrix instructions of a 32 x 32 x 64 product
    constexpr int kLoads = (kStepLoads + TM * TN - 1) / (TM * TN);
    constexpr int kReads = (2 * (TM + TN) + TM * TN - 1) / (TM * TN);
    static_assert(kWindow % kStages == 0, "a step's buffer goes by its place in the window");
    auto step = [&](int s, auto byte) {
        constexpr int buffer = decltype(byte)::value % kStages;
        read(buffer, 1);
        multiply(0, byte);
#pragma unroll
        for (int i = 0; i < TM * TN; i++) {
            __builtin_amdgcn_sched_group_barrier(0x008, kProducts, 0);  // MFMA
            __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);     // LDS read
        }
        __builtin_amdgcn_sched_barrier(0);
        wait_loads<(kStages - 2) * kStepLoads>();
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
        load_step(s + kStages, buffer);
        read((buffer + 1) % kStages, 0);
        multiply(1, byte);
#pragma unroll
        for (int i = 0; i < TM * TN; i++) {
            __builtin_amdgcn_sched_group_barrier(0x008, kProducts, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
            __builtin_amdgcn_sched_group_barrier(0x020, kLoads, 0);  // loads
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    if (begin < end) {
        load_scales(begin);
#pragma unroll
        for (int i = 0; i < kStages; i++) load_step(begin + i, i);
        wait_loads<(kStages - 1) * kStepLoads>();
        lds_barrier();
        take_scales(begin);
        read(0, 0);
        for (int s = begin; s < end; s += kWindow) {
            load_scales(s + kWindow);
            step(s, std::integral_constant<int, 0>{});
            if (s + 1 < end) step(s + 1, std::integral_constant<int, 1>{});
            if (s + 2 < end) step(s + 2, std::integral_constant<int, 2>{});
            if (s + 3 < end) step(s + 3, std::integral_constant<int, 3>{});
            take_scales(s + kWindow);
        }
        wait_loads<0>();  // (the last steps' zeros: LDS is not given back before they have arrived)
    }

    if (splits > 1) {  // fp32 sums of this split, [M, N] of its own
        float* const part = parts + (int64_t)split * M * N;
#pragma unroll
        for (int i = 0; i < TM; i++)
#pragma unroll
            for (int j = 0; j < TN; j++) {
                const int col = wn * WN + 32 * j + (lane & 31);
#pragma unroll
                for (int r = 0; r < 16; r++) {
                    const int row = wm * WM + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                    if (row < a_rows && col < w_rows) part[(m0 + row) * N + n0 + col] = acc[i][j][r];
                }
            }
        return;
    }
    // lane: column lane % 32 of a block, rows 8 (r / 4) + 4 (lane / 32) + r % 4.  The
    // stores go through a buffer resource over the tile's rows that exist: one
    // vector offset per lane, and a store past M is dropped.  C of the largest tiles is more
    // than the caches hold, and goes past them (non-temporal) where its rows are whole lines (5000 x
    // 5000 x 512 58 us past them, 43 through them; 8192 x 28672 x 8192 1470, 1495).
    constexpr int kSize = kBf16 ? 2 : 4;
    if ((uint64_t)ldc * (kSize * BM) < (1ull << 31)) {
        const uint32_t ld = (uint32_t)ldc * kSize;
        const __amdgpu_buffer_rsrc_t rc = __builtin_amdgcn_make_buffer_rsrc(
            reinterpret_cast<uint8_t*>(c) + (m0 * ldc + n0) * kSize, 0, (int)((uint32_t)a_rows * ld),
            kRawBufferFlags);
        const uint32_t vo = (uint32_t)(lane & 31) * kSize + (uint32_t)(4 * (lane >> 5)) * ld;
        const auto store = [&](auto policy) {
            constexpr int kPolicy = decltype(policy)::value;
#pragma unroll
            for (int j = 0; j < TN; j++) {
                const int col = wn * WN + 32 * j;
                if (col + (lane & 31) >= w_rows) continue;
#pragma unroll
                for (int i = 0; i < TM; i++)
#pragma unroll
                    for (int r = 0; r < 16; r++) {
                        const uint32_t so = (uint32_t)(wm * WM + 32 * i + 8 * (r >> 2) + (r & 3)) * ld +
                                            col * kSize;
                        if constexpr (kBf16)
                            __builtin_amdgcn_raw_buffer_store_b16(
                                __builtin_bit_cast(short, (__bf16)acc[i][j][r]), rc, (int)vo, (int)so, kPolicy);
                        else
                            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[i][j][r]), rc,
                                                                  (int)vo, (int)so, kPolicy);
                    }
            }
        };
        if (BM == 256 && ((reinterpret_cast<uintptr_t>(c) | ld) & 127) == 0)
            store(std::integral_constant<int, 2>{});
        else
            store(std::integral_constant<int, 0>{});
        return;
    }
#pragma unroll
    for (int i = 0; i < TM; i++)
#pragma unroll
        for (int j = 0; j < TN; j++) {
            const int64_t col = n0 + wn * WN + 32 * j + (lane & 31);
#pragma unroll
            for (int r = 0; r < 16; r++) {
                const int64_t row = m0 + wm * WM + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                if (row < M && col < N) {
                    if constexpr (kBf16)
                        reinterpret_cast<__bf16*>(c)[row * ldc + col] = (__bf16)acc[i][j][r];
                    else
                        reinterpret_cast<float*>(c)[row * ldc + col] = acc[i][j][r];
                }
            }
        }
}

// Few rows of A (M <= 16): the bytes of W bound the call, and each is used by one wave only, so
// that they go from memory to registers, four blocks ahead, with no LDS.  A workgroup has 16
// rows of W and all rows of A (16 x 16 x 128 products, W's rows in the accumulators'
// registers); its 8 waves take shares of K, whose sums are added up in LDS in their order.
// M = 1, N = 6144, K = 4096 (25 MB): 7.5 us, 3.4 TB/s, of which the launch and the first
// answer from memory are about half.
constexpr int kFewWaves = 8, kFewThreads = 64 * kFewWaves;

// The two pieces of 16 bytes of a lane's 32 codes of block s: row `row` of the resource,
// zeros past K.
__device__ __forceinline__ int8v load_codes(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, int k, int s,
                                            int64_t K) {
    const bool a = (int64_t)s * BK + k < K, b = (int64_t)s * BK + k + 16 < K;
    const int4v x = __builtin_bit_cast(int4v, __builtin_amdgcn_raw_buffer_load_b128(
                                                  rsrc, a ? (int)voff : (int)0x80000000, s * BK, 0));
    const int4v y = __builtin_bit_cast(int4v, __builtin_amdgcn_raw_buffer_load_b128(
                                                  rsrc, b ? (int)(voff + 16) : (int)0x80000000, s * BK, 0));
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <bool kBf16, bool kBytes>
__global__ void __launch_bounds__(kFewThreads)
few_kernel(const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_scales,
           const uint8_t* __restrict__ w_codes, const uint8_t* __restrict__ w_scales,
           int w_square, int64_t M, int64_t N, int64_t K, void* __restrict__ c, int64_t ldc) {
    __shared__ float4v sums[kFewWaves][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int w_rows = N - n0 < 16 ? (int)(N - n0) : 16;
    const int steps = (int)((K + BK - 1) / BK);
    const int share = ((steps + kFewWaves - 1) / kFewWaves + kWindow - 1) & ~(kWindow - 1);
    const int from = wave * share, to = from + share < steps ? from + share : steps;

    float4v acc = {0.0f, 0.0f, 0.0f, 0.0f};
    if (from < to) {
        const int r = lane & 15, k = 32 * (lane >> 4);
        const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
            (void*)(w_codes + n0 * K), 0, (int)(w_rows * K), kRawBufferFlags);
        const __amdgpu_buffer_rsrc_t ra =
            __builtin_amdgcn_make_buffer_rsrc((void*)a_codes, 0, (int)(M * K), kRawBufferFlags);
        // (rows past M and N read as zeros or as the last row's, and are not stored)
        const uint32_t vw = (uint32_t)r * (uint32_t)K + k;
        const int64_t w_first = w_square ? n0 / BK : n0;
        const Scales<kBytes> scales_w(w_scales, w_first, w_square ? (N + BK - 1) / BK : N, steps);
        const Scales<kBytes> scales_a(a_scales, 0, M, steps);
        const int off_w = (w_square ? 0 : r < w_rows ? r : w_rows - 1) * steps;
        const int m = r < M ? r : (int)M - 1;
        const uint32_t va = (uint32_t)m * (uint32_t)K + k;
        const int off_a = m * steps;
        // W of four blocks at once, those of the next four on their way
        int8v w[2][kWindow];
        uint32_t ew[2], ea[2];
        const auto load = [&](int which, int s) {
#pragma unroll
            for (int u = 0; u < kWindow; u++) w[which][u] = load_codes(rw, vw, k, s + u, K);
            ew[which] = scales_w.window(off_w + s);
            ea[which] = scales_a.window(off_a + s);
        };
        const auto multiply = [&](auto which, int s) {
            constexpr int b = decltype(which)::value;
            const uint32_t sw = scales_w.take(ew[b], off_w + s), sa = scales_a.take(ea[b], off_a + s);
            int8v a[kWindow];
#pragma unroll
            for (int u = 0; u < kWindow; u++) a[u] = load_codes(ra, va, k, s + u, K);
#pragma unroll
            for (int u = 0; u < kWindow; u++) {
                // (blocks past the last are zeros, and their bytes another row's: not NaN then)
                const bool past = s + u >= steps;
                const uint32_t eu = past ? 127u : sw >> (8 * u), fu = past ? 127u : sa >> (8 * u);
                if constexpr (kBf16) {
                    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[b][u], a[u], acc, 0, 0, 0, (int)eu, 0,
                                                                           (int)fu);
                } else {
                    bf16x8 x[4], y[4];
                    widen(w[b][u], eu, x);
                    widen(a[u], fu, y);
#pragma unroll
                    for (int q = 0; q < 4; q++) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[q], y[q], acc, 0, 0, 0);
                }
            }
        };
        load(0, from);
        for (int s = from; s < to; s += 2 * kWindow) {
            load(1, s + kWindow);
            multiply(std::integral_constant<int, 0>{}, s);
            if (s + kWindow >= to) break;
            load(0, s + 2 * kWindow);
            multiply(std::integral_constant<int, 1>{}, s + kWindow);
        }
    }
    sums[wave][lane] = acc;
    __syncthreads();
    if (wave != 0) return;
    for (int p = 1; p < kFewWaves; p++) acc += sums[p][lane];
    // lane: row lane % 16 of A, columns n0 + 4 (lane / 16) .. + 3
    const int64_t row = lane & 15, col = n0 + 4 * (lane >> 4);
    if (row >= M) return;
#pragma unroll
    for (int r = 0; r < 4; r++) {
        if (col + r >= N) continue;
        if constexpr (kBf16)
            reinterpret_cast<__bf16*>(c)[row * ldc + col + r] = (__bf16)acc[r];
        else
            reinterpret_cast<float*>(c)[row * ldc + col + r] = acc[r];
    }
}

template <bool kBf16, bool kBytes>
hipError_t launch_few(const Fp8Gemm& g, hipStream_t stream) {
    const int64_t groups = (g.N + 15) / 16;
    if (!launchable(groups, kFewThreads)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((few_kernel<kBf16, kBytes>), dim3((unsigned)groups), dim3(kFewThreads), 0, stream,
                       g.a_codes, g.a_scales, g.w_codes, g.w_scales, g.w_square, g.M, g.N, g.K, g.c, g.ldc);
    return hipGetLastError();
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

// The splits' sums, added in their order.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads)
join_kernel(const float* __restrict__ parts, int splits, int64_t M, int64_t N, void* __restrict__ c, int64_t ldc) {
    const int64_t total = M * N;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        float v = parts[i];
        for (int p = 1; p < splits; p++) v += parts[p * total + i];
        const int64_t at = i / N * ldc + i % N;
        if constexpr (kBf16)
            reinterpret_cast<__bf16*>(c)[at] = (__bf16)v;
        else
            reinterpret_cast<float*>(c)[at] = v;
    }
}

// How a product is cut: the tile, and the splits of K.
struct Plan {
    int tile;  // 0: few_kernel; rows and columns of a tile else
    int splits;
};

// Tiles whose workgroups fill the CUs (128: half of them, for what two parts of K then
// bring), and few_kernel for few rows.  In us, results in bf16, W from memory:
//   few_kernel and tiles of 64:  1 x 6144 x 4096  8.4, 10.7;  4  9.0, 10.8;  16  10.9, 11.2;
//                                16 x 28672 x 8192  72, 53 (W's tiles fill the CUs)
//   64 and 128:   256 x 6144 x 4096  24, 27;  512  38, 36;  1024 x 4096 x 4096  35, 27
//   128 and 256:  2048 x 4096 x 4096  44, 100;  4096 x 4096 x 4096  82, 68
// Where tiles of 256 fill the CUs too, an estimate of the time decides: rounds of 256 of
// them, or of 512 of the smaller, times steps and what a tile has besides, its results above
// all (more where rows of C are no whole lines), from fits to measured times.  128 and 256 in
// bf16 and fp32:  4096 x 5004 x 2048  66, 77 and 93, 121;  1929 x 25702 x 2320  199, 201 and 261,
// 304;  8192 x 8192 x 1024  118, 89 and 151, 146;  1024 x 28672 x 8192  286, 216 and 393, 375.
// K is parted where tiles leave CUs free, so that there are up to two workgroups on each, of 8
// steps at least; parted and whole:  64 x 6144 x 4096  16.0, 22.8;  300 x 1024 x 16384  26,
// 78;  512 x 6144 x 4096  36, 34 (its results are many for what is gained).
constexpr int kCus = 256;

bool wide_tiles(int64_t M, int64_t N, int64_t steps, bool bf16, bool whole_lines) {
    const int64_t wide = ((M + 255) / 256) * ((N + 255) / 256), narrow = ((M + 127) / 128) * ((N + 127) / 128);
    if (wide < kCus) return false;
    // us of a step, and of a tile's start and end (no sizes overflow)
    const double a = bf16 ? 1.6 : 3.0, b = bf16 ? 1.1 : 1.71;
    const double ea = (bf16 ? 9.0 : 12.0) + (whole_lines ? 0.0 : 8.0), eb = bf16 ? 5.6 : 5.2;
    return (double)((wide + kCus - 1) / kCus) * (a * (double)steps + ea) <=
           (double)((narrow + 2 * kCus - 1) / (2 * kCus)) * (b * (double)steps + eb);
}

// (results' type and lines choose between tiles that both leave K whole: no workspace depends
// on them)
Plan plan_of(int64_t M, int64_t N, int64_t K, bool bf16, bool whole_lines) {
    const auto tiles = [&](int64_t t) { return ((M + t - 1) / t) * ((N + t - 1) / t); };
    if (M <= 4 || (M <= 16 && tiles(64) < kCus)) return {0, 1};
    Plan p;
    const int64_t steps = (K + BK - 1) / BK;
    p.tile = M <= 64 || 2 * tiles(128) < kCus ? 64 : wide_tiles(M, N, steps, bf16, whole_lines) ? 256 : 128;
    const int64_t count = tiles(p.tile);
    int64_t splits = count >= kCus ? 1 : 2 * kCus / count;
    splits = splits < steps / (2 * kWindow) ? splits : steps / (2 * kWindow);
    p.splits = (int)(splits < 1 ? 1 : splits > 16 ? 16 : splits);
    return p;
}

template <int BM, int BN, int kWavesM, int kWavesN, int kStages, bool kBf16, bool kBytes>
hipError_t launch_tile(const Fp8Gemm& g, int splits, hipStream_t stream) {
    constexpr int kSmem = kStages * (BM + BN) * BK;
    const auto kernel = tile_kernel<BM, BN, kWavesM, kWavesN, kStages, kBf16, kBytes>;
    const int64_t tiles_m = (g.M + BM - 1) / BM, tiles_n = (g.N + BN - 1) / BN;
    if (!launchable(tiles_m * tiles_n * splits, 64 * kWavesM * kWavesN)) return hipErrorInvalidConfiguration;
    // dynamic LDS above 64 KB must be allowed per kernel (idempotent, any device)
    const hipError_t err =
        hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (err != hipSuccess) return err;
    float* const parts = reinterpret_cast<float*>(g.workspace);
    hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles_m * tiles_n * splits)), dim3(64 * kWavesM * kWavesN), kSmem, stream, g.a_codes,
                       g.a_scales, g.w_codes, g.w_scales, g.w_square, g.M, g.N, g.K, g.c, g.ldc, (int)tiles_m,
                       (int)tiles_n, parts, splits);
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess || splits == 1) return st;
    const int64_t blocks = (g.M * g.N + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(join_kernel<kBf16>, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(kThreads), 0, stream,
                       parts, splits, g.M, g.N, g.c, g.ldc);
    return hipGetLastError();
}

// Whether rows of C are whole lines of the caches.
bool whole_lines(const Fp8Gemm& g) {
    return ((reinterpret_cast<uintptr_t>(g.c) | (uintptr_t)(g.ldc * (g.c_bf16 ? 2 : 4))) & 127) == 0;
}

template <bool kBf16, bool kBytes>
hipError_t launch_of(const Fp8Gemm& g, hipStream_t stream) {
    const Plan p = plan_of(g.M, g.N, g.K, kBf16, whole_lines(g));
    if (p.tile == 0) return launch_few<kBf16, kBytes>(g, stream);
    if (kBytes || p.tile == 64) return launch_tile<64, 64, 2, 2, 4, kBf16, kBytes>(g, p.splits, stream);
    if constexpr (!kBytes) {
        if (p.tile == 128) return launch_tile<128, 128, 2, 2, 2, kBf16, false>(g, p.splits, stream);
        return launch_tile<256, 256, 2, 2, 2, kBf16, false>(g, p.splits, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace

int64_t fp8_gemm_workspace(int64_t M, int64_t N, int64_t K) {
    const Plan p = plan_of(M, N, K, true, true);
    return p.splits > 1 ? p.splits * M * N * 4 : 0;
}

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
    if (g.c_bf16) return bytes ? launch_of<true, true>(g, stream) : launch_of<true, false>(g, stream);
    return bytes ? launch_of<false, true>(g, stream) : launch_of<false, false>(g, stream);
}

}  // namespace if4
