// Choosing the tokens that stay in the paged IF4 KV cache and moving them together, for
// gfx950 (definitions in include/if4_kv_evict.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_evict_internal.h"
#include "kv_internal.h"

namespace if4 {
namespace {

// ---------------------------------------------------------------------------
// Select.  One workgroup per sequence and kv head finds the sum that is the last to be kept,
// eleven (then eleven and ten) bits of its order at a time: the numbers of sums with each
// next digit, in LDS.  Then it goes through the tokens in order once more and writes those
// above it, and of those equal to it the first.
//
// Bound by the latency of one workgroup's passes over its sums: a thread asks for 8 at once
// when it counts and 4 when it writes.  Sums of one size are many (zeros, above all), and
// atomics on one place of LDS wait for one another: the lanes with the first lane's digit
// add once.

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kDigits = 2048;

// Bits that order sums as numbers do: zeros equal, NaN above all.
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t u = __float_as_uint(v);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    if ((u & 0x7FFFFFFFu) == 0) return 0x80000000u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct SelectArgs {
    if4_kv_mass mass;
    const int32_t* seq_lens;
    int32_t* kept;
    int kv_heads, keep, recent, sinks;
};

__device__ __forceinline__ uint32_t rank_in(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// One more of `digit` for each lane with `on`.
__device__ __forceinline__ void count_digit(uint32_t* count, uint32_t digit, bool on) {
    const uint64_t live = __builtin_amdgcn_ballot_w64(on);
    if (live == 0) return;
    const int leader = __builtin_ctzll(live);
    const uint32_t first = (uint32_t)__builtin_amdgcn_readlane((int)digit, leader);
    const bool same = on && digit == first;
    const uint64_t alike = __builtin_amdgcn_ballot_w64(same);
    if ((int)(threadIdx.x & 63) == leader)
        atomicAdd(&count[first], (uint32_t)__builtin_popcountll(alike));
    else if (on && !same)
        atomicAdd(&count[digit], 1u);
}

__global__ void __launch_bounds__(kThreads) select_kernel(const SelectArgs p) {
    __shared__ uint32_t count[kDigits];
    __shared__ uint32_t sums[kWaves], found[2];
    __shared__ uint32_t before[2][kWaves];  // above, and equal << 16, of each wave
    const int b = blockIdx.x / p.kv_heads, head = blockIdx.x - b * p.kv_heads;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = p.mass.rows ? p.mass.rows[b] : b;
    int32_t* const kept = p.kept + (int64_t)blockIdx.x * p.keep;
    int n = 0;
    if (row >= 0 && row < p.mass.mass_rows) {
        n = p.seq_lens[b];
        n = n < 0 ? 0 : n > p.mass.width ? (int)p.mass.width : n;
    }
    const float* const in = p.mass.in + row * p.mass.in_stride_row + head * p.mass.in_stride_head;
    float* const out = p.mass.out ? p.mass.out + row * p.mass.out_stride_row + head * p.mass.out_stride_head : nullptr;
    if (n <= p.keep) {
        for (int i = tid; i < p.keep; i += kThreads) {
            kept[i] = i < n ? i : -1;
            if (out && out != in && i < n) out[i] = in[i];
        }
        return;
    }
    const int first = p.sinks, last = n - p.recent;  // (sinks + recent <= keep < n)
    uint32_t need = (uint32_t)(p.keep - p.sinks - p.recent);  // of those between, fewer than they are
    uint32_t prefix = 0;
    int shift = 32;
    while (need && shift > 0) {
        const int bits = shift > 11 ? 11 : shift, below = shift - bits;
        for (int i = tid; i < kDigits; i += kThreads) count[i] = 0;
        __syncthreads();
        const uint32_t mask = (1u << bits) - 1;
        for (int base = first; base < last; base += 8 * kThreads) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int i = base + j * kThreads + tid;
                v[j] = i < last ? in[i] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t o = order_of(v[j]);
                const bool on = base + j * kThreads + tid < last && (shift == 32 || o >> shift == prefix);
                count_digit(count, (o >> below) & mask, on);
            }
        }
        __syncthreads();
        // digits from the largest down, two to a thread; sums of the waves before
        uint32_t c[2], sum = 0;
#pragma unroll
        for (int j = 0; j < 2; j++) sum += c[j] = count[kDigits - 1 - 2 * tid - j];
        uint32_t upto = sum;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t o = (uint32_t)__shfl_up((int)upto, d);
            upto += lane >= d ? o : 0;
        }
        if (lane == 63) sums[wave] = upto;
        __syncthreads();
        for (int w = 0; w < wave; w++) upto += sums[w];
        const uint32_t above = upto - sum;
        if (above < need && need <= upto) {
            const int j = above + c[0] < need;
            found[0] = (uint32_t)(kDigits - 1 - 2 * tid - j);
            found[1] = need - above - (j ? c[0] : 0);
        }
        __syncthreads();
        prefix = prefix << bits | found[0];
        need = found[1];  // of those with this prefix
        shift = below;
    }
    if (shift == 32) prefix = 0xFFFFFFFFu;  // none between, NaN neither (need is 0)
    // Position i goes to the number of those above before it, and of those equal as many as are
    // kept.  (A chunk's sums have been read before any of its outputs is written, and these
    // lie no further than the chunk: `out` may be `in`.)
    uint32_t aboves = 0, equals = 0;
    int turn = 0;
    const auto load = [&](int base, float (&v)[4]) {
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] = base + 4 * tid + j < n ? in[base + 4 * tid + j] : 0.0f;
    };
    float next[4];
    load(0, next);
    for (int base = 0; base < n; base += 4 * kThreads, turn ^= 1) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] = next[j];
        load(base + 4 * kThreads, next);
        bool up[4], equal[4];
        uint32_t a = 0, e = 0, wave_a = 0, wave_e = 0;  // before this thread's first, in the wave
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int i = base + 4 * tid + j;
            const uint32_t o = order_of(v[j]);
            const bool between = i >= first && i < last;
            up[j] = i < n && (!between || o > prefix);
            equal[j] = between && o == prefix;
            const uint64_t am = __builtin_amdgcn_ballot_w64(up[j]), em = __builtin_amdgcn_ballot_w64(equal[j]);
            a += rank_in(am);
            e += rank_in(em);
            wave_a += (uint32_t)__builtin_popcountll(am);
            wave_e += (uint32_t)__builtin_popcountll(em);
        }
        if (lane == 0) before[turn][wave] = wave_a | wave_e << 16;
        __syncthreads();
        uint32_t of_waves = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kWaves; w++) {
            const uint32_t c = before[turn][w];
            of_waves += w < wave ? c : 0;
            all += c;
        }
        a += aboves + (of_waves & 0xFFFFu);
        e += equals + (of_waves >> 16);
        aboves += all & 0xFFFFu;
        equals += all >> 16;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (up[j] || (equal[j] && e < need)) {
                const uint32_t at = a + (e < need ? e : need);
                kept[at] = base + 4 * tid + j;
                if (out) out[at] = v[j];
            }
            a += up[j];
            e += equal[j];
        }
    }
}

// ---------------------------------------------------------------------------
// Compact.  A workgroup fills one tile of 16 tokens of one sequence and kv head: V's 16
// pieces of each token lie 16 tokens apart, so that a whole tile is written in one piece
// of 8 D bytes, and what is read of a source tile is read by one workgroup and its
// neighbours.

constexpr int kCopyThreads = 256;

struct CompactArgs {
    if4_kv_cache cache;
    const int32_t *page_table, *kept, *new_table;
    int64_t table_stride, new_stride, keep;
    int tiles_of_keep;
    Divisor tiles;  // of 16 tokens in a page
};

template <int D>
__global__ void __launch_bounds__(kCopyThreads) compact_kernel(const CompactArgs p) {
    __shared__ int64_t from[16];  // cache rows of the tile's tokens, -1: none
    const int kv_heads = (int)p.cache.kv_heads;
    const int bh = blockIdx.x / p.tiles_of_keep, tile = blockIdx.x - bh * p.tiles_of_keep;
    const int b = bh / kv_heads, head = bh - b * kv_heads, tid = threadIdx.x;
    const uint32_t np = p.tiles.into((uint32_t)tile);
    if (np >= p.new_stride) return;
    const int page = p.new_table[b * p.new_stride + np];
    if (page < 0 || page >= p.cache.pages) return;
    const int64_t to = ((int64_t)page * kv_heads + head) * p.tiles.n + (tile - np * p.tiles.n);
    if (tid < 16) {
        const int64_t i = (int64_t)tile * 16 + tid;
        const int j = i < p.keep ? p.kept[(int64_t)bh * p.keep + i] : -1;
        int64_t row = -1;
        if (j >= 0) {
            const uint32_t t = (uint32_t)j >> 4, sp = p.tiles.into(t);
            if (sp < p.table_stride) {
                int src = p.page_table[b * p.table_stride + sp];
                src = src < p.cache.pages - 1 ? src : (int)p.cache.pages - 1;
                src = src > 0 ? src : 0;
                row = (((int64_t)src * kv_heads + head) * p.tiles.n + (t - sp * p.tiles.n)) * 16 + (j & 15);
            }
        }
        from[tid] = row;
    }
    __syncthreads();
    {  // V codes: thread (piece, token)
        const int tok = tid & 15, piece = tid >> 4;
        const int64_t row = from[tok];
        if (row >= 0) {
            const uint8_t* const x = p.cache.v_codes + (row >> 4) * (8 * D) + (piece * 16 + (row & 15)) * (D / 32);
            uint8_t* const y = p.cache.v_codes + to * (8 * D) + tid * (D / 32);
            if constexpr (D == 64)
                *reinterpret_cast<uint16_t*>(y) = *reinterpret_cast<const uint16_t*>(x);
            else if constexpr (D == 128)
                *reinterpret_cast<uint32_t*>(y) = *reinterpret_cast<const uint32_t*>(x);
            else
                *reinterpret_cast<uint2*>(y) = *reinterpret_cast<const uint2*>(x);
        }
    }
    if (tid < D) {  // V scales: thread (group, token)
        const int tok = tid & 15, g = tid >> 4;
        const int64_t row = from[tok];
        if (row >= 0) p.cache.v_scales[to * D + tid] = p.cache.v_scales[(row >> 4) * D + g * 16 + (row & 15)];
    }
    if (tid < D / 2) {  // K codes: 16 bytes, D/32 threads to a token
        const int tok = tid / (D / 32), c = tid % (D / 32);
        const int64_t row = from[tok];
        if (row >= 0)
            reinterpret_cast<uint4*>(p.cache.k_codes)[(to * 16 + tok) * (D / 32) + c] =
                reinterpret_cast<const uint4*>(p.cache.k_codes)[row * (D / 32) + c];
    } else if (tid >= kCopyThreads - D / 4) {  // K scales: 4 bytes, D/64 threads to a token
        const int i = tid - (kCopyThreads - D / 4), tok = i / (D / 64), c = i % (D / 64);
        const int64_t row = from[tok];
        if (row >= 0)
            reinterpret_cast<uint32_t*>(p.cache.k_scales)[(to * 16 + tok) * (D / 64) + c] =
                reinterpret_cast<const uint32_t*>(p.cache.k_scales)[row * (D / 64) + c];
    }
}

}  // namespace

hipError_t launch_kv_select(const if4_kv_mass& m, const int32_t* seq_lens, int64_t batch,
                            int64_t kv_heads, int64_t keep, int64_t recent, int64_t sinks,
                            int32_t* kept, hipStream_t stream) {
    const SelectArgs p = {m, seq_lens, kept, (int)kv_heads, (int)keep, (int)recent, (int)sinks};
    hipLaunchKernelGGL(select_kernel, dim3((unsigned)(batch * kv_heads)), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_kv_compact(const if4_kv_cache& c, const int32_t* page_table,
                             int64_t table_stride, const int32_t* kept, int64_t batch,
                             int64_t keep, const int32_t* new_table, int64_t new_stride,
                             hipStream_t stream) {
    const int64_t tiles = (keep + 15) / 16;
    if (tiles > 0x7FFFFFFF / (batch * c.kv_heads)) return hipErrorInvalidValue;
    const CompactArgs p = {c, page_table, kept, new_table, table_stride, new_stride, keep, (int)tiles, Divisor(c.page_size / 16)};
    const dim3 grid((unsigned)(batch * c.kv_heads * tiles));
    const auto k = c.head_dim == 64 ? compact_kernel<64> : c.head_dim == 128 ? compact_kernel<128> : compact_kernel<256>;
    hipLaunchKernelGGL(k, grid, dim3(kCopyThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace if4
