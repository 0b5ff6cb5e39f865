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
// eight bits of its order at a time (the numbers of sums with each next byte, in LDS),
// then goes through the tokens in order once more and writes those above it, and of those
// equal to it the first.

constexpr int kThreads = 1024, kWaves = kThreads / 64;

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

__global__ void __launch_bounds__(kThreads) select_kernel(const SelectArgs p) {
    __shared__ uint32_t count[256];
    __shared__ uint32_t above[2][kWaves];
    __shared__ uint32_t found[2];
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
    if (need) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) count[tid] = 0;
            __syncthreads();
            for (int i = first + tid; i < last; i += kThreads) {
                const uint32_t o = order_of(in[i]);
                if (shift == 24 || o >> (shift + 8) == prefix) atomicAdd(&count[(o >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (tid < 64) {  // from the largest byte down, four to a lane
                uint32_t c[4], sum = 0;
                for (int j = 0; j < 4; j++) sum += c[j] = count[255 - 4 * tid - j];
                uint32_t upto = sum;
                for (int d = 1; d < 64; d *= 2) {
                    const uint32_t o = (uint32_t)__shfl_up((int)upto, d);
                    upto += lane >= d ? o : 0;
                }
                uint32_t before = upto - sum;
                if (before < need && need <= upto) {
                    int j = 0;
                    while (before + c[j] < need) before += c[j++];
                    found[0] = 255u - 4u * (uint32_t)tid - (uint32_t)j;
                    found[1] = need - before;
                }
            }
            __syncthreads();
            prefix = prefix << 8 | found[0];
            need = found[1];  // of those with this prefix
            __syncthreads();
        }
    } else {
        prefix = 0xFFFFFFFFu;  // none between, NaN neither (need is 0)
    }
    // (a chunk's sums have been read before any of its outputs is written, and these lie no
    // further than the chunk: `out` may be `in`)
    uint32_t written = 0, equals = 0;
    for (int base = 0; base < n; base += kThreads) {
        const int i = base + tid;
        const float v = i < n ? in[i] : 0.0f;
        const uint32_t o = order_of(v);
        const bool fixed = i < n && (i < first || i >= last), free = i < n && !fixed;
        const bool equal = free && o == prefix;
        const uint64_t lower = ((uint64_t)1 << lane) - 1;
        const uint64_t em = __builtin_amdgcn_ballot_w64(equal);
        if (lane == 0) above[0][wave] = (uint32_t)__builtin_popcountll(em);
        __syncthreads();
        uint32_t er = equals + (uint32_t)__builtin_popcountll(em & lower);
        for (int w = 0; w < kWaves; w++) {
            er += w < wave ? above[0][w] : 0;
            equals += above[0][w];
        }
        const bool take = fixed || (free && o > prefix) || (equal && er < need);
        const uint64_t tm = __builtin_amdgcn_ballot_w64(take);
        if (lane == 0) above[1][wave] = (uint32_t)__builtin_popcountll(tm);
        __syncthreads();
        uint32_t at = written + (uint32_t)__builtin_popcountll(tm & lower);
        for (int w = 0; w < kWaves; w++) {
            at += w < wave ? above[1][w] : 0;
            written += above[1][w];
        }
        if (take) {
            kept[at] = i;
            if (out) out[at] = v;
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
