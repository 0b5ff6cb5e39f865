// Choosing the tokens that stay in the paged IF4 KV cache and moving them together, for
// gfx950 (definitions in include/if4_kv_evict.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_evict_internal.h"
#include "kv_internal.h"
#include "launch_limit.h"

namespace if4 {
namespace {

// ---------------------------------------------------------------------------
// Select.  The sum that is the last to be kept is found eleven (then eleven and ten) bits of
// its order at a time: the numbers of sums with each next digit, in LDS.  Then the tokens
// are gone through in order once more, and those above it are written, and of those equal to
// it the first.
//
// One workgroup per sequence and kv head does all of it (select_kernel) where rows are
// short, or are many.  Bound by the latency of its four passes, with one workgroup on a CU: a
// thread asks for 8 sums at once when it counts and 4 when it writes (256 rows of 16384 sums
// 28 us, of which the first pass reads memory and the others the caches).  Sums of one size
// are many (zeros, above all), and atomics on one place of LDS wait for one another: the lanes
// with the first lane's digit add once.
//
// Of long rows a workgroup takes a segment, and the passes are launches (segment kernels):
// each leaves its digits' numbers in the workspace, and each workgroup of the next adds them
// up itself.  16 rows of 131071 sums: 41 us, 155 in one workgroup each.

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

// A row of sums, as its workgroups see it.
struct Row {
    int n, first, last;  // tokens; those first .. last - 1 are chosen from
    const float* in;
    float* out;
    int32_t* kept;
    __device__ __forceinline__ Row(const SelectArgs& p, int pair) {
        const int b = pair / p.kv_heads, head = pair - b * p.kv_heads;
        const int64_t row = p.mass.rows ? p.mass.rows[b] : b;
        n = 0;
        if (row >= 0 && row < p.mass.mass_rows) {
            n = p.seq_lens[b];
            n = n < 0 ? 0 : n > p.mass.width ? (int)p.mass.width : n;
        }
        first = p.sinks;  // (sinks + recent <= keep)
        last = n - p.recent;
        in = p.mass.in + row * p.mass.in_stride_row + head * p.mass.in_stride_head;
        out = p.mass.out ? p.mass.out + row * p.mass.out_stride_row + head * p.mass.out_stride_head : nullptr;
        kept = p.kept + (int64_t)pair * p.keep;
    }
};

constexpr int bits_of(int level) { return level < 2 ? 11 : 10; }
constexpr int below(int level) { return level == 0 ? 21 : level == 1 ? 10 : 0; }

// Counts the digits of sums from .. to - 1 that have the prefix of the levels before.
__device__ __forceinline__ void count_digits(uint32_t* count, const float* in, int from, int to, int level,
                                             uint32_t prefix) {
    for (int i = threadIdx.x; i < kDigits; i += kThreads) count[i] = 0;
    __syncthreads();
    const int under = below(level), width = bits_of(level);
    const uint32_t mask = (1u << width) - 1;
    for (int base = from; base < to; base += 8 * kThreads) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int i = base + j * kThreads + threadIdx.x;
            v[j] = i < to ? in[i] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const uint32_t o = order_of(v[j]);
            const bool on = base + j * kThreads + (int)threadIdx.x < to && (level == 0 || o >> (under + width) == prefix);
            count_digit(count, (o >> under) & mask, on);
        }
    }
    __syncthreads();
}

// The digit that the sum number `need` from the largest has, of c[0] and c[1] sums with this
// thread's digits kDigits - 1 - 2 t and the one below: found[0]; and its number among those
// with the digit: found[1].
struct Shared {
    uint32_t sums[kWaves], found[2];
};
__device__ __forceinline__ void find_digit(Shared& sh, const uint32_t (&c)[2], uint32_t need) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t sum = c[0] + c[1];
    uint32_t upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = (uint32_t)__shfl_up((int)upto, d);
        upto += lane >= d ? o : 0;
    }
    if (lane == 63) sh.sums[wave] = upto;
    __syncthreads();
    for (int w = 0; w < wave; w++) upto += sh.sums[w];
    const uint32_t above = upto - sum;
    if (above < need && need <= upto) {
        const int j = above + c[0] < need;
        sh.found[0] = (uint32_t)(kDigits - 1 - 2 * tid - j);
        sh.found[1] = need - above - (j ? c[0] : 0);
    }
    __syncthreads();
}

// Writes the tokens from .. to - 1 that stay: position i goes to the number of those above
// before it, and of those equal as many as are kept; `aboves` (the first and last ones of a row
// among them) and `equals` lie before `from`.  A chunk's sums have been read before any
// of its outputs is written, and these lie no further than the chunk: `out` may be `in`
// where one workgroup writes the row.  (Two sequences of one row, written in place, count
// each other's sums in between, and may come to more than `keep`: none goes past it.)
__device__ __forceinline__ void write_kept(const Row& row, float* out, int keep, int from, int to, uint32_t prefix,
                                           uint32_t need, uint32_t aboves, uint32_t equals) {
    __shared__ uint32_t before[2][kWaves];  // above, and equal << 16, of each wave
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int turn = 0;
    const auto load = [&](int base, float (&v)[4]) {
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] = base + 4 * tid + j < to ? row.in[base + 4 * tid + j] : 0.0f;
    };
    float next[4];
    load(from, next);
    for (int base = from; base < to; base += 4 * kThreads, turn ^= 1) {
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
            const bool between = i >= row.first && i < row.last;
            up[j] = i < to && (!between || o > prefix);
            equal[j] = i < to && between && o == prefix;
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
                if (at < (uint32_t)keep) {
                    row.kept[at] = base + 4 * tid + j;
                    if (out) out[at] = v[j];
                }
            }
            a += up[j];
            e += equal[j];
        }
    }
}

// A prefix that no sum between has above or at it: none of them stays.
constexpr uint32_t kNone = 0xFFFFFFFFu;

__global__ void __launch_bounds__(kThreads) select_kernel(const SelectArgs p) {
    __shared__ uint32_t count[kDigits];
    __shared__ Shared sh;
    const Row row(p, blockIdx.x);
    if (row.n <= p.keep) {
        for (int i = threadIdx.x; i < p.keep; i += kThreads) {
            row.kept[i] = i < row.n ? i : -1;
            if (row.out && row.out != row.in && i < row.n) row.out[i] = row.in[i];
        }
        return;
    }
    uint32_t need = (uint32_t)(p.keep - p.sinks - p.recent);  // of those between, fewer than they are
    uint32_t prefix = need ? 0 : kNone;
    for (int level = 0; level < 3 && need; level++) {
        count_digits(count, row.in, row.first, row.last, level, prefix);
        const uint32_t c[2] = {count[kDigits - 1 - 2 * threadIdx.x], count[kDigits - 2 - 2 * threadIdx.x]};
        find_digit(sh, c, need);
        prefix = prefix << bits_of(level) | sh.found[0];
        need = sh.found[1];  // of those with this prefix
    }
    write_kept(row, row.out, p.keep, 0, row.n, prefix, need, 0, 0);
}

// Workspace of the segment kernels: [3][rows][segments][kDigits] numbers, then [rows][segments]
// States, then the sums of rows that are written in place, [rows][keep].
struct State {
    uint32_t prefix, need;  // of the row, after the levels so far
    uint32_t above;         // sums above it in the segments before this one
    uint32_t unused;
};
struct SegmentArgs {
    SelectArgs s;
    uint32_t* counts;
    State* states;
    float* moved;  // NULL: out is another tensor
    int rows, segments, segment;  // segments of a row, sums of each
};

// What the levels before `level` say, from their numbers; `equals` are the sums equal to
// the prefix in the segments before.
__device__ __forceinline__ State resolve(const SegmentArgs& p, Shared& sh, int pair, int segment, int level,
                                         uint32_t& equals) {
    __shared__ uint32_t part[2];
    State st = {0, (uint32_t)(p.s.keep - p.s.sinks - p.s.recent), 0, 0};
    equals = 0;
    if (level == 0) return st;
    State* const own = p.states + (int64_t)pair * p.segments + segment;
    if (level > 1) st = *own;
    const int tid = threadIdx.x;
    const uint32_t* const at = p.counts + (((int64_t)(level - 1) * p.rows + pair) * p.segments) * kDigits;
    uint32_t c[2] = {0, 0}, mine[2] = {0, 0};
    for (int g = 0; g < p.segments; g++)
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const uint32_t v = at[(int64_t)g * kDigits + kDigits - 1 - 2 * tid - j];
            c[j] += v;
            mine[j] += g < segment ? v : 0;
        }
    if (tid < 2) part[tid] = 0;
    find_digit(sh, c, st.need);
    const uint32_t digit = sh.found[0];
    uint32_t up = 0;
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const uint32_t d = (uint32_t)(kDigits - 1 - 2 * tid - j);
        up += d > digit ? mine[j] : 0;
        if (d == digit) part[1] = mine[j];
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) up += (uint32_t)__shfl_xor((int)up, d);
    if ((tid & 63) == 0 && up) atomicAdd(&part[0], up);
    __syncthreads();
    st.prefix = st.prefix << bits_of(level - 1) | digit;
    st.need = sh.found[1];
    st.above += part[0];
    equals = part[1];
    if (tid == 0) *own = st;
    return st;
}

// (a segment's part of the tokens that are chosen from)
template <int kLevel>
__global__ void __launch_bounds__(kThreads) segment_count_kernel(const SegmentArgs p) {
    __shared__ uint32_t count[kDigits];
    __shared__ Shared sh;
    const int pair = blockIdx.x / p.segments, segment = blockIdx.x - pair * p.segments;
    const Row row(p.s, pair);
    if (row.n <= p.s.keep || p.s.keep == p.s.sinks + p.s.recent) return;
    uint32_t equals;
    const State st = resolve(p, sh, pair, segment, kLevel, equals);
    const int from = segment * p.segment, to = from + p.segment;
    count_digits(count, row.in, from > row.first ? from : row.first, to < row.last ? to : row.last, kLevel, st.prefix);
    uint32_t* const at = p.counts + (((int64_t)kLevel * p.rows + pair) * p.segments + segment) * kDigits;
    for (int i = threadIdx.x; i < kDigits; i += kThreads) at[i] = count[i];
}

__global__ void __launch_bounds__(kThreads) segment_write_kernel(const SegmentArgs p) {
    __shared__ Shared sh;
    const int pair = blockIdx.x / p.segments, segment = blockIdx.x - pair * p.segments;
    const Row row(p.s, pair);
    const int from = segment * p.segment, to = from + p.segment < row.n ? from + p.segment : row.n;
    if (row.n <= p.s.keep) {
        for (int i = from + threadIdx.x; i < from + p.segment && i < p.s.keep; i += kThreads) {
            row.kept[i] = i < row.n ? i : -1;
            if (row.out && row.out != row.in && i < row.n) row.out[i] = row.in[i];
        }
        return;
    }
    State st = {kNone, 0, 0, 0};
    uint32_t equals = 0;
    if (p.s.keep > p.s.sinks + p.s.recent) st = resolve(p, sh, pair, segment, 3, equals);
    const int fixed = (from < row.first ? from : row.first) + (from > row.last ? from - row.last : 0);
    write_kept(row, p.moved ? p.moved + (int64_t)pair * p.s.keep : row.out, p.s.keep, from, to, st.prefix, st.need,
               st.above + (uint32_t)fixed, equals);
}

// The sums of rows that are written in place, once all of them have been read.
__global__ void __launch_bounds__(kThreads) segment_move_kernel(const SegmentArgs p) {
    const int pair = blockIdx.x / p.segments, segment = blockIdx.x - pair * p.segments;
    const Row row(p.s, pair);
    if (row.n <= p.s.keep) return;
    const int from = segment * p.segment;
    for (int i = from + threadIdx.x; i < from + p.segment && i < p.s.keep; i += kThreads)
        row.out[i] = p.moved[(int64_t)pair * p.s.keep + i];
}

// Sums of a segment, 0 where one workgroup takes a row: rows that are short, or so many that
// they keep the chip busy without being parted.  A workgroup for each CU, and 16 segments of a
// row at most, because each workgroup reads the numbers of all segments of its row (64 rows of
// 131071 sums in segments of 8192: 113 us).  In us, one workgroup a row and segments:
//   8 rows of 16384 sums 25, 26, of 24000 34, 27, of 131071 153, 41, of 300000 347, 57;
//   64 rows of 16384 26, 28, of 24000 35, 31, of 131071 159, 64;
//   128 rows of 24000 35, 39, of 40000 54, 49, of 131071 168, 103;  256 of 24000 37, 66.
int64_t segment_of(const if4_kv_mass& m, int64_t rows, int64_t keep) {
    constexpr int64_t kUnit = 8 * kThreads;
    if (m.width <= (rows > 64 ? 4 : 2) * kUnit || rows > 128 || keep >= m.width) return 0;
    const int64_t each = (m.width * (rows > 16 ? rows : 16) + 255) / 256;
    const int64_t segment = (each + kUnit - 1) / kUnit * kUnit;
    return segment < m.width ? segment : 0;
}

// ---------------------------------------------------------------------------
// Compact.  A workgroup fills one tile of 16 tokens of one sequence and kv head: V's 16
// pieces of each token lie 16 tokens apart, so that a whole tile is written in one piece
// of 8 D bytes, and what is read of a source tile is read by one workgroup and its
// neighbours.  Bound by memory, and by how it is laid out: of a source tile with any token
// kept, V's every 64-byte line is read, whichever of its 16 tokens stay.  32 sequences of about 7100
// tokens and 8 kv heads of 128, of which 2048 stay (so that nearly every tile has one; 254
// MB read and written, 130 of them V's tiles), other ones in each call: 69 us, 3.7 TB/s.

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

int64_t kv_select_workspace(const if4_kv_mass& m, int64_t batch, int64_t kv_heads, int64_t keep) {
    const int64_t rows = batch * kv_heads, segment = segment_of(m, rows, keep);
    if (!segment) return 0;
    const int64_t segments = (m.width + segment - 1) / segment;
    return rows * (segments * (3 * kDigits * 4 + (int64_t)sizeof(State)) + keep * 4);
}

hipError_t launch_kv_select(const if4_kv_mass& m, const int32_t* seq_lens, int64_t batch,
                            int64_t kv_heads, int64_t keep, int64_t recent, int64_t sinks,
                            int32_t* kept, void* workspace, hipStream_t stream) {
    const SelectArgs s = {m, seq_lens, kept, (int)kv_heads, (int)keep, (int)recent, (int)sinks};
    const int64_t rows = batch * kv_heads, segment = segment_of(m, rows, keep);
    if (segment == 0) {
        if (!launchable(rows, kThreads)) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL(select_kernel, dim3((unsigned)rows), dim3(kThreads), 0, stream, s);
        return hipGetLastError();
    }
    const int64_t segments = (m.width + segment - 1) / segment;
    SegmentArgs p;
    p.s = s;
    p.rows = (int)rows;
    p.segment = (int)segment;
    p.segments = (int)segments;
    p.counts = reinterpret_cast<uint32_t*>(workspace);
    p.states = reinterpret_cast<State*>(p.counts + 3 * rows * segments * kDigits);
    p.moved = m.out == m.in ? reinterpret_cast<float*>(p.states + rows * segments) : nullptr;
    const dim3 grid((unsigned)(rows * segments));
    hipLaunchKernelGGL(segment_count_kernel<0>, grid, dim3(kThreads), 0, stream, p);
    hipLaunchKernelGGL(segment_count_kernel<1>, grid, dim3(kThreads), 0, stream, p);
    hipLaunchKernelGGL(segment_count_kernel<2>, grid, dim3(kThreads), 0, stream, p);
    hipLaunchKernelGGL(segment_write_kernel, grid, dim3(kThreads), 0, stream, p);
    if (p.moved) hipLaunchKernelGGL(segment_move_kernel, grid, dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_kv_compact(const if4_kv_cache& c, const int32_t* page_table,
                             int64_t table_stride, const int32_t* kept, int64_t batch,
                             int64_t keep, const int32_t* new_table, int64_t new_stride,
                             hipStream_t stream) {
    const int64_t tiles = (keep + 15) / 16, each = c.kv_heads * tiles;  // workgroups of a sequence
    if (!launchable(each, kCopyThreads)) return hipErrorInvalidConfiguration;
    const auto k = c.head_dim == 64 ? compact_kernel<64> : c.head_dim == 128 ? compact_kernel<128> : compact_kernel<256>;
    // as many sequences at once as a launch holds
    const int64_t most = most_groups(kCopyThreads) / each;
    for (int64_t b = 0; b < batch; b += most) {
        const CompactArgs p = {c, page_table + b * table_stride, kept + b * c.kv_heads * keep, new_table + b * new_stride,
                               table_stride, new_stride, keep, (int)tiles, Divisor(c.page_size / 16)};
        const dim3 grid((unsigned)((batch - b < most ? batch - b : most) * each));
        hipLaunchKernelGGL(k, grid, dim3(kCopyThreads), 0, stream, p);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace if4
