// Norm and rotation of queries and keys in one pass, and its gradients, for gfx950.
// The formulas are those of include/if4_qk.h.
//
// A vector of D values lies in L = D/8 lanes (rounded up to a power of two), 8 values in
// each: two runs of 4, chosen so that both members of a rotated pair are in one lane.
// The mean of the squares is then three to five exchanges between lanes, and the rotation
// none.  Bound by memory: each value is read and written once; a wave keeps its token's
// cosines and sines while it goes through several heads.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "qk_internal.h"

namespace if4 {
namespace {

constexpr int kThreads = 256;

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

template <bool kBf16>
__device__ __forceinline__ void load4(const void* p, int64_t at, float* v) {
    if constexpr (kBf16) {
        const bf16x4 w = *reinterpret_cast<const bf16x4*>(reinterpret_cast<const uint16_t*>(p) + at);
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = (float)w[i];
    } else {
        const float4 w = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at);
        v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    }
}

template <bool kBf16>
__device__ __forceinline__ void store4(void* p, int64_t at, const float* v) {
    if constexpr (kBf16) {
        bf16x4 w;
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = (__bf16)v[i];
        *reinterpret_cast<bf16x4*>(reinterpret_cast<uint16_t*>(p) + at) = w;
    } else {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at) = make_float4(v[0], v[1], v[2], v[3]);
    }
}

// Sum over L neighbouring lanes, the same bits in all of them.
template <int L>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
    for (int d = 1; d < L; d *= 2) v += __shfl_xor(v, d);
    return v;
}

// What a lane holds of every vector: values at[0] .. + 3 and at[1] .. + 3, which are pairs
// 4 i .. 4 i + 3 where i < rotary / 8.
struct Place {
    int at[2];
    bool in, turned;
    __device__ __forceinline__ Place(int i, int dim, int rotary, bool interleaved) {
        in = 8 * i < dim;
        turned = 8 * i < rotary;
        at[0] = turned && !interleaved ? 4 * i : 8 * i;
        at[1] = turned && !interleaved ? rotary / 2 + 4 * i : 8 * i + 4;
    }
};

// (a, b) -> (a c - b s, a s + b c) for the lane's four pairs.
template <bool kInterleaved>
__device__ __forceinline__ void turn(float (&v)[8], const float (&c)[4], const float (&s)[4]) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int x = kInterleaved ? 2 * j : j, y = kInterleaved ? 2 * j + 1 : 4 + j;
        const float a = v[x], b = v[y];
        v[x] = fmaf(a, c[j], -(b * s[j]));
        v[y] = fmaf(a, s[j], b * c[j]);
    }
}

struct Args {
    if4_qk_part part[2];
    const float* table;
    const int64_t* positions;
    int64_t tokens, table_rows;
    int dim, rotary, heads;  // heads: of both parts
    int per, chunks;         // vectors of a lane, and waves of a token
    float eps;
};

// Cosines and sines of a token for this lane; false: the token is skipped.
__device__ __forceinline__ bool load_turn(const Args& p, int64_t token, int i, const Place& at,
                                          float (&c)[4], float (&s)[4]) {
    const int64_t pos = p.positions[token];
    if (pos < 0 || pos >= p.table_rows) return false;
    if (at.turned) {
        load4<false>(p.table, pos * p.rotary + 4 * i, c);
        load4<false>(p.table, pos * p.rotary + p.rotary / 2 + 4 * i, s);
    }
    return true;
}

// A wave per token and chunk of its heads; its 64 / L lane groups take them in turn.
template <int L, bool kIn, bool kOut, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) forward_kernel(const Args p) {
    constexpr int G = 64 / L;
    const int lane = threadIdx.x & 63, i = lane % L;
    const int64_t wave = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
    const int64_t token = wave / p.chunks;
    if (token >= p.tokens) return;
    const Place at(i, p.dim, p.rotary, kInterleaved);
    float c[4], s[4];
    if (!load_turn(p, token, i, at, c, s)) return;
    int h = (int)(wave - token * p.chunks) * p.per * G + lane / L;
    const float inv = 1.0f / (float)p.dim;
    for (int n = 0; n < p.per; n++, h += G) {
        const bool there = h < p.heads && at.in;
        const int kind = h < p.part[0].heads ? 0 : 1;
        const if4_qk_part& part = p.part[kind];
        const int head = kind ? h - (int)p.part[0].heads : h;
        float v[8] = {}, w[8] = {};
        if (there) {
            const int64_t x = token * part.x_stride_token + head * part.x_stride_head;
            load4<kIn>(part.x, x + at.at[0], v);
            load4<kIn>(part.x, x + at.at[1], v + 4);
            load4<false>(part.weight, at.at[0], w);
            load4<false>(part.weight, at.at[1], w + 4);
        }
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++) ss = fmaf(v[j], v[j], ss);
        const float r = rsqrtf(fmaf(sum_lanes<L>(ss), inv, p.eps));
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = v[j] * r * w[j];
        if (at.turned) turn<kInterleaved>(v, c, s);
        if (there) {
            const int64_t y = token * part.y_stride_token + head * part.y_stride_head;
            store4<kOut>(part.y, y + at.at[0], v);
            store4<kOut>(part.y, y + at.at[1], v + 4);
        }
    }
}

// dz = the rotation undone on g, r = 1 / sqrt(mean x^2 + eps):
//     dx = r (dz w - x r^2 mean(dz w x)),   dw = sum dz x r.
// Each lane keeps its sums of dw over all vectors that it sees; a workgroup joins them
// through LDS and writes one row of the workspace, and join_kernel adds the rows.
template <int L, bool kIn, bool kOut, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) backward_kernel(const Args p, float* __restrict__ sums) {
    constexpr int G = 64 / L, kWaves = kThreads / 64;
    __shared__ float shared[kWaves * G][2][8 * L];
    const int lane = threadIdx.x & 63, i = lane % L;
    const Place at(i, p.dim, p.rotary, kInterleaved);
    float w[2][8] = {}, dw[2][8] = {};
#pragma unroll
    for (int kind = 0; kind < 2; kind++)
        if (p.part[kind].heads && at.in) {
            load4<false>(p.part[kind].weight, at.at[0], w[kind]);
            load4<false>(p.part[kind].weight, at.at[1], w[kind] + 4);
        }
    const float inv = 1.0f / (float)p.dim;
    const int64_t waves = (int64_t)gridDim.x * kWaves;
    for (int64_t unit = (int64_t)blockIdx.x * kWaves + threadIdx.x / 64; unit < p.tokens * p.chunks; unit += waves) {
        const int64_t token = unit / p.chunks;
        float c[4] = {}, s[4] = {};
        const bool live = load_turn(p, token, i, at, c, s);
        int h = (int)(unit - token * p.chunks) * p.per * G + lane / L;
        for (int n = 0; n < p.per; n++, h += G) {
            const bool there = h < p.heads && at.in;
            const int kind = h < p.part[0].heads ? 0 : 1;
            const if4_qk_part& part = p.part[kind];
            const int head = kind ? h - (int)p.part[0].heads : h;
            float x[8] = {}, g[8] = {};
            if (there && live) {
                const int64_t xo = token * part.x_stride_token + head * part.x_stride_head;
                const int64_t go = token * part.g_stride_token + head * part.g_stride_head;
                load4<kIn>(part.x, xo + at.at[0], x);
                load4<kIn>(part.x, xo + at.at[1], x + 4);
                load4<kOut>(part.g, go + at.at[0], g);
                load4<kOut>(part.g, go + at.at[1], g + 4);
            }
            if (at.turned) {
                const float back[4] = {-s[0], -s[1], -s[2], -s[3]};
                turn<kInterleaved>(g, c, back);
            }
            float ss = 0.0f, dot = 0.0f;
            float gw[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                gw[j] = g[j] * (kind ? w[1][j] : w[0][j]);
                ss = fmaf(x[j], x[j], ss);
                dot = fmaf(gw[j], x[j], dot);
            }
            const float r = rsqrtf(fmaf(sum_lanes<L>(ss), inv, p.eps));
            const float mean = sum_lanes<L>(dot) * inv * r * r;
            float dx[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float d = there && live ? g[j] * x[j] * r : 0.0f;
                dw[0][j] += kind ? 0.0f : d;
                dw[1][j] += kind ? d : 0.0f;
                dx[j] = live ? r * fmaf(-x[j], mean, gw[j]) : 0.0f;
            }
            if (there) {
                const int64_t y = token * part.y_stride_token + head * part.y_stride_head;
                store4<kIn>(part.y, y + at.at[0], dx);
                store4<kIn>(part.y, y + at.at[1], dx + 4);
            }
        }
    }
    const int row = threadIdx.x / L;
    if (at.in) {
#pragma unroll
        for (int kind = 0; kind < 2; kind++)
#pragma unroll
            for (int j = 0; j < 8; j++) shared[row][kind][at.at[j / 4] + j % 4] = dw[kind][j];
    }
    __syncthreads();
    for (int d = threadIdx.x; d < 2 * p.dim; d += kThreads) {
        const int kind = d >= p.dim, e = kind ? d - p.dim : d;
        float t = 0.0f;
        for (int q = 0; q < kWaves * G; q++) t += shared[q][kind][e];
        sums[(int64_t)blockIdx.x * 2 * p.dim + d] = t;
    }
}

// Adds `rows` rows (kRows at most) of 2 dim sums: 16 columns per workgroup, 64 threads each,
// so that a thread's few loads are on their way at once (16 threads of 64 loads each: 20 us).
constexpr int kRows = 1024;
constexpr int kJoinThreads = 1024, kJoinParts = kJoinThreads / 16;
__global__ void __launch_bounds__(kJoinThreads)
join_kernel(const float* __restrict__ sums, int rows, int dim, float* dq, float* dk) {
    __shared__ float shared[kJoinParts][17];
    const int c = threadIdx.x % 16, col = blockIdx.x * 16 + c, part = threadIdx.x / 16;
    float v[kRows / kJoinParts], t = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows / kJoinParts; i++) {
        const int r = part + i * kJoinParts;
        v[i] = r < rows ? sums[(int64_t)r * 2 * dim + col] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kRows / kJoinParts; i++) t += v[i];
    shared[part][c] = t;
    __syncthreads();
    if (part == 0) {
        for (int q = 1; q < kJoinParts; q++) t += shared[q][c];
        float* const to = col < dim ? dq : dk;
        if (to) to[col < dim ? col : col - dim] = t;
    }
}

// Vectors of a lane: as many as leave this many waves, for the chip to be full; the
// backward pass has no more workgroups than kRows rows of sums.
constexpr int kFullWaves = 256 * 16;

Args make_args(const if4_qk_args& a, int lanes) {
    Args p;
    p.part[0] = a.q;
    p.part[1] = a.k;
    p.table = a.table;
    p.positions = a.positions;
    p.tokens = a.tokens;
    p.table_rows = a.table_rows;
    p.dim = (int)a.head_dim;
    p.rotary = (int)a.rotary;
    p.heads = (int)(a.q.heads + a.k.heads);
    const int groups = 64 / lanes, turns = (p.heads + groups - 1) / groups;
    const int64_t each = a.tokens * turns / kFullWaves;
    p.per = each < 1 ? 1 : each > turns ? turns : (int)each;
    p.chunks = (turns + p.per - 1) / p.per;
    p.per = (turns + p.chunks - 1) / p.chunks;  // even shares
    p.eps = a.eps;
    return p;
}

int lanes_of(int64_t dim) { return dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

template <int L, bool kIn, bool kOut, bool kInterleaved>
hipError_t forward(const if4_qk_args& a, hipStream_t stream) {
    const Args p = make_args(a, L);
    const int64_t groups = (a.tokens * p.chunks + kThreads / 64 - 1) / (kThreads / 64);
    hipLaunchKernelGGL((forward_kernel<L, kIn, kOut, kInterleaved>), dim3((unsigned)groups),
                       dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

int backward_rows(const if4_qk_args& a) {
    const Args p = make_args(a, lanes_of(a.head_dim));
    const int64_t groups = (a.tokens * p.chunks + kThreads / 64 - 1) / (kThreads / 64);
    return (int)(groups < kRows ? groups : kRows);
}

template <int L, bool kIn, bool kOut, bool kInterleaved>
hipError_t backward(const if4_qk_args& a, float* sums, hipStream_t stream) {
    const int rows = backward_rows(a);
    if (rows) {
        hipLaunchKernelGGL((backward_kernel<L, kIn, kOut, kInterleaved>), dim3(rows), dim3(kThreads),
                           0, stream, make_args(a, L), sums);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)(2 * a.head_dim / 16)), dim3(kJoinThreads), 0, stream,
                       sums, rows, (int)a.head_dim, a.q.heads ? a.q.d_weight : nullptr,
                       a.k.heads ? a.k.d_weight : nullptr);
    return hipGetLastError();
}

template <class F>
hipError_t by_types(const if4_qk_args& a, F f) {
    const bool in = a.dtype == IF4_BF16, out = a.out_dtype == IF4_BF16, il = a.interleaved != 0;
    using T = std::true_type;
    using N = std::false_type;
    if (il)
        return in ? out ? f(T{}, T{}, T{}) : f(T{}, N{}, T{}) : out ? f(N{}, T{}, T{}) : f(N{}, N{}, T{});
    return in ? out ? f(T{}, T{}, N{}) : f(T{}, N{}, N{}) : out ? f(N{}, T{}, N{}) : f(N{}, N{}, N{});
}

template <int L>
hipError_t forward_of(const if4_qk_args& a, hipStream_t stream) {
    return by_types(a, [&](auto in, auto out, auto il) {
        return forward<L, decltype(in)::value, decltype(out)::value, decltype(il)::value>(a, stream);
    });
}

template <int L>
hipError_t backward_of(const if4_qk_args& a, float* sums, hipStream_t stream) {
    return by_types(a, [&](auto in, auto out, auto il) {
        return backward<L, decltype(in)::value, decltype(out)::value, decltype(il)::value>(a, sums, stream);
    });
}

}  // namespace

int64_t norm_rotate_backward_workspace(const if4_qk_args& a) {
    return (int64_t)kRows * 2 * a.head_dim * 4;
}

hipError_t launch_norm_rotate(const if4_qk_args& a, hipStream_t stream) {
    const int lanes = lanes_of(a.head_dim);
    return lanes == 8 ? forward_of<8>(a, stream) : lanes == 16 ? forward_of<16>(a, stream) : forward_of<32>(a, stream);
}

hipError_t launch_norm_rotate_backward(const if4_qk_args& a, void* workspace, hipStream_t stream) {
    const int lanes = lanes_of(a.head_dim);
    float* const sums = reinterpret_cast<float*>(workspace);
    return lanes == 8    ? backward_of<8>(a, sums, stream)
           : lanes == 16 ? backward_of<16>(a, sums, stream)
                         : backward_of<32>(a, sums, stream);
}

}  // namespace if4
