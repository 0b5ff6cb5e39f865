// Norm and rotation of queries and keys in one pass, and its gradients, for gfx950.
// The formulas are those of include/if4_qk.h.
//
// A vector of D values lies in L = D/8 lanes (rounded up to a power of two), 8 neighbours in
// each, so that a lane's 16 (or 32) bytes are one access.  The mean of the squares is three
// to five exchanges between lanes, in registers; pairs of two halves lie in two lanes, which
// trade their values, and neighbouring pairs in one.  Bound by memory: each value is read and
// written once; a wave keeps its token's cosines and sines while it goes through several
// heads.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "launch_limit.h"
#include "qk_internal.h"

namespace if4 {
namespace {

constexpr int kThreads = 256;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <bool kBf16>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
    if constexpr (kBf16) {
        const bf16x8 w = *reinterpret_cast<const bf16x8*>(reinterpret_cast<const uint16_t*>(p) + at);
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = (float)w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float4 w = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at)[i];
            v[4 * i] = w.x, v[4 * i + 1] = w.y, v[4 * i + 2] = w.z, v[4 * i + 3] = w.w;
        }
    }
}

// Keeps the compiler from making one store of the two kinds, which would be the ordinary.
__device__ __forceinline__ void apart() { asm volatile(""); }

// `past`: past the caches.
typedef float f32x4 __attribute__((ext_vector_type(4)));
template <bool kBf16>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&v)[8], bool past) {
    if constexpr (kBf16) {
        bf16x8 w;
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = (__bf16)v[i];
        bf16x8* const to = reinterpret_cast<bf16x8*>(reinterpret_cast<uint16_t*>(p) + at);
        if (past) {
            apart();
            __builtin_nontemporal_store(w, to);
            apart();
        } else {
            *to = w;
        }
    } else {
        f32x4* const to = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + at);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const f32x4 w = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
            if (past) {
                apart();
                __builtin_nontemporal_store(w, to + i);
                apart();
            } else {
                to[i] = w;
            }
        }
    }
}

// v of the lane that a DPP control names.
template <int kControl>
__device__ __forceinline__ float moved(float v) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), kControl, 0xF, 0xF, true));
}

// Sum over L neighbouring lanes, the same bits in all of them.
template <int L>
__device__ __forceinline__ float sum_lanes(float v) {
    v += moved<0xB1>(v);   // quad_perm 1,0,3,2
    v += moved<0x4E>(v);   // quad_perm 2,3,0,1
    v += moved<0x141>(v);  // half row mirrored
    if constexpr (L >= 16) v += moved<0x140>(v);  // row mirrored
    if constexpr (L >= 32) v += __shfl_xor(v, 16);
    return v;
}

// What lane i of a vector's holds: values 8 i .. 8 i + 7.  Of pairs of two halves (a, b)
// lanes below rotary / 16 hold the a's of pairs 8 i .., as many after them the b's; of
// neighbouring pairs lane i holds pairs 4 i ...
template <bool kInterleaved>
struct Place {
    int at;         // its first value
    int pair;       // its first pair
    bool in, turned;
    bool second;    // holds b's
    int partner;    // lane of the wave with the other members
    __device__ __forceinline__ Place(int lane, int i, int dim, int rotary) {
        at = 8 * i;
        in = at < dim;
        turned = at < rotary;
        const int half = rotary / 16;
        second = i >= half;
        pair = kInterleaved ? 4 * i : 8 * (second ? i - half : i);
        partner = turned ? lane + (second ? -half : half) : lane;
    }
};

// Cosines and sines of a lane's pairs.
template <bool kInterleaved>
struct Turn {
    static constexpr int kPairs = kInterleaved ? 4 : 8;
    float c[kPairs], s[kPairs];
    // (`sign` -1: the other way round.  Of pairs of two halves the b's sine is the other one.)
    __device__ __forceinline__ void load(const float* row, int rotary, const Place<kInterleaved>& at, float sign) {
#pragma unroll
        for (int i = 0; i < kPairs; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(row + at.pair + i);
            const float4 y = *reinterpret_cast<const float4*>(row + rotary / 2 + at.pair + i);
            c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
            s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
        }
        if (!kInterleaved && !at.second) sign = -sign;
#pragma unroll
        for (int i = 0; i < kPairs; i++) s[i] *= sign;
    }
    // (a, b) -> (a c - b s, a s + b c)
    __device__ __forceinline__ void operator()(float (&v)[8], const Place<kInterleaved>& at) const {
        if constexpr (kInterleaved) {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float a = v[2 * j], b = v[2 * j + 1];
                v[2 * j] = at.turned ? fmaf(a, c[j], -(b * s[j])) : a;
                v[2 * j + 1] = at.turned ? fmaf(a, s[j], b * c[j]) : b;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float other = __shfl(v[j], at.partner);  // (all lanes take part)
                v[j] = at.turned ? fmaf(v[j], c[j], other * s[j]) : v[j];
            }
        }
    }
};

struct Args {
    if4_qk_part part[2];
    const float* table;
    const int64_t* positions;
    int64_t tokens, table_rows;
    int dim, rotary, heads;  // heads: of both parts
    int per, chunks;         // vectors of a lane, and waves of a token
    float eps;
    int past;  // whether results go past the caches
};

// One lane's part of a vector: which kind it is, and its values.
struct Vector {
    int kind, head;
    bool there;
    __device__ __forceinline__ Vector(const Args& p, int h) {
        there = h < p.heads;
        kind = h < (int)p.part[0].heads ? 0 : 1;
        head = kind ? h - (int)p.part[0].heads : h;
    }
};

// The two weights' values of a lane.
struct Weights {
    float w[2][8] = {};
    __device__ __forceinline__ Weights(const Args& p, int at, bool in) {
#pragma unroll
        for (int kind = 0; kind < 2; kind++)
            if (p.part[kind].heads && in) load8<false>(p.part[kind].weight, at, w[kind]);
    }
    __device__ __forceinline__ float operator()(int kind, int j) const { return kind ? w[1][j] : w[0][j]; }
};

// A wave per token and chunk of its heads; its 64 / L lane groups take them in turn.  8192
// tokens of 72 vectors of 128 in bf16 (304 MB moved), other ones in each call: 72.7 us, 4.2
// TB/s, with up to 8 vectors to a lane and stores past the caches; up to 2, 3, 4, 12, 18: 81,
// 75, 77, 79, 93; ordinary stores 73.2; the next vector on its way while one is turned
// 77.  The same tensors in each call, which the caches hold in part: 52.5, up to 4 57, up to 18
// 59, ordinary stores 69.  64 tokens: 4.2 us, the time of a launch.
template <int L, bool kIn, bool kOut, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) forward_kernel(const Args p) {
    constexpr int G = 64 / L;
    const int lane = threadIdx.x & 63, i = lane % L;
    const int64_t wave = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
    const int64_t token = wave / p.chunks;
    if (token >= p.tokens) return;
    const int64_t pos = p.positions[token];
    if (pos < 0 || pos >= p.table_rows) return;
    const Place<kInterleaved> at(lane, i, p.dim, p.rotary);
    Turn<kInterleaved> turn = {};
    if (at.turned) turn.load(p.table + pos * p.rotary, p.rotary, at, 1.0f);
    const Weights w(p, at.at, at.in);
    const float inv = 1.0f / (float)p.dim;
    int h = (int)(wave - token * p.chunks) * p.per * G + lane / L;
    for (int n = 0; n < p.per; n++, h += G) {
        const Vector x(p, h);
        const if4_qk_part& part = p.part[x.kind];
        float v[8] = {};
        if (x.there && at.in) load8<kIn>(part.x, token * part.x_stride_token + x.head * part.x_stride_head + at.at, v);
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++) ss = fmaf(v[j], v[j], ss);
        const float r = rsqrtf(fmaf(sum_lanes<L>(ss), inv, p.eps));
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = v[j] * r * w(x.kind, j);
        turn(v, at);
        if (x.there && at.in)
            store8<kOut>(part.y, token * part.y_stride_token + x.head * part.y_stride_head + at.at, v, p.past);
    }
}

// dz = the rotation undone on g, r = 1 / sqrt(mean x^2 + eps):
//     dx = r (dz w - x r^2 mean(dz w x)),   dw = sum dz x r.
// Each lane keeps its sums of dw over all vectors that it sees; a workgroup joins them
// through LDS and writes one row of the workspace, and join_kernel adds the rows.  4099 tokens
// of 40 vectors of 128 in bf16 (126 MB): 28 us and 4.7 of the join, 3.9 TB/s.
template <int L, bool kIn, bool kOut, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) backward_kernel(const Args p, float* __restrict__ sums) {
    constexpr int G = 64 / L, kWaves = kThreads / 64;
    __shared__ float shared[kWaves * G][2][8 * L];
    const int lane = threadIdx.x & 63, i = lane % L;
    const Place<kInterleaved> at(lane, i, p.dim, p.rotary);
    const Weights w(p, at.at, at.in);
    float dw[2][8] = {};
    const float inv = 1.0f / (float)p.dim;
    const int64_t waves = (int64_t)gridDim.x * kWaves;
    for (int64_t unit = (int64_t)blockIdx.x * kWaves + threadIdx.x / 64; unit < p.tokens * p.chunks; unit += waves) {
        const int64_t token = unit / p.chunks;
        const int64_t pos = p.positions[token];
        const bool live = pos >= 0 && pos < p.table_rows;
        Turn<kInterleaved> back = {};
        if (live && at.turned) back.load(p.table + pos * p.rotary, p.rotary, at, -1.0f);
        int h = (int)(unit - token * p.chunks) * p.per * G + lane / L;
        for (int n = 0; n < p.per; n++, h += G) {
            const Vector v(p, h);
            const if4_qk_part& part = p.part[v.kind];
            const bool there = v.there && at.in;
            float x[8] = {}, g[8] = {};
            if (there && live) {
                load8<kIn>(part.x, token * part.x_stride_token + v.head * part.x_stride_head + at.at, x);
                load8<kOut>(part.g, token * part.g_stride_token + v.head * part.g_stride_head + at.at, g);
            }
            back(g, at);
            float ss = 0.0f, dot = 0.0f, gw[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                gw[j] = g[j] * w(v.kind, j);
                ss = fmaf(x[j], x[j], ss);
                dot = fmaf(gw[j], x[j], dot);
            }
            const float r = rsqrtf(fmaf(sum_lanes<L>(ss), inv, p.eps));
            const float mean = sum_lanes<L>(dot) * inv * r * r;
            float dx[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float d = there && live ? g[j] * x[j] * r : 0.0f;
                dw[0][j] += v.kind ? 0.0f : d;
                dw[1][j] += v.kind ? d : 0.0f;
                dx[j] = live ? r * fmaf(-x[j], mean, gw[j]) : 0.0f;
            }
            if (there) store8<kIn>(part.y, token * part.y_stride_token + v.head * part.y_stride_head + at.at, dx, p.past);
        }
    }
    const int row = threadIdx.x / L;
    if (at.in) {
#pragma unroll
        for (int kind = 0; kind < 2; kind++)
#pragma unroll
            for (int j = 0; j < 8; j++) shared[row][kind][at.at + j] = dw[kind][j];
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

// Vectors of a lane: as many as leave this many waves, for the chip to be full, and no more
// than kMostTurns; the backward pass has no more workgroups than kRows rows of sums.
constexpr int kFullWaves = 256 * 16, kMostTurns = 8;
// Results of more bytes than the caches of the chip's eight parts hold go past them.
constexpr int64_t kCaches = (int64_t)32 << 20;

Args make_args(const if4_qk_args& a, int lanes, int y_size) {
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
    p.per = each < 1 ? 1 : each > kMostTurns ? kMostTurns : (int)each;
    p.chunks = (turns + p.per - 1) / p.per;
    p.per = (turns + p.chunks - 1) / p.chunks;  // even shares
    p.eps = a.eps;
    p.past = a.tokens * p.heads * p.dim * y_size > kCaches;
    return p;
}

int lanes_of(int64_t dim) { return dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

template <int L, bool kIn, bool kOut, bool kInterleaved>
hipError_t forward(const if4_qk_args& a, hipStream_t stream) {
    const Args p = make_args(a, L, kOut ? 2 : 4);
    const int64_t groups = (a.tokens * p.chunks + kThreads / 64 - 1) / (kThreads / 64);
    if (!launchable(groups, kThreads)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((forward_kernel<L, kIn, kOut, kInterleaved>), dim3((unsigned)groups),
                       dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

int backward_rows(const if4_qk_args& a) {
    const Args p = make_args(a, lanes_of(a.head_dim), 4);
    const int64_t groups = (a.tokens * p.chunks + kThreads / 64 - 1) / (kThreads / 64);
    return (int)(groups < kRows ? groups : kRows);
}

template <int L, bool kIn, bool kOut, bool kInterleaved>
hipError_t backward(const if4_qk_args& a, float* sums, hipStream_t stream) {
    const int rows = backward_rows(a);
    if (rows) {
        hipLaunchKernelGGL((backward_kernel<L, kIn, kOut, kInterleaved>), dim3(rows), dim3(kThreads),
                           0, stream, make_args(a, L, kIn ? 2 : 4), sums);
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
