// ssd_channel.cuh -- device pieces shared by the channel scan's kernels.
//
// The scan: per channel d with N states (one decay per channel and state)
//   delta = softplus(dt + dt_bias),  h_n <- exp(delta A_n) h_n + delta x B_n,
//   y = sum_n h_n C_n + D x  (times silu(z)).
//
// A warp owns 32 channels of one group, in one of two arrangements:
//   one channel a lane (Tile<N, 1, 1>): a lane has its channel's N states and
//     its delta in registers and sums over states by itself; B and C are read
//     from shared memory as broadcasts, N / 2 reads of 16 bytes a token;
//   square (Tile<N, Q, Q>): lane l = cg * Q + q has the M = N / Q states q * M ..
//     of the Q channels cg * Q ..: a third of the reads, an eighth of the
//     lanes to sum dB and dC over, but sums over a channel's states go through
//     shuffles, transposed on the way so that lane l ends with channel l.
// The forward kernel and the chunk summaries take the first, the gradient
// inside chunks the second.  Either way what is per channel and token
// (softplus, gates, D x, loads and stores, whatever the alignment of rows) is
// done by lane l for channel l.
#pragma once

#include "ssd_layer.cuh"

namespace ssd {

// Two fp32 values in one register pair.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// p ? fma2(a, b, c) : c, as a predicated instruction rather than two selects
__device__ __forceinline__ f2 fma2_if(bool p, f2 a, f2 b, f2 c) {
    asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t@p fma.rn.f32x2 %0, %1, %2, %0;\n\t}"
        : "+l"(c)
        : "l"(a), "l"(b), "r"((unsigned)p));
    return c;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 ex2x2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return pack2(ex2(a), ex2(b));
}
__device__ __forceinline__ float sum2(f2 v) {
    float a, b;
    unpack2(v, a, b);
    return a + b;
}

// log(1 + exp(v)) = max(v, 0) + log(1 + e), e = exp(-|v|): no overflow, and no
// cancellation for v far below zero, where the result is e.  With s = e / (2 + e),
// log(1 + e) = 2 atanh(s) = s q(s^2); q is the polynomial of degree 4 of least
// relative error (4e-9, by the exchange algorithm) on s^2 in [0, 1/9].  In
// fp32 the rounded product in e adds 7e-8 |v| to the 3e-7 of the rest: 6e-7
// relative at -8.7, a few 1e-6 at -80.  (Adding the product's rounding error
// back gives 3.5e-7 there and leaves the scan's outputs as far from exact as
// they are, for 829 instead of 805 us at 8 x 4096 x 5120.)
__device__ __forceinline__ float softplus(float v) {
    const float e = ex2(-kLog2e * fabsf(v));
    const float s = e * rcp(2.f + e), w = s * s;
    float q = fmaf(0.28178334f, w, 0.27960601f);
    q = fmaf(q, w, 0.40024909f);
    q = fmaf(q, w, 0.66666317f);
    q = fmaf(q, w, 2.f);
    return fmaf(s, q, fmaxf(v, 0.f));
}

// Tile shape for N states: K channels on Q lanes.
template <int N_, int Q_, int K_>
struct Tile {
    static constexpr int N = N_, Q = Q_, K = K_;
    static constexpr int M = N / Q, M2 = M / 2;  // states a lane holds of each channel
    static constexpr int E4 = K * M / 4;         // float4s a lane holds
    using Regs = f2[K][M2];
};

// The sequences: equal lengths, or packed offsets, which travel in the launch's
// parameters when they are few and otherwise lie in the workspace.
constexpr int kInline = 96;
struct Seqs {
    const int *start;  // nullptr: in `few` (packed) or none
    int n, L, packed;
    int few[kInline];
    // (of a __grid_constant__ parameter)
    __device__ __forceinline__ const int *offsets() const { return start ? start : few; }
};

__device__ __forceinline__ int seq_of(const int *start, int n, int t) {  // start[s] <= t < start[s + 1]
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int m = (lo + hi) / 2;
        (start[m] <= t ? lo : hi) = m;
    }
    while (start[lo + 1] <= t) ++lo;  // (empty sequences share an offset)
    return lo;
}

// Empty sequences hand a state on unchanged: dst[s] = src[s] (zero without
// src) for every s with start[s] == start[s + 1]; `each` floats, a multiple
// of four.  Run by the last `blocks` blocks of a launch, several a sequence.
__device__ inline void pass_empty_states(const int *start, int n, int64_t each, const float *src, float *dst, int block,
                                         int blocks) {
    const int parts = blocks > n ? blocks / n : 1, part = block / n;
    if (part >= parts) return;
    for (int s = block % n; s < n; s += blocks) {
        if (start[s] != start[s + 1]) continue;
        const float4 *from = reinterpret_cast<const float4 *>(src + s * each);
        float4 *to = reinterpret_cast<float4 *>(dst + s * each);
        for (int64_t i = (int64_t)part * blockDim.x + threadIdx.x; i < each / 4; i += (int64_t)parts * blockDim.x)
            to[i] = src ? from[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

// Channel block: cw channels (or what is left) of one group.
struct Block {
    int g, c0, nc;
};
__device__ __forceinline__ Block block_of(int blk, int per, int nblk_g, int cw) {
    const int g = blk / nblk_g, k = blk % nblk_g;
    return {g, g * per + cw * k, min(cw, per - cw * k)};
}

// Lane-tile access of a [ch, N] fp32 array at channel c0: channels past nc
// read as zero and are not written.
template <typename G>
__device__ __forceinline__ void load_tile(const float *p, int lane, int nc, typename G::Regs &v) {
    const int cg = lane / G::Q, q = lane % G::Q;
#pragma unroll
    for (int i = 0; i < G::K; ++i) {
        const int c = cg * G::K + i;
#pragma unroll
        for (int j = 0; j < G::M; j += 4) {
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < nc) r = *reinterpret_cast<const float4 *>(p + (int64_t)c * G::N + q * G::M + j);
            v[i][j / 2] = pack2(r.x, r.y);
            v[i][j / 2 + 1] = pack2(r.z, r.w);
        }
    }
}
template <typename G>
__device__ __forceinline__ void store_tile(float *p, int lane, int nc, const typename G::Regs &v) {
    const int cg = lane / G::Q, q = lane % G::Q;
#pragma unroll
    for (int i = 0; i < G::K; ++i) {
        const int c = cg * G::K + i;
#pragma unroll
        for (int j = 0; j < G::M; j += 4) {
            float4 r;
            unpack2(v[i][j / 2], r.x, r.y);
            unpack2(v[i][j / 2 + 1], r.z, r.w);
            if (c < nc) *reinterpret_cast<float4 *>(p + (int64_t)c * G::N + q * G::M + j) = r;
        }
    }
}
// The same through a lane-interleaved scratch array [E4][32] of float4.
template <typename G>
__device__ __forceinline__ void load_lanes(const float4 *p, int lane, typename G::Regs &v) {
#pragma unroll
    for (int f = 0; f < G::E4; ++f) {
        const float4 r = p[f * 32 + lane];
        v[4 * f / G::M][4 * f % G::M / 2] = pack2(r.x, r.y);
        v[4 * f / G::M][4 * f % G::M / 2 + 1] = pack2(r.z, r.w);
    }
}
template <typename G>
__device__ __forceinline__ void store_lanes(float4 *p, int lane, const typename G::Regs &v) {
#pragma unroll
    for (int f = 0; f < G::E4; ++f) {
        float4 r;
        unpack2(v[4 * f / G::M][4 * f % G::M / 2], r.x, r.y);
        unpack2(v[4 * f / G::M][4 * f % G::M / 2 + 1], r.z, r.w);
        p[f * 32 + lane] = r;
    }
}
template <typename G>
__device__ __forceinline__ void zero_tile(typename G::Regs &v) {
#pragma unroll
    for (int i = 0; i < G::K; ++i)
#pragma unroll
        for (int j = 0; j < G::M2; ++j) v[i][j] = 0;
}

// K consecutive floats of shared (or global) memory.
template <int K>
__device__ __forceinline__ void load_k(const float *p, float (&v)[K]) {
    if constexpr (K == 2) {
        const float2 r = *reinterpret_cast<const float2 *>(p);
        v[0] = r.x, v[1] = r.y;
    } else {
        const float4 r = *reinterpret_cast<const float4 *>(p);
        v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
    }
}
// M consecutive floats as pairs.
template <int M>
__device__ __forceinline__ void load_m(const float *p, f2 (&v)[M / 2]) {
#pragma unroll
    for (int j = 0; j < M; j += 4) {
        const ulonglong2 r = *reinterpret_cast<const ulonglong2 *>(p + j);
        v[j / 2] = r.x, v[j / 2 + 1] = r.y;
    }
}

// Sums over the Q lanes of a group, R of each of Q values: lane q ends with
// the R sums of value q.
template <int Q, int R>
__device__ __forceinline__ void group_sums(float (&v)[Q][R], int lane, float (&out)[R]) {
    if constexpr (Q == 4) {
        const bool up = lane & 2;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float s0 = up ? v[0][r] : v[2][r], s1 = up ? v[1][r] : v[3][r];
            v[0][r] = (up ? v[2][r] : v[0][r]) + __shfl_xor_sync(0xffffffffu, s0, 2);
            v[1][r] = (up ? v[3][r] : v[1][r]) + __shfl_xor_sync(0xffffffffu, s1, 2);
        }
    }
    const bool up = lane & 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float s = up ? v[0][r] : v[1][r];
        out[r] = (up ? v[1][r] : v[0][r]) + __shfl_xor_sync(0xffffffffu, s, 1);
    }
}

}  // namespace ssd
