// ssd_channel.cuh -- device pieces shared by the channel scan's kernels.
//
// The scan: per channel d with N states (one decay per channel and state)
//   delta = softplus(dt + dt_bias),  h_n <- exp(delta A_n) h_n + delta x B_n,
//   y = sum_n h_n C_n + D x  (times silu(z)).
//
// A warp owns 32 channels of one group.  Lane l = cg * K + q holds, for the K
// channels cg * K .. cg * K + K - 1, the M = N / K states q * M ..: a tile of
// K x M states, so that one token's B and C (M values each) serve K channels
// and its delta and delta x (K values each) serve M states.  Four operations,
// one exponential and (M + K) / (K M) * 8 bytes of shared memory a state: with
// one channel a lane the shared-memory reads alone would take twice the time
// of the arithmetic.  Everything per channel (softplus, gates, D x, loads and
// stores) is done by lane l for channel l, whatever the alignment of rows;
// sums over the states of a channel are transposed on the way through the
// shuffles so that lane l ends with channel l.
#pragma once

#include "ssd_layer.cuh"

namespace ssd {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
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

// log(1 + exp(v)) = max(v, 0) + log1p(exp(-|v|)): no overflow, and accurate
// for v far below zero, where the result is exp(v).
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(__expf(-fabsf(v))); }

// Tile shape for N states.
template <int N>
struct Tile {
    static constexpr int K = N == 8 ? 2 : 4;  // channels a lane holds, and lanes a channel's states lie on
    static constexpr int M = N / K;           // states a lane holds of each
    static constexpr int M2 = M / 2;
    static constexpr int E4 = N / 4;  // float4s a lane holds (K * M == N)
};

// A sequence's stretch of a chunk: tokens [a, e) of sequence s = [S, E).
struct Span {
    int s, a, e, S, E;
};

// Sequence offsets on the device (packed batches), or equal lengths.
struct Seqs {
    const int *start;  // nullptr: equal lengths
    int n, L;
};

__device__ __forceinline__ int seq_of(const Seqs &q, int t) {  // start[s] <= t < start[s + 1]
    int lo = 0, hi = q.n;
    while (hi - lo > 1) {
        const int m = (lo + hi) / 2;
        (q.start[m] <= t ? lo : hi) = m;
    }
    while (q.start[lo + 1] <= t) ++lo;  // (empty sequences share an offset)
    return lo;
}

// Channel block: 32 channels (or what is left) of one group.
struct Block {
    int g, c0, nc;
};
__device__ __forceinline__ Block block_of(int blk, int per, int nblk_g) {
    const int g = blk / nblk_g, k = blk % nblk_g;
    return {g, g * per + 32 * k, min(32, per - 32 * k)};
}

// Lane-tile access of a [ch, N] fp32 array at channel c0: channels past nc
// read as zero and are not written.
template <int N>
__device__ __forceinline__ void load_tile(const float *p, int lane, int nc, f2 (&v)[Tile<N>::K][Tile<N>::M2]) {
    constexpr int K = Tile<N>::K, M = Tile<N>::M;
    const int cg = lane / K, q = lane % K;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int c = cg * K + i;
#pragma unroll
        for (int j = 0; j < M; j += 4) {
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < nc) r = *reinterpret_cast<const float4 *>(p + (int64_t)c * N + q * M + j);
            v[i][j / 2] = pack2(r.x, r.y);
            v[i][j / 2 + 1] = pack2(r.z, r.w);
        }
    }
}
template <int N>
__device__ __forceinline__ void store_tile(float *p, int lane, int nc, const f2 (&v)[Tile<N>::K][Tile<N>::M2]) {
    constexpr int K = Tile<N>::K, M = Tile<N>::M;
    const int cg = lane / K, q = lane % K;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int c = cg * K + i;
#pragma unroll
        for (int j = 0; j < M; j += 4) {
            float4 r;
            unpack2(v[i][j / 2], r.x, r.y);
            unpack2(v[i][j / 2 + 1], r.z, r.w);
            if (c < nc) *reinterpret_cast<float4 *>(p + (int64_t)c * N + q * M + j) = r;
        }
    }
}
// The same through a lane-interleaved scratch array [E4][32] of float4.
template <int N>
__device__ __forceinline__ void load_lanes(const float4 *p, int lane, f2 (&v)[Tile<N>::K][Tile<N>::M2]) {
    constexpr int M = Tile<N>::M;
#pragma unroll
    for (int f = 0; f < Tile<N>::E4; ++f) {
        const float4 r = p[f * 32 + lane];
        v[4 * f / M][4 * f % M / 2] = pack2(r.x, r.y);
        v[4 * f / M][4 * f % M / 2 + 1] = pack2(r.z, r.w);
    }
}
template <int N>
__device__ __forceinline__ void store_lanes(float4 *p, int lane, const f2 (&v)[Tile<N>::K][Tile<N>::M2]) {
    constexpr int M = Tile<N>::M;
#pragma unroll
    for (int f = 0; f < Tile<N>::E4; ++f) {
        float4 r;
        unpack2(v[4 * f / M][4 * f % M / 2], r.x, r.y);
        unpack2(v[4 * f / M][4 * f % M / 2 + 1], r.z, r.w);
        p[f * 32 + lane] = r;
    }
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

// Sums over lanes whose index differs in the bits below K, of R values for
// each of K channels: lane q of the K ends with the R sums of channel q.
template <int K, int R>
__device__ __forceinline__ void channel_sums(float (&v)[K][R], int lane, float (&out)[R]) {
    if constexpr (K == 4) {
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
