// ssd_channel_bwd.cu -- gradient of the channel scan.
//
// With g = dy silu(z), a_t = exp(delta_t A) and the gradient dh_t of the
// state after token t:
//   dh_t = g_t C_t + a_{t+1} dh_{t+1}
//   dC_t = sum_c g_t h_t,  dB_t = sum_c delta_t x_t dh_t
//   du_t = sum_n dh_t B_t,  w_t = dh_t a_t h_{t-1}
//   dx_t = delta_t du_t + D g_t,  ddelta_t = x_t du_t + sum_n w_t A,  dA = sum_t w_t delta_t
// Four launches over chunks of 28 tokens (32 with 8 states, 16 with 32):
//   1 chunk summaries: the state a chunk leaves from a zero start, the
//     gradient its outputs send back to the state before it, its sum of
//     deltas (exp(A sum delta) is its decay);
//   2 the two recurrences over chunks, in place: the state entering and the
//     gradient leaving every chunk;
//   3 per chunk: forward once, keeping every fourth state in shared memory;
//     then backward TB tokens at a time, whose states and decays are formed
//     again and stay in registers.  dB and dC are summed over the lanes of a
//     warp, then over the block's 128 channels; dA, dD and ddt_bias over the
//     chunks a block walks;
//   4 the sums over channel blocks and over blocks, in a fixed order.
// Bound by instruction issue.  At 4 x 2048 x 1536, 16 states, bf16 with gate
// a call takes 393 us, the launches each by itself with cold caches 93, 19, 280
// and 9: 162 and 459 instructions a token and warp in 1 and 3, 48 and 125 of
// them packed multiply-adds of two issue cycles each.  3 runs eight warps an SM (254 registers: the states and decays of four
// tokens are 128 of them) at 55 % issue; what its loads cost it was hidden by
// taking a chunk's values half a chunk at a time, all in flight (618 -> 272 us
// with a grid of one wave).
#include <type_traits>

#include "ssd_channel.h"

namespace ssd {
namespace {

constexpr int kWarps = 4;

template <int N>
struct Geo {
    // tokens per chunk: with 16 states what lets eight warps share an SM's memory
    static constexpr int CH = N == 32 ? 16 : N == 16 ? 28 : 32;
    static constexpr int TB = N == 32 ? 2 : 4;  // tokens whose states are in registers
    static constexpr int EV = 4;                // tokens between states kept in shared memory
    static constexpr int NK = EV == TB ? CH / EV - 1 : CH / EV;  // how many (the last TB's stays in registers)
};

template <typename T>
struct BwdArgs {
    ChannelArgs<T> f;  // the forward call's arguments
    Rows<const T> dy;
    Rows<T> dx, ddt, dz, dB, dC;
    const float *dfinal;
    float *dA, *dD, *dbias, *dinit;
    float4 *back;       // [unit][block][N / 4][32]: gradient for the state before (2: after) the chunk
    int *flags;         // [unit]: 1 a sequence starts in the chunk, 2 the one at its first token ends in it
    float *part_bc;     // [group][quad][token][2 N]
    float *part_a;      // [slot][block][N + 2][32]
    int quads, slots;   // quads of channel blocks per group; blocks that share a quad's chunks
    int64_t tokens;
};

// The square tile: 32 channels a warp, lane l the one channel l.
template <int N>
using BwdTile = std::conditional_t<N == 8, Tile<8, 2, 2>, Tile<N, 4, 4>>;

template <typename T, int N>
__device__ __forceinline__ void load_decay(const ChannelArgs<T> &a, const Block &k, int lane,
                                           typename BwdTile<N>::Regs &A2) {
    load_tile<BwdTile<N>>(a.A + (int64_t)k.c0 * N, lane, k.nc, A2);
#pragma unroll
    for (int i = 0; i < BwdTile<N>::K; ++i)
#pragma unroll
        for (int j = 0; j < BwdTile<N>::M2; ++j) A2[i][j] = mul2(A2[i][j], pack2(kLog2e, kLog2e));
}

// The channel's delta before and after softplus.
template <typename T>
__device__ __forceinline__ float delta_of(const ChannelArgs<T> &a, float pre) {
    return a.soft ? softplus(pre) : pre;
}

// ---------------------------------------------------------------------------
// 1: chunk summaries.  One forward walk: with P the decay from the chunk's
// start to t, the gradient for the state before the chunk is sum_t P g_t C_t.
// ---------------------------------------------------------------------------
// A lane is a channel, as in the forward kernel; the results are stored as the
// square tiles of 3 hold them.
template <int N>
__device__ __forceinline__ void store_square(float4 *p, int c, const f2 (&v)[1][N / 2]) {
    using G = BwdTile<N>;
    const int cg = c / G::K, i = c % G::K;
#pragma unroll
    for (int n = 0; n < N; n += 4) {
        float4 r;
        unpack2(v[0][n / 2], r.x, r.y);
        unpack2(v[0][n / 2 + 1], r.z, r.w);
        p[(i * G::M + n % G::M) / 4 * 32 + cg * G::K + n / G::M] = r;
    }
}

template <typename T, int N, bool GATE>
__global__ void __launch_bounds__(kWarps * 32, N == 32 ? 2 : 3) channel_bwd_chunk_kernel(const __grid_constant__ BwdArgs<T> b) {
    using G = Tile<N, 1, 1>;
    constexpr int N2 = N / 2, TB = 4, NB = TB * 2 * N / 32;
    __shared__ __align__(16) float stage[kWarps][TB][2 * N];
    const ChannelArgs<T> &a = b.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t id = (int64_t)blockIdx.x * kWarps + warp;
    launch_next();
    wait_previous();
    if (id >= (int64_t)a.units * a.nblk) return;
    const int blk = (int)(id % a.nblk), unit = (int)(id / a.nblk);
    auto &sm = stage[warp];
    const Block k = block_of(blk, a.per, a.nblk_g, 32);
    const bool mine = lane < k.nc;
    const int own = k.c0 + (mine ? lane : 0);
    const bool packed = a.seqs.packed;
    const int *start = a.seqs.offsets();
    const int row = packed ? 0 : unit / a.nchunk;
    const int t0 = (packed ? unit : unit % a.nchunk) * a.chunk, t1 = min(a.seqs.L, t0 + a.chunk);
    int s = row, S = 0, E = a.seqs.L;
    if (packed) {
        s = seq_of(start, a.seqs.n, t0);
        S = start[s], E = start[s + 1];
    }
    if (blk == 0 && lane == 0) {
        const bool starts = S == t0 || E < t1;  // (E < t1: another sequence starts at or after E, inside)
        b.flags[unit] = (starts ? 1 : 0) | (E <= t1 ? 2 : 0);
    }
    typename G::Regs A2, h, P, R;
    load_tile<G>(a.A + (int64_t)k.c0 * N, lane, k.nc, A2);
#pragma unroll
    for (int m = 0; m < N2; ++m) A2[0][m] = mul2(A2[0][m], pack2(kLog2e, kLog2e));
    const float bias = a.bias ? a.bias[own] : 0.f;
    const int64_t at = (int64_t)unit * a.nblk + blk;
    int t = t0;
    while (true) {
        const int e = min(t1, E);
        const bool head = t == t0 && S < t0;  // a gradient goes back to the chunk before
        const bool tail = E > t1;             // a state goes on to the chunk after
        if (head || tail) {
            zero_tile<G>(h), zero_tile<G>(R);
            if (t == S && a.init) load_tile<G>(a.init + ((int64_t)s * a.ch + k.c0) * N, lane, k.nc, h);
#pragma unroll
            for (int m = 0; m < N2; ++m) P[0][m] = pack2(1.f, 1.f);
            float total = 0.f;
            // (tokens past the piece read its last one, lanes without a channel the block's first: delta = g = 0)
            T rd[TB], rx[TB], rg[TB], rz[TB], rbc[NB];
            auto fetch = [&](int tb) {
#pragma unroll
                for (int j = 0; j < TB; ++j) {
                    const int tt = min(tb + j, e - 1);
                    rd[j] = a.dt.at(row, tt)[own];
                    rx[j] = a.x.at(row, tt)[own];
                    rg[j] = b.dy.at(row, tt)[own];
                    if (GATE) rz[j] = a.z.at(row, tt)[own];
                }
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int el = i * 32 + lane, tt = min(tb + el / (2 * N), e - 1), w = el % (2 * N);
                    rbc[i] = w < N ? a.B.at(row, tt)[k.g * N + w] : a.C.at(row, tt)[k.g * N + w - N];
                }
            };
            fetch(t);
            for (int tb = t; tb < e; tb += TB) {
                float d[TB], u[TB], g[TB];
#pragma unroll
                for (int j = 0; j < TB; ++j) {
                    d[j] = to_f32(rd[j]) + bias, u[j] = to_f32(rx[j]), g[j] = to_f32(rg[j]);
                    if (GATE) g[j] *= silu(to_f32(rz[j]));
                }
                if (a.soft) {
#pragma unroll
                    for (int j = 0; j < TB; ++j) d[j] = softplus(d[j]);
                }
#pragma unroll
                for (int j = 0; j < TB; ++j) {
                    const bool in = tb + j < e && mine;
                    d[j] = in ? d[j] : 0.f, u[j] = in ? d[j] * u[j] : 0.f, g[j] = in ? g[j] : 0.f;
                    total += d[j];
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int el = i * 32 + lane;
                    (&sm[0][0])[el] = tb + el / (2 * N) < e ? to_f32(rbc[i]) : 0.f;
                }
                __syncwarp();
                if (tb + TB < e) fetch(tb + TB);
#pragma unroll
                for (int j = 0; j < TB; ++j) {
                    const f2 dd = pack2(d[j], d[j]), uu = pack2(u[j], u[j]), gg = pack2(g[j], g[j]);
#pragma unroll
                    for (int m = 0; m < N2; m += 2) {
                        const ulonglong2 B = *reinterpret_cast<const ulonglong2 *>(&sm[j][2 * m]);
                        const ulonglong2 C = *reinterpret_cast<const ulonglong2 *>(&sm[j][N + 2 * m]);
                        const f2 d0 = ex2x2(mul2(A2[0][m], dd)), d1 = ex2x2(mul2(A2[0][m + 1], dd));
                        h[0][m] = fma2(d0, h[0][m], mul2(uu, B.x));
                        h[0][m + 1] = fma2(d1, h[0][m + 1], mul2(uu, B.y));
                        P[0][m] = mul2(P[0][m], d0);
                        P[0][m + 1] = mul2(P[0][m + 1], d1);
                        R[0][m] = fma2(P[0][m], mul2(gg, C.x), R[0][m]);
                        R[0][m + 1] = fma2(P[0][m + 1], mul2(gg, C.y), R[0][m + 1]);
                    }
                }
            }
            if (head) {
                if (e == E && b.dfinal) {
                    typename G::Regs f;
                    load_tile<G>(b.dfinal + ((int64_t)s * a.ch + k.c0) * N, lane, k.nc, f);
#pragma unroll
                    for (int m = 0; m < N2; ++m) R[0][m] = fma2(P[0][m], f[0][m], R[0][m]);
                }
                store_square<N>(b.back + at * (N / 4 * 32), lane, R);
            }
            if (tail) store_square<N>(a.local + at * (N / 4 * 32), lane, h);
            if (tail && head) a.sums[at * 32 + lane] = total;
        }
        if (e == t1) return;
        t = e;
        do ++s;
        while (start[s + 1] <= t);
        S = start[s], E = start[s + 1];
    }
}

// ---------------------------------------------------------------------------
// 2: the recurrences over chunks.  A block owns one float4 a lane of a channel
// block's states over all chunks of a sequence row; blockIdx.y picks the
// direction.  One warp walks them all where there are enough blocks (at 4 x
// 2048 x 1536 60 MB of both directions read in 19 us, what is written stays in
// L2).  The latency of the loads bounds it, and with few blocks RUNS warps take a run of
// chunks each: every warp combines its run from zero, then starts it again
// from the runs before (257 chunks of 640 channels: 37 -> 25 us).
// ---------------------------------------------------------------------------
template <typename T, int N, int RUNS>
__global__ void __launch_bounds__(RUNS * 32) channel_bwd_pass_kernel(const __grid_constant__ BwdArgs<T> b) {
    constexpr int K = BwdTile<N>::K, M = BwdTile<N>::M, AHEAD = RUNS == 1 ? 16 : 8;
    __shared__ float4 end[RUNS][32];
    __shared__ float sum[RUNS][32];
    __shared__ int reset[RUNS];
    const ChannelArgs<T> &a = b.f;
    launch_next();
    wait_previous();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, f = (int)(blockIdx.x % (N / 4));
    const int blk = (int)(blockIdx.x / (N / 4) % a.nblk), row = (int)(blockIdx.x / (N / 4) / a.nblk);
    const Block k = block_of(blk, a.per, a.nblk_g, 32);
    const int cg = lane / K, q = lane % K, c = cg * K + 4 * f / M;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < k.nc) A = *reinterpret_cast<const float4 *>(a.A + (int64_t)(k.c0 + c) * N + q * M + 4 * f % M);
    A.x *= kLog2e, A.y *= kLog2e, A.z *= kLog2e, A.w *= kLog2e;
    const bool fwd = blockIdx.y == 0;
    float4 *arr = fwd ? a.local : b.back;
    const int n = a.nchunk, u0 = row * n;
    const int per = (n + RUNS - 1) / RUNS, i_begin = min(n, warp * per), i_end = min(n, i_begin + per);
    float4 carry;
    // what leaves a chunk: its own value, and unless that is the whole of it the decayed rest
    auto combine = [&](bool whole, float sd, const float4 &v) {
        if (whole) {
            carry = v;
        } else {
            carry.x = fmaf(ex2(A.x * sd), carry.x, v.x);
            carry.y = fmaf(ex2(A.y * sd), carry.y, v.y);
            carry.z = fmaf(ex2(A.z * sd), carry.z, v.z);
            carry.w = fmaf(ex2(A.w * sd), carry.w, v.w);
        }
    };
    float4 v[AHEAD];
    float sd[AHEAD];
    int fl[AHEAD];
    auto load = [&](int i0) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (RUNS == 1 && i0 + j >= i_end) break;
            const int i = min(i0 + j, i_end - 1), u = u0 + (fwd ? i : n - 1 - i);
            const int64_t at = (int64_t)u * a.nblk + blk;
            v[j] = arr[at * (N / 4 * 32) + f * 32 + lane];
            sd[j] = a.sums[at * 32 + c];
            fl[j] = b.flags[u] & (fwd ? 1 : 2);
        }
    };
    carry = make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (RUNS > 1) {
        float total = 0.f;
        int whole = 0;
        for (int i0 = i_begin; i0 < i_end; i0 += AHEAD) {
            load(i0);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                if (i0 + j < i_end) {
                    combine(fl[j], sd[j], v[j]);
                    total += sd[j];
                    whole |= fl[j];
                }
            }
        }
        end[warp][lane] = carry, sum[warp][lane] = total;
        if (lane == 0) reset[warp] = whole;
        __syncthreads();
        carry = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < warp; ++w) combine(reset[w], sum[w][lane], end[w][lane]);
    }
    for (int i0 = i_begin; i0 < i_end; i0 += AHEAD) {
        load(i0);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (i0 + j < i_end) {
                const int u = u0 + (fwd ? i0 + j : n - 1 - i0 - j);
                arr[((int64_t)u * a.nblk + blk) * (N / 4 * 32) + f * 32 + lane] = carry;
                combine(fl[j], sd[j], v[j]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// 3: the gradients inside chunks
// ---------------------------------------------------------------------------
template <int N>
struct alignas(16) GradStage {
    float4 kept[Geo<N>::NK][N / 4 * 32];         // the state before every EV tokens
    float d[Geo<N>::CH][32], u[Geo<N>::CH][32], g[Geo<N>::CH][32];  // by token of the piece
    float bc[Geo<N>::CH + 1][2 * N];                                // by token of the chunk, turning into the warp's dB and dC; a zero row
};

// Sums over the lanes whose index differs in the bits from K up, of V values:
// halving the values while there are any to halve.  Lane l ends with the
// V / left values from `first` on.
template <int K, int V>
struct LaneSums {
    static constexpr int LANES = 32 / K, LEFT = V > LANES ? V / LANES : 1;
    static __device__ __forceinline__ int reduce(float (&v)[V], int lane) {
        int first = 0;
        int cnt = V;
#pragma unroll
        for (int bit = 16; bit >= K; bit >>= 1) {
            const bool up = lane & bit;
            if (cnt > 1) {
                cnt >>= 1;
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    if (i < cnt) {
                        const float s = up ? v[i] : v[i + cnt];
                        v[i] = (up ? v[i + cnt] : v[i]) + __shfl_xor_sync(0xffffffffu, s, bit);
                    }
                }
                if (up) first += cnt;
            } else {
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
            }
        }
        return first;
    }
};

template <typename T, int N, bool GATE>
__global__ void __launch_bounds__(kWarps * 32) channel_bwd_kernel(const __grid_constant__ BwdArgs<T> b) {
    constexpr int K = BwdTile<N>::K, M = BwdTile<N>::M, M2 = BwdTile<N>::M2, TB = Geo<N>::TB, CH = Geo<N>::CH;
    constexpr int EV = Geo<N>::EV;
    constexpr int R = GATE ? 3 : 2, LEFT = LaneSums<BwdTile<N>::K, 2 * BwdTile<N>::M>::LEFT;
    extern __shared__ __align__(16) char smem[];
    const ChannelArgs<T> &a = b.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    GradStage<N> *all = reinterpret_cast<GradStage<N> *>(smem);
    GradStage<N> &sm = all[warp];
    const int gq = blockIdx.x % (b.quads * (a.nblk / a.nblk_g)), slot = blockIdx.x / (b.quads * (a.nblk / a.nblk_g));
    const int grp = gq / b.quads, quad = gq % b.quads;
    const int in_g = quad * kWarps + warp;
    const bool live = in_g < a.nblk_g;  // a warp without channels only joins the barriers
    const int lives = min(kWarps, a.nblk_g - quad * kWarps);
    const int blk = grp * a.nblk_g + (live ? in_g : 0);
    Block k = block_of(blk, a.per, a.nblk_g, 32);
    if (!live) k.nc = 0;
    const int cg = lane / K, q = lane % K;
    const bool mine = lane < k.nc;
    const int own = k.c0 + (mine ? lane : 0);
    const bool packed = a.seqs.packed;
    const int *start = a.seqs.offsets();

    f2 A2[K][M2], dA[K][M2];
    load_decay<T, N>(a, k, lane, A2);
    zero_tile<BwdTile<N>>(dA);
    const float bias = a.bias ? a.bias[own] : 0.f;
    const float D = a.D && mine ? a.D[own] : 0.f;
    float dD = 0.f, dbias = 0.f;
    for (int i = lane; i < 2 * N; i += 32) sm.bc[CH][i] = 0.f;
    launch_next();
    wait_previous();

    for (int unit = slot; unit < a.units; unit += b.slots) {
        const int row = packed ? 0 : unit / a.nchunk;
        const int t0 = (packed ? unit : unit % a.nchunk) * CH, t1 = min(a.seqs.L, t0 + CH);
        const int64_t at = (int64_t)unit * a.nblk + blk;
        // the chunk's pieces of sequences, last one first
        int s = row, S = 0, E = a.seqs.L, e = t1;
        if (packed) {
            s = seq_of(start, a.seqs.n, t1 - 1);
            S = start[s], E = start[s + 1];
        }
        while (live) {
            const int begin = max(t0, S), off = begin - t0, ns = (e - begin + TB - 1) / TB;
            f2 h[K][M2], r[K][M2];
            if (begin == S) {
                zero_tile<BwdTile<N>>(h);
                if (a.init) load_tile<BwdTile<N>>(a.init + ((int64_t)s * a.ch + k.c0) * N, lane, k.nc, h);
            } else {
                load_lanes<BwdTile<N>>(a.local + at * (N / 4 * 32), lane, h);
            }
            if (e == E) {
                zero_tile<BwdTile<N>>(r);
                if (b.dfinal) load_tile<BwdTile<N>>(b.dfinal + ((int64_t)s * a.ch + k.c0) * N, lane, k.nc, r);
            } else {
                load_lanes<BwdTile<N>>(b.back + at * (N / 4 * 32), lane, r);
            }
            // forward, keeping the state before every TB tokens.  (Many loads at a
            // time; tokens past the piece read its last one, lanes without a
            // channel the block's first: delta = g = 0.)
            __syncwarp();
            constexpr int AT = CH / 2, AB = AT * 2 * N / 32;
            for (int j0 = 0; j0 < ns * TB; j0 += AT) {
                T rd[AT], rx[AT], rg[AT], rz[AT], rb[AB];
#pragma unroll
                for (int j = 0; j < AT; ++j) {
                    const int t = min(begin + j0 + j, e - 1);
                    rd[j] = a.dt.at(row, t)[own];
                    rx[j] = a.x.at(row, t)[own];
                    rg[j] = b.dy.at(row, t)[own];
                    if (GATE) rz[j] = a.z.at(row, t)[own];
                }
#pragma unroll
                for (int i = 0; i < AB; ++i) {
                    const int el = i * 32 + lane, t = min(begin + j0 + el / (2 * N), e - 1), w = el % (2 * N);
                    rb[i] = w < N ? a.B.at(row, t)[k.g * N + w] : a.C.at(row, t)[k.g * N + w - N];
                }
#pragma unroll
                for (int j = 0; j < AT; ++j) {
                    float d = delta_of(a, to_f32(rd[j]) + bias), u = d * to_f32(rx[j]), g = to_f32(rg[j]);
                    if (GATE) g *= silu(to_f32(rz[j]));
                    if (begin + j0 + j >= e || !mine) d = u = g = 0.f;
                    sm.d[j0 + j][lane] = d, sm.u[j0 + j][lane] = u, sm.g[j0 + j][lane] = g;
                }
#pragma unroll
                for (int i = 0; i < AB; ++i) {
                    const int el = i * 32 + lane, j = j0 + el / (2 * N);
                    if (begin + j < e) sm.bc[off + j][el % (2 * N)] = to_f32(rb[i]);
                }
            }
            __syncwarp();
            auto advance = [&](int sb) {  // the state over TB tokens of the piece
#pragma unroll
                for (int jj = 0; jj < TB; ++jj) {
                    const int j = sb * TB + jj;
                    float d[K], u[K];
                    f2 B[M2];
                    load_k<K>(&sm.d[j][cg * K], d);
                    load_k<K>(&sm.u[j][cg * K], u);
                    load_m<M>(&sm.bc[off + j][q * M], B);
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        const f2 dd = pack2(d[i], d[i]), uu = pack2(u[i], u[i]);
#pragma unroll
                        for (int m = 0; m < M2; ++m)
                            h[i][m] = fma2(ex2x2(mul2(A2[i][m], dd)), h[i][m], mul2(uu, B[m]));
                    }
                }
            };
            for (int sb = 0; sb < ns; ++sb) {
                if (sb * TB % EV == 0 && (EV != TB || sb + 1 < ns)) store_lanes<BwdTile<N>>(sm.kept[sb * TB / EV], lane, h);
                if (sb + 1 < ns) advance(sb);
            }
            // backward
            for (int sb = ns - 1; sb >= 0; --sb) {
                const int left = e - begin - sb * TB;  // tokens of these TB that are the piece's
                // this channel's values, in flight until the outputs
                T rx[TB], rg[TB], rz[TB], rd[TB];
#pragma unroll
                for (int jj = 0; jj < TB; ++jj) {
                    const int t = min(begin + sb * TB + jj, e - 1);
                    rx[jj] = a.x.at(row, t)[own];
                    rg[jj] = b.dy.at(row, t)[own];
                    rd[jj] = a.dt.at(row, t)[own];
                    if (GATE) rz[jj] = a.z.at(row, t)[own];
                }
                if (sb + 1 < ns) load_lanes<BwdTile<N>>(sm.kept[sb * TB / EV], lane, h);
                if (EV != TB && sb + 1 < ns) {
                    for (int s2 = sb * TB / EV * EV / TB; s2 < sb; ++s2) advance(s2);
                }
                f2 before[TB][K][M2], decay[TB][K][M2];
#pragma unroll
                for (int jj = 0; jj < TB; ++jj) {
                    const int j = sb * TB + jj;
                    float d[K], u[K];
                    f2 B[M2];
                    load_k<K>(&sm.d[j][cg * K], d);
                    load_k<K>(&sm.u[j][cg * K], u);
                    // (tokens past the piece: delta = g = 0 and the zero row)
                    load_m<M>(&sm.bc[begin + j < e ? off + j : CH][q * M], B);
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        const f2 dd = pack2(d[i], d[i]), uu = pack2(u[i], u[i]);
#pragma unroll
                        for (int m = 0; m < M2; ++m) {
                            before[jj][i][m] = h[i][m];
                            decay[jj][i][m] = ex2x2(mul2(A2[i][m], dd));
                            h[i][m] = fma2(decay[jj][i][m], h[i][m], mul2(uu, B[m]));
                        }
                    }
                }
                float o[TB][R], dbc[TB][LEFT];
                int first = 0;
#pragma unroll
                for (int jj = TB - 1; jj >= 0; --jj) {
                    const int j = sb * TB + jj, t = begin + j;
                    float d[K], u[K], g[K];
                    f2 B[M2], C[M2], dBp[M2], dCp[M2];
                    load_k<K>(&sm.d[j][cg * K], d);
                    load_k<K>(&sm.u[j][cg * K], u);
                    load_k<K>(&sm.g[j][cg * K], g);
                    const int at_bc = t < e ? off + j : CH;
                    load_m<M>(&sm.bc[at_bc][q * M], B);
                    load_m<M>(&sm.bc[at_bc][N + q * M], C);
#pragma unroll
                    for (int m = 0; m < M2; ++m) dBp[m] = 0, dCp[m] = 0;
                    float sums[K][R];
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        const f2 dd = pack2(d[i], d[i]), uu = pack2(u[i], u[i]), gg = pack2(g[i], g[i]);
                        f2 du = 0, dd_A = 0, yy = 0;
#pragma unroll
                        for (int m = 0; m < M2; ++m) {
                            const f2 after = jj + 1 < TB ? before[jj + 1 < TB ? jj + 1 : 0][i][m] : h[i][m];
                            const f2 dh = fma2(gg, C[m], r[i][m]);
                            if (GATE) yy = fma2(after, C[m], yy);
                            dCp[m] = fma2(gg, after, dCp[m]);
                            dBp[m] = fma2(uu, dh, dBp[m]);
                            du = fma2(dh, B[m], du);
                            r[i][m] = mul2(decay[jj][i][m], dh);
                            const f2 w = mul2(r[i][m], before[jj][i][m]);
                            dd_A = fma2(w, A2[i][m], dd_A);
                            // (past the piece w may be 0 times an infinity)
                            dA[i][m] = jj == 0 ? fma2(w, dd, dA[i][m]) : fma2_if(jj < left, w, dd, dA[i][m]);
                        }
                        sums[i][0] = sum2(du);
                        sums[i][1] = sum2(dd_A);
                        if (GATE) sums[i][R - 1] = sum2(yy);
                    }
                    group_sums<K, R>(sums, lane, o[jj]);
                    float v[2 * M];
#pragma unroll
                    for (int m = 0; m < M2; ++m) {
                        unpack2(dBp[m], v[2 * m], v[2 * m + 1]);
                        unpack2(dCp[m], v[M + 2 * m], v[M + 2 * m + 1]);
                    }
                    first = LaneSums<K, 2 * M>::reduce(v, lane);
#pragma unroll
                    for (int i = 0; i < LEFT; ++i) dbc[jj][i] = v[i];
                }
                // (outputs only here: a branch inside the loop would keep its tokens from overlapping)
                __syncwarp();
#pragma unroll
                for (int jj = 0; jj < TB; ++jj) {
                    if (jj < left) {
#pragma unroll
                        for (int i = 0; i < LEFT; ++i) {
                            const int w = first + i;  // < M: dB, else dC, of state q M + w % M
                            sm.bc[off + sb * TB + jj][(w < M ? 0 : N) + q * M + w % M] = dbc[jj][i];
                        }
                    }
                }
                if (mine) {
#pragma unroll
                    for (int jj = 0; jj < TB; ++jj) {
                        if (jj >= left) break;
                        const int t = begin + sb * TB + jj;
                        const float delta = sm.d[sb * TB + jj][lane], gx = sm.g[sb * TB + jj][lane], x = to_f32(rx[jj]);
                        float ddl = x * o[jj][0] + kLn2 * o[jj][1];
                        if (a.soft) ddl *= sigmoid(to_f32(rd[jj]) + bias);
                        b.dx.at(row, t)[own] = from_f32<T>(fmaf(delta, o[jj][0], D * gx));
                        b.ddt.at(row, t)[own] = from_f32<T>(ddl);
                        dD = fmaf(gx, x, dD);
                        dbias += ddl;
                        if (GATE) {
                            const float y = fmaf(D, x, o[jj][R - 1]), z = to_f32(rz[jj]);
                            b.dz.at(row, t)[own] = from_f32<T>(to_f32(rg[jj]) * y * silu_slope(z, sigmoid(z)));
                        }
                    }
                }
            }
            if (begin == S && b.dinit) store_tile<BwdTile<N>>(b.dinit + ((int64_t)s * a.ch + k.c0) * N, lane, k.nc, r);
            if (begin == t0) break;
            e = begin;
            do --s;
            while (start[s] == start[s + 1]);
            S = start[s], E = start[s + 1];
        }
        // add the block's warps
        __syncthreads();
        float4 *dst = reinterpret_cast<float4 *>(b.part_bc + ((int64_t)gq * b.tokens + (int64_t)row * a.seqs.L + t0) * (2 * N));
        for (int el = threadIdx.x; el < (t1 - t0) * (2 * N / 4); el += kWarps * 32) {
            float4 v = reinterpret_cast<const float4 *>(all[0].bc)[el];
            for (int w = 1; w < lives; ++w) {
                const float4 o = reinterpret_cast<const float4 *>(all[w].bc)[el];
                v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
            }
            dst[el] = v;
        }
        __syncthreads();
    }
    if (live) {
        float *dst = b.part_a + ((int64_t)slot * a.nblk + blk) * ((N + 2) * 32);
        store_lanes<BwdTile<N>>(reinterpret_cast<float4 *>(dst), lane, dA);
        dst[N * 32 + lane] = dD;
        dst[(N + 1) * 32 + lane] = dbias;
    }
}

// ---------------------------------------------------------------------------
// 4: sums over channel blocks (dB, dC) and over slots (dA, dD, ddt_bias)
// ---------------------------------------------------------------------------
template <typename T, int N>
__global__ void __launch_bounds__(256) channel_bwd_reduce_kernel(const __grid_constant__ BwdArgs<T> b, int64_t bc_blocks,
                                                                 unsigned blocks) {
    constexpr int K = BwdTile<N>::K, M = BwdTile<N>::M;
    const ChannelArgs<T> &a = b.f;
    wait_previous();
    if (blockIdx.x >= blocks) {
        pass_empty_states(a.seqs.offsets(), a.seqs.n, (int64_t)a.ch * N, b.dfinal, b.dinit, blockIdx.x - blocks,
                          gridDim.x - blocks);
        return;
    }
    if (blockIdx.x < bc_blocks) {
        const int groups = a.nblk / a.nblk_g;
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
        if (i >= b.tokens * groups * 2 * N) return;
        const int w = (int)(i % (2 * N)), g = (int)(i / (2 * N) % groups);
        const int64_t token = i / (2 * N) / groups;
        const float *src = b.part_bc + ((int64_t)g * b.quads * b.tokens + token) * (2 * N) + w;
        float s = 0.f;
        for (int q = 0; q < b.quads; ++q) s += src[(int64_t)q * b.tokens * (2 * N)];
        const int row = (int)(token / a.seqs.L), t = (int)(token % a.seqs.L);
        if (w < N)
            b.dB.at(row, t)[g * N + w] = from_f32<T>(s);
        else
            b.dC.at(row, t)[g * N + w - N] = from_f32<T>(s);
        return;
    }
    constexpr int each = (N + 2) * 32;
    const int64_t i = ((int64_t)blockIdx.x - bc_blocks) * 256 + threadIdx.x;
    if (i >= (int64_t)a.nblk * each) return;
    const int blk = (int)(i / each), idx = (int)(i % each);
    float s = 0.f;
    for (int q = 0; q < b.slots; ++q) s += b.part_a[((int64_t)q * a.nblk + blk) * each + idx];
    const Block k = block_of(blk, a.per, a.nblk_g, 32);
    if (idx >= N * 32) {
        const int lane = idx % 32;
        float *dst = idx < (N + 1) * 32 ? b.dD : b.dbias;
        if (dst && lane < k.nc) dst[k.c0 + lane] = s;
        return;
    }
    const int lane = idx / 4 % 32, el = idx / 128 * 4 + idx % 4;
    const int c = lane / K * K + el / M, n = lane % K * M + el % M;
    if (b.dA && c < k.nc) b.dA[(int64_t)(k.c0 + c) * N + n] = s;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int N>
struct BwdPlan {
    int nchunk, quads, slots;
    int64_t units, nblk;
    size_t offsets, flags, local, back, sums, part_bc, part_a, bytes;

    BwdPlan(const ssd_channel_shape_t *s, const int64_t *cu, int64_t nseq) {
        const int64_t nblk_g = (s->channels / s->ngroups + 31) / 32;
        nblk = s->ngroups * nblk_g;
        quads = (int)((nblk_g + kWarps - 1) / kWarps);
        nchunk = (int)((s->seqlen + Geo<N>::CH - 1) / Geo<N>::CH);
        units = (cu ? 1 : s->batch) * nchunk;
        // at most one wave of the blocks that fit two to an SM
        int64_t want = 152 * 2 / (s->ngroups * quads);
        if (want < 1) want = 1;
        slots = (int)(units < want ? units : want);
        size_t at = 0;
        auto take = [&at](size_t n) {
            const size_t r = at;
            at += align256(n);
            return r;
        };
        offsets = take(offsets_bytes(cu, nseq));
        flags = take(sizeof(int) * units);
        local = take(sizeof(float) * units * nblk * N * 32);
        back = take(sizeof(float) * units * nblk * N * 32);
        sums = take(sizeof(float) * units * nblk * 32);
        part_bc = take(sizeof(float) * s->ngroups * quads * s->batch * s->seqlen * 2 * N);
        part_a = take(sizeof(float) * slots * nblk * (N + 2) * 32);
        bytes = at;
    }
};

template <typename T, int N>
ssd_status_t run_bwd(BwdArgs<T> &b, const ssd_channel_shape_t *s, const int64_t *cu, int64_t nseq, char *ws,
                     size_t ws_bytes, cudaStream_t st) {
    const BwdPlan<N> p(s, cu, nseq);
    if (p.bytes > 0 && (!ws || ws_bytes < p.bytes || !aligned(ws, 16))) return SSD_ERR_WORKSPACE;
    ChannelArgs<T> &a = b.f;
    timing_begin(st);
    cudaError_t e = cudaSuccess;
    bool after = false;
    if (s->seqlen == 0 && b.dinit && nseq > 0)
        e = copy_states(b.dfinal, b.dinit, nseq * s->channels * s->dstate, st);
    else if (cu)
        e = place_offsets(cu, nseq, reinterpret_cast<int *>(ws + p.offsets), a.seqs, &after, st);
    if (e != cudaSuccess) return status_of(e);
    a.chunk = Geo<N>::CH, a.nchunk = p.nchunk, a.units = (int)p.units;
    a.local = reinterpret_cast<float4 *>(ws + p.local);
    a.sums = reinterpret_cast<float *>(ws + p.sums);
    b.back = reinterpret_cast<float4 *>(ws + p.back);
    b.flags = reinterpret_cast<int *>(ws + p.flags);
    b.part_bc = reinterpret_cast<float *>(ws + p.part_bc);
    b.part_a = reinterpret_cast<float *>(ws + p.part_a);
    b.quads = p.quads, b.slots = p.slots;
    b.tokens = s->batch * s->seqlen;
    if (p.units > 0) {
        const int64_t warps = (p.units * p.nblk + kWarps - 1) / kWarps;
        const int64_t passes = (int64_t)(cu ? 1 : s->batch) * p.nblk * (N / 4);
        const int64_t grads = (int64_t)s->ngroups * p.quads * p.slots;
        if (warps > 0x7FFFFFFF || passes > 0x7FFFFFFF || grads > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
        if (p.nchunk > 1) {
            e = launch(a.z.p ? channel_bwd_chunk_kernel<T, N, true> : channel_bwd_chunk_kernel<T, N, false>,
                       dim3((unsigned)warps), kWarps * 32, 0, st, after, b);
            timing_mark(st, "channel_bwd_chunk");
            if (e == cudaSuccess)
                e = passes < 304 ? launch(channel_bwd_pass_kernel<T, N, 8>, dim3((unsigned)passes, 2), 256, 0, st, true, b)
                                 : launch(channel_bwd_pass_kernel<T, N, 1>, dim3((unsigned)passes, 2), 32, 0, st, true, b);
            timing_mark(st, "channel_bwd_pass");
            if (e != cudaSuccess) return status_of(e);
            after = true;
        }
        const size_t smem = sizeof(GradStage<N>) * kWarps;
        auto kernel = a.z.p ? channel_bwd_kernel<T, N, true> : channel_bwd_kernel<T, N, false>;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) e = launch(kernel, dim3((unsigned)grads), kWarps * 32, smem, st, after, b);
        timing_mark(st, "channel_bwd");
        if (e != cudaSuccess) return status_of(e);
    }
    const int64_t bc = (b.tokens * s->ngroups * 2 * N + 255) / 256, ab = (p.nblk * (N + 2) * 32 + 255) / 256;
    if (bc + ab > 0x7FFFF000) return SSD_ERR_UNSUPPORTED;
    const unsigned blocks = (unsigned)(bc + ab), empty = cu && b.dinit && s->seqlen > 0 ? empty_blocks(cu, nseq) : 0;
    e = launch(channel_bwd_reduce_kernel<T, N>, dim3(blocks + empty), 256, 0, st, p.units > 0, b, bc, blocks);
    timing_mark(st, "channel_bwd_reduce");
    return status_of(e);
}

template <typename T>
ssd_status_t bwd_typed(const ssd_channel_shape_t *s, const int64_t *cu, int64_t nseq, const ssd_rows_t *dy,
                       const ssd_channel_inputs_t *in, const float *dfinal, const ssd_channel_grads_t *out, void *ws,
                       size_t ws_bytes, cudaStream_t st) {
    BwdArgs<T> b{};
    b.f = channel_args<T>(s, in, nseq);
    b.dy = rows_of<const T>(*dy);
    b.dx = rows_of<T>(out->dx), b.ddt = rows_of<T>(out->ddt), b.dz = rows_of<T>(out->dz);
    b.dB = rows_of<T>(out->dB), b.dC = rows_of<T>(out->dC);
    b.dfinal = dfinal;
    b.dA = out->dA, b.dD = out->dD, b.dbias = out->ddt_bias, b.dinit = out->dinit_state;
    char *w = static_cast<char *>(ws);
    if (s->dstate == 8) return run_bwd<T, 8>(b, s, cu, nseq, w, ws_bytes, st);
    if (s->dstate == 16) return run_bwd<T, 16>(b, s, cu, nseq, w, ws_bytes, st);
    return run_bwd<T, 32>(b, s, cu, nseq, w, ws_bytes, st);
}

}  // namespace
}  // namespace ssd

extern "C" {

size_t ssd_channel_scan_bwd_workspace_size(const ssd_channel_shape_t *shape, const int64_t *cu_seqlens, int64_t nseq) {
    using namespace ssd;
    if (check_channel(shape, cu_seqlens, nseq) != SSD_OK) return 0;
    if (shape->dstate == 8) return BwdPlan<8>(shape, cu_seqlens, nseq).bytes;
    if (shape->dstate == 16) return BwdPlan<16>(shape, cu_seqlens, nseq).bytes;
    return BwdPlan<32>(shape, cu_seqlens, nseq).bytes;
}

ssd_status_t ssd_channel_scan_bwd(const ssd_channel_shape_t *shape, const int64_t *cu_seqlens, int64_t nseq,
                                  const ssd_rows_t *dy, const ssd_channel_inputs_t *in, const float *dfinal_state,
                                  const ssd_channel_grads_t *out, void *workspace, size_t workspace_bytes,
                                  cudaStream_t stream) {
    using namespace ssd;
    const ssd_status_t st = check_channel(shape, cu_seqlens, nseq);
    if (st != SSD_OK) return st;
    if (!cu_seqlens) nseq = shape->batch;
    const bool rows = shape->seqlen > 0 && nseq > 0;
    if (!channel_inputs_ok(shape, in, rows) || !dy || !out || !aligned(dfinal_state, 16) || !aligned(out->dA, 4) ||
        !aligned(out->dD, 4) || !aligned(out->ddt_bias, 4) || !aligned(out->dinit_state, 16))
        return SSD_ERR_INVALID_ARG;
    if (rows) {
        const size_t es = dtype_size(shape->dtype);
        const int64_t b = shape->batch, L = shape->seqlen, gn = shape->ngroups * shape->dstate;
        if (!rows_in_ok(*dy, es) || !rows_out_ok(out->dx, es, b, L, shape->channels) ||
            !rows_out_ok(out->ddt, es, b, L, shape->channels) || !rows_out_ok(out->dB, es, b, L, gn) ||
            !rows_out_ok(out->dC, es, b, L, gn))
            return SSD_ERR_INVALID_ARG;
        if (in->z.data && !rows_out_ok(out->dz, es, b, L, shape->channels)) return SSD_ERR_INVALID_ARG;
    }
    return shape->dtype == SSD_DTYPE_BF16
               ? bwd_typed<bf16>(shape, cu_seqlens, nseq, dy, in, dfinal_state, out, workspace, workspace_bytes, stream)
               : bwd_typed<float>(shape, cu_seqlens, nseq, dy, in, dfinal_state, out, workspace, workspace_bytes, stream);
}

}  // extern "C"
