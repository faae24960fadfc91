// ssd_conv.cu -- the short causal convolution before a scan: forward over
// prompts, gradient, and one token at a time.
//
//   p[t, c] = bias[c] + sum_k weight[c, k] x[t - (W-1) + k, c],  y = silu(p)
//
// W + 5 operations an element against 2 (forward) or 3 (gradient) element
// transfers: bound by memory, with instruction issue not far behind in bf16.
// A thread owns four channels and walks down the tokens with the last W-1 rows
// in registers, so each row is read once (and W-1 rows more per tile); a warp
// reads 256 (bf16) or 512 consecutive bytes of a row, and the next four rows
// are in flight while four are computed.  (Eight channels a thread halve the
// address arithmetic but leave 16 warps an SM instead of 24: 259 against 244
// us at 65536 x 5376.)  Channels are independent, so y is written straight into the x, B and C
// arrays a scan takes, out of the projection's rows in place.
// bf16, W 4: 65537 packed tokens x 5376 channels in 246 us, 5.7 TB/s; the
// gradient at 4 x 4095 x 2560 in 59 us with the sums, 4.2 TB/s.  fp32 spills
// registers: 8 x 2048 x 5120 in 126 us, 5.3 TB/s; the gradient at 4 x 4095 x
// 2560 in 138 us, 3.6 TB/s.
//
// Tokens are cut into tiles without regard to sequences: a tile walks its
// pieces of sequences one after another and rebuilds the window (from the
// sequence's initial rows where it begins), so ragged batches stay balanced.
#include <type_traits>

#include "ssd_layer.cuh"

namespace ssd {
namespace {

constexpr int kVec = 4;       // channels per thread (8 bytes of bf16, 16 of fp32)
constexpr int kLanes = 32;    // channel vectors per block
constexpr int kSub = 8;       // tiles of tokens per block, one per warp
constexpr int kAhead = 4;     // rows in flight, forward
constexpr int kStep = 4;      // and in the gradient (of x and of dy)
constexpr int kMaxSet = 960;  // sequences whose offsets fit one launch's parameters

// Offsets of the packed sequences first .. first + n - 1.
struct SeqSet {
    int n, first;
    int start[kMaxSet + 1];
};
struct NoSet {};

template <typename T>
struct ConvArgs {
    Rows<const T> x;
    Rows<T> y[SSD_CONV_MAX_PARTS];  // forward: outputs; gradient: dy (read only)
    int part_end[SSD_CONV_MAX_PARTS];
    Rows<T> dx;
    const float *weight, *bias;
    const T *init;    // [nseq, W-1, C]
    const T *dfinal;  // gradient: [nseq, W-1, C]
    T *final_state;   // forward: [nseq, W-1, C]; gradient: dinit
    float *partial;   // gradient: [slots, W+1, C]
    int C, nvec, ncb;  // channels, channel vectors, blocks of vectors
    int L, nseq;       // equal lengths
    int tile, ntiles;  // tokens per tile, tiles
    int64_t tblocks;   // blocks that walk tiles (the rest copy states)
    int use_silu;
};

// One sequence's stretch of a tile: tokens [a, e) of sequence s = [S, E).
struct Piece {
    int s, a, e, S, E;
};

// Calls f(piece, batch row) for each stretch of the tile.
template <bool PACKED, typename Set, typename F>
__device__ __forceinline__ void for_pieces(int64_t tile, int tile_len, int L, const Set &set, F f) {
    if constexpr (!PACKED) {
        const int tps = (L + tile_len - 1) / tile_len;
        const int s = (int)(tile / tps), a = (int)(tile % tps) * tile_len;
        f(Piece{s, a, min(L, a + tile_len), 0, L}, s);
    } else {
        int t = set.start[0] + (int)(tile * tile_len);
        const int end = min(set.start[set.n], t + tile_len);
        int lo = 0, hi = set.n;  // start[lo] <= t < start[hi]
        while (hi - lo > 1) {
            const int m = (lo + hi) / 2;
            (set.start[m] <= t ? lo : hi) = m;
        }
        while (t < end) {
            while (set.start[lo + 1] <= t) ++lo;  // past empty sequences
            const int E = set.start[lo + 1], e = min(end, E);
            f(Piece{set.first + lo, t, e, set.start[lo], E}, 0);
            t = e;
        }
    }
}

template <typename T>
__device__ __forceinline__ Rows<T> part_of(const ConvArgs<T> &a, int c0) {
    Rows<T> r = a.y[0];
    int begin = 0;
#pragma unroll
    for (int i = 1; i < SSD_CONV_MAX_PARTS; ++i)
        if (c0 >= a.part_end[i - 1]) r = a.y[i], begin = a.part_end[i - 1];
    r.p += c0 - begin;
    return r;
}

// The row that precedes or belongs to a sequence: x, or its initial rows.
template <typename T, int W, int V>
__device__ __forceinline__ Vec<T, V> row_at(const ConvArgs<T> &a, const Rows<const T> &x, const Piece &p, int row, int t,
                                            int c0) {
    if (t >= p.S) return load_vec<T, V>(x.at(row, t));
    if (!a.init) return zero_vec<T, V>();
    return load_vec<T, V>(a.init + ((int64_t)p.s * (W - 1) + (t - p.S + W - 1)) * a.C + c0);
}

template <typename T, int W, int V>
__device__ __forceinline__ void load_weights(const ConvArgs<T> &a, int c0, float (&w)[W][V], float (&b)[V]) {
    const float *src = a.weight + (int64_t)c0 * W;  // V W floats: 16-byte aligned where V is 4 or 8
    float f[W * V];
    if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < W * V / 4; ++i) widen<float, 4>(load_vec<float, 4>(src + 4 * i), f + 4 * i);
    } else {
#pragma unroll
        for (int i = 0; i < W * V; ++i) f[i] = src[i];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][v] = f[v * W + k];
        b[v] = a.bias ? a.bias[c0 + v] : 0.f;
    }
}

// p = bias + sum_k w[k] (window, then cur): the window moves up by one.
template <int W, int V>
__device__ __forceinline__ void taps(const float (&w)[W][V], const float (&bias)[V], float (&win)[W - 1][V],
                                     const float (&cur)[V], float (&p)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float s = bias[v];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) s = fmaf(w[k][v], win[k][v], s);
        p[v] = fmaf(w[W - 1][v], cur[v], s);
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) win[k][v] = win[k + 1][v];
        win[W - 2][v] = cur[v];
    }
}

// The states that sequences leave behind, copied bit by bit: row j is token
// E - (W-1) + j, or an initial row where the sequence is shorter than that.
// In the gradient (GRAD) only empty sequences are copied here.
template <typename T, int W, int V, bool PACKED, bool GRAD, typename Set>
__device__ void copy_states(const ConvArgs<T> &a, const Set &set, int64_t block) {
    int n = a.nseq;
    if constexpr (PACKED) n = set.n;
    const int64_t items = (int64_t)n * (W - 1) * a.nvec;
    const int64_t i = block * (kLanes * kSub) + threadIdx.y * kLanes + threadIdx.x;
    if (i >= items) return;
    const int c0 = (int)(i % a.nvec) * V;
    const int j = (int)(i / a.nvec % (W - 1)), q = (int)(i / a.nvec / (W - 1));
    Piece p{q, 0, 0, 0, a.L};
    int row = q;
    if constexpr (PACKED) p = Piece{set.first + q, 0, 0, set.start[q], set.start[q + 1]}, row = 0;
    T *dst = a.final_state + ((int64_t)p.s * (W - 1) + j) * a.C + c0;
    if constexpr (GRAD) {
        if (p.E > p.S) return;
        const Vec<T, V> v =
            a.dfinal ? load_vec<T, V>(a.dfinal + ((int64_t)p.s * (W - 1) + j) * a.C + c0) : zero_vec<T, V>();
        store_vec<T, V>(dst, v);
    } else {
        Rows<const T> x = a.x;
        x.p += c0;
        store_vec<T, V>(dst, row_at<T, W, V>(a, x, p, row, p.E - (W - 1) + j, c0));
    }
}

template <typename T, int W, int V, bool PACKED, bool SILU, typename Set>
__global__ void __launch_bounds__(kLanes *kSub, 3) conv_fwd_kernel(const __grid_constant__ ConvArgs<T> a,
                                                                const __grid_constant__ Set set) {
    if (blockIdx.x >= a.tblocks) {
        copy_states<T, W, V, PACKED, false>(a, set, blockIdx.x - a.tblocks);
        return;
    }
    const int vec = (int)(blockIdx.x % a.ncb) * kLanes + threadIdx.x;
    const int64_t tile = blockIdx.x / a.ncb * kSub + threadIdx.y;
    if (vec >= a.nvec || tile >= a.ntiles) return;
    const int c0 = vec * V;
    float w[W][V], bias[V];
    load_weights<T, W, V>(a, c0, w, bias);
    Rows<const T> x = a.x;
    x.p += c0;
    const Rows<T> y = part_of<T>(a, c0);
    for_pieces<PACKED>(tile, a.tile, a.L, set, [&](const Piece &p, int row) {
        Vec<T, V> nxt[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) nxt[i] = zero_vec<T, V>();
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (p.a + i < p.e) nxt[i] = load_vec<T, V>(x.at(row, p.a + i));
        float win[W - 1][V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const Vec<T, V> v = row_at<T, W, V>(a, x, p, row, p.a - (W - 1) + j, c0);
            widen<T, V>(v, win[j]);
        }
#pragma unroll 2  // (two steps swap the rows in flight and those computed without copies)
        for (int t = p.a; t < p.e; t += kAhead) {
            const int n = p.e - t;
            float o[kAhead][V];
            Vec<T, V> cur[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) cur[i] = nxt[i];
            if (n >= 2 * kAhead) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) nxt[i] = load_vec<T, V>(x.at(row, t + kAhead + i));
            } else {
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    if (kAhead + i < n) nxt[i] = load_vec<T, V>(x.at(row, t + kAhead + i));
            }
            // (rows past the end are computed from what was loaded last and not stored)
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                float c[V];
                widen<T, V>(cur[i], c);
                taps<W, V>(w, bias, win, c, o[i]);
            }
            if constexpr (SILU) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
#pragma unroll
                    for (int v = 0; v < V; ++v) o[i][v] = silu(o[i][v]);
            }
            if (n >= kAhead) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) store_vec<T, V>(y.at(row, t + i), narrow<T, V>(o[i]));
            } else {
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    if (i < n) store_vec<T, V>(y.at(row, t + i), narrow<T, V>(o[i]));
            }
        }
    });
}

// Gradient.  Walking down the tokens, step t forms
//   dp[t] = dy[t] silu'(p[t]),  dweight[k] += dp[t] x[t - (W-1) + k],
// and with the last W dp at hand the row W-1 before it is complete:
//   dx[t - (W-1)] = sum_k weight[k] dp[t - k].
// A tile walks W-1 tokens past its end (only for dp), and a sequence's first
// W-1 steps complete the rows before it, its initial state's gradient.  The
// sums over tokens stay in fp32 registers over all tiles of a block, are
// added over the block's warps, and the blocks' partial sums by a second
// kernel in a fixed order.
template <typename T, int W, int V, bool PACKED, bool SILU, typename Set>
__global__ void __launch_bounds__(kLanes *kSub, 2) conv_bwd_kernel(const __grid_constant__ ConvArgs<T> a,
                                                                const __grid_constant__ Set set, int slots, int slot0) {
    if (blockIdx.x >= a.tblocks) {
        copy_states<T, W, V, PACKED, true>(a, set, blockIdx.x - a.tblocks);
        return;
    }
    const int vec = (int)(blockIdx.x % a.ncb) * kLanes + threadIdx.x;
    const int slot = (int)(blockIdx.x / a.ncb);
    const int c0 = vec * V;
    float dw[W][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][v] = 0.f;
    }
    if (vec < a.nvec) {
        float w[W][V], bias[V];
        load_weights<T, W, V>(a, c0, w, bias);
        Rows<const T> x = a.x;
        x.p += c0;
        const Rows<T> dy = part_of<T>(a, c0);
        Rows<T> dx = a.dx;
        dx.p += c0;
        for (int64_t tile = (int64_t)slot * kSub + threadIdx.y; tile < a.ntiles; tile += (int64_t)slots * kSub) {
            for_pieces<PACKED>(tile, a.tile, a.L, set, [&](const Piece &p, int row) {
                // a sequence's first rows complete the rows before it
                const bool back = p.a == p.S && a.final_state;
                const int tail = a.dfinal ? p.E - (W - 1) : p.E;  // rows from here on add the final state's gradient
                float win[W - 1][V], dpw[W - 1][V];
                Vec<T, V> nx[kStep], ng[kStep];
                auto fetch = [&](int t) {
                    // (rows past the sequence read its last one; their dp is set to zero)
#pragma unroll
                    for (int i = 0; i < kStep; ++i) {
                        const int tt = min(t + i, p.E - 1);
                        nx[i] = load_vec<T, V>(x.at(row, tt));
                        ng[i] = load_vec<T, V>(dy.at(row, tt));
                    }
                };
                fetch(p.a);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    const Vec<T, V> v = row_at<T, W, V>(a, x, p, row, p.a - (W - 1) + j, c0);
                    widen<T, V>(v, win[j]);
#pragma unroll
                    for (int v2 = 0; v2 < V; ++v2) dpw[j][v2] = 0.f;
                }
                // one token: dp from x and dy, dweight's and dbias' terms, and the row that it completes
                auto token = [&](auto inside, const float (&c)[V], float (&g)[V], bool in_seq, bool mine, float (&o)[V]) {
                    float old[W - 1][V], s[V];
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
#pragma unroll
                        for (int v = 0; v < V; ++v) old[k][v] = win[k][v];
                    taps<W, V>(w, bias, win, c, s);
                    if constexpr (SILU) {
#pragma unroll
                        for (int v = 0; v < V; ++v) g[v] *= silu_slope(s[v], sigmoid(s[v]));
                    }
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if constexpr (!decltype(inside)::value) g[v] = in_seq ? g[v] : 0.f;
                        float own = g[v], last = c[v];
                        if constexpr (!decltype(inside)::value) {
                            // a token past the tile only completes rows, and must not bring in 0 times an infinity
                            own = mine ? own : 0.f, last = mine ? last : 0.f;
#pragma unroll
                            for (int k = 0; k < W - 1; ++k) old[k][v] = mine ? old[k][v] : 0.f;
                        }
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) dw[k][v] = fmaf(own, old[k][v], dw[k][v]);
                        dw[W - 1][v] = fmaf(own, last, dw[W - 1][v]);
                        db[v] += own;
                        // dpw holds the last W-1 dp
                        float r = w[0][v] * g[v];
#pragma unroll
                        for (int k = 1; k < W; ++k) r = fmaf(w[k][v], dpw[W - 1 - k][v], r);
                        o[v] = r;
#pragma unroll
                        for (int k = 0; k + 1 < W - 1; ++k) dpw[k][v] = dpw[k + 1][v];
                        dpw[W - 2][v] = g[v];
                    }
                };
                const int end = p.e + W - 1, plain = min(p.e, tail);
                for (int t = p.a; t < end; t += kStep) {
                    const int r0 = t - (W - 1);
                    Vec<T, V> cx[kStep], cg[kStep];
#pragma unroll
                    for (int i = 0; i < kStep; ++i) cx[i] = nx[i], cg[i] = ng[i];
                    if (t + kStep < end) fetch(t + kStep);
                    if (r0 >= p.a && t + kStep <= plain) {  // nothing special about these tokens and rows
#pragma unroll
                        for (int i = 0; i < kStep; ++i) {
                            float c[V], g[V], o[V];
                            widen<T, V>(cx[i], c), widen<T, V>(cg[i], g);
                            token(std::true_type{}, c, g, true, true, o);
                            store_vec<T, V>(dx.at(row, r0 + i), narrow<T, V>(o));
                        }
                        continue;
                    }
#pragma unroll
                    for (int i = 0; i < kStep; ++i) {
                        float c[V], g[V], o[V];
                        widen<T, V>(cx[i], c), widen<T, V>(cg[i], g);
                        token(std::false_type{}, c, g, t + i < p.E, t + i < p.e, o);
                        const int r = r0 + i;
                        if (r >= p.e || (r < p.a && !back)) continue;
                        if (a.dfinal && r >= tail) {
                            float f[V];
                            widen<T, V>(load_vec<T, V>(a.dfinal + ((int64_t)p.s * (W - 1) + (r - tail)) * a.C + c0), f);
#pragma unroll
                            for (int v = 0; v < V; ++v) o[v] += f[v];
                        }
                        if (r >= p.a)
                            store_vec<T, V>(dx.at(row, r), narrow<T, V>(o));
                        else
                            store_vec<T, V>(a.final_state + ((int64_t)p.s * (W - 1) + (r - p.S + W - 1)) * a.C + c0,
                                            narrow<T, V>(o));
                    }
                }
            });
        }
    }
    // add the block's warps, one tap after another
    __shared__ float red[kSub][kLanes * V];
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) red[threadIdx.y][v * kLanes + threadIdx.x] = k < W ? dw[k < W ? k : 0][v] : db[v];
        __syncthreads();
        for (int i = threadIdx.y * kLanes + threadIdx.x; i < kLanes * V; i += kLanes * kSub) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < kSub; ++q) s += red[q][i];
            const int c = (int)(blockIdx.x % a.ncb) * kLanes * V + (i % kLanes) * V + i / kLanes;
            if (c < a.C) a.partial[((int64_t)(slot0 + slot) * (W + 1) + k) * a.C + c] = s;
        }
    }
}

// Sum of the slots' partial sums in slot order: dweight[c, k], dbias[c].
__global__ void __launch_bounds__(256) conv_reduce_kernel(const float *__restrict__ partial, int slots, int W, int C,
                                                          float *__restrict__ dweight, float *__restrict__ dbias) {
    __shared__ float red[8][32];
    const int c = blockIdx.x * 32 + threadIdx.x, k = blockIdx.y;
    float s = 0.f;
    if (c < C)
        for (int q = threadIdx.y; q < slots; q += 8) s += partial[((int64_t)q * (W + 1) + k) * C + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < C) {
#pragma unroll
        for (int q = 1; q < 8; ++q) s += red[q][threadIdx.x];
        if (k < W) {
            if (dweight) dweight[(int64_t)c * W + k] = s;
        } else if (dbias) {
            dbias[c] = s;
        }
    }
}

// One token per sequence: the state's rows move up by one, in place.
template <typename T, int W, int V>
__global__ void __launch_bounds__(128) conv_step_kernel(const __grid_constant__ ConvArgs<T> a, T *state) {
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (i >= (int64_t)a.nseq * a.nvec) return;
    const int c0 = (int)(i % a.nvec) * V;
    const int b = (int)(i / a.nvec);
    T *st = state + (int64_t)b * (W - 1) * a.C + c0;
    Vec<T, V> row[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) row[k] = load_vec<T, V>(st + (int64_t)k * a.C);
    row[W - 1] = load_vec<T, V>(a.x.at(b, 0) + c0);
    float w[W][V], o[V];
    load_weights<T, W, V>(a, c0, w, o);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        float f[V];
        widen<T, V>(row[k], f);
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = fmaf(w[k][v], f[v], o[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = a.use_silu ? silu(o[v]) : o[v];
    store_vec<T, V>(a.y[0].at(b, 0) + c0, narrow<T, V>(o));
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_vec<T, V>(st + (int64_t)k * a.C, row[k + 1]);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 4096;  // tokens are counted in 32 bits, offsets in 64

ssd_status_t check(const ssd_conv_shape_t *s, const int64_t *cu, int64_t nseq) {
    if (!s || s->batch < 0 || s->seqlen < 0 || s->channels <= 0 || s->width <= 0) return SSD_ERR_INVALID_ARG;
    if (s->dtype != SSD_DTYPE_F32 && s->dtype != SSD_DTYPE_BF16) return SSD_ERR_INVALID_ARG;
    if (s->nparts < 1 || s->nparts > SSD_CONV_MAX_PARTS) return SSD_ERR_INVALID_ARG;
    int64_t left = s->channels;
    for (int64_t i = 0; i < s->nparts; ++i) {
        if (s->part[i] <= 0 || s->part[i] > left) return SSD_ERR_INVALID_ARG;
        left -= s->part[i];
    }
    if (left != 0) return SSD_ERR_INVALID_ARG;
    if (s->width < 2 || s->width > 4 || s->channels > (1 << 24)) return SSD_ERR_UNSUPPORTED;
    if (s->seqlen > kMaxTokens || s->batch > kMaxTokens) return SSD_ERR_UNSUPPORTED;
    if (cu) {
        if (s->batch != 1 || nseq > kMaxTokens || !offsets_ok(cu, nseq, s->seqlen)) return SSD_ERR_INVALID_ARG;
    }
    return SSD_OK;
}

// Tokens per tile: the longest of 128, 64, .. 8 that still makes 16 warps an SM
// (a tile reads W-1 rows beyond its own).
int pick_tile(int64_t ncb, int64_t tokens) {
    int tile = 128;
    while (tile > 8 && ncb * (tokens / tile) < 152 * 16) tile /= 2;
    return tile;
}

template <typename T>
bool fill(const ssd_conv_shape_t *s, int64_t nseq, const ssd_rows_t *x, const ssd_rows_t *y, const ssd_rows_t *dx,
          std::initializer_list<const void *> states, int V, ConvArgs<T> &a) {
    const size_t es = sizeof(T);
    bool vec = aligned(a.weight, 16) && s->channels * es % 16 == 0 && rows_vec(*x, es, s->batch, s->seqlen);
    if (dx) vec = vec && rows_vec(*dx, es, s->batch, s->seqlen);
    int64_t end = 0;
    for (int i = 0; i < SSD_CONV_MAX_PARTS; ++i) {
        if (i < s->nparts) {
            end += s->part[i];
            vec = vec && s->part[i] * es % 16 == 0 && rows_vec(y[i], es, s->batch, s->seqlen);
            a.y[i] = rows_of<T>(y[i]);
        } else {
            a.y[i] = a.y[0];
        }
        a.part_end[i] = (int)end;
    }
    for (const void *p : states) vec = vec && (!p || aligned(p, 16));
    a.x = rows_of<const T>(*x);
    a.C = (int)s->channels;
    a.nvec = vec ? a.C / V : a.C;
    a.ncb = (a.nvec + kLanes - 1) / kLanes;
    a.L = (int)s->seqlen;
    a.nseq = (int)nseq;
    a.use_silu = s->silu != 0;
    return vec;
}

bool states_ok(std::initializer_list<const void *> states, size_t es) {
    for (const void *p : states)
        if (p && !aligned(p, es)) return false;
    return true;
}

// The next launch's sequences of a packed batch: as many as fit its
// parameters.  Sequences are taken in order, so a set's tokens are one run.
int next_set(const int64_t *cu, int64_t nseq, int64_t first, SeqSet &set) {
    set.n = (int)(nseq - first < kMaxSet ? nseq - first : kMaxSet);
    set.first = (int)first;
    for (int i = 0; i <= set.n; ++i) set.start[i] = (int)cu[first + i];
    return set.n;
}

template <typename T, int W, int V, bool PACKED, typename Set>
ssd_status_t launch_fwd(ConvArgs<T> &a, const Set &set, int64_t tokens, int64_t nseq, cudaStream_t st) {
    a.tile = pick_tile(a.ncb, tokens);
    a.ntiles = PACKED ? (int)((tokens + a.tile - 1) / a.tile) : (int)(nseq * ((a.L + a.tile - 1) / a.tile));
    a.tblocks = (int64_t)a.ncb * ((a.ntiles + kSub - 1) / kSub);
    int64_t blocks = a.tblocks;
    if (a.final_state) blocks += (nseq * (W - 1) * a.nvec + kLanes * kSub - 1) / (kLanes * kSub);
    if (blocks > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
    if (blocks == 0) return SSD_OK;
    if (a.use_silu)
        conv_fwd_kernel<T, W, V, PACKED, true, Set><<<(unsigned)blocks, dim3(kLanes, kSub), 0, st>>>(a, set);
    else
        conv_fwd_kernel<T, W, V, PACKED, false, Set><<<(unsigned)blocks, dim3(kLanes, kSub), 0, st>>>(a, set);
    timing_mark(st, "conv_fwd");
    return status_of(cudaGetLastError());
}

template <typename T, int W, int V>
ssd_status_t run_fwd(ConvArgs<T> &a, const ssd_conv_shape_t *s, const int64_t *cu, int64_t nseq, cudaStream_t st) {
    timing_begin(st);
    if (!cu) return launch_fwd<T, W, V, false>(a, NoSet{}, s->batch * s->seqlen, s->batch, st);
    SeqSet set;
    for (int64_t first = 0; first < nseq; first += kMaxSet) {
        next_set(cu, nseq, first, set);
        const ssd_status_t e =
            launch_fwd<T, W, V, true>(a, set, set.start[set.n] - set.start[0], set.n, st);
        if (e != SSD_OK) return e;
    }
    return SSD_OK;
}

// The gradient's blocks per channel block (a slot's block walks every
// slots-th group of kSub tiles), two an SM, and tiles of 32 to 256 tokens that
// give every warp of them the same number.
struct BwdPlan {
    int slots, tile;
    int64_t ntiles;
};
BwdPlan plan_bwd(int64_t ncb, int64_t rows, int64_t L) {
    int64_t want = 152 * 2 / ncb;
    if (want < 1) want = 1;
    const int64_t warps = want * kSub, tokens = rows * L;
    const int64_t each = (tokens + warps - 1) / warps, rounds = (each + 255) / 256;
    int64_t tile = rounds ? (each + rounds - 1) / rounds : 32;
    if (tile < 32) tile = 32;
    BwdPlan p;
    p.tile = (int)tile;
    p.ntiles = rows * ((L + tile - 1) / tile);
    const int64_t groups = (p.ntiles + kSub - 1) / kSub;
    p.slots = (int)(groups < want ? groups : want);
    return p;
}
// The most slots that the call may use: with vectors of kVec channels (single
// ones make more channel blocks and so fewer slots).
int64_t total_slots(const ssd_conv_shape_t *s, const int64_t *cu, int64_t nseq) {
    const int64_t ncb = ((s->channels + kVec - 1) / kVec + kLanes - 1) / kLanes;
    int64_t want = 152 * 2 / ncb;
    if (want < 1) want = 1;
    return want * (cu ? (nseq + kMaxSet - 1) / kMaxSet : 1);
}

template <typename T, int W, int V, bool PACKED, typename Set>
ssd_status_t launch_bwd(ConvArgs<T> &a, const ssd_conv_shape_t *s, const Set &set, int64_t tokens, int64_t nseq, int slot0,
                        int *used, cudaStream_t st) {
    const BwdPlan p = plan_bwd(a.ncb, PACKED ? 1 : s->batch, PACKED ? tokens : s->seqlen);
    a.tile = p.tile, a.ntiles = (int)p.ntiles;
    const int slots = p.slots;
    a.tblocks = (int64_t)a.ncb * slots;
    int64_t blocks = a.tblocks;
    if (a.final_state) blocks += (nseq * (W - 1) * a.nvec + kLanes * kSub - 1) / (kLanes * kSub);
    *used = slots;
    if (blocks > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
    if (blocks == 0) return SSD_OK;
    if (a.use_silu)
        conv_bwd_kernel<T, W, V, PACKED, true, Set><<<(unsigned)blocks, dim3(kLanes, kSub), 0, st>>>(a, set, slots, slot0);
    else
        conv_bwd_kernel<T, W, V, PACKED, false, Set><<<(unsigned)blocks, dim3(kLanes, kSub), 0, st>>>(a, set, slots, slot0);
    timing_mark(st, "conv_bwd");
    return status_of(cudaGetLastError());
}

template <typename T, int W, int V>
ssd_status_t run_bwd(ConvArgs<T> &a, const ssd_conv_shape_t *s, const int64_t *cu, int64_t nseq, float *dweight,
                     float *dbias, cudaStream_t st) {
    timing_begin(st);
    int slots = 0, used = 0;
    if (!cu) {
        const ssd_status_t e =
            launch_bwd<T, W, V, false>(a, s, NoSet{}, s->batch * s->seqlen, s->batch, 0, &used, st);
        if (e != SSD_OK) return e;
        slots = used;
    } else {
        SeqSet set;
        for (int64_t first = 0; first < nseq; first += kMaxSet) {
            next_set(cu, nseq, first, set);
            const ssd_status_t e = launch_bwd<T, W, V, true>(a, s, set, set.start[set.n] - set.start[0], set.n, slots,
                                                             &used, st);
            if (e != SSD_OK) return e;
            slots += used;
        }
    }
    if (!dweight && !dbias) return SSD_OK;
    conv_reduce_kernel<<<dim3((unsigned)((a.C + 31) / 32), (unsigned)(W + 1)), dim3(32, 8), 0, st>>>(
        a.partial, slots, W, a.C, dweight, dbias);
    timing_mark(st, "conv_reduce");
    return status_of(cudaGetLastError());
}

template <int N>
using Int = std::integral_constant<int, N>;

// f(W, V) as compile-time constants, for the width and the vector length (1
// where rows are not 16-byte aligned).
template <int V, typename F>
ssd_status_t dispatch(int64_t width, bool vec, F f) {
    if (width == 2) return vec ? f(Int<2>{}, Int<V>{}) : f(Int<2>{}, Int<1>{});
    if (width == 3) return vec ? f(Int<3>{}, Int<V>{}) : f(Int<3>{}, Int<1>{});
    return vec ? f(Int<4>{}, Int<V>{}) : f(Int<4>{}, Int<1>{});
}

template <typename T>
ssd_status_t fwd_typed(const ssd_conv_shape_t *s, const int64_t *cu, int64_t nseq, const ssd_rows_t *x,
                       const float *weight, const float *bias, const void *init, const ssd_rows_t *y, void *fin,
                       cudaStream_t st) {
    ConvArgs<T> a{};
    a.weight = weight, a.bias = bias;
    const bool vec = fill<T>(s, nseq, x, y, nullptr, {init, fin}, kVec, a);
    a.init = static_cast<const T *>(init), a.final_state = static_cast<T *>(fin);
    return dispatch<kVec>(s->width, vec, [&](auto w, auto v) {
        return run_fwd<T, decltype(w)::value, decltype(v)::value>(a, s, cu, nseq, st);
    });
}

template <typename T>
ssd_status_t bwd_typed(const ssd_conv_shape_t *s, const int64_t *cu, int64_t nseq, const ssd_rows_t *dy,
                       const ssd_rows_t *x, const float *weight, const float *bias, const void *init, const void *dfin,
                       const ssd_rows_t *dx, float *dweight, float *dbias, void *dinit, void *ws, cudaStream_t st) {
    ConvArgs<T> a{};
    a.weight = weight, a.bias = bias;
    const bool vec = fill<T>(s, nseq, x, dy, dx, {init, dfin, dinit}, kVec, a);
    a.dx = rows_of<T>(*dx);
    a.init = static_cast<const T *>(init), a.dfinal = static_cast<const T *>(dfin);
    a.final_state = static_cast<T *>(dinit);
    a.partial = static_cast<float *>(ws);
    return dispatch<kVec>(s->width, vec, [&](auto w, auto v) {
        return run_bwd<T, decltype(w)::value, decltype(v)::value>(a, s, cu, nseq, dweight, dbias, st);
    });
}

template <typename T>
ssd_status_t step_typed(const ssd_conv_shape_t *s, const ssd_rows_t *x, const float *weight, const float *bias,
                        void *state, const ssd_rows_t *y, cudaStream_t st) {
    ConvArgs<T> a{};
    a.weight = weight, a.bias = bias;
    const bool vec = fill<T>(s, s->batch, x, y, nullptr, {state}, kVec, a);
    return dispatch<kVec>(s->width, vec, [&](auto w, auto v) {
        const int64_t blocks = (s->batch * a.nvec + 127) / 128;
        if (blocks > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
        timing_begin(st);
        conv_step_kernel<T, decltype(w)::value, decltype(v)::value>
            <<<(unsigned)blocks, 128, 0, st>>>(a, static_cast<T *>(state));
        timing_mark(st, "conv_step");
        return status_of(cudaGetLastError());
    });
}

}  // namespace
}  // namespace ssd

extern "C" {

ssd_status_t ssd_conv_fwd(const ssd_conv_shape_t *shape, const int64_t *cu_seqlens, int64_t nseq, const ssd_rows_t *x,
                          const float *weight, const float *bias, const void *init_state, const ssd_rows_t *y,
                          void *final_state, cudaStream_t stream) {
    using namespace ssd;
    const ssd_status_t st = check(shape, cu_seqlens, nseq);
    if (st != SSD_OK) return st;
    const size_t es = dtype_size(shape->dtype);
    if (!cu_seqlens) nseq = shape->batch;
    if (nseq == 0) return SSD_OK;
    if (!x || !y || !weight || !aligned(weight, 4) || !aligned(bias, 4)) return SSD_ERR_INVALID_ARG;
    if (!states_ok({init_state, final_state}, es)) return SSD_ERR_INVALID_ARG;
    if (final_state && final_state == init_state) return SSD_ERR_INVALID_ARG;  // one is read while the other is written
    if (shape->seqlen > 0) {
        if (!rows_in_ok(*x, es)) return SSD_ERR_INVALID_ARG;
        for (int64_t i = 0; i < shape->nparts; ++i)
            if (!rows_out_ok(y[i], es, shape->batch, shape->seqlen, shape->part[i])) return SSD_ERR_INVALID_ARG;
    }
    if (shape->batch * shape->seqlen > kMaxTokens) return SSD_ERR_UNSUPPORTED;
    return shape->dtype == SSD_DTYPE_BF16
               ? fwd_typed<bf16>(shape, cu_seqlens, nseq, x, weight, bias, init_state, y, final_state, stream)
               : fwd_typed<float>(shape, cu_seqlens, nseq, x, weight, bias, init_state, y, final_state, stream);
}

size_t ssd_conv_bwd_workspace_size(const ssd_conv_shape_t *shape, const int64_t *cu_seqlens, int64_t nseq) {
    using namespace ssd;
    if (check(shape, cu_seqlens, nseq) != SSD_OK) return 0;
    // (one-element lanes make more channel blocks and so no more slots)
    return sizeof(float) * total_slots(shape, cu_seqlens, nseq) * (shape->width + 1) * shape->channels;
}

ssd_status_t ssd_conv_bwd(const ssd_conv_shape_t *shape, const int64_t *cu_seqlens, int64_t nseq, const ssd_rows_t *dy,
                          const ssd_rows_t *x, const float *weight, const float *bias, const void *init_state,
                          const void *dfinal_state, const ssd_rows_t *dx, float *dweight, float *dbias,
                          void *dinit_state, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace ssd;
    const ssd_status_t st = check(shape, cu_seqlens, nseq);
    if (st != SSD_OK) return st;
    const size_t es = dtype_size(shape->dtype);
    if (!cu_seqlens) nseq = shape->batch;
    if (!x || !dy || !dx || !weight || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(dweight, 4) ||
        !aligned(dbias, 4))
        return SSD_ERR_INVALID_ARG;
    if (!states_ok({init_state, dfinal_state, dinit_state}, es)) return SSD_ERR_INVALID_ARG;
    if (shape->seqlen > 0 && nseq > 0) {
        if (!rows_in_ok(*x, es) || !rows_out_ok(*dx, es, shape->batch, shape->seqlen, shape->channels))
            return SSD_ERR_INVALID_ARG;
        for (int64_t i = 0; i < shape->nparts; ++i)
            if (!rows_in_ok(dy[i], es)) return SSD_ERR_INVALID_ARG;
    }
    if (shape->batch * shape->seqlen > kMaxTokens) return SSD_ERR_UNSUPPORTED;
    const size_t need = ssd_conv_bwd_workspace_size(shape, cu_seqlens, nseq);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return SSD_ERR_WORKSPACE;
    return shape->dtype == SSD_DTYPE_BF16
               ? bwd_typed<bf16>(shape, cu_seqlens, nseq, dy, x, weight, bias, init_state, dfinal_state, dx, dweight,
                                 dbias, dinit_state, workspace, stream)
               : bwd_typed<float>(shape, cu_seqlens, nseq, dy, x, weight, bias, init_state, dfinal_state, dx, dweight,
                                  dbias, dinit_state, workspace, stream);
}

ssd_status_t ssd_conv_step(const ssd_conv_shape_t *shape, const ssd_rows_t *x, const float *weight, const float *bias,
                           void *state, const ssd_rows_t *y, cudaStream_t stream) {
    using namespace ssd;
    ssd_conv_shape_t one;
    if (!shape) return SSD_ERR_INVALID_ARG;
    one = *shape;
    one.seqlen = 1;
    const ssd_status_t st = check(&one, nullptr, 0);
    if (st != SSD_OK) return st;
    if (one.nparts != 1) return SSD_ERR_INVALID_ARG;
    if (one.batch == 0) return SSD_OK;
    const size_t es = dtype_size(one.dtype);
    if (!x || !y || !weight || !state || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(state, es))
        return SSD_ERR_INVALID_ARG;
    if (!rows_in_ok(*x, es) || !rows_out_ok(*y, es, one.batch, 1, one.channels)) return SSD_ERR_INVALID_ARG;
    return one.dtype == SSD_DTYPE_BF16 ? step_typed<bf16>(&one, x, weight, bias, state, y, stream)
                                       : step_typed<float>(&one, x, weight, bias, state, y, stream);
}

}  // extern "C"
