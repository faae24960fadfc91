// ssd_channel.cu -- the channel scan over prompts and single tokens, and the
// host side of all its entry points.  (Gradient kernels: ssd_channel_bwd.cu.)
//
// Forward.  With b * channels / 32 warps enough to fill the SMs, one pass
// walks every sequence.  With fewer, the tokens are cut into chunks: a first
// launch forms every chunk's end state from a zero start (or from the
// sequence's own start) and the sum of its deltas; the second starts a chunk
// from the combination of the earlier ones, where a chunk's decay is
// exp(A sum delta), and writes y.  That costs up to 1.75 times the arithmetic
// on SMs that would otherwise idle.  Chunks are cut without regard to
// sequences, which restart the state inside a chunk.
#include "ssd_channel.h"

namespace ssd {
namespace {

constexpr int kTB = 8;     // tokens staged at a time
constexpr int kWarps = 4;  // warps per block

template <int N>
struct alignas(16) Stage {
    float d[kTB][32], u[kTB][32], bc[kTB][2 * N];
};

// What a lane has in flight for the next kTB tokens: its own channel's
// values and its share of their B and C.
template <typename T, int N, bool FULL>
struct Ahead {
    static constexpr int NB = kTB * 2 * N / 32;
    T x[kTB], dt[kTB], z[FULL ? kTB : 1], bc[NB];

    __device__ __forceinline__ void load(const ChannelArgs<T> &a, const Block &k, int row, int t, int n, int lane) {
        const bool mine = lane < k.nc;
        const int c = k.c0 + lane;
#pragma unroll
        for (int j = 0; j < kTB; ++j) {
            const bool in = j < n && mine;
            x[j] = in ? a.x.at(row, t + j)[c] : from_f32<T>(0.f);
            dt[j] = in ? a.dt.at(row, t + j)[c] : from_f32<T>(0.f);
            if (FULL && a.z.p) z[FULL ? j : 0] = in ? a.z.at(row, t + j)[c] : from_f32<T>(0.f);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int e = i * 32 + lane, j = e / (2 * N), w = e % (2 * N);
            T v = from_f32<T>(0.f);
            if (j < n && (FULL || w < N))
                v = w < N ? a.B.at(row, t + j)[k.g * N + w] : a.C.at(row, t + j)[k.g * N + w - N];
            bc[i] = v;
        }
    }
};

// FULL: outputs; otherwise only the chunk's end state and sum of deltas.
template <typename T, int N, bool FULL>
__global__ void __launch_bounds__(kWarps * 32) channel_fwd_kernel(const __grid_constant__ ChannelArgs<T> a) {
    constexpr int K = Tile<N>::K, M = Tile<N>::M, M2 = Tile<N>::M2;
    __shared__ Stage<N> stage[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t id = (int64_t)blockIdx.x * kWarps + warp;
    if (id >= (int64_t)a.units * a.nblk) return;  // whole warps; only warp barriers below
    const int blk = (int)(id % a.nblk), unit = (int)(id / a.nblk);
    Stage<N> &sm = stage[warp];
    const Block k = block_of(blk, a.per, a.nblk_g);
    const int cg = lane / K, q = lane % K;
    const bool mine = lane < k.nc;
    const int own = k.c0 + (mine ? lane : 0);

    f2 A2[K][M2], h[K][M2];
    load_tile<N>(a.A + (int64_t)k.c0 * N, lane, k.nc, A2);
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
        for (int j = 0; j < M2; ++j) A2[i][j] = mul2(A2[i][j], pack2(kLog2e, kLog2e));
    const float bias = a.bias && mine ? a.bias[own] : 0.f;
    const float D = FULL && a.D && mine ? a.D[own] : 0.f;

    // this unit's tokens
    const bool packed = a.seqs.start != nullptr;
    const int seq0 = packed ? 0 : unit / a.nchunk, row = seq0;
    const int c_in = packed ? unit : unit % a.nchunk;
    const int t0 = c_in * a.chunk, t1 = min(a.seqs.L, t0 + a.chunk);
    int s = seq0, S = 0, E = a.seqs.L, t = t0;
    if (packed) {
        s = seq_of(a.seqs, FULL ? t0 : t1 - 1);
        S = a.seqs.start[s], E = a.seqs.start[s + 1];
        if (!FULL) t = max(t, S);  // only what reaches the chunk's end
    }
    if (!FULL && E <= t1) return;  // nothing passes to the next chunk

    while (true) {
        const int e = min(t1, E);
        // the state before token t
        if (t == S) {
            if (a.init) {
                load_tile<N>(a.init + ((int64_t)s * a.ch + k.c0) * N, lane, k.nc, h);
            } else {
#pragma unroll
                for (int i = 0; i < K; ++i)
#pragma unroll
                    for (int j = 0; j < M2; ++j) h[i][j] = 0;
            }
        } else if (FULL) {
            const int first = packed ? S / a.chunk : unit - c_in;
            load_lanes<N>(a.local + ((int64_t)first * a.nblk + blk) * (N / 4 * 32), lane, h);
            for (int c = first + 1; c < unit; ++c) {
                const int64_t at = (int64_t)c * a.nblk + blk;
                f2 l[K][M2];
                float sd[K];
                load_lanes<N>(a.local + at * (N / 4 * 32), lane, l);
                load_k<K>(a.sums + at * 32 + cg * K, sd);
#pragma unroll
                for (int i = 0; i < K; ++i)
#pragma unroll
                    for (int j = 0; j < M2; ++j)
                        h[i][j] = fma2(ex2x2(mul2(A2[i][j], pack2(sd[i], sd[i]))), h[i][j], l[i][j]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < K; ++i)
#pragma unroll
                for (int j = 0; j < M2; ++j) h[i][j] = 0;
        }
        float total = 0.f;
        Ahead<T, N, FULL> nxt;
        nxt.load(a, k, row, t, e - t, lane);
        for (; t < e; t += kTB) {
            float x[kTB], z[kTB];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kTB; ++j) {
                // tokens past the end have delta = 0: they leave the state alone
                float d = to_f32(nxt.dt[j]) + bias;
                if (a.soft) d = softplus(d);
                if (t + j >= e || !mine) d = 0.f;
                x[j] = to_f32(nxt.x[j]);
                if (FULL && a.z.p) z[j] = to_f32(nxt.z[FULL ? j : 0]);
                if (!FULL) total += d;
                sm.d[j][lane] = d;
                sm.u[j][lane] = d * x[j];
            }
#pragma unroll
            for (int i = 0; i < Ahead<T, N, FULL>::NB; ++i) (&sm.bc[0][0])[i * 32 + lane] = to_f32(nxt.bc[i]);
            __syncwarp();
            if (t + kTB < e) nxt.load(a, k, row, t + kTB, e - t - kTB, lane);
#pragma unroll
            for (int j = 0; j < kTB; ++j) {
                float d[K], u[K];
                f2 B[M2], C[M2];
                load_k<K>(&sm.d[j][cg * K], d);
                load_k<K>(&sm.u[j][cg * K], u);
                load_m<M>(&sm.bc[j][q * M], B);
                if (FULL) load_m<M>(&sm.bc[j][N + q * M], C);
                float p[K][1];
#pragma unroll
                for (int i = 0; i < K; ++i) {
                    const f2 dd = pack2(d[i], d[i]), uu = pack2(u[i], u[i]);
                    f2 acc = 0;
#pragma unroll
                    for (int m = 0; m < M2; ++m) {
                        const f2 decay = ex2x2(mul2(A2[i][m], dd));
                        h[i][m] = fma2(decay, h[i][m], mul2(uu, B[m]));
                        if (FULL) acc = fma2(h[i][m], C[m], acc);
                    }
                    p[i][0] = sum2(acc);
                }
                if (FULL) {
                    float y[1];
                    channel_sums<K, 1>(p, lane, y);
                    float o = fmaf(D, x[j], y[0]);
                    if (a.z.p) o *= silu(z[j]);
                    if (mine && t + j < e) a.y.at(row, t + j)[own] = from_f32<T>(o);
                }
            }
        }
        if (!FULL) {
            const int64_t at = (int64_t)unit * a.nblk + blk;
            store_lanes<N>(a.local + at * (N / 4 * 32), lane, h);
            a.sums[at * 32 + lane] = total;
            return;
        }
        if (e == E && a.fin) store_tile<N>(a.fin + ((int64_t)s * a.ch + k.c0) * N, lane, k.nc, h);
        if (e == t1) return;
        t = e;
        do ++s;
        while (a.seqs.start[s + 1] <= t);
        S = a.seqs.start[s], E = a.seqs.start[s + 1];
    }
}

// One token per sequence.  The fp32 state is read and written once, all else
// is small: bound by memory.  N / 4 lanes hold a channel's states, a float4
// each; a thread has kUnroll channels' states in flight.
constexpr int kUnroll = 4;
template <typename T, int N>
__global__ void __launch_bounds__(256) channel_step_kernel(const __grid_constant__ ChannelArgs<T> a, float *state) {
    constexpr int Q = N / 4;
    const int64_t total = (int64_t)a.nseq * a.ch * Q;  // float4s
    const int64_t base = (int64_t)blockIdx.x * (256 * kUnroll) + threadIdx.x;
    float4 *s4 = reinterpret_cast<float4 *>(state);
    float4 h[kUnroll];
#pragma unroll
    for (int r = 0; r < kUnroll; ++r)
        if (base + r * 256 < total) h[r] = __ldcs(s4 + base + r * 256);
#pragma unroll
    for (int r = 0; r < kUnroll; ++r) {
        const int64_t i = base + r * 256;
        const bool in = i < total;  // whole groups of Q lanes
        const int64_t bc = in ? i / Q : 0;
        const int q = (int)(i % Q), b = (int)(bc / a.ch), c = (int)(bc % a.ch);
        const int g = c / a.per;
        const float x = to_f32(a.x.at(b, 0)[c]);
        float d = to_f32(a.dt.at(b, 0)[c]) + (a.bias ? a.bias[c] : 0.f);
        if (a.soft) d = softplus(d);
        const float u = d * x;
        const float4 A = *reinterpret_cast<const float4 *>(a.A + (int64_t)c * N + 4 * q);
        const T *Bp = a.B.at(b, 0) + g * N + 4 * q, *Cp = a.C.at(b, 0) + g * N + 4 * q;
        float4 v = h[r];
        d *= kLog2e;
        v.x = fmaf(ex2(d * A.x), v.x, u * to_f32(Bp[0]));
        v.y = fmaf(ex2(d * A.y), v.y, u * to_f32(Bp[1]));
        v.z = fmaf(ex2(d * A.z), v.z, u * to_f32(Bp[2]));
        v.w = fmaf(ex2(d * A.w), v.w, u * to_f32(Bp[3]));
        if (in) __stcs(s4 + i, v);
        float y = fmaf(v.x, to_f32(Cp[0]),
                       fmaf(v.y, to_f32(Cp[1]), fmaf(v.z, to_f32(Cp[2]), v.w * to_f32(Cp[3]))));
#pragma unroll
        for (int off = Q / 2; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
        if (in && q == 0) {
            float o = fmaf(a.D ? a.D[c] : 0.f, x, y);
            if (a.z.p) o *= silu(to_f32(a.z.at(b, 0)[c]));
            a.y.at(b, 0)[c] = from_f32<T>(o);
        }
    }
}

}  // namespace

// Packed offsets, a launch's parameters at a time, into the workspace.
constexpr int kMaxSet = 960;
struct OffsetSet {
    int n, first;
    int v[kMaxSet];
};
static __global__ void __launch_bounds__(256) write_offsets_kernel(const __grid_constant__ OffsetSet s, int *dst) {
    for (int i = threadIdx.x; i < s.n; i += 256) dst[s.first + i] = s.v[i];
}
cudaError_t write_offsets(const int64_t *cu, int64_t nseq, int *dst, cudaStream_t st) {
    OffsetSet set;
    for (int64_t f = 0; f <= nseq; f += kMaxSet) {
        set.first = (int)f;
        set.n = (int)(nseq + 1 - f < kMaxSet ? nseq + 1 - f : kMaxSet);
        for (int i = 0; i < set.n; ++i) set.v[i] = (int)cu[f + i];
        write_offsets_kernel<<<1, 256, 0, st>>>(set, dst);
        timing_mark(st, "write_offsets");
    }
    return cudaGetLastError();
}

// Empty sequences hand a state on unchanged: dst[s] = src[s] (zero without
// src) for every s with start[s] == start[s + 1], or for all (start null).
static __global__ void __launch_bounds__(256) empty_states_kernel(const int *start, int64_t each, const float *src,
                                                                  float *dst) {
    const int64_t s = blockIdx.x;
    if (start && start[s] != start[s + 1]) return;
    for (int64_t i = (int64_t)blockIdx.y * 256 + threadIdx.x; i < each; i += (int64_t)gridDim.y * 256)
        dst[s * each + i] = src ? src[s * each + i] : 0.f;
}
cudaError_t pass_empty_states(const int *start, int64_t nseq, int64_t each, const float *src, float *dst,
                              cudaStream_t st) {
    empty_states_kernel<<<dim3((unsigned)nseq, 8), 256, 0, st>>>(start, each, src, dst);
    timing_mark(st, "empty_states");
    return cudaGetLastError();
}

ssd_status_t check_channel(const ssd_channel_shape_t *s, const int64_t *cu, int64_t nseq) {
    if (!s || s->batch < 0 || s->seqlen < 0 || s->channels <= 0 || s->dstate <= 0 || s->ngroups <= 0)
        return SSD_ERR_INVALID_ARG;
    if (s->dtype != SSD_DTYPE_F32 && s->dtype != SSD_DTYPE_BF16) return SSD_ERR_INVALID_ARG;
    if (s->channels % s->ngroups != 0) return SSD_ERR_INVALID_ARG;
    if (s->dstate != 8 && s->dstate != 16 && s->dstate != 32) return SSD_ERR_UNSUPPORTED;
    if (s->channels > (1 << 24) || s->seqlen > kMaxTokens || s->batch > kMaxTokens || s->batch * s->seqlen > kMaxTokens)
        return SSD_ERR_UNSUPPORTED;
    if (cu && (s->batch != 1 || nseq > kMaxTokens || !offsets_ok(cu, nseq, s->seqlen))) return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

bool channel_inputs_ok(const ssd_channel_shape_t *s, const ssd_channel_inputs_t *in, bool rows) {
    const size_t es = dtype_size(s->dtype);
    if (!in || !in->A || !aligned(in->A, 16) || !aligned(in->D, 4) || !aligned(in->dt_bias, 4) ||
        !aligned(in->init_state, 16))
        return false;
    if (!rows) return true;
    if (in->z.data && !rows_in_ok(in->z, es)) return false;
    return rows_in_ok(in->x, es) && rows_in_ok(in->dt, es) && rows_in_ok(in->B, es) && rows_in_ok(in->C, es);
}

namespace {

// Chunks: one per sequence where the warps suffice, otherwise enough for
// about eight warps an SM, of at least 64 tokens.
struct FwdPlan {
    int chunk, nchunk;  // tokens per chunk; chunks of a sequence (equal lengths) or of the batch (packed)
    int64_t units;
    size_t offsets, local, sums, bytes;  // workspace offsets
};
FwdPlan plan_fwd(const ssd_channel_shape_t *s, const int64_t *cu, int64_t nseq) {
    FwdPlan p{};
    const int64_t nblk = s->ngroups * ((s->channels / s->ngroups + 31) / 32);
    const int64_t rows = cu ? 1 : s->batch, L = s->seqlen;
    const int64_t base = nblk * (rows > 0 ? rows : 1);
    int64_t want = base >= 152 * 6 ? 1 : (152 * 8 + base - 1) / base;
    if (want > (L + 63) / 64) want = (L + 63) / 64;
    if (want < 1) want = 1;
    p.chunk = (int)(((L + want - 1) / want + kTB - 1) / kTB * kTB);
    if (p.chunk < kTB) p.chunk = kTB;
    p.nchunk = (int)((L + p.chunk - 1) / p.chunk);
    p.units = rows * p.nchunk;
    size_t at = 0;
    p.offsets = at;
    if (cu) at += align256(sizeof(int) * (nseq + 1));
    p.local = at;
    if (p.nchunk > 1) at += align256(sizeof(float) * p.units * nblk * s->dstate * 32);
    p.sums = at;
    if (p.nchunk > 1) at += align256(sizeof(float) * p.units * nblk * 32);
    p.bytes = at;
    return p;
}

template <typename T, int N>
ssd_status_t run_fwd(ChannelArgs<T> &a, const ssd_channel_shape_t *s, const int64_t *cu, int64_t nseq, char *ws,
                     cudaStream_t st) {
    const FwdPlan p = plan_fwd(s, cu, nseq);
    timing_begin(st);
    cudaError_t e = cudaSuccess;
    if (cu) {
        int *dst = reinterpret_cast<int *>(ws + p.offsets);
        e = write_offsets(cu, nseq, dst, st);
        if (e != cudaSuccess) return status_of(e);
        a.seqs.start = dst;
        bool empty = false;
        for (int64_t i = 0; i < nseq && !empty; ++i) empty = cu[i] == cu[i + 1];
        if (empty && a.fin) e = pass_empty_states(dst, nseq, s->channels * s->dstate, a.init, a.fin, st);
    } else if (s->seqlen == 0 && a.fin) {
        e = pass_empty_states(nullptr, nseq, s->channels * s->dstate, a.init, a.fin, st);
    }
    if (e != cudaSuccess) return status_of(e);
    if (s->seqlen == 0) return SSD_OK;
    a.chunk = p.chunk, a.nchunk = p.nchunk, a.units = (int)p.units;
    a.local = reinterpret_cast<float4 *>(ws + p.local);
    a.sums = reinterpret_cast<float *>(ws + p.sums);
    const int64_t blocks = (p.units * a.nblk + kWarps - 1) / kWarps;
    if (blocks > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
    if (p.nchunk > 1) {
        channel_fwd_kernel<T, N, false><<<(unsigned)blocks, kWarps * 32, 0, st>>>(a);
        timing_mark(st, "channel_chunk_state");
    }
    channel_fwd_kernel<T, N, true><<<(unsigned)blocks, kWarps * 32, 0, st>>>(a);
    timing_mark(st, "channel_scan");
    return status_of(cudaGetLastError());
}

template <typename T>
ssd_status_t fwd_typed(const ssd_channel_shape_t *s, const int64_t *cu, int64_t nseq, const ssd_channel_inputs_t *in,
                       const ssd_rows_t *y, float *fin, void *ws, cudaStream_t st) {
    ChannelArgs<T> a = channel_args<T>(s, in, nseq);
    a.y = rows_of<T>(*y);
    a.fin = fin;
    char *w = static_cast<char *>(ws);
    if (s->dstate == 8) return run_fwd<T, 8>(a, s, cu, nseq, w, st);
    if (s->dstate == 16) return run_fwd<T, 16>(a, s, cu, nseq, w, st);
    return run_fwd<T, 32>(a, s, cu, nseq, w, st);
}

template <typename T>
ssd_status_t step_typed(const ssd_channel_shape_t *s, const ssd_channel_inputs_t *in, float *state, const ssd_rows_t *y,
                        cudaStream_t st) {
    ChannelArgs<T> a = channel_args<T>(s, in, s->batch);
    a.y = rows_of<T>(*y);
    const int64_t blocks = (s->batch * s->channels * (s->dstate / 4) + 256 * kUnroll - 1) / (256 * kUnroll);
    if (blocks > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
    timing_begin(st);
    if (s->dstate == 8)
        channel_step_kernel<T, 8><<<(unsigned)blocks, 256, 0, st>>>(a, state);
    else if (s->dstate == 16)
        channel_step_kernel<T, 16><<<(unsigned)blocks, 256, 0, st>>>(a, state);
    else
        channel_step_kernel<T, 32><<<(unsigned)blocks, 256, 0, st>>>(a, state);
    timing_mark(st, "channel_step");
    return status_of(cudaGetLastError());
}

}  // namespace
}  // namespace ssd

extern "C" {

size_t ssd_channel_scan_workspace_size(const ssd_channel_shape_t *shape, const int64_t *cu_seqlens, int64_t nseq) {
    using namespace ssd;
    if (check_channel(shape, cu_seqlens, nseq) != SSD_OK) return 0;
    return plan_fwd(shape, cu_seqlens, nseq).bytes;
}

ssd_status_t ssd_channel_scan_fwd(const ssd_channel_shape_t *shape, const int64_t *cu_seqlens, int64_t nseq,
                                  const ssd_channel_inputs_t *in, const ssd_rows_t *y, float *final_state,
                                  void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace ssd;
    const ssd_status_t st = check_channel(shape, cu_seqlens, nseq);
    if (st != SSD_OK) return st;
    if (!cu_seqlens) nseq = shape->batch;
    if (nseq == 0) return SSD_OK;
    const bool rows = shape->seqlen > 0;
    if (!channel_inputs_ok(shape, in, rows) || !y || !aligned(final_state, 16)) return SSD_ERR_INVALID_ARG;
    if (rows && !rows_out_ok(*y, dtype_size(shape->dtype), shape->batch, shape->seqlen, shape->channels))
        return SSD_ERR_INVALID_ARG;
    const size_t need = plan_fwd(shape, cu_seqlens, nseq).bytes;
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return SSD_ERR_WORKSPACE;
    return shape->dtype == SSD_DTYPE_BF16 ? fwd_typed<bf16>(shape, cu_seqlens, nseq, in, y, final_state, workspace, stream)
                                          : fwd_typed<float>(shape, cu_seqlens, nseq, in, y, final_state, workspace, stream);
}

ssd_status_t ssd_channel_scan_step(const ssd_channel_shape_t *shape, const ssd_channel_inputs_t *in, float *state,
                                   const ssd_rows_t *y, cudaStream_t stream) {
    using namespace ssd;
    if (!shape) return SSD_ERR_INVALID_ARG;
    ssd_channel_shape_t one = *shape;
    one.seqlen = 1;
    const ssd_status_t st = check_channel(&one, nullptr, 0);
    if (st != SSD_OK) return st;
    if (one.batch == 0) return SSD_OK;
    if (!channel_inputs_ok(&one, in, true) || !y || !state || !aligned(state, 16)) return SSD_ERR_INVALID_ARG;
    if (!rows_out_ok(*y, dtype_size(one.dtype), one.batch, 1, one.channels)) return SSD_ERR_INVALID_ARG;
    return one.dtype == SSD_DTYPE_BF16 ? step_typed<bf16>(&one, in, state, y, stream)
                                       : step_typed<float>(&one, in, state, y, stream);
}

}  // extern "C"
