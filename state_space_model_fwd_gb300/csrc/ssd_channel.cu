// ssd_channel.cu -- the channel scan over prompts and single tokens, and the
// host side of all its entry points.  (Gradient kernels: ssd_channel_bwd.cu.)
//
// Forward.  A block row is 32 channels of a sequence row, one warp's work.  Where
// there are two for every warp scheduler, one pass walks every sequence.  With
// fewer, the tokens are cut into chunks: a first launch forms every chunk's end
// state from a zero start (or from the sequence's own start) and the sum of its
// deltas; the second starts a chunk from the combination of the earlier ones,
// where a chunk's decay is exp(A sum delta), and writes y.  That costs up to
// 1.6 times the arithmetic on SMs that would otherwise idle, and on top one
// step a chunk for every earlier chunk of its sequence: few beside its tokens,
// except where one or two block rows are cut into a thousand chunks (1 x 100000
// x 32, 1137 chunks of 88 tokens: 17 us for the first launch, 152 for the
// second).  Chunks are cut without regard to sequences, which restart the state
// inside a chunk.
//
// Bound by instruction issue and what two warps a scheduler leave uncovered of
// the instructions' latencies: 108 instructions a token and warp (16 states), 32
// of them packed multiply-adds that take two issue cycles, 16 exponentials; 805
// us at 8 x 4096 x 5120 bf16 with gate, an instruction in 58 % of the main
// launch's cycles, 75 % with the packed ones' second cycle.  The bytes would
// take 199 us, the fp32 results alone (4 a state) 290 us.
#include <type_traits>

#include "ssd_channel.h"

namespace ssd {
namespace {

constexpr int kTB = 8;     // tokens staged at a time
constexpr int kWarps = 4;  // warps per block, one for each of an SM's schedulers

// What a lane has in flight for the next kTB tokens: its channel's values and
// its share of B and C.  A lane without a channel reads the block's first one:
// its states have A = 0 and are never stored.
template <typename T, int N, bool FULL, bool GATE>
struct Ahead {
    static constexpr int NB = kTB * 2 * N / 32;
    T x[kTB], dt[kTB], z[GATE ? kTB : 1], bc[NB];

    __device__ __forceinline__ void load(const T *px, const T *pdt, const T *pz, const T *pb, const T *pc,
                                         const ChannelArgs<T> &a, int n, int lane) {
        if (n >= kTB) {
#pragma unroll
            for (int j = 0; j < kTB; ++j) {
                x[j] = px[a.x.step(j)];
                dt[j] = pdt[a.dt.step(j)];
                if (GATE) z[GATE ? j : 0] = pz[a.z.step(j)];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kTB; ++j) {
                x[j] = j < n ? px[a.x.step(j)] : from_f32<T>(0.f);
                dt[j] = j < n ? pdt[a.dt.step(j)] : from_f32<T>(0.f);
                if (GATE) z[GATE ? j : 0] = j < n ? pz[a.z.step(j)] : from_f32<T>(0.f);
            }
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int j = (i * 32 + lane) / (2 * N);
            const bool is_b = (i * 32 + lane) % (2 * N) < N;
            bc[i] = from_f32<T>(0.f);
            if (j < n && (FULL || is_b)) bc[i] = is_b ? pb[a.B.step(j)] : pc[a.C.step(j)];
        }
    }
};

// A lane is a channel: its N states, their decay rates and its delta stay in
// registers, nothing is summed over lanes, and B and C come from shared
// memory as broadcasts, N / 2 reads of 16 bytes a token.  A square tile of
// channels and states a lane reads a third of that but needs 25 instructions
// more a token to stage delta and to transpose the sums.
// Nothing branches between the staging and the stores: with the gate's switch
// and predicated stores inside the token loop, tokens did not overlap and the
// same case took 1400 us.
//
// FULL: outputs; otherwise only the chunk's end state and sum of deltas.  The
// warps of a block share nothing.
template <typename T, int N, bool FULL, bool GATE>
__global__ void __launch_bounds__(kWarps * 32, 2) channel_fwd_kernel(const __grid_constant__ ChannelArgs<T> a) {
    using G = Tile<N, 1, 1>;
    constexpr int N2 = N / 2, E = N / 4;
    __shared__ __align__(16) float stage[kWarps][kTB][2 * N];
    const int lane = threadIdx.x % 32;
    auto &sm = stage[threadIdx.x / 32];
    const bool packed = a.seqs.packed;
    const int *start = a.seqs.offsets();
    launch_next();
    if (a.seqs.start) wait_previous();  // the offsets
    if (FULL && blockIdx.x >= a.blocks) {
        pass_empty_states(start, a.seqs.n, (int64_t)a.ch * N, a.init, a.fin, blockIdx.x - a.blocks, gridDim.x - a.blocks);
        return;
    }
    const int64_t warp = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (warp >= (FULL ? a.whole : 0) + (int64_t)a.cut * a.nchunk) return;  // (only warp barriers below)
    // a block row is a channel block of a sequence row; those from a.whole on
    // are cut into chunks
    const bool whole = FULL && warp < a.whole;
    const int id = (int)warp - (FULL ? a.whole : 0);
    const int r = whole ? 0 : id % a.cut, c_in = whole ? 0 : id / a.cut, brow = whole ? (int)warp : a.whole + r;
    const int blk = brow % a.nblk, row = brow / a.nblk;
    const Block k = block_of(blk, a.per, a.nblk_g, 32);
    const bool mine = lane < k.nc;
    const int own = k.c0 + (mine ? lane : 0);

    typename G::Regs A2, h;
    load_tile<G>(a.A + (int64_t)k.c0 * N, lane, k.nc, A2);
#pragma unroll
    for (int m = 0; m < N2; ++m) A2[0][m] = mul2(A2[0][m], pack2(kLog2e, kLog2e));
    const float bias = a.bias ? a.bias[own] : 0.f;
    const float D = FULL && a.D ? a.D[own] : 0.f;

    // this warp's tokens
    // (the last chunk's end is formed from what is left: t0 + a.chunk may pass 2^31)
    const int t0 = c_in * a.chunk, t1 = whole || a.seqs.L - t0 <= a.chunk ? a.seqs.L : t0 + a.chunk;
    int s = row, S0 = 0, S1 = a.seqs.L, t = t0;
    if (packed) {
        s = seq_of(start, a.seqs.n, FULL ? t0 : t1 - 1);
        S0 = start[s], S1 = start[s + 1];
        if (!FULL) t = max(t, S0);  // only what reaches the chunk's end
    }
    if (!FULL && S1 <= t1) return;  // nothing passes to the next chunk
    // (pointers may come to stand past the last token: they are read through only where a token is)
    const T *px = a.x.at(row, t) + own, *pdt = a.dt.at(row, t) + own;
    const T *pz = GATE ? a.z.at(row, t) + own : nullptr;
    const T *pb = a.B.at(row, t) + k.g * N + lane % N, *pc = a.C.at(row, t) + k.g * N + lane % N;
    T *py = FULL ? a.y.at(row, t) + own : nullptr;

    while (true) {
        const int e = min(t1, S1);
        Ahead<T, N, FULL, GATE> nxt;
        nxt.load(px, pdt, pz, pb, pc, a, e - t, lane);
        // the state before token t
        zero_tile<G>(h);
        if (t == S0) {
            if (a.init) load_tile<G>(a.init + ((int64_t)s * a.ch + k.c0) * N, lane, k.nc, h);
        } else if (FULL) {
            wait_previous();
            const int first = S0 / a.chunk;
            load_lanes<G>(a.local + ((int64_t)first * a.cut + r) * (E * 32), lane, h);
#pragma unroll 4
            for (int c = first + 1; c < c_in; ++c) {
                const int64_t at = (int64_t)c * a.cut + r;
                typename G::Regs l;
                load_lanes<G>(a.local + at * (E * 32), lane, l);
                const float sd = a.sums[at * 32 + lane];
#pragma unroll
                for (int m = 0; m < N2; ++m)
                    h[0][m] = fma2(ex2x2(mul2(A2[0][m], pack2(sd, sd))), h[0][m], l[0][m]);
            }
        }
        float total = 0.f;
        for (; t < e; t += kTB) {
            const int n = e - t;
            // (straight-line code from here to the stores, so that the tokens' chains overlap)
            float d[kTB], x[kTB], z[GATE ? kTB : 1], o[kTB];
#pragma unroll
            for (int j = 0; j < kTB; ++j) {
                d[j] = to_f32(nxt.dt[j]) + bias;
                x[j] = to_f32(nxt.x[j]);
                if (GATE) z[GATE ? j : 0] = to_f32(nxt.z[GATE ? j : 0]);
            }
            if (a.soft) {
#pragma unroll
                for (int j = 0; j < kTB; ++j) d[j] = softplus(d[j]);
            }
            if (n < kTB) {  // tokens past the end leave the state alone
#pragma unroll
                for (int j = 0; j < kTB; ++j) d[j] = j < n ? d[j] : 0.f;
            }
            if (!FULL) {
#pragma unroll
                for (int j = 0; j < kTB; ++j) total += d[j];
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < Ahead<T, N, FULL, GATE>::NB; ++i) (&sm[0][0])[i * 32 + lane] = to_f32(nxt.bc[i]);
            __syncwarp();
            px += a.x.step(kTB), pdt += a.dt.step(kTB), pb += a.B.step(kTB), pc += a.C.step(kTB);
            if (GATE) pz += a.z.step(kTB);
            if (n > kTB) nxt.load(px, pdt, pz, pb, pc, a, n - kTB, lane);
#pragma unroll
            for (int j = 0; j < kTB; ++j) {
                f2 acc[2] = {0, 0};
                const f2 dd = pack2(d[j], d[j]), uu = pack2(d[j] * x[j], d[j] * x[j]);
#pragma unroll
                for (int m = 0; m < N2; m += 2) {
                    const ulonglong2 B = *reinterpret_cast<const ulonglong2 *>(&sm[j][2 * m]);
                    h[0][m] = fma2(ex2x2(mul2(A2[0][m], dd)), h[0][m], mul2(uu, B.x));
                    h[0][m + 1] = fma2(ex2x2(mul2(A2[0][m + 1], dd)), h[0][m + 1], mul2(uu, B.y));
                    if (FULL) {
                        const ulonglong2 C = *reinterpret_cast<const ulonglong2 *>(&sm[j][N + 2 * m]);
                        acc[0] = m ? fma2(h[0][m], C.x, acc[0]) : mul2(h[0][m], C.x);
                        acc[1] = m ? fma2(h[0][m + 1], C.y, acc[1]) : mul2(h[0][m + 1], C.y);
                    }
                }
                if (FULL) {
                    o[j] = fmaf(D, x[j], sum2(add2(acc[0], acc[1])));
                    if (GATE) o[j] *= silu(z[GATE ? j : 0]);
                }
            }
            if (FULL && mine) {
                if (n >= kTB) {
#pragma unroll
                    for (int j = 0; j < kTB; ++j) py[a.y.step(j)] = from_f32<T>(o[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < kTB; ++j)
                        if (j < n) py[a.y.step(j)] = from_f32<T>(o[j]);
                }
            }
            if (FULL) py += a.y.step(kTB);
        }
        if (!FULL) {
            const int64_t at = (int64_t)c_in * a.cut + r;
            store_lanes<G>(a.local + at * (E * 32), lane, h);
            a.sums[at * 32 + lane] = total;
            return;
        }
        if (e == S1 && a.fin) store_tile<G>(a.fin + ((int64_t)s * a.ch + k.c0) * N, lane, k.nc, h);
        if (e == t1) return;
        const int over = t - e;  // the last step went past the piece
        px -= a.x.step(over), pdt -= a.dt.step(over), pb -= a.B.step(over), pc -= a.C.step(over);
        py -= a.y.step(over);
        if (GATE) pz -= a.z.step(over);
        t = e;
        do ++s;
        while (start[s + 1] <= t);
        S0 = start[s], S1 = start[s + 1];
    }
}

// One token per sequence.  The fp32 state is read and written once, all else
// is small: bound by memory.  N / 4 lanes hold a channel's states, a float4
// each, for kRows sequences at a time: kRows state loads in flight, the decay
// rates read once for all of them.  What is per channel and sequence is done
// by one lane (lane q for sequences q, q + N / 4, ..) and passed on by
// shuffles, and the sums over states are transposed back to that lane.
constexpr int kRows = 4;
template <typename T, int N, bool VEC>
__global__ void __launch_bounds__(256) channel_step_kernel(const __grid_constant__ ChannelArgs<T> a, float *state) {
    constexpr int Q = N / 4, MINE = kRows / Q > 0 ? kRows / Q : 1;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const bool in = i < (int64_t)a.ch * Q;  // whole groups of Q lanes
    const int c = in ? (int)(i / Q) : 0, q = threadIdx.x % Q, g = c / a.per;
    const int b0 = blockIdx.y * kRows, nb = min(kRows, a.nseq - b0);
    float4 *s4 = reinterpret_cast<float4 *>(state) + ((int64_t)b0 * a.ch + c) * Q + q;
    const int64_t row4 = (int64_t)a.ch * Q;
    float4 h[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        if (in && r < nb) h[r] = __ldcs(s4 + r * row4);
    // this lane's sequences
    float d[MINE], x[MINE], z[MINE];
    const float bias = a.bias ? a.bias[c] : 0.f;
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
        const int r = q + k * Q;
        d[k] = x[k] = z[k] = 0.f;
        if (r < nb) {
            d[k] = to_f32(a.dt.at(b0 + r, 0)[c]) + bias;
            x[k] = to_f32(a.x.at(b0 + r, 0)[c]);
            if (a.z.p) z[k] = to_f32(a.z.at(b0 + r, 0)[c]);
            if (a.soft) d[k] = softplus(d[k]);
        }
    }
    float4 A = *reinterpret_cast<const float4 *>(a.A + (int64_t)c * N + 4 * q);
    A.x *= kLog2e, A.y *= kLog2e, A.z *= kLog2e, A.w *= kLog2e;
    float y[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int k = r / Q < MINE ? r / Q : 0;
        const float dr = __shfl_sync(0xffffffffu, d[k], r % Q, Q);
        const float ur = dr * __shfl_sync(0xffffffffu, x[k], r % Q, Q);
        y[r] = 0.f;
        if (in && r < nb) {
            float B[4], C[4];
            const T *pb = a.B.at(b0 + r, 0) + g * N + 4 * q, *pc = a.C.at(b0 + r, 0) + g * N + 4 * q;
            if constexpr (VEC) {
                widen<T, 4>(load_vec<T, 4>(pb), B);
                widen<T, 4>(load_vec<T, 4>(pc), C);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) B[j] = to_f32(pb[j]), C[j] = to_f32(pc[j]);
            }
            float4 v = h[r];
            v.x = fmaf(ex2(dr * A.x), v.x, ur * B[0]);
            v.y = fmaf(ex2(dr * A.y), v.y, ur * B[1]);
            v.z = fmaf(ex2(dr * A.z), v.z, ur * B[2]);
            v.w = fmaf(ex2(dr * A.w), v.w, ur * B[3]);
            __stcs(s4 + r * row4, v);
            y[r] = fmaf(v.x, C[0], fmaf(v.y, C[1], fmaf(v.z, C[2], v.w * C[3])));
        }
    }
    // lane q ends with the sums of its own sequences
    float o[MINE];
    if constexpr (Q == 2) {
        float v[2][2] = {{y[0], y[2]}, {y[1], y[3]}};
        group_sums<2, 2>(v, threadIdx.x, o);
    } else {
        if constexpr (Q == 8) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) y[r] += __shfl_xor_sync(0xffffffffu, y[r], 4);
        }
        float v[4][1] = {{y[0]}, {y[1]}, {y[2]}, {y[3]}};
        group_sums<4, 1>(v, threadIdx.x, o);
    }
    const float D = a.D ? a.D[c] : 0.f;
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
        const int r = q + k * Q;
        if (in && r < nb) {
            float v = fmaf(D, x[k], o[k]);
            if (a.z.p) v *= silu(z[k]);
            a.y.at(b0 + r, 0)[c] = from_f32<T>(v);
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
    launch_next();
    for (int i = threadIdx.x; i < s.n; i += 256) dst[s.first + i] = s.v[i];
}
cudaError_t place_offsets(const int64_t *cu, int64_t nseq, int *dst, Seqs &seqs, bool *launched, cudaStream_t st) {
    seqs.packed = 1;
    *launched = nseq + 1 > kInline;
    if (!*launched) {
        for (int64_t i = 0; i <= nseq; ++i) seqs.few[i] = (int)cu[i];
        return cudaSuccess;
    }
    seqs.start = dst;
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

int empty_blocks(const int64_t *cu, int64_t nseq) {
    int64_t n = 0;
    for (int64_t i = 0; i < nseq; ++i) n += cu[i] == cu[i + 1];
    return (int)(n == 0 ? 0 : nseq <= 64 ? nseq * 16 : 1024);
}

cudaError_t copy_states(const float *src, float *dst, int64_t count, cudaStream_t st) {
    return src ? cudaMemcpyAsync(dst, src, sizeof(float) * count, cudaMemcpyDeviceToDevice, st)
               : cudaMemsetAsync(dst, 0, sizeof(float) * count, st);
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

// How block rows (a channel block of a sequence row, one warp each) are cut.
// An SM has four warp schedulers and the kernel two warps for each (its
// registers: with 168 instead of 255 a third warp fits, but one warp's tokens
// overlap less: 1097 against 790 us at 8 x 4096 x 5120).  As many block rows
// as give every scheduler the same number run whole; the rest, which would
// set the time on a few schedulers, are cut into chunks that spread over all.
// With fewer than two a scheduler all are cut, in chunks of at least 64
// tokens.
constexpr int64_t kSched = 152 * 4;
struct FwdPlan {
    int chunk, nchunk;  // tokens per chunk, chunks of a block row that is cut
    int64_t whole, cut;
    size_t offsets, local, sums, bytes;  // workspace offsets
};
FwdPlan plan_fwd(const ssd_channel_shape_t *s, const int64_t *cu, int64_t nseq) {
    FwdPlan p{};
    const int64_t nblk = s->ngroups * ((s->channels / s->ngroups + 31) / 32);
    const int64_t L = s->seqlen, base = nblk * (cu ? 1 : s->batch);
    p.whole = cu || base < 2 * kSched ? 0 : base / kSched * kSched;
    p.cut = base - p.whole;
    // A tail of more than 7/8 of a warp for every scheduler, or behind eight of them, is not worth cutting
    // (11 x 2048 x 5120, 2.9 warps each: 626 us whole, 645 cut; 60 x 512 x 5120, 15.8: 748 and 776; on the
    // other side 8 x 4096 x 5120, 2.1: 1237 and 805).
    if (p.whole && (p.cut * 8 > kSched * 7 || base >= 8 * kSched)) p.whole = base, p.cut = 0;
    int64_t want = p.cut ? 2 * kSched / p.cut : 1;  // two for every scheduler, at most
    if (want > (L + 63) / 64) want = (L + 63) / 64;
    if (want < 1) want = 1;
    if (want == 1) p.whole = cu ? 0 : base, p.cut = base - p.whole;
    p.chunk = (int)(((L + want - 1) / want + kTB - 1) / kTB * kTB);
    if (p.chunk < kTB) p.chunk = kTB;
    p.nchunk = (int)((L + p.chunk - 1) / p.chunk);
    size_t at = 0;
    p.offsets = at;
    at += offsets_bytes(cu, nseq);
    p.local = at;
    if (p.nchunk > 1) at += align256(sizeof(float) * p.cut * p.nchunk * s->dstate * 32);
    p.sums = at;
    if (p.nchunk > 1) at += align256(sizeof(float) * p.cut * p.nchunk * 32);
    p.bytes = at;
    return p;
}

template <typename T, int N>
ssd_status_t run_fwd(ChannelArgs<T> &a, const ssd_channel_shape_t *s, const int64_t *cu, int64_t nseq, char *ws,
                     cudaStream_t st) {
    const FwdPlan p = plan_fwd(s, cu, nseq);
    timing_begin(st);
    cudaError_t e = cudaSuccess;
    if (s->seqlen == 0) return status_of(a.fin ? copy_states(a.init, a.fin, nseq * s->channels * s->dstate, st) : e);
    bool after = false;
    if (cu) e = place_offsets(cu, nseq, reinterpret_cast<int *>(ws + p.offsets), a.seqs, &after, st);
    if (e != cudaSuccess) return status_of(e);
    a.chunk = p.chunk, a.nchunk = p.nchunk;
    a.local = reinterpret_cast<float4 *>(ws + p.local);
    a.sums = reinterpret_cast<float *>(ws + p.sums);
    const int64_t cut = p.cut * p.nchunk;
    if (p.whole + cut > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
    a.whole = (int)p.whole, a.cut = (int)p.cut;
    a.blocks = (unsigned)((p.whole + cut + kWarps - 1) / kWarps);
    const unsigned blocks = a.blocks + (cu && a.fin ? empty_blocks(cu, nseq) : 0);
    if (p.cut && p.nchunk > 1) {
        e = launch(channel_fwd_kernel<T, N, false, false>, dim3((unsigned)((cut + kWarps - 1) / kWarps)), kWarps * 32, 0, st,
                   after, a);
        timing_mark(st, "channel_chunk_state");
        if (e != cudaSuccess) return status_of(e);
        after = true;
    }
    e = launch(a.z.p ? channel_fwd_kernel<T, N, true, true> : channel_fwd_kernel<T, N, true, false>, dim3(blocks),
               kWarps * 32, 0, st, after, a);
    timing_mark(st, "channel_scan");
    return status_of(e);
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
    const int64_t blocks = (s->channels * (s->dstate / 4) + 255) / 256, rows = (s->batch + kRows - 1) / kRows;
    if (blocks > 0x7FFFFFFF || rows > 65535) return SSD_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks, (unsigned)rows);
    const bool vec = rows_vec(in->B, sizeof(T), s->batch, 1) && rows_vec(in->C, sizeof(T), s->batch, 1);
    timing_begin(st);
    auto launch = [&](auto n) {
        constexpr int N = decltype(n)::value;
        if (vec)
            channel_step_kernel<T, N, true><<<grid, 256, 0, st>>>(a, state);
        else
            channel_step_kernel<T, N, false><<<grid, 256, 0, st>>>(a, state);
    };
    if (s->dstate == 8)
        launch(std::integral_constant<int, 8>{});
    else if (s->dstate == 16)
        launch(std::integral_constant<int, 16>{});
    else
        launch(std::integral_constant<int, 32>{});
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
    if (final_state && final_state == in->init_state) return SSD_ERR_INVALID_ARG;  // one is read while the other is written
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
