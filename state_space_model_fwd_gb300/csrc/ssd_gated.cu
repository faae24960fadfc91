// ssd_gated.cu -- gated scan: prompts (equal and packed lengths) and single
// tokens.  The gradient is in ssd_gated_bwd.cu, the shared pieces and what a
// tile is in ssd_gated.cuh.
#include "ssd_gated.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 8;  // of a tile; fewer where a row has fewer tokens
constexpr int S = 16;      // tokens a warp
constexpr int kBlocks = 2;  // an SM

// What a warp knows of its tokens.
template <typename T, bool PAIRS>
struct Warp {
    Lane<PAIRS> k;
    int b, t0, L;
    Cuts cut;
    f2 rate;
    __device__ __forceinline__ float2 init_of(const GatedArgs<T> &a, int s) const {
        return load_state(a.init ? a.init + (int64_t)seq_from(a.seqs, cut.seq, t0 + s) * a.ch : nullptr, k);
    }
};

// The tokens' decays and inputs, and the run they make.  PLAIN: S tokens of one sequence that neither begins nor ends among
// them, decays with m <= 1.
template <typename T, bool PAIRS, bool PACKED, bool PLAIN>
__device__ __forceinline__ void run_tokens(const GatedArgs<T> &a, const Warp<T, PAIRS> &w, f2 (&av)[S], f2 (&uv)[S], f2 &A, f2 &H) {
    Two<T> x[S], r[S], g[S];
    const T *px = a.x.at(w.b, w.t0), *pr = a.r.at(w.b, w.t0), *pi = a.i.p ? a.i.at(w.b, w.t0) : nullptr;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        // past the end, and in channels that are none: a = 1 and nothing enters
        r[s] = two_of(T(), -30000.f), x[s] = two_of(T(), 0.f), g[s] = two_of(T(), 128.f);
        if (PLAIN || w.t0 + s < w.L) {
            r[s] = load_two<T, PAIRS>(pr + a.r.step(s), w.k, -30000.f);
            x[s] = load_two<T, PAIRS>(px + a.x.step(s), w.k, 0.f);
            if (pi) g[s] = load_two<T, PAIRS>(pi + a.i.step(s), w.k, 128.f);  // without it s(i) = s(128) = 1
        }
    }
    A = splat(1.f), H = splat(0.f);
#pragma unroll
    for (int s = 0; s < S; ++s) {
        f2 v;
        decay2<PLAIN>(mul2(w.rate, both(sigmoid2(widen(r[s])))), v, av[s]);
        const float2 b2 = apart(fma2(v, av[s], v));
        const f2 beta = pack2(sqrt_approx(b2.x), sqrt_approx(b2.y));
        uv[s] = mul2(mul2(beta, both(sigmoid2(widen(g[s])))), both(widen(x[s])));
        if (PACKED && !PLAIN && (w.cut.first >> s & 1)) H = both(w.init_of(a, s));
        A = mul2(A, av[s]);
        H = fma2(av[s], H, uv[s]);
    }
    if (PACKED && !PLAIN && w.cut.first) A = splat(-1.f);
}

// The outputs, from the state that enters.
template <typename T, bool PAIRS, bool GATE, bool PACKED, bool PLAIN>
__device__ __forceinline__ void write_tokens(const GatedArgs<T> &a, const Warp<T, PAIRS> &w, const f2 (&av)[S], const f2 (&uv)[S],
                                             const Two<T> (&z)[S], f2 hv) {
    T *py = a.y.at(w.b, w.t0);
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (!PLAIN && w.t0 + s >= w.L) break;
        if (PACKED && !PLAIN && (w.cut.first >> s & 1)) hv = both(w.init_of(a, s));
        hv = fma2(av[s], hv, uv[s]);
        f2 o = hv;
        if constexpr (GATE) {
            const float2 zf = widen(z[s]);
            o = mul2(o, mul2(both(zf), both(sigmoid2(zf))));
        }
        store_two<T, PAIRS>(py + a.y.step(s), w.k, apart(o));
        if (!PLAIN && (w.cut.last >> s & 1) && a.fin) {
            const int q = PACKED ? seq_from(a.seqs, w.cut.seq, w.t0 + s) : w.b;
            store_state(a.fin + (int64_t)q * a.ch, w.k, apart(hv));
        }
    }
}

template <typename T, bool PAIRS, bool GATE, bool PACKED>
__global__ void __launch_bounds__(kWarps * 32, kBlocks) gated_fwd_kernel(const __grid_constant__ GatedArgs<T> a) {
    __shared__ float4 runs[kWarps][32];
    __shared__ float4 tiles[kGroup][32];
    __shared__ float2 enter[32];
    __shared__ unsigned ticket;
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32, nw = blockDim.x / 32;
    unsigned n = blockIdx.x;
    if (a.links.run) {
        if (threadIdx.x == 0) ticket = atomicAdd(a.links.ticket, 1u) + 1u;  // (it starts at -1)
        __syncthreads();
        n = (unsigned)uniform((int)ticket);
    }
    const int rows = a.nblk * a.batch, tile = n / rows, row = n % rows, b = row / a.nblk, L = a.seqs.L;
    Warp<T, PAIRS> w{Lane<PAIRS>(row % a.nblk, lane, a.ch), b, (tile * nw + warp) * S, L, Cuts{0, 0, b}, 0};
    const Lane<PAIRS> &k = w.k;
    if (w.t0 < L) {
        if constexpr (PACKED) {
            w.cut = cuts_of<S>(a.seqs, w.t0);
            w.cut.first = (unsigned)uniform((int)w.cut.first), w.cut.last = (unsigned)uniform((int)w.cut.last);
            w.cut.seq = uniform(w.cut.seq);
        } else if (w.t0 + S >= L) {
            w.cut.last = 1u << (L - 1 - w.t0);
        }
    }
    const float2 dec = load_state(a.decay, k);
    const float ra = decay_rate(dec.x, a.rate), rb = decay_rate(dec.y, a.rate);
    w.rate = pack2(ra, rb);
    const bool plain = w.t0 + S <= L && !(w.cut.first | w.cut.last) && __all_sync(0xffffffffu, (ra <= 1.f || !k.in0) && (rb <= 1.f || !k.in1));

    f2 av[S], uv[S], A, H;
    if (plain)
        run_tokens<T, PAIRS, PACKED, true>(a, w, av, uv, A, H);
    else
        run_tokens<T, PAIRS, PACKED, false>(a, w, av, uv, A, H);
    Two<T> z[S];  // (in flight while the tiles exchange their runs)
    if constexpr (GATE) {
        const T *pz = a.z.at(b, w.t0);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            z[s] = two_of(T(), 0.f);
            if (a.y.p && w.t0 + s < L) z[s] = load_two<T, PAIRS>(pz + a.z.step(s), k, 0.f);
        }
    }
    if (nw > 1) {
        const float2 fa = apart(A), fh = apart(H);
        runs[warp][lane] = make_float4(fa.x, fa.y, fh.x, fh.y);
        __syncthreads();
    }
    auto run_of = [](const float4 &v) { return Run{make_float2(v.x, v.y), make_float2(v.z, v.w)}; };

    // The state that enters the tile.
    float2 h = !PACKED ? load_state(a.init ? a.init + (int64_t)b * a.ch : nullptr, k) : make_float2(0.f, 0.f);
    if (a.links.run) {
        unsigned long long *mine = a.links.run + ((int64_t)row * a.ntile + tile) * kCols + lane;
        const int64_t groups = (a.ntile + kGroup - 1) / kGroup;
        unsigned long long *entry = a.links.entry + (int64_t)row * groups * kCols + lane;
        const int in_group = tile % kGroup, group = tile / kGroup;
        Run all{};
        if (warp == 0) {
            all = run_of(runs[0][lane]);
            for (int j = 1; j < nw; ++j) all = then(all, run_of(runs[j][lane]));
            if (in_group != kGroup - 1 && tile + 1 < a.ntile) link_store(mine, all);
        }
        for (int j = in_group - 1 - warp; j >= 0; j -= nw) {
            const Run q = link_wait(mine - (int64_t)(in_group - j) * kCols, a.links.status);
            tiles[j][lane] = make_float4(q.A.x, q.A.y, q.H.x, q.H.y);
        }
        if (warp == 0 && group > 0) h = link_wait(entry + (int64_t)group * kCols, a.links.status).H;
        __syncthreads();
        if (warp == 0) {
            for (int j = 0; j < in_group; ++j) h = through(run_of(tiles[j][lane]), h);
            if (in_group == kGroup - 1 && tile + 1 < a.ntile)
                link_store(entry + (int64_t)(group + 1) * kCols, Run{make_float2(0.f, 0.f), through(all, h)});
            enter[lane] = h;
        }
        __syncthreads();
        h = enter[lane];
    }
    for (int j = 0; j < warp; ++j) h = through(run_of(runs[j][lane]), h);
    if (a.keep && w.t0 % kStateEvery == 0 && w.t0 < L)
        store_state(a.keep + ((int64_t)b * a.nkeep + w.t0 / kStateEvery) * a.ch, k, h);
    if (!a.y.p) return;
    if (plain)
        write_tokens<T, PAIRS, GATE, PACKED, true>(a, w, av, uv, z, both(h));
    else
        write_tokens<T, PAIRS, GATE, PACKED, false>(a, w, av, uv, z, both(h));
}

__global__ void __launch_bounds__(256) gated_empty_kernel(const __grid_constant__ Seqs q, int64_t ch, const float *src, float *dst) {
    const int *start = q.offsets();
    for (int s = blockIdx.x; s < q.n; s += gridDim.x) {
        if (start[s] != start[s + 1]) continue;
        for (int64_t c = threadIdx.x; c < ch; c += 256) dst[s * ch + c] = src ? src[s * ch + c] : 0.f;
    }
}

template <typename T, bool PAIRS>
__global__ void __launch_bounds__(128) gated_step_kernel(const __grid_constant__ GatedArgs<T> a, float *state) {
    const int n = blockIdx.x * 4 + threadIdx.x / 32;
    const Lane<PAIRS> k(n % a.nblk, threadIdx.x % 32, a.ch);
    const int b = n / a.nblk;
    if (b >= a.batch) return;
    const Two<T> x = load_two<T, PAIRS>(a.x.at(b, 0), k, 0.f), r = load_two<T, PAIRS>(a.r.at(b, 0), k, 0.f);
    const Two<T> g = a.i.p ? load_two<T, PAIRS>(a.i.at(b, 0), k, 0.f) : two_of(T(), 128.f);
    const Two<T> z = a.z.p ? load_two<T, PAIRS>(a.z.at(b, 0), k, 0.f) : two_of(T(), 0.f);
    float *h = state + (int64_t)b * a.ch;
    const f2 old = both(load_state(h, k));
    const float2 dec = load_state(a.decay, k);
    f2 v, av;
    decay2<false>(mul2(pack2(decay_rate(dec.x, a.rate), decay_rate(dec.y, a.rate)), both(sigmoid2(widen(r)))), v, av);
    const float2 w = apart(fma2(v, av, v));
    const f2 u = mul2(mul2(pack2(sqrt_approx(w.x), sqrt_approx(w.y)), both(sigmoid2(widen(g)))), both(widen(x)));
    const f2 now = fma2(av, old, u);
    store_state(h, k, apart(now));
    f2 o = now;
    if (a.z.p) {
        const float2 zf = widen(z);
        o = mul2(o, mul2(both(zf), both(sigmoid2(zf))));
    }
    store_two<T, PAIRS>(a.y.at(b, 0), k, apart(o));
}

int64_t fwd_tokens(int64_t L) {  // of a tile
    const int64_t w = (L + S - 1) / S;
    return S * (w < kWarps ? (w < 1 ? 1 : w) : kWarps);
}

}  // namespace

ssd_status_t check_gated(const ssd_gated_shape_t *s, const int64_t *cu, int64_t nseq) {
    if (!s || s->batch < 0 || s->seqlen < 0 || s->channels <= 0 || !(s->rate > 0.f) || s->rate > 3e38f) return SSD_ERR_INVALID_ARG;
    if (s->dtype != SSD_DTYPE_F32 && s->dtype != SSD_DTYPE_BF16) return SSD_ERR_INVALID_ARG;
    if (s->channels > (1 << 24) || s->seqlen > kMaxTokens || s->batch > kMaxTokens || s->batch * s->seqlen > kMaxTokens)
        return SSD_ERR_UNSUPPORTED;
    if (cu && (s->batch != 1 || nseq > kMaxTokens || !offsets_ok(cu, nseq, s->seqlen))) return SSD_ERR_INVALID_ARG;
    // one block a tile: their number is counted in 31 bits
    const int64_t rows = gated_blocks(s) * (s->batch ? s->batch : 1);
    if (rows > 0x7FFFFFFF || rows * ((s->seqlen + 31) / 32 + 1) > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

bool gated_inputs_ok(const ssd_gated_shape_t *s, const ssd_gated_inputs_t *in, bool rows) {
    const size_t es = dtype_size(s->dtype);
    if (!in || !in->decay || !aligned(in->decay, 4) || !aligned(in->init_state, 4)) return false;
    if (!rows) return true;
    if ((in->i.data && !rows_in_ok(in->i, es)) || (in->z.data && !rows_in_ok(in->z, es))) return false;
    return rows_in_ok(in->x, es) && rows_in_ok(in->r, es);
}

bool rows_pairs(const ssd_rows_t &r, size_t esize, int64_t b, int64_t L) {
    return aligned(r.data, 2 * esize) && (b <= 1 || r.batch_stride % 2 == 0) && (L <= 1 || r.row_stride % 2 == 0);
}
bool gated_pairs(const ssd_gated_shape_t *s, const ssd_gated_inputs_t *in) {
    const size_t es = dtype_size(s->dtype);
    if (s->channels % 2) return false;
    for (const ssd_rows_t *r : {&in->x, &in->r, &in->i, &in->z})
        if (r->data && !rows_pairs(*r, es, s->batch, s->seqlen)) return false;
    return true;
}

template <typename T>
GatedArgs<T> gated_args(const ssd_gated_shape_t *s, const ssd_gated_inputs_t *in, int64_t nseq) {
    GatedArgs<T> a{};
    a.x = rows_of<const T>(in->x), a.r = rows_of<const T>(in->r), a.i = rows_of<const T>(in->i), a.z = rows_of<const T>(in->z);
    a.decay = in->decay, a.init = in->init_state, a.rate = s->rate;
    a.ch = (int)s->channels, a.nblk = (int)gated_blocks(s), a.batch = (int)s->batch, a.nkeep = (int)gated_kept(s);
    a.seqs.n = (int)nseq, a.seqs.L = (int)s->seqlen;
    return a;
}
template GatedArgs<float> gated_args<float>(const ssd_gated_shape_t *, const ssd_gated_inputs_t *, int64_t);
template GatedArgs<bf16> gated_args<bf16>(const ssd_gated_shape_t *, const ssd_gated_inputs_t *, int64_t);

size_t links_bytes(int64_t rows, int64_t ntile) {
    if (ntile <= 1) return 0;
    return align256(8 * kCols * rows * (ntile + (ntile + kGroup - 1) / kGroup) + 256);
}
cudaError_t place_links(char *ws, int64_t rows, int64_t ntile, Links &l, cudaStream_t st) {
    l = Links{};
    const size_t bytes = links_bytes(rows, ntile);
    if (!bytes) return cudaSuccess;
    cudaError_t e = device_status_word(&l.status);
    if (e != cudaSuccess) return e;
    l.ticket = reinterpret_cast<unsigned *>(ws);
    l.run = reinterpret_cast<unsigned long long *>(ws + 256);
    l.entry = l.run + kCols * rows * ntile;
    e = cudaMemsetAsync(ws, 0xFF, bytes, st);
    timing_mark(st, "gated_links");
    return e;
}

cudaError_t launch_empty(const Seqs &q, const int64_t *cu, int64_t nseq, int64_t ch, const float *src, float *dst, cudaStream_t st) {
    bool any = false;
    for (int64_t s = 0; s < nseq && !any; ++s) any = cu[s] == cu[s + 1];
    if (!any) return cudaSuccess;
    gated_empty_kernel<<<(unsigned)(nseq < 1024 ? nseq : 1024), 256, 0, st>>>(q, ch, src, dst);
    timing_mark(st, "gated_empty");
    return cudaGetLastError();
}

size_t gated_fwd_links(const ssd_gated_shape_t *s) {
    const int64_t per = fwd_tokens(s->seqlen);
    return links_bytes(gated_blocks(s) * s->batch, (s->seqlen + per - 1) / per);
}

template <typename T>
cudaError_t launch_gated_fwd(GatedArgs<T> &a, const ssd_gated_shape_t *s, bool pairs, bool packed, char *links, cudaStream_t st) {
    const int64_t per = fwd_tokens(s->seqlen), ntile = (s->seqlen + per - 1) / per;
    a.ntile = (int)ntile;
    cudaError_t e = place_links(links, gated_blocks(s) * s->batch, ntile, a.links, st);
    if (e != cudaSuccess) return e;
    const unsigned blocks = (unsigned)(ntile * a.nblk * a.batch), threads = (unsigned)(per / S * 32);
    auto go = [&](auto p, auto g, auto c) {
        gated_fwd_kernel<T, decltype(p)::value, decltype(g)::value, decltype(c)::value><<<blocks, threads, 0, st>>>(a);
    };
    auto with_cuts = [&](auto p, auto g) { packed ? go(p, g, std::true_type{}) : go(p, g, std::false_type{}); };
    auto with_gate = [&](auto p) { a.z.p && a.y.p ? with_cuts(p, std::true_type{}) : with_cuts(p, std::false_type{}); };
    pairs ? with_gate(std::true_type{}) : with_gate(std::false_type{});
    timing_mark(st, a.y.p ? "gated_scan" : "gated_states");
    return cudaGetLastError();
}
template cudaError_t launch_gated_fwd<float>(GatedArgs<float> &, const ssd_gated_shape_t *, bool, bool, char *, cudaStream_t);
template cudaError_t launch_gated_fwd<bf16>(GatedArgs<bf16> &, const ssd_gated_shape_t *, bool, bool, char *, cudaStream_t);

namespace {

template <typename T>
ssd_status_t fwd_typed(const ssd_gated_shape_t *s, const int64_t *cu, int64_t nseq, const ssd_gated_inputs_t *in,
                       const ssd_rows_t *y, float *fin, float *keep, char *ws, cudaStream_t st) {
    timing_begin(st);
    if (s->seqlen == 0)
        return status_of(fin ? copy_states(in->init_state, fin, nseq * s->channels, st) : cudaSuccess);
    GatedArgs<T> a = gated_args<T>(s, in, nseq);
    a.y = rows_of<T>(*y);
    a.fin = fin, a.keep = keep;
    cudaError_t e = cudaSuccess;
    if (cu) {
        bool launched;
        e = place_offsets(cu, nseq, reinterpret_cast<int *>(ws), a.seqs, &launched, st);
        if (e == cudaSuccess && fin) e = launch_empty(a.seqs, cu, nseq, s->channels, a.init, fin, st);
        if (e != cudaSuccess) return status_of(e);
        ws += offsets_bytes(cu, nseq);
    }
    return status_of(launch_gated_fwd(a, s, gated_pairs(s, in) && rows_pairs(*y, sizeof(T), s->batch, s->seqlen), cu != nullptr, ws, st));
}

template <typename T>
ssd_status_t step_typed(const ssd_gated_shape_t *s, const ssd_gated_inputs_t *in, float *state, const ssd_rows_t *y, cudaStream_t st) {
    GatedArgs<T> a = gated_args<T>(s, in, s->batch);
    a.y = rows_of<T>(*y);
    timing_begin(st);
    const unsigned blocks = (unsigned)(((int64_t)a.nblk * a.batch + 3) / 4);
    if (gated_pairs(s, in) && rows_pairs(*y, sizeof(T), s->batch, 1))
        gated_step_kernel<T, true><<<blocks, 128, 0, st>>>(a, state);
    else
        gated_step_kernel<T, false><<<blocks, 128, 0, st>>>(a, state);
    timing_mark(st, "gated_step");
    return status_of(cudaGetLastError());
}

}  // namespace
}  // namespace ssd

extern "C" {

int64_t ssd_gated_scan_chunk_states(const ssd_gated_shape_t *shape) {
    return ssd::check_gated(shape, nullptr, 0) == SSD_OK ? ssd::gated_kept(shape) : 0;
}

size_t ssd_gated_scan_workspace_size(const ssd_gated_shape_t *shape, const int64_t *cu_seqlens, int64_t nseq) {
    using namespace ssd;
    if (check_gated(shape, cu_seqlens, nseq) != SSD_OK || shape->batch == 0 || shape->seqlen == 0) return 0;
    return (cu_seqlens ? offsets_bytes(cu_seqlens, nseq) : 0) + gated_fwd_links(shape);
}

ssd_status_t ssd_gated_scan_fwd(const ssd_gated_shape_t *shape, const int64_t *cu_seqlens, int64_t nseq,
                                const ssd_gated_inputs_t *in, const ssd_rows_t *y, float *final_state, float *chunk_states,
                                void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace ssd;
    const ssd_status_t st = check_gated(shape, cu_seqlens, nseq);
    if (st != SSD_OK) return st;
    if (!cu_seqlens) nseq = shape->batch;
    if (nseq == 0) return SSD_OK;
    const bool rows = shape->seqlen > 0;
    if (!gated_inputs_ok(shape, in, rows) || !y || !aligned(final_state, 4) || !aligned(chunk_states, 4)) return SSD_ERR_INVALID_ARG;
    if (final_state && final_state == in->init_state) return SSD_ERR_INVALID_ARG;  // one is read while the other is written
    if (rows && !rows_out_ok(*y, dtype_size(shape->dtype), shape->batch, shape->seqlen, shape->channels)) return SSD_ERR_INVALID_ARG;
    const size_t need = ssd_gated_scan_workspace_size(shape, cu_seqlens, nseq);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return SSD_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    return shape->dtype == SSD_DTYPE_BF16 ? fwd_typed<bf16>(shape, cu_seqlens, nseq, in, y, final_state, chunk_states, ws, stream)
                                          : fwd_typed<float>(shape, cu_seqlens, nseq, in, y, final_state, chunk_states, ws, stream);
}

ssd_status_t ssd_gated_scan_step(const ssd_gated_shape_t *shape, const ssd_gated_inputs_t *in, float *state, const ssd_rows_t *y,
                                 cudaStream_t stream) {
    using namespace ssd;
    if (!shape) return SSD_ERR_INVALID_ARG;
    ssd_gated_shape_t one = *shape;
    one.seqlen = 1;
    const ssd_status_t st = check_gated(&one, nullptr, 0);
    if (st != SSD_OK) return st;
    if (one.batch == 0) return SSD_OK;
    if (!gated_inputs_ok(&one, in, true) || !y || !state || !aligned(state, 4)) return SSD_ERR_INVALID_ARG;
    if (!rows_out_ok(*y, dtype_size(one.dtype), one.batch, 1, one.channels)) return SSD_ERR_INVALID_ARG;
    return one.dtype == SSD_DTYPE_BF16 ? step_typed<bf16>(&one, in, state, y, stream) : step_typed<float>(&one, in, state, y, stream);
}

}  // extern "C"
