// ssd_gated.cu -- gated scan: prompts (equal and packed lengths) and single
// tokens.  The gradient is in ssd_gated_bwd.cu, the shared pieces and what a
// tile is in ssd_gated.cuh.
//
// What bounds the prompt's kernel: issue and waiting in turn.  A token and warp
// of 64 channels takes 89 instructions (8 of the special function unit a
// channel with a gate), issued in half of the cycles: with 128 registers for 16
// tokens' a and beta s(i) x there are four warps a scheduler, and a tile's two
// meetings with the links cost 2000 of its 13000 cycles.  The special function
// unit is active for 47% of the time.  4 x 4096 x 2560 bf16 with a gate 103 us,
// 50% of the DRAM rate; 8 tokens a warp in 32 warps an SM
// are as fast (less to wait for, twice the meetings), tiles of 64 tokens too.
#include "ssd_gated.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 8;  // of a tile; fewer where a row has fewer tokens
constexpr int kBlocks = 2;  // an SM
template <typename T>
constexpr int kTokens = 32 / sizeof(T);  // a warp: fp32 takes twice the shared memory

// The next tile's x, r and i, and two tiles' z: each lane's own.
template <typename T, int ALIGN>
struct Stage {
    static constexpr int S = kTokens<T>;
    Slot<T, ALIGN> in[3][S][kWarps], z[2][S][kWarps];
};

// What a warp knows of its tokens.
template <typename T, int ALIGN>
struct Warp {
    Lane<ALIGN> k;
    int tile, row, b, t0;
    // (A block's rows past the last one count as a tile behind it: no token is there.)
    __device__ __forceinline__ Warp(const GatedArgs<T> &a, int n, int in_block, int in_row, int lane, int tokens)
        : k(((n * a.per + in_block) % (a.nblk * a.batch)) % a.nblk, lane, a.ch) {
        const int rows = a.nblk * a.batch, q = n * a.per + in_block;
        tile = q / rows, row = q % rows, b = row / a.nblk, t0 = tile * tokens + in_row * kTokens<T>;
    }
};
template <typename T, int ALIGN>
__device__ __forceinline__ float2 init_of(const GatedArgs<T> &a, const Warp<T, ALIGN> &w, const Cuts &cut, int s) {
    return load_state(a.init ? a.init + (int64_t)seq_from(a.seqs, cut.seq, w.t0 + s) * a.ch : nullptr, w.k);
}

// Starts the copies of a tile's inputs.
template <typename T, int ALIGN, bool GATE>
__device__ __forceinline__ void fetch_tile(const GatedArgs<T> &a, const Warp<T, ALIGN> &w, Stage<T, ALIGN> &st, int warp, int lane, int zbuf) {
    // past the end, and in channels that are none: a = 1 and nothing enters
    const int left = a.seqs.L - w.t0;
    auto rows = [&](Slot<T, ALIGN> *dst, const Rows<const T> &r, float fill) {
        fetch_rows<T, ALIGN, kTokens<T>, kWarps>(dst, r, w.b, w.t0, w.k, lane, left, a.ch, fill);
    };
    rows(&st.in[1][0][warp], a.r, -30000.f);
    rows(&st.in[0][0][warp], a.x, 0.f);
    if (a.i.p) rows(&st.in[2][0][warp], a.i, 128.f);
    if (GATE) rows(&st.z[zbuf][0][warp], a.z, 0.f);
}

// The tokens' decays and inputs, and the run they make.  PLAIN: S tokens of one sequence that neither begins nor ends among
// them, decays with m <= 1.
template <typename T, int ALIGN, bool PACKED, bool PLAIN, int S>
__device__ __forceinline__ void run_tokens(const GatedArgs<T> &a, const Warp<T, ALIGN> &w, const Cuts &cut, f2 rate, const Stage<T, ALIGN> &st,
                                           int warp, int lane, f2 (&av)[S], f2 (&uv)[S], f2 &A, f2 &H) {
    A = splat(1.f), H = splat(0.f);
    const Skew<T, ALIGN> sx(a.x, w.b, w.t0), sr(a.r, w.b, w.t0), si(a.i, w.b, w.t0);
    auto in = [&](int which, int s, const Skew<T, ALIGN> &skew) { return widen(two_in(st.in[which][s][warp], lane, skew(s))); };
#pragma unroll
    for (int s = 0; s < S; ++s) {
        f2 v;
        decay2<PLAIN>(mul2(rate, both(sigmoid2(in(1, s, sr)))), v, av[s]);
        const float2 b2 = apart(fma2(v, av[s], v));
        uv[s] = mul2(mul2(pack2(sqrt_approx(b2.x), sqrt_approx(b2.y)), both(sigmoid2(in(2, s, si)))),
                     both(in(0, s, sx)));
        if (PACKED && !PLAIN && (cut.first >> s & 1)) H = both(init_of(a, w, cut, s));
        A = mul2(A, av[s]);
        H = fma2(av[s], H, uv[s]);
    }
    if (PACKED && !PLAIN && cut.first) A = splat(-1.f);
}

// The outputs, from the state that enters.
template <typename T, int ALIGN, bool GATE, bool PACKED, bool PLAIN, int S>
__device__ __forceinline__ void write_tokens(const GatedArgs<T> &a, const Warp<T, ALIGN> &w, const Cuts &cut, const Stage<T, ALIGN> &st, int warp,
                                             int lane, int zbuf, const f2 (&av)[S], const f2 (&uv)[S], f2 hv) {
    T *py = a.y.at(w.b, w.t0);
    const int L = a.seqs.L;
    const Skew<T, ALIGN> sz(a.z, w.b, w.t0);
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (!PLAIN && w.t0 + s >= L) break;
        if (PACKED && !PLAIN && (cut.first >> s & 1)) hv = both(init_of(a, w, cut, s));
        hv = fma2(av[s], hv, uv[s]);
        f2 o = hv;
        if constexpr (GATE) {
            const float2 zf = widen(two_in(st.z[zbuf][s][warp], lane, sz(s)));
            o = mul2(o, mul2(both(zf), both(sigmoid2(zf))));
        }
        store_two<T, ALIGN>(py + a.y.step(s), w.k, apart(o));
        if (!PLAIN && (cut.last >> s & 1) && a.fin) {
            const int q = PACKED ? seq_from(a.seqs, cut.seq, w.t0 + s) : w.b;
            store_state(a.fin + (int64_t)q * a.ch, w.k, apart(hv));
        }
    }
}

template <typename T, int ALIGN, bool GATE, bool PACKED>
__global__ void __launch_bounds__(kWarps * 32, kBlocks) gated_fwd_kernel(const __grid_constant__ GatedArgs<T> a) {
    constexpr int S = kTokens<T>;
    extern __shared__ __align__(16) uint8_t dynamic[];
    Stage<T, ALIGN> &st = *reinterpret_cast<Stage<T, ALIGN> *>(dynamic);
    __shared__ float4 runs[2][kWarps][32];
    __shared__ LinkShared sh;
    __shared__ unsigned ticket[2];
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32, nw = blockDim.x / 32, tokens = a.sub * S, L = a.seqs.L;
    const int in_block = uniform(warp / a.sub), in_row = warp - in_block * a.sub;  // this warp's row of the block's, its place in it
    const bool linked = a.links.run != nullptr;
    auto run_of = [](const float4 &v) { return Run{make_float2(v.x, v.y), make_float2(v.z, v.w)}; };
    auto next = [&](unsigned n) { return linked ? atomicAdd(a.links.ticket, 1u) + 1u : n + gridDim.x; };  // (it starts at -1)
    if (!a.i.p) {  // no input gate: s(128) = 1
#pragma unroll
        for (int s = 0; s < S; ++s) fill_slot(st.in[2][s][warp], lane, 128.f);
    }
    wait_previous();
    if (threadIdx.x == 0) ticket[1] = next(blockIdx.x - gridDim.x);
    __syncthreads();
    int n = uniform((int)ticket[1]);
    Warp<T, ALIGN> w(a, n, in_block, in_row, lane, tokens);
    float2 rate = make_float2(0.f, 0.f);
    Cuts cut{};
    auto cuts = [&](const Warp<T, ALIGN> &w) {
        Cuts c{0, 0, w.b};
        if (w.t0 < L) {
            if constexpr (PACKED)
                c = cuts_of<S>(a.seqs, w.t0);
            else if (w.t0 + S >= L)
                c.last = 1u << (L - 1 - w.t0);
        }
        return c;
    };
    if (n < a.tiles) {
        rate = rates_of(a, w.k);
        fetch_tile<T, ALIGN, GATE>(a, w, st, warp, lane, 0);
        cut = cuts(w);
    }
    for (int p = 0; n < a.tiles; p ^= 1) {
        const Lane<ALIGN> &k = w.k;
        if (threadIdx.x == 0) ticket[p] = next((unsigned)n);
        const bool plain = w.t0 + S <= L && !(cut.first | cut.last) && __all_sync(0xffffffffu, rate.x <= 1.f && rate.y <= 1.f);
        // The state that enters the row, or the group of tiles.
        float2 h = !PACKED && w.tile < kGroup ? load_state(a.init ? a.init + (int64_t)w.b * a.ch : nullptr, k) : make_float2(0.f, 0.f);

        const Place place(a.links, w.row, w.tile, linked ? a.ntile : 1, lane);
        copies_done();
        __syncwarp();
        f2 av[S], uv[S], A, H;
        if (plain)
            run_tokens<T, ALIGN, PACKED, true>(a, w, cut, both(rate), st, warp, lane, av, uv, A, H);
        else
            run_tokens<T, ALIGN, PACKED, false>(a, w, cut, both(rate), st, warp, lane, av, uv, A, H);
        const float2 fa = apart(A), fh = apart(H);
        runs[p][warp][lane] = make_float4(fa.x, fa.y, fh.x, fh.y);
        __syncthreads();
        Run all{};
        if (linked && warp == 0) {
            all = run_of(runs[p][0][lane]);
            for (int j = 1; j < nw; ++j) all = then(all, run_of(runs[p][j][lane]));
            place.publish(all);
        }
        n = uniform((int)ticket[p]);
        const Warp<T, ALIGN> after(a, n, in_block, in_row, lane, tokens);
        Cuts next_cut{};
        if (n < a.tiles) {
            rate = rates_of(a, after.k);
            fetch_tile<T, ALIGN, GATE>(a, after, st, warp, lane, p ^ 1);
            next_cut = cuts(after);  // (while others' runs are on their way)
        }

        if (linked) h = pass_links(place, a.links, sh, h, all, w.tile >= kGroup, warp, nw, lane);
        for (int j = warp - in_row; j < warp; ++j) h = through(run_of(runs[p][j][lane]), h);
        if (a.keep && w.t0 % kStateEvery == 0 && w.t0 < L)
            store_state(a.keep + ((int64_t)w.b * a.nkeep + w.t0 / kStateEvery) * a.ch, k, h);
        if (a.y.p) {
            if (plain)
                write_tokens<T, ALIGN, GATE, PACKED, true>(a, w, cut, st, warp, lane, p, av, uv, both(h));
            else
                write_tokens<T, ALIGN, GATE, PACKED, false>(a, w, cut, st, warp, lane, p, av, uv, both(h));
        }
        w = after, cut = next_cut;
    }
    if (PACKED && a.some_empty) pass_empty(a.seqs, a.ch, a.init, a.fin);
}

template <typename T, int ALIGN>
__global__ void __launch_bounds__(128) gated_step_kernel(const __grid_constant__ GatedArgs<T> a, float *state) {
    const int n = blockIdx.x * 4 + threadIdx.x / 32;
    const Lane<ALIGN> k(n % a.nblk, threadIdx.x % 32, a.ch);
    const int b = n / a.nblk;
    if (b >= a.batch) return;
    const Two<T> x = load_two<T, ALIGN>(a.x.at(b, 0), k, 0.f), r = load_two<T, ALIGN>(a.r.at(b, 0), k, 0.f);
    const Two<T> g = a.i.p ? load_two<T, ALIGN>(a.i.at(b, 0), k, 0.f) : two_of(T(), 128.f);
    const Two<T> z = a.z.p ? load_two<T, ALIGN>(a.z.at(b, 0), k, 0.f) : two_of(T(), 0.f);
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
    store_two<T, ALIGN>(a.y.at(b, 0), k, apart(o));
}

int64_t fwd_warps(const ssd_gated_shape_t *s) {
    const int64_t per = 32 / dtype_size(s->dtype), w = (s->seqlen + per - 1) / per;
    return w < kWarps ? (w < 1 ? 1 : w) : kWarps;
}
int64_t fwd_tokens(const ssd_gated_shape_t *s) { return 32 / dtype_size(s->dtype) * fwd_warps(s); }  // of a tile

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
Align gated_align(const ssd_gated_shape_t *s, const ssd_gated_inputs_t *in) {
    const size_t es = dtype_size(s->dtype);
    bool pairs = s->channels % 2 == 0, sixteen = s->channels * es % 16 == 0;
    for (const ssd_rows_t *r : {&in->x, &in->r, &in->i, &in->z})
        if (r->data) pairs = pairs && rows_pairs(*r, es, s->batch, s->seqlen), sixteen = sixteen && rows_vec(*r, es, s->batch, s->seqlen);
    return sixteen ? kSixteen : pairs ? kPairs : kElements;
}

template <typename T>
GatedArgs<T> gated_args(const ssd_gated_shape_t *s, const ssd_gated_inputs_t *in, int64_t nseq) {
    GatedArgs<T> a{};
    a.x = gated_rows<const T>(s, in->x), a.r = gated_rows<const T>(s, in->r);
    a.i = gated_rows<const T>(s, in->i), a.z = gated_rows<const T>(s, in->z);
    a.decay = in->decay, a.init = in->init_state, a.rate = s->rate;
    a.ch = (int)s->channels, a.nblk = (int)gated_blocks(s), a.batch = (int)s->batch, a.nkeep = (int)gated_kept(s);
    a.seqs.n = (int)nseq, a.seqs.L = (int)s->seqlen;
    return a;
}
template GatedArgs<float> gated_args<float>(const ssd_gated_shape_t *, const ssd_gated_inputs_t *, int64_t);
template GatedArgs<bf16> gated_args<bf16>(const ssd_gated_shape_t *, const ssd_gated_inputs_t *, int64_t);

namespace {
__global__ void __launch_bounds__(256) gated_prepare_kernel(uint4 *links, int64_t n, const float *decay, float rate, float *rates, int ch) {
    launch_next();
    const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t c = first; c < ch; c += step) rates[c] = decay_rate(decay[c], rate);
    for (int64_t i = first; i < n; i += step) links[i] = make_uint4(kUnset, kUnset, kUnset, kUnset);
}
}  // namespace

size_t links_bytes(int64_t ch, int64_t rows, int64_t ntile) {
    if (ntile <= 1) return 0;
    return align256(sizeof(float) * ch) + align256(8 * kCols * rows * (ntile + (ntile + kGroup - 1) / kGroup) + 256);
}
template <typename T>
cudaError_t prepare(GatedArgs<T> &a, char *ws, int64_t rows, int64_t ntile, cudaStream_t st) {
    a.links = Links{};
    a.rates = nullptr;
    if (ntile <= 1) return cudaSuccess;
    const cudaError_t e = device_status_word(&a.links.status);
    if (e != cudaSuccess) return e;
    a.rates = reinterpret_cast<float *>(ws);
    const size_t before = align256(sizeof(float) * a.ch), bytes = links_bytes(a.ch, rows, ntile) - before;
    ws += before;
    a.links.ticket = reinterpret_cast<unsigned *>(ws);
    a.links.run = reinterpret_cast<unsigned long long *>(ws + 256);
    a.links.entry = a.links.run + kCols * rows * ntile;
    const int64_t want = (int64_t)(bytes / 16 + 1023) / 1024 + a.ch / 256;
    gated_prepare_kernel<<<(unsigned)(want < 1 ? 1 : want < 4 * kSMs ? want : 4 * kSMs), 256, 0, st>>>(
        reinterpret_cast<uint4 *>(ws), (int64_t)(bytes / 16), a.decay, a.rate, a.rates, a.ch);
    timing_mark(st, "gated_prepare");
    return cudaGetLastError();
}
template cudaError_t prepare<float>(GatedArgs<float> &, char *, int64_t, int64_t, cudaStream_t);
template cudaError_t prepare<bf16>(GatedArgs<bf16> &, char *, int64_t, int64_t, cudaStream_t);

bool any_empty(const int64_t *cu, int64_t nseq) {
    for (int64_t s = 0; s < nseq; ++s)
        if (cu[s] == cu[s + 1]) return true;
    return false;
}

size_t gated_fwd_links(const ssd_gated_shape_t *s) {
    const int64_t per = fwd_tokens(s);
    return links_bytes(s->channels, gated_blocks(s) * s->batch, (s->seqlen + per - 1) / per);
}

template <typename T>
cudaError_t launch_gated_fwd(GatedArgs<T> &a, const ssd_gated_shape_t *s, Align align, bool packed, char *links, cudaStream_t st) {
    const int64_t tokens = fwd_tokens(s), ntile = (s->seqlen + tokens - 1) / tokens, rows = gated_blocks(s) * s->batch;
    a.ntile = (int)ntile;
    a.sub = (int)fwd_warps(s);
    a.per = rows_of_block(rows, ntile, a.sub, kWarps, kSMs * kBlocks);
    a.tiles = (int)(ntile * ((rows + a.per - 1) / a.per));
    cudaError_t e = prepare(a, links, rows, ntile, st);
    if (e != cudaSuccess) return e;
    const unsigned blocks = (unsigned)(a.tiles < kSMs * kBlocks ? a.tiles : kSMs * kBlocks), threads = (unsigned)(a.sub * a.per * 32);
    auto go = [&](auto p, auto g, auto c) {
        constexpr int kStage = (int)sizeof(Stage<T, decltype(p)::value>);
        auto kernel = gated_fwd_kernel<T, decltype(p)::value, decltype(g)::value, decltype(c)::value>;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStage);
        if (e == cudaSuccess) e = launch(kernel, dim3(blocks), (int)threads, kStage, st, a.rates != nullptr, a);
    };
    auto with_cuts = [&](auto p, auto g) { packed ? go(p, g, std::true_type{}) : go(p, g, std::false_type{}); };
    auto with_gate = [&](auto p) { a.z.p && a.y.p ? with_cuts(p, std::true_type{}) : with_cuts(p, std::false_type{}); };
    by_align(align, with_gate);
    timing_mark(st, a.y.p ? "gated_scan" : "gated_states");
    return e;
}
template cudaError_t launch_gated_fwd<float>(GatedArgs<float> &, const ssd_gated_shape_t *, Align, bool, char *, cudaStream_t);
template cudaError_t launch_gated_fwd<bf16>(GatedArgs<bf16> &, const ssd_gated_shape_t *, Align, bool, char *, cudaStream_t);

namespace {

template <typename T>
ssd_status_t fwd_typed(const ssd_gated_shape_t *s, const int64_t *cu, int64_t nseq, const ssd_gated_inputs_t *in,
                       const ssd_rows_t *y, float *fin, float *keep, char *ws, cudaStream_t st) {
    timing_begin(st);
    if (s->seqlen == 0)
        return status_of(fin ? copy_states(in->init_state, fin, nseq * s->channels, st) : cudaSuccess);
    GatedArgs<T> a = gated_args<T>(s, in, nseq);
    a.y = gated_rows<T>(s, *y);
    a.fin = fin, a.keep = keep;
    cudaError_t e = cudaSuccess;
    if (cu) {
        bool launched;
        e = place_offsets(cu, nseq, reinterpret_cast<int *>(ws), a.seqs, &launched, st);
        a.some_empty = fin && any_empty(cu, nseq);
        if (e != cudaSuccess) return status_of(e);
        ws += offsets_bytes(cu, nseq);
    }
    const Align align = rows_pairs(*y, sizeof(T), s->batch, s->seqlen) ? gated_align(s, in) : kElements;
    return status_of(launch_gated_fwd(a, s, align, cu != nullptr, ws, st));
}

template <typename T>
ssd_status_t step_typed(const ssd_gated_shape_t *s, const ssd_gated_inputs_t *in, float *state, const ssd_rows_t *y, cudaStream_t st) {
    GatedArgs<T> a = gated_args<T>(s, in, s->batch);
    a.y = gated_rows<T>(s, *y);
    timing_begin(st);
    const unsigned blocks = (unsigned)(((int64_t)a.nblk * a.batch + 3) / 4);
    if (gated_align(s, in) != kElements && rows_pairs(*y, sizeof(T), s->batch, 1))
        gated_step_kernel<T, kPairs><<<blocks, 128, 0, st>>>(a, state);
    else
        gated_step_kernel<T, kElements><<<blocks, 128, 0, st>>>(a, state);
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
