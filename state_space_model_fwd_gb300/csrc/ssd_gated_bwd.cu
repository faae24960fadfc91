// ssd_gated_bwd.cu -- gradient of the gated scan.
//
// With g_t the gradient of h_t and d_t = dy_t silu(z_t):
//   g_t = d_t + a_{t+1} g_{t+1}
//   dx = g beta s(i),  di = g beta x s(i) (1 - s(i)),  dz = dy h silu'(z)
//   dl = g (a h_{t-1} - s(i) x a^2 / beta),  dr = dl l (1 - s(r)),
//   ddecay = softplus'/softplus sum_t dl l       (l = log a)
// l / beta goes to zero with l, so dl l is formed as one: no division by beta.
//
// A block is a tile as in the forward kernel, later tokens first: the state
// that enters comes from those kept every 64 tokens, what comes back from
// later tokens (c_t = a_t g_t, so c -> P c + Q over a run of tokens) through
// the links.  Everything is read once and written once.
//
// What bounds it: issue and waiting in turn, 211 instructions a token and warp
// in half of the cycles, with 15 registers a token kept between the passes (4 x
// 4096 x 2560 bf16 with a gate 226 us, 40% of the DRAM rate, the special
// function unit active for 29%).  16 warps of 4
// tokens or of 8 are slower (8 x 4096 x 2560: 606 and 559 us against 471 at the
// time), and so is keeping beta s(i) x instead of forming it again (477);
// leaving x in shared memory instead of registers gives 0.5%.
#include "ssd_gated.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 8;
constexpr int S = 8;        // tokens a warp
constexpr int kBlocks = 2;  // an SM
constexpr int kTile = kWarps * S;
static_assert(kTile % kStateEvery == 0, "a tile starts at a kept state");

// The next tile's x, r, i, dy and z: each lane's own.
template <typename T, int ALIGN>
struct Stage {
    Slot<T, ALIGN> in[5][S][kWarps];
};

template <typename T, int ALIGN>
struct Warp {
    Lane<ALIGN> k;
    int later, tile, row, b, t0;  // later: tiles behind this one
    __device__ __forceinline__ Warp(const GatedArgs<T> &a, int n, int in_block, int in_row, int lane, int tokens)
        : k(((n * a.per + in_block) % (a.nblk * a.batch)) % a.nblk, lane, a.ch) {
        const int rows = a.nblk * a.batch, q = n * a.per + in_block;
        later = q / rows, tile = max(a.ntile - 1 - later, 0), row = q % rows, b = row / a.nblk, t0 = tile * tokens + in_row * S;
        if (later >= a.ntile) t0 = a.seqs.L;  // a block's row past the last one: no token is there
    }
};
template <typename T, int ALIGN>
__device__ __forceinline__ f2 state_of(const GatedArgs<T> &a, const Warp<T, ALIGN> &w, const Cuts &cut, const float *states, int s) {
    return both(load_state(states ? states + (int64_t)seq_from(a.seqs, cut.seq, w.t0 + s) * a.ch : nullptr, w.k));
}

// Starts the copies of a tile's inputs.
template <typename T, int ALIGN, bool GATE>
__device__ __forceinline__ void fetch_tile(const GatedArgs<T> &a, const Warp<T, ALIGN> &w, Stage<T, ALIGN> &st, int warp, int lane) {
    const int left = a.seqs.L - w.t0;
    auto rows = [&](int which, const Rows<const T> &r, float fill) {
        fetch_rows<T, ALIGN, S, kWarps>(&st.in[which][0][warp], r, w.b, w.t0, w.k, lane, left, a.ch, fill);
    };
    rows(1, a.r, -30000.f);
    rows(0, a.x, 0.f);
    if (a.i.p) rows(2, a.i, 128.f);
    rows(3, a.dy, 0.f);
    if (GATE) rows(4, a.z, 0.f);
}

// What is kept of a token between the passes, two channels each: the gates, the decay, x, the gradient of h_t by its own
// output, and dy times the slope of the output's gate.
template <typename T>
struct Kept {
    f2 sr, si, w, d, e;
    Two<T> x;
};
__device__ __forceinline__ f2 one_minus(f2 v) { return fma2(v, splat(-1.f), splat(1.f)); }
// The decay in one register: v = 1 - a, or -a where v is above a half and 1 - v would have lost a's digits (6% of it at
// a = e^-14).  The sign bit says which, as a may be 0.  (8 x 4096 x 2560 bf16 whose warps all hold some such channel: this kernel
// 517 us for 502; a formed again from m wherever it is needed takes twice the spills.)
struct Decay {
    f2 v, a;
};
template <bool PLAIN>
__device__ __forceinline__ f2 kept_decay(f2 v, f2 a) {
    if constexpr (PLAIN) return v;
    const float2 vv = apart(v), aa = apart(a);
    return pack2(vv.x > 0.5f ? -aa.x : vv.x, vv.y > 0.5f ? -aa.y : vv.y);
}
template <bool PLAIN>
__device__ __forceinline__ Decay decay_of(f2 w) {
    if constexpr (PLAIN) return {w, one_minus(w)};
    const float2 f = apart(w);
    const f2 p = pack2(fabsf(f.x), fabsf(f.y));
    const float2 g = apart(p), o = apart(one_minus(p));
    const bool x = signbit(f.x), y = signbit(f.y);
    return {pack2(x ? o.x : g.x, y ? o.y : g.y), pack2(x ? g.x : o.x, y ? g.y : o.y)};
}
__device__ __forceinline__ f2 input_of(const Decay &q, f2 si, f2 x) {  // beta s(i) x
    const float2 b2 = apart(fma2(q.v, q.a, q.v));
    return mul2(mul2(pack2(sqrt_approx(b2.x), sqrt_approx(b2.y)), si), x);
}

// PLAIN as in the forward kernel, and every channel of the block exists.
template <typename T, int ALIGN, bool GATE, bool PACKED, bool PLAIN>
__device__ __forceinline__ void read_tokens(const GatedArgs<T> &a, const Warp<T, ALIGN> &w, const Cuts &cut, f2 rate, const Stage<T, ALIGN> &st,
                                            int warp, int lane, Kept<T> (&t)[S], f2 &A, f2 &H, f2 &Q) {
    A = splat(1.f), H = splat(0.f), Q = splat(0.f);
    const Skew<T, ALIGN> sx(a.x, w.b, w.t0), sr(a.r, w.b, w.t0), si(a.i, w.b, w.t0), sdy(a.dy, w.b, w.t0), sz(a.z, w.b, w.t0);
    auto in = [&](int which, int s, const Skew<T, ALIGN> &skew) { return two_in(st.in[which][s][warp], lane, skew(s)); };
#pragma unroll
    for (int s = 0; s < S; ++s) {
        t[s].x = in(0, s, sx);
        t[s].sr = both(sigmoid2(widen(in(1, s, sr))));
        t[s].si = both(sigmoid2(widen(in(2, s, si))));
        Decay q;
        decay2<PLAIN>(mul2(rate, t[s].sr), q.v, q.a);
        t[s].w = kept_decay<PLAIN>(q.v, q.a);
        if (PACKED && !PLAIN && (cut.first >> s & 1)) H = state_of(a, w, cut, a.init, s);
        A = mul2(A, q.a);
        H = fma2(q.a, H, input_of(q, t[s].si, both(widen(t[s].x))));
        t[s].d = both(widen(in(3, s, sdy)));
        t[s].e = splat(0.f);
        if constexpr (GATE) {
            // silu(z) = z s, its slope s + z s (1 - s)
            const float2 z = widen(in(4, s, sz));
            const f2 zf = both(z), open = both(sigmoid2(z)), gate = mul2(zf, open);
            t[s].e = mul2(t[s].d, fma2(gate, one_minus(open), open));
            t[s].d = mul2(t[s].d, gate);
        }
    }
#pragma unroll
    for (int s = S - 1; s >= 0; --s) {
        if (PACKED && !PLAIN && (cut.last >> s & 1)) Q = state_of(a, w, cut, a.dfinal, s);
        Q = mul2(decay_of<PLAIN>(t[s].w).a, add2(t[s].d, Q));
    }
}

// h: the state that enters; c: what comes back from later tokens, and on return what goes back to earlier ones.
template <typename T, int ALIGN, bool GATE, bool PACKED, bool PLAIN>
__device__ __forceinline__ void write_tokens(const GatedArgs<T> &a, const Warp<T, ALIGN> &w, const Cuts &cut, f2 rate, Kept<T> (&t)[S], f2 h,
                                             f2 &c, f2 &sum) {
    const int L = a.seqs.L;
    // Stores without a condition each: forward and gradient of 8 x 4096 x 2560 bf16 643 us for 668.  (Without a gate it costs
    // registers that are spilled: 566 us, 547 so.)
    constexpr bool ALL = PLAIN && GATE;
    f2 prev[S];
    T *pz = GATE ? a.dz.at(w.b, w.t0) : nullptr;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (PACKED && !PLAIN && (cut.first >> s & 1)) h = state_of(a, w, cut, a.init, s);
        prev[s] = h;
        const Decay q = decay_of<PLAIN>(t[s].w);
        h = fma2(q.a, h, input_of(q, t[s].si, both(widen(t[s].x))));
        if (GATE && (PLAIN || w.t0 + s < L)) store_two<T, ALIGN, ALL>(pz + a.dz.step(s), w.k, apart(mul2(t[s].e, h)));
    }
    T *px = a.dx.at(w.b, w.t0), *pr = a.dr.at(w.b, w.t0), *pi = a.i.p ? a.di.at(w.b, w.t0) : nullptr;
    sum = splat(0.f);
#pragma unroll
    for (int s = S - 1; s >= 0; --s) {
        if (PACKED && !PLAIN && (cut.last >> s & 1)) c = state_of(a, w, cut, a.dfinal, s);
        const Decay q = decay_of<PLAIN>(t[s].w);
        const f2 av = q.a, gh = add2(t[s].d, c), xf = both(widen(t[s].x)), m = mul2(rate, t[s].sr);
        const float2 b2 = apart(fma2(q.v, av, q.v));
        const f2 rb = pack2(rsqrt_approx(fmaxf(b2.x, 1e-37f)), rsqrt_approx(fmaxf(b2.y, 1e-37f))), beta = mul2(both(b2), rb);
        c = mul2(gh, av);
        // dl l = g a (s(i) x a m / beta - m h_{t-1}),  l = -m
        const f2 sx = mul2(t[s].si, xf);
        const f2 dll = mul2(mul2(c, m), fma2(mul2(sx, av), rb, mul2(prev[s], splat(-1.f))));
        sum = add2(sum, dll);
        if (PACKED && !PLAIN && (cut.first >> s & 1) && a.dinit)
            store_state(a.dinit + (int64_t)seq_from(a.seqs, cut.seq, w.t0 + s) * a.ch, w.k, apart(c));
        if (PLAIN || w.t0 + s < L) {
            const f2 gx = mul2(mul2(gh, beta), t[s].si);
            store_two<T, ALIGN, ALL>(px + a.dx.step(s), w.k, apart(gx));
            store_two<T, ALIGN, ALL>(pr + a.dr.step(s), w.k, apart(mul2(dll, one_minus(t[s].sr))));
            if (pi) store_two<T, ALIGN, ALL>(pi + a.di.step(s), w.k, apart(mul2(mul2(gx, xf), one_minus(t[s].si))));
        }
    }
}

template <typename T, int ALIGN, bool GATE, bool PACKED>
__global__ void __launch_bounds__(kWarps * 32, kBlocks) gated_bwd_kernel(const __grid_constant__ GatedArgs<T> a) {
    extern __shared__ __align__(16) uint8_t dynamic[];
    Stage<T, ALIGN> &st = *reinterpret_cast<Stage<T, ALIGN> *>(dynamic);
    __shared__ float4 fore[2][kWarps][32], back[2][kWarps][32];
    __shared__ LinkShared sh;
    __shared__ float2 sums[2][kWarps - 1][32];
    __shared__ unsigned ticket[2];
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32, nw = blockDim.x / 32, tokens = a.sub * S, L = a.seqs.L;
    const int in_block = uniform(warp / a.sub), in_row = warp - in_block * a.sub, own = warp - in_row;  // (own: the row's first)
    const bool linked = a.links.run != nullptr;
    auto next = [&](unsigned n) { return linked ? atomicAdd(a.links.ticket, 1u) + 1u : n + gridDim.x; };
    auto run_of = [](const float4 &v) { return Run{make_float2(v.x, v.y), make_float2(v.z, v.w)}; };
    if (!a.i.p) {  // no input gate: s(128) = 1
#pragma unroll
        for (int s = 0; s < S; ++s) fill_slot(st.in[2][s][warp], lane, 128.f);
    }
    wait_previous();
    if (threadIdx.x == 0) ticket[1] = next(blockIdx.x - gridDim.x);
    __syncthreads();
    int n = uniform((int)ticket[1]);
    Warp<T, ALIGN> w(a, n, in_block, in_row, lane, tokens);
    auto entering = [&](const Warp<T, ALIGN> &w) {
        return load_state(a.kept + ((int64_t)w.b * a.nkeep + w.tile * (kTile / kStateEvery)) * a.ch, w.k);
    };
    float2 rate = make_float2(0.f, 0.f), kept = rate;
    Cuts cut{0, 0, w.b};
    if (n < a.tiles) {
        rate = rates_of(a, w.k), kept = entering(w);
        fetch_tile<T, ALIGN, GATE>(a, w, st, warp, lane);
        if (PACKED && w.t0 < L) cut = cuts_of<S>(a.seqs, w.t0);
    }
    for (int p = 0; n < a.tiles; p ^= 1) {
        const Lane<ALIGN> &k = w.k;
        if (threadIdx.x == 0) ticket[p] = next((unsigned)n);
        float2 h = kept;
        const f2 rates = both(rate);
        // What comes back from behind the row, or the group of tiles.
        float2 c = !PACKED && w.later < kGroup ? load_state(a.dfinal ? a.dfinal + (int64_t)w.b * a.ch : nullptr, k) : make_float2(0.f, 0.f);
        const bool plain = w.t0 + S <= L && !(cut.first | cut.last) && __all_sync(0xffffffffu, k.in1 && rate.x <= 1.f && rate.y <= 1.f);

        copies_done();
        __syncwarp();
        Kept<T> t[S];
        f2 A, H, Q;
        if (plain)
            read_tokens<T, ALIGN, GATE, PACKED, true>(a, w, cut, rates, st, warp, lane, t, A, H, Q);
        else
            read_tokens<T, ALIGN, GATE, PACKED, false>(a, w, cut, rates, st, warp, lane, t, A, H, Q);
        {
            const float2 fa = apart(A), fh = apart(H), fq = apart(Q);
            fore[p][warp][lane] = cut.first ? make_float4(-1.f, -1.f, fh.x, fh.y) : make_float4(fa.x, fa.y, fh.x, fh.y);
            back[p][warp][lane] = cut.last ? make_float4(-1.f, -1.f, fq.x, fq.y) : make_float4(fa.x, fa.y, fq.x, fq.y);
        }
        __syncthreads();
        Run all{};
        if (linked && warp == 0) {
            all = run_of(back[p][nw - 1][lane]);
            for (int j = nw - 2; j >= 0; --j) all = then(all, run_of(back[p][j][lane]));
            Place(a.links, w.row, w.later, a.ntile, lane).publish(all);
        }
        n = uniform((int)ticket[p]);
        const Warp<T, ALIGN> after(a, n, in_block, in_row, lane, tokens);
        Cuts next_cut{0, 0, after.b};
        if (n < a.tiles) {
            rate = rates_of(a, after.k), kept = entering(after);
            fetch_tile<T, ALIGN, GATE>(a, after, st, warp, lane);
            if (PACKED && after.t0 < L) next_cut = cuts_of<S>(a.seqs, after.t0);
        }

        if (linked)
            c = pass_links(Place(a.links, w.row, w.later, a.ntile, lane), a.links, sh, c, all, w.later >= kGroup, warp, nw, lane);
        for (int j = own + a.sub - 1; j > warp; --j) c = through(run_of(back[p][j][lane]), c);
        for (int j = own; j < warp; ++j) h = through(run_of(fore[p][j][lane]), h);

        f2 cv = both(c), sum;
        if (plain)
            write_tokens<T, ALIGN, GATE, PACKED, true>(a, w, cut, rates, t, both(h), cv, sum);
        else
            write_tokens<T, ALIGN, GATE, PACKED, false>(a, w, cut, rates, t, both(h), cv, sum);
        if (!PACKED && w.t0 == 0 && a.dinit) store_state(a.dinit + (int64_t)w.b * a.ch, k, apart(cv));
        if (a.ddecay_part) {
            if (warp != own) sums[p][warp - 1][lane] = apart(sum);
            __syncthreads();
            if (warp == own && w.t0 < L) {
                float2 s = apart(sum);
                for (int j = own; j < own + a.sub - 1; ++j) s.x += sums[p][j][lane].x, s.y += sums[p][j][lane].y;
                store_state(a.ddecay_part + ((int64_t)w.tile * a.batch + w.b) * a.ch, k, s);
            }
        }
        w = after, cut = next_cut;
    }
    if (PACKED && a.some_empty) pass_empty(a.seqs, a.ch, a.dfinal, a.dinit);
}

// ddecay[c] = softplus'(decay) / softplus(decay) sum over the tiles' parts, in a fixed order.  The quotient's limit for
// decay -> -inf is 1.
__global__ void __launch_bounds__(1024) gated_ddecay_kernel(const float *part, int64_t n, int64_t ch, const float *decay, float *out) {
    __shared__ float sums[32][33];
    launch_next();
    wait_previous();
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < ch) {
        int64_t t = w;
        for (; t + 96 < n; t += 128) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += part[(t + 32 * j) * ch + c];
        }
        for (; t < n; t += 32) v[0] += part[t * ch + c];
    }
    sums[w][lane] = (v[0] + v[1]) + (v[2] + v[3]);
    __syncthreads();
    if (w == 0 && c < ch) {
        float s = 0.f;
        for (int j = 0; j < 32; ++j) s += sums[j][lane];
        const float d = decay[c], sp = fmaxf(d, 0.f) + log1pf(expf(-fabsf(d)));
        out[c] = s * (d < -15.f ? 1.f : 1.f / (1.f + expf(-d)) / sp);
    }
}

int64_t bwd_warps(int64_t L) {
    const int64_t w = (L + S - 1) / S;
    return w < 1 ? 1 : w < kWarps ? w : kWarps;
}

int64_t bwd_tiles(int64_t L) { return (L + kTile - 1) / kTile; }

struct BwdPlan {
    size_t kept, fwd_links, links, part, bytes;
};
BwdPlan plan_bwd(const ssd_gated_shape_t *s, const int64_t *cu, int64_t nseq, bool with_states) {
    BwdPlan p{};
    const int64_t rows = gated_blocks(s) * s->batch, ntile = bwd_tiles(s->seqlen);
    size_t at = cu ? offsets_bytes(cu, nseq) : 0;
    p.kept = at;
    if (!with_states) at += align256(sizeof(float) * s->batch * gated_kept(s) * s->channels);
    p.fwd_links = at;
    if (!with_states) at += gated_fwd_links(s);
    p.links = at;
    at += links_bytes(s->channels, rows, ntile);
    p.part = at;
    at += align256(sizeof(float) * ntile * s->batch * s->channels);
    p.bytes = at;
    return p;
}

template <typename T>
ssd_status_t bwd_typed(const ssd_gated_shape_t *s, const int64_t *cu, int64_t nseq, const ssd_rows_t *dy,
                       const ssd_gated_inputs_t *in, const float *dfinal, const float *kept, const ssd_gated_grads_t *out,
                       char *ws, cudaStream_t st) {
    timing_begin(st);
    cudaError_t e = cudaSuccess;
    if (s->seqlen == 0) {
        if (out->dinit_state) e = copy_states(dfinal, out->dinit_state, nseq * s->channels, st);
        if (e == cudaSuccess && out->ddecay) e = cudaMemsetAsync(out->ddecay, 0, sizeof(float) * s->channels, st);
        return status_of(e);
    }
    const BwdPlan p = plan_bwd(s, cu, nseq, kept != nullptr);
    GatedArgs<T> a = gated_args<T>(s, in, nseq);
    if (cu) {
        bool launched;
        e = place_offsets(cu, nseq, reinterpret_cast<int *>(ws), a.seqs, &launched, st);
        if (e != cudaSuccess) return status_of(e);
    }
    Align align = gated_align(s, in);
    if (!kept) {
        a.keep = reinterpret_cast<float *>(ws + p.kept);
        e = launch_gated_fwd(a, s, align, cu != nullptr, ws + p.fwd_links, st);
        if (e != cudaSuccess) return status_of(e);
        kept = a.keep;
    }
    a.kept = kept, a.dfinal = dfinal;
    a.dy = gated_rows<const T>(s, *dy);
    a.dx = gated_rows<T>(s, out->dx), a.dr = gated_rows<T>(s, out->dr), a.di = gated_rows<T>(s, out->di), a.dz = gated_rows<T>(s, out->dz);
    a.dinit = out->dinit_state;
    a.ddecay_part = out->ddecay ? reinterpret_cast<float *>(ws + p.part) : nullptr;
    if (align == kSixteen && !rows_vec(*dy, sizeof(T), s->batch, s->seqlen)) align = kPairs;
    bool pairs = rows_pairs(*dy, sizeof(T), s->batch, s->seqlen);
    for (const ssd_rows_t *r : {&out->dx, &out->dr}) pairs = pairs && rows_pairs(*r, sizeof(T), s->batch, s->seqlen);
    if (in->i.data) pairs = pairs && rows_pairs(out->di, sizeof(T), s->batch, s->seqlen);
    if (in->z.data) pairs = pairs && rows_pairs(out->dz, sizeof(T), s->batch, s->seqlen);
    if (!pairs) align = kElements;
    const int64_t ntile = bwd_tiles(s->seqlen), rows = gated_blocks(s) * s->batch;
    const int most = kSMs * kBlocks;
    a.ntile = (int)ntile;
    a.sub = (int)bwd_warps(s->seqlen);
    a.per = rows_of_block(rows, ntile, a.sub, kWarps, most);
    a.tiles = (int)(ntile * ((rows + a.per - 1) / a.per));
    e = prepare(a, ws + p.links, rows, ntile, st);
    if (e != cudaSuccess) return status_of(e);
    a.some_empty = cu && a.dinit && any_empty(cu, nseq);
    const unsigned blocks = (unsigned)(a.tiles < most ? a.tiles : most);
    auto go = [&](auto pr, auto g, auto c) {
        constexpr int kStage = (int)sizeof(Stage<T, decltype(pr)::value>);
        constexpr int kBeside = (int)(4 * kWarps * 32 * sizeof(float4) + sizeof(LinkShared) + 2 * (kWarps - 1) * 32 * sizeof(float2) + 8);
        static_assert(kBlocks * (kStage + kBeside + 1024) <= 228 * 1024, "two blocks an SM");
        auto kernel = gated_bwd_kernel<T, decltype(pr)::value, decltype(g)::value, decltype(c)::value>;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStage);
        if (e == cudaSuccess) e = launch(kernel, dim3(blocks), a.sub * a.per * 32, kStage, st, a.rates != nullptr, a);
    };
    auto with_cuts = [&](auto pr, auto g) { cu ? go(pr, g, std::true_type{}) : go(pr, g, std::false_type{}); };
    auto with_gate = [&](auto pr) { a.z.p ? with_cuts(pr, std::true_type{}) : with_cuts(pr, std::false_type{}); };
    by_align(align, with_gate);
    timing_mark(st, "gated_bwd");
    if (e != cudaSuccess || !out->ddecay) return status_of(e);
    e = launch(gated_ddecay_kernel, dim3((unsigned)((s->channels + 31) / 32)), 1024, 0, st, true, a.ddecay_part,
               ntile * s->batch, s->channels, a.decay, out->ddecay);
    timing_mark(st, "gated_ddecay");
    return status_of(e);
}

}  // namespace
}  // namespace ssd

extern "C" {

size_t ssd_gated_scan_bwd_workspace_size(const ssd_gated_shape_t *shape, const int64_t *cu_seqlens, int64_t nseq,
                                         int with_chunk_states) {
    using namespace ssd;
    if (check_gated(shape, cu_seqlens, nseq) != SSD_OK || shape->batch == 0 || shape->seqlen == 0) return 0;
    return plan_bwd(shape, cu_seqlens, nseq, with_chunk_states != 0).bytes;
}

ssd_status_t ssd_gated_scan_bwd(const ssd_gated_shape_t *shape, const int64_t *cu_seqlens, int64_t nseq, const ssd_rows_t *dy,
                                const ssd_gated_inputs_t *in, const float *dfinal_state, const float *chunk_states,
                                const ssd_gated_grads_t *out, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace ssd;
    const ssd_status_t st = check_gated(shape, cu_seqlens, nseq);
    if (st != SSD_OK) return st;
    if (!cu_seqlens) nseq = shape->batch;
    if (!in || !out || !dy) return SSD_ERR_INVALID_ARG;
    if (nseq == 0) {
        if (out->ddecay)
            return status_of(cudaMemsetAsync(out->ddecay, 0, sizeof(float) * shape->channels, stream));
        return SSD_OK;
    }
    const bool rows = shape->seqlen > 0;
    const size_t es = dtype_size(shape->dtype);
    if (!gated_inputs_ok(shape, in, rows) || !aligned(dfinal_state, 4) || !aligned(chunk_states, 4) || !aligned(out->ddecay, 4) ||
        !aligned(out->dinit_state, 4) || (out->dinit_state && out->dinit_state == dfinal_state))
        return SSD_ERR_INVALID_ARG;
    if (rows) {
        const int64_t b = shape->batch, L = shape->seqlen, ch = shape->channels;
        if (!rows_in_ok(*dy, es) || !rows_out_ok(out->dx, es, b, L, ch) || !rows_out_ok(out->dr, es, b, L, ch)) return SSD_ERR_INVALID_ARG;
        if (in->i.data && !rows_out_ok(out->di, es, b, L, ch)) return SSD_ERR_INVALID_ARG;
        if (in->z.data && !rows_out_ok(out->dz, es, b, L, ch)) return SSD_ERR_INVALID_ARG;
    }
    const size_t need = ssd_gated_scan_bwd_workspace_size(shape, cu_seqlens, nseq, chunk_states != nullptr);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return SSD_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    return shape->dtype == SSD_DTYPE_BF16
               ? bwd_typed<bf16>(shape, cu_seqlens, nseq, dy, in, dfinal_state, chunk_states, out, ws, stream)
               : bwd_typed<float>(shape, cu_seqlens, nseq, dy, in, dfinal_state, chunk_states, out, ws, stream);
}

}  // extern "C"
