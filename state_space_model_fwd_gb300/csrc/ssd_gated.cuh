// ssd_gated.cuh -- pieces shared by the gated scan's kernels.
//
// Per channel, with s(v) = 1 / (1 + exp(-v)):
//   m = rate softplus(decay) s(r),  a = exp(-m),  beta = sqrt(1 - a^2),
//   h <- a h + beta s(i) x,  y = h (times silu(z)).
// Everything is formed from v = 1 - a = -expm1(-m): 1 - a^2 = v + v a keeps
// its digits where a is close to 1, which is where such layers work.
//
// The blocks of the prompt's kernels, a few on each SM, take one tile after
// another: kCols channels, two a lane, and kWarps x S consecutive tokens, S a
// warp, whose inputs stay in registers from the one read to the output; the
// next tile's are copied into shared memory meanwhile.  What a run of tokens
// does to the state is h -> A h + H; warps exchange their (A, H) through shared
// memory, tiles theirs through the workspace (Links).  A run that holds a
// sequence's boundary does not let the state through, whatever its value:
// A = -1 says so.
//
// Why one pass: a pass that only sums tiles up, and another from the states
// that enter them, would read x, r and i twice (1.6 times the bytes).
#pragma once

#include "ssd_channel.h"
#include "ssd_status.h"
#include "tc_ptx.cuh"

namespace ssd {

constexpr int kCols = 64;        // channels of a block
constexpr int kStateEvery = 64;  // tokens between the states kept for the gradient
constexpr int kGroup = 16;       // tiles from one entry state to the next

// Two channels of one token as they lie in memory.
template <typename T>
struct Two;
template <>
struct Two<bf16> {
    uint32_t w;
};
template <>
struct Two<float> {
    float2 w;
};
__device__ __forceinline__ Two<bf16> two_of(bf16, float v) {
    const __nv_bfloat162 h = __float2bfloat162_rn(v);
    return {*reinterpret_cast<const uint32_t *>(&h)};
}
__device__ __forceinline__ Two<float> two_of(float, float v) { return {make_float2(v, v)}; }
__device__ __forceinline__ float2 widen(const Two<bf16> &v) {
    return make_float2(__uint_as_float(v.w << 16), __uint_as_float(v.w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 widen(const Two<float> &v) { return v.w; }

// How rows lie: anywhere, their pairs of channels on their own size's boundary,
// or each on a 16-byte boundary.
enum Align { kElements, kPairs, kSixteen };
// A lane's channels: c0 and c1 of the block's 64.  Rows whose pairs lie on
// their own size's boundary are read in pairs, two neighbours a lane; others
// one element at a time, 32 neighbours a warp.
template <int ALIGN>
struct Lane {
    int c0;
    int step;       // from c0 to the second channel
    bool in0, in1;  // which exist
    __device__ __forceinline__ Lane(int blk, int lane, int ch) {
        c0 = blk * kCols + (ALIGN ? 2 * lane : lane);
        step = ALIGN ? 1 : 32;
        in0 = c0 < ch, in1 = c0 + step < ch;
    }
};

// The lane's place in a row.  Rows are the same in all lanes and lanes keep one 32-bit offset: an access needs no
// arithmetic of its own.
template <typename P, int ALIGN>
__device__ __forceinline__ P *place(P *row, const Lane<ALIGN> &k) {
    using B = std::conditional_t<std::is_const_v<P>, const char, char>;
    return reinterpret_cast<P *>(reinterpret_cast<B *>(row) + (size_t)((unsigned)k.c0 * (unsigned)sizeof(P)));
}
template <typename T, int ALIGN>
__device__ __forceinline__ Two<T> load_two(const T *row, const Lane<ALIGN> &k, float fill) {
    const T *p = place(row, k);
    Two<T> v = two_of(T(), fill);
    if constexpr (ALIGN) {
        if (k.in0) v.w = *reinterpret_cast<const decltype(v.w) *>(p);
    } else if constexpr (sizeof(T) == 2) {
        uint32_t lo = v.w & 0xFFFFu, hi = v.w >> 16;
        if (k.in0) lo = *reinterpret_cast<const uint16_t *>(p);
        if (k.in1) hi = *reinterpret_cast<const uint16_t *>(p + 32);
        v.w = lo | hi << 16;
    } else {
        if (k.in0) v.w.x = p[0];
        if (k.in1) v.w.y = p[32];
    }
    return v;
}
// A warp's 64 channels of one token in shared memory.  Rows on 16-byte boundaries lie as the lanes read them; others as they
// lie in memory from the boundary before them on, so that they are copied 16 bytes at a time all the same.  (What is read
// before a row is not used.  It is in the row's allocation, which begins on such a boundary; nothing is read behind a row.)
template <typename T, int ALIGN>
struct alignas(16) Slot {
    char b[kCols * sizeof(T) + (ALIGN == kSixteen ? 0 : 16)];
};
// Where a row lies in its slot, token by token.
template <typename T, int ALIGN>
struct Skew {
    unsigned first = 0, step = 0;
    __device__ __forceinline__ Skew(const Rows<const T> &r, int b, int t0) {
        if constexpr (ALIGN != kSixteen) first = (unsigned)reinterpret_cast<uintptr_t>(r.at(b, t0)), step = (unsigned)r.rs * (unsigned)sizeof(T);
    }
    __device__ __forceinline__ unsigned operator()(int s) const { return ALIGN == kSixteen ? 0 : (first + s * step) & 15; }
};
template <typename T, int ALIGN>
__device__ __forceinline__ Two<T> two_in(const Slot<T, ALIGN> &slot, int lane, unsigned skew) {
    if constexpr (ALIGN != kElements) {
        return reinterpret_cast<const Two<T> *>(slot.b + skew)[lane];
    } else if constexpr (sizeof(T) == 2) {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(slot.b + skew) + lane;
        return {(uint32_t)p[0] | (uint32_t)p[32] << 16};
    } else {
        const float *p = reinterpret_cast<const float *>(slot.b + skew) + lane;
        return {make_float2(p[0], p[32])};
    }
}
template <typename T, int ALIGN>
__device__ __forceinline__ void fill_slot(Slot<T, ALIGN> &slot, int lane, float v) {
    const Two<T> f = two_of(T(), v);
    for (int i = lane; i < (int)(sizeof(slot) / sizeof(f)); i += 32) reinterpret_cast<Two<T> *>(slot.b)[i] = f;
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Asynchronous copies of a warp's S tokens of one array from token t0 on, `left` of which exist, to every STRIDE-th slot
// (others: `fill`).  A lane copies 16 bytes of one of the rows that an instruction spans, for others to read.  65537 x 2560
// packed bf16, rows of 2560: 447 us; of 2562 516 (copied by the lanes that read them, four bytes each: 527); of 2561 532
// (through registers: 1092).
template <typename T, int ALIGN, int S, int STRIDE>
__device__ __forceinline__ void fetch_rows(Slot<T, ALIGN> *dst, const Rows<const T> &r, int b, int t0, const Lane<ALIGN> &k, int lane,
                                           int left, int ch, float fill) {
    constexpr int CHUNKS = kCols * sizeof(T) / 16, ROWS = 32 / CHUNKS, EACH = 16 / sizeof(T);
    const int64_t step = (int64_t)r.rs * (int)sizeof(T);
    const int first = lane / CHUNKS, q = lane % CHUNKS, c0 = k.c0 - (ALIGN ? 2 : 1) * lane;
    const Two<T> f = two_of(T(), fill);
    auto fill16 = [&](char *d) {
#pragma unroll
        for (int i = 0; i < EACH / 2; ++i) reinterpret_cast<Two<T> *>(d)[i] = f;
    };
    if constexpr (ALIGN == kSixteen) {
        const int c = c0 + q * EACH;
        const char *src = reinterpret_cast<const char *>(r.at(b, t0) + c) + first * step;
        char *d = dst[first * STRIDE].b + q * 16;
#pragma unroll
        for (int s = 0; s < S; s += ROWS) {
            if (s + first < left && c < ch)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(d)), "l"(src) : "memory");
            else
                fill16(d);
            src += step * ROWS, d += ROWS * STRIDE * sizeof(*dst);
        }
    } else {
        const int before = c0 * (int)sizeof(T), row = ch * (int)sizeof(T);  // bytes of the row before the block's, in all
        const char *src = reinterpret_cast<const char *>(r.at(b, t0)) + before;
        auto one = [&](int s, int c, const char *p) {  // the c-th 16 bytes of token s, whose channels begin at p
            const int at = c * 16 - (int)(reinterpret_cast<uintptr_t>(p) & 15), valid = row - before - at;
            char *d = dst[s * STRIDE].b + c * 16;
            if (s < left && valid > 0)  // (of fewer than 16 bytes zeros behind them)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(d)), "l"(p + at), "r"(min(valid, 16))
                             : "memory");
            else
                fill16(d);
        };
#pragma unroll 2
        for (int s = 0; s < S; s += ROWS) one(s + first, q, src + (s + first) * step);
        if (lane < S) one(lane, CHUNKS, src + lane * step);
    }
}
// ALL: every channel of the block exists.
template <typename T, int ALIGN, bool ALL = false>
__device__ __forceinline__ void store_two(T *row, const Lane<ALIGN> &k, float2 f) {
    T *p = place(row, k);
    if constexpr (ALIGN) {
        if (!ALL && !k.in0) return;
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint32_t *>(p) = tc::pack_bf16x2(f.x, f.y);
        else
            *reinterpret_cast<float2 *>(p) = f;
    } else {
        if (ALL || k.in0) p[0] = from_f32<T>(f.x);
        if (ALL || k.in1) p[32] = from_f32<T>(f.y);
    }
}
// The same for fp32 arrays of the channels (states, parameters): p is the array's row.
template <int ALIGN>
__device__ __forceinline__ float2 load_state(const float *p, const Lane<ALIGN> &k) {
    return make_float2(p && k.in0 ? p[k.c0] : 0.f, p && k.in1 ? p[k.c0 + k.step] : 0.f);
}
template <int ALIGN>
__device__ __forceinline__ void store_state(float *p, const Lane<ALIGN> &k, float2 v) {
    if (k.in0) p[k.c0] = v.x;
    if (k.in1) p[k.c0 + k.step] = v.y;
}

// rate softplus(decay), by the library's functions: once a call and channel, by the kernel that clears the links, where
// there are any
__device__ __forceinline__ float decay_rate(float decay, float rate) {
    return rate * (fmaxf(decay, 0.f) + log1pf(expf(-fabsf(decay))));
}

__device__ __forceinline__ f2 splat(float v) { return pack2(v, v); }
__device__ __forceinline__ f2 both(float2 v) { return pack2(v.x, v.y); }
__device__ __forceinline__ float2 apart(f2 v) {
    float2 r;
    unpack2(v, r.x, r.y);
    return r;
}

__device__ __forceinline__ float2 sigmoid2(float2 v) {
    const float2 t = apart(mul2(both(v), splat(-kLog2e)));
    const float2 d = apart(add2(pack2(ex2(t.x), ex2(t.y)), splat(1.f)));
    return make_float2(rcp(d.x), rcp(d.y));
}

// v = 1 - a and a from m = -log a >= 0.  Up to m = 1, v = m q(m), q the
// polynomial of degree 6 of least relative error (2.5e-9, by the exchange
// algorithm) to (1 - e^-m) / m on [0, 1]: 1.4e-7 in fp32.  Beyond, 1 - e^-m,
// whose absolute error of 2^-24 or so is 1e-7 of v >= 0.63.  SMALL: no m is
// above 1.  (Layers keep their states for tens of tokens: rate softplus(decay)
// is below 1 throughout, which a warp finds out from its channels' decays;
// the test and the second form cost 14 of 80 instructions a token.)
template <bool SMALL>
__device__ __forceinline__ void decay2(f2 m, f2 &v, f2 &a) {
    f2 q = fma2(m, splat(1.2838072e-4f), splat(-1.2986638e-3f));
    q = fma2(q, m, splat(8.2730958e-3f));
    q = fma2(q, m, splat(-4.1645579e-2f));
    q = fma2(q, m, splat(0.1666631f));
    q = fma2(q, m, splat(-0.49999976f));
    q = fma2(q, m, splat(1.f));
    v = mul2(q, m);
    if constexpr (SMALL) {
        a = fma2(v, splat(-1.f), splat(1.f));
    } else {
        const float2 s = apart(v), e = apart(mul2(m, splat(-kLog2e))), mv = apart(m);
        const float ex = ex2(e.x), ey = ex2(e.y);
        const bool nx = mv.x <= 1.f, ny = mv.y <= 1.f;
        const float vx = nx ? s.x : 1.f - ex, vy = ny ? s.y : 1.f - ey;
        v = pack2(vx, vy);
        a = pack2(nx ? 1.f - vx : ex, ny ? 1.f - vy : ey);
    }
}
__device__ __forceinline__ float sqrt_approx(float v) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rsqrt_approx(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// What a run of tokens does to the state that enters it.
struct Run {
    float2 A, H;
};
__device__ __forceinline__ float through(float A, float H, float h) { return A < 0.f ? H : fmaf(A, h, H); }
__device__ __forceinline__ float2 through(const Run &r, float2 h) {
    return make_float2(through(r.A.x, r.H.x, h.x), through(r.A.y, r.H.y, h.y));
}
// r, then s
__device__ __forceinline__ Run then(const Run &r, const Run &s) {
    Run o;
    o.H = through(s, r.H);
    o.A.x = s.A.x < 0.f || r.A.x < 0.f ? -1.f : r.A.x * s.A.x;
    o.A.y = s.A.y < 0.f || r.A.y < 0.f ? -1.f : r.A.y * s.A.y;
    return o;
}

// What tiles of a block row (one channel block of one sequence row) hand on,
// [row][tile][64] in the workspace: every tile's (A, H), and the state that
// enters every group of kGroup tiles.  The words are their own flags: the
// workspace is filled with ones before the launch, and no A is that NaN (a
// computed NaN is the canonical one, and -1 stands for a boundary).  A tile's
// run does not depend on other tiles, so a tile waits for the entry state of
// its group and the runs before it in the group, in one round of loads; the
// last of a group hands the next entry state on.  The order of every sum is
// fixed.  Tiles are numbered by a counter, earlier tokens first, and a block
// finishes its tiles in that order, so the first unfinished one never waits.
// Groups of 16: one sequence of 65537 tokens, 64 channels 35 us (8: 58, 32:
// 26), 48 packed ones of 2560 channels out of rows of 2568 461 (455, 487).
struct Links {
    unsigned long long *run, *entry;  // null: one tile a row, nothing to wait for
    unsigned *ticket;
    unsigned *status;
};
constexpr unsigned kUnset = 0xFFFFFFFFu;
__device__ __forceinline__ unsigned long long link_word(float A, float H) {
    // (a NaN that came in through an operand may have any bits)
    const unsigned a = A != A ? 0x7FFFFFFFu : __float_as_uint(A);
    return (unsigned long long)a << 32 | __float_as_uint(H);
}
__device__ __forceinline__ void link_store(unsigned long long *p, const Run &r) {
    asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(link_word(r.A.x, r.H.x)) : "memory");
    asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p + 32), "l"(link_word(r.A.y, r.H.y)) : "memory");
}
__device__ __forceinline__ unsigned long long link_load(const unsigned long long *p) {
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
// Waits until both words are there; gives up after 100 ms and says so in the status word.
__device__ __forceinline__ Run link_wait(const unsigned long long *p, unsigned *status) {
    unsigned long long u = link_load(p), v = link_load(p + 32);
    auto unset = [&] { return (unsigned)(u >> 32) == kUnset || (unsigned)(v >> 32) == kUnset; };
    if (unset()) {
        const uint64_t t0 = tc::globaltimer_ns();
        do {
            __nanosleep(40);  // (other warps of the SM need the issue slots)
            u = link_load(p), v = link_load(p + 32);
            const uint64_t spent = tc::globaltimer_ns() - t0;
            if (spent > 100000000ull) atomicOr(status, 1u);
            if (spent > 1000000ull && *reinterpret_cast<volatile unsigned *>(status)) break;  // (another block's, too)
        } while (unset());
    }
    Run r;
    r.A = make_float2(__uint_as_float((unsigned)(u >> 32)), __uint_as_float((unsigned)(v >> 32)));
    r.H = make_float2(__uint_as_float((unsigned)u), __uint_as_float((unsigned)v));
    return r;
}

// A tile's place among the links: number `at` of its row in the order in which states pass.
struct Place {
    unsigned long long *mine, *entry;  // this tile's run; the state that enters its group
    int in_group;
    bool more;  // a tile follows in the row
    __device__ __forceinline__ Place(const Links &l, int row, int at, int ntile, int lane) {
        const int groups = (ntile + kGroup - 1) / kGroup;
        mine = l.run + ((int64_t)row * ntile + at) * kCols + lane;
        entry = l.entry + ((int64_t)row * groups + at / kGroup) * kCols + lane;
        in_group = at % kGroup, more = at + 1 < ntile;
    }
    __device__ __forceinline__ void publish(const Run &all) const {
        if (in_group != kGroup - 1 && more) link_store(mine, all);
    }
};
struct LinkShared {
    float4 tiles[kGroup - 1][32];
    float2 group[32], enter[32];
};
// The state that enters the tile; `first`: the one that enters the row, for its first group.  `all`: the tile's own run,
// published, in warp 0.  Warp j looks after the j-th run before it in its group (and the (j + nw)-th), the last warp after the
// state that enters the group; warp 0 puts them together.
__device__ __forceinline__ float2 pass_links(const Place &q, const Links &l, LinkShared &sh, float2 first, const Run &all, bool has_entry,
                                             int warp, int nw, int lane) {
    for (int j = warp; j < q.in_group; j += nw) {
        const Run r = link_wait(q.mine - (int64_t)(j + 1) * kCols, l.status);
        sh.tiles[j][lane] = make_float4(r.A.x, r.A.y, r.H.x, r.H.y);
    }
    if (warp == nw - 1 && has_entry) sh.group[lane] = link_wait(q.entry, l.status).H;
    __syncthreads();
    if (warp == 0) {
        float2 h = has_entry ? sh.group[lane] : first;
        for (int j = q.in_group - 1; j >= 0; --j) {
            const float4 v = sh.tiles[j][lane];
            h = through(Run{make_float2(v.x, v.y), make_float2(v.z, v.w)}, h);
        }
        if (q.in_group == kGroup - 1 && q.more) link_store(q.entry + kCols, Run{make_float2(0.f, 0.f), through(all, h)});
        sh.enter[lane] = h;
    }
    __syncthreads();
    return sh.enter[lane];
}

// The number of a value that is the same in all lanes, as the compiler cannot know.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Sequence boundaries in a warp's tokens t0 .. t0 + S - 1 (the same in all lanes).
struct Cuts {
    unsigned first, last;  // bit s: token t0 + s is its sequence's first, last
    int seq;               // of token t0
};
template <int S>
__device__ __forceinline__ Cuts cuts_of(const Seqs &q, int t0) {
    const int *start = q.offsets();
    Cuts c{0, 0, seq_of(start, q.n, t0)};
    if (start[c.seq] == t0) c.first = 1;
    for (int s = c.seq + 1; s <= q.n; ++s) {  // (an empty sequence has the next one's bit, or none past the last token)
        const int d = start[s] - t0;
        if (d > S) break;
        if (d < S && start[s] < q.L) c.first |= 1u << d;
        c.last |= 1u << (d - 1);
    }
    c.first = (unsigned)uniform((int)c.first), c.last = (unsigned)uniform((int)c.last), c.seq = uniform(c.seq);
    return c;
}
// Every empty sequence's dst = src (zeros without src).
__device__ __forceinline__ void pass_empty(const Seqs &q, int ch, const float *src, float *dst) {
    const int *start = q.offsets();
    for (int s = blockIdx.x; s < q.n; s += gridDim.x) {
        if (start[s] != start[s + 1]) continue;
#pragma unroll 4
        for (int c = threadIdx.x; c < ch; c += blockDim.x) dst[(int64_t)s * ch + c] = src ? src[(int64_t)s * ch + c] : 0.f;
    }
}

// The sequence of token t, at or after sequence s.
__device__ __forceinline__ int seq_from(const Seqs &q, int s, int t) {
    const int *start = q.offsets();
    while (start[s + 1] <= t) ++s;
    return s;
}

template <typename T>
struct GatedArgs {
    Rows<const T> x, r, i, z, dy;  // i.p, z.p null: absent
    Rows<T> y, dx, dr, di, dz;     // y.p null: only the kept states are wanted
    const float *decay, *init, *dfinal, *kept;
    float *rates;  // [ch] rate softplus(decay); null: formed by the tiles (one a row)
    float *fin, *keep, *dinit, *ddecay_part;  // keep, kept: [b][ceil(L / 64)][ch] states entering every 64 tokens
    float rate;
    int ch, nblk, batch, ntile, nkeep;
    int sub, per;           // warps of a row's tile; rows of a block (linked rows: 1)
    int tiles, some_empty;  // tiles in all (of `per` rows each); whether a sequence has no tokens
    Seqs seqs;
    Links links;
};

// Rows of one short tile each: as many to a block as leave every place of a block filled (4096 x 16 x 2560 bf16 394 us, one a
// block 1729; gradient with the states formed again 1068, 3617).
inline int rows_of_block(int64_t rows, int64_t ntile, int sub, int warps, int places) {
    if (ntile > 1) return 1;
    const int64_t most = warps / sub, want = (rows + places - 1) / places;
    return (int)(want < most ? want : most);
}

template <typename T, int ALIGN>
__device__ __forceinline__ float2 rates_of(const GatedArgs<T> &a, const Lane<ALIGN> &k) {
    if (a.rates) return load_state(a.rates, k);
    const float2 d = load_state(a.decay, k);
    return make_float2(k.in0 ? decay_rate(d.x, a.rate) : 0.f, k.in1 ? decay_rate(d.y, a.rate) : 0.f);
}

// An operand's rows as the kernels get them.  A stride between rows of which there is one, or none, is 0 whatever the caller
// left there: alignment goes by the strides that mean something, and Skew steps by the row stride over all tokens of a warp,
// those past the end too.
template <typename P>
Rows<P> gated_rows(const ssd_gated_shape_t *s, const ssd_rows_t &r) {
    Rows<P> v = rows_of<P>(r);
    if (!r.data || s->batch <= 1) v.bs = 0;
    if (!r.data || s->seqlen <= 1) v.rs = 0;
    return v;
}

// host side (ssd_gated.cu)
ssd_status_t check_gated(const ssd_gated_shape_t *s, const int64_t *cu, int64_t nseq);
bool gated_inputs_ok(const ssd_gated_shape_t *s, const ssd_gated_inputs_t *in, bool rows);
inline int64_t gated_blocks(const ssd_gated_shape_t *s) { return (s->channels + kCols - 1) / kCols; }
inline int64_t gated_kept(const ssd_gated_shape_t *s) { return (s->seqlen + kStateEvery - 1) / kStateEvery; }
// Workspace of the rates and of the links of `rows` block rows of `ntile` tiles each (none of one tile each); their place in
// it, and the launch that prepares them.
size_t links_bytes(int64_t ch, int64_t rows, int64_t ntile);
template <typename T>
cudaError_t prepare(GatedArgs<T> &a, char *ws, int64_t rows, int64_t ntile, cudaStream_t st);
template <typename F>
void by_align(Align a, F &&f) {
    a == kSixteen ? f(std::integral_constant<int, kSixteen>{})
    : a == kPairs ? f(std::integral_constant<int, kPairs>{})
                  : f(std::integral_constant<int, kElements>{});
}
// Pairs of channels that lie on their own size's boundary in every row.
bool rows_pairs(const ssd_rows_t &r, size_t esize, int64_t b, int64_t L);
template <typename T>
GatedArgs<T> gated_args(const ssd_gated_shape_t *s, const ssd_gated_inputs_t *in, int64_t nseq);
// of the rows that are read
Align gated_align(const ssd_gated_shape_t *s, const ssd_gated_inputs_t *in);
bool any_empty(const int64_t *cu, int64_t nseq);
template <typename T>
cudaError_t launch_gated_fwd(GatedArgs<T> &a, const ssd_gated_shape_t *s, Align align, bool packed, char *links, cudaStream_t st);
size_t gated_fwd_links(const ssd_gated_shape_t *s);

}  // namespace ssd
