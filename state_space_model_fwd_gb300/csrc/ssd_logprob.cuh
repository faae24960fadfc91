// ssd_logprob.cuh -- the statistics of a row of logits and the gradient of
// what is formed from them, shared by the operators that read logits and that
// form them.
#pragma once

#include "ssd_channel.h"

namespace ssd {

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// What is known of a set of logits: the largest, m, and over all z
//   sum = sum 2^t,  moment = sum 2^t t,  t = z log2(e) - ref(m).
// t is one fused multiply-add: ref(m) is m log2(e) rounded, and what it was
// rounded by comes back in lse_of.  Entropies do not depend on the reference.
// Far from zero, where the rounding would not be small, t = (z - m) log2(e).
struct Stat {
    float m, sum, moment;
};
constexpr float kFar = 65536.f;
__device__ __forceinline__ bool is_far(float m) { return !(fabsf(m) <= kFar); }
// A z below kLeast counts as kLeast, an exponent below kNothing as kNothing: they add nothing in fp32, and minus infinity
// stays out of the moment.
constexpr float kLeast = -1e38f, kNothing = -200.f;
// (Not contracted with what uses it: the same m has to give the same reference.)
__device__ __forceinline__ float ref_of(float m) { return __fmul_rn(m, kLog2e); }
// What t of a set with the maximum m0 changes by when m takes its place.
__device__ __forceinline__ float shift_of(float m0, float m) {
    if (m0 == m) return 0.f;
    float d;
    if (is_far(m))
        d = is_far(m0) ? (m0 - m) * kLog2e : fmaf(-m, kLog2e, ref_of(m0));
    else
        d = is_far(m0) ? fmaf(m0, kLog2e, -ref_of(m)) : ref_of(m0) - ref_of(m);
    return fmaxf(d, kNothing);
}
__device__ __forceinline__ void move_to(Stat &s, float m) {
    const float d = shift_of(s.m, m), f = ex2(d);
    s.moment = f * fmaf(d, s.sum, s.moment), s.sum *= f, s.m = m;
}
// Of two disjoint sets; an empty one has sum 0 and m = -inf.
__device__ __forceinline__ Stat join(Stat a, Stat b) {
    const float m = max_nan(a.m, b.m);
    move_to(a, m), move_to(b, m);
    return Stat{m, a.sum + b.sum, a.moment + b.moment};
}
// Of the 32 (or, 16 lanes wide, 16) sets of a warp's lanes, in all lanes; one order of additions.
template <int WIDTH>
__device__ __forceinline__ Stat join_lanes(Stat s) {
    float m = s.m;
#pragma unroll
    for (int d = WIDTH / 2; d; d /= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d, WIDTH));
    move_to(s, m);
#pragma unroll
    for (int d = WIDTH / 2; d; d /= 2) {
        s.sum += __shfl_xor_sync(0xffffffffu, s.sum, d, WIDTH);
        s.moment += __shfl_xor_sync(0xffffffffu, s.moment, d, WIDTH);
    }
    return s;
}

// N more logits whose maximum is m.
template <int N>
__device__ __forceinline__ void add_to(Stat &s, const float (&z)[N], float m) {
    if (!(m <= s.m)) move_to(s, max_nan(s.m, m));  // (or NaN)
    if (is_far(s.m)) {
        if (s.m == -INFINITY) return;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float t = fmaxf((z[i] - s.m) * kLog2e, kNothing), e = ex2(t);
            s.sum += e, s.moment = fmaf(e, t, s.moment);
        }
        return;
    }
    const float ref = -ref_of(s.m);
    if constexpr (N % 2 == 0) {
        f2 sum = pack2(s.sum, 0.f), moment = pack2(s.moment, 0.f);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const f2 t = fma2(pack2(fmaxf(z[i], kLeast), fmaxf(z[i + 1], kLeast)), pack2(kLog2e, kLog2e), pack2(ref, ref));
            const f2 e = ex2x2(t);
            sum = add2(sum, e);
            moment = fma2(e, t, moment);
        }
        s.sum = sum2(sum), s.moment = sum2(moment);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float t = fmaf(fmaxf(z[i], kLeast), kLog2e, ref), e = ex2(t);
            s.sum += e, s.moment = fmaf(e, t, s.moment);
        }
    }
}
template <int N>
__device__ __forceinline__ void add_to(Stat &s, const float (&z)[N]) {
    float m = z[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = max_nan(m, z[i]);
    add_to(s, z, m);
}
// The same for pairs of bf16 as they lie in memory: the maximum and the clamp work on two at once.
template <int NW>
__device__ __forceinline__ void add_to(Stat &s, const uint32_t (&w)[NW]) {
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(w);
    __nv_bfloat162 top = p[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) top = __hmax2_nan(top, p[i]);
    const float m = max_nan(__low2float(top), __high2float(top));
    if (!(m <= s.m)) move_to(s, max_nan(s.m, m));
    if (is_far(s.m)) {
        float z[2 * NW];
#pragma unroll
        for (int i = 0; i < NW; ++i) z[2 * i] = __low2float(p[i]), z[2 * i + 1] = __high2float(p[i]);
        add_to(s, z, m);
        return;
    }
    const float ref = -ref_of(s.m);
    const __nv_bfloat162 least = __float2bfloat162_rn(kLeast);
    f2 sum = pack2(s.sum, 0.f), moment = pack2(s.moment, 0.f);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const __nv_bfloat162 c = __hmax2_nan(p[i], least);
        const uint32_t u = *reinterpret_cast<const uint32_t *>(&c);
        const f2 z = pack2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
        const f2 t = fma2(z, pack2(kLog2e, kLog2e), pack2(ref, ref)), e = ex2x2(t);
        sum = add2(sum, e);
        moment = fma2(e, t, moment);
    }
    s.sum = sum2(sum), s.moment = sum2(moment);
}

// The numbers of a row from its joined statistics and the given token's logit.
__device__ __forceinline__ float lse_of(const Stat &s) {
    if (s.m == -INFINITY || s.m == INFINITY) return s.m;
    const float off = !is_far(s.m) ? fmaf(s.m, kLog2e, -ref_of(s.m)) : 0.f;
    return s.m + (logf(s.sum) - kLn2 * off);
}
// nothing left in the row: 0; infinity or NaN in it: NaN
__device__ __forceinline__ float entropy_of(const Stat &s) {
    return s.m == -INFINITY ? 0.f : (s.m - s.m) + (logf(s.sum) - kLn2 * s.moment / s.sum);
}
__device__ __forceinline__ float logprob_of(float z, float lse) { return lse == -INFINITY ? z : z - lse; }

// dz = p (dlse - dlogprob - dentropy (log p + entropy)) + dlogprob [v = target]
struct RowGrad {
    float lse, coef, ent, dent, dlp, dlse;
    int target;
    bool none;  // nothing left in the row: zeros
};
struct RowGradIn {
    const int64_t *targets;
    const float *lse, *entropy, *dlogprob, *dlse, *dentropy;  // the latter three null: zero
};
__device__ __forceinline__ RowGrad row_grad(const RowGradIn &a, int64_t row, int vocab) {
    RowGrad g;
    const int64_t t = a.targets ? a.targets[row] : -1;
    g.target = t >= 0 && t < vocab ? (int)t : -1;
    g.lse = a.lse[row];
    g.dlp = a.dlogprob && t >= 0 ? a.dlogprob[row] : 0.f;
    if (t >= vocab) g.dlp = __uint_as_float(0x7FC00000u);
    g.dlse = a.dlse ? a.dlse[row] : 0.f;
    g.coef = g.dlse - g.dlp;
    g.dent = a.dentropy ? a.dentropy[row] : 0.f;
    g.ent = a.dentropy ? a.entropy[row] : 0.f;
    g.none = g.lse == -INFINITY;
    return g;
}
template <bool ENT>
__device__ __forceinline__ float grad_of(const RowGrad &g, float z) {
    const float t = z - g.lse, p = ex2(t * kLog2e);
    if constexpr (ENT) return p * fmaf(-g.dent, fmaxf(t, kNothing) + g.ent, g.coef);  // (a masked element's p is 0)
    return p * g.coef;
}

// The given token's: dlogprob (1 - p) keeps its digits where p is close to 1.
template <bool ENT>
__device__ __forceinline__ float given_grad(const RowGrad &g, float z) {
    const float t = z - g.lse, p = ex2(t * kLog2e);
    const float other = ENT ? p * fmaf(-g.dent, fmaxf(t, kNothing) + g.ent, g.dlse) : p * g.dlse;
    return fmaf(-g.dlp, expm1f(t), other);
}

// Rows at one stride, which may be as far apart as batches elsewhere (the last rows of long prompts' logits).
inline bool far_rows_ok(const ssd_rows_t &r, size_t esize) { return rows_in_ok(ssd_rows_t{r.data, r.row_stride, 0}, esize); }
inline bool far_rows_out_ok(const ssd_rows_t &r, size_t esize, int64_t rows, int64_t cols) {
    return rows_out_ok(ssd_rows_t{r.data, r.row_stride, 0}, esize, rows, 1, cols);
}

}  // namespace ssd
