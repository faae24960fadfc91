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

struct Stat {
    float m, sum, moment;
};
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }
// Exponents below this add nothing in fp32; clamping keeps minus infinity out of the moment.
constexpr float kNothing = -200.f;
// Of two disjoint sets.
__device__ __forceinline__ Stat join(const Stat &a, const Stat &b) {
    const float m = max_nan(a.m, b.m), base = base_of(m);
    Stat r{m, 0.f, 0.f};
    if (a.sum > 0.f) {
        const float d = fmaxf((a.m - base) * kLog2e, kNothing), f = ex2(d);
        r.sum = f * a.sum, r.moment = f * fmaf(d, a.sum, a.moment);
    }
    if (b.sum > 0.f) {
        const float d = fmaxf((b.m - base) * kLog2e, kNothing), f = ex2(d);
        r.sum += f * b.sum, r.moment += f * fmaf(d, b.sum, b.moment);
    }
    return r;
}

template <int N>
__device__ __forceinline__ void add_to(Stat &s, const float (&z)[N]) {
    float m = z[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = max_nan(m, z[i]);
    if (!(m <= s.m)) {  // (or NaN)
        const float top = max_nan(s.m, m);
        if (s.sum > 0.f) {
            const float d = fmaxf((s.m - top) * kLog2e, kNothing), f = ex2(d);
            s.moment = f * fmaf(d, s.sum, s.moment), s.sum *= f;
        }
        s.m = top;
    }
    const float base = base_of(s.m);
    f2 sum = pack2(s.sum, 0.f), moment = pack2(s.moment, 0.f);
    const f2 minus = pack2(-base, -base), scale = pack2(kLog2e, kLog2e);
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            float t0, t1;
            unpack2(mul2(add2(pack2(z[i], z[i + 1]), minus), scale), t0, t1);
            t0 = fmaxf(t0, kNothing), t1 = fmaxf(t1, kNothing);
            const f2 e = pack2(ex2(t0), ex2(t1));
            sum = add2(sum, e);
            moment = fma2(e, pack2(t0, t1), moment);
        }
        s.sum = sum2(sum), s.moment = sum2(moment);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float t = fmaxf((z[i] - base) * kLog2e, kNothing), e = ex2(t);
            s.sum += e, s.moment = fmaf(e, t, s.moment);
        }
    }
}

// The numbers of a row from its joined statistics and the given token's logit.
__device__ __forceinline__ float lse_of(const Stat &s) {
    return s.m == -INFINITY || s.m == INFINITY ? s.m : s.m + logf(s.sum);
}
// nothing left in the row: 0; infinity or NaN in it: NaN
__device__ __forceinline__ float entropy_of(const Stat &s) {
    return s.m == -INFINITY ? 0.f : (s.m - s.m) + (logf(s.sum) - kLn2 * s.moment / s.sum);
}
__device__ __forceinline__ float logprob_of(float z, float lse) { return lse == -INFINITY ? z : z - lse; }

// dz = p (dlse - dlogprob - dentropy (log p + entropy)) + dlogprob [v = target]
struct RowGrad {
    float lse, coef, ent, dent, dlp;
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
    g.coef = (a.dlse ? a.dlse[row] : 0.f) - g.dlp;
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

}  // namespace ssd
