// ssd_norm.cu -- the norms before and after a block, fused with the gate and
// the scaled residual.
//
//   v = x (silu(z)),  s = residual + scale v,  out = s rsqrt(mean s^2 + eps) w (silu(z))
//
// the mean over groups of `group` columns; forward and gradient.  A few
// operations an element against 2 to 6 element transfers: bound by memory.
// A (row, group) is read once, all its loads in flight together, reduced over
// a team of threads and written from registers.  The team is a warp for short
// groups, several to a block, and otherwise a block of just enough threads
// for NV vectors each, so that few threads idle whatever the width.  The gate
// is fixed at compile time for widths up to 8192 (read at run time inside the
// loops: 91 us instead of 71 for the gradient at 4096 x 5120 gated, 89 instead
// of 82 forward at 16384 x 5120).
// bf16: 16384 x 5120 gated in 81 us, 6.2 TB/s; the gradient with an fp32
// residual and scale at 8191 x 2560 in 75 us with the sums, 5.1 TB/s.  Gated
// gradients, fp32 and groups over 8192 columns spill registers: 8191 x 2560
// gated in 62 us against 31 for its bytes, 2048 x 16384 in 296 against 30.
#include <type_traits>

#include "ssd_layer.cuh"

namespace ssd {
namespace {

constexpr int64_t kMaxGroup = 32768;

enum Gate : int { kNone, kBefore, kAfter };

// A [rows, dim] array; a thread's place in it.
template <typename T>
struct Mat {
    T *p;
    int rs;
    __device__ __forceinline__ T *at(int row, int c) const { return p + (int64_t)row * rs + c; }
};

template <typename T, typename TR>
struct NormArgs {
    Mat<const T> x, z;
    Mat<const TR> res;  // forward: the residual; gradient: the stored sum (p null: none)
    const float *weight, *scale;
    Mat<T> out;
    Mat<TR> res_out;  // forward: the sum; gradient: the residual's gradient
    // gradient
    Mat<const T> dout;
    Mat<const TR> dres;  // gradient of the sum from elsewhere (p null: zero)
    Mat<T> dx, dz;
    float *partial;  // [slots][2][dim]: dweight, dscale
    int64_t rows;
    int dim, group, ngroups, gate;
    float eps, inv_group;
};

// V consecutive elements as loaded: 16 bytes an access, or one element (V = 1).
template <typename T, int V>
struct Raw {
    static constexpr int N = V == 1 ? 1 : V * (int)sizeof(T) / 16, W = V / N;
    Vec<T, W> p[N];
    __device__ __forceinline__ void load(const T *src) {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = load_vec<T, W>(src + i * W);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = zero_vec<T, W>();
    }
    __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) widen<T, W>(p[i], f + i * W);
    }
    static __device__ __forceinline__ void store(T *dst, const float (&f)[V]) {
#pragma unroll
        for (int i = 0; i < N; ++i) store_vec<T, W>(dst + i * W, narrow<T, W>(f + i * W));
    }
};
template <int V>
__device__ __forceinline__ void load_param(const float *p, float (&f)[V]) {
    Raw<float, V> r;
    r.load(p);
    r.get(f);
}

// Sum over a team: a warp, or the whole block (one barrier; the caller
// alternates between two arrays when it sums again).
template <bool WARP, int R>
__device__ __forceinline__ void team_sum(float (&v)[R], float (&smem)[32 * R]) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], off);
    if constexpr (!WARP) {
        const int warps = blockDim.x / 32;
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) smem[threadIdx.x / 32 * R + r] = v[r];
        __syncthreads();
        const int lane = threadIdx.x % 32;
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = lane < warps ? smem[lane * R + r] : 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
#pragma unroll
            for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], off);
    }
}

constexpr int kWarpTeams = 4;  // warp teams per block
constexpr int kAnyGate = -1;   // the gate is read at run time (rare widths)

// NV vectors of V values per thread cover the group.
template <typename T, typename TR, int V, int NV, bool WARP, int GATE>
__global__ void __launch_bounds__(WARP ? kWarpTeams * 32 : GATE == kAnyGate ? 1024 : 512, WARP || GATE == kAnyGate ? 1 : 3)
    norm_fwd_kernel(const __grid_constant__ NormArgs<T, TR> a) {
    __shared__ float smem[32];
    const int gate = GATE == kAnyGate ? a.gate : GATE;
    const int team = WARP ? 32 : blockDim.x, lane = WARP ? threadIdx.x % 32 : threadIdx.x;
    const int64_t id = WARP ? (int64_t)blockIdx.x * kWarpTeams + threadIdx.x / 32 : blockIdx.x;
    if (id >= a.rows * a.ngroups) return;  // (whole teams)
    const int row = (int)(a.ngroups == 1 ? id : id / a.ngroups);
    const int c0 = a.ngroups == 1 ? 0 : (int)(id % a.ngroups) * a.group;
    Raw<T, V> x[NV], z[NV];
    Raw<TR, V> res[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i * team + lane) * V, c = c0 + at;
        x[i].zero(), z[i].zero(), res[i].zero();
        if (at < a.group) {
            x[i].load(a.x.at(row, c));
            if (gate != kNone) z[i].load(a.z.at(row, c));
            if (a.res.p) res[i].load(a.res.at(row, c));
        }
    }
    float s[NV][V];
    float sq[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i * team + lane) * V, c = c0 + at;
        x[i].get(s[i]);
        if (gate == kBefore) {
            float f[V];
            z[i].get(f);
#pragma unroll
            for (int v = 0; v < V; ++v) s[i][v] *= silu(f[v]);
        }
        if (a.scale && at < a.group) {
            float f[V];
            load_param<V>(a.scale + c, f);
#pragma unroll
            for (int v = 0; v < V; ++v) s[i][v] *= f[v];
        }
        if (a.res.p) {
            float f[V];
            res[i].get(f);
#pragma unroll
            for (int v = 0; v < V; ++v) s[i][v] += f[v];
            if (at < a.group) Raw<TR, V>::store(a.res_out.at(row, c), s[i]);
        }
        // (vectors past the group are zero)
#pragma unroll
        for (int v = 0; v < V; ++v) sq[0] = fmaf(s[i][v], s[i][v], sq[0]);
    }
    team_sum<WARP, 1>(sq, smem);
    const float rstd = rsqrtf(fmaf(sq[0], a.inv_group, a.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i * team + lane) * V, c = c0 + at;
        if (at >= a.group) break;
        float w[V];
        load_param<V>(a.weight + c, w);
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] *= s[i][v] * rstd;
        if (gate == kAfter) {
            float f[V];
            z[i].get(f);
#pragma unroll
            for (int v = 0; v < V; ++v) w[v] *= silu(f[v]);
        }
        Raw<T, V>::store(a.out.at(row, c), w);
    }
}

__device__ __forceinline__ void prefetch(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Gradient.  With hat = s rstd and gw = dout (silu z) w:
//   ds = rstd (gw - hat mean(gw hat)) + dres,  both means from one reduction;
//   dresidual = ds, dv = scale ds, dscale = sum_rows ds v, dweight = sum_rows dout (silu z) hat.
// A team walks rows of its own group of columns, its column sums in
// registers; the teams' partial sums are added by a second kernel in a fixed
// order.
template <typename T, typename TR, int V, int NV, bool WARP, int GATE>
__global__ void __launch_bounds__(WARP ? kWarpTeams * 32 : GATE == kAnyGate ? 1024 : 512, WARP ? 3 : 1)
    norm_bwd_kernel(const __grid_constant__ NormArgs<T, TR> a, int slots) {
    __shared__ float smem[2][64];
    const int gate = GATE == kAnyGate ? a.gate : GATE;
    const int team = WARP ? 32 : blockDim.x, lane = WARP ? threadIdx.x % 32 : threadIdx.x;
    const int64_t id = WARP ? (int64_t)blockIdx.x * kWarpTeams + threadIdx.x / 32 : blockIdx.x;
    if (id >= (int64_t)slots * a.ngroups) return;  // (whole teams)
    const int g = (int)(id % a.ngroups), slot = (int)(id / a.ngroups);
    const int c0 = g * a.group;
    float dw[NV][V], dsc[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[i][v] = dsc[i][v] = 0.f;
    const bool need_x = !a.res.p || gate == kBefore || a.scale;
    int turn = 0;
    for (int64_t r64 = slot; r64 < a.rows; r64 += slots, turn ^= 1) {
        const int row = (int)r64;
        Raw<T, V> x[NV], z[NV], go[NV];
        Raw<TR, V> res[NV], dres[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (i * team + lane) * V, c = c0 + at;
            x[i].zero(), z[i].zero(), go[i].zero(), res[i].zero(), dres[i].zero();
            if (at < a.group) {
                go[i].load(a.dout.at(row, c));
                if (a.res.p) res[i].load(a.res.at(row, c));
                if (need_x) x[i].load(a.x.at(row, c));
                if (gate != kNone) z[i].load(a.z.at(row, c));
                if (a.dres.p) dres[i].load(a.dres.at(row, c));
            }
        }
        // the next row on its way to L2 meanwhile (4096 x 5120 gated: 71 us, 85 without; 512 columns: 32 and 33)
        if (r64 + slots < a.rows) {
            const int next = row + slots;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int at = (i * team + lane) * V, c = c0 + at;
                if (at < a.group) {
                    prefetch(a.dout.at(next, c));
                    if (a.res.p) prefetch(a.res.at(next, c));
                    if (need_x) prefetch(a.x.at(next, c));
                    if (gate != kNone) prefetch(a.z.at(next, c));
                    if (a.dres.p) prefetch(a.dres.at(next, c));
                }
            }
        }
        float s[NV][V], w[NV][V];
        float sums[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (i * team + lane) * V, c = c0 + at;
            float gw[V];
#pragma unroll
            for (int v = 0; v < V; ++v) w[i][v] = 0.f;
            if (at < a.group) load_param<V>(a.weight + c, w[i]);
            go[i].get(gw);
            if (a.res.p)
                res[i].get(s[i]);
            else
                x[i].get(s[i]);
            if (gate != kNone) {
                float f[V];
                z[i].get(f);
#pragma unroll
                for (int v = 0; v < V; ++v) f[v] = silu(f[v]);
                if (gate == kAfter) {
#pragma unroll
                    for (int v = 0; v < V; ++v) gw[v] *= f[v];
                } else if (!a.res.p) {
#pragma unroll
                    for (int v = 0; v < V; ++v) s[i][v] *= f[v];
                }
            }
            if (a.scale && !a.res.p && at < a.group) {
                float f[V];
                load_param<V>(a.scale + c, f);
#pragma unroll
                for (int v = 0; v < V; ++v) s[i][v] *= f[v];
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                sums[0] = fmaf(s[i][v], s[i][v], sums[0]);
                sums[1] = fmaf(gw[v] * w[i][v], s[i][v], sums[1]);
            }
        }
        team_sum<WARP, 2>(sums, smem[turn]);
        const float rstd = rsqrtf(fmaf(sums[0], a.inv_group, a.eps));
        const float proj = sums[1] * a.inv_group * rstd * rstd * rstd;  // mean(gw hat) rstd, per unit of s
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (i * team + lane) * V, c = c0 + at;
            if (at >= a.group) break;
            float zf[V], gf[V], dz[V], ds[V];
            go[i].get(gf);
            if (gate != kNone) z[i].get(zf);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float hat = s[i][v] * rstd;
                if (gate == kAfter) {
                    const float sg = sigmoid(zf[v]);
                    dz[v] = gf[v] * hat * w[i][v] * silu_slope(zf[v], sg);
                    gf[v] *= zf[v] * sg;
                }
                dw[i][v] = fmaf(gf[v], hat, dw[i][v]);
                ds[v] = fmaf(-proj, s[i][v], rstd * (gf[v] * w[i][v]));
            }
            if (a.res.p) {
                float f[V];
                dres[i].get(f);
#pragma unroll
                for (int v = 0; v < V; ++v) ds[v] += f[v];
                Raw<TR, V>::store(a.res_out.at(row, c), ds);
            }
            if (a.scale) {
                float f[V], xv[V];
                x[i].get(xv);
                load_param<V>(a.scale + c, f);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    dsc[i][v] = fmaf(ds[v], gate == kBefore ? xv[v] * silu(zf[v]) : xv[v], dsc[i][v]);
                    ds[v] *= f[v];
                }
            }
            if (gate == kBefore) {
                float xv[V];
                x[i].get(xv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float sg = sigmoid(zf[v]);
                    dz[v] = ds[v] * xv[v] * silu_slope(zf[v], sg);
                    ds[v] *= zf[v] * sg;
                }
            }
            Raw<T, V>::store(a.dx.at(row, c), ds);
            if (gate != kNone) Raw<T, V>::store(a.dz.at(row, c), dz);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i * team + lane) * V;
        if (at >= a.group) break;
        float *dst = a.partial + (int64_t)slot * 2 * a.dim + c0 + at;
#pragma unroll
        for (int v = 0; v < V; ++v) dst[v] = dw[i][v], dst[a.dim + v] = dsc[i][v];
    }
}

__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float *__restrict__ partial, int slots, int dim,
                                                           float *__restrict__ dweight, float *__restrict__ dscale) {
    __shared__ float red[32][32];
    const int c = blockIdx.x * 32 + threadIdx.x, k = blockIdx.y;
    float s = 0.f;
    if (c < dim)
#pragma unroll 4
        for (int q = threadIdx.y; q < slots; q += 32) s += partial[((int64_t)q * 2 + k) * dim + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < dim) {
#pragma unroll
        for (int q = 1; q < 32; ++q) s += red[q][threadIdx.x];
        float *dst = k ? dscale : dweight;
        if (dst) dst[c] = s;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int N>
using Int = std::integral_constant<int, N>;

// f(V, NV, WARP, GATE, threads): a warp a group for up to 512 values, for
// more a block of just enough warps; one value at a time where rows are not
// 16-byte aligned.
template <int VF, typename F>
ssd_status_t pick_team(int64_t group, bool vec, int gate, F f) {
    auto threads = [](int64_t n, int nv) { return (int)((n + 32 * nv - 1) / (32 * nv) * 32); };
    if (!vec) {
        if (group <= 8192) return f(Int<1>{}, Int<8>{}, Int<0>{}, Int<kAnyGate>{}, threads(group, 8));
        return f(Int<1>{}, Int<32>{}, Int<0>{}, Int<kAnyGate>{}, threads(group, 32));
    }
    constexpr int NV = 16 / VF;  // 16 values a thread
    const int64_t n = group / VF;
    if (group > 8192) return f(Int<VF>{}, Int<2 * NV>{}, Int<0>{}, Int<kAnyGate>{}, threads(n, 2 * NV));
    auto gated = [&](auto w, int t) {
        if (gate == kNone) return f(Int<VF>{}, Int<NV>{}, w, Int<kNone>{}, t);
        if (gate == kBefore) return f(Int<VF>{}, Int<NV>{}, w, Int<kBefore>{}, t);
        return f(Int<VF>{}, Int<NV>{}, w, Int<kAfter>{}, t);
    };
    return group <= 512 ? gated(Int<1>{}, 32) : gated(Int<0>{}, threads(n, NV));
}

ssd_status_t check(const ssd_norm_shape_t *s) {
    if (!s || s->rows < 0 || s->dim <= 0 || s->group_size <= 0 || s->dim % s->group_size != 0) return SSD_ERR_INVALID_ARG;
    if (s->dtype != SSD_DTYPE_F32 && s->dtype != SSD_DTYPE_BF16) return SSD_ERR_INVALID_ARG;
    if (s->residual_dtype != SSD_DTYPE_F32 && s->residual_dtype != s->dtype) return SSD_ERR_INVALID_ARG;
    if (!(s->eps >= 0.f)) return SSD_ERR_INVALID_ARG;
    if (s->group_size > kMaxGroup || s->dim > (1 << 24) || s->rows > (int64_t(1) << 31) - 1) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Teams that share the rows of a group of columns in the gradient: one wave
// of 12 warps an SM (warp teams) or of the blocks whose warps are 15 at most,
// of the 16 that the registers allow (21 M elements, bf16 with an fp32 residual
// and scale, as rows of 1024, 2048, 4096 and 5120: 77, 73, 75 and 75 us, although
// one block of 8 warps stands on an SM at 4096).
int64_t bwd_slots(const ssd_norm_shape_t *s) {
    const int64_t ngroups = s->dim / s->group_size, warps = (s->group_size + 511) / 512;
    const int64_t per_sm = warps == 1 ? 12 : warps < 15 ? 15 / warps : 1;
    int64_t slots = 152 * per_sm / ngroups;
    if (slots < 1) slots = 1;
    if (slots > s->rows) slots = s->rows;
    return slots;
}

bool row_ok(const ssd_rows_t &r, size_t es) { return rows_in_ok(r, es); }

template <typename T>
Mat<T> mat(const ssd_rows_t &r) {
    return {static_cast<T *>(r.data), (int)r.row_stride};
}

template <typename T, typename TR>
ssd_status_t fwd_typed(const ssd_norm_shape_t *s, const ssd_rows_t *x, const float *weight, const ssd_rows_t *z,
                       const ssd_rows_t *res, const float *scale, const ssd_rows_t *out, const ssd_rows_t *res_out,
                       cudaStream_t st) {
    NormArgs<T, TR> a{};
    a.x = mat<const T>(*x);
    if (z) a.z = mat<const T>(*z);
    if (res) {
        a.res = mat<const TR>(*res);
        a.res_out = mat<TR>(*res_out);
    }
    a.weight = weight, a.scale = scale;
    a.out = mat<T>(*out);
    a.rows = s->rows, a.dim = (int)s->dim, a.group = (int)s->group_size, a.ngroups = (int)(s->dim / s->group_size);
    a.eps = s->eps, a.inv_group = 1.f / (float)s->group_size;
    constexpr int VF = 16 / sizeof(T);
    const size_t es = sizeof(T);
    bool vec = s->group_size % VF == 0 && rows_vec(*x, es, 1, s->rows) && rows_vec(*out, es, 1, s->rows);
    if (z) vec = vec && rows_vec(*z, es, 1, s->rows);
    if (res) vec = vec && rows_vec(*res, sizeof(TR), 1, s->rows) && rows_vec(*res_out, sizeof(TR), 1, s->rows);
    vec = vec && aligned(weight, 16) && aligned(scale, 16);
    a.gate = !z ? kNone : s->gate_after ? kAfter : kBefore;
    return pick_team<VF>(s->group_size, vec, a.gate, [&](auto v, auto nv, auto w, auto gt, int threads) {
        constexpr int V = decltype(v)::value, NV = decltype(nv)::value, GATE = decltype(gt)::value;
        constexpr bool WARP = decltype(w)::value;
        const int64_t teams = s->rows * a.ngroups, blocks = WARP ? (teams + kWarpTeams - 1) / kWarpTeams : teams;
        if (blocks > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
        timing_begin(st);
        norm_fwd_kernel<T, TR, V, NV, WARP, GATE><<<(unsigned)blocks, WARP ? kWarpTeams * 32 : threads, 0, st>>>(a);
        timing_mark(st, "norm_fwd");
        return status_of(cudaGetLastError());
    });
}

template <typename T, typename TR>
ssd_status_t bwd_typed(const ssd_norm_shape_t *s, const ssd_rows_t *dout, const ssd_rows_t *x, const float *weight,
                       const ssd_rows_t *z, const float *scale, const ssd_rows_t *sum, const ssd_rows_t *dsum,
                       const ssd_rows_t *dx, float *dweight, const ssd_rows_t *dz, const ssd_rows_t *dres, float *dscale,
                       void *ws, cudaStream_t st) {
    NormArgs<T, TR> a{};
    a.x = mat<const T>(*x);
    if (z) {
        a.z = mat<const T>(*z);
        a.dz = mat<T>(*dz);
    }
    if (sum) {
        a.res = mat<const TR>(*sum);
        a.res_out = mat<TR>(*dres);
        if (dsum) a.dres = mat<const TR>(*dsum);
    }
    a.weight = weight, a.scale = scale;
    a.dout = mat<const T>(*dout);
    a.dx = mat<T>(*dx);
    a.partial = static_cast<float *>(ws);
    a.rows = s->rows, a.dim = (int)s->dim, a.group = (int)s->group_size, a.ngroups = (int)(s->dim / s->group_size);
    a.eps = s->eps, a.inv_group = 1.f / (float)s->group_size;
    constexpr int VF = 16 / sizeof(T);
    const size_t es = sizeof(T);
    bool vec = s->group_size % VF == 0 && rows_vec(*x, es, 1, s->rows) && rows_vec(*dout, es, 1, s->rows) &&
               rows_vec(*dx, es, 1, s->rows);
    if (z) vec = vec && rows_vec(*z, es, 1, s->rows) && rows_vec(*dz, es, 1, s->rows);
    if (sum) vec = vec && rows_vec(*sum, sizeof(TR), 1, s->rows) && rows_vec(*dres, sizeof(TR), 1, s->rows);
    if (dsum) vec = vec && rows_vec(*dsum, sizeof(TR), 1, s->rows);
    vec = vec && aligned(weight, 16) && aligned(scale, 16);
    a.gate = !z ? kNone : s->gate_after ? kAfter : kBefore;
    const int slots = (int)bwd_slots(s);
    timing_begin(st);
    if (slots > 0) {
        const ssd_status_t e = pick_team<VF>(s->group_size, vec, a.gate, [&](auto v, auto nv, auto w, auto gt, int threads) {
            constexpr int V = decltype(v)::value, NV = decltype(nv)::value, GATE = decltype(gt)::value;
            constexpr bool WARP = decltype(w)::value;
            const int64_t teams = (int64_t)slots * a.ngroups, blocks = WARP ? (teams + kWarpTeams - 1) / kWarpTeams : teams;
            if (blocks > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
            norm_bwd_kernel<T, TR, V, NV, WARP, GATE>
                <<<(unsigned)blocks, WARP ? kWarpTeams * 32 : threads, 0, st>>>(a, slots);
            timing_mark(st, "norm_bwd");
            return status_of(cudaGetLastError());
        });
        if (e != SSD_OK) return e;
    }
    norm_reduce_kernel<<<dim3((unsigned)((a.dim + 31) / 32), scale && dscale ? 2 : 1), dim3(32, 32), 0, st>>>(
        a.partial, slots, a.dim, dweight, dscale);
    timing_mark(st, "norm_reduce");
    return status_of(cudaGetLastError());
}

}  // namespace
}  // namespace ssd

extern "C" {

ssd_status_t ssd_block_norm_fwd(const ssd_norm_shape_t *shape, const ssd_rows_t *x, const float *weight,
                                const ssd_rows_t *z, const ssd_rows_t *residual, const float *scale,
                                const ssd_rows_t *out, const ssd_rows_t *residual_out, cudaStream_t stream) {
    using namespace ssd;
    const ssd_status_t st = check(shape);
    if (st != SSD_OK) return st;
    if (shape->rows == 0) return SSD_OK;
    const size_t es = dtype_size(shape->dtype), rs = dtype_size(shape->residual_dtype);
    if (!x || !weight || !out || !aligned(weight, 4) || !aligned(scale, 4) || !row_ok(*x, es) || (z && !row_ok(*z, es)))
        return SSD_ERR_INVALID_ARG;
    if (!rows_out_ok(*out, es, 1, shape->rows, shape->dim)) return SSD_ERR_INVALID_ARG;
    if (residual && (!row_ok(*residual, rs) || !residual_out || !rows_out_ok(*residual_out, rs, 1, shape->rows, shape->dim)))
        return SSD_ERR_INVALID_ARG;
    if (shape->dtype == SSD_DTYPE_F32)
        return fwd_typed<float, float>(shape, x, weight, z, residual, scale, out, residual_out, stream);
    if (shape->residual_dtype == SSD_DTYPE_F32)
        return fwd_typed<bf16, float>(shape, x, weight, z, residual, scale, out, residual_out, stream);
    return fwd_typed<bf16, bf16>(shape, x, weight, z, residual, scale, out, residual_out, stream);
}

size_t ssd_block_norm_bwd_workspace_size(const ssd_norm_shape_t *shape) {
    using namespace ssd;
    if (check(shape) != SSD_OK) return 0;
    return sizeof(float) * bwd_slots(shape) * 2 * shape->dim;
}

ssd_status_t ssd_block_norm_bwd(const ssd_norm_shape_t *shape, const ssd_rows_t *dout, const ssd_rows_t *x,
                                const float *weight, const ssd_rows_t *z, const float *scale,
                                const ssd_rows_t *residual_out, const ssd_rows_t *dresidual_out, const ssd_rows_t *dx,
                                float *dweight, const ssd_rows_t *dz, const ssd_rows_t *dresidual, float *dscale,
                                void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace ssd;
    const ssd_status_t st = check(shape);
    if (st != SSD_OK) return st;
    const size_t es = dtype_size(shape->dtype), rs = dtype_size(shape->residual_dtype);
    const int64_t rows = shape->rows, dim = shape->dim;
    if (!dout || !x || !weight || !dx || !aligned(weight, 4) || !aligned(scale, 4) || !aligned(dweight, 4) ||
        !aligned(dscale, 4))
        return SSD_ERR_INVALID_ARG;
    if ((z && !dz) || (residual_out && !dresidual) || (dresidual_out && !residual_out)) return SSD_ERR_INVALID_ARG;
    // a gradient of what is absent would be left unwritten
    if ((dz && !z) || (dresidual && !residual_out) || (dscale && !scale)) return SSD_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!row_ok(*dout, es) || !row_ok(*x, es) || !rows_out_ok(*dx, es, 1, rows, dim)) return SSD_ERR_INVALID_ARG;
        if (z && (!row_ok(*z, es) || !rows_out_ok(*dz, es, 1, rows, dim))) return SSD_ERR_INVALID_ARG;
        if (residual_out && (!row_ok(*residual_out, rs) || !rows_out_ok(*dresidual, rs, 1, rows, dim)))
            return SSD_ERR_INVALID_ARG;
        if (dresidual_out && !row_ok(*dresidual_out, rs)) return SSD_ERR_INVALID_ARG;
    }
    const size_t need = ssd_block_norm_bwd_workspace_size(shape);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return SSD_ERR_WORKSPACE;
    if (shape->dtype == SSD_DTYPE_F32)
        return bwd_typed<float, float>(shape, dout, x, weight, z, scale, residual_out, dresidual_out, dx, dweight, dz,
                                       dresidual, dscale, workspace, stream);
    if (shape->residual_dtype == SSD_DTYPE_F32)
        return bwd_typed<bf16, float>(shape, dout, x, weight, z, scale, residual_out, dresidual_out, dx, dweight, dz,
                                      dresidual, dscale, workspace, stream);
    return bwd_typed<bf16, bf16>(shape, dout, x, weight, z, scale, residual_out, dresidual_out, dx, dweight, dz,
                                 dresidual, dscale, workspace, stream);
}

}  // extern "C"
