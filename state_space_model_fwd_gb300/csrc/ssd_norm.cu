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
// for NV vectors each, so that few threads idle whatever the width.
#include <type_traits>

#include "ssd_layer.cuh"

namespace ssd {
namespace {

constexpr int64_t kMaxGroup = 32768;

enum Gate : int { kNone, kBefore, kAfter };

template <typename T, typename TR>
struct NormArgs {
    const T *x, *z;
    int64_t x_rs, z_rs;
    const TR *res;  // forward: the residual; gradient: the stored sum
    int64_t res_rs;
    const float *weight, *scale;
    T *out;
    int64_t out_rs;
    TR *res_out;  // forward: the sum; gradient: the residual's gradient
    int64_t res_out_rs;
    // gradient
    const T *dout;
    int64_t dout_rs;
    const TR *dres;  // gradient of the sum from elsewhere (null: zero)
    int64_t dres_rs;
    T *dx, *dz;
    int64_t dx_rs, dz_rs;
    float *partial;  // [slots][2][dim]: dweight, dscale
    int64_t rows;
    int dim, group, ngroups, gate;
    float eps;
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

// Sum over a team: a warp, or the whole block.
template <bool WARP, int R>
__device__ __forceinline__ void team_sum(float (&v)[R], float *smem) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], off);
    if constexpr (!WARP) {
        const int warps = blockDim.x / 32;
        __syncthreads();
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) smem[threadIdx.x / 32 * R + r] = v[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = 0.f;
        for (int w = 0; w < warps; ++w)
#pragma unroll
            for (int r = 0; r < R; ++r) v[r] += smem[w * R + r];
    }
}

constexpr int kWarpTeams = 4;  // warp teams per block

// NV vectors of V values per thread cover the group.
template <typename T, typename TR, int V, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarpTeams * 32 : V == 1 || NV * V > 16 ? 1024 : 512, 1)
    norm_fwd_kernel(const __grid_constant__ NormArgs<T, TR> a) {
    __shared__ float smem[32];
    const int team = WARP ? 32 : blockDim.x, lane = WARP ? threadIdx.x % 32 : threadIdx.x;
    const int64_t id = WARP ? (int64_t)blockIdx.x * kWarpTeams + threadIdx.x / 32 : blockIdx.x;
    if (id >= a.rows * a.ngroups) return;  // (whole teams)
    const int64_t row = id / a.ngroups;
    const int c0 = (int)(id % a.ngroups) * a.group;
    Raw<T, V> x[NV], z[NV];
    Raw<TR, V> res[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i * team + lane) * V, c = c0 + at;
        x[i].zero(), z[i].zero(), res[i].zero();
        if (at < a.group) {
            x[i].load(a.x + row * a.x_rs + c);
            if (a.gate != kNone) z[i].load(a.z + row * a.z_rs + c);
            if (a.res) res[i].load(a.res + row * a.res_rs + c);
        }
    }
    float s[NV][V];
    float sq[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i * team + lane) * V, c = c0 + at;
        x[i].get(s[i]);
        if (a.gate == kBefore) {
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
        if (a.res) {
            float f[V];
            res[i].get(f);
#pragma unroll
            for (int v = 0; v < V; ++v) s[i][v] += f[v];
            if (at < a.group) Raw<TR, V>::store(a.res_out + row * a.res_out_rs + c, s[i]);
        }
        // (vectors past the group are zero)
#pragma unroll
        for (int v = 0; v < V; ++v) sq[0] = fmaf(s[i][v], s[i][v], sq[0]);
    }
    team_sum<WARP, 1>(sq, smem);
    const float rstd = rsqrtf(sq[0] / (float)a.group + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int at = (i * team + lane) * V, c = c0 + at;
        if (at >= a.group) break;
        float w[V];
        load_param<V>(a.weight + c, w);
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] *= s[i][v] * rstd;
        if (a.gate == kAfter) {
            float f[V];
            z[i].get(f);
#pragma unroll
            for (int v = 0; v < V; ++v) w[v] *= silu(f[v]);
        }
        Raw<T, V>::store(a.out + row * a.out_rs + c, w);
    }
}

// Gradient.  With hat = s rstd and gw = dout (silu z) w:
//   ds = rstd (gw - hat mean(gw hat)) + dres,  both means from one reduction;
//   dresidual = ds, dv = scale ds, dscale = sum_rows ds v, dweight = sum_rows dout (silu z) hat.
// A team walks rows of its own group of columns, its column sums in
// registers; the teams' partial sums are added by a second kernel in a fixed
// order.
template <typename T, typename TR, int V, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? kWarpTeams * 32 : V == 1 || NV * V > 16 ? 1024 : 512, 1)
    norm_bwd_kernel(const __grid_constant__ NormArgs<T, TR> a, int slots) {
    __shared__ float smem[64];
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
    const bool need_x = !a.res || a.gate == kBefore || a.scale;
    for (int64_t row = slot; row < a.rows; row += slots) {
        Raw<T, V> x[NV], z[NV], go[NV];
        Raw<TR, V> res[NV], dres[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (i * team + lane) * V, c = c0 + at;
            x[i].zero(), z[i].zero(), go[i].zero(), res[i].zero(), dres[i].zero();
            if (at < a.group) {
                go[i].load(a.dout + row * a.dout_rs + c);
                if (a.res) res[i].load(a.res + row * a.res_rs + c);
                if (need_x) x[i].load(a.x + row * a.x_rs + c);
                if (a.gate != kNone) z[i].load(a.z + row * a.z_rs + c);
                if (a.dres) dres[i].load(a.dres + row * a.dres_rs + c);
            }
        }
        float s[NV][V];
        float sums[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (i * team + lane) * V, c = c0 + at;
            float gw[V];
            go[i].get(gw);
            if (a.res)
                res[i].get(s[i]);
            else
                x[i].get(s[i]);
            if (a.gate != kNone) {
                float f[V];
                z[i].get(f);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float gate = silu(f[v]);
                    if (a.gate == kAfter)
                        gw[v] *= gate;
                    else if (!a.res)
                        s[i][v] *= gate;
                }
            }
            if (at < a.group) {
                float f[V];
                if (a.scale && !a.res) {
                    load_param<V>(a.scale + c, f);
#pragma unroll
                    for (int v = 0; v < V; ++v) s[i][v] *= f[v];
                }
                load_param<V>(a.weight + c, f);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    sums[0] = fmaf(s[i][v], s[i][v], sums[0]);
                    sums[1] = fmaf(gw[v] * f[v], s[i][v], sums[1]);
                }
            }
        }
        team_sum<WARP, 2>(sums, smem);
        const float rstd = rsqrtf(sums[0] / (float)a.group + a.eps);
        const float proj = sums[1] / (float)a.group * rstd * rstd;  // mean(gw hat) rstd, per unit of s
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (i * team + lane) * V, c = c0 + at;
            if (at >= a.group) break;
            float zf[V], f[V], gf[V], dz[V], ds[V];
            go[i].get(gf);
            z[i].get(zf);
            load_param<V>(a.weight + c, f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float hat = s[i][v] * rstd;
                if (a.gate == kAfter) {
                    const float sg = sigmoid(zf[v]);
                    dz[v] = gf[v] * hat * f[v] * silu_slope(zf[v], sg);
                    gf[v] *= zf[v] * sg;
                }
                dw[i][v] = fmaf(gf[v], hat, dw[i][v]);
                ds[v] = rstd * (gf[v] * f[v] - s[i][v] * proj);
            }
            if (a.res) {
                dres[i].get(f);
#pragma unroll
                for (int v = 0; v < V; ++v) ds[v] += f[v];
                Raw<TR, V>::store(a.res_out + row * a.res_out_rs + c, ds);
            }
            float xv[V];
            x[i].get(xv);
            if (a.scale) {
                load_param<V>(a.scale + c, f);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    dsc[i][v] = fmaf(ds[v], a.gate == kBefore ? xv[v] * silu(zf[v]) : xv[v], dsc[i][v]);
                    ds[v] *= f[v];
                }
            }
            if (a.gate == kBefore) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float sg = sigmoid(zf[v]);
                    dz[v] = ds[v] * xv[v] * silu_slope(zf[v], sg);
                    ds[v] *= zf[v] * sg;
                }
            }
            Raw<T, V>::store(a.dx + row * a.dx_rs + c, ds);
            if (a.gate != kNone) Raw<T, V>::store(a.dz + row * a.dz_rs + c, dz);
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

__global__ void __launch_bounds__(256) norm_reduce_kernel(const float *__restrict__ partial, int slots, int dim,
                                                          float *__restrict__ dweight, float *__restrict__ dscale) {
    __shared__ float red[8][32];
    const int c = blockIdx.x * 32 + threadIdx.x, k = blockIdx.y;
    float s = 0.f;
    if (c < dim)
        for (int q = threadIdx.y; q < slots; q += 8) s += partial[((int64_t)q * 2 + k) * dim + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < dim) {
#pragma unroll
        for (int q = 1; q < 8; ++q) s += red[q][threadIdx.x];
        float *dst = k ? dscale : dweight;
        if (dst) dst[c] = s;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int N>
using Int = std::integral_constant<int, N>;

// f(V, NV, WARP, threads): a warp a group for up to 512 values, for more a
// block of just enough warps; one value at a time where rows are not 16-byte
// aligned.
template <int VF, typename F>
ssd_status_t pick_team(int64_t group, bool vec, F f) {
    auto threads = [](int64_t n, int nv) { return (int)((n + 32 * nv - 1) / (32 * nv) * 32); };
    if (!vec) {
        if (group <= 8192) return f(Int<1>{}, Int<8>{}, Int<0>{}, threads(group, 8));
        return f(Int<1>{}, Int<32>{}, Int<0>{}, threads(group, 32));
    }
    constexpr int NV = 16 / VF;    // 16 values a thread
    const int64_t n = group / VF;  // vectors
    if (group <= 512) return f(Int<VF>{}, Int<NV>{}, Int<1>{}, 32);
    if (group <= 8192) return f(Int<VF>{}, Int<NV>{}, Int<0>{}, threads(n, NV));
    return f(Int<VF>{}, Int<2 * NV>{}, Int<0>{}, threads(n, 2 * NV));
}

ssd_status_t check(const ssd_norm_shape_t *s) {
    if (!s || s->rows < 0 || s->dim <= 0 || s->group_size <= 0 || s->dim % s->group_size != 0) return SSD_ERR_INVALID_ARG;
    if (s->dtype != SSD_DTYPE_F32 && s->dtype != SSD_DTYPE_BF16) return SSD_ERR_INVALID_ARG;
    if (s->residual_dtype != SSD_DTYPE_F32 && s->residual_dtype != s->dtype) return SSD_ERR_INVALID_ARG;
    if (!(s->eps >= 0.f)) return SSD_ERR_INVALID_ARG;
    if (s->group_size > kMaxGroup || s->dim > (1 << 24) || s->rows > (int64_t(1) << 31) - 1) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Teams that share the rows of a group of columns in the gradient: enough to
// fill the SMs (16 warps each), one at least for each row where there are few.
int64_t bwd_slots(const ssd_norm_shape_t *s) {
    const int64_t ngroups = s->dim / s->group_size, warps = (s->group_size + 511) / 512;
    int64_t slots = 152 * 16 / (ngroups * warps);
    if (slots < 1) slots = 1;
    if (slots > s->rows) slots = s->rows;
    return slots;
}

bool row_ok(const ssd_rows_t &r, size_t es) { return rows_in_ok(r, es); }

template <typename T, typename TR>
ssd_status_t fwd_typed(const ssd_norm_shape_t *s, const ssd_rows_t *x, const float *weight, const ssd_rows_t *z,
                       const ssd_rows_t *res, const float *scale, const ssd_rows_t *out, const ssd_rows_t *res_out,
                       cudaStream_t st) {
    NormArgs<T, TR> a{};
    a.x = static_cast<const T *>(x->data), a.x_rs = x->row_stride;
    if (z) a.z = static_cast<const T *>(z->data), a.z_rs = z->row_stride;
    if (res) {
        a.res = static_cast<const TR *>(res->data), a.res_rs = res->row_stride;
        a.res_out = static_cast<TR *>(res_out->data), a.res_out_rs = res_out->row_stride;
    }
    a.weight = weight, a.scale = scale;
    a.out = static_cast<T *>(out->data), a.out_rs = out->row_stride;
    a.rows = s->rows, a.dim = (int)s->dim, a.group = (int)s->group_size, a.ngroups = (int)(s->dim / s->group_size);
    a.eps = s->eps;
    constexpr int VF = 16 / sizeof(T);
    const size_t es = sizeof(T);
    bool vec = s->group_size % VF == 0 && rows_vec(*x, es, 1, s->rows) && rows_vec(*out, es, 1, s->rows);
    if (z) vec = vec && rows_vec(*z, es, 1, s->rows);
    if (res) vec = vec && rows_vec(*res, sizeof(TR), 1, s->rows) && rows_vec(*res_out, sizeof(TR), 1, s->rows);
    vec = vec && aligned(weight, 16) && aligned(scale, 16);
    a.gate = !z ? kNone : s->gate_after ? kAfter : kBefore;
    return pick_team<VF>(s->group_size, vec, [&](auto v, auto nv, auto w, int threads) {
        constexpr int V = decltype(v)::value, NV = decltype(nv)::value;
        constexpr bool WARP = decltype(w)::value;
        const int64_t teams = s->rows * a.ngroups, blocks = WARP ? (teams + kWarpTeams - 1) / kWarpTeams : teams;
        if (blocks > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
        timing_begin(st);
        norm_fwd_kernel<T, TR, V, NV, WARP><<<(unsigned)blocks, WARP ? kWarpTeams * 32 : threads, 0, st>>>(a);
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
    a.x = static_cast<const T *>(x->data), a.x_rs = x->row_stride;
    if (z) {
        a.z = static_cast<const T *>(z->data), a.z_rs = z->row_stride;
        a.dz = static_cast<T *>(dz->data), a.dz_rs = dz->row_stride;
    }
    if (sum) {
        a.res = static_cast<const TR *>(sum->data), a.res_rs = sum->row_stride;
        a.res_out = static_cast<TR *>(dres->data), a.res_out_rs = dres->row_stride;
        if (dsum) a.dres = static_cast<const TR *>(dsum->data), a.dres_rs = dsum->row_stride;
    }
    a.weight = weight, a.scale = scale;
    a.dout = static_cast<const T *>(dout->data), a.dout_rs = dout->row_stride;
    a.dx = static_cast<T *>(dx->data), a.dx_rs = dx->row_stride;
    a.partial = static_cast<float *>(ws);
    a.rows = s->rows, a.dim = (int)s->dim, a.group = (int)s->group_size, a.ngroups = (int)(s->dim / s->group_size);
    a.eps = s->eps;
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
        const ssd_status_t e = pick_team<VF>(s->group_size, vec, [&](auto v, auto nv, auto w, int threads) {
            constexpr int V = decltype(v)::value, NV = decltype(nv)::value;
            constexpr bool WARP = decltype(w)::value;
            const int64_t teams = (int64_t)slots * a.ngroups, blocks = WARP ? (teams + kWarpTeams - 1) / kWarpTeams : teams;
            if (blocks > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
            norm_bwd_kernel<T, TR, V, NV, WARP>
                <<<(unsigned)blocks, WARP ? kWarpTeams * 32 : threads, 0, st>>>(a, slots);
            timing_mark(st, "norm_bwd");
            return status_of(cudaGetLastError());
        });
        if (e != SSD_OK) return e;
    }
    norm_reduce_kernel<<<dim3((unsigned)((a.dim + 31) / 32), scale && dscale ? 2 : 1), dim3(32, 8), 0, st>>>(
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
