// ssd_layer.cuh -- what the operators around the scan share: strided rows,
// packed-sequence tables, small device math and host checks.
#pragma once

#include <utility>

#include "ssd_common.cuh"

namespace ssd {

// ---------------------------------------------------------------------------
// device math
// ---------------------------------------------------------------------------
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// 1 / (1 + exp(-v)); exp(-v) overflows to inf for v < -88, whose reciprocal
// is the limit 0.
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(-kLog2e * v)); }
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
// d/dv [v sigmoid(v)] given s = sigmoid(v)
__device__ __forceinline__ float silu_slope(float v, float s) { return s * fmaf(v, 1.f - s, 1.f); }

// ---------------------------------------------------------------------------
// V consecutive elements as fp32: one access of 16 bytes (8 for bf16 with
// V = 4), or one element (V = 1) where rows are not 16-byte aligned.
// ---------------------------------------------------------------------------
template <typename T, int V>
struct Vec {
    T e[V];
};
template <>
struct Vec<bf16, 8> {
    uint4 r;
};
template <>
struct Vec<bf16, 4> {
    uint2 r;
};
template <>
struct Vec<float, 4> {
    float4 r;
};

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T *p) {
    Vec<T, V> v;
    if constexpr (V == 1)
        v.e[0] = *p;
    else
        v.r = *reinterpret_cast<const decltype(v.r) *>(p);
    return v;
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> zero_vec() {
    Vec<T, V> v;
    if constexpr (V == 1)
        v.e[0] = from_f32<T>(0.f);
    else if constexpr (V == 8)
        v.r = make_uint4(0, 0, 0, 0);
    else if constexpr (sizeof(T) == 2)
        v.r = make_uint2(0, 0);
    else
        v.r = make_float4(0.f, 0.f, 0.f, 0.f);
    return v;
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const Vec<T, V> &v) {
    if constexpr (V == 1)
        *p = v.e[0];
    else
        *reinterpret_cast<decltype(v.r) *>(p) = v.r;
}
template <typename T, int V>
__device__ __forceinline__ void widen(const Vec<T, V> &v, float *f) {
    if constexpr (V == 1) {
        f[0] = to_f32(v.e[0]);
    } else if constexpr (V == 8) {
        const uint32_t w[4] = {v.r.x, v.r.y, v.r.z, v.r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else if constexpr (sizeof(T) == 2) {
        f[0] = __uint_as_float(v.r.x << 16), f[1] = __uint_as_float(v.r.x & 0xFFFF0000u);
        f[2] = __uint_as_float(v.r.y << 16), f[3] = __uint_as_float(v.r.y & 0xFFFF0000u);
    } else {
        f[0] = v.r.x, f[1] = v.r.y, f[2] = v.r.z, f[3] = v.r.w;
    }
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> narrow(const float *f) {
    Vec<T, V> v;
    if constexpr (V == 1) {
        v.e[0] = from_f32<T>(f[0]);
    } else if constexpr (V == 8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        v.r = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 h0 = __floats2bfloat162_rn(f[0], f[1]), h1 = __floats2bfloat162_rn(f[2], f[3]);
        v.r = make_uint2(*reinterpret_cast<const uint32_t *>(&h0), *reinterpret_cast<const uint32_t *>(&h1));
    } else {
        v.r = make_float4(f[0], f[1], f[2], f[3]);
    }
    return v;
}

template <typename T>
struct Rows {
    T *p;
    int64_t bs;  // elements between batch rows
    int rs;      // and between tokens (32 bits: one multiplication an address)
    __device__ __forceinline__ int64_t step(int tokens) const { return (int64_t)tokens * rs; }
    __device__ __forceinline__ T *at(int64_t b, int t) const { return p + b * bs + step(t); }
};

// Programmatic dependency between the launches of one call: a kernel lets the
// next one start once all its blocks run, and waits for the whole of the
// previous one (and so, one after another, of all before it) before it reads
// what that wrote.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------------------
// host checks
// ---------------------------------------------------------------------------
// `after`: with a programmatic dependency on the launch before.  A call's first
// launch has none, so it waits for everything before it on the stream.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, bool after, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

inline ssd_status_t status_of(cudaError_t e) {
    if (e == cudaSuccess) return SSD_OK;
    (void)cudaGetLastError();  // a failed call also records itself as the thread's last error
    return SSD_ERR_CUDA;
}

inline bool aligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

inline size_t dtype_size(ssd_dtype_t t) { return t == SSD_DTYPE_BF16 ? 2 : 4; }

constexpr int kSMs = 152;

constexpr int64_t kMaxBatchStride = int64_t(1) << 40;  // keeps every offset far inside 63 bits
constexpr int64_t kMaxRowStride = int64_t(1) << 31;

// A readable array of rows: element-aligned, strides not negative.
inline bool rows_in_ok(const ssd_rows_t &r, size_t esize) {
    return r.data && aligned(r.data, esize) && r.batch_stride >= 0 && r.row_stride >= 0 && r.batch_stride < kMaxBatchStride &&
           r.row_stride < kMaxRowStride;
}
// A writable one: no two rows share an element.
inline bool rows_out_ok(const ssd_rows_t &r, size_t esize, int64_t b, int64_t L, int64_t cols) {
    if (!rows_in_ok(r, esize)) return false;
    const __int128 rs = r.row_stride, bs = r.batch_stride;
    if (L > 1 && rs < cols) return false;
    if (b > 1 && bs < cols) return false;
    return b <= 1 || L <= 1 || bs >= (L - 1) * rs + cols || rs >= (b - 1) * bs + cols;
}
// Whether every row starts on a 16-byte boundary.
inline bool rows_vec(const ssd_rows_t &r, size_t esize, int64_t b, int64_t L) {
    return aligned(r.data, 16) && (b <= 1 || r.batch_stride * esize % 16 == 0) && (L <= 1 || r.row_stride * esize % 16 == 0);
}

// A packed batch's offsets: 0 first, total last, non-decreasing.
inline bool offsets_ok(const int64_t *cu, int64_t nseq, int64_t total) {
    if (nseq < 0 || cu[0] != 0 || cu[nseq] != total) return false;
    for (int64_t s = 0; s < nseq; ++s)
        if (cu[s + 1] < cu[s]) return false;
    return true;
}

template <typename T>
inline Rows<T> rows_of(const ssd_rows_t &r) {
    return {static_cast<T *>(r.data), r.batch_stride, (int)r.row_stride};
}

}  // namespace ssd
