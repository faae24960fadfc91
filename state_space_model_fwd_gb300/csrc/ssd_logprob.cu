// ssd_logprob.cu -- from rows of logits: the log-probability of a given
// token, the log of the sum of exponentials, the entropy, the top
// alternatives; and the gradient of the first three.
//
// A row is read once.  Each thread keeps the maximum m of what it has seen,
//   sum = sum e^(z - m)  and  moment = sum e^(z - m) (z - m) log2(e),
// rescaled where m grows; from the joined ones
//   lse = m + log(sum),  entropy = log(sum) - ln 2 moment / sum.
// Alternatives: the k-th largest of the maxima of groups of threads, tau, is
// not above the k-th largest element.  Only what the few threads hold whose
// maximum reaches tau is looked through again, and what reaches tau is ranked
// by (value, lowest index).
#include <cooperative_groups.h>

#include "ssd_logprob.cuh"

namespace ssd {
namespace {

namespace cg = cooperative_groups;

// A row is 100 KB: a block spends as long on joining its threads' statistics
// and on the alternatives as on loads, so small blocks, many of them, keep
// memory busy (forward and gradient of 8192 x 50280 bf16 / five alternatives of
// 2047 x 65537: eight blocks of 256 an SM 399 / 60 us, six 408 / 65, three of
// 512 419 / 70, two of 512 449 / 77, one of 1024 580 / 115).
constexpr int kThreads = 256, kBlocks = 8;
constexpr int kLoads = 4;  // in flight a thread (2: 404 / 58 us, 1: 438 / 71)
constexpr int kMaxTop = SSD_LOGPROB_MAX_TOP;
constexpr int kFound = 1024;  // candidates kept: above tau
constexpr int kSame = 512;    // and equal to it

template <typename T>
struct LogprobArgs {
    const T *logits;
    int64_t row_stride;
    T *dlogits;
    int64_t drow_stride;
    const int64_t *targets;
    float *logprob, *lse, *entropy, *top_logprob;
    int64_t *top_index;
    RowGradIn grad;
    int vocab, top, parts;
};

// The elements of a row as slots of 16 aligned bytes.  The first and the last slot may be cut; a part of a row is a range
// of slots.  What a cut slot has is read element by element.
template <typename T>
struct Slots {
    static constexpr int V = 16 / sizeof(T);
    const T *p;     // the row
    int skew, n;    // elements of slot 0 that lie before the row; the row's elements
    int lo, hi;     // this part's slots
    int full0, full1;  // and the whole ones among them
    __device__ __forceinline__ Slots(const T *row, int vocab, int part, int parts) {
        p = row, n = vocab;
        skew = (int)(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
        const int all = (skew + n + V - 1) / V;
        lo = (int)((int64_t)all * part / parts), hi = (int)((int64_t)all * (part + 1) / parts);
        full0 = lo == 0 && skew ? 1 : lo;
        full1 = hi == all && (skew + n) % V ? hi - 1 : hi;
        if (full1 < full0) full1 = full0;
    }
    __device__ __forceinline__ int first(int slot) const { return slot * V - skew; }  // its first element's index
    // f(index, element) for the elements of this part's cut slots that thread t has (t < V the first, 32 <= t < 32 + V the last)
    template <typename F>
    __device__ __forceinline__ void cut(int t, F &&f) const {
        if (t < V && full0 > lo) {
            const int i = first(lo) + t;
            if (i >= 0 && i < n) f(i, to_f32(p[i]));
        }
        if (t >= 32 && t < 32 + V && full1 < hi && hi - 1 >= full0) {
            const int i = first(hi - 1) + t - 32;
            if (i >= 0 && i < n) f(i, to_f32(p[i]));
        }
    }
    __device__ __forceinline__ Vec<T, V> load(int slot) const { return load_vec<T, V>(p + first(slot)); }
};

// Larger is larger; NaN is above everything, as in a sort; -0 is 0.
__device__ __forceinline__ unsigned key_of(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const unsigned u = __float_as_uint(v + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned key) {
    return key == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
// The larger value first, then the lower index.
__device__ __forceinline__ unsigned long long entry_of(float v, int index) {
    return (unsigned long long)key_of(v) << 32 | (0xFFFFFFFFu - (unsigned)index);
}

// tau is found among the maxima of groups of threads, twice as many as alternatives can be asked for: then about
// n log(n / (n - k)) <= 1.4 k elements reach it.
constexpr int kGroups = 2 * kMaxTop, kWide = kThreads / kGroups;
static_assert(kWide >= 1 && 32 % kWide == 0, "");

struct TopShared {
    unsigned maxima[kGroups];
    unsigned long long found[kFound + kSame];
    unsigned long long best[kMaxTop];  // sorted
    short threads[kThreads];
    unsigned tau;
    int above, equal, holders, warps[kThreads / 32];
};

// The k largest of the `n` entries, sorted, to best: each entry's rank is counted.
__device__ __forceinline__ void rank(const unsigned long long *e, int n, int k, unsigned long long *best) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
        int r = 0;
        for (int j = 0; j < n; ++j) r += e[j] > e[i];
        if (r < k) best[r] = e[i];
    }
}

// The largest key that k of a warp's values reach, bit by bit; the lower half of a bf16 value's key is zeros, a
// negative one's ones.
template <typename T, int N>
__device__ __forceinline__ unsigned reached_by(const unsigned (&v)[N], int k) {
    unsigned tau = 0;
    for (int bit = 31; bit >= (sizeof(T) == 2 ? 16 : 0); --bit) {
        const unsigned want = tau | 1u << bit;
        int n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) n += v[i] >= want;
        if ((int)__reduce_add_sync(0xffffffffu, n) >= k) tau = want;
    }
    return sizeof(T) == 2 && !(tau & 0x80000000u) ? tau | 0xFFFFu : tau;
}

// The part's k largest elements, sorted, in t.best (fewer elements: zeros, below every entry).  m: this thread's maximum.
template <typename T>
__device__ void top_of_part(const Slots<T> &s, float m, bool any, int k, TopShared &t) {
    constexpr int V = Slots<T>::V;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const unsigned mine = any ? key_of(m) : 0;
    unsigned g = mine;
#pragma unroll
    for (int d = 1; d < kWide; d *= 2) g = max(g, __shfl_xor_sync(0xffffffffu, g, d));
    if (tid % kWide == 0) t.maxima[tid / kWide] = g;
    if (tid < k) t.best[tid] = 0;
    if (tid == 0) t.above = t.equal = t.holders = 0;
    __syncthreads();
    if (warp == 0) {
        unsigned v[kGroups / 32];
#pragma unroll
        for (int i = 0; i < kGroups / 32; ++i) v[i] = t.maxima[i * 32 + lane];
        const unsigned tau = reached_by<T>(v, k);
        if (lane == 0) t.tau = tau;
    }
    __syncthreads();
    const unsigned tau = t.tau;
    auto look = [&](int i, float z) {
        const unsigned key = key_of(z);
        if (key < tau) return;
        if (key == tau) {
            const int at = atomicAdd(&t.equal, 1);
            if (at < kSame) t.found[kFound + at] = entry_of(z, i);
            return;
        }
        const int at = atomicAdd(&t.above, 1);
        if (at < kFound) t.found[at] = entry_of(z, i);
    };
    // The threads that hold something of tau or above; all threads share their slots.
    if (any && mine >= tau) {
        t.threads[atomicAdd(&t.holders, 1)] = (short)tid;
        s.cut(tid, look);
    }
    __syncthreads();
    {
        const int each = (s.full1 - s.full0 + kThreads - 1) / kThreads, n = t.holders * each;
        for (int q = tid; q < n; q += kThreads) {
            const int j = s.full0 + t.threads[q / each] + q % each * kThreads;
            if (j >= s.full1) continue;
            float z[V];
            widen<T, V>(s.load(j), z);
#pragma unroll
            for (int i = 0; i < V; ++i) look(s.first(j) + i, z[i]);
        }
    }
    __syncthreads();
    const int above = t.above, equal = t.equal;
    if (above + kSame <= kFound && equal <= kSame) {
        for (int i = tid; i < equal; i += kThreads) t.found[above + i] = t.found[kFound + i];
        __syncthreads();
        rank(t.found, above + equal, k, t.best);
        __syncthreads();
        return;
    }
    if (above + kMaxTop <= kFound) {
        // Of those that equal tau the first ones in the row: threads go through it in order until there are k.
        int have = above;
        const int first = max(s.first(s.lo), 0), last = min(s.first(s.hi), s.n);
        for (int i0 = first; i0 < last && have < k; i0 += kThreads * V) {
            // thread by thread V neighbouring elements
            float z[V];
            int n = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int at = i0 + tid * V + i;
                z[i] = at < last ? to_f32(s.p[at]) : 0.f;
                n += at < last && key_of(z[i]) == tau;
            }
            int before = n;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int o = __shfl_up_sync(0xffffffffu, before, d);
                if (lane >= d) before += o;
            }
            if (lane == 31) t.warps[warp] = before;
            __syncthreads();
            int total = 0, base = 0;
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) base += t.warps[w];
                total += t.warps[w];
            }
            int at = have + base + before - n;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int idx = i0 + tid * V + i;
                if (idx < last && key_of(z[i]) == tau) {
                    if (at < k) t.found[at] = entry_of(z[i], idx);
                    ++at;
                }
            }
            have = min(have + total, k);
            __syncthreads();
        }
        rank(t.found, max(have, above), k, t.best);
        __syncthreads();
        return;
    }
    // More above tau than there is room for (they sit in fewer than k threads): one after another, the largest below the last.
    unsigned long long last = 0;
    unsigned long long *part = t.found;
    for (int r = 0; r < k; ++r) {
        unsigned long long big = 0;
        auto look = [&](int i, float z) {
            const unsigned long long e = entry_of(z, i);
            if ((r == 0 || e < last) && e > big) big = e;  // (a NaN of the first token is the largest entry there is)
        };
        s.cut(tid, look);
        for (int j = s.full0 + tid; j < s.full1; j += kThreads) {
            float z[V];
            widen<T, V>(s.load(j), z);
#pragma unroll
            for (int i = 0; i < V; ++i) look(s.first(j) + i, z[i]);
        }
        for (int d = 16; d; d /= 2) {
            const unsigned long long o = __shfl_xor_sync(0xffffffffu, big, d);
            big = o > big ? o : big;
        }
        __syncthreads();
        if (lane == 0) part[warp] = big;
        __syncthreads();
        big = part[0];
        for (int w = 1; w < kThreads / 32; ++w) big = part[w] > big ? part[w] : big;
        if (tid == 0) t.best[r] = big;
        last = big;
    }
    __syncthreads();
}

template <int U>
__device__ __forceinline__ void add_vecs(Stat &st, const Vec<bf16, 8> (&v)[U]) {
    uint32_t w[4 * U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[4 * u] = v[u].r.x, w[4 * u + 1] = v[u].r.y, w[4 * u + 2] = v[u].r.z, w[4 * u + 3] = v[u].r.w;
    add_to(st, w);
}
template <int U>
__device__ __forceinline__ void add_vecs(Stat &st, const Vec<float, 4> (&v)[U]) {
    float z[4 * U];
#pragma unroll
    for (int u = 0; u < U; ++u) z[4 * u] = v[u].r.x, z[4 * u + 1] = v[u].r.y, z[4 * u + 2] = v[u].r.z, z[4 * u + 3] = v[u].r.w;
    add_to(st, z);
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, kBlocks) logprob_fwd_kernel(const __grid_constant__ LogprobArgs<T> a) {
    constexpr int V = Slots<T>::V;
    __shared__ Stat stats[kThreads / 32], joined;
    __shared__ std::conditional_t<TOP, TopShared, char> top;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, part = blockIdx.x % a.parts;
    const int64_t row = blockIdx.x / a.parts;
    const T *p = a.logits + row * a.row_stride;
    const Slots<T> s(p, a.vocab, part, a.parts);

    Stat st{-INFINITY, 0.f, 0.f};
    bool any = s.full0 + tid < s.full1;
    s.cut(tid, [&](int, float z) {
        const float one[1] = {z};
        add_to(st, one);
        any = true;
    });
    constexpr int U = kLoads;
    int j = s.full0 + tid;
    for (; j + (U - 1) * kThreads < s.full1; j += U * kThreads) {
        Vec<T, V> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = s.load(j + u * kThreads);
        add_vecs(st, v);
    }
    for (; j < s.full1; j += kThreads) {
        const Vec<T, V> v[1] = {s.load(j)};
        add_vecs(st, v);
    }
    const float mine = st.m;
    st = join_lanes<32>(st);
    if (lane == 0) stats[warp] = st;
    __syncthreads();
    if (warp == 0) {
        st = join_lanes<kThreads / 32>(stats[lane % (kThreads / 32)]);
        if (tid == 0) joined = st;
    }
    if constexpr (TOP) top_of_part(s, mine, any, a.top, top);

    if (a.parts > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        if (part == 0) {
            if (tid == 0) {
                st = joined;
                for (int q = 1; q < a.parts; ++q) st = join(st, *cluster.map_shared_rank(&joined, q));
            }
            if constexpr (TOP) {
                // a.parts sorted lists of a.top entries: into one and ranked
                const int n = a.parts * a.top;
                for (int i = tid; i < n; i += kThreads)
                    top.found[i] = cluster.map_shared_rank(&top.best[0], i / a.top)[i % a.top];
            }
        }
        cluster.sync();  // (no block ends before it was read)
        if (part) return;
        if constexpr (TOP) {
            rank(top.found, a.parts * a.top, a.top, top.best);
        }
    }
    if (tid == 0) {
        const float lse = lse_of(st);
        if (a.lse) a.lse[row] = lse;
        if (a.entropy) a.entropy[row] = entropy_of(st);
        if (a.logprob) {
            const int64_t t = a.targets[row];
            float v = 0.f;
            if (t >= a.vocab)
                v = __uint_as_float(0x7FC00000u);
            else if (t >= 0)
                v = logprob_of(to_f32(p[t]), lse);
            a.logprob[row] = v;
        }
        joined.m = lse;
    }
    if constexpr (TOP) {
        __syncthreads();
        const float lse = joined.m;
        if (tid < a.top) {
            const unsigned long long e = top.best[tid];
            a.top_logprob[row * a.top + tid] = logprob_of(value_of((unsigned)(e >> 32)), lse);
            a.top_index[row * a.top + tid] = (int64_t)(0xFFFFFFFFu - (unsigned)e);
        }
    }
}

template <typename T, bool ENT>
__global__ void __launch_bounds__(256) logprob_bwd_kernel(const __grid_constant__ LogprobArgs<T> a) {
    constexpr int V = Slots<T>::V, U = 4;
    const int64_t row = blockIdx.x / a.parts;
    const int part = blockIdx.x % a.parts;
    const T *p = a.logits + row * a.row_stride;
    T *d = a.dlogits + row * a.drow_stride;
    const Slots<T> s(p, a.vocab, part, a.parts);
    const RowGrad g = row_grad(a.grad, row, a.vocab);
    auto one = [&](int i, float z) {
        const float v = g.none ? 0.f : grad_of<ENT>(g, z) + (i == g.target ? g.dlp : 0.f);
        d[i] = from_f32<T>(v);
    };
    if ((reinterpret_cast<uintptr_t>(d) - reinterpret_cast<uintptr_t>(p)) % 16 != 0) {  // no common slots
        // Neighbouring elements in neighbouring threads, several in flight (8192 x 50277 from rows of 50304 376 us; one by one 873;
        // with common slots 271).
        constexpr int E = 8;
        const int first = max(s.first(s.lo), 0), last = min(s.first(s.hi), s.n);
        for (int i = first + threadIdx.x; i < last; i += E * 256) {
            T v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = p[min(i + e * 256, last - 1)];
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (i + e * 256 < last) one(i + e * 256, to_f32(v[e]));
        }
        return;
    }
    s.cut(threadIdx.x, one);
    for (int j = s.full0 + threadIdx.x; j < s.full1; j += U * 256) {
        Vec<T, V> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u * 256 < s.full1) v[u] = s.load(j + u * 256);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u * 256 >= s.full1) break;
            float z[V];
            widen<T, V>(v[u], z);
            const int i0 = s.first(j + u * 256);
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] = g.none ? 0.f : grad_of<ENT>(g, z[i]);
            if ((unsigned)(g.target - i0) < (unsigned)V && g.target >= 0 && !g.none) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i0 + i == g.target) z[i] += g.dlp;
            }
            store_vec<T, V>(d + i0, narrow<T, V>(z));
        }
    }
}

ssd_status_t check_logprob(const ssd_logprob_shape_t *s) {
    if (!s || s->rows < 0 || s->vocab <= 0 || s->top < 0 || s->top > s->vocab) return SSD_ERR_INVALID_ARG;
    if (s->dtype != SSD_DTYPE_F32 && s->dtype != SSD_DTYPE_BF16) return SSD_ERR_INVALID_ARG;
    if (s->top > kMaxTop || s->vocab > (1 << 30) || s->rows > (1 << 28)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

template <typename T>
ssd_status_t fwd_typed(const ssd_logprob_shape_t *s, const ssd_rows_t *logits, const int64_t *targets, float *logprob, float *lse,
                       float *entropy, float *top_logprob, int64_t *top_index, cudaStream_t st) {
    LogprobArgs<T> a{};
    a.logits = static_cast<const T *>(logits->data), a.row_stride = logits->row_stride;
    a.targets = targets, a.logprob = logprob, a.lse = lse, a.entropy = entropy;
    a.top_logprob = top_logprob, a.top_index = top_index;
    a.vocab = (int)s->vocab, a.top = (int)s->top;
    // Few long rows: up to four blocks, a cluster, share one (4 rows with eight alternatives in a graph: of 131072 15.5 us by
    // one block, 12.0 by two, 9.5 by four or eight; of 50280 9.5, -, 9.3, 10.4; of 8192 6.5 by one, 8.1 by two), as long as
    // that gives no SM more than two (152 rows of 50280: 10 us, by four blocks each 20).
    a.parts = 1;
    while (a.parts < 4 && s->rows * a.parts * 2 <= 2 * kSMs && s->vocab / (a.parts * 2) >= 12288) a.parts *= 2;
    timing_begin(st);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(s->rows * a.parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.parts, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.parts > 1 ? 1 : 0;
    const cudaError_t e = a.top ? cudaLaunchKernelEx(&cfg, logprob_fwd_kernel<T, true>, a)
                                : cudaLaunchKernelEx(&cfg, logprob_fwd_kernel<T, false>, a);
    timing_mark(st, "token_logprob");
    return status_of(e);
}

template <typename T>
ssd_status_t bwd_typed(const ssd_logprob_shape_t *s, const ssd_rows_t *logits, const int64_t *targets, const float *lse,
                       const float *entropy, const float *dlogprob, const float *dlse, const float *dentropy,
                       const ssd_rows_t *dlogits, cudaStream_t st) {
    LogprobArgs<T> a{};
    a.logits = static_cast<const T *>(logits->data), a.row_stride = logits->row_stride;
    a.dlogits = static_cast<T *>(dlogits->data), a.drow_stride = dlogits->row_stride;
    a.grad = RowGradIn{targets, lse, entropy, dlogprob, dlse, dentropy};
    a.vocab = (int)s->vocab;
    const int64_t per = 256 * 4 * Slots<T>::V;  // elements of a block: one round of loads
    a.parts = (int)((s->vocab + per - 1) / per);
    if (s->rows * a.parts > 0x7FFFFFFF) return SSD_ERR_UNSUPPORTED;
    timing_begin(st);
    const unsigned blocks = (unsigned)(s->rows * a.parts);
    if (dentropy)
        logprob_bwd_kernel<T, true><<<blocks, 256, 0, st>>>(a);
    else
        logprob_bwd_kernel<T, false><<<blocks, 256, 0, st>>>(a);
    timing_mark(st, "token_logprob_bwd");
    return status_of(cudaGetLastError());
}

}  // namespace
}  // namespace ssd

extern "C" {

ssd_status_t ssd_token_logprob_fwd(const ssd_logprob_shape_t *shape, const ssd_rows_t *logits, const int64_t *targets,
                                   float *logprob, float *lse, float *entropy, float *top_logprob, int64_t *top_index,
                                   cudaStream_t stream) {
    using namespace ssd;
    const ssd_status_t st = check_logprob(shape);
    if (st != SSD_OK) return st;
    if (shape->rows == 0) return SSD_OK;
    if (!logits || !far_rows_ok(*logits, dtype_size(shape->dtype)) || !aligned(targets, 8) || !aligned(logprob, 4) ||
        !aligned(lse, 4) || !aligned(entropy, 4) || !aligned(top_logprob, 4) || !aligned(top_index, 8))
        return SSD_ERR_INVALID_ARG;
    if ((logprob && !targets) || (shape->top && (!top_logprob || !top_index))) return SSD_ERR_INVALID_ARG;
    return shape->dtype == SSD_DTYPE_BF16
               ? fwd_typed<bf16>(shape, logits, targets, logprob, lse, entropy, top_logprob, top_index, stream)
               : fwd_typed<float>(shape, logits, targets, logprob, lse, entropy, top_logprob, top_index, stream);
}

ssd_status_t ssd_token_logprob_bwd(const ssd_logprob_shape_t *shape, const ssd_rows_t *logits, const int64_t *targets,
                                   const float *lse, const float *entropy, const float *dlogprob, const float *dlse,
                                   const float *dentropy, const ssd_rows_t *dlogits, cudaStream_t stream) {
    using namespace ssd;
    const ssd_status_t st = check_logprob(shape);
    if (st != SSD_OK) return st;
    if (shape->rows == 0) return SSD_OK;
    const size_t es = dtype_size(shape->dtype);
    if (!logits || !dlogits || !far_rows_ok(*logits, es) || !far_rows_out_ok(*dlogits, es, shape->rows, shape->vocab) || !lse ||
        !aligned(lse, 4) || !aligned(entropy, 4) || !aligned(targets, 8) || !aligned(dlogprob, 4) || !aligned(dlse, 4) ||
        !aligned(dentropy, 4))
        return SSD_ERR_INVALID_ARG;
    if ((dlogprob && !targets) || (dentropy && !entropy)) return SSD_ERR_INVALID_ARG;
    return shape->dtype == SSD_DTYPE_BF16
               ? bwd_typed<bf16>(shape, logits, targets, lse, entropy, dlogprob, dlse, dentropy, dlogits, stream)
               : bwd_typed<float>(shape, logits, targets, lse, entropy, dlogprob, dlse, dentropy, dlogits, stream);
}

}  // extern "C"
