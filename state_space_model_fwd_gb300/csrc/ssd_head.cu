// ssd_head.cu -- the head's log-probabilities: z = hidden weight^T is formed
// tile by tile on the tensor cores and never stored; what a row of logits is
// needed for is taken from the accumulator.  The gradient forms z again, stores
// dz in bf16 and multiplies it with the weights and with the hidden states.
//
// All products run in one kernel: a block (one on each SM) walks over tiles of
// 128 rows and up to 256 columns.  One warp copies operands by TMA into a ring
// of stages, one issues the MMAs into one of two accumulators in TMEM, eight
// read the other accumulator meanwhile, half a row of the tile a thread, and
// store bf16 results by TMA.
//
// Where there are rows enough, two blocks, a cluster on neighbouring SMs, share
// tiles of 256 rows (PAIR): each copies its 128 rows of A and half of B, the
// first one's MMAs read both, and each has its 128 rows of the sum in its own
// TMEM.  B's copies and reads are halved.
//
// The tensor cores add into fp32 with truncation, so a sum over K comes out
// too small by 2^-25 or so of itself for every 16 of K: 2.6e-6 at K = 2560,
// which scales all logits alike and shows in the entropy (1.2e-6 of it).  A
// tile's sum of logits is therefore taken in shares of at most kShare chunks,
// which are added in registers with rounding: 5.5e-7, for 856 instead of 839 us
// at 8192 x 2560 x 32000 (16 chunks: 884 us).  The gradient takes the same
// shares (4095 x 2560 x 50277: 694 us for 681): p = exp(z - lse) needs the z that
// is in lse.  Where a given token is nearly certain its dz, dlogprob (1 - p), is
// a difference of the two, and 2.6e-6 of z = 30 would be 80% of it at p = 0.9999.
//
// What bounds it: the tensor cores under the power limit (1.05 TFLOP for dz in
// 640 us, 1.65 PFLOP/s; a library product sustains 1.71).  Pairs: forward and
// gradient of 4095 x 2560 x 50277 2617 us, single blocks 2928.  Below dim 512
// or so the readers bound it: 8192 x 128 x 32000 in 94 us, 4.5 instructions and
// one exponential a logit with two warps a scheduler (storing by thread and
// taking the maximum anew every 16 columns: 243).  With few rows the weights'
// one pass does: 16 x 2560 x 50280 in 51 us, 38 at the copy rate.
#include <cudaTypedefs.h>

#include "ssd_logprob.cuh"
#include "ssd_status.h"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

using namespace tc;

constexpr int kBM = 128, kBN = 256, kBK = 64;
constexpr int kMaxStages = 8, kRing = 4 * (kBM + kBN) * kBK * 2;  // bytes of the ring: four stages of full tiles
constexpr int kReaders = 8;  // warps that read the accumulators, 32 rows and half of the columns each
constexpr int kSmem = kRing + kReaders * 4096 + 1024;
constexpr int kShare = 20;      // chunks of K
constexpr int kLongest = 4096;  // and at most in one sum of the gradient: 2.7e-4 too small, a tenth of a step of its bf16 result
constexpr uint64_t kWaitNs = 100000000ull;
constexpr int kNoLead = 0x7FFFFFFF;  // above every row

// What becomes of an accumulator: statistics of the logits, their gradient (of sums in one share, or in several), the product.
enum Use { kStats, kGrad, kGradShares, kStore };
constexpr int kGemmThreads = 128 + 32 * kReaders;  // warps: copy, MMA, TMEM, -, the readers

// dz is rounded to bf16 (2^-8 relative at most, as its products' other operands are), which would show where one element
// outweighs all others: the given token's.  What its rounding left, `rest`, is kept in fp32 and added to the products:
//   dhidden[row] += rest[row] weight[target[row]],   dweight[v] += sum over rows with target v of rest[row] hidden[row],
// the latter summed by head_fix_kernel and found by way of lead[v], one of those rows.  (4095 x 2560 x 50277: error against
// 64 bits 1.4 times a bf16 rounding without it, 1.0 with it, for 1% of the time; with few rows up to 1.8 times.)
struct Fix {
    const int64_t *targets;  // dhidden
    const float *rest;
    const bf16 *weight;
    int64_t weight_pitch;
    int vocab;
    const int *lead;         // dweight
    const float *sums;
    int64_t dim;
};
// What is added to 8 columns of a row of the product: a multiple of the given token's weights, or a row of the sums.
struct FixRow {
    const bf16 *w;
    const float *e;
    float scale;
};
__device__ __forceinline__ FixRow fix_row(const Fix &f, int row, bool live) {
    FixRow r{nullptr, nullptr, 0.f};
    if (!live) return r;
    if (f.targets) {
        const int64_t t = f.targets[row];
        if (t >= 0 && t < f.vocab) r.w = f.weight + t * f.weight_pitch, r.scale = f.rest[row];
    } else if (f.lead) {
        const int first = f.lead[row];
        if (first != kNoLead) r.e = f.sums + first * f.dim;
    }
    return r;
}
__device__ __forceinline__ void fix_add(const FixRow &r, int col, float *z) {  // 8 columns
    if (r.w) {
        float w[8];
        widen<bf16, 8>(load_vec<bf16, 8>(r.w + col), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = fmaf(r.scale, w[i], z[i]);
    } else if (r.e) {
        const float4 a = *reinterpret_cast<const float4 *>(r.e + col), b = *reinterpret_cast<const float4 *>(r.e + col + 4);
        z[0] += a.x, z[1] += a.y, z[2] += a.z, z[3] += a.w, z[4] += b.x, z[5] += b.y, z[6] += b.z, z[7] += b.w;
    }
}

struct GemmArgs {
    int M, N, K;          // D[M, N] = A[M, K] B[N, K]^T
    int pair;             // tiles of 256 rows, two blocks each
    int bn, mt, nt, kc;   // columns of a tile; tiles; chunks of kBK
    int arows;            // rows that are copied of a row tile: what lies behind them is read, and only by rows that are none
    int stages, abytes, stage_bytes;
    int shares;           // of K, for the statistics
    int group;            // row tiles that are walked together before the next column tile
    int units, whole, split;  // the first `whole` tiles are a unit each, the others `split` units, a share of K each
    // kStats, kGrad: rows are tokens, columns the vocabulary
    const int64_t *targets;
    float4 *stats;        // [nt][halves][M] (m, sum, moment, 0)
    float *given;         // [M] the given tokens' logits
    RowGradIn grad;
    float *rest;          // [M] what rounding left of the given token's dz (0 without one)
    int *lead;            // [N] set to kNoLead (null: not wanted)
    // kStore
    bf16 *out;
    int64_t out_pitch;
    Fix fix;
    float *parts;         // [units - whole][rows of a tile][bn] of the tiles that are split
    unsigned *status;
};

struct Unit {
    int m, n, k0, k1, part;  // part < 0: a whole tile
};
__device__ __forceinline__ Unit unit_of(const GemmArgs &a, int u) {
    Unit r;
    int tile = u;
    r.k0 = 0, r.k1 = a.kc, r.part = -1;
    if (u >= a.whole) {
        const int e = u - a.whole, q = e % a.split;
        tile = a.whole + e / a.split;
        r.part = e;
        r.k0 = (int)((int64_t)a.kc * q / a.split), r.k1 = (int)((int64_t)a.kc * (q + 1) / a.split);
    }
    const int per = a.group * a.nt, g = tile / per, in = tile % per, gm = min(a.group, a.mt - g * a.group);
    r.m = g * a.group + in % gm, r.n = in / gm;
    return r;
}

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}

// ---- the pair: this block's number in it, the first one's address of something in shared memory, the barrier of both
__device__ __forceinline__ uint32_t pair_rank() {
    uint32_t r;
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t at_first(const void *p) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}
__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// A copy into this block's memory that counts on a barrier of the pair's first block.
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    if (accumulate)
        asm volatile("tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, 1;" ::"r"(d), "l"(a), "l"(b), "r"(idesc) : "memory");
    else
        asm volatile("tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, 0;" ::"r"(d), "l"(a), "l"(b), "r"(idesc) : "memory");
}
// Arrives on the same barrier of both blocks (or of this one) once the MMAs issued so far are complete.
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}
__device__ __forceinline__ void mma_commit_pair_here(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
                 "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(smem_u32(dst)),
                 "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages], ready[2], taken[2], drain;
    uint32_t tmem;
    int gave_up;
};
// False once any wait of the block has given up.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, Bars *b) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity, 20000)) return true;
        if (*reinterpret_cast<volatile int *>(&b->gave_up)) return false;
        if (globaltimer_ns() - t0 > kWaitNs) {
            *reinterpret_cast<volatile int *>(&b->gave_up) = 1;
            return false;
        }
    }
}

__device__ __forceinline__ void store16(bf16 *p, const float *v) {
    uint4 w;
    w.x = pack_bf16x2(v[0], v[1]), w.y = pack_bf16x2(v[2], v[3]);
    w.z = pack_bf16x2(v[4], v[5]), w.w = pack_bf16x2(v[6], v[7]);
    *reinterpret_cast<uint4 *>(p) = w;
}

// Tiled copy shared -> global; elements outside the tensor are not written.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1)
                 : "memory");
}

// Waits for the loads from TMEM; nothing that uses their results moves before.
template <int N>
__device__ __forceinline__ void loaded(float (&z)[N]) {
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(z[i]));
}

// One column, of the warp's 32 rows.
__device__ __forceinline__ float tmem_column(uint32_t at) {
    float v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=f"(v) : "r"(at));
    tmem_ld_wait();
    asm volatile("" : "+f"(v));
    return v;
}
// One of 128 registers.
__device__ __forceinline__ float pick(const float (&z)[4][32], int at) {
    float v = 0.f;
#pragma unroll
    for (int c = 0; c < 128; c += 16) {
        int in = at - c;
        asm volatile("" : "+r"(in));  // (or all of z is kept in memory and indexed)
        if (in >= 0 && in < 16) {
            v = z[c / 32][c % 32];
#pragma unroll
            for (int i = 1; i < 16; ++i) v = in == i ? z[c / 32][c % 32 + i] : v;
        }
    }
    return v;
}

// The statistics of finite logits (and of any, but for the entropy, which minus infinity makes NaN): the maximum first, then
// four sums side by side, so that no addition waits for the one before.
__device__ __forceinline__ Stat stat_of(const float (&z)[4][32]) {
    constexpr int N = 128;
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = z[0][i];
#pragma unroll
    for (int i = 8; i < N; ++i) m[i % 8] = max_nan(m[i % 8], z[i / 32][i % 32]);
#pragma unroll
    for (int d = 4; d; d /= 2)
#pragma unroll
        for (int i = 0; i < d; ++i) m[i] = max_nan(m[i], m[i + d]);
    Stat s{m[0], 0.f, 0.f};
    if (is_far(s.m)) {
        if (s.m == -INFINITY) return s;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float t = fmaxf((z[i / 32][i % 32] - s.m) * kLog2e, kNothing), e = ex2(t);
            s.sum += e, s.moment = fmaf(e, t, s.moment);
        }
        return s;
    }
    const float ref = -ref_of(s.m);
    f2 sum[4] = {0, 0, 0, 0}, moment[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const f2 t = fma2(pack2(z[i / 16][2 * i % 32], z[i / 16][2 * i % 32 + 1]), pack2(kLog2e, kLog2e), pack2(ref, ref)), e = ex2x2(t);
        sum[i % 4] = add2(sum[i % 4], e);
        moment[i % 4] = fma2(e, t, moment[i % 4]);
    }
    s.sum = sum2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
    s.moment = sum2(add2(add2(moment[0], moment[1]), add2(moment[2], moment[3])));
    return s;
}

// A place in the ring.
struct Ring {
    int stages, s = 0;
    uint32_t round = 0;
    __device__ __forceinline__ explicit Ring(int n) : stages(n) {}
    __device__ __forceinline__ void next() {
        if (++s == stages) s = 0, ++round;
    }
};

// A_MN, B_MN: the operand lies with its rows (M or N) contiguous, in blocks of 64 rows by kBK.
template <int USE, bool A_MN, bool B_MN, bool ENT, bool PAIR>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mo,
                const __grid_constant__ GemmArgs a) {
    extern __shared__ uint8_t raw[];
    __shared__ Bars bars;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = PAIR ? pair_rank() : 0;
    const int first_unit = PAIR ? blockIdx.x / 2 : blockIdx.x, every = PAIR ? gridDim.x / 2 : gridDim.x;
    constexpr int HALF = PAIR ? 2 : 1;  // blocks that share B and the columns' work
    constexpr bool GRAD = USE == kGrad || USE == kGradShares, SHARES = USE == kStats || USE == kGradShares;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&bars.ready[i], 1), mbar_init(&bars.taken[i], HALF * kReaders);
        mbar_init(&bars.drain, 1);
        bars.gave_up = 0;
        fence_mbar_init();
        prefetch_tmap(&ma), prefetch_tmap(&mb);
    }
    if (warp == 2) {
        if constexpr (PAIR) {
            tmem_alloc_pair(&bars.tmem, 512);
        } else {
            tmem_alloc(&bars.tmem, 512);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) pair_sync();  // both blocks' barriers are there
    tc_fence_after();
    const uint32_t tmem = bars.tmem;
    const int shares = SHARES ? a.shares : 1;
    // (Where there are shares the readers' sums take 128 registers.  384 threads are launched with 168 each: 128 x 56 + 256 x 224.)
    if (warp < 4) {
        if constexpr (SHARES) reg_dec<56>();
        if (warp == 0 && lane == 0) {
            const int bn = a.bn / HALF;  // columns that this block copies
            const uint32_t bytes = HALF * (a.arows + bn) * kBK * 2;
            Ring r(a.stages);
            uint32_t it = 0;
            bool ok = true;
            for (int u = first_unit; u < a.units && ok; u += every) {
                const Unit t = unit_of(a, u);
                const int m0 = (t.m * HALF + rank) * kBM, n0 = t.n * a.bn + rank * bn;
                for (int k = t.k0; k < t.k1; ++k, ++it, r.next()) {
                    if (r.round > 0 && !(ok = wait_for(&bars.empty[r.s], (r.round - 1) & 1, &bars))) break;
                    uint64_t *full = &bars.full[r.s];
                    const uint32_t full_first = PAIR ? at_first(full) : 0;
                    auto load = [&](uint8_t *dst, const CUtensorMap *map, int c0, int c1) {
                        if constexpr (PAIR)
                            tma_load_2d_pair(dst, map, full_first, c0, c1);
                        else
                            tma_load_2d(dst, map, full, c0, c1);
                    };
                    uint8_t *sa = smem + r.s * a.stage_bytes, *sb = sa + a.abytes;
                    if (rank == 0) mbar_arrive_expect_tx(full, bytes);  // (both blocks' copies)
                    if constexpr (A_MN) {
                        for (int j = 0; j < kBM / 64; ++j) load(sa + j * 8192, &ma, m0 + j * 64, k * kBK);
                    } else {
                        load(sa, &ma, k * kBK, m0);
                    }
                    if constexpr (B_MN) {
                        for (int j = 0; j < bn / 64; ++j) load(sb + j * 8192, &mb, n0 + j * 64, k * kBK);
                    } else {
                        load(sb, &mb, k * kBK, n0);
                    }
                }
            }
            // no block ends with copies in flight (the pair's second waits for the first at the end)
            if (rank == 0)
                for (uint32_t i = it < (uint32_t)a.stages ? 0 : it - a.stages; i < it; ++i)
                    mbar_wait(&bars.full[i % a.stages], (i / a.stages) & 1, kWaitNs / 5);
        } else if (warp == 1 && lane == 0 && rank == 0) {
            const uint32_t idesc = idesc_bf16(HALF * kBM, a.bn, A_MN, B_MN);
            auto commit = [](uint64_t *bar) {
                if constexpr (PAIR)
                    mma_commit_pair(bar);
                else
                    mma_commit(bar);
            };
            Ring r(a.stages);
            uint32_t n = 0;
            bool ok = true;
            for (int u = first_unit; u < a.units && ok; u += every) {
                const Unit t = unit_of(a, u);
                for (int q = 0; q < shares && ok; ++q, ++n) {
                    const int k0 = SHARES ? a.kc * q / shares : t.k0, k1 = SHARES ? a.kc * (q + 1) / shares : t.k1;
                    const uint32_t acc = n & 1, d = tmem + acc * kBN;
                    if (n >= 2 && !(ok = wait_for(&bars.taken[acc], (n / 2 - 1) & 1, &bars))) break;
                    tc_fence_after();
                    for (int k = k0; k < k1; ++k, r.next()) {
                        if (!(ok = wait_for(&bars.full[r.s], r.round & 1, &bars))) break;
                        tc_fence_after();
                        const uint32_t sa = smem_u32(smem + r.s * a.stage_bytes), sb = sa + a.abytes;
                        const uint64_t da = A_MN ? sdesc(sa, 8192, 1024) : sdesc(sa, 16, 1024);
                        const uint64_t db = B_MN ? sdesc(sb, 8192, 1024) : sdesc(sb, 16, 1024);
#pragma unroll
                        for (int j = 0; j < kBK / 16; ++j) {
                            const uint64_t dj = desc_add(da, j * (A_MN ? 2048 : 32)), ej = desc_add(db, j * (B_MN ? 2048 : 32));
                            if constexpr (PAIR)
                                mma_bf16_pair(d, dj, ej, idesc, j > 0 || k > k0);
                            else
                                mma_bf16(d, dj, ej, idesc, j > 0 || k > k0);
                        }
                        commit(&bars.empty[r.s]);
                    }
                    if (ok) commit(&bars.ready[acc]);
                }
            }
            if constexpr (PAIR)
                mma_commit_pair_here(&bars.drain);  // nor with MMAs
            else
                mma_commit(&bars.drain);
            mbar_wait(&bars.drain, 0, kWaitNs / 5);
        }
    } else {
        if constexpr (SHARES) reg_inc<224>();
        const int q = warp % 4, half = (warp - 4) / 4, first = half * (kBN / 2);  // (a warp reads the 32 rows of its number mod 4)
        uint8_t *stage = smem + kRing + (warp - 4) * 4096;
        uint32_t n = 0;
        auto taken = [&](uint32_t acc) {
            tc_fence_before();
            __syncwarp();
            if (lane != 0) return;
            if (rank == 0)
                mbar_arrive(&bars.taken[acc]);
            else
                mbar_arrive_at(at_first(&bars.taken[acc]));
        };
        // The sums of this warp's columns (`limit` of them) over all shares; false: a wait gave up.
        auto sum_shares = [&](uint32_t lanes, int limit, float (&z)[4][32]) {
            for (int share = 0; share < shares; ++share, ++n) {
                const uint32_t acc = n & 1, at = lanes + acc * kBN + first;
                if (!wait_for(&bars.ready[acc], (n / 2) & 1, &bars)) return false;
                tc_fence_after();
                if (share == 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (32 * j < limit) tmem_ld32(at + 32 * j, z[j]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) loaded(z[j]);
                } else {
#pragma unroll
                    for (int c = 0; c < kBN / 2; c += 16) {
                        if (c < limit) {
                            float v[16];
                            tmem_ld16(at + c, v);
                            loaded(v);
#pragma unroll
                            for (int i = 0; i < 16; ++i) z[c / 32][c % 32 + i] += v[i];
                        }
                    }
                }
                taken(acc);
            }
            return true;
        };
        for (int u = first_unit; u < a.units; u += every) {
            const Unit t = unit_of(a, u);
            const int row = (t.m * HALF + rank) * kBM + q * 32 + lane, c0 = t.n * a.bn;
            const bool live = row < a.M;
            const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
            if constexpr (USE == kStats) {
                const int limit = min(min(a.N - c0, a.bn) - first, kBN / 2);  // of this warp's columns
                const int64_t given = live && a.targets ? a.targets[row] - c0 - first : -1;
                const int target = given >= 0 && given < limit ? (int)given : -1;
                float z[4][32];
                if (!sum_shares(lanes, limit, z)) break;
                if (limit < kBN / 2) {
#pragma unroll
                    for (int i = 0; i < kBN / 2; ++i) z[i / 32][i % 32] = i < limit ? z[i / 32][i % 32] : kLeast;
                }
                if (target >= 0) a.given[row] = pick(z, target);
                const Stat st = stat_of(z);
                if (live && first < a.bn)
                    a.stats[((int64_t)t.n * (a.bn > kBN / 2 ? 2 : 1) + half) * a.M + row] = make_float4(st.m, st.sum, st.moment, 0.f);
            } else {
                const int row0 = row - lane, limit = min(min(a.N - c0, a.bn) - first, kBN / 2);  // of this warp's columns
                RowGrad g{};
                FixRow fix{};
                if constexpr (GRAD) {
                    if (live) g = row_grad(a.grad, row, a.N);
                    if (live && t.n == 0 && half == 0 && (g.target < 0 || g.none)) a.rest[row] = 0.f;
                    if (a.lead && t.m == 0 && rank == 0 && q == 0)
                        for (int c = lane; c < limit; c += 32) a.lead[c0 + first + c] = kNoLead;
                } else if (t.part < 0) {
                    fix = fix_row(a.fix, row, live);
                }
                // The given token, where it is among this warp's columns, and its dz.
                const int in = g.target - c0 - first, target = GRAD && live && !g.none && g.target >= 0 && in >= 0 && in < limit ? in : -1;
                float given = 0.f;
                auto give = [&](float z) {
                    given = given_grad<ENT>(g, z);
                    a.rest[row] = given - to_f32(from_f32<bf16>(given));
                };
                // What becomes of 32 of the columns, from the c-th on.
                auto put = [&](float (&now)[32], int c) {
                    const int col = c0 + first + c;
                    if constexpr (GRAD) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) now[i] = g.none ? 0.f : grad_of<ENT>(g, now[i]);
                        if (target >= c && target < c + 32) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) now[i] = c + i == target ? given : now[i];
                        }
                    }
                    if (USE == kStore && t.part >= 0) {
                        float *p = a.parts + (((int64_t)t.part * HALF + rank) * kBM + q * 32 + lane) * a.bn + first + c;
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4 *>(p + i) = make_float4(now[i], now[i + 1], now[i + 2], now[i + 3]);
                    } else if (row0 < a.M) {
                        // by way of shared memory, 32 rows of 64 columns in the layout that the copy expects
                        if (c % 64 == 0) {
                            if (lane == 0) bulk_wait_read_all();
                            __syncwarp();
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            if (USE == kStore && col + i < a.N) fix_add(fix, col + i, now + i);
                            store16(reinterpret_cast<bf16 *>(stage + lane * 128 + (((c % 64 + i) / 8 ^ (lane & 7)) * 16)), now + i);
                        }
                        if (c % 64 == 32 || c + 32 >= limit) {
                            fence_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                tma_store_2d(&mo, stage, col / 64 * 64, row0);
                                bulk_commit_group();
                            }
                        }
                    }
                };
                if constexpr (SHARES) {
                    float z[4][32] = {};
                    if (!sum_shares(lanes, limit, z)) break;
                    if (target >= 0) give(pick(z, target));
#pragma unroll
                    for (int c = 0; c < kBN / 2; c += 32)
                        if (c < limit) put(z[c / 32], c);
                } else {
                    const uint32_t acc = n & 1, at = lanes + acc * kBN + first;
                    if (!wait_for(&bars.ready[acc], (n / 2) & 1, &bars)) break;
                    ++n;
                    tc_fence_after();
                    if constexpr (GRAD) {  // (as many columns as there are different given tokens: few or none)
                        float zt = 0.f;
                        for (unsigned todo = __ballot_sync(0xffffffffu, target >= 0); todo;) {
                            const int c = __shfl_sync(0xffffffffu, target, __ffs(todo) - 1);
                            const float v = tmem_column(at + c);
                            if (target == c) zt = v;
                            todo &= ~__ballot_sync(0xffffffffu, target == c);
                        }
                        if (target >= 0) give(zt);
                    }
                    float z[2][32] = {};
                    if (limit > 0) {
                        tmem_ld32(at, z[0]);
                        loaded(z[0]);
                    }
#pragma unroll
                    for (int c = 0; c < kBN / 2; c += 32) {
                        if (c >= limit) continue;
                        if (c + 32 < kBN / 2 && c + 32 < limit) tmem_ld32(at + c + 32, z[(c / 32 + 1) % 2]);
                        put(z[c / 32 % 2], c);
                        loaded(z[(c / 32 + 1) % 2]);
                    }
                    taken(acc);
                }
            }
        }
        if (USE != kStats && lane == 0) bulk_wait_all();  // the copies have read what they store
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && bars.gave_up) atomicOr(a.status, 1u);
    if constexpr (PAIR) {
        pair_sync();  // nothing is on its way to either block
        if (warp == 2) tmem_dealloc_pair(tmem, 512);
    } else {
        if (warp == 2) tmem_dealloc(tmem, 512);
    }
}

// The numbers of every row from its tiles' statistics.  A block has `per` neighbouring rows (1, or 8 where there are many) and
// joins a row's tiles in 256 / per threads, then those, in a fixed order.
__global__ void __launch_bounds__(256) head_rows_kernel(const float4 *stats, const float *given, const int64_t *targets, int rows,
                                                        int nt, int vocab, int per, float *logprob, float *lse, float *entropy) {
    __shared__ Stat part[256];
    wait_previous();
    const int in = threadIdx.x % per, w = threadIdx.x / per, step = 256 / per, row = blockIdx.x * per + in;
    Stat st{-INFINITY, 0.f, 0.f};
    if (row < rows) {
        for (int n = w; n < nt; n += 4 * step) {
            float4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = n + i * step < nt ? stats[(int64_t)(n + i * step) * rows + row] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) st = join(st, Stat{v[i].x, v[i].y, v[i].z});
        }
    }
    part[threadIdx.x] = st;
    for (int d = step / 2; d; d /= 2) {
        __syncthreads();
        if (w < d) part[threadIdx.x] = st = join(st, part[threadIdx.x + d * per]);
    }
    if (w || row >= rows) return;
    const float l = lse_of(st);
    if (lse) lse[row] = l;
    if (entropy) entropy[row] = entropy_of(st);
    if (logprob) {
        const int64_t t = targets[row];
        logprob[row] = t < 0 ? 0.f : t >= vocab ? __uint_as_float(0x7FC00000u) : logprob_of(given[row], l);
    }
}

// The tiles that were split: their parts' sum, in order.
__global__ void __launch_bounds__(256) head_parts_kernel(const __grid_constant__ GemmArgs a) {
    const int per = a.bn / 8, tall = a.pair ? 2 * kBM : kBM, blocks = (tall * per + 255) / 256;
    const int tile = blockIdx.x / blocks, i = blockIdx.x % blocks * 256 + threadIdx.x;
    const Unit t = unit_of(a, a.whole + tile * a.split);
    if (i >= tall * per) return;
    const int r = i / per, c = i % per * 8, row = t.m * tall + r, col = t.n * a.bn + c;
    if (row >= a.M || col >= a.N) return;
    float v[8] = {};
    for (int k = 0; k < a.split; ++k) {
        const float4 *p = reinterpret_cast<const float4 *>(a.parts + (((int64_t)tile * a.split + k) * tall + r) * a.bn + c);
        const float4 x = p[0], y = p[1];
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w, v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
    }
    fix_add(fix_row(a.fix, row, true), col, v);
    store16(a.out + row * a.out_pitch + col, v);
}

// What dweight's rows are given for rounding dz: sums[r] = sum of rest[row] hidden[row] over the rows with row r's target, in
// two steps so that neither many rows nor many of one target cost more than their share.  Rows are taken in chunks of
// fix_chunk(); the first row of a target in each chunk (a block a row, 8 columns a thread) sums the chunk's, in order, and
// enters the target's chain of chunks.  (4095 x 2560 x 50277, random targets 35 us, one for all rows 86; 131072 rows 1.1 ms of
// 72.  One scan of all rows by the first of each target: 27 us, 3.8 ms and 8.2 ms.)
constexpr int kFixRows = 4096, kFixChunks = 1024;  // the largest chunk, and how many there are at most
static_assert((int64_t)kFixRows * kFixChunks >= 1 << 22, "every number of rows that is supported");
int fix_chunk(int64_t rows) {
    const int64_t c = (rows + kFixChunks - 1) / kFixChunks;
    return (int)((c + 255) / 256 * 256);
}
__global__ void __launch_bounds__(256, 4) head_fix_kernel(const int64_t *targets, const float *rest, const bf16 *hidden, int64_t pitch,
                                                       int rows, int dim, int vocab, int chunk, int *lead, int *next, float *sums) {
    __shared__ int list[kFixRows], counts[8];
    const int r = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t t = targets[r];
    if (t < 0 || t >= vocab) return;
    const int begin = r / chunk * chunk, end = min(begin + chunk, rows);
    int n = 0;
    for (int base = begin; base < end; base += 256) {
        const int row = base + threadIdx.x;
        const bool same = row < end && targets[row] == t;
        const unsigned which = __ballot_sync(0xffffffffu, same);
        if (lane == 0) counts[warp] = __popc(which);
        if (__syncthreads_or(same && row < r)) return;  // not the first
        int at = n;
        for (int w = 0; w < 8; ++w) {
            if (w < warp) at += counts[w];
            n += counts[w];
        }
        if (same) list[at + __popc(which & ((1u << lane) - 1))] = row;
        __syncthreads();
    }
    constexpr int U = 8;
    for (int c = threadIdx.x * 8; c < dim; c += 2048) {
        float v[8] = {};
        int k = 0;
        for (; k + U <= n; k += U) {
            Vec<bf16, 8> h[U];
            float q[U];
#pragma unroll
            for (int u = 0; u < U; ++u) h[u] = load_vec<bf16, 8>(hidden + list[k + u] * pitch + c), q[u] = rest[list[k + u]];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[8];
                widen<bf16, 8>(h[u], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = fmaf(q[u], f[i], v[i]);
            }
        }
        for (; k < n; ++k) {
            float f[8];
            widen<bf16, 8>(load_vec<bf16, 8>(hidden + list[k] * pitch + c), f);
            const float q = rest[list[k]];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(q, f[i], v[i]);
        }
        float *out = sums + (int64_t)r * dim + c;
        *reinterpret_cast<float4 *>(out) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(out + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
    if (threadIdx.x == 0) next[r] = atomicExch(&lead[t], r);
}
// The chunks of each target, in the order of their rows, to sums of the row that the chain begins with (any of them: rows
// enter as blocks end).
__global__ void __launch_bounds__(256) head_chains_kernel(const int64_t *targets, const int *lead, const int *next, int dim, int vocab,
                                                          float *sums) {
    __shared__ int chain[kFixChunks], sorted[kFixChunks], count;
    const int r = blockIdx.x;
    wait_previous();
    const int64_t t = targets[r];
    if (t < 0 || t >= vocab || lead[t] != r || next[r] == kNoLead) return;
    if (threadIdx.x == 0) {
        int n = 0;
        for (int q = r; q != kNoLead && n < kFixChunks; q = next[q]) chain[n++] = q;
        count = n;
    }
    __syncthreads();
    const int n = count;
    for (int i = threadIdx.x; i < n; i += 256) {
        int before = 0;
        for (int j = 0; j < n; ++j) before += chain[j] < chain[i];
        sorted[before] = chain[i];
    }
    __syncthreads();
    for (int c = threadIdx.x * 4; c < dim; c += 1024) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(sums + (int64_t)sorted[i] * dim + c);
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        *reinterpret_cast<float4 *>(sums + (int64_t)r * dim + c) = v;
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// [rows][cols] bf16, boxes of 64 columns and `box` rows, 128-byte swizzle; what lies outside reads as 0.
bool map_of(CUtensorMap *m, const void *p, int64_t rows, int64_t cols, int64_t pitch, int box) {
    const auto enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, str[1] = {(cuuint64_t)pitch * 2};
    const cuuint32_t b[2] = {64, (cuuint32_t)box}, es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, str, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tiles of 256 rows where they leave no more than an eighth of the rows empty and sums are long enough for a pair's longer
// start.  8192 x 256 x 32000 120 us, in pairs 134; x 512 193 and 199.  Forward and gradient of T x 2560 x 50277, T = 300: 349 us,
// with pairs for dweight, a sum over T, 362; T = 1000: 793 us, without any pairs 875.
bool takes_pairs(int64_t M, int64_t K, int bn) {
    const int64_t padded = (M + 2 * kBM - 1) / (2 * kBM) * (2 * kBM);
    return bn % 128 == 0 && K >= 640 && padded - M <= padded / 8;
}

// Tiles and units of a product.  `split`: tiles beyond the last full round of blocks are cut along K, so that every SM has a share
// (forward and gradient of 300 x 2560 x 50277, at the time 478 us: whole tiles only 709; of 64 rows: 349 and 606).
GemmArgs plan_gemm(int64_t M, int64_t N, int64_t K, int bn, bool split, bool a_mn = false) {
    GemmArgs a{};
    a.M = (int)M, a.N = (int)N, a.K = (int)K, a.bn = bn;
    a.pair = takes_pairs(M, K, bn);
    const int tall = a.pair ? 2 * kBM : kBM, places = a.pair ? kSMs / 2 : kSMs;
    a.mt = (int)((M + tall - 1) / tall), a.nt = (int)((N + bn - 1) / bn), a.kc = (int)((K + kBK - 1) / kBK);
    a.group = a.pair ? 16 : 32;
    a.arows = M < kBM && !a_mn ? (int)((M + 7) / 8 * 8) : kBM;
    a.abytes = (a.arows * kBK * 2 + 1023) / 1024 * 1024, a.stage_bytes = a.abytes + (bn / (a.pair ? 2 : 1) * kBK * 2 + 1023) / 1024 * 1024;
    a.stages = kRing / a.stage_bytes < kMaxStages ? kRing / a.stage_bytes : kMaxStages;
    a.shares = (a.kc + kShare - 1) / kShare;
    const int tiles = a.mt * a.nt;
    a.whole = tiles, a.split = 1;
    const int rest = tiles % places;
    if (split && rest) {
        int s = places / rest;
        if (s > a.kc / 4) s = a.kc / 4;  // (a share of fewer chunks is mostly filling the ring)
        if (s > 1) a.whole = tiles - rest, a.split = s;
    }
    if (split && a.kc > kLongest) a.whole = 0, a.split = (a.kc + kLongest - 1) / kLongest;
    a.units = a.whole + (tiles - a.whole) * a.split;
    return a;
}
size_t parts_bytes(const GemmArgs &a) { return align256(sizeof(float) * (size_t)(a.units - a.whole) * (a.pair ? 2 : 1) * kBM * a.bn); }

int fit_columns(int64_t n) { return n >= 256 ? 256 : (int)((n + 63) / 64 * 64); }

// Up to 128 rows the weights' one pass is what takes time: tiles of the statistics as wide as gives every SM the same number
// (in a graph, 16 x 2560 x 50280 48.2 us, tiles of 256 52.1; of 131072 106.6, 109.0; 128 x 2560 x 20000 26.5, 28.2), unless
// they were narrow (16 x 2560 x 5000 22.1, 21.1).
int forward_columns(int64_t rows, int64_t vocab) {
    const int64_t rounds = (vocab + kBN * kSMs - 1) / (kBN * kSMs), n = (vocab + rounds * kSMs - 1) / (rounds * kSMs);
    return rows > kBM || n < 64 ? fit_columns(vocab) : (int)(n + 15) / 16 * 16;
}

int halves(const GemmArgs &a) { return a.bn > kBN / 2 ? 2 : 1; }

struct HeadPlan {
    size_t stats, given, dz, rest, lead, next, sums, parts, bytes;
    int64_t pitch;
    GemmArgs z, dh, dw;
};
HeadPlan plan_fwd(const ssd_head_shape_t *s) {
    HeadPlan p{};
    p.z = plan_gemm(s->rows, s->vocab, s->dim, forward_columns(s->rows, s->vocab), false);
    p.stats = 0;
    p.given = align256(sizeof(float4) * p.z.nt * halves(p.z) * s->rows);
    p.bytes = p.given + align256(sizeof(float) * s->rows);
    return p;
}
HeadPlan plan_bwd(const ssd_head_shape_t *s) {
    HeadPlan p{};
    p.z = plan_gemm(s->rows, s->vocab, s->dim, fit_columns(s->vocab), false);
    p.dh = plan_gemm(s->rows, s->dim, s->vocab, fit_columns(s->dim), true);
    p.dw = plan_gemm(s->vocab, s->dim, s->rows, fit_columns(s->dim), true, true);
    p.pitch = (s->vocab + 63) / 64 * 64;
    p.dz = 0;
    p.rest = align256(2 * s->rows * p.pitch);
    p.lead = p.rest + align256(sizeof(float) * s->rows);
    p.next = p.lead + align256(sizeof(int) * s->vocab);
    p.sums = p.next + align256(sizeof(int) * s->rows);
    p.parts = p.sums + align256(sizeof(float) * s->rows * s->dim);
    const size_t a = parts_bytes(p.dh), b = parts_bytes(p.dw);
    p.bytes = p.parts + (a > b ? a : b);
    return p;
}

template <int USE, bool A_MN, bool B_MN, bool ENT>
cudaError_t run_gemm(const CUtensorMap &ma, const CUtensorMap &mb, const CUtensorMap &mo, const GemmArgs &a, const char *name,
                     cudaStream_t st) {
    auto kernel = a.pair ? gemm_kernel<USE, A_MN, B_MN, ENT, true> : gemm_kernel<USE, A_MN, B_MN, ENT, false>;
    // (set on every call: cheap, and right for each device and context)
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int blocks = a.pair ? 2 : 1, places = kSMs / blocks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * (a.units < places ? a.units : places)));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)blocks, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.pair ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kernel, ma, mb, mo, a);
    timing_mark(st, name);
    return e;
}

cudaError_t run_parts(const GemmArgs &a, cudaStream_t st) {
    const int tiles = (a.units - a.whole) / a.split;
    if (a.units == a.whole) return cudaSuccess;
    const int64_t blocks = ((a.pair ? 2 : 1) * kBM * (a.bn / 8) + 255) / 256;
    if (blocks * tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
    head_parts_kernel<<<(unsigned)(blocks * tiles), 256, 0, st>>>(a);
    timing_mark(st, "head_parts");
    return cudaGetLastError();
}

ssd_status_t check_head(const ssd_head_shape_t *s) {
    if (!s || s->rows < 0 || s->dim <= 0 || s->vocab <= 0) return SSD_ERR_INVALID_ARG;
    if (s->dtype != SSD_DTYPE_F32 && s->dtype != SSD_DTYPE_BF16) return SSD_ERR_INVALID_ARG;
    if (s->dtype != SSD_DTYPE_BF16 || s->dim % 8 || s->dim > (1 << 20) || s->vocab > (1 << 22) || s->rows > (1 << 22))
        return SSD_ERR_UNSUPPORTED;
    // tiles and their parts are counted in 31 bits
    const int64_t most = 1 << 28;
    if ((s->rows / kBM + 1) * (s->vocab / 64 + 1) > most ||
        (s->vocab / kBM + 1) * (s->dim / 64 + 1) * (s->rows / (kLongest * kBK) + 1) > most / 64 ||
        (s->rows / kBM + 1) * (s->dim / 64 + 1) * (s->vocab / (kLongest * kBK) + 1) > most / 64)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}
// Rows that TMA reads: 16-byte aligned, each of them.
bool tma_rows(const ssd_rows_t &r, int64_t rows, int64_t dim) {
    return far_rows_ok(r, 2) && aligned(r.data, 16) &&
           (rows <= 1 || (r.row_stride % 8 == 0 && r.row_stride >= dim && r.row_stride < kMaxBatchStride / 2));
}
int64_t pitch_of(const ssd_rows_t &r, int64_t rows, int64_t dim) { return rows > 1 ? r.row_stride : dim; }

}  // namespace
}  // namespace ssd

extern "C" {

size_t ssd_head_logprob_workspace_size(const ssd_head_shape_t *shape) {
    using namespace ssd;
    return check_head(shape) != SSD_OK || shape->rows == 0 ? 0 : plan_fwd(shape).bytes;
}
size_t ssd_head_logprob_bwd_workspace_size(const ssd_head_shape_t *shape) {
    using namespace ssd;
    return check_head(shape) != SSD_OK || shape->rows == 0 ? 0 : plan_bwd(shape).bytes;
}

ssd_status_t ssd_head_logprob_fwd(const ssd_head_shape_t *shape, const ssd_rows_t *hidden, const ssd_rows_t *weight,
                                  const int64_t *targets, float *logprob, float *lse, float *entropy, void *workspace,
                                  size_t workspace_bytes, cudaStream_t stream) {
    using namespace ssd;
    const ssd_status_t ok = check_head(shape);
    if (ok != SSD_OK) return ok;
    if (shape->rows == 0) return SSD_OK;
    const int64_t T = shape->rows, V = shape->vocab, D = shape->dim;
    if (!hidden || !weight || !tma_rows(*hidden, T, D) || !tma_rows(*weight, V, D) || !aligned(targets, 8) || !aligned(logprob, 4) ||
        !aligned(lse, 4) || !aligned(entropy, 4) || (logprob && !targets))
        return SSD_ERR_INVALID_ARG;
    HeadPlan p = plan_fwd(shape);
    if (!workspace || workspace_bytes < p.bytes || !aligned(workspace, 16)) return SSD_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    CUtensorMap mh, mw;
    if (!map_of(&mh, hidden->data, T, D, pitch_of(*hidden, T, D), p.z.arows) ||
        !map_of(&mw, weight->data, V, D, pitch_of(*weight, V, D), p.z.bn / (p.z.pair ? 2 : 1)))
        return SSD_ERR_CUDA;
    GemmArgs a = p.z;
    a.targets = logprob ? targets : nullptr;
    a.stats = reinterpret_cast<float4 *>(ws + p.stats);
    a.given = reinterpret_cast<float *>(ws + p.given);
    cudaError_t e = device_status_word(&a.status);
    if (e != cudaSuccess) return status_of(e);
    timing_begin(stream);
    e = run_gemm<kStats, false, false, false>(mh, mw, mw, a, "head_logprob", stream);
    if (e != cudaSuccess) return status_of(e);
    const int per = T > 8 * kSMs ? 8 : 1;
    e = launch(head_rows_kernel, dim3((unsigned)((T + per - 1) / per)), 256, 0, stream, true, a.stats, a.given, a.targets, (int)T,
               a.nt * halves(a), (int)V, per, logprob, lse, entropy);
    timing_mark(stream, "head_rows");
    return status_of(e);
}

ssd_status_t ssd_head_logprob_bwd(const ssd_head_shape_t *shape, const ssd_rows_t *hidden, const ssd_rows_t *weight,
                                  const int64_t *targets, const float *lse, const float *entropy, const float *dlogprob,
                                  const float *dlse, const float *dentropy, const ssd_rows_t *dhidden, const ssd_rows_t *dweight,
                                  void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace ssd;
    const ssd_status_t ok = check_head(shape);
    if (ok != SSD_OK) return ok;
    const int64_t T = shape->rows, V = shape->vocab, D = shape->dim;
    if (dweight && (!tma_rows(*dweight, V, D) || !far_rows_out_ok(*dweight, 2, V, D))) return SSD_ERR_INVALID_ARG;
    if (T == 0) {
        if (!dweight) return SSD_OK;
        return status_of(cudaMemset2DAsync(dweight->data, pitch_of(*dweight, V, D) * 2, 0, D * 2, V, stream));
    }
    if (!hidden || !weight || !tma_rows(*hidden, T, D) || !tma_rows(*weight, V, D) || !lse || !aligned(lse, 4) || !aligned(entropy, 4) ||
        !aligned(targets, 8) || !aligned(dlogprob, 4) || !aligned(dlse, 4) || !aligned(dentropy, 4) || (dlogprob && !targets) ||
        (dentropy && !entropy))
        return SSD_ERR_INVALID_ARG;
    if (dhidden && (!tma_rows(*dhidden, T, D) || !far_rows_out_ok(*dhidden, 2, T, D))) return SSD_ERR_INVALID_ARG;
    if (!dhidden && !dweight) return SSD_OK;
    HeadPlan p = plan_bwd(shape);
    if (!workspace || workspace_bytes < p.bytes || !aligned(workspace, 16)) return SSD_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    bf16 *dz = reinterpret_cast<bf16 *>(ws + p.dz);
    const int64_t hp = pitch_of(*hidden, T, D), wp = pitch_of(*weight, V, D);
    CUtensorMap mh, mw, mz, mz_t, mw_t, mh_t, mz_out, mdh, mdw;
    // dz: only its V columns are read, whatever lies behind them
    if (!map_of(&mh, hidden->data, T, D, hp, p.z.arows) || !map_of(&mw, weight->data, V, D, wp, p.z.bn / (p.z.pair ? 2 : 1)) ||
        !map_of(&mz, dz, T, V, p.pitch, p.dh.arows) || !map_of(&mw_t, weight->data, V, D, wp, kBK) ||
        !map_of(&mz_t, dz, T, V, p.pitch, kBK) || !map_of(&mh_t, hidden->data, T, D, hp, kBK) ||
        !map_of(&mz_out, dz, T, V, p.pitch, 32) || (dhidden && !map_of(&mdh, dhidden->data, T, D, pitch_of(*dhidden, T, D), 32)) ||
        (dweight && !map_of(&mdw, dweight->data, V, D, pitch_of(*dweight, V, D), 32)))
        return SSD_ERR_CUDA;
    unsigned *status = nullptr;
    cudaError_t e = device_status_word(&status);
    if (e != cudaSuccess) return status_of(e);
    timing_begin(stream);
    GemmArgs a = p.z;
    a.status = status;
    a.grad = RowGradIn{targets, lse, entropy, dlogprob, dlse, dentropy};
    a.rest = reinterpret_cast<float *>(ws + p.rest);
    const bool given = targets && dlogprob;  // otherwise no element of dz stands out
    int *lead = dweight && given ? reinterpret_cast<int *>(ws + p.lead) : nullptr;
    a.lead = lead;
    auto dlogits = [&](auto use, auto ent) {
        e = run_gemm<decltype(use)::value, false, false, decltype(ent)::value>(mh, mw, mz_out, a, "head_dlogits", stream);
    };
    auto with_shares = [&](auto ent) {
        a.shares > 1 ? dlogits(std::integral_constant<int, kGradShares>{}, ent) : dlogits(std::integral_constant<int, kGrad>{}, ent);
    };
    dentropy ? with_shares(std::true_type{}) : with_shares(std::false_type{});
    if (e == cudaSuccess && dhidden) {
        GemmArgs b = p.dh;
        b.status = status;
        b.out = static_cast<bf16 *>(dhidden->data), b.out_pitch = pitch_of(*dhidden, T, D);
        b.parts = reinterpret_cast<float *>(ws + p.parts);
        if (given) b.fix = Fix{targets, a.rest, static_cast<const bf16 *>(weight->data), wp, (int)V, nullptr, nullptr, D};
        e = run_gemm<kStore, false, true, false>(mz, mw_t, mdh, b, "head_dhidden", stream);
        if (e == cudaSuccess) e = run_parts(b, stream);
    }
    if (e == cudaSuccess && dweight) {
        GemmArgs b = p.dw;
        b.status = status;
        b.out = static_cast<bf16 *>(dweight->data), b.out_pitch = pitch_of(*dweight, V, D);
        b.parts = reinterpret_cast<float *>(ws + p.parts);
        if (lead) {
            float *sums = reinterpret_cast<float *>(ws + p.sums);
            int *next = reinterpret_cast<int *>(ws + p.next);
            const int chunk = fix_chunk(T);
            head_fix_kernel<<<(unsigned)T, 256, 0, stream>>>(targets, a.rest, static_cast<const bf16 *>(hidden->data), hp, (int)T, (int)D,
                                                             (int)V, chunk, lead, next, sums);
            timing_mark(stream, "head_fix");
            e = cudaGetLastError();
            if (e == cudaSuccess && T > chunk) {
                e = launch(head_chains_kernel, dim3((unsigned)T), 256, 0, stream, true, targets, lead, next, (int)D, (int)V, sums);
                timing_mark(stream, "head_chains");
            }
            if (e != cudaSuccess) return status_of(e);
            b.fix = Fix{nullptr, nullptr, nullptr, 0, (int)V, lead, sums, D};
        }
        e = run_gemm<kStore, true, true, false>(mz_t, mh_t, mdw, b, "head_dweight", stream);
        if (e == cudaSuccess) e = run_parts(b, stream);
    }
    return status_of(e);
}

}  // extern "C"
