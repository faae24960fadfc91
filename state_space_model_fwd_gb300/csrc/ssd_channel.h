// ssd_channel.h -- arguments and host helpers of the channel scan's kernels.
#pragma once

#include "ssd_channel.cuh"

namespace ssd {

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 4096;  // tokens are counted in 32 bits, offsets in 64

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

template <typename T>
struct ChannelArgs {
    Rows<const T> x, dt, z, B, C;  // z.p null: no gate
    Rows<T> y;
    const float *A, *D, *bias, *init;
    float *fin;
    int ch, per, nblk_g, nblk;  // channels, channels per group, blocks of 32 per group and in all
    int nseq, soft;
    Seqs seqs;
    int chunk, nchunk;  // tokens per chunk; chunks of a sequence row
    int whole, cut;     // forward: block rows run whole, and cut into chunks
    unsigned blocks;    // forward: blocks of these (more pass empty sequences' states on)
    int units;          // gradient: chunks in all
    float4 *local;      // a chunk's own end state, [N / 4][32] each: by [chunk][cut] forward, [unit][block] gradient
    float *sums;        // sum of a chunk's deltas, [32] each
};

template <typename T>
ChannelArgs<T> channel_args(const ssd_channel_shape_t *s, const ssd_channel_inputs_t *in, int64_t nseq) {
    ChannelArgs<T> a{};
    a.x = rows_of<const T>(in->x), a.dt = rows_of<const T>(in->dt), a.z = rows_of<const T>(in->z);
    a.B = rows_of<const T>(in->B), a.C = rows_of<const T>(in->C);
    a.A = in->A, a.D = in->D, a.bias = in->dt_bias, a.init = in->init_state;
    a.ch = (int)s->channels, a.per = (int)(s->channels / s->ngroups);
    a.nblk_g = (a.per + 31) / 32, a.nblk = a.nblk_g * (int)s->ngroups;
    a.nseq = (int)nseq, a.soft = s->dt_softplus != 0;
    a.seqs.n = (int)nseq, a.seqs.L = (int)s->seqlen;
    return a;
}

ssd_status_t check_channel(const ssd_channel_shape_t *s, const int64_t *cu, int64_t nseq);
bool channel_inputs_ok(const ssd_channel_shape_t *s, const ssd_channel_inputs_t *in, bool rows);

// Where the offsets of a packed batch go: into the launches' parameters, or
// (true: a launch was made) into the workspace.
inline size_t offsets_bytes(const int64_t *cu, int64_t nseq) {
    return cu && nseq + 1 > kInline ? align256(sizeof(int) * (nseq + 1)) : 0;
}
cudaError_t place_offsets(const int64_t *cu, int64_t nseq, int *dst, Seqs &seqs, bool *launched, cudaStream_t st);
// Blocks to add for the empty sequences of a packed batch (0: there are none).
int empty_blocks(const int64_t *cu, int64_t nseq);
// Every sequence is empty: dst = src, or zero.
cudaError_t copy_states(const float *src, float *dst, int64_t count, cudaStream_t st);

}  // namespace ssd
