// paged_move.h -- parameters of the kernels behind kvevict_paged_append and
// kvevict_paged_gather.
#pragma once

#include "paged_common.cuh"

namespace kvevict {

constexpr int kPagedThreads = 256;
constexpr int kAppendTokens = 32;  // of a CTA, at most
constexpr int kAppendOwnBatch = 4; // units of a thread at once, own type
constexpr int kGatherRows = 64;    // of a CTA

struct AppendParams {
    PagedCache c;
    const void *x[2];        // k, v
    long long xs[2][2];      // strides in elements: head, token
    const int32_t *starts;
    const double *freq;
    const void *pos;
    long long ps;
    int pos64, R, inter, per;
    float scale;
    int tokens;
    int tokens_per, heads_per, head_blocks;  // a CTA's share; heads: n_kv_heads of k, then of v
};

struct GatherParams {
    PagedCache c;
    void *y[2];
    long long ys[2][3];  // strides in elements: sequence, head, token
    const int32_t *k_starts;
    int rows, tiles;     // rows of a sequence (padded) or in all (packed); row tiles
};

// Which kernel takes a call. Pages of the keys' own type: the rotary part is whole
// 16-byte chunks (pairs of them). 4 bits: whole eights of
// channels turn (pairs of them). (All else: the general one.) elem: bytes of dtype, 2 or 4.
inline bool append_own(const AppendParams &p, int elem, bool q4) { return !q4 && (p.inter ? p.R * elem % 16 == 0 : p.R / 2 * elem % 16 == 0); }
inline bool append_q4(const AppendParams &p, bool q4) { return q4 && (p.inter ? p.R % 8 == 0 : p.R / 2 % 8 == 0); }
cudaError_t launch_append(const AppendParams &p, int head_dim, int elem, bool q4, cudaStream_t st);
cudaError_t launch_gather(const GatherParams &p, int head_dim, int elem, bool q4, cudaStream_t st);

}  // namespace kvevict
