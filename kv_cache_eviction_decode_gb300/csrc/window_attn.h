// window_attn.h -- parameters of the attention kernels behind
// kvevict_window_attention and kvevict_shared_prefix_attention.
//
// One launch works on one or two problems (the shared prefix and the
// suffixes). A problem is a grid of units (sequence, KV head); a unit's query
// rows are its (token, group head) pairs, row = token * G + g, so that the G
// query heads of a KV head share every key tile. An item of work is a tile of
// rows of one unit against one of `splits` parts of the key tiles those rows
// see; with more than one part, each writes its own normalised output and log2
// normaliser to a slot of the workspace and launch_attn_join joins the slots.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace kvevict {

struct AttnProblem {
    const void *q, *k, *v;
    long long qs[3], ks[3], vs[3];  // strides in elements: sequence, head, token
    long long os[3], rs[3];         // the output's, and the row index's (lse and workspace slots)
    const int32_t *q_starts, *k_starts, *q_lens, *k_lens;
    int q_rows, k_rows, max_q;
    int batch, causal, n_sink, window;  // window 0: none
    int q_tiles, splits, slot0;         // slot0: the first part's slot
    int n_items;
    int pair;                           // tensor cores: the rows fit one tile, two tiles share the keys
};

struct AttnParams {
    AttnProblem pr[2];
    int n_problems;
    int G, Hq, Hkv;
    float scale_log2;   // log2(e) * scale
    void *out;
    float *lse;         // may be null
    float *part_o;      // [slots][rows][d], and
    float *part_l;      // [slots][rows] log2 normalisers, where slots > 1
    long long rows;     // query rows in all
    int slots;
    uint32_t *err;
};

constexpr int kAttnF32Rows = 64, kAttnF32FewRows = 16, kAttnF32Keys = 64, kAttnF32FewKeys = 32;

// Tensor maps of one problem: q as (d, group head, token, KV head, sequence),
// boxes of 64 x G x (128 / G) tokens; k and v as (d, key, KV head, sequence),
// boxes of 64 x 128 keys; 128-byte swizzle.
struct alignas(64) AttnTmap {
    uint64_t word[16];
};
struct AttnTcMaps {
    AttnTmap q, k, v;
};
struct AttnTcParams {
    AttnTcMaps maps[2];
    AttnParams a;
};

constexpr int kAttnTcRows = 128, kAttnTcKeys = 128;

// bf16 attention on the tensor cores.
cudaError_t launch_attn_tc(const AttnTcParams &p, int head_dim, cudaStream_t st);
// fp32 attention on the CUDA cores; `few`: tiles of 16 rows, else 64.
cudaError_t launch_attn_f32(const AttnParams &p, int head_dim, bool few, cudaStream_t st);
// Joins the slots: out = sum_s 2^(l_s - l) o_s, l = log2 sum_s 2^(l_s).
cudaError_t launch_attn_join(const AttnParams &p, int head_dim, bool bf16, cudaStream_t st);

}  // namespace kvevict
