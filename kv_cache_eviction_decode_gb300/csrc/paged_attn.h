// paged_attn.h -- parameters of the attention kernels on a paged cache
// (kvevict_paged_attention).
//
// A unit is a (sequence, KV head); its query rows are (token, group head) pairs,
// row = token * G + g, so that the G query heads of a KV head share every key. An
// item of work is a tile of rows of one unit against one of `splits` parts of the
// 16-key tiles that those rows see (a tile lies in one page). Up to eight parts are
// the CTAs of a cluster, which join them through distributed shared memory; of more,
// each writes its own normalised output and log2 normaliser to the workspace, and
// launch_paged_join joins them.
#pragma once

#include "paged_common.cuh"
#include "window_attn_common.cuh"

namespace kvevict {

constexpr int kPagedTile = 16;  // keys

struct PagedAttnParams {
    PagedCache c;
    AttnProblem mask;  // causal, n_sink, window, and q_starts (what attn_keys and attn_first_fall read)
    const void *q;
    void *out;
    float *lse;        // may be null
    long long qs[2], os[2];  // strides in elements: head, token
    int tokens, per, max_q;
    int G, Hq;
    float scale_log2;
    int splits, q_tiles;
    int clusters;      // the parts are joined in their cluster
    float *part_o;     // [splits][tokens * Hq][d], and
    float *part_l;     // [splits][tokens * Hq] log2 normalisers, where splits > 1 and not clusters
};

// A sequence's new tokens and keys: rows q0 .. q0 + n - 1, the first of them at
// position p0 (negative where there are more of them than keys), m keys.
struct PagedSeq {
    int q0, n, m, p0;
    bool bad;
};

// `sound`: none of the starts 0 .. b falls; else the sequence is left out.
__device__ __forceinline__ PagedSeq paged_sequence(const PagedAttnParams &p, int b, bool sound)
{
    const PagedRows r = paged_rows(p.mask.q_starts, b, p.per, p.tokens);
    PagedSeq s;
    s.q0 = r.q0;
    s.n = sound ? paged_min(r.n, p.max_q) : 0;
    const int len = p.c.kv_lens[b];
    const long long room = static_cast<long long>(p.c.width) << p.c.log2_s;
    s.m = paged_max(len, 0);
    if (s.m > room) s.m = static_cast<int>(room);
    s.bad = r.bad || !sound || s.n != r.n || s.m != len;
    s.p0 = paged_max(s.m - r.given, -(1 << 30));
    return s;
}

// Four values of a CTA of the cluster (an address from peer_addr).
__device__ __forceinline__ float4 ld_peer_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// Eight channels of a row, joined over the cluster's parts: each has its maximum (to
// base 2), its sum and its unnormalised output at the same places of its shared
// memory. Returns the sum, and the maximum in `big`.
__device__ __forceinline__ float paged_join_peers(const float *o, const float *m, const float *l, int parts, float (&v)[8], float &big)
{
    big = -INFINITY;
    for (int s = 0; s < parts; ++s) big = fmaxf(big, ld_peer_f32(peer_addr(m, s)));
    const float base = big == -INFINITY ? 0.f : big;
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    for (int s = 0; s < parts; ++s) {
        const float f = exp2f(ld_peer_f32(peer_addr(m, s)) - base);
        total = fmaf(f, ld_peer_f32(peer_addr(l, s)), total);
        const uint32_t at = peer_addr(o, s);
        const float4 a = ld_peer_f32x4(at), b = ld_peer_f32x4(at + 16);
        v[0] = fmaf(f, a.x, v[0]); v[1] = fmaf(f, a.y, v[1]); v[2] = fmaf(f, a.z, v[2]); v[3] = fmaf(f, a.w, v[3]);
        v[4] = fmaf(f, b.x, v[4]); v[5] = fmaf(f, b.y, v[5]); v[6] = fmaf(f, b.z, v[6]); v[7] = fmaf(f, b.w, v[7]);
    }
    return total;
}

// CTAs that an SM holds, by their registers (which the launch bounds hold to this) and,
// bf16 pages, their rings. What the planner counts on: with three of every fp32 kernel,
// where some have room for two and others for five, clusters ran in waves, 26 us for 8
// sequences of 1008 tokens, 8 heads of 128, instead of 17.
constexpr int paged_simt_ctas(bool q4, int head_dim, int rows)
{
    return rows == 8 ? 2 : !q4 ? (head_dim == 128 ? 2 : rows == 1 ? 4 : 3) : head_dim == 128 ? (rows == 4 ? 3 : 4) : rows == 4 ? 4 : 5;
}
constexpr int paged_mma_ctas(bool q4, int rows) { return q4 && rows == 8 ? 3 : 2; }

// fp32 queries on the CUDA cores; rows: 1, 2, 4 or 8 of an item.
cudaError_t launch_paged_simt(const PagedAttnParams &p, int head_dim, bool q4, int rows, cudaStream_t st);
// bf16 queries on the tensor cores; rows: 8 or 16 of an item.
constexpr int kPagedMmaWarps = 4;
cudaError_t launch_paged_mma(const PagedAttnParams &p, int head_dim, bool q4, int rows, cudaStream_t st);
// Joins the parts: out = sum_s 2^(l_s - l) o_s, l = log2 sum_s 2^(l_s).
cudaError_t launch_paged_join(const PagedAttnParams &p, int head_dim, bool bf16, cudaStream_t st);

}  // namespace kvevict
