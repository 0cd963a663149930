// window_attn_common.cuh -- what the attention kernels share: a sequence's
// lengths as read (and clamped) from the device, and the key tiles that a
// range of query positions sees.
#pragma once

#include "device_common.cuh"
#include "kvevict_ops.h"
#include "window_attn.h"

namespace kvevict {

__device__ __forceinline__ void attn_flag(uint32_t *err, uint32_t bit)
{
    if (err) atomicOr(err, bit);
}

// One sequence: where its rows start (token index), how many there are, and
// the position of its first query (negative where there are more queries than
// keys). Values from the device are clamped to the tensors.
struct AttnSeq {
    int q0, n, k0, m, p0;
    bool bad;
};

__device__ __forceinline__ AttnSeq attn_sequence(const AttnProblem &p, int b)
{
    AttnSeq s;
    s.bad = false;
    if (p.q_starts) {
        const int a0 = p.q_starts[b], a1 = p.q_starts[b + 1], c0 = p.k_starts[b], c1 = p.k_starts[b + 1];
        s.q0 = min(max(a0, 0), p.q_rows);
        const int q1 = min(max(a1, s.q0), p.q_rows);
        s.n = min(q1 - s.q0, p.max_q);
        s.k0 = min(max(c0, 0), p.k_rows);
        const int k1 = min(max(c1, s.k0), p.k_rows);
        s.m = k1 - s.k0;
        s.bad = s.q0 != a0 || q1 != a1 || s.n != q1 - s.q0 || s.k0 != c0 || k1 != c1;
        if (b > 0 && p.q_starts[b - 1] > a0) {  // its rows would be an earlier sequence's
            s.n = 0;
            s.bad = true;
        }
    } else {
        s.q0 = s.k0 = 0;
        const int n = p.q_lens ? p.q_lens[b] : p.q_rows, m = p.k_lens ? p.k_lens[b] : p.k_rows;
        s.n = min(max(n, 0), p.q_rows);
        s.m = min(max(m, 0), p.k_rows);
        s.bad = s.n != n || s.m != m;
    }
    s.p0 = s.m - s.n;
    return s;
}

// The keys that queries at positions pa .. pb (pa <= pb) see between them:
// [0, sink) and [lo, hi), sink <= lo unless empty; as tiles of `tile` keys, a
// list of `count`: sink_tiles first tiles, then those from main0 on.
struct AttnKeys {
    int sink, lo, hi;
    int sink_tiles, main0, count;
};

__device__ __forceinline__ AttnKeys attn_keys(const AttnProblem &p, int m, int pa, int pb, int tile)
{
    AttnKeys r;
    if (!p.causal) pa = pb = m - 1;
    r.hi = min(pb, m - 1) + 1;
    if (r.hi <= 0) {
        r.sink = r.lo = r.hi = r.sink_tiles = r.main0 = r.count = 0;
        return r;
    }
    r.lo = p.window > 0 && pa >= p.window ? pa - p.window + 1 : 0;
    r.sink = min(p.n_sink, r.lo);
    r.sink_tiles = (r.sink + tile - 1) / tile;
    r.main0 = max(r.lo / tile, r.sink_tiles);
    const int end = (r.hi + tile - 1) / tile;
    r.count = r.sink_tiles + max(0, end - r.main0);
    return r;
}

__device__ __forceinline__ int attn_tile_at(const AttnKeys &r, int i)
{
    return i < r.sink_tiles ? i : r.main0 + i - r.sink_tiles;
}

}  // namespace kvevict
