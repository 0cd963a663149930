// window_attn_common.cuh -- what the attention kernels share: a sequence's
// lengths as read (and clamped) from the device, and the key tiles that a
// range of query positions sees.
#pragma once

#include <climits>

#include "device_common.cuh"
#include "kvevict_ops.h"
#include "window_attn.h"

namespace kvevict {

__device__ __forceinline__ void attn_flag(uint32_t *err, uint32_t bit) { atomicOr(err, bit); }

__host__ __device__ __forceinline__ int attn_min(int a, int b) { return a < b ? a : b; }
__host__ __device__ __forceinline__ int attn_max(int a, int b) { return a > b ? a : b; }

// One sequence: where its rows start (token index), how many there are, and
// the position of the first (negative where there are more queries than keys).
// Values from the device are clamped to the tensors and to max_q; the position
// is counted from the queries given, so that the rows of a sequence cut at its
// end see no key that lies behind them.
struct AttnSeq {
    int q0, n, k0, m, p0;
    bool bad;
};

// Whether sequence j of a packed batch ends before it starts.
__host__ __device__ __forceinline__ bool attn_falls(const AttnProblem &p, int j) { return p.q_starts[j] > p.q_starts[j + 1]; }

// The first of the sequences 0 .. upto that does, or INT_MAX; by a whole warp.
__device__ __forceinline__ int attn_first_fall(const AttnProblem &p, int upto, int lane)
{
    for (int j0 = 0; j0 <= upto; j0 += 128) {
        int at = INT_MAX;
#pragma unroll
        for (int u = 3; u >= 0; --u) {
            const int j = j0 + 32 * u + lane;
            if (j <= upto && attn_falls(p, j)) at = j;
        }
        at = __reduce_min_sync(0xffffffffu, at);
        if (at != INT_MAX) return at;
    }
    return INT_MAX;
}

// `sound`: none of the sequences 0 .. b of a packed batch falls. Otherwise b is
// left out: its rows could be an earlier sequence's, and a comparison with its
// neighbours alone would not show that (starts 0, 20, 10, 15, 40: the last one
// ascends again, inside the first one's rows). The rows of sound sequences are
// disjoint, because their starts ascend.
__host__ __device__ __forceinline__ AttnSeq attn_sequence(const AttnProblem &p, int b, bool sound)
{
    AttnSeq s;
    s.bad = false;
    int given;  // queries from the first row to the end given
    if (p.q_starts) {
        const int a0 = p.q_starts[b], a1 = p.q_starts[b + 1], c0 = p.k_starts[b], c1 = p.k_starts[b + 1];
        s.q0 = attn_min(attn_max(a0, 0), p.q_rows);
        given = attn_max(a1, s.q0) - s.q0;
        const int q1 = attn_min(s.q0 + given, p.q_rows);
        s.n = attn_min(q1 - s.q0, p.max_q);
        s.k0 = attn_min(attn_max(c0, 0), p.k_rows);
        const int k1 = attn_min(attn_max(c1, s.k0), p.k_rows);
        s.m = k1 - s.k0;
        s.bad = s.q0 != a0 || q1 != a1 || s.n != q1 - s.q0 || s.k0 != c0 || k1 != c1;
        if (!sound) {
            s.n = 0;
            s.bad = true;
        }
    } else {
        s.q0 = s.k0 = 0;
        const int n = p.q_lens ? p.q_lens[b] : p.q_rows, m = p.k_lens ? p.k_lens[b] : p.k_rows;
        s.n = attn_min(attn_max(n, 0), p.q_rows);
        s.m = attn_min(attn_max(m, 0), p.k_rows);
        s.bad = s.n != n || s.m != m;
        given = attn_max(n, 0);
    }
    // (a position below -2^30 sees nothing, nor does any of the 2^30 rows behind it)
    s.p0 = attn_max(s.m - given, -(1 << 30));
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
