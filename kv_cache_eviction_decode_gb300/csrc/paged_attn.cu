// paged_attn.cu -- attention of fp32 queries over a paged cache, fp32 or 4 bits, on
// the CUDA cores, and the join of an attention's parts.
//
// out_i = sum_j 2^(z_ij - M_i) v_j / sum_j 2^(z_ij - M_i), z = q . k * scale *
// log2(e), M the running maximum of one pass. A warp takes tiles of 16 keys; a lane
// holds eight channels of up to eight query rows and of their outputs, D / 8 lanes a key.
// The partial products of a key are added up so that each lane ends with one row's
// logit (halving exchanges), which is also how softmax is spread. 8 sequences to 8000
// tokens, 8 heads of 128, one token each: 74 us (5.2 TB/s; with items of eight rows
// whatever there are and nothing read ahead the first version took 233); 32 heads over
// 8: 88 (237).
#include <cmath>

#include "launch.h"
#include "paged_attn.h"

namespace kvevict {

namespace {

constexpr int kSimtWarps = 4;
constexpr float kLn2 = 0.69314718055994531f;
constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Eight channels as they lie in a page: fp32, or the codes and the group's base and
// step.
template <bool Q4> struct Raw {
    static constexpr int kWords = Q4 ? 2 : 8;
    uint32_t w[kWords];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;  // (4 bits: base and step 0)
    }
    // Channels 8 s .. 8 s + 7 of row `slot` of a head's block in a page.
    template <int D> __device__ __forceinline__ void load(const char *block, int slot, long long token_bytes, int S, int s)
    {
        if constexpr (Q4) {
            const int j = s / 4, g = s % 4 * 2;
            const char *codes = block + slot * (D / 2) + 2 * j;
            w[0] = *reinterpret_cast<const uint16_t *>(codes + (D / 16) * g) |
                   static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(codes + (D / 16) * (g + 1))) << 16;
            w[1] = *reinterpret_cast<const uint32_t *>(block + S * (D / 2) + slot * (D / 8) + 4 * j);
        } else {
            const char *p = block + slot * token_bytes + 32 * s;
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(p + 4 * i);
                w[i] = x.x; w[i + 1] = x.y; w[i + 2] = x.z; w[i + 3] = x.w;
            }
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        if constexpr (Q4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(static_cast<float>(static_cast<int>(w[0] >> (4 * i) & 15u) - 8), q4_step(w[1]), q4_base(w[1]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
        }
    }
};

// R rows of an item: the arithmetic is per row, so an item of few is not computed as
// one of eight. With up to four, V's rows and the next tile's K are on their way
// while a tile's logits and products are made.
template <bool Q4, int D, int R>
__global__ void __launch_bounds__(kSimtWarps * 32, paged_simt_ctas(Q4, D, R)) paged_simt_kernel(const __grid_constant__ PagedAttnParams p)
{
    constexpr int kLanes = D / 8, kKeys = 32 / kLanes, U = kPagedTile / kKeys;  // lanes a key, keys at once, steps a tile
    constexpr int kShift = R == 8 ? (D == 128 ? 1 : 0) : R == 4 ? (D == 128 ? 2 : 1) : R == 2 ? (D == 128 ? 3 : 2) : (D == 128 ? 4 : 3);
    constexpr bool kAhead = R <= 4;
    __shared__ __align__(16) float s_o[kSimtWarps][R][D];
    __shared__ float s_m[kSimtWarps][R], s_l[kSimtWarps][R], s_cm[R], s_cl[R];  // a warp's, the CTA's
    grid_dependency_wait();
    const PagedCache &c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int item = blockIdx.x;
    const int part = item % p.splits;
    item /= p.splits;
    const int tile = item % p.q_tiles, unit = item / p.q_tiles;
    const int b = unit / c.Hkv, kvh = unit - b * c.Hkv;
    const PagedSeq sq = paged_sequence(p, b, !p.mask.q_starts || attn_first_fall(p.mask, b, lane) == INT_MAX);
    if (sq.bad && threadIdx.x == 0) atomicOr(c.err, KVEVICT_DEV_BAD_LENGTH);
    const int r0 = tile * R, nr = min(R, sq.n * p.G - r0);
    if (nr <= 0) return;
    const AttnKeys keys = attn_keys(p.mask, sq.m, sq.p0 + r0 / p.G, sq.p0 + (r0 + nr - 1) / p.G, kPagedTile);
    const int i_lo = static_cast<int>(static_cast<long long>(keys.count) * part / p.splits);
    const int i_hi = static_cast<int>(static_cast<long long>(keys.count) * (part + 1) / p.splits);

    const int s = lane & (kLanes - 1), kk = lane / kLanes;  // channels, key of a step
    float q[R][8], o[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[r][i] = o[r][i] = 0.f;
        if (r < nr) {
            const int t = (r0 + r) / p.G, g = r0 + r - t * p.G;
            load8(static_cast<const float *>(p.q) + (kvh * p.G + g) * p.qs[0] + (sq.q0 + t) * p.qs[1] + 8 * s, q[r]);
#pragma unroll
            for (int i = 0; i < 8; ++i) q[r][i] *= p.scale_log2;
        }
    }
    // the row whose softmax this lane keeps, and the keys it sees: j <= top, and j < n_sink or j >= low
    const int mine = s >> kShift;
    const int pos = sq.p0 + (r0 + mine) / p.G;
    const int top = mine < nr ? pos : -1, low = p.mask.window > 0 && pos >= p.mask.window ? pos - p.mask.window + 1 : 0;
    float m = -INFINITY, l = 0.f;

    auto seen = [&](int j) { return j < keys.sink || (j >= keys.lo && j < keys.hi); };
    // tile i's first key and page; the next one's page is looked up one tile ahead
    auto first_key = [&](int i) { return attn_tile_at(keys, i) * kPagedTile; };
    auto page_at = [&](int i) { return i < i_hi ? paged_page(c, b, first_key(i)) : -1; };
    auto load_tile = [&](Raw<Q4>(&x)[U], int which, int j0, int page) {
        const char *block = c.pages[which] + max(page, 0) * c.page_bytes[which] + kvh * c.head_bytes[which];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = u * kKeys + kk;
            x[u].zero();
            if (page >= 0 && seen(j0 + key)) x[u].template load<D>(block, (j0 & (c.S - 1)) + key, c.token_bytes[which], c.S, s);
        }
    };
    Raw<Q4> ks[kAhead ? U : 1], vs[kAhead ? U : 1];
    int page = page_at(i_lo + warp), page_next = page_at(i_lo + warp + kSimtWarps);
    if constexpr (kAhead) {
        if (i_lo + warp < i_hi) load_tile(ks, 0, first_key(i_lo + warp), page);
    }
    for (int i = i_lo + warp; i < i_hi; i += kSimtWarps) {
        const int j0 = first_key(i), page_after = page_at(i + 2 * kSimtWarps);
        if (page < 0) {
            if (lane == 0) atomicOr(c.err, KVEVICT_DEV_BAD_PAGE);
            if constexpr (kAhead) {
                if (i + kSimtWarps < i_hi) load_tile(ks, 0, first_key(i + kSimtWarps), page_next);
            }
            page = page_next;
            page_next = page_after;
            continue;
        }
        const char *kb = c.pages[0] + page * c.page_bytes[0] + kvh * c.head_bytes[0];
        const char *vb = c.pages[1] + page * c.page_bytes[1] + kvh * c.head_bytes[1];
        const int slot0 = j0 & (c.S - 1);
        if constexpr (kAhead) load_tile(vs, 1, j0, page);
        float z[U], mx = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = u * kKeys + kk, j = j0 + key;
            float k[8], d[R];
            if constexpr (kAhead) {
                ks[u].get(k);
            } else {
                Raw<Q4> x;
                x.zero();
                if (seen(j)) x.template load<D>(kb, slot0 + key, c.token_bytes[0], c.S, s);
                x.get(k);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                d[r] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) d[r] = fmaf(q[r][e], k[e], d[r]);
            }
            // a lane keeps the rows whose bits are its own, and sends the others; then the lanes of one row add up
#pragma unroll
            for (int w = R / 2; w; w >>= 1) {
                const int o_ = w << kShift;
                const bool high = s & o_;
#pragma unroll
                for (int r = 0; r < w; ++r) {
                    const float keep = high ? d[r + w] : d[r], send = high ? d[r] : d[r + w];
                    d[r] = keep + __shfl_xor_sync(kAll, send, o_);
                }
            }
#pragma unroll
            for (int o_ = (1 << kShift) / 2; o_; o_ >>= 1) d[0] += __shfl_xor_sync(kAll, d[0], o_);
            z[u] = seen(j) && j <= top && (j < p.mask.n_sink || j >= low) ? d[0] : -INFINITY;
            mx = fmaxf(mx, z[u]);
        }
        if constexpr (kAhead) {
            if (i + kSimtWarps < i_hi) load_tile(ks, 0, first_key(i + kSimtWarps), page_next);
        }
#pragma unroll
        for (int o_ = kLanes; o_ < 32; o_ <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, o_));
        const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn, f = exp2f(m - ms);
        m = mn;
        l *= f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            z[u] = exp2f(z[u] - ms);
            l += z[u];
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float fr = __shfl_sync(kAll, f, r << kShift);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[r][e] *= fr;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = u * kKeys + kk;
            float v[8];
            if constexpr (kAhead) {
                vs[u].get(v);
            } else {
                Raw<Q4> x;
                x.zero();
                if (seen(j0 + key)) x.template load<D>(vb, slot0 + key, c.token_bytes[1], c.S, s);
                x.get(v);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float w = __shfl_sync(kAll, z[u], (lane & ~(kLanes - 1)) | r << kShift);
                // (4 bits: a row that does not see the key takes nothing of it, whatever it stands for)
                if (Q4 && w == 0.f) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[r][e] = fmaf(w, v[e], o[r][e]);
            }
        }
        page = page_next;
        page_next = page_after;
    }

    // the keys of a step, then the warps
#pragma unroll
    for (int o_ = kLanes; o_ < 32; o_ <<= 1) {
        l += __shfl_xor_sync(kAll, l, o_);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) o[r][e] += __shfl_xor_sync(kAll, o[r][e], o_);
    }
    if (kk == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) s_o[warp][r][8 * s + e] = o[r][e];
        if ((s & ((1 << kShift) - 1)) == 0) {
            s_m[warp][mine] = m;
            s_l[warp][mine] = l;
        }
    }
    __syncthreads();
    auto join_warps = [&](int r, int ch, float(&v)[8], float &big) {
        float total = 0.f;
        big = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll
        for (int w = 0; w < kSimtWarps; ++w) big = fmaxf(big, s_m[w][r]);
        const float base = big == -INFINITY ? 0.f : big;
#pragma unroll
        for (int w = 0; w < kSimtWarps; ++w) {
            const float f = exp2f(s_m[w][r] - base);
            total = fmaf(f, s_l[w][r], total);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(f, s_o[w][r][ch + i], v[i]);
        }
        return total;
    };
    if (p.clusters) {
        // into the place of the first warp's part, where only this thread reads; then each CTA of the cluster joins a share
        for (int e = threadIdx.x; e < nr * kLanes; e += kSimtWarps * 32) {
            const int r = e / kLanes, ch = e % kLanes * 8;
            float v[8], big;
            const float total = join_warps(r, ch, v, big);
            store8(&s_o[0][r][ch], v);
            if (ch == 0) {
                s_cm[r] = big;
                s_cl[r] = total;
            }
        }
        cluster_sync();
    }
    const int share = p.clusters ? p.splits : 1, from = p.clusters ? part : 0;
    for (int e = threadIdx.x * share + from; e < nr * kLanes; e += kSimtWarps * 32 * share) {
        const int r = e / kLanes, ch = e % kLanes * 8;
        float v[8], big;
        const float total = p.clusters ? paged_join_peers(&s_o[0][r][ch], &s_cm[r], &s_cl[r], p.splits, v, big) : join_warps(r, ch, v, big);
        const float inv = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= inv;
        const float lse2 = total == 0.f ? -INFINITY : big + log2f(total);
        const int t = sq.q0 + (r0 + r) / p.G, h = kvh * p.G + (r0 + r) % p.G;
        const long long row = static_cast<long long>(t) * p.Hq + h;
        if (p.splits > 1 && !p.clusters) {
            const long long at = static_cast<long long>(part) * p.tokens * p.Hq + row;
            store8(p.part_o + at * D + ch, v);
            if (ch == 0) p.part_l[at] = lse2;
        } else {
            store8(static_cast<float *>(p.out) + h * p.os[0] + t * p.os[1] + ch, v);
            if (ch == 0 && p.lse) p.lse[row] = lse2 * kLn2;
        }
    }
    if (p.clusters) cluster_sync();  // no CTA's shared memory goes while another reads it
}

// One warp per query row: the parts' weights from their log2 normalisers, then
// D / 32 columns a lane.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedAttnParams p)
{
    constexpr int N = D / 32;
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long long rows = static_cast<long long>(p.c.batch) * p.Hq * p.max_q, slots = static_cast<long long>(p.tokens) * p.Hq;
    for (long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); w < rows; w += static_cast<long long>(gridDim.x) * 8) {
        const int h = static_cast<int>(w % p.Hq);
        const long long bt = w / p.Hq;
        const int b = static_cast<int>(bt / p.max_q), t0 = static_cast<int>(bt - static_cast<long long>(b) * p.max_q);
        const PagedSeq sq = paged_sequence(p, b, !p.mask.q_starts || attn_first_fall(p.mask, b, lane) == INT_MAX);
        if (t0 >= sq.n) continue;
        const int t = sq.q0 + t0;
        const long long row = static_cast<long long>(t) * p.Hq + h;
        float top = -INFINITY;
        for (int s = lane; s < p.splits; s += 32) top = fmaxf(top, p.part_l[s * slots + row]);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        const float base = top == -INFINITY ? 0.f : top;
        float acc[N], total = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.f;
        for (int s = 0; s < p.splits; ++s) {
            const float wgt = exp2f(p.part_l[s * slots + row] - base);
            if (wgt == 0.f) continue;  // nothing seen in this part
            float v[N];
            load_f32<float, N>(p.part_o + (s * slots + row) * D + lane * N, v);
            total += wgt;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(wgt, v[i], acc[i]);
        }
        const float inv = total > 0.f ? 1.f / total : total;
        T *po = static_cast<T *>(p.out) + h * p.os[0] + t * p.os[1] + lane * N;
#pragma unroll
        for (int i = 0; i < N; ++i) po[i] = Elem<T>::from_f32(acc[i] * inv);
        if (lane == 0 && p.lse) p.lse[row] = (total == 0.f ? -INFINITY : top + log2f(total)) * kLn2;
    }
}

template <int D, int R> cudaError_t simt_rows(const PagedAttnParams &p, bool q4, cudaStream_t st)
{
    const unsigned grid = static_cast<unsigned>(p.c.batch) * p.c.Hkv * p.q_tiles * p.splits;
    return launch_dependent(q4 ? paged_simt_kernel<true, D, R> : paged_simt_kernel<false, D, R>, grid, kSimtWarps * 32, 0, st, p,
                            p.clusters ? static_cast<unsigned>(p.splits) : 1u);
}

template <int D> cudaError_t simt_for(const PagedAttnParams &p, bool q4, int rows, cudaStream_t st)
{
    return rows == 1 ? simt_rows<D, 1>(p, q4, st) : rows == 2 ? simt_rows<D, 2>(p, q4, st) : rows == 4 ? simt_rows<D, 4>(p, q4, st) : simt_rows<D, 8>(p, q4, st);
}

template <typename T, int D> cudaError_t join_for(const PagedAttnParams &p, cudaStream_t st)
{
    const long long blocks = (static_cast<long long>(p.c.batch) * p.Hq * p.max_q + 7) / 8;
    return launch_dependent(paged_join_kernel<T, D>, static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, st, p);
}

}  // namespace

cudaError_t launch_paged_simt(const PagedAttnParams &p, int head_dim, bool q4, int rows, cudaStream_t st)
{
    return head_dim == 64 ? simt_for<64>(p, q4, rows, st) : simt_for<128>(p, q4, rows, st);
}

cudaError_t launch_paged_join(const PagedAttnParams &p, int head_dim, bool bf16, cudaStream_t st)
{
    if (bf16) return head_dim == 64 ? join_for<__nv_bfloat16, 64>(p, st) : join_for<__nv_bfloat16, 128>(p, st);
    return head_dim == 64 ? join_for<float, 64>(p, st) : join_for<float, 128>(p, st);
}

}  // namespace kvevict
