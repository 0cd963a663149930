// paged_attn.cu -- attention over a paged cache on the CUDA cores, and the join of
// an attention's parts.
//
// out_i = sum_j 2^(z_ij - M_i) v_j / sum_j 2^(z_ij - M_i), z = q . k * scale *
// log2(e), M the running maximum of one pass. A warp takes tiles of 16 keys; a lane
// holds eight channels of eight query rows and of their outputs, D / 8 lanes a key.
// The partial products of a key are added up so that each lane ends with one row's
// logit (three halving exchanges), which is also how softmax is spread.
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
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8])
{
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    bf16x2_to_f32(w.x, v[0], v[1]);
    bf16x2_to_f32(w.y, v[2], v[3]);
    bf16x2_to_f32(w.z, v[4], v[5]);
    bf16x2_to_f32(w.w, v[6], v[7]);
}

template <typename T> __device__ __forceinline__ void store8(T *p, const float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = Elem<T>::from_f32(v[i]);
}

// Channels 8 s .. 8 s + 7 of row `slot` of a head's block in a page.
template <typename T, bool Q4, int D>
__device__ __forceinline__ void page_row8(const char *block, int slot, long long token_bytes, int S, int s, float (&v)[8])
{
    if constexpr (Q4) {
        const int j = s / 4, g = s % 4 * 2;
        const char *codes = block + slot * (D / 2) + 2 * j;
        const uint32_t w = *reinterpret_cast<const uint16_t *>(codes + (D / 16) * g) |
                           static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(codes + (D / 16) * (g + 1))) << 16;
        const uint32_t bs = *reinterpret_cast<const uint32_t *>(block + S * (D / 2) + slot * (D / 8) + 4 * j);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fmaf(static_cast<float>(static_cast<int>(w >> (4 * i) & 15u) - 8), q4_step(bs), q4_base(bs));
    } else {
        load8(reinterpret_cast<const T *>(block + slot * token_bytes) + 8 * s, v);
    }
}

template <typename T, bool Q4, int D>
__global__ void __launch_bounds__(kSimtWarps * 32) paged_simt_kernel(const __grid_constant__ PagedAttnParams p)
{
    constexpr int R = kPagedSimtRows, kLanes = D / 8, kKeys = 32 / kLanes, U = kPagedTile / kKeys;  // keys at once, steps a tile
    constexpr int kRowShift = D == 128 ? 1 : 0;  // D = 128: two lanes hold the same row's logit
    __shared__ float s_o[kSimtWarps][R][D], s_m[kSimtWarps][R], s_l[kSimtWarps][R];
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
            load8(static_cast<const T *>(p.q) + (kvh * p.G + g) * p.qs[0] + (sq.q0 + t) * p.qs[1] + 8 * s, q[r]);
#pragma unroll
            for (int i = 0; i < 8; ++i) q[r][i] *= p.scale_log2;
        }
    }
    // the row whose softmax this lane keeps, and the keys it sees: j <= top, and j < n_sink or j >= low
    const int mine = s >> kRowShift;
    const int pos = sq.p0 + (r0 + mine) / p.G;
    const int top = mine < nr ? pos : -1, low = p.mask.window > 0 && pos >= p.mask.window ? pos - p.mask.window + 1 : 0;
    float m = -INFINITY, l = 0.f;

    for (int i = i_lo + warp; i < i_hi; i += kSimtWarps) {
        const int j0 = attn_tile_at(keys, i) * kPagedTile;
        const int page = paged_page(c, b, j0);
        if (page < 0) {
            if (lane == 0) atomicOr(c.err, KVEVICT_DEV_BAD_PAGE);
            continue;
        }
        const char *kb = c.pages[0] + page * c.page_bytes[0] + kvh * c.head_bytes[0];
        const char *vb = c.pages[1] + page * c.page_bytes[1] + kvh * c.head_bytes[1];
        const int slot0 = j0 & (c.S - 1);
        float z[U], mx = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = u * kKeys + kk, j = j0 + key;
            const bool seen = j < keys.sink || (j >= keys.lo && j < keys.hi);
            float k[8], d[R];
#pragma unroll
            for (int e = 0; e < 8; ++e) k[e] = 0.f;
            if (seen) page_row8<T, Q4, D>(kb, slot0 + key, c.token_bytes[0], c.S, s, k);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                d[r] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) d[r] = fmaf(q[r][e], k[e], d[r]);
            }
            // a lane keeps the rows whose bits are its own, and sends the others
#pragma unroll
            for (int w = 4; w; w >>= 1) {
                const int o_ = w << kRowShift;
                const bool high = s & o_;
#pragma unroll
                for (int r = 0; r < w; ++r) {
                    const float keep = high ? d[r + w] : d[r], send = high ? d[r] : d[r + w];
                    d[r] = keep + __shfl_xor_sync(kAll, send, o_);
                }
            }
            if (kRowShift) d[0] += __shfl_xor_sync(kAll, d[0], 1);
            z[u] = seen && j <= top && (j < p.mask.n_sink || j >= low) ? d[0] : -INFINITY;
            mx = fmaxf(mx, z[u]);
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
            const float fr = __shfl_sync(kAll, f, r << kRowShift);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[r][e] *= fr;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int key = u * kKeys + kk, j = j0 + key;
            const bool seen = j < keys.sink || (j >= keys.lo && j < keys.hi);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
            if (seen) page_row8<T, Q4, D>(vb, slot0 + key, c.token_bytes[1], c.S, s, v);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float w = __shfl_sync(kAll, z[u], (lane & ~(kLanes - 1)) | r << kRowShift);
                // (4 bits: a row that does not see the key takes nothing of it, whatever it stands for)
                if (Q4 && w == 0.f) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[r][e] = fmaf(w, v[e], o[r][e]);
            }
        }
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
        if ((s & ((1 << kRowShift) - 1)) == 0) {
            s_m[warp][mine] = m;
            s_l[warp][mine] = l;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < nr * kLanes; e += kSimtWarps * 32) {
        const int r = e / kLanes, ch = e % kLanes * 8;
        float big = -INFINITY, total = 0.f, v[8];
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
        const float inv = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= inv;
        const float lse2 = total == 0.f ? -INFINITY : big + log2f(total);
        const int t = sq.q0 + (r0 + r) / p.G, h = kvh * p.G + (r0 + r) % p.G;
        const long long row = static_cast<long long>(t) * p.Hq + h;
        if (p.splits > 1) {
            const long long at = static_cast<long long>(part) * p.tokens * p.Hq + row;
            store8(p.part_o + at * D + ch, v);
            if (ch == 0) p.part_l[at] = lse2;
        } else {
            store8(static_cast<T *>(p.out) + h * p.os[0] + t * p.os[1] + ch, v);
            if (ch == 0 && p.lse) p.lse[row] = lse2 * kLn2;
        }
    }
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

template <typename T, int D> cudaError_t simt_for(const PagedAttnParams &p, bool q4, cudaStream_t st)
{
    const unsigned grid = static_cast<unsigned>(p.c.batch) * p.c.Hkv * p.q_tiles * p.splits;
    return launch_dependent(q4 ? paged_simt_kernel<T, true, D> : paged_simt_kernel<T, false, D>, grid, kSimtWarps * 32, 0, st, p);
}

template <typename T, int D> cudaError_t join_for(const PagedAttnParams &p, cudaStream_t st)
{
    const long long blocks = (static_cast<long long>(p.c.batch) * p.Hq * p.max_q + 7) / 8;
    return launch_dependent(paged_join_kernel<T, D>, static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, st, p);
}

}  // namespace

cudaError_t launch_paged_simt(const PagedAttnParams &p, int head_dim, bool bf16, bool q4, cudaStream_t st)
{
    if (bf16) return head_dim == 64 ? simt_for<__nv_bfloat16, 64>(p, q4, st) : simt_for<__nv_bfloat16, 128>(p, q4, st);
    return head_dim == 64 ? simt_for<float, 64>(p, q4, st) : simt_for<float, 128>(p, q4, st);
}

cudaError_t launch_paged_join(const PagedAttnParams &p, int head_dim, bool bf16, cudaStream_t st)
{
    if (bf16) return head_dim == 64 ? join_for<__nv_bfloat16, 64>(p, st) : join_for<__nv_bfloat16, 128>(p, st);
    return head_dim == 64 ? join_for<float, 64>(p, st) : join_for<float, 128>(p, st);
}

}  // namespace kvevict
