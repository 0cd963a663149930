// paged_move.cu -- tokens into the pages of a cache (kvevict_paged_append) and out
// of them (kvevict_paged_gather). Both are bound by bytes.
#include "launch.h"
#include "paged_move.h"
#include "rotary_common.cuh"

namespace kvevict {

namespace {

// Four neighbouring elements as fp32 values, and back.
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p)
{
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    float4 v;
    bf16x2_to_f32(w.x, v.x, v.y);
    bf16x2_to_f32(w.y, v.z, v.w);
    return v;
}
__device__ __forceinline__ void store4(float *p, const float (&v)[4]) { *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&v)[4])
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// The places of the tokens tok0 .. tok0 + nt - 1 and their positions, by a whole
// block; ends with a barrier.
struct Places {
    int seq[kAppendTokens], page[kAppendTokens], slot[kAppendTokens], fall;
    long long pos[kAppendTokens];
};

__device__ __forceinline__ void find_places(const AppendParams &p, int tok0, int nt, Places &s)
{
    const PagedCache &c = p.c;
    const int tid = threadIdx.x;
    uint32_t bits = 0;
    if (p.starts) paged_owners<kPagedThreads>(p.starts, c.batch, p.tokens, tok0, nt, s.seq, &s.fall, bits);
    if (tid < nt) {
        const int t = tok0 + tid, b = p.starts ? s.seq[tid] : t / p.per;
        int page = -1, slot = 0;
        long long pos = 0;
        if (b >= 0) {
            const PagedRows r = paged_rows(p.starts, b, p.per, p.tokens);
            const long long i = static_cast<long long>(c.kv_lens[b]) - r.given + (t - r.q0);  // the token's place
            if (i < 0 || i >= static_cast<long long>(c.width) << c.log2_s) {
                bits |= KVEVICT_DEV_BAD_LENGTH;
            } else {
                page = paged_page(c, b, i);
                if (page < 0) bits |= KVEVICT_DEV_BAD_PAGE;
                slot = static_cast<int>(i) & (c.S - 1);
            }
            pos = !p.pos ? i : p.pos64 ? static_cast<const long long *>(p.pos)[t * p.ps] : static_cast<const int *>(p.pos)[t * p.ps];
        }
        s.page[tid] = page;
        s.slot[tid] = slot;
        s.pos[tid] = pos;
    }
    if (bits) atomicOr(c.err, bits);
    __syncthreads();
}

// Pages of the keys' own type, rotary parts in whole 16-byte chunks. A unit of one
// thread is two chunks of a head (a pair rotary_dim / 2 apart, or neighbours), and a
// thread's units, kBatch of them, are all on their way while the CTA looks up its
// tokens' places and forms its cosines: three dependent reads, which took longer
// than the copying.
template <typename T, int D>
__global__ void __launch_bounds__(kPagedThreads) append_own_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int N = Vec<T>::N, kLanes = D / N / 2, kAtOnce = kPagedThreads / kLanes, kBatch = kAppendOwnBatch;
    extern __shared__ float2 cs[];  // [tokens_per][R / 2] cos, sin
    __shared__ Places s;
    grid_dependency_wait();
    const PagedCache &c = p.c;
    const int tid = threadIdx.x, u = tid % kLanes;
    const int tok0 = static_cast<int>(blockIdx.x / p.head_blocks) * p.tokens_per;
    const int nt = min(p.tokens_per, p.tokens - tok0);
    const int h0 = static_cast<int>(blockIdx.x % p.head_blocks) * p.heads_per, nh = min(p.heads_per, 2 * c.Hkv - h0);
    const int half = p.R / 2, rows = nt * nh, pairs = p.inter ? 0 : half / N;
    // this lane's chunks of a key; a value's are the two halves of a row
    const int ka = p.inter ? 2 * u * N : u < pairs ? u * N : p.R + 2 * (u - pairs) * N, kb = !p.inter && u < pairs ? ka + half : ka + N;
    bool ready = false;
    for (int row0 = 0; row0 < rows; row0 += kAtOnce * kBatch) {
        uint4 a[kBatch], b[kBatch];
        int lt[kBatch], hh[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int row = row0 + i * kAtOnce + tid / kLanes;
            lt[i] = row / nh;
            hh[i] = row < rows ? h0 + row - lt[i] * nh : -1;
            if (hh[i] < 0) continue;
            const int v = hh[i] >= c.Hkv, h = v ? hh[i] - c.Hkv : hh[i];
            const T *x = static_cast<const T *>(p.x[v]) + h * p.xs[v][0] + (tok0 + lt[i]) * p.xs[v][1];
            a[i] = *reinterpret_cast<const uint4 *>(x + (v ? u * N : ka));
            b[i] = *reinterpret_cast<const uint4 *>(x + (v ? u * N + D / 2 : kb));
        }
        if (!ready) {
            find_places(p, tok0, nt, s);
            if (half && h0 < c.Hkv) {
                for (int i = tid; i < nt * half; i += kPagedThreads) {
                    const int t = i / half;
                    cs[i] = rot_cos_sin(p.freq[i - t * half], s.pos[t], p.scale, false);
                }
                __syncthreads();
            }
            ready = true;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (hh[i] < 0 || s.page[lt[i]] < 0) continue;
            const int v = hh[i] >= c.Hkv, h = v ? hh[i] - c.Hkv : hh[i];
            T *y = reinterpret_cast<T *>(c.pages[v] + s.page[lt[i]] * c.page_bytes[v] + h * c.head_bytes[v] + s.slot[lt[i]] * c.token_bytes[v]);
            if (!v && ka < p.R) {
                const float2 *k = cs + lt[i] * half;
                float x[N], z[N];
                unpack16(a[i], x);
                unpack16(b[i], z);
                if (p.inter) {
#pragma unroll
                    for (int l = 0; l < 2; ++l) {
                        float(&w)[N] = l ? z : x;
                        const int ch = l ? kb : ka;
                        if (ch >= p.R) continue;
#pragma unroll
                        for (int j = 0; j < N; j += 2) {
                            const float2 f = k[ch / 2 + j / 2];
                            const float e = w[j], o = w[j + 1];
                            w[j] = e * f.x - o * f.y;
                            w[j + 1] = e * f.y + o * f.x;
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float2 f = k[ka + j];
                        const float e = x[j], o = z[j];
                        x[j] = e * f.x - o * f.y;
                        z[j] = e * f.y + o * f.x;
                    }
                }
                a[i] = pack16(x);
                b[i] = pack16(z);
            }
            *reinterpret_cast<uint4 *>(y + (v ? u * N : ka)) = a[i];
            *reinterpret_cast<uint4 *>(y + (v ? u * N + D / 2 : kb)) = b[i];
        }
    }
}

// Four neighbouring channels a lane: channels 32 j + 4 g + i are lane 8 j + g of a
// head's D / 4 lanes, so that a group of 32 is eight lanes, whose minimum and
// maximum take three shuffles, and a lane's four codes are two bytes side by side.
// A channel's mate in the rotation is in the lane itself (interleaved) or a whole
// number of lanes away (rotary_dim a multiple of 8); only other rotary dims read
// it from memory. For 4 bits, and for rotary parts that no whole chunks make up. A CTA takes `tokens_per` tokens x `heads_per` of the heads of k
// and v; its places in the pages and its cosines are found once. kBatch heads a warp
// (D = 64: two at a time) are in flight.
template <typename T, bool Q4, int D>
__global__ void __launch_bounds__(kPagedThreads) append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int kLanes = D / 4, kAtOnce = kPagedThreads / kLanes, kBatch = 4;
    extern __shared__ float2 cs[];  // [tokens_per][R / 2] cos, sin
    __shared__ Places s;
    grid_dependency_wait();
    const PagedCache &c = p.c;
    const int tid = threadIdx.x;
    const int tok0 = static_cast<int>(blockIdx.x / p.head_blocks) * p.tokens_per;
    const int nt = min(p.tokens_per, p.tokens - tok0);
    const int h0 = static_cast<int>(blockIdx.x % p.head_blocks) * p.heads_per, nh = min(p.heads_per, 2 * c.Hkv - h0);
    find_places(p, tok0, nt, s);
    const int half = p.R / 2;
    if (half && h0 < c.Hkv) {
        for (int i = tid; i < nt * half; i += kPagedThreads) {
            const int lt = i / half;
            cs[i] = rot_cos_sin(p.freq[i - lt * half], s.pos[lt], p.scale, false);
        }
        __syncthreads();
    }

    const int lane = tid % kLanes, ch = lane * 4;
    // where a lane's mates are: in itself, `far` lanes off, or (found one by one) anywhere
    const bool by_lane = !p.inter && half % 4 == 0, turns = ch < p.R;
    const bool first = ch < half;
    const int far = first ? half / 4 : -(half / 4);
    const int rows = nt * nh;
    for (int row0 = 0; row0 < rows; row0 += kAtOnce * kBatch) {
        float4 x[kBatch];
        int lt[kBatch], hh[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int row = row0 + u * kAtOnce + tid / kLanes;
            x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            lt[u] = row / nh;
            hh[u] = h0 + row - lt[u] * nh;
            if (row >= rows) {
                hh[u] = -1;
                continue;
            }
            const int v = hh[u] >= c.Hkv, h = v ? hh[u] - c.Hkv : hh[u];
            x[u] = load4(static_cast<const T *>(p.x[v]) + h * p.xs[v][0] + (tok0 + lt[u]) * p.xs[v][1] + ch);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const bool real = hh[u] >= 0, key = real && hh[u] < c.Hkv;
            float v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            if (by_lane && half) {  // (the same for every thread)
                const int mate = (tid & 31) + (turns ? far : 0);
                const float o[4] = {__shfl_sync(0xffffffffu, v[0], mate), __shfl_sync(0xffffffffu, v[1], mate),
                                    __shfl_sync(0xffffffffu, v[2], mate), __shfl_sync(0xffffffffu, v[3], mate)};
                if (key && turns) {
                    const float2 *k = cs + lt[u] * half + (first ? ch : ch - half);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = first ? v[i] * k[i].x - o[i] * k[i].y : o[i] * k[i].y + v[i] * k[i].x;
                }
            } else if (key && turns) {
                const float2 *k = cs + lt[u] * half;
                if (p.inter) {
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        if (ch + i >= p.R) continue;
                        const float2 w = k[ch / 2 + i / 2];
                        const float a = v[i], b = v[i + 1];
                        v[i] = a * w.x - b * w.y;
                        v[i + 1] = a * w.y + b * w.x;
                    }
                } else {
                    const T *xr = static_cast<const T *>(p.x[0]) + hh[u] * p.xs[0][0] + (tok0 + lt[u]) * p.xs[0][1];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int d = ch + i;
                        if (d >= p.R) continue;
                        const bool low = d < half;
                        const float o = Elem<T>::to_f32(xr[low ? d + half : d - half]);
                        const float2 w = k[low ? d : d - half];
                        v[i] = low ? v[i] * w.x - o * w.y : o * w.y + v[i] * w.x;
                    }
                }
            }
            const int page = real ? s.page[lt[u]] : -1, slot = real ? s.slot[lt[u]] : 0;
            const int which = real && !key, h = which ? hh[u] - c.Hkv : hh[u];
            char *block = c.pages[which] + page * c.page_bytes[which] + h * c.head_bytes[which];
            if constexpr (Q4) {
                float lo = fminf(fminf(v[0], v[1]), fminf(v[2], v[3])), hi = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
                bool fine = true;
#pragma unroll
                for (int i = 0; i < 4; ++i) fine = fine && isfinite(v[i]);
#pragma unroll
                for (int o = 4; o; o >>= 1) {
                    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
                    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                }
                const uint32_t all = __ballot_sync(0xffffffffu, fine) >> (tid & 24) & 0xffu;
                if (page < 0) continue;
                uint32_t params, codes = 0;
                float base, step;
                q4_group(lo, hi, all == 0xffu, params, base, step);
#pragma unroll
                for (int i = 0; i < 4; ++i) codes |= q4_code(v[i], base, step) << (4 * i);
                const int g = lane & 7, j = lane >> 3;
                *reinterpret_cast<uint16_t *>(block + slot * (D / 2) + (D / 16) * g + 2 * j) = static_cast<uint16_t>(codes);
                if (g == 0) *reinterpret_cast<uint32_t *>(block + c.S * (D / 2) + slot * (D / 8) + 4 * j) = params;
            } else {
                if (page < 0) continue;
                store4(reinterpret_cast<T *>(block + slot * c.token_bytes[which]) + ch, v);
            }
        }
    }
}

// A CTA takes kGatherRows rows of one head, keys and values, which it finds in the
// pages once. Own type: 16-byte chunks, eight of a thread in flight. 4 bits: a unit
// of one thread is an eighth of a row's codes twice (neighbouring g: eight channels
// side by side of every group), so that the results go out in 16-byte chunks.
template <typename T, bool Q4, int D>
__global__ void __launch_bounds__(kPagedThreads) gather_kernel(const __grid_constant__ GatherParams p)
{
    __shared__ int s_seq[kGatherRows], s_page[kGatherRows], s_slot[kGatherRows], s_fall;
    grid_dependency_wait();
    const PagedCache &c = p.c;
    const int tid = threadIdx.x;
    const int h = static_cast<int>(blockIdx.x % c.Hkv);
    const int rest = static_cast<int>(blockIdx.x / c.Hkv), tile = rest % p.tiles, b0 = rest / p.tiles;
    const int row0 = tile * kGatherRows, count = min(kGatherRows, p.rows - row0);
    uint32_t bits = 0;
    if (p.k_starts) paged_owners<kPagedThreads>(p.k_starts, c.batch, p.rows, row0, count, s_seq, &s_fall, bits);
    if (tid < count) {
        const int b = p.k_starts ? s_seq[tid] : b0;
        int page = -1;
        long long i = row0 + tid;
        if (b >= 0) {
            const int len = c.kv_lens[b];
            const long long room = min(static_cast<long long>(c.width) << c.log2_s, static_cast<long long>(INT_MAX));
            long long most = p.rows;
            if (p.k_starts) {
                const PagedRows r = paged_rows(p.k_starts, b, 0, p.rows);
                i -= r.q0;
                most = r.n;
            }
            if (len < 0 || len > room || len > most) bits |= KVEVICT_DEV_BAD_LENGTH;
            if (i < len && i < room) {
                page = paged_page(c, b, i);
                if (page < 0) bits |= KVEVICT_DEV_BAD_PAGE;
            }
        }
        s_page[tid] = page;
        s_slot[tid] = static_cast<int>(i) & (c.S - 1);
    }
    if (bits) atomicOr(c.err, bits);
    __syncthreads();
    constexpr int N = 16 / sizeof(T);
    if constexpr (!Q4) {
        constexpr int kChunks = D / N, kUnits = kGatherRows * 2 * kChunks / kPagedThreads, kBatch = kUnits < 8 ? kUnits : 8;
#pragma unroll
        for (int u0 = 0; u0 < kUnits; u0 += kBatch) {
            uint4 v[kBatch];
            T *y[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int e = (u0 + u) * kPagedThreads + tid, which = e / (kGatherRows * kChunks), r = e / kChunks % kGatherRows;
                const int ch = e % kChunks * N;
                y[u] = nullptr;
                if (r >= count || s_page[r] < 0) continue;
                const int row = row0 + r;
                y[u] = static_cast<T *>(p.y[which]) + (p.k_starts ? 0 : b0 * p.ys[which][0]) + h * p.ys[which][1] + row * p.ys[which][2] + ch;
                v[u] = *reinterpret_cast<const uint4 *>(c.pages[which] + s_page[r] * c.page_bytes[which] + h * c.head_bytes[which] +
                                                        s_slot[r] * c.token_bytes[which] + ch * static_cast<int>(sizeof(T)));
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (y[u]) *reinterpret_cast<uint4 *>(y[u]) = v[u];
        }
    } else {
        constexpr int kUnits = kGatherRows * 2 * 4 / kPagedThreads, kGroups = D / 32, kWords = D / 32;  // words of codes a unit
        uint32_t w[kUnits][kWords], bs[kUnits][kGroups];
        T *y[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int e = u * kPagedThreads + tid, which = e / (kGatherRows * 4), r = e / 4 % kGatherRows, t = e % 4;
            y[u] = nullptr;
            if (r >= count || s_page[r] < 0) continue;
            y[u] = static_cast<T *>(p.y[which]) + (p.k_starts ? 0 : b0 * p.ys[which][0]) + h * p.ys[which][1] + (row0 + r) * p.ys[which][2] + 8 * t;
            const char *block = c.pages[which] + s_page[r] * c.page_bytes[which] + h * c.head_bytes[which];
            const char *codes = block + s_slot[r] * (D / 2) + t * (D / 8), *params = block + c.S * (D / 2) + s_slot[r] * (D / 8);
            if constexpr (D == 128) {
                *reinterpret_cast<uint4 *>(w[u]) = *reinterpret_cast<const uint4 *>(codes);
                *reinterpret_cast<uint4 *>(bs[u]) = *reinterpret_cast<const uint4 *>(params);
            } else {
                *reinterpret_cast<uint2 *>(w[u]) = *reinterpret_cast<const uint2 *>(codes);
                *reinterpret_cast<uint2 *>(bs[u]) = *reinterpret_cast<const uint2 *>(params);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            if (!y[u]) continue;
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                // group j: half-word j of the first g's codes, then of the second's
                const uint32_t eight = __byte_perm(w[u][j / 2], w[u][kWords / 2 + j / 2], j % 2 ? 0x7632 : 0x5410);
                const float base = q4_base(bs[u][j]), step = q4_step(bs[u][j]);
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = fmaf(static_cast<float>(static_cast<int>(eight >> (4 * i) & 15u) - 8), step, base);
                if constexpr (sizeof(T) == 2) {
                    *reinterpret_cast<uint4 *>(y[u] + 32 * j) = pack16(v);
                } else {
                    *reinterpret_cast<float4 *>(y[u] + 32 * j) = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4 *>(y[u] + 32 * j + 4) = make_float4(v[4], v[5], v[6], v[7]);
                }
            }
        }
    }
}

template <int D> cudaError_t append_for(const AppendParams &p, int elem, bool q4, cudaStream_t st)
{
    const unsigned grid = static_cast<unsigned>((p.tokens + p.tokens_per - 1) / p.tokens_per) * p.head_blocks;
    const size_t smem = static_cast<size_t>(p.tokens_per) * (p.R / 2) * sizeof(float2);
    auto kern = elem == 4 ? (q4 ? append_kernel<float, true, D> : append_kernel<float, false, D>)
                          : (q4 ? append_kernel<__nv_bfloat16, true, D> : append_kernel<__nv_bfloat16, false, D>);
    if (append_own(p, elem, q4)) kern = elem == 4 ? append_own_kernel<float, D> : append_own_kernel<__nv_bfloat16, D>;
    return launch_dependent(kern, grid, kPagedThreads, smem, st, p);
}

template <int D> cudaError_t gather_for(const GatherParams &p, int elem, bool q4, cudaStream_t st)
{
    const unsigned grid = static_cast<unsigned>(p.tiles) * p.c.Hkv * (p.k_starts ? 1 : p.c.batch);
    auto kern = elem == 4 ? (q4 ? gather_kernel<float, true, D> : gather_kernel<float, false, D>)
                          : (q4 ? gather_kernel<__nv_bfloat16, true, D> : gather_kernel<__nv_bfloat16, false, D>);
    return launch_dependent(kern, grid, kPagedThreads, 0, st, p);
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, int head_dim, int elem, bool q4, cudaStream_t st)
{
    return head_dim == 64 ? append_for<64>(p, elem, q4, st) : append_for<128>(p, elem, q4, st);
}

cudaError_t launch_gather(const GatherParams &p, int head_dim, int elem, bool q4, cudaStream_t st)
{
    return head_dim == 64 ? gather_for<64>(p, elem, q4, st) : gather_for<128>(p, elem, q4, st);
}

}  // namespace kvevict
