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
    long long turns[64];  // of a pair, see rot_turns
    int seq[kAppendTokens], page[kAppendTokens], slot[kAppendTokens], fall;
    long long pos[kAppendTokens];
};

__device__ __forceinline__ void find_places(const AppendParams &p, int tok0, int nt, Places &s)
{
    const PagedCache &c = p.c;
    const int tid = threadIdx.x;
    uint32_t bits = 0;
    if (tid >= kPagedThreads - p.R / 2) s.turns[kPagedThreads - 1 - tid] = rot_turns(p.freq[kPagedThreads - 1 - tid]);
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

// [tokens][R / 2] cosines and sines of the tokens' positions, by a whole block; ends
// with a barrier (and begins with one behind find_places).
__device__ __forceinline__ void form_cosines(const AppendParams &p, int nt, Places &s, float2 *cs)
{
    const int half = p.R / 2;
    for (int i = threadIdx.x; i < nt * half; i += kPagedThreads) {
        const int t = i / half;
        cs[i] = rot_cos_sin(s.turns[i - t * half], s.pos[t], p.scale);
    }
    __syncthreads();
}

// Pages of the keys' own type, rotary parts in whole 16-byte chunks. A unit of one
// thread is two chunks of a head (a pair rotary_dim / 2 apart, or neighbours), and a
// thread's units, kBatch of them, are all on their way while the CTA looks up its
// tokens' places and forms its cosines: three dependent reads, which took longer
// than the copying (13 prompts to 4097 tokens, 8 heads of 128, bf16: 28 us, 74% of the
// copy bandwidth; 73 with eight bytes a lane loaded behind the reads).
template <typename T, int D>
__global__ void __launch_bounds__(kPagedThreads) append_own_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int N = Vec<T>::N, kLanes = D / N / 2, kAtOnce = kPagedThreads / kLanes, kBatch = kAppendOwnBatch;
    extern __shared__ __align__(16) float2 cs[];  // [tokens_per][R / 2] cos, sin
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
            if (half && h0 < c.Hkv) form_cosines(p, nt, s, cs);
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

// Eight neighbouring elements as they are in memory.
template <typename T> struct Eight {
    static constexpr int kWords = 2 * sizeof(T);
    uint32_t w[kWords];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const char *p)
    {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(p + 4 * i);
            w[i] = x.x; w[i + 1] = x.y; w[i + 2] = x.z; w[i + 3] = x.w;
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 2) bf16x2_to_f32(w[i], v[2 * i], v[2 * i + 1]);
            else v[i] = __uint_as_float(w[i]);
        }
    }
    // Another lane's.
    __device__ __forceinline__ void from(int lane, float (&v)[8]) const
    {
        Eight o;
#pragma unroll
        for (int i = 0; i < kWords; ++i) o.w[i] = __shfl_sync(0xffffffffu, w[i], lane);
        o.get(v);
    }
};

// 4 bits. Eight neighbouring channels a lane: 32 j + 8 t .. of lane 4 j + t, so that a
// group of 32 is four lanes, whose minimum and maximum take two shuffles each, and
// goes out as two bytes for each of two neighbouring g. A channel's mate in the
// rotation is in the lane itself (interleaved) or a whole number of lanes away.
// Instructions bound it, not bytes, so that rows are walked by strides, keys first
// and then values, which need no rotation; kBatch rows of a thread are on their way
// at once, the first ones while the CTA looks up its tokens' places. (15,505 tokens
// of 8 heads of 128: 42 us, 3.4 times its bytes; before quotients were put right 38,
// and with four channels a lane 52.)
template <typename T, int D>
__global__ void __launch_bounds__(kPagedThreads) append_q4_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int kLanes = D / 8, kAtOnce = kPagedThreads / kLanes, kBatch = 4;
    extern __shared__ __align__(16) float2 cs[];  // [tokens_per][R / 2] cos, sin
    __shared__ Places s;
    __shared__ char *s_codes[2][kAppendTokens], *s_groups[2][kAppendTokens];
    grid_dependency_wait();
    const PagedCache &c = p.c;
    const int tid = threadIdx.x, lane = tid % kLanes, ch = lane * 8;
    const int tok0 = static_cast<int>(blockIdx.x / p.head_blocks) * p.tokens_per;
    const int nt = min(p.tokens_per, p.tokens - tok0);
    const int h0 = static_cast<int>(blockIdx.x % p.head_blocks) * p.heads_per, nh_all = min(p.heads_per, 2 * c.Hkv - h0);
    const int half = p.R / 2;
    const bool turns = ch < p.R, first = ch < half;
    const int mate = (tid & 31) + (p.inter || !turns ? 0 : first ? half / 8 : -(half / 8)), ang = p.inter ? ch / 2 : first ? ch : ch - half;
    const int byte = (D / 16) * 2 * (lane & 3) + 2 * (lane >> 2);
    bool ready = false;
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
        const int ha = w ? max(h0 - c.Hkv, 0) : h0, hz = w ? h0 + nh_all - c.Hkv : min(h0 + nh_all, c.Hkv), nh = hz - ha;
        if (nh <= 0) continue;
        const long long strides[3] = {0, p.xs[w][0], p.xs[w][1]};
        Walk in;
        const T *x0 = static_cast<const T *>(p.x[w]) + ha * p.xs[w][0] + ch;
        in.start(const_cast<char *>(reinterpret_cast<const char *>(x0)), strides, sizeof(T), 0, tok0, nh, kAtOnce, tid / kLanes, INT_MAX);
        const long long head_bytes = c.head_bytes[w];
        const int trips = (nt * nh + kAtOnce - 1) / kAtOnce;
#pragma unroll 1
        for (int trip = 0; trip < trips; trip += kBatch) {
            Eight<T> x[kBatch];
            int tk[kBatch], hd[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                x[u].zero();
                tk[u] = in.t;
                hd[u] = in.h;
                if (in.t < nt) x[u].load(in.p);
                in.on();
            }
            if (!ready) {
                find_places(p, tok0, nt, s);
                for (int i = tid; i < 2 * nt; i += kPagedThreads) {
                    const int v = i / nt, t = i - v * nt;
                    char *block = s.page[t] < 0 ? nullptr : c.pages[v] + s.page[t] * c.page_bytes[v];
                    s_codes[v][t] = block ? block + s.slot[t] * (D / 2) : nullptr;
                    s_groups[v][t] = block ? block + c.S * (D / 2) + s.slot[t] * (D / 8) : nullptr;
                }
                if (half && h0 < c.Hkv) form_cosines(p, nt, s, cs);
                else __syncthreads();
                ready = true;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (trip + u >= trips) break;
                float v[8];
                x[u].get(v);
                const int t = min(tk[u], nt - 1);
                if (!w && half) {  // (the same for every thread)
                    if (p.inter) {
                        if (turns) {
#pragma unroll
                            for (int i = 0; i < 8; i += 4) {
                                const float4 f = *reinterpret_cast<const float4 *>(cs + t * half + ang + i / 2);
                                const float a0 = v[i], b0 = v[i + 1], a1 = v[i + 2], b1 = v[i + 3];
                                v[i] = a0 * f.x - b0 * f.y;
                                v[i + 1] = a0 * f.y + b0 * f.x;
                                v[i + 2] = a1 * f.z - b1 * f.w;
                                v[i + 3] = a1 * f.w + b1 * f.z;
                            }
                        }
                    } else {
                        float o[8];
                        x[u].from(mate, o);
                        if (turns) {
                            const float sg = first ? -1.f : 1.f;
#pragma unroll
                            for (int i = 0; i < 8; i += 2) {
                                const float4 f = *reinterpret_cast<const float4 *>(cs + t * half + ang + i);
                                v[i] = v[i] * f.x + sg * o[i] * f.y;
                                v[i + 1] = v[i + 1] * f.z + sg * o[i + 1] * f.w;
                            }
                        }
                    }
                }
                float lo = v[0], hi = v[0], none = v[0] * 0.f;  // (none: NaN where one is not finite)
#pragma unroll
                for (int i = 1; i < 8; ++i) {
                    lo = fminf(lo, v[i]);
                    hi = fmaxf(hi, v[i]);
                    none = fmaf(v[i], 0.f, none);
                }
#pragma unroll
                for (int o = 2; o; o >>= 1) {
                    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
                    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                }
                const uint32_t fine = __ballot_sync(0xffffffffu, none == 0.f) >> (tid & 28) & 0xfu;
                uint32_t params;
                float base, step;
                q4_group(lo, hi, fine == 0xfu, params, base, step);
                char *const to = s_codes[w][t];
                if (tk[u] < nt && to) {
                    const long long head = (ha + hd[u]) * head_bytes;
                    q4_in_range(v, base, step);
                    const float inverse = q4_inverse(step);
                    *reinterpret_cast<uint16_t *>(to + head + byte) = q4_codes(v, base, step, inverse);
                    *reinterpret_cast<uint16_t *>(to + head + byte + D / 16) = q4_codes(v + 4, base, step, inverse);
                    if ((lane & 3) == 0) *reinterpret_cast<uint32_t *>(s_groups[w][t] + head + 4 * (lane >> 2)) = params;
                }
            }
        }
    }
}

// Rotary parts that the two kernels above do not take, own type and 4 bits, with the
// latter's layout; a channel's mate in the rotation is read from memory.
template <typename T, bool Q4, int D>
__global__ void __launch_bounds__(kPagedThreads) append_kernel(const __grid_constant__ AppendParams p)
{
    constexpr int kLanes = D / 4, kAtOnce = kPagedThreads / kLanes, kBatch = 4;
    extern __shared__ __align__(16) float2 cs[];  // [tokens_per][R / 2] cos, sin
    __shared__ Places s;
    grid_dependency_wait();
    const PagedCache &c = p.c;
    const int tid = threadIdx.x;
    const int tok0 = static_cast<int>(blockIdx.x / p.head_blocks) * p.tokens_per;
    const int nt = min(p.tokens_per, p.tokens - tok0);
    const int h0 = static_cast<int>(blockIdx.x % p.head_blocks) * p.heads_per, nh = min(p.heads_per, 2 * c.Hkv - h0);
    const int half = p.R / 2;
    bool ready = false;

    const int lane = tid % kLanes, ch = lane * 4;
    const bool turns = ch < p.R;
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
        if (!ready) {  // (the first loads are under way)
            find_places(p, tok0, nt, s);
            if (half && h0 < c.Hkv) form_cosines(p, nt, s, cs);
            ready = true;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const bool real = hh[u] >= 0, key = real && hh[u] < c.Hkv;
            float v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            if (key && turns) {
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
                uint32_t params;
                float base, step;
                q4_group(lo, hi, all == 0xffu, params, base, step);
                const int g = lane & 7, j = lane >> 3;
                q4_in_range(v, base, step);
                *reinterpret_cast<uint16_t *>(block + slot * (D / 2) + (D / 16) * g + 2 * j) = q4_codes(v, base, step, q4_inverse(step));
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
// side by side of every group), so that the results go out in 16-byte chunks. (16
// sequences to 16384 tokens, 8 heads of 128, 4 bits to bf16: 168 us, 99% of the copy
// bandwidth.)
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
    if (p.k_starts && blockIdx.x == 0) {  // (what has no rows is in no CTA's share)
        for (int j = tid; j < c.batch; j += kPagedThreads)
            if (paged_rows(p.k_starts, j, 0, p.rows).n == 0 && c.kv_lens[j] != 0) bits |= KVEVICT_DEV_BAD_LENGTH;
    }
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
    if (append_q4(p, q4)) kern = elem == 4 ? append_q4_kernel<float, D> : append_q4_kernel<__nv_bfloat16, D>;
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
