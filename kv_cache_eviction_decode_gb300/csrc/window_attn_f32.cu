// window_attn_f32.cu -- attention on the CUDA cores in fp32, and the join of
// an attention's parts.
//
// out_i = sum_j 2^(z_ij - M_i) v_j / sum_j 2^(z_ij - M_i), z = q . k * scale *
// log2(e), M the running maximum of one pass over the key tiles (each new
// maximum rescales the sum and the output by 2^(old - new)). A CTA of 16 x 16
// threads holds a tile of R query rows and walks the key tiles that the rows
// see; each thread owns R/16 rows x (tile / 16) keys of the logits and R/16 rows
// x D/16 columns of the output. V is copied while the logits are made and the
// next K during the product with V (cp.async, no registers between).
//
// R = 64, tiles of 64 keys: per 64 FFMA a warp issues 8 shared-memory loads (12
// wavefronts, below the 16 cycles that the FFMAs take at four warps a cycle). 8
// heads of 2048 x 128, causal: 415 us, 21 TFLOP/s, a quarter of the FP32 rate
// (518 with K and V loaded in turn into one buffer). With one CTA of 8 warps an SM
// (118,784 bytes of shared memory) the FMA pipe is busy in 48% of the cycles of an
// SM at work; and over the launch in 28%, because blocks start with a prompt's
// shortest tiles and the end waits for the longest.
// R = 16, tiles of 32 keys, four CTAs an SM: for few rows, where K and V are read
// for little arithmetic. 8 sequences of 8 heads, one token over 8000 keys of 128:
// 99 us, 5.3 TB/s (285 while the warps without rows computed theirs too: bound by
// shared-memory reads).
#include <cmath>

#include "launch.h"
#include "window_attn.h"
#include "window_attn_common.cuh"

namespace kvevict {

namespace {

constexpr int kThreadsF32 = 256;
constexpr float kLn2 = 0.69314718055994531f;

template <int D, int R> struct F32Layout {
    static constexpr int kBK = R == kAttnF32FewRows ? kAttnF32FewKeys : kAttnF32Keys;
    static constexpr int kQ = D + 4;    // padded rows: four floats apart, 8 rows cover the 32 banks
    static constexpr int kP = kBK + 4;
    static constexpr int kFloats = R * kQ + 2 * kBK * kQ + R * kP;
    static constexpr int kBytes = kFloats * 4;
    static constexpr int kCtas = kBytes <= 56 * 1024 ? 4 : kBytes <= 113 * 1024 ? 2 : 1;  // that an SM holds
};

// 16 bytes global -> shared without a register between, or 16 zero bytes.
__device__ __forceinline__ void copy16(float *dst, const float *src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All groups but the newest N have landed (this thread's own; a barrier makes them everyone's).
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }

__device__ __forceinline__ float half_max(float v)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float half_sum(float v)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// kPacked: starts give the sequences; apart, because their check costs a spill at
// 64 registers (8 x 8 heads, one token over 8000 keys of 128: 101.5 us with it in
// every kernel, 99 without).
template <int D, int R, bool kPacked>
__global__ void __launch_bounds__(kThreadsF32, (F32Layout<D, R>::kCtas)) attn_f32_kernel(const __grid_constant__ AttnParams ap)
{
    using L = F32Layout<D, R>;
    constexpr int kBK = L::kBK;
    constexpr int RM = R / 16;      // rows of a thread
    constexpr int KM = kBK / 16;    // keys of a thread
    constexpr int CV = D / 64;      // float4 columns of a thread's output
    extern __shared__ __align__(16) float fsm[];
    float *sQ = fsm, *sK = sQ + R * L::kQ, *sV = sK + kBK * L::kQ, *sP = sV + kBK * L::kQ;

    grid_dependency_wait();
    int item = blockIdx.x;
    const bool second = item >= ap.pr[0].n_items;
    if (second) item -= ap.pr[0].n_items;
    const AttnProblem &p = ap.pr[second ? 1 : 0];
    const int G = ap.G;
    const int part = item % p.splits;
    item /= p.splits;
    const int tile = item % p.q_tiles;
    const int unit = item / p.q_tiles;
    const int b = unit / ap.Hkv, kvh = unit - b * ap.Hkv;
    AttnSeq sq = attn_sequence(p, b, true);
    if constexpr (kPacked) {
        // (1,024 sequences of up to two tokens, 8 heads, the dearest case seen: 92 us, 85 without this)
        bool falls = false;
        for (int j = threadIdx.x; j <= b; j += kThreadsF32) falls = falls || attn_falls(p, j);
        if (__syncthreads_or(falls)) sq = attn_sequence(p, b, false);
    }
    if (sq.bad && threadIdx.x == 0) attn_flag(ap.err, KVEVICT_DEV_BAD_LENGTH);
    const int per = R / G;          // tokens of a tile
    const int t0 = tile * per;
    if (t0 >= sq.n) return;
    const int nt = min(per, sq.n - t0), nrows = nt * G;
    const AttnKeys keys = attn_keys(p, sq.m, sq.p0 + t0, sq.p0 + t0 + nt - 1, kBK);
    const int i_lo = static_cast<int>(static_cast<long long>(keys.count) * part / p.splits);
    const int i_hi = static_cast<int>(static_cast<long long>(keys.count) * (part + 1) / p.splits);

    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const float *qb = static_cast<const float *>(p.q) + (p.q_starts ? 0 : b * p.qs[0]) +
                  static_cast<long long>(kvh) * G * p.qs[1] + static_cast<long long>(sq.q0 + t0) * p.qs[2];
    const float *kb = static_cast<const float *>(p.k) + (p.k_starts ? 0 : b * p.ks[0]) + kvh * p.ks[1] + sq.k0 * p.ks[2];
    const float *vb = static_cast<const float *>(p.v) + (p.k_starts ? 0 : b * p.vs[0]) + kvh * p.vs[1] + sq.k0 * p.vs[2];

    for (int e = tid; e < R * (D / 4); e += kThreadsF32) {
        const int r = e / (D / 4), c = (e - r * (D / 4)) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < nrows) {
            const int t = r / G, g = r - t * G;
            v = load4(qb + g * p.qs[1] + t * p.qs[2] + c);
            v.x *= ap.scale_log2; v.y *= ap.scale_log2; v.z *= ap.scale_log2; v.w *= ap.scale_log2;
        }
        *reinterpret_cast<float4 *>(sQ + r * L::kQ + c) = v;
    }

    // the key positions that a thread's rows see: j <= top, and j < n_sink or j >= low
    int top[RM], low[RM];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const int pos = p.causal ? sq.p0 + t0 + (ty * RM + i) / G : sq.m - 1;
        top[i] = ty * RM + i < nrows ? pos : -1;
        low[i] = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
    }
    // a warp whose rows (two of the 16 row groups) all lie behind the last one only helps copying:
    // with a single row the others' shared-memory reads were what bound the loop
    const bool busy = (tid >> 5) * 2 * RM < nrows;
    float m[RM], l[RM];
    float4 o[RM][CV];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < CV; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }

    // Copies a K or V tile into shared memory, one group; the keys that no row of this tile of rows
    // sees are not read (their rows: zeros).
    auto load_tile = [&](float *dst, const float *base, long long stride, int j0) {
        for (int e = tid; e < kBK * (D / 4); e += kThreadsF32) {
            const int r = e / (D / 4), c = (e - r * (D / 4)) * 4;
            const int j = j0 + r;
            const bool seen = j < keys.sink || (j >= keys.lo && j < keys.hi);
            copy16(dst + r * L::kQ + c, seen ? base + j * stride + c : base, seen);
        }
        copies_close();
    };
    if (i_lo < i_hi) load_tile(sK, kb, p.ks[2], attn_tile_at(keys, i_lo) * kBK);

    for (int i = i_lo; i < i_hi; ++i) {
        const int j0 = attn_tile_at(keys, i) * kBK;
        __syncthreads();  // the previous tile's V has been used
        load_tile(sV, vb, p.vs[2], j0);
        copies_wait<1>();  // K; V lands while the logits are made
        __syncthreads();
        if (busy) {
            float s[RM][KM];
#pragma unroll
            for (int a = 0; a < RM; ++a)
#pragma unroll
                for (int c = 0; c < KM; ++c) s[a][c] = 0.f;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 qv[RM], kv[KM];
#pragma unroll
                for (int a = 0; a < RM; ++a) qv[a] = *reinterpret_cast<const float4 *>(sQ + (ty * RM + a) * L::kQ + d);
#pragma unroll
                for (int c = 0; c < KM; ++c) kv[c] = *reinterpret_cast<const float4 *>(sK + (tx + 16 * c) * L::kQ + d);
#pragma unroll
                for (int a = 0; a < RM; ++a)
#pragma unroll
                    for (int c = 0; c < KM; ++c) {
                        s[a][c] = fmaf(qv[a].x, kv[c].x, s[a][c]);
                        s[a][c] = fmaf(qv[a].y, kv[c].y, s[a][c]);
                        s[a][c] = fmaf(qv[a].z, kv[c].z, s[a][c]);
                        s[a][c] = fmaf(qv[a].w, kv[c].w, s[a][c]);
                    }
            }
#pragma unroll
            for (int a = 0; a < RM; ++a) {
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < KM; ++c) {
                    const int j = j0 + tx + 16 * c;
                    if (!(j <= top[a] && (j < p.n_sink || j >= low[a]))) s[a][c] = -INFINITY;
                    mx = fmaxf(mx, s[a][c]);
                }
                const float mn = fmaxf(m[a], half_max(mx));
                const float ms = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m[a] - ms);
                m[a] = mn;
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < KM; ++c) {
                    const float e = exp2f(s[a][c] - ms);
                    sum += e;
                    sP[(ty * RM + a) * L::kP + tx + 16 * c] = e;
                }
                l[a] = l[a] * f + half_sum(sum);
#pragma unroll
                for (int c = 0; c < CV; ++c) {
                    o[a][c].x *= f; o[a][c].y *= f; o[a][c].z *= f; o[a][c].w *= f;
                }
            }
        }
        __syncthreads();  // every thread has used K and written its probabilities
        if (i + 1 < i_hi) {
            load_tile(sK, kb, p.ks[2], attn_tile_at(keys, i + 1) * kBK);  // lands during the product with V
            copies_wait<1>();
        } else {
            copies_wait<0>();
        }
        __syncthreads();
        if (!busy) continue;
#pragma unroll 4
        for (int j = 0; j < kBK; j += 4) {
            float4 pv[RM];
#pragma unroll
            for (int a = 0; a < RM; ++a) pv[a] = *reinterpret_cast<const float4 *>(sP + (ty * RM + a) * L::kP + j);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
                for (int c = 0; c < CV; ++c) {
                    const float4 v = *reinterpret_cast<const float4 *>(sV + (j + jj) * L::kQ + tx * 4 + c * 64);
#pragma unroll
                    for (int a = 0; a < RM; ++a) {
                        const float w = jj == 0 ? pv[a].x : jj == 1 ? pv[a].y : jj == 2 ? pv[a].z : pv[a].w;
                        o[a][c].x = fmaf(w, v.x, o[a][c].x);
                        o[a][c].y = fmaf(w, v.y, o[a][c].y);
                        o[a][c].z = fmaf(w, v.z, o[a][c].z);
                        o[a][c].w = fmaf(w, v.w, o[a][c].w);
                    }
                }
            }
        }
    }

#pragma unroll
    for (int a = 0; a < RM; ++a) {
        const int r = ty * RM + a;
        if (r >= nrows) continue;
        const int t = sq.q0 + t0 + r / G, h = kvh * G + r % G;
        const long long row = b * p.rs[0] + h * p.rs[1] + t * p.rs[2];
        const float inv = l[a] > 0.f ? 1.f / l[a] : (l[a] == 0.f ? 0.f : l[a]);
        const float lse2 = l[a] == 0.f ? -INFINITY : m[a] + log2f(l[a]);
        if (ap.slots > 1) {
            const long long at = (p.slot0 + part) * ap.rows + row;
            float *po = ap.part_o + at * D;
#pragma unroll
            for (int c = 0; c < CV; ++c)
                store4(po + tx * 4 + c * 64, make_float4(o[a][c].x * inv, o[a][c].y * inv, o[a][c].z * inv, o[a][c].w * inv));
            if (tx == 0) ap.part_l[at] = lse2;
        } else {
            float *po = static_cast<float *>(ap.out) + b * p.os[0] + h * p.os[1] + t * p.os[2];
#pragma unroll
            for (int c = 0; c < CV; ++c)
                store4(po + tx * 4 + c * 64, make_float4(o[a][c].x * inv, o[a][c].y * inv, o[a][c].z * inv, o[a][c].w * inv));
            if (tx == 0 && ap.lse) ap.lse[row] = lse2 * kLn2;
        }
    }
}

// One warp per query row: the slots' weights from their log2 normalisers, then
// D / 32 columns a lane. Reads slots * (D + 1) * 4 bytes a row, written just
// before (they are in L2).
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnParams ap)
{
    constexpr int N = D / 32;
    const AttnProblem &p = ap.pr[ap.n_problems - 1];
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long long rows = static_cast<long long>(p.batch) * ap.Hq * p.max_q;
    for (long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); w < rows;
         w += static_cast<long long>(gridDim.x) * 8) {
        const int h = static_cast<int>(w % ap.Hq);
        const long long bt = w / ap.Hq;
        const int b = static_cast<int>(bt / p.max_q), t0 = static_cast<int>(bt - static_cast<long long>(b) * p.max_q);
        const AttnSeq sq = attn_sequence(p, b, !p.q_starts || attn_first_fall(p, b, lane) == INT_MAX);
        if (t0 >= sq.n) continue;
        const int t = sq.q0 + t0;
        const long long row = b * p.rs[0] + h * p.rs[1] + t * p.rs[2];
        float top = -INFINITY;
        for (int s = lane; s < ap.slots; s += 32) top = fmaxf(top, ap.part_l[s * ap.rows + row]);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float base = top == -INFINITY ? 0.f : top;
        float acc[N], total = 0.f;
#pragma unroll
        for (int c = 0; c < N; ++c) acc[c] = 0.f;
        for (int s = 0; s < ap.slots; ++s) {
            const float wgt = exp2f(ap.part_l[s * ap.rows + row] - base);
            if (wgt == 0.f) continue;  // nothing seen in this part (its output is not read)
            float v[N];
            load_f32<float, N>(ap.part_o + (s * ap.rows + row) * D + lane * N, v);
            total += wgt;
#pragma unroll
            for (int c = 0; c < N; ++c) acc[c] = fmaf(wgt, v[c], acc[c]);
        }
        const float inv = total > 0.f ? 1.f / total : total;
        T *po = static_cast<T *>(ap.out) + b * p.os[0] + h * p.os[1] + t * p.os[2] + lane * N;
#pragma unroll
        for (int c = 0; c < N; ++c) po[c] = Elem<T>::from_f32(acc[c] * inv);
        if (lane == 0 && ap.lse) ap.lse[row] = (total == 0.f ? -INFINITY : top + log2f(total)) * kLn2;
    }
}

template <int D, int R> cudaError_t launch_f32(const AttnParams &p, cudaStream_t st)
{
    auto kern = p.pr[0].q_starts ? attn_f32_kernel<D, R, true> : attn_f32_kernel<D, R, false>;
    constexpr int bytes = F32Layout<D, R>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, p.pr[0].n_items + (p.n_problems > 1 ? p.pr[1].n_items : 0), kThreadsF32, bytes, st, p);
}

template <typename T, int D> cudaError_t launch_join(const AttnParams &p, cudaStream_t st)
{
    const AttnProblem &q = p.pr[p.n_problems - 1];
    const long long rows = static_cast<long long>(q.batch) * p.Hq * q.max_q;
    const long long blocks = (rows + 7) / 8;
    return launch_dependent(attn_join_kernel<T, D>, static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, st, p);
}

}  // namespace

cudaError_t launch_attn_f32(const AttnParams &p, int head_dim, bool few, cudaStream_t st)
{
    if (head_dim == 64) return few ? launch_f32<64, 16>(p, st) : launch_f32<64, 64>(p, st);
    return few ? launch_f32<128, 16>(p, st) : launch_f32<128, 64>(p, st);
}

cudaError_t launch_attn_join(const AttnParams &p, int head_dim, bool bf16, cudaStream_t st)
{
    if (bf16) return head_dim == 64 ? launch_join<__nv_bfloat16, 64>(p, st) : launch_join<__nv_bfloat16, 128>(p, st);
    return head_dim == 64 ? launch_join<float, 64>(p, st) : launch_join<float, 128>(p, st);
}

}  // namespace kvevict
