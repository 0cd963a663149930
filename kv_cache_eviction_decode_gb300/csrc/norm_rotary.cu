// norm_rotary.cu -- kvevict_norm_rotary: the root-mean-square norm of every head
// of queries and keys and its rotary positions, in one launch.
//
// y = x w r, r = 1 / sqrt(mean x^2 + eps), then every pair of y turns. A head is read
// once and written once; beside these bytes the instructions count (121 us for 16384
// tokens of 64 + 8 heads of 128 with an address worked out for each head, 108 now,
// 103 for the rotation alone in rotary.cu). So a head's lanes, a
// power of two of neighbours in a warp, take two 16-byte chunks each (a pair
// rotary_dim / 2 apart, or two of neighbouring pairs or of elements that do not
// turn), walk from head to head by adding strides, keep the weights as fp32, and
// fold r into cosine and sine. What a thread reads comes through places of its own
// in shared memory, three heads ahead, without registers and (since it reads only
// its own copies) without a barrier. All in fp32, rounded once.
#include <algorithm>
#include <cmath>

#include "launch.h"
#include "norm_rotary.h"
#include "rotary_common.cuh"

namespace kvevict {

namespace {

struct NormParams {
    RotParams r;
    const void *w[2];  // q's, k's weights
    float eps;
    uint32_t lanes;    // of a head: a power of two, at least half its chunks
};

// 16 bytes global -> shared without a register between.
__device__ __forceinline__ void copy16(uint4 *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T, bool INTER>
__global__ void __launch_bounds__(kRotThreads, 4) norm_rotary_kernel(const __grid_constant__ NormParams np)
{
    constexpr int N = Vec<T>::N, kLines = INTER ? N / 4 : N / 2;  // 16-byte lines of cosines and sines of a chunk (pair)
    const RotParams &p = np.r;
    extern __shared__ __align__(16) char sh[];
    uint4 *const own = reinterpret_cast<uint4 *>(sh) + threadIdx.x;                                     // [stages][2][threads]
    float4 *const cs = reinterpret_cast<float4 *>(sh + kNormStages * 2 * kRotThreads * 16);  // [tokens_per][lines][R / N, or half of it]
    __shared__ long long turns[kNormPairs];
    grid_dependency_wait();
    const int half = p.R / 2, chunks = p.D / N, turning = INTER ? p.R / N : half / N;  // (half layout: pairs of chunks)
    const int tok0 = blockIdx.x / p.head_blocks * p.tokens_per;
    const int nt = min(static_cast<int>(p.tokens_per), static_cast<int>(p.total - tok0));
    const int h0 = blockIdx.x % p.head_blocks * p.heads_per;
    const int nh_all = min(static_cast<int>(p.heads_per), p.heads[0] + p.heads[1] - h0);
    const int step = kRotThreads / np.lanes, first = threadIdx.x / np.lanes, u = threadIdx.x & (np.lanes - 1);
    const int tokens = static_cast<int>(p.tokens);
    const long long b0 = tok0 / tokens;
    const int t0 = tok0 - static_cast<int>(b0) * tokens;
    // this lane's chunks, and which lines of the table they use
    const bool mine = 2 * u < chunks, turn = INTER ? 2 * u < turning : u < turning, turn2 = INTER && 2 * u + 1 < turning;
    const int ca = !mine ? 0 : INTER ? 2 * u * N : u < turning ? u * N : p.R + 2 * (u - turning) * N;
    const int cb = !mine ? 0 : !INTER && u < turning ? ca + half : ca + N;
    const float over_d = 1.f / static_cast<float>(p.D);
    const int per_token = kLines * turning;
    bool ready = false;
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {  // queries, keys
        const int ha = w ? max(h0 - p.heads[0], 0) : h0, hz = w ? h0 + nh_all - p.heads[0] : min(h0 + nh_all, p.heads[0]);
        const int nh = hz - ha;
        if (nh <= 0) continue;
        Walk in, out;
        in.start(const_cast<char *>(static_cast<const char *>(p.x[w])) + (ha * p.xs[w][1] + ca) * static_cast<int>(sizeof(T)), p.xs[w], sizeof(T), b0, t0, nh, step,
                 first, tokens);
        out.start(static_cast<char *>(p.y[w]) + (ha * p.ys[w][1] + ca) * static_cast<int>(sizeof(T)), p.ys[w], sizeof(T), b0, t0, nh, step, first, tokens);
        const int apart = (cb - ca) * static_cast<int>(sizeof(T));
        int to = 0;
        auto load = [&]() {
            if (in.t < nt && mine) {
                copy16(own + to, in.p);
                copy16(own + to + kRotThreads, in.p + apart);
            }
            copies_close();
            to = to == (kNormStages - 1) * 2 * kRotThreads ? 0 : to + 2 * kRotThreads;
            in.on();
        };
#pragma unroll
        for (int i = 0; i < kNormStages - 1; ++i) load();
        float wa[N], wb[N];
        unpack16(*reinterpret_cast<const uint4 *>(static_cast<const T *>(np.w[w]) + ca), wa);
        unpack16(*reinterpret_cast<const uint4 *>(static_cast<const T *>(np.w[w]) + cb), wb);
        if (!ready) {
            for (int i = threadIdx.x; i < half; i += kRotThreads) turns[i] = rot_turns(p.freq[i]);
            __syncthreads();
            // pair f: (INTER) chunk 2 f / N, else pair of chunks f / N; lines of two pairs lie beside those of the other chunks
            for (int i = threadIdx.x; i < nt * half; i += kRotThreads) {
                const int lt = i / half, f = i - lt * half, in_chunk = INTER ? N / 2 : N;
                const int q = f / in_chunk, e = f - q * in_chunk;
                const int bt = tok0 + lt, b = bt / tokens;
                reinterpret_cast<float2 *>(cs)[((lt * kLines + e / 2) * turning + q) * 2 + (e & 1)] =
                    rot_cos_sin(turns[f], rot_position(p, b, bt - static_cast<long long>(b) * tokens), p.scale);
            }
            __syncthreads();
            ready = true;
        }
        const int trips = (nt * nh + step - 1) / step;
        int at = 0;
#pragma unroll 1
        for (int trip = 0; trip < trips; ++trip) {
            copies_wait<kNormStages - 2>();
            float v[N], z[N], sum = 0.f;
            const bool real = out.t < nt && mine;
            unpack16(real ? own[at] : make_uint4(0, 0, 0, 0), v);
            unpack16(real ? own[at + kRotThreads] : make_uint4(0, 0, 0, 0), z);
            at = at == (kNormStages - 1) * 2 * kRotThreads ? 0 : at + 2 * kRotThreads;
            load();
#pragma unroll
            for (int j = 0; j < N; ++j) {
                sum = fmaf(v[j], v[j], sum);
                sum = fmaf(z[j], z[j], sum);
            }
            for (uint32_t o = np.lanes / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float r = rsqrtf(fmaf(sum, over_d, np.eps));
            if (real) {
                const float4 *k = cs + out.t * per_token;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    v[j] *= wa[j];
                    z[j] *= wb[j];
                }
                if constexpr (INTER) {
#pragma unroll
                    for (int l = 0; l < 2; ++l) {
                        float(&x)[N] = l ? z : v;
                        if (l ? turn2 : turn) {
#pragma unroll
                            for (int j = 0; j < N; j += 4) {
                                const float4 c = k[j / 4 * turning + 2 * u + l];
                                const float a0 = x[j] * r, b0_ = x[j + 1] * r, a1 = x[j + 2] * r, b1 = x[j + 3] * r;
                                x[j] = a0 * c.x - b0_ * c.y;
                                x[j + 1] = a0 * c.y + b0_ * c.x;
                                x[j + 2] = a1 * c.z - b1 * c.w;
                                x[j + 3] = a1 * c.w + b1 * c.z;
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < N; ++j) x[j] *= r;
                        }
                    }
                } else if (turn) {
#pragma unroll
                    for (int j = 0; j < N; j += 2) {
                        const float4 c = k[j / 2 * turning + u];
                        const float c0 = c.x * r, s0 = c.y * r, c1 = c.z * r, s1 = c.w * r;
                        const float a0 = v[j], a1 = v[j + 1], e0 = z[j], e1 = z[j + 1];
                        v[j] = a0 * c0 - e0 * s0;
                        z[j] = a0 * s0 + e0 * c0;
                        v[j + 1] = a1 * c1 - e1 * s1;
                        z[j + 1] = a1 * s1 + e1 * c1;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        v[j] *= r;
                        z[j] *= r;
                    }
                }
                *reinterpret_cast<uint4 *>(out.p) = pack16(v);
                *reinterpret_cast<uint4 *>(out.p + apart) = pack16(z);
            }
            out.on();
        }
        copies_wait<0>();
    }
}

// Heads of more than 64 or an odd number of chunks, and rotary parts whose pairs do
// not fall into 16-byte chunks. One CTA per token, a warp per head, which passes through shared
// memory as fp32; it is read whole before any of it is written, so that in place
// needs no care.
template <typename T>
__global__ void __launch_bounds__(kRotThreads) norm_rotary_any_kernel(const __grid_constant__ NormParams np)
{
    constexpr int N = Vec<T>::N;
    const RotParams &p = np.r;
    extern __shared__ __align__(16) float2 cs[];  // [R / 2] cos, sin, then [8][D] floats
    const int half = p.R / 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *line = reinterpret_cast<float *>(cs + half) + warp * p.D;
    grid_dependency_wait();
    const long long bt = blockIdx.x;
    const long long b = bt / p.tokens, t = bt - b * p.tokens;
    if (half) {
        const long long pos = rot_position(p, b, t);
        for (int i = threadIdx.x; i < half; i += kRotThreads) cs[i] = rot_cos_sin(p.freq[i], pos, p.scale, false);
    }
    __syncthreads();
    for (int hh = warp; hh < p.heads[0] + p.heads[1]; hh += kRotThreads / 32) {
        const int k = hh >= p.heads[0], h = k ? hh - p.heads[0] : hh;
        const T *x = static_cast<const T *>(p.x[k]) + b * p.xs[k][0] + t * p.xs[k][2] + h * p.xs[k][1];
        T *y = static_cast<T *>(p.y[k]) + b * p.ys[k][0] + t * p.ys[k][2] + h * p.ys[k][1];
        const T *w = static_cast<const T *>(np.w[k]);
        float sum = 0.f;
        for (int c = lane * N; c < p.D; c += 32 * N) {
            float v[N];
            unpack16(*reinterpret_cast<const uint4 *>(x + c), v);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                sum = fmaf(v[j], v[j], sum);
                line[c + j] = v[j];
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float r = rsqrtf(sum / static_cast<float>(p.D) + np.eps);
        __syncwarp();
        for (int c = lane * N; c < p.D; c += 32 * N) {
            float v[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int d = c + j;
                v[j] = line[d] * (r * Elem<T>::to_f32(w[d]));
                if (d >= p.R) continue;
                const bool first = p.interleaved ? !(d & 1) : d < half;
                const int f = p.interleaved ? d >> 1 : (first ? d : d - half);
                const int mate = p.interleaved ? d ^ 1 : (first ? d + half : d - half);
                const float o = line[mate] * (r * Elem<T>::to_f32(w[mate]));
                v[j] = first ? v[j] * cs[f].x - o * cs[f].y : o * cs[f].y + v[j] * cs[f].x;
            }
            *reinterpret_cast<uint4 *>(y + c) = pack16(v);
        }
        __syncwarp();  // the line has been used
    }
}

long long norm_shares(NormParams &np)
{
    RotParams &p = np.r;
    const long long heads = p.heads[0] + p.heads[1], step = kRotThreads / np.lanes;
    p.heads_per = static_cast<uint32_t>(heads);
    p.head_blocks = 1;
    p.tokens_per = 1;
    if (p.total < kNormSlots / 2) {
        // few tokens: two trips of a CTA's threads at most
        const long long want = std::max(step, p.total * heads / (kNormSlots / 2));
        p.heads_per = static_cast<uint32_t>(std::min(heads, want));
        p.head_blocks = static_cast<uint32_t>((heads + p.heads_per - 1) / p.heads_per);
        return p.total * p.head_blocks;
    }
    p.tokens_per = static_cast<uint32_t>(norm_tokens(p.total, heads, step, p.R));
    return (p.total + p.tokens_per - 1) / p.tokens_per;
}

template <typename T> cudaError_t launch_norm(NormParams &np, bool chunks, uint32_t units, cudaStream_t st, int &rc)
{
    RotParams &p = np.r;
    if (chunks) {
        np.lanes = 1;
        while (np.lanes < units) np.lanes *= 2;
        const long long blocks = norm_shares(np);
        if (blocks >= (1LL << 31)) {
            rc = KVEVICT_ERR_INVALID_ARG;
            return cudaSuccess;
        }
        const size_t smem = static_cast<size_t>(p.tokens_per) * (p.R / 2) * sizeof(float2) + kNormOwn;
        auto kern = p.interleaved ? norm_rotary_kernel<T, true> : norm_rotary_kernel<T, false>;
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormOwn + kNormTable);
        if (e != cudaSuccess) return e;
        return launch_dependent(kern, static_cast<unsigned>(blocks), kRotThreads, smem, st, np);
    }
    const size_t smem = static_cast<size_t>(p.R / 2) * sizeof(float2) + static_cast<size_t>(kRotThreads / 32) * p.D * 4;
    return launch_dependent(norm_rotary_any_kernel<T>, static_cast<unsigned>(p.total), kRotThreads, smem, st, np);
}

}  // namespace

}  // namespace kvevict

using namespace kvevict;

extern "C" int kvevict_norm_rotary(const kvevict_norm_rotary_args *a, void *cuda_stream)
{
    if (!a) return KVEVICT_ERR_INVALID_ARG;
    NormParams np{};
    bool nothing;
    int rc = rot_prepare(&a->r, true, np.r, nothing);
    if (rc != KVEVICT_OK) return rc;
    if (!(a->eps >= 0.f) || !std::isfinite(a->eps)) return KVEVICT_ERR_INVALID_ARG;
    if (nothing) return KVEVICT_OK;
    RotParams &p = np.r;
    np.w[0] = a->q_weight;
    np.w[1] = a->k_weight;
    np.eps = a->eps;
    if (!a->k_weight != !a->r.k) return KVEVICT_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i)
        if (p.heads[i] && (!np.w[i] || (reinterpret_cast<uintptr_t>(np.w[i]) & 15))) return KVEVICT_ERR_INVALID_ARG;
    const int n = a->r.dtype == KVEVICT_F32 ? 4 : 8;  // elements of a chunk
    const uint32_t units = static_cast<uint32_t>(p.D / n / 2);  // pairs of chunks a head
    const bool chunks = p.D % (2 * n) == 0 && (p.interleaved ? p.R % n == 0 : p.R / 2 % n == 0) && units <= 32;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = n == 4 ? launch_norm<float>(np, chunks, units, st, rc) : launch_norm<__nv_bfloat16>(np, chunks, units, st, rc);
    return rc != KVEVICT_OK ? rc : e == cudaSuccess ? KVEVICT_OK : KVEVICT_ERR_CUDA;
}
