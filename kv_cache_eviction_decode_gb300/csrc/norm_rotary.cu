// norm_rotary.cu -- kvevict_norm_rotary: the root-mean-square norm of every head
// of queries and keys and its rotary positions, in one launch.
//
// y = x r w, r = 1 / sqrt(mean x^2 + eps), then every pair of y turns. Bound by
// bytes: a head is read once and written once, so its lanes keep it in registers
// while its squares are summed. A head's lanes are a power of two of neighbours in
// a warp (its units of 16-byte chunks, as in rotary.cu: a pair of chunks
// rotary_dim / 2 apart, a chunk of neighbouring pairs, or one that does not turn);
// the sum takes log2 of them shuffles, and nothing else is exchanged. All in fp32,
// rounded once.
#include <algorithm>
#include <cmath>

#include "launch.h"
#include "rotary_common.cuh"

namespace kvevict {

namespace {

struct NormParams {
    RotParams r;
    const void *w[2];  // q's, k's weights
    float eps;
    uint32_t lanes;    // of a head: a power of two, at least its units
};

// Units of one thread, as in rotary_kernel. A thread's unit within the head stays;
// it walks the CTA's heads, kBatch of them in flight.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kRotThreads, 4) norm_rotary_kernel(const __grid_constant__ NormParams np)
{
    constexpr int N = Vec<T>::N, kBatch = INTER ? 4 : 2;
    const RotParams &p = np.r;
    extern __shared__ float2 cs[];  // [tokens_per][R / 2] cos, sin
    grid_dependency_wait();
    const uint32_t half = p.R / 2;
    const uint32_t pairs = INTER ? 0 : half / N;
    const uint32_t units = INTER ? p.D / N : pairs + (p.D - p.R) / N;
    const uint32_t tok0 = blockIdx.x / p.head_blocks * p.tokens_per;
    const uint32_t nt = min(p.tokens_per, static_cast<uint32_t>(p.total) - tok0);
    const uint32_t h0 = blockIdx.x % p.head_blocks * p.heads_per;
    const uint32_t nh = min(p.heads_per, static_cast<uint32_t>(p.heads[0] + p.heads[1]) - h0);
    const uint32_t step = kRotThreads / np.lanes, u = threadIdx.x & (np.lanes - 1);
    const bool mine = u < units;
    const bool two = !INTER && u < pairs;
    const uint32_t c = !mine ? 0 : INTER || u < pairs ? u * N : p.R + (u - pairs) * N;
    const uint32_t rows = nt * nh;
    uint32_t row = threadIdx.x / np.lanes;
    const float over_d = 1.f / static_cast<float>(p.D);
    bool ready = false;
    for (uint32_t row0 = 0; row0 < rows; row0 += step * kBatch) {
        uint4 a[kBatch], b[kBatch];
        T *y[kBatch];
        uint32_t tk[kBatch];
        bool key[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i, row += step) {
            y[i] = nullptr;
            key[i] = false;
            a[i] = b[i] = make_uint4(0, 0, 0, 0);
            tk[i] = row / nh;
            if (row >= rows || !mine) continue;
            const uint32_t hh = h0 + row - tk[i] * nh;
            const bool k = hh >= static_cast<uint32_t>(p.heads[0]);
            const uint32_t hl = k ? hh - p.heads[0] : hh;
            const uint32_t bt = tok0 + tk[i], bb = bt / static_cast<uint32_t>(p.tokens), t = bt - bb * static_cast<uint32_t>(p.tokens);
            const T *x = static_cast<const T *>(p.x[k]) + bb * p.xs[k][0] + t * p.xs[k][2] + hl * p.xs[k][1] + c;
            y[i] = static_cast<T *>(p.y[k]) + bb * p.ys[k][0] + t * p.ys[k][2] + hl * p.ys[k][1] + c;
            key[i] = k;
            a[i] = *reinterpret_cast<const uint4 *>(x);
            if (two) b[i] = *reinterpret_cast<const uint4 *>(x + half);
        }
        if (!ready) {
            for (uint32_t i = threadIdx.x; i < nt * half; i += kRotThreads) {
                const uint32_t t0 = i / half, bt = tok0 + t0, bb = bt / static_cast<uint32_t>(p.tokens);
                const long long t = bt - bb * static_cast<uint32_t>(p.tokens);
                cs[i] = rot_cos_sin(p.freq[i - t0 * half], rot_position(p, bb, t), p.scale, false);
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float v[N], z[N], sum = 0.f;
            unpack16(a[i], v);
            unpack16(b[i], z);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                sum = fmaf(v[j], v[j], sum);
                if (!INTER) sum = fmaf(z[j], z[j], sum);
            }
            for (uint32_t o = np.lanes / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (!y[i]) continue;
            const float r = rsqrtf(fmaf(sum, over_d, np.eps));
            const T *wp = static_cast<const T *>(np.w[key[i]]) + c;
            const float2 *k = cs + tk[i] * half + (INTER ? c / 2 : c);
            float w[N];
            unpack16(*reinterpret_cast<const uint4 *>(wp), w);
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] *= r * w[j];
            if (INTER) {
                if (c < static_cast<uint32_t>(p.R)) {
#pragma unroll
                    for (int j = 0; j < N; j += 2) {
                        const float x = v[j], e = v[j + 1];
                        v[j] = x * k[j / 2].x - e * k[j / 2].y;
                        v[j + 1] = x * k[j / 2].y + e * k[j / 2].x;
                    }
                }
            } else if (two) {
                unpack16(*reinterpret_cast<const uint4 *>(wp + half), w);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float x = v[j], e = z[j] * (r * w[j]);
                    v[j] = x * k[j].x - e * k[j].y;
                    z[j] = x * k[j].y + e * k[j].x;
                }
                *reinterpret_cast<uint4 *>(y[i] + half) = pack16(z);
            }
            *reinterpret_cast<uint4 *>(y[i]) = pack16(v);
        }
    }
}

// Heads of more than 32 units, and rotary parts whose pairs do not fall into
// 16-byte chunks. One CTA per token, a warp per head, which passes through shared
// memory as fp32; it is read whole before any of it is written, so that in place
// needs no care.
template <typename T>
__global__ void __launch_bounds__(kRotThreads) norm_rotary_any_kernel(const __grid_constant__ NormParams np)
{
    constexpr int N = Vec<T>::N;
    const RotParams &p = np.r;
    extern __shared__ float2 cs[];  // [R / 2] cos, sin, then [8][D] floats
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

template <typename T> cudaError_t launch_norm(NormParams &np, bool chunks, uint32_t units, cudaStream_t st, int &rc)
{
    RotParams &p = np.r;
    if (chunks) {
        np.lanes = 1;
        while (np.lanes < units) np.lanes *= 2;
        const long long blocks = rot_shares(p, units);
        if (blocks >= (1LL << 31)) {
            rc = KVEVICT_ERR_INVALID_ARG;
            return cudaSuccess;
        }
        const size_t smem = static_cast<size_t>(p.tokens_per) * (p.R / 2) * sizeof(float2);
        auto kern = p.interleaved ? norm_rotary_kernel<T, true> : norm_rotary_kernel<T, false>;
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
    const uint32_t units = static_cast<uint32_t>(p.interleaved ? p.D / n : p.R / 2 / n + (p.D - p.R) / n);
    const bool chunks = (p.interleaved ? p.R % n == 0 : p.R / 2 % n == 0) && p.D % n == 0 && units <= 32;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = n == 4 ? launch_norm<float>(np, chunks, units, st, rc) : launch_norm<__nv_bfloat16>(np, chunks, units, st, rc);
    return rc != KVEVICT_OK ? rc : e == cudaSuccess ? KVEVICT_OK : KVEVICT_ERR_CUDA;
}
