// rotary.cu -- kvevict_rotary: rotary positions for queries and keys, in one
// launch.
//
// Bound by bytes: x is read once and written once. The angle of (token, pair)
// is the same for every head, so a CTA takes one token, forms its cosines and
// sines once in shared memory and applies them to all heads of q and k. The
// angle itself is formed in turns as a 64-bit binary fraction: with F =
// round(inv_freq / 2 pi * 2^64), pos * F mod 2^64 is the angle modulo one turn,
// exactly up to F's own rounding -- an integer multiply does the range
// reduction, for any position, where an fp32 product would have lost the
// fraction past a few thousand turns.
#include <cmath>
#include <cstdint>

#include "device_common.cuh"
#include "kvevict_ops.h"

namespace kvevict {

namespace {

constexpr int kRotThreads = 256;

struct RotParams {
    const void *x[2];      // q, k
    void *y[2];
    long long xs[2][3], ys[2][3];
    int heads[2];
    const void *pos;
    int pos64;
    long long ps0, ps1, pos_start;
    const double *freq;
    float scale;
    int D, R, interleaved, inverse;
    long long tokens, total;  // total = batch * tokens
};

// 16-byte vectors of T as fp32 values.
template <typename T> struct Vec {
    static constexpr int N = 16 / sizeof(T);
};

__device__ __forceinline__ void ld16(const float *p, float (&v)[4])
{
    const float4 w = *reinterpret_cast<const float4 *>(p);
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
}
__device__ __forceinline__ void ld16(const __nv_bfloat16 *p, float (&v)[8])
{
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    bf16x2_to_f32(w.x, v[0], v[1]);
    bf16x2_to_f32(w.y, v[2], v[3]);
    bf16x2_to_f32(w.z, v[4], v[5]);
    bf16x2_to_f32(w.w, v[6], v[7]);
}
__device__ __forceinline__ void st16(float *p, const float (&v)[4])
{
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void st16(__nv_bfloat16 *p, const float (&v)[8])
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                               pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ float2 rot_cos_sin(double freq, long long pos, float scale, bool inverse)
{
    // freq in [-pi, pi]: half a turn at most, so the fraction fits a signed 64-bit integer
    const long long f = __double2ll_rn(freq * (0.15915494309189535 * 18446744073709551616.0));
    const long long frac = static_cast<long long>(static_cast<unsigned long long>(pos) * static_cast<unsigned long long>(f));
    const float half_turns = static_cast<float>(frac) * 1.0842021724855044e-19f;  // 2^-63
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * scale, inverse ? -s * scale : s * scale);
}

// One CTA per token. A thread takes 16-byte chunks of the output; an element
// of the rotary part reads its partner element by itself (from L1: another
// thread of the warp reads the same line). In place, all reads of a pass come
// before its writes.
template <typename T>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotParams p)
{
    constexpr int N = Vec<T>::N;
    extern __shared__ float2 cs[];  // [R / 2] cos, sin
    const long long bt = blockIdx.x;
    const long long b = bt / p.tokens, t = bt - b * p.tokens;
    const long long at = b * p.ps0 + t * p.ps1;
    const long long pos = !p.pos ? p.pos_start + t
                                 : (p.pos64 ? static_cast<const long long *>(p.pos)[at]
                                            : static_cast<long long>(static_cast<const int *>(p.pos)[at]));
    const int half = p.R / 2;
    for (int i = threadIdx.x; i < half; i += kRotThreads) cs[i] = rot_cos_sin(p.freq[i], pos, p.scale, p.inverse);
    __syncthreads();
    const int chunks = p.D / N;
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
        const T *x = static_cast<const T *>(p.x[w]) + b * p.xs[w][0] + t * p.xs[w][2];
        T *y = static_cast<T *>(p.y[w]) + b * p.ys[w][0] + t * p.ys[w][2];
        const int per = kRotThreads / chunks;  // whole heads a pass
        const int lh = threadIdx.x / chunks, c = (threadIdx.x - lh * chunks) * N;
        for (int h0 = 0; h0 < p.heads[w]; h0 += per) {
            const int h = h0 + lh;
            const bool mine = lh < per && h < p.heads[w];
            float v[N];
            if (mine) {
                const T *xr = x + h * p.xs[w][1];
                ld16(xr + c, v);
                if (c < p.R) {
#pragma unroll
                    for (int u = 0; u < N; ++u) {
                        const int d = c + u;
                        if (d >= p.R) continue;
                        const int f = p.interleaved ? d >> 1 : (d < half ? d : d - half);
                        const bool first = p.interleaved ? !(d & 1) : d < half;
                        const int mate = p.interleaved ? d ^ 1 : (first ? d + half : d - half);
                        const float o = Elem<T>::to_f32(xr[mate]);
                        const float2 k = cs[f];
                        v[u] = first ? v[u] * k.x - o * k.y : o * k.y + v[u] * k.x;
                    }
                }
            }
            if (x == y) __syncthreads();
            if (mine) st16(y + h * p.ys[w][1] + c, v);
        }
    }
}

bool rot_tensor_ok(const void *x, const void *y, const int64_t (&xs)[3], const int64_t (&ys)[3], int elem)
{
    if (!x || !y || (reinterpret_cast<uintptr_t>(x) & 15) || (reinterpret_cast<uintptr_t>(y) & 15)) return false;
    for (int i = 0; i < 3; ++i) {
        if ((xs[i] * elem) % 16 || (ys[i] * elem) % 16) return false;
        if (x == y && xs[i] != ys[i]) return false;
    }
    return true;
}

}  // namespace

}  // namespace kvevict

using namespace kvevict;

extern "C" int kvevict_rotary(const kvevict_rotary_args *a, void *cuda_stream)
{
    if (!a) return KVEVICT_ERR_INVALID_ARG;
    if (a->dtype != KVEVICT_F32 && a->dtype != KVEVICT_BF16) return KVEVICT_ERR_INVALID_ARG;
    const int elem = a->dtype == KVEVICT_F32 ? 4 : 2;
    if (a->head_dim < 8 || a->head_dim > 1024 || a->head_dim % 8 || a->rotary_dim < 2 || a->rotary_dim > a->head_dim ||
        a->rotary_dim % 2)
        return KVEVICT_ERR_INVALID_ARG;
    if ((a->interleaved | a->inverse | a->positions_64) & ~1) return KVEVICT_ERR_INVALID_ARG;
    if (a->batch < 0 || a->tokens < 0 || a->n_q_heads < 0 || a->n_k_heads < 0 || a->n_q_heads > 65535 || a->n_k_heads > 65535)
        return KVEVICT_ERR_INVALID_ARG;
    if (!std::isfinite(a->scale) || !a->inv_freq || (reinterpret_cast<uintptr_t>(a->inv_freq) & 7))
        return KVEVICT_ERR_INVALID_ARG;
    if (a->batch >= (1LL << 31) || a->tokens >= (1LL << 31) || a->batch * a->tokens >= (1LL << 31))
        return KVEVICT_ERR_INVALID_ARG;
    const bool has_q = a->n_q_heads > 0, has_k = a->k != nullptr && a->n_k_heads > 0;
    const long long total = a->batch * a->tokens;
    if (total == 0 || (!has_q && !has_k)) return KVEVICT_OK;
    if (has_q && !rot_tensor_ok(a->q, a->q_out, a->q_stride, a->q_out_stride, elem)) return KVEVICT_ERR_INVALID_ARG;
    if (has_k && !rot_tensor_ok(a->k, a->k_out, a->k_stride, a->k_out_stride, elem)) return KVEVICT_ERR_INVALID_ARG;
    if (a->positions && (reinterpret_cast<uintptr_t>(a->positions) & (a->positions_64 ? 7 : 3))) return KVEVICT_ERR_INVALID_ARG;
    RotParams p{};
    p.x[0] = a->q; p.y[0] = a->q_out;
    p.x[1] = a->k; p.y[1] = a->k_out;
    for (int i = 0; i < 3; ++i) {
        p.xs[0][i] = a->q_stride[i]; p.ys[0][i] = a->q_out_stride[i];
        p.xs[1][i] = a->k_stride[i]; p.ys[1][i] = a->k_out_stride[i];
    }
    p.heads[0] = has_q ? a->n_q_heads : 0;
    p.heads[1] = has_k ? a->n_k_heads : 0;
    p.pos = a->positions;
    p.pos64 = a->positions_64;
    p.ps0 = a->pos_stride[0];
    p.ps1 = a->pos_stride[1];
    p.pos_start = a->pos_start;
    p.freq = a->inv_freq;
    p.scale = a->scale;
    p.D = a->head_dim;
    p.R = a->rotary_dim;
    p.interleaved = a->interleaved;
    p.inverse = a->inverse;
    p.tokens = a->tokens;
    p.total = total;
    const size_t smem = static_cast<size_t>(p.R / 2) * sizeof(float2);
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if (elem == 4) rotary_kernel<float><<<static_cast<unsigned>(total), kRotThreads, smem, st>>>(p);
    else rotary_kernel<__nv_bfloat16><<<static_cast<unsigned>(total), kRotThreads, smem, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? KVEVICT_OK : KVEVICT_ERR_CUDA;
}
