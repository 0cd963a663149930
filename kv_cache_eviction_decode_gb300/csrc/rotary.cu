// rotary.cu -- kvevict_rotary: rotary positions for queries and keys, in one
// launch.
//
// Bound by bytes: x is read once and written once. The angle of (token, pair)
// is the same for every head, so a CTA takes one token, forms its cosines and
// sines once in shared memory and applies them to all heads of q and k. The
// angle itself is formed in turns as a 64-bit binary fraction: with F =
// round(inv_freq / 2 pi * 2^64), pos * F mod 2^64 is the angle modulo one turn
// but for F's error -- an integer multiply does the range reduction, for any
// position, where an fp32 product would have lost the fraction past a few
// thousand turns. F's error is that of the fp64 product inv_freq * (1 / 2 pi),
// 1.6 * 2^-53 of it at most, and that of its last bit, 2^-64 at most.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "device_common.cuh"
#include "kvevict_ops.h"
#include "launch.h"
#include "rotary_common.cuh"

namespace kvevict {

namespace {

// Rotary parts whose pairs do not fall into 16-byte chunks (half layout:
// rotary_dim / 2, interleaved: rotary_dim no multiple of a chunk). One CTA per
// token. A thread takes 16-byte chunks of the output; an element of the rotary
// part reads its partner element by itself (from L1: another thread of the warp
// reads the same line). In place, all reads of a pass come before its writes.
template <typename T>
__global__ void __launch_bounds__(kRotThreads) rotary_any_kernel(const __grid_constant__ RotParams p)
{
    constexpr int N = Vec<T>::N;
    extern __shared__ __align__(16) float2 cs[];  // [R / 2] cos, sin
    grid_dependency_wait();
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
                unpack16(*reinterpret_cast<const uint4 *>(xr + c), v);
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
            if (mine) *reinterpret_cast<uint4 *>(y + h * p.ys[w][1] + c) = pack16(v);
        }
    }
}

// Rotary parts in whole 16-byte chunks. The work is units of one thread: a pair
// of chunks rotary_dim / 2 apart (half layout), a chunk of neighbouring pairs
// (interleaved), or a chunk that is only copied; a unit reads all that it writes
// over, so that in place needs no care. A CTA takes `tokens_per` tokens x
// `heads_per` heads of q and k together; a thread has 64 bytes of loads in
// flight (two units of two chunks, four of one), the first ones while the CTA
// forms its cosines and sines. With 128 bytes a thread fewer CTAs fit an SM, and
// prompts of 16384 tokens, 64 + 8 heads of 128, took 133 us instead of 105 (85% of
// the copy bandwidth); with CTAs of 576 units instead of about 2300, which share a
// token's cosines among fewer rows, 110.

template <typename T, bool INTER>
__global__ void __launch_bounds__(kRotThreads, 4) rotary_kernel(const __grid_constant__ RotParams p)
{
    constexpr int N = Vec<T>::N, kBatch = INTER ? 4 : 2;
    extern __shared__ __align__(16) float2 cs[];  // [tokens_per][R / 2] cos, sin
    grid_dependency_wait();
    const uint32_t half = p.R / 2;
    const uint32_t pairs = INTER ? 0 : half / N;                       // units of two chunks a head
    const uint32_t units = INTER ? p.D / N : pairs + (p.D - p.R) / N;  // units a head
    const uint32_t tok0 = blockIdx.x / p.head_blocks * p.tokens_per;
    const uint32_t nt = min(p.tokens_per, static_cast<uint32_t>(p.total) - tok0);
    const uint32_t h0 = blockIdx.x % p.head_blocks * p.heads_per;
    const uint32_t nh = min(p.heads_per, static_cast<uint32_t>(p.heads[0] + p.heads[1]) - h0);
    // a thread's chunk within the head stays; it walks the CTA's (token, head) rows
    const uint32_t step = kRotThreads / units, u = threadIdx.x % units;
    const bool two = !INTER && u < pairs;
    const uint32_t c = INTER || u < pairs ? u * N : p.R + (u - pairs) * N;
    uint32_t h = threadIdx.x / units, lt = threadIdx.x < step * units ? 0 : nt;  // head, token of the CTA
    long long xq = 0, xk = 0, yq = 0, yk = 0;                                    // where the token starts
    auto settle = [&]() {
        while (h >= nh && lt < nt) {
            h -= nh;
            ++lt;
        }
    };
    auto token = [&]() {
        const uint32_t bt = tok0 + lt, b = bt / static_cast<uint32_t>(p.tokens), t = bt - b * static_cast<uint32_t>(p.tokens);
        xq = b * p.xs[0][0] + t * p.xs[0][2];
        xk = b * p.xs[1][0] + t * p.xs[1][2];
        yq = b * p.ys[0][0] + t * p.ys[0][2];
        yk = b * p.ys[1][0] + t * p.ys[1][2];
    };
    settle();
    if (lt < nt) token();
    bool ready = false;
    for (bool more = true; more;) {
        uint4 a[kBatch], b[kBatch];
        T *y[kBatch];
        uint32_t tk[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            y[i] = nullptr;
            tk[i] = lt;
            if (lt >= nt) continue;
            const uint32_t hh = h0 + h;
            const bool k = hh >= static_cast<uint32_t>(p.heads[0]);
            const uint32_t hl = k ? hh - p.heads[0] : hh;
            const T *x = static_cast<const T *>(p.x[k]) + (k ? xk : xq) + hl * p.xs[k][1] + c;
            y[i] = static_cast<T *>(p.y[k]) + (k ? yk : yq) + hl * p.ys[k][1] + c;
            a[i] = *reinterpret_cast<const uint4 *>(x);
            if (two) b[i] = *reinterpret_cast<const uint4 *>(x + half);
            const uint32_t was = lt;
            h += step;
            settle();
            if (lt != was && lt < nt) token();
        }
        if (!ready) {
            for (uint32_t i = threadIdx.x; i < nt * half; i += kRotThreads) {
                const uint32_t t0 = i / half, bt = tok0 + t0, bb = bt / static_cast<uint32_t>(p.tokens);
                const long long t = bt - bb * static_cast<uint32_t>(p.tokens), at = bb * p.ps0 + t * p.ps1;
                const long long pos = !p.pos ? p.pos_start + t
                                             : (p.pos64 ? static_cast<const long long *>(p.pos)[at]
                                                        : static_cast<long long>(static_cast<const int *>(p.pos)[at]));
                cs[i] = rot_cos_sin(p.freq[i - t0 * half], pos, p.scale, p.inverse);
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (!y[i]) continue;
            const float2 *k = cs + tk[i] * half + (INTER ? c / 2 : c);
            float v[N];
            if (INTER) {
                if (c < static_cast<uint32_t>(p.R)) {
                    unpack16(a[i], v);
#pragma unroll
                    for (int j = 0; j < N; j += 2) {
                        const float x = v[j], w = v[j + 1];
                        v[j] = x * k[j / 2].x - w * k[j / 2].y;
                        v[j + 1] = x * k[j / 2].y + w * k[j / 2].x;
                    }
                    a[i] = pack16(v);
                }
            } else if (two) {
                float z[N];
                unpack16(a[i], v);
                unpack16(b[i], z);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float x = v[j], w = z[j];
                    v[j] = x * k[j].x - w * k[j].y;
                    z[j] = x * k[j].y + w * k[j].x;
                }
                a[i] = pack16(v);
                *reinterpret_cast<uint4 *>(y[i] + half) = pack16(z);
            }
            *reinterpret_cast<uint4 *>(y[i]) = a[i];
        }
        more = lt < nt;
    }
}

// The stride of an axis of one entry is not looked at. Over any other the
// output's must not be 0: its entries would share a row.
bool rot_tensor_ok(const void *x, const void *y, const int64_t (&xs)[3], const int64_t (&ys)[3], const int64_t (&sizes)[3], int elem)
{
    if (!x || !y || (reinterpret_cast<uintptr_t>(x) & 15) || (reinterpret_cast<uintptr_t>(y) & 15)) return false;
    for (int i = 0; i < 3; ++i) {
        if (sizes[i] <= 1) continue;
        if (ys[i] == 0) return false;
        if ((xs[i] * elem) % 16 || (ys[i] * elem) % 16) return false;
        if (x == y && xs[i] != ys[i]) return false;
    }
    return true;
}

}  // namespace

long long rot_shares(RotParams &p, uint32_t units)
{
    const uint32_t heads = static_cast<uint32_t>(p.heads[0] + p.heads[1]);
    const long long all = p.total * heads * units;
    const long long want = std::min<long long>(10 * kRotThreads, std::max<long long>(kRotThreads / 2, all / 304));
    p.heads_per = static_cast<uint32_t>(std::min<long long>(heads, std::max<long long>(1, want / units)));
    p.head_blocks = (heads + p.heads_per - 1) / p.heads_per;
    p.tokens_per = 1;
    if (p.head_blocks == 1)
        p.tokens_per = static_cast<uint32_t>(std::max<long long>(1, std::min<long long>(want / (heads * units), 8192 / std::max(p.R, 2))));
    return (p.total + p.tokens_per - 1) / p.tokens_per * p.head_blocks;
}

int rot_prepare(const kvevict_rotary_args *a, bool norm, RotParams &p, bool &nothing)
{
    nothing = false;
    if (!a) return KVEVICT_ERR_INVALID_ARG;
    if (a->dtype != KVEVICT_F32 && a->dtype != KVEVICT_BF16) return KVEVICT_ERR_INVALID_ARG;
    const int elem = a->dtype == KVEVICT_F32 ? 4 : 2;
    const bool turns = !norm || a->rotary_dim != 0;
    if (a->head_dim < 8 || a->head_dim > 1024 || a->head_dim % 8 || a->rotary_dim < (norm ? 0 : 2) || a->rotary_dim > a->head_dim ||
        a->rotary_dim % 2)
        return KVEVICT_ERR_INVALID_ARG;
    if ((a->interleaved | a->inverse | a->positions_64) & ~1) return KVEVICT_ERR_INVALID_ARG;
    if (norm && a->inverse) return KVEVICT_ERR_INVALID_ARG;
    if (a->batch < 0 || a->tokens < 0 || a->n_q_heads < 0 || a->n_k_heads < 0 || a->n_q_heads > 65535 || a->n_k_heads > 65535)
        return KVEVICT_ERR_INVALID_ARG;
    if (!std::isfinite(a->scale) || (turns && !a->inv_freq) || (reinterpret_cast<uintptr_t>(a->inv_freq) & 7))
        return KVEVICT_ERR_INVALID_ARG;
    if (a->batch >= (1LL << 31) || a->tokens >= (1LL << 31) || a->batch * a->tokens >= (1LL << 31))
        return KVEVICT_ERR_INVALID_ARG;
    const bool has_q = a->n_q_heads > 0, has_k = a->k != nullptr && a->n_k_heads > 0;
    const long long total = a->batch * a->tokens;
    if (total == 0 || (!has_q && !has_k)) {
        nothing = true;
        return KVEVICT_OK;
    }
    const int64_t qn[3] = {a->batch, a->n_q_heads, a->tokens}, kn[3] = {a->batch, a->n_k_heads, a->tokens};
    if (has_q && !rot_tensor_ok(a->q, a->q_out, a->q_stride, a->q_out_stride, qn, elem)) return KVEVICT_ERR_INVALID_ARG;
    if (has_k && !rot_tensor_ok(a->k, a->k_out, a->k_stride, a->k_out_stride, kn, elem)) return KVEVICT_ERR_INVALID_ARG;
    if (a->positions && (reinterpret_cast<uintptr_t>(a->positions) & (a->positions_64 ? 7 : 3))) return KVEVICT_ERR_INVALID_ARG;
    p = RotParams{};
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
    return KVEVICT_OK;
}

}  // namespace kvevict

using namespace kvevict;

extern "C" int kvevict_rotary(const kvevict_rotary_args *a, void *cuda_stream)
{
    RotParams p;
    bool nothing;
    const int rc = rot_prepare(a, false, p, nothing);
    if (rc != KVEVICT_OK || nothing) return rc;
    const int elem = a->dtype == KVEVICT_F32 ? 4 : 2;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const int n = 16 / elem;  // elements of a chunk
    cudaError_t e;
    if (a->interleaved ? p.R % n == 0 : p.R / 2 % n == 0) {
        const uint32_t units = static_cast<uint32_t>(a->interleaved ? p.D / n : p.R / 2 / n + (p.D - p.R) / n);
        const long long blocks = rot_shares(p, units);
        if (blocks >= (1LL << 31)) return KVEVICT_ERR_INVALID_ARG;
        const unsigned g = static_cast<unsigned>(blocks);
        const size_t smem = static_cast<size_t>(p.tokens_per) * (p.R / 2) * sizeof(float2);
        if (a->interleaved) {
            if (elem == 4) e = launch_dependent(rotary_kernel<float, true>, g, kRotThreads, smem, st, p);
            else e = launch_dependent(rotary_kernel<__nv_bfloat16, true>, g, kRotThreads, smem, st, p);
        } else {
            if (elem == 4) e = launch_dependent(rotary_kernel<float, false>, g, kRotThreads, smem, st, p);
            else e = launch_dependent(rotary_kernel<__nv_bfloat16, false>, g, kRotThreads, smem, st, p);
        }
    } else {
        const size_t smem = static_cast<size_t>(p.R / 2) * sizeof(float2);
        if (elem == 4) e = launch_dependent(rotary_any_kernel<float>, static_cast<unsigned>(p.total), kRotThreads, smem, st, p);
        else e = launch_dependent(rotary_any_kernel<__nv_bfloat16>, static_cast<unsigned>(p.total), kRotThreads, smem, st, p);
    }
    return e == cudaSuccess ? KVEVICT_OK : KVEVICT_ERR_CUDA;
}
