// paged_common.cuh -- what the kernels on a paged cache share: its parameters,
// the new tokens of a sequence as read (and clamped) from the device, the place of
// a token in the pages, and the groups of 4-bit pages.
#pragma once

#include <climits>

#include "device_common.cuh"
#include "kvevict_paged.h"

namespace kvevict {

struct PagedCache {
    char *pages[2];                                             // keys, values
    long long page_bytes[2], head_bytes[2], token_bytes[2];     // strides (4 bits: no token stride)
    const int32_t *table, *kv_lens;
    long long table_stride;
    uint32_t *err;
    int Hkv, S, log2_s, batch, width, n_pages;
};

__host__ __device__ __forceinline__ int paged_min(int a, int b) { return a < b ? a : b; }
__host__ __device__ __forceinline__ int paged_max(int a, int b) { return a > b ? a : b; }

// The rows of new tokens that a sequence owns: `n` of them from row q0 on, the
// first ones of `given`. Starts out of range are clamped, so that every row lies in
// the tensor; the rows of sequences whose starts ascend are disjoint.
struct PagedRows {
    int q0, n, given;
    bool bad;
};

__host__ __device__ __forceinline__ PagedRows paged_rows(const int32_t *starts, int b, int per, int rows)
{
    PagedRows r;
    if (!starts) {
        r.q0 = b * per;
        r.n = r.given = per;
        r.bad = false;
        return r;
    }
    const int a0 = starts[b], a1 = starts[b + 1];
    r.q0 = paged_min(paged_max(a0, 0), rows);
    r.given = paged_max(a1, r.q0) - r.q0;
    r.n = paged_min(r.given, rows - r.q0);
    r.bad = r.q0 != a0 || r.q0 + r.n != a1;
    return r;
}

// The page of token i (>= 0) of sequence b, or -1 where the table names none.
__device__ __forceinline__ int paged_page(const PagedCache &c, int b, long long i)
{
    const int page = c.table[b * c.table_stride + (i >> c.log2_s)];
    return page >= 0 && page < c.n_pages ? page : -1;
}

// A whole block of threads, NT of them, finds the sequences of the rows row0 ..
// row0 + count - 1 of packed tokens: seq[i] is the one that owns row0 + i, or -1.
// From the first sequence that ends before it starts, the batch is left out (its
// rows could be an earlier one's). `bits`: set where starts are out of order or
// range. Uses *fall (shared); ends with a barrier.
template <int NT>
__device__ __forceinline__ void paged_owners(const int32_t *starts, int batch, int rows, int row0, int count, int *seq, int *fall,
                                             uint32_t &bits)
{
    for (int i = threadIdx.x; i < count; i += NT) seq[i] = -1;
    if (threadIdx.x == 0) *fall = INT_MAX;
    __syncthreads();
    for (int j0 = 0; j0 < batch; j0 += NT) {
        const int j = j0 + static_cast<int>(threadIdx.x);
        if (j < batch && starts[j] > starts[j + 1]) atomicMin(fall, j);
        __syncthreads();
        const int first = *fall;
        if (j < batch && j < first) {
            const PagedRows r = paged_rows(starts, j, 0, rows);
            if (r.bad) bits |= KVEVICT_DEV_BAD_LENGTH;
            const int hi = paged_min(r.q0 + r.n, row0 + count);
            for (int t = paged_max(r.q0, row0); t < hi; ++t) seq[t - row0] = j;
        }
        __syncthreads();
        if (first != INT_MAX) {
            bits |= KVEVICT_DEV_BAD_LENGTH;
            break;
        }
    }
}

// ------------------------------------------------------------- 4-bit groups
// d / by from the reciprocal, put right once: exact wherever the quotient is an fp32
// value. Channels of bf16 keys and steps in bf16 make codes that lie just between two
// (k + 1/2) and steps that need no rounding common, so that those have to be.
__device__ __forceinline__ float q4_divide(float d, float by, float inverse)
{
    const float q = d * inverse;
    return fmaf(fmaf(-q, by, d), inverse, q);
}

// A group's base and step for values between lo and hi.
__device__ __forceinline__ void q4_group(float lo, float hi, bool finite, uint32_t &base_step, float &base, float &step)
{
    // (8 hi + 7 lo) / 15, by sixteenths so that it cannot overflow
    base = __bfloat162float(__float2bfloat16_rn(q4_divide(fmaf(hi, 0.5f, lo * 0.4375f), 0.9375f, 1.f / 0.9375f)));
    // (by eighths, as base - lo can pass the largest fp32 value)
    step = fmaxf(q4_divide(hi - base, 7.f, 1.f / 7.f), base * 0.125f - lo * 0.125f);
    step = __uint_as_float((__float_as_uint(step) + 0xFFFFu) & 0xFFFF0000u);  // (>= 0: up)
    if (!finite) {
        base = __uint_as_float(0x7FC00000u);
        step = 0.f;
    }
    base_step = (__float_as_uint(base) >> 16) | (__float_as_uint(step) & 0xFFFF0000u);
}

// Values of a group for q4_code: those of a step of 2^100 and more are scaled by 2^-64, so that no difference to the base
// overflows, those of a step below 2^-64 by 2^64, so that the step has a reciprocal and a quotient's remainder its bits
// (they are no larger than 2^-35: a difference to the base below 2^-61 needs such neighbours). Nothing but the codes
// may be taken from them then.
template <int N> __device__ __forceinline__ void q4_in_range(float (&v)[N], float &base, float &step)
{
    if ((step >= 5.4210109e-20f && step < 1.2676506e30f) || step == 0.f) return;
    const float by = step < 1.f ? 1.8446744e19f : 5.4210109e-20f;
    base *= by;
    step *= by;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= by;
}

// 1 / step, 0 for none.
__device__ __forceinline__ float q4_inverse(float step) { return step > 0.f ? __fdividef(1.f, step) : 0.f; }

// A code in the low bits of 2^23 + 2^22 + code, where fp32's step is 1: the sum rounds
// (k + 1/2 to the even code).
__device__ __forceinline__ uint32_t q4_code(float x, float base, float step, float inverse)
{
    const float least = 12582912.f;
    return __float_as_uint(fminf(fmaxf(q4_divide(x - base, step, inverse) + (least + 8.f), least), least + 15.f));
}
// Four of them side by side, in the low 16 bits.
__device__ __forceinline__ uint16_t q4_codes(const float *v, float base, float step, float inverse)
{
    return static_cast<uint16_t>(q4_code(v[0], base, step, inverse) + q4_code(v[1], base, step, inverse) * 16u +
                                 q4_code(v[2], base, step, inverse) * 256u + q4_code(v[3], base, step, inverse) * 4096u);
}

__device__ __forceinline__ float q4_base(uint32_t base_step) { return __uint_as_float(base_step << 16); }
__device__ __forceinline__ float q4_step(uint32_t base_step) { return __uint_as_float(base_step & 0xFFFF0000u); }

}  // namespace kvevict
