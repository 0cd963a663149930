// rotary_common.cuh -- what the kernels with rotary positions share: their
// parameters, 16-byte vectors as fp32 values, the cosine and sine of a
// (frequency, position), and the host's checks.
#pragma once

#include <cstdint>

#include "device_common.cuh"
#include "kvevict_ops.h"

namespace kvevict {

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
    uint32_t tokens_per, heads_per, head_blocks;  // rotary_kernel: a CTA's share
};

// 16-byte vectors of T as fp32 values.
template <typename T> struct Vec {
    static constexpr int N = 16 / sizeof(T);
};

__device__ __forceinline__ void unpack16(const uint4 &w, float (&v)[4])
{
    v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y); v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack16(const uint4 &w, float (&v)[8])
{
    bf16x2_to_f32(w.x, v[0], v[1]);
    bf16x2_to_f32(w.y, v[2], v[3]);
    bf16x2_to_f32(w.z, v[4], v[5]);
    bf16x2_to_f32(w.w, v[6], v[7]);
}
__device__ __forceinline__ uint4 pack16(const float (&v)[4])
{
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack16(const float (&v)[8])
{
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// (The angle as a 64-bit binary fraction of a turn: see rotary.cu.)
__device__ __forceinline__ float2 rot_cos_sin(double freq, long long pos, float scale, bool inverse)
{
    // whole turns a position drop out; half a turn at most is left, and fits a signed 64-bit integer
    const double turns = freq * 0.15915494309189535;
    const long long f = __double2ll_rn((turns - rint(turns)) * 18446744073709551616.0);
    const long long frac = static_cast<long long>(static_cast<unsigned long long>(pos) * static_cast<unsigned long long>(f));
    const float half_turns = static_cast<float>(frac) * 1.0842021724855044e-19f;  // 2^-63
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * scale, inverse ? -s * scale : s * scale);
}

// The same in two parts: a frequency's turns a position as a fraction, once for many
// tokens (fp64 instructions are scarce: 16 cycles of an SM for a warp's), and a
// position's cosine and sine from it.
__device__ __forceinline__ long long rot_turns(double freq)
{
    const double turns = freq * 0.15915494309189535;
    return __double2ll_rn((turns - rint(turns)) * 18446744073709551616.0);
}
__device__ __forceinline__ float2 rot_cos_sin(long long turns, long long pos, float scale)
{
    const long long frac = static_cast<long long>(static_cast<unsigned long long>(pos) * static_cast<unsigned long long>(turns));
    float s, c;
    sincospif(static_cast<float>(frac) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    return make_float2(c * scale, s * scale);
}

// Position of token t of sequence b.
__device__ __forceinline__ long long rot_position(const RotParams &p, long long b, long long t)
{
    const long long at = b * p.ps0 + t * p.ps1;
    return !p.pos ? p.pos_start + t
                  : (p.pos64 ? static_cast<const long long *>(p.pos)[at]
                             : static_cast<long long>(static_cast<const int *>(p.pos)[at]));
}

// A thread's way through the (token, head) rows of a CTA, `step` rows at a time: a
// pointer that follows the strides.
struct Walk {
    char *p;
    int h, t, ts;  // head, token of the CTA, token of its sequence
    int nh, tokens, heads_on, tokens_on;           // a step: so many heads and whole tokens on
    long long by_step, by_token, by_seq;           // bytes: a step; from behind the last head to the next token; over a sequence's end

    __device__ __forceinline__ void start(char *base, const long long (&s)[3], int elem, long long b, int token, int heads, int step, int first, int per)
    {
        nh = heads;
        tokens = per;
        heads_on = step % nh;
        tokens_on = step / nh;
        by_token = (s[2] - nh * s[1]) * elem;
        by_step = (heads_on * s[1] + tokens_on * s[2]) * elem;
        by_seq = static_cast<long long>(static_cast<unsigned long long>(s[0]) - static_cast<unsigned long long>(tokens) * s[2]) * elem;
        h = first % nh;
        t = first / nh;
        ts = token + t;
        p = base + (b * s[0] + ts * s[2] + h * s[1]) * elem;
        ends();
    }
    __device__ __forceinline__ void ends()
    {
        if (ts >= tokens) {
            const int n = ts / tokens;
            ts -= n * tokens;
            p += n * by_seq;
        }
    }
    __device__ __forceinline__ void on()
    {
        int dt = tokens_on;
        h += heads_on;
        p += by_step;
        if (h >= nh) {
            h -= nh;
            p += by_token;
            ++dt;
        }
        t += dt;
        ts += dt;
        ends();
    }
};

constexpr int kRotThreads = 256;

// A CTA's share of tokens and heads (rotary.cu has the figures): its units,
// `units` a head, are ten for each of its threads, or, where that would leave SMs
// idle, what gives every SM two CTAs, but a unit for every second thread at least.
// Returns the number of CTAs.
long long rot_shares(RotParams &p, uint32_t units);

// kvevict_rotary's checks (norm: kvevict_norm_rotary's, rotary_dim may be 0 and
// there is no inverse), and its parameters. `nothing`: no token or head.
int rot_prepare(const kvevict_rotary_args *a, bool norm, RotParams &p, bool &nothing);

}  // namespace kvevict
