// paged_attn_mma.cu -- attention of a few bf16 queries over a paged cache, bf16 or
// 4 bits, on the tensor cores.
//
// A few rows over many keys are bound by the keys' bytes, so a warp works by
// itself: it walks tiles of 16 keys through a ring of its own in shared memory
// (cp.async), keeps its own softmax, and only at the end are a CTA's warps joined.
// The products are transposed, S^T = K Q^T and O^T = V^T P^T, with keys and then
// channels on the 16-wide axis of mma.m16n8k16 and query rows on the 8-wide one:
// eight query heads of a KV head fill an instruction. (tcgen05 would want 64 or 128
// rows.) P^T comes from S^T by transposing 8 x 8 blocks in registers (movmatrix).
//
// 4 bits: a code needs a mask and nothing else to be a matrix operand. bf16's bit
// patterns 0 .. 255 are the values 0 .. 255 times 2^-133 (its subnormals and, with
// the same spacing, the first normal numbers), so c and 16 c are read off as they
// lie in a half word, two bits of work a channel. Queries are scaled by a power of
// two to at most 2^101, a sixteenth of it for every second channel, and
//   S_ij = sum_groups step (sum_c c q) + (base - 8 step) (sum q),
// the sums over a group in fp32. In the second product the step goes into the
// probabilities, which are then rounded to bf16, once, and scaled by a power of two
// that follows the largest step seen:
//   O_i = sum_j (p_ij step_j) (c_j - 8) + sum_j p_ij base_j,
// the 8 taken off by an instruction with constant codes, the base's part in fp32.
//
// The running maximum is moved only where a logit exceeds it by 2^8 or more: then,
// and only then, sums and outputs are rescaled. Probabilities below 2^8 instead of
// below 1 cost no precision.
#include <cfloat>
#include <cmath>

#include "launch.h"
#include "paged_attn.h"

namespace kvevict {

namespace {

constexpr int kWarps = kPagedMmaWarps;
constexpr float kLn2 = 0.69314718055994531f;
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kSlack = 8.f;  // powers of two that a logit may exceed the maximum by

template <int D, bool Q4> struct Ring {
    static constexpr int kRow = Q4 ? D / 2 : D * 2;                            // bytes of a key, codes only
    static constexpr int kParams = Q4 ? D / 8 : 0;                             // and its groups
    static constexpr int kStage = 2 * kPagedTile * (kRow + kParams);           // K codes, V codes, K groups, V groups
    static constexpr int kStages = Q4 ? (D == 128 ? 6 : 8) : (D == 128 ? 3 : 6);
    static constexpr int kWarpBytes = kStage * kStages;
};

template <int D, bool Q4, int NT> constexpr int smem_bytes()
{
    constexpr int ring = Ring<D, Q4>::kWarpBytes * kWarps, join = kWarps * 8 * NT * (D + 4 + 2) * 4;
    return ring > join ? ring : join;
}

__device__ __forceinline__ void copy16(uint32_t dst, const char *src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// D = A B + C with C = 0.
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_next(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    const uint32_t a[4] = {a0, a1, a2, a3};
    mma_bf16_16816(d, a, b0, b1);
}

// 2^x, off by two steps at most; 0 below 2^-126.
__device__ __forceinline__ float pow2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Codes of two keys or channels, one in each half word, as bf16: c 2^-133, and
// from the next nibble 16 c 2^-133.
__device__ __forceinline__ uint32_t code(uint32_t x) { return x & 0x000F000Fu; }
__device__ __forceinline__ uint32_t code16(uint32_t x) { return x & 0x00F000F0u; }
constexpr uint32_t kMinus8 = 0x80088008u, kMinus8x16 = 0x80808080u;  // -8 as such a code

__device__ __forceinline__ float exponent_of(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // 2^e

constexpr int kMinE = -40;  // of the steps' power of two; the probabilities' is 2^(kProbE - E)
constexpr int kProbE = 80;
constexpr int kCodeE = -133;

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// W words of shared memory.
template <int W> __device__ __forceinline__ void lds(uint32_t (&v)[W], uint32_t a)
{
    if constexpr (W == 4) {
        const uint4 x = lds128(a);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else if constexpr (W == 2) {
        const uint2 x = lds64(a);
        v[0] = x.x; v[1] = x.y;
    } else {
        v[0] = lds32(a);
    }
}

// Row r (0 .. 7) of an 8 x 8 block of S^T is this key of a 4-bit tile's half, so
// that after the transpose a lane's keys lie four apart: t and 4 + t. Its loads of
// V, one row of codes a key, then take neighbouring rows side by side.
__device__ __forceinline__ int key_of(int r) { return (r & 1) * 4 + (r >> 1); }

template <int D, bool Q4, int NT>
__global__ void __launch_bounds__(kWarps * 32, (NT == 1 ? 3 : 2)) paged_mma_kernel(const __grid_constant__ PagedAttnParams p)
{
    using L = Ring<D, Q4>;
    constexpr int R = 8 * NT, kGroups = D / 32, kSteps = D / 16;  // rows; groups; 16-channel steps, or tiles of O^T
    extern __shared__ __align__(16) char ring[];
    grid_dependency_wait();
    const PagedCache &c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    int item = blockIdx.x;
    const int tile = item % p.q_tiles;
    item /= p.q_tiles;
    const int part = item % p.splits, unit = item / p.splits;
    const int b = unit / c.Hkv, kvh = unit - b * c.Hkv;
    const PagedSeq sq = paged_sequence(p, b, !p.mask.q_starts || attn_first_fall(p.mask, b, lane) == INT_MAX);
    if (sq.bad && threadIdx.x == 0) atomicOr(c.err, KVEVICT_DEV_BAD_LENGTH);
    const int r0 = tile * R, nr = min(R, sq.n * p.G - r0);
    if (nr <= 0) return;
    const int pa = sq.p0 + r0 / p.G, pb = sq.p0 + (r0 + nr - 1) / p.G;  // the rows' positions
    const AttnKeys keys = attn_keys(p.mask, sq.m, pa, pb, kPagedTile);
    const int i_lo = static_cast<int>(static_cast<long long>(keys.count) * part / p.splits);
    const int i_hi = static_cast<int>(static_cast<long long>(keys.count) * (part + 1) / p.splits);
    const int n_mine = max(0, (i_hi - i_lo - warp + kWarps - 1) / kWarps);  // tiles i_lo + warp + kWarps k
    const int low_b = p.mask.window > 0 && pb >= p.mask.window ? pb - p.mask.window + 1 : 0;

    // pages of the next 32 of this warp's tiles, one a lane; the 32 after them are on their way
    auto pages_from = [&](int k0) {
        const int k = k0 + lane;
        return k < n_mine ? paged_page(c, b, static_cast<long long>(attn_tile_at(keys, i_lo + warp + kWarps * k)) * kPagedTile) : -1;
    };
    int pages = pages_from(0), pages_next = -1;

    // ------------------------------------------------------------ copies into the ring
    const uint32_t my_ring = smem_u32(ring) + warp * L::kWarpBytes;
    const char *const kbase = c.pages[0] + kvh * c.head_bytes[0], *const vbase = c.pages[1] + kvh * c.head_bytes[1];
    // 4 bits: what a lane copies. K's rows go in by eights in key_of's order; V's as they are, with the 16-byte chunks of
    // every second pair of rows swapped (D = 128), so that four rows' parts lie in different banks.
    constexpr int kPc = L::kParams;  // 16-byte chunks of a tile's groups, of K and of V
    const int cr = lane / (L::kRow / 16), cch = lane % (L::kRow / 16);
    const int k_from = ((cr & 8) + key_of(cr & 7)) * L::kRow + cch * 16, v_from = cr * L::kRow + (D == 128 ? cch ^ (cr & 2) : cch) * 16;
    const int p_from = Q4 ? c.S * L::kRow + lane % max(kPc, 1) * 16 : 0;
    uint32_t bad = 0;  // bit s: stage s holds a tile without a page
    int next = 0;      // the stage that the next copies go to
    auto issue = [&](int k) {
        if (k < n_mine) {
            if (k && (k & 31) == 0) pages = pages_next;
            if ((k & 31) == 0) pages_next = pages_from(k + 32);
            const int page = __shfl_sync(kAll, pages, k & 31);
            const int s = next, j0 = attn_tile_at(keys, i_lo + warp + kWarps * k) * kPagedTile, slot0 = j0 & (c.S - 1);
            const uint32_t dst = my_ring + s * L::kStage;
            bad = page < 0 ? bad | 1u << s : bad & ~(1u << s);
            if (page < 0) {
                if (lane == 0) atomicOr(c.err, KVEVICT_DEV_BAD_PAGE);
            }
            const char *kp = kbase + max(page, 0) * c.page_bytes[0], *vp = vbase + max(page, 0) * c.page_bytes[1];
            if constexpr (Q4) {
                if (page >= 0) {
                    const char *kc = kp + slot0 * L::kRow + k_from, *vc = vp + slot0 * L::kRow + v_from;
                    const char *pc = (lane < kPc ? kp : vp) + slot0 * L::kParams + p_from;
                    const uint32_t to = dst + lane * 16;
#pragma unroll
                    for (int e0 = 0; e0 < kPagedTile * L::kRow; e0 += 512) {
                        copy16(to + e0, kc + e0, true);
                        copy16(to + kPagedTile * L::kRow + e0, vc + e0, true);
                    }
                    if (lane < 2 * kPc) copy16(to + 2 * kPagedTile * L::kRow, pc, true);
                }
            } else {
                // 16-byte chunks swapped by row, so that the eight rows of a matrix load lie in different banks
                constexpr int kChunks = L::kRow / 16;
#pragma unroll
                for (int e0 = 0; e0 < kPagedTile * kChunks; e0 += 32) {
                    const int e = e0 + lane, r = e / kChunks, ch = e % kChunks, j = j0 + r;
                    const bool real = page >= 0 && (j < keys.sink || (j >= keys.lo && j < keys.hi));
                    const uint32_t at = r * L::kRow + ((ch & ~7) | ((ch ^ r) & 7)) * 16;
                    copy16(dst + at, kp + (slot0 + r) * c.token_bytes[0] + ch * 16, real);
                    copy16(dst + kPagedTile * L::kRow + at, vp + (slot0 + r) * c.token_bytes[1] + ch * 16, real);
                }
            }
        }
        next = next + 1 == L::kStages ? 0 : next + 1;
        copies_close();
    };
#pragma unroll 1
    for (int k = 0; k < L::kStages - 1; ++k) issue(k);

    // ---------------------------------------------------------------- queries, row n = 8 a + g
    uint32_t qf[NT][kSteps][2];
    float qsum[NT][kGroups][2];  // 4 bits: of a group, rows 2 t and 2 t + 1, times 2^-133 like the products
    float sl2[NT][2];            // what turns those rows' products into logits to base 2
#pragma unroll
    for (int a = 0; a < NT; ++a) {
        const int r = 8 * a + g, tk = (r0 + r) / p.G, hd = r0 + r - tk * p.G;
        const __nv_bfloat16 *qr = static_cast<const __nv_bfloat16 *>(p.q) + (kvh * p.G + hd) * p.qs[0] + (sq.q0 + tk) * p.qs[1];
        sl2[a][0] = sl2[a][1] = p.scale_log2;
        if constexpr (Q4) {
            float x[kGroups][8], top = 0.f;
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                uint4 w = make_uint4(0, 0, 0, 0);
                if (r < nr) w = *reinterpret_cast<const uint4 *>(qr + 32 * j + 8 * t);
                bf16x2_to_f32(w.x, x[j][0], x[j][1]);
                bf16x2_to_f32(w.y, x[j][2], x[j][3]);
                bf16x2_to_f32(w.z, x[j][4], x[j][5]);
                bf16x2_to_f32(w.w, x[j][6], x[j][7]);
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[j][i]));
            }
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
            // the row times 2^(100 - e), 2^e the power of two of its largest element (far ones, where fp32 would end, left as they are)
            const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -20), 90);
            const float up = exponent_of(100 - e), back = p.scale_log2 * exponent_of(e - 100 - kCodeE);
            sl2[a][0] = __shfl_sync(kAll, back, 8 * t);
            sl2[a][1] = __shfl_sync(kAll, back, 8 * t + 4);
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[j][i] *= up;
                    sum += x[j][i] * exponent_of(-100);
                }
                // step 2 j + h: channels (2 h, 4 + 2 h) and, a sixteenth, (2 h + 1, 5 + 2 h) of the lane's eight
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    qf[a][2 * j + h][0] = pack_bf16x2(x[j][2 * h], x[j][4 + 2 * h]);
                    qf[a][2 * j + h][1] = pack_bf16x2(x[j][2 * h + 1] * 0.0625f, x[j][5 + 2 * h] * 0.0625f);
                }
                sum += __shfl_xor_sync(kAll, sum, 1);
                sum += __shfl_xor_sync(kAll, sum, 2);
                sum *= exponent_of(100 + kCodeE);
                qsum[a][j][0] = __shfl_sync(kAll, sum, 8 * t);
                qsum[a][j][1] = __shfl_sync(kAll, sum, 8 * t + 4);
            }
        } else {
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    qf[a][s][i] = r < nr ? *reinterpret_cast<const uint32_t *>(qr + 16 * s + 8 * i + 2 * t) : 0u;
        }
    }

    // nm: minus the running maximum (to base 2); over: the product above which it is moved
    float nm[NT][2], over[NT][2], l[NT][2], o[NT][kSteps][4], ob[NT][kGroups][2];  // ob: sum of p base (4 bits), this lane's keys
    int step_e = kMinE;                                                           // 4 bits: 2^e of the largest step seen,
    uint32_t step_over = 0;                                                       // and the group from which on it is moved
    float prob = exponent_of(kProbE - kMinE);
#pragma unroll
    for (int a = 0; a < NT; ++a) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            nm[a][i] = FLT_MAX;
            over[a][i] = -INFINITY;
            l[a][i] = 0.f;
#pragma unroll
            for (int j = 0; j < kGroups; ++j) ob[a][j][i] = 0.f;
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[a][s][i] = 0.f;
    }
    // this lane's keys of a tile: k0 and k0 + 8
    const int k0 = Q4 ? key_of(g) : g;
    const int kw_at = g * L::kRow + t * (D / 8), vw_at = kPagedTile * L::kRow + t * L::kRow + (D == 128 ? (g >> 1 ^ (t & 2)) * 16 + (g & 1) * 8 : g * 4);
    const int p_at = 2 * kPagedTile * L::kRow + k0 * L::kParams;

#pragma unroll 1
    for (int k = 0, s = 0; k < n_mine; ++k, s = s + 1 == L::kStages ? 0 : s + 1) {
        copies_wait<L::kStages - 2>();
        __syncwarp();
        issue(k + L::kStages - 1);
        const uint32_t at = my_ring + s * L::kStage;
        const int j0 = attn_tile_at(keys, i_lo + warp + kWarps * k) * kPagedTile;
        // every row sees every key of the tile
        const bool whole = j0 + kPagedTile - 1 <= min(pa, sq.m - 1) && (j0 + kPagedTile <= p.mask.n_sink || j0 >= low_b) && !(bad >> s & 1);

        // ---------------------------------------------------------- logits
        float z[NT][4];
        if constexpr (Q4) {
            constexpr int W = D / 32;  // words of codes: an eighth of a row twice
            uint32_t w0[W], w1[W], ps0[kGroups], ps1[kGroups];
            lds(w0, at + kw_at);
            lds(w1, at + kw_at + 8 * L::kRow);
            lds(ps0, at + p_at);
            lds(ps1, at + p_at + 8 * L::kParams);
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                // half word j of both eighths: channels 8 t + i below, 8 t + 4 + i above
                const uint32_t sel = j % 2 ? 0x7632 : 0x5410;
                const uint32_t x0 = __byte_perm(w0[j / 2], w0[W / 2 + j / 2], sel), x1 = __byte_perm(w1[j / 2], w1[W / 2 + j / 2], sel);
                const uint32_t y0 = x0 >> 8, y1 = x1 >> 8;
                const float st0 = q4_step(ps0[j]), st1 = q4_step(ps1[j]);
                const float ba0 = fmaf(-8.f, st0, q4_base(ps0[j])), ba1 = fmaf(-8.f, st1, q4_base(ps1[j]));
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    float d[4];
                    mma_first(d, code(x0), code(x1), code16(x0), code16(x1), qf[a][2 * j][0], qf[a][2 * j][1]);
                    mma_next(d, code(y0), code(y1), code16(y0), code16(y1), qf[a][2 * j + 1][0], qf[a][2 * j + 1][1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float base = i < 2 ? ba0 : ba1;
                        z[a][i] = fmaf(i < 2 ? st0 : st1, d[i], j ? fmaf(base, qsum[a][j][i & 1], z[a][i]) : base * qsum[a][j][i & 1]);
                    }
                }
            }
        } else {
            uint32_t f[4];
#pragma unroll
            for (int s2 = 0; s2 < kSteps; ++s2) {
                // matrices: keys 0-7 / 8-15, channels 16 s / 16 s + 8
                const int r = lane & 15, ch = 2 * s2 + (lane >> 4);
                ldsm_x4(at + r * L::kRow + ((ch & ~7) | ((ch ^ r) & 7)) * 16, f[0], f[1], f[2], f[3]);
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    if (s2 == 0) mma_first(z[a], f[0], f[1], f[2], f[3], qf[a][s2][0], qf[a][s2][1]);
                    else mma_next(z[a], f[0], f[1], f[2], f[3], qf[a][s2][0], qf[a][s2][1]);
                }
            }
        }

        // --------------------------------------------------------- softmax
        if (!whole) {
#pragma unroll
            for (int a = 0; a < NT; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = j0 + k0 + (i < 2 ? 0 : 8), r = min(8 * a + 2 * t + (i & 1), nr - 1), pos = sq.p0 + (r0 + r) / p.G;
                    const bool see = j <= pos && j < sq.m && (p.mask.window <= 0 || j < p.mask.n_sink || j > pos - p.mask.window);
                    if (!see || (bad >> s & 1)) z[a][i] = -INFINITY;
                }
        }
        const uint32_t av = at + kPagedTile * L::kRow;
        uint32_t vs0[kGroups], vs1[kGroups];  // 4 bits: V's groups, keys k0 and k0 + 8
        bool move = false;
        if constexpr (Q4) {
            lds(vs0, at + p_at + 16 * L::kParams);
            lds(vs1, at + p_at + 24 * L::kParams);
            if (!whole) {
                // a row takes nothing of a key that it does not see, whatever that stands for; one that sees NaN gets it
                const int ja = j0 + k0, jb = ja + 8;
                const bool none0 = !(ja < keys.sink || (ja >= keys.lo && ja < keys.hi)) || (bad >> s & 1);
                const bool none1 = !(jb < keys.sink || (jb >= keys.lo && jb < keys.hi)) || (bad >> s & 1);
#pragma unroll
                for (int j = 0; j < kGroups; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t &v = e ? vs1[j] : vs0[j];
                        if (e ? none1 : none0) v = 0;
                        if ((v & 0x7F80u) != 0x7F80u && (v & 0x7F800000u) != 0x7F800000u) continue;
                        v = 0;
#pragma unroll
                        for (int a = 0; a < NT; ++a)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (z[a][2 * e + i] != -INFINITY) ob[a][j][i] = __uint_as_float(0x7FC00000u);
                    }
            }
            uint32_t largest = max(vs0[0], vs1[0]);
#pragma unroll
            for (int j = 1; j < kGroups; ++j) largest = max(largest, max(vs0[j], vs1[j]));
            move = largest >= step_over;
        }
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int i = 0; i < 2; ++i) move = move || fmaxf(z[a][i], z[a][i + 2]) > over[a][i];
        if (__any_sync(kAll, move)) {
            float less = 1.f;
            if constexpr (Q4) {
                uint32_t largest = 0;
#pragma unroll
                for (int j = 0; j < kGroups; ++j) {
                    const uint32_t e0 = vs0[j] & 0x7F800000u, e1 = vs1[j] & 0x7F800000u;
                    largest = max(largest, max(e0 == 0x7F800000u ? 0 : e0, e1 == 0x7F800000u ? 0 : e1));
                }
                const int e = max(step_e, static_cast<int>(__reduce_max_sync(kAll, largest) >> 23) - 127);
                less = exponent_of(max(step_e - e, -126));
                step_e = e;
                step_over = min(static_cast<uint32_t>(e + 127 + static_cast<int>(kSlack)), 255u) << 23;
                prob = exponent_of(kProbE - e);
            }
#pragma unroll
            for (int a = 0; a < NT; ++a)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float mx = fmaxf(z[a][i], z[a][i + 2]) * sl2[a][i];
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, w));
                    const float mn = fmaxf(-nm[a][i], mx), f = pow2(-nm[a][i] - mn), fo = f * less;
                    nm[a][i] = -mn;
                    over[a][i] = mn == -FLT_MAX ? -INFINITY : (mn + kSlack) / sl2[a][i];
                    l[a][i] *= f;
#pragma unroll
                    for (int j = 0; j < kGroups; ++j) ob[a][j][i] *= f;
#pragma unroll
                    for (int s2 = 0; s2 < kSteps; ++s2) {
                        o[a][s2][i] *= fo;
                        o[a][s2][i + 2] *= fo;
                    }
                }
        }
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                z[a][i] = pow2(fmaf(z[a][i], sl2[a][i & 1], nm[a][i & 1]));
                l[a][i & 1] += z[a][i];
            }

        // --------------------------------------------------------- outputs
        if constexpr (Q4) {
            constexpr int W = D / 64;  // words of an eighth of a row
            uint32_t w[4][W];
#pragma unroll
            for (int i = 0; i < 4; ++i) lds(w[i], at + vw_at + 4 * i * L::kRow);
            float zp[NT][4];
#pragma unroll
            for (int a = 0; a < NT; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) zp[a][i] = z[a][i] * prob;
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                const uint32_t sel = j % 2 ? 0x7632 : 0x5410;
                const uint32_t x0 = __byte_perm(w[0][j / 2], w[1][j / 2], sel), x1 = __byte_perm(w[2][j / 2], w[3][j / 2], sel);
                const uint32_t y0 = x0 >> 8, y1 = x1 >> 8;
                const float st0 = q4_step(vs0[j]), st1 = q4_step(vs1[j]), ba0 = q4_base(vs0[j]), ba1 = q4_base(vs1[j]);
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    const uint32_t b0 = transpose8x8(pack_bf16x2(zp[a][0] * st0, zp[a][1] * st0));
                    const uint32_t b1 = transpose8x8(pack_bf16x2(zp[a][2] * st1, zp[a][3] * st1));
#pragma unroll
                    for (int i = 0; i < 2; ++i) ob[a][j][i] = fmaf(z[a][i + 2], ba1, fmaf(z[a][i], ba0, ob[a][j][i]));
                    mma_next(o[a][2 * j], kMinus8, kMinus8x16, kMinus8, kMinus8x16, b0, b1);
                    mma_next(o[a][2 * j + 1], kMinus8, kMinus8x16, kMinus8, kMinus8x16, b0, b1);
                    mma_next(o[a][2 * j], code(x0), code16(x0), code(x1), code16(x1), b0, b1);
                    mma_next(o[a][2 * j + 1], code(y0), code16(y0), code(y1), code16(y1), b0, b1);
                }
            }
        } else {
            uint32_t b0[NT], b1[NT], f[4];
#pragma unroll
            for (int a = 0; a < NT; ++a) {
                b0[a] = transpose8x8(pack_bf16x2(z[a][0], z[a][1]));
                b1[a] = transpose8x8(pack_bf16x2(z[a][2], z[a][3]));
            }
#pragma unroll
            for (int s2 = 0; s2 < kSteps; ++s2) {
                // matrices, transposed: channels 16 s / 16 s + 8, keys 0-7 / 8-15
                const int r = (lane & 7) + (lane >> 4) * 8, ch = 2 * s2 + (lane >> 3 & 1);
                ldsm_x4_trans(av + r * L::kRow + ((ch & ~7) | ((ch ^ r) & 7)) * 16, f[0], f[1], f[2], f[3]);
#pragma unroll
                for (int a = 0; a < NT; ++a) mma_next(o[a][s2], f[0], f[1], f[2], f[3], b0[a], b1[a]);
            }
        }
    }

    // -------------------------------------------------------------- the warps' parts
    copies_wait<0>();
#pragma unroll
    for (int w = 4; w < 32; w <<= 1)
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[a][i] += __shfl_xor_sync(kAll, l[a][i], w);
                if constexpr (Q4) {
#pragma unroll
                    for (int j = 0; j < kGroups; ++j) ob[a][j][i] += __shfl_xor_sync(kAll, ob[a][j][i], w);
                }
            }
    __syncthreads();  // the rings have been used
    constexpr int kPad = D + 4;
    float *const so = reinterpret_cast<float *>(ring), *const sm = so + kWarps * R * kPad, *const sl = sm + kWarps * R;
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float *row = so + (warp * R + 8 * a + 2 * t + (i & 1)) * kPad;
#pragma unroll
            for (int s2 = 0; s2 < kSteps; ++s2) {
                // 4 bits: tile 2 j + h has channels 32 j + 4 g + 2 h, and the next one
                if constexpr (Q4)
                    row[32 * (s2 / 2) + 4 * g + 2 * (s2 % 2) + i / 2] =
                        fmaf(o[a][s2][i] * exponent_of((i < 2 ? 0 : -4) - kProbE - kCodeE), exponent_of(step_e), ob[a][s2 / 2][i & 1]);
                else row[16 * s2 + g + 8 * (i / 2)] = o[a][s2][i];
            }
            if (g == 0 && i < 2) {
                sm[warp * R + 8 * a + 2 * t + i] = -nm[a][i];
                sl[warp * R + 8 * a + 2 * t + i] = l[a][i];
            }
        }
    __syncthreads();
    for (int e = threadIdx.x; e < nr * (D / 8); e += kWarps * 32) {
        const int r = e / (D / 8), ch = e % (D / 8) * 8;
        float big = -FLT_MAX, total = 0.f, v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) big = fmaxf(big, sm[w * R + r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = pow2(sm[w * R + r] - big);
            total = fmaf(f, sl[w * R + r], total);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(f, so[(w * R + r) * kPad + ch + i], v[i]);
        }
        const float inv = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= inv;
        const float lse2 = total == 0.f ? -INFINITY : big + log2f(total);
        const int tk = (r0 + r) / p.G, h = kvh * p.G + r0 + r - tk * p.G;
        const long long row = static_cast<long long>(sq.q0 + tk) * p.Hq + h;
        if (p.splits > 1) {
            const long long slot = static_cast<long long>(part) * p.tokens * p.Hq + row;
            float4 *po = reinterpret_cast<float4 *>(p.part_o + slot * D + ch);
            po[0] = make_float4(v[0], v[1], v[2], v[3]);
            po[1] = make_float4(v[4], v[5], v[6], v[7]);
            if (ch == 0) p.part_l[slot] = lse2;
        } else {
            __nv_bfloat16 *po = static_cast<__nv_bfloat16 *>(p.out) + h * p.os[0] + (sq.q0 + tk) * p.os[1] + ch;
            *reinterpret_cast<uint4 *>(po) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            if (ch == 0 && p.lse) p.lse[row] = lse2 * kLn2;
        }
    }
}

template <int D, bool Q4, int NT> cudaError_t mma_for(const PagedAttnParams &p, cudaStream_t st)
{
    constexpr int bytes = smem_bytes<D, Q4, NT>();
    auto kern = paged_mma_kernel<D, Q4, NT>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, static_cast<unsigned>(p.c.batch) * p.c.Hkv * p.q_tiles * p.splits, kWarps * 32, bytes, st, p);
}

template <int D, bool Q4> cudaError_t mma_rows(const PagedAttnParams &p, int rows, cudaStream_t st)
{
    return rows == 8 ? mma_for<D, Q4, 1>(p, st) : mma_for<D, Q4, 2>(p, st);
}

}  // namespace

cudaError_t launch_paged_mma(const PagedAttnParams &p, int head_dim, bool q4, int rows, cudaStream_t st)
{
    if (head_dim == 64) return q4 ? mma_rows<64, true>(p, rows, st) : mma_rows<64, false>(p, rows, st);
    return q4 ? mma_rows<128, true>(p, rows, st) : mma_rows<128, false>(p, rows, st);
}

}  // namespace kvevict
