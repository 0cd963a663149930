// paged_attn_mma.cu -- attention of a few bf16 queries over a paged cache, bf16 or
// 4 bits, on the tensor cores.
//
// A few rows over many keys are bound by the keys' bytes, so a warp works by
// itself: it walks tiles of 16 keys through a ring of its own in shared memory
// (cp.async), keeps its own softmax, and only at the end are a CTA's warps joined.
// The products are transposed, S^T = K Q^T and O^T = V^T P^T, with keys and then
// channels on the 16-wide axis of mma.m16n8k16 and query rows on the 8-wide one:
// eight query heads of a KV head fill an instruction. (tcgen05 could have the keys on
// its long axis in the same way, but takes them from shared or tensor memory as bf16:
// four times the bytes of 4-bit codes, written there first. bf16 pages are at their
// bytes without it.) P^T comes from S^T by transposing 8 x 8 blocks in registers
// (movmatrix).
//
// 4 bits: a code needs a mask and nothing else to be a matrix operand. bf16's bit
// patterns 0 .. 255 are the values 0 .. 255 times 2^-133 (its subnormals and, with
// the same spacing, the first normal numbers), so c, 16 c and a byte
// of two codes are read off as they lie in a half word. Queries are scaled by a power
// of two to at most 2^101, a sixteenth of it for every second channel, and
//   S_ij = sum_groups step (sum_c c q) + (base - 8 step) (sum q),
// the sums over a group in fp32. In the second product the step goes into the
// probabilities, which are then rounded to bf16, once, and scaled by a power of two
// that follows the largest step seen:
//   O_i = sum_j (p_ij step_j) (c_j - 8) + sum_j p_ij base_j,
// the 8 taken off the codes, exactly, the base's part in an instruction of its own.
//
// The running maximum (to base 2) is moved only where a logit exceeds it by more than
// 8: then, and only then, sums and outputs are rescaled. Probabilities below 2^8
// instead of below 1 cost no precision.
//
// bf16 pages are bound by their bytes: 32 sequences to 10240 tokens, 32 query heads over
// 8 of 128, 151 us, 94% of the copy bandwidth. 4 bits are not: 32 to 32768, 64 heads
// over 8, 212 us, 69%. Instructions of 16 keys x 128 channels on an SM quarter: about
// 140 of the logic unit at two cycles (masks, shifts, permutes, steps out of their
// words), 19 products at eight, ten transposes at four, 340 in all, against 437 cycles
// for the bytes; 580 are taken, because three warps a quarter (168 registers) do not
// cover a warp's chain. Two tiles at a time give it a second one (252 us with one); four
// spill (272 at that stage), and four CTAs of 128 registers with one tile gained nothing
// (250).
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

template <int D, bool Q4, int NT> struct Ring {
    static constexpr int kRow = Q4 ? D / 2 : D * 2;                            // bytes of a key, codes only
    static constexpr int kParams = Q4 ? D / 8 : 0;                             // and its groups
    static constexpr int kTile = 2 * kPagedTile * (kRow + kParams);            // K codes, V codes, K groups, V groups
    // of a stage. 16 rows: one, two spill (30.5 us against 26.1 for to 5 tokens of 16 sequences, 2048 keys, 32 heads over 8)
    static constexpr int kTiles = Q4 && NT == 1 ? 2 : 1;
    static constexpr int kStage = kTiles * kTile;
    static constexpr int kStages = Q4 ? (D == 128 ? 6 : 8) / kTiles : (D == 128 ? 3 : 6);
    static constexpr int kWarpBytes = kStage * kStages;
};

template <int D, bool Q4, int NT> constexpr int smem_bytes()
{
    constexpr int ring = Ring<D, Q4, NT>::kWarpBytes * kWarps, join = (kWarps * (D + 4 + 2) + 2) * 8 * NT * 4;
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
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// D = A B, and D += A B. (Not volatile: what they need is in their operands, and the compiler may move them.)
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_next(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^x, off by two steps at most; 0 below 2^-126.
__device__ __forceinline__ float pow2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Codes of two keys or channels, one in each half word, as bf16: c 2^-133, and
// from the next nibble 16 c 2^-133. Or a byte of each, c + 16 c' of two nibbles.
__device__ __forceinline__ uint32_t code(uint32_t x) { return x & 0x000F000Fu; }
__device__ __forceinline__ uint32_t code16(uint32_t x) { return x & 0x00F000F0u; }
// Such a code less 8, such a byte less 136 (8 of either nibble): exact.
template <int N> __device__ __forceinline__ uint32_t less(uint32_t x)
{
    uint32_t y;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(N * 0x00010001u));
    return y;
}
__device__ __forceinline__ uint32_t low_bytes(uint32_t x) { return x & 0x00FF00FFu; }
__device__ __forceinline__ uint32_t high_bytes(uint32_t x) { return __byte_perm(x, 0u, 0x4341); }
__device__ __forceinline__ bool finite_group(uint32_t v) { return (v & 0x7F80u) != 0x7F80u && (v & 0x7F800000u) != 0x7F800000u; }

__device__ __forceinline__ float exponent_of(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // 2^e

constexpr int kMinE = -20;  // of the steps' power of two E, from which the maximum is counted kProbE lower (see below)
constexpr int kProbE = 40;
constexpr int kCodeE = -133;

// The upper, middle and lower eight bits of an fp32 value (i = 0, 1, 2), or 0.
__device__ __forceinline__ float bf16_part(float x, int i)
{
    const float hi = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u), r = x - hi;
    const float mid = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u);
    return i == 0 ? hi : i == 1 ? mid : i == 2 ? r - mid : 0.f;
}

// W words of shared memory.
template <int W> __device__ __forceinline__ void lds(uint32_t (&v)[W], const char *a)
{
    if constexpr (W == 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(a);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else if constexpr (W == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(a);
        v[0] = x.x; v[1] = x.y;
    } else {
        v[0] = *reinterpret_cast<const uint32_t *>(a);
    }
}

// Row r (0 .. 7) of an 8 x 8 block of S^T is this key of a 4-bit tile's half, so
// that after the transpose a lane's keys lie four apart: t and 4 + t. Its loads of
// V, one row of codes a key, then take neighbouring rows side by side.
__device__ __forceinline__ int key_of(int r) { return (r & 1) * 4 + (r >> 1); }

template <int D, bool Q4, int NT>
__global__ void __launch_bounds__(kWarps * 32, (NT == 1 ? 3 : 2)) paged_mma_kernel(const __grid_constant__ PagedAttnParams p)
{
    using L = Ring<D, Q4, NT>;
    constexpr int R = 8 * NT, kGroups = D / 32, kSteps = D / 16;  // rows; groups; 16-channel steps, or tiles of O^T
    constexpr int kTiles = L::kTiles;
    extern __shared__ __align__(16) char ring[];
    grid_dependency_wait();
    const PagedCache &c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    int item = blockIdx.x;
    const int part = item % p.splits;
    item /= p.splits;
    const int tile = item % p.q_tiles, unit = item / p.q_tiles;
    const int b = unit / c.Hkv, kvh = unit - b * c.Hkv;
    const PagedSeq sq = paged_sequence(p, b, !p.mask.q_starts || attn_first_fall(p.mask, b, lane) == INT_MAX);
    if (sq.bad && threadIdx.x == 0) atomicOr(c.err, KVEVICT_DEV_BAD_LENGTH);
    const int r0 = tile * R, nr = min(R, sq.n * p.G - r0);
    if (nr <= 0) return;
    const int pa = sq.p0 + r0 / p.G, pb = sq.p0 + (r0 + nr - 1) / p.G;  // the rows' positions
    const AttnKeys keys = attn_keys(p.mask, sq.m, pa, pb, kPagedTile);
    const int i_lo = static_cast<int>(static_cast<long long>(keys.count) * part / p.splits);
    const int i_hi = static_cast<int>(static_cast<long long>(keys.count) * (part + 1) / p.splits);
    // this warp's tiles come kTiles at a time: number k is i_lo + kTiles (kWarps (k / kTiles) + warp) + k % kTiles, and an
    // odd last one is followed by one without a page
    const int n_all = i_hi - i_lo, n_rounds = n_all / (kTiles * kWarps), n_rest = n_all - n_rounds * (kTiles * kWarps) - kTiles * warp;
    const int n_mine = n_rounds * kTiles + min(max(n_rest, 0), kTiles);
    const int n_stages = (n_mine + kTiles - 1) / kTiles;
    const int low_b = p.mask.window > 0 && pb >= p.mask.window ? pb - p.mask.window + 1 : 0;

    // Of 32 of this warp's tiles, one a lane: where their pages' blocks are, the first key, and whether every row sees
    // every key (kWhole) or there is no page (kNoPage). The next 32 tiles' pages are on their way.
    constexpr int kWhole = 1, kNoPage = 2;
    auto first_key = [&](int k) { return attn_tile_at(keys, i_lo + kTiles * (k / kTiles * kWarps + warp) + k % kTiles) * kPagedTile; };
    auto page_at = [&](int k) { return k < n_mine ? paged_page(c, b, first_key(k)) : 0; };
    const char *block[2] = {};
    int what = 0, page_next = page_at(lane);
    auto next_tiles = [&](int k) {  // the tiles k .. k + 31
        const int page = page_next;
        page_next = page_at(k + 32 + lane);
        const int j0 = first_key(k + lane);
        const bool none = page < 0 || k + lane >= n_mine;
        const bool whole = !none && j0 + kPagedTile - 1 <= min(pa, sq.m - 1) && (j0 + kPagedTile <= p.mask.n_sink || j0 >= low_b);
        what = j0 | (whole ? kWhole : 0) | (none ? kNoPage : 0);
        if (page < 0) atomicOr(c.err, KVEVICT_DEV_BAD_PAGE);
#pragma unroll
        for (int i = 0; i < 2; ++i) block[i] = c.pages[i] + max(page, 0) * c.page_bytes[i] + kvh * c.head_bytes[i];
    };

    // ------------------------------------------------------------ copies into the ring
    const uint32_t my_ring = smem_u32(ring) + warp * L::kWarpBytes, ring_end = my_ring + L::kWarpBytes;
    // 4 bits: what a lane copies. K's rows go in by eights in key_of's order; V's as they are, with the 16-byte chunks of
    // every second pair of rows swapped (D = 128), so that four rows' parts lie in different banks.
    constexpr int kPc = L::kParams;  // 16-byte chunks of a tile's groups, of K and of V
    const int cr = lane / (L::kRow / 16), cch = lane % (L::kRow / 16);
    const int k_from = ((cr & 8) + key_of(cr & 7)) * L::kRow + cch * 16, v_from = cr * L::kRow + (D == 128 ? cch ^ (cr & 2) : cch) * 16;
    const int p_from = Q4 ? c.S * L::kRow + lane % max(kPc, 1) * 16 : 0;
    uint32_t to = my_ring;  // the stage that the next copies go to
    auto issue = [&](int k) {  // stage k
        if (k < n_stages) {
            if ((k * kTiles & 31) == 0) next_tiles(k * kTiles);
#pragma unroll
            for (int h = 0; h < kTiles; ++h) {
                const int from = (k * kTiles + h) & 31;
                const int w = __shfl_sync(kAll, what, from);
                const char *kb = reinterpret_cast<const char *>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(block[0]), from));
                const char *vb = reinterpret_cast<const char *>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(block[1]), from));
                const int slot0 = w & (c.S - kPagedTile);
                if constexpr (Q4) {
                    if (!(w & kNoPage)) {
                        const char *kc = kb + (slot0 * L::kRow + k_from), *vc = vb + (slot0 * L::kRow + v_from);
                        const char *pc = (lane < kPc ? kb : vb) + (slot0 * L::kParams + p_from);
                        const uint32_t dst = to + h * L::kTile + lane * 16;
#pragma unroll
                        for (int e0 = 0; e0 < kPagedTile * L::kRow; e0 += 512) {
                            copy16(dst + e0, kc + e0, true);
                            copy16(dst + kPagedTile * L::kRow + e0, vc + e0, true);
                        }
                        if (lane < 2 * kPc) copy16(dst + 2 * kPagedTile * L::kRow, pc, true);
                    }
                } else {
                    // 16-byte chunks swapped by row, so that the eight rows of a matrix load lie in different banks
                    constexpr int kChunks = L::kRow / 16;
                    const int j0 = w & ~(kPagedTile - 1);
#pragma unroll
                    for (int e0 = 0; e0 < kPagedTile * kChunks; e0 += 32) {
                        const int e = e0 + lane, r = e / kChunks, ch = e % kChunks, j = j0 + r;
                        const bool real = !(w & kNoPage) && (j < keys.sink || (j >= keys.lo && j < keys.hi));
                        const uint32_t at = r * L::kRow + ((ch & ~7) | ((ch ^ r) & 7)) * 16;
                        // (zeros where no row sees the key; the address of a tile without a page is the first page's)
                        copy16(to + at, kb + (slot0 + r) * c.token_bytes[0] + ch * 16, real);
                        copy16(to + kPagedTile * L::kRow + at, vb + (slot0 + r) * c.token_bytes[1] + ch * 16, real);
                    }
                }
            }
        }
        to += L::kStage;
        if (to == ring_end) to = my_ring;
        copies_close();
    };
#pragma unroll 1
    for (int k = 0; k < L::kStages - 1; ++k) issue(k);

    // ---------------------------------------------------------------- queries, row n = 8 a + g
    uint32_t qf[NT][kSteps][2];
    uint32_t qs[NT][2][2];       // 4 bits: of each group the sum of row g, and -8 of it, in bf16 parts (see below)
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
            float qg[kGroups];
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
                qg[j] = sum * exponent_of(100 + kCodeE);  // times 2^-133 like the products
            }
            // An instruction's 16 channels hold the groups' bases (or steps): D = 128, lane t groups 2 (t & 1) and the next;
            // they meet the sums' upper parts (t < 2), middle (t >= 2) and, eight further, lower parts (t < 2). D = 64: both
            // groups in every lane, with the upper, middle and lower part for t = 0, 1, 2.
            const int pair = D == 128 ? t & 1 : 0, part0 = D == 128 ? t >> 1 : t, part1 = D == 128 && t < 2 ? 2 : 3;
            const float s0 = pair ? qg[kGroups - 2] : qg[0], s1 = pair ? qg[kGroups - 1] : qg[1];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float f = i ? -8.f : 1.f;
                qs[a][i][0] = pack_bf16x2(f * bf16_part(s0, part0), f * bf16_part(s1, part0));
                qs[a][i][1] = pack_bf16x2(f * bf16_part(s0, part1), f * bf16_part(s1, part1));
            }
        } else {
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    qf[a][s][i] = r < nr ? *reinterpret_cast<const uint32_t *>(qr + 16 * s + 8 * i + 2 * t) : 0u;
        }
    }

    // nm: minus the running maximum (to base 2), 4 bits: counted kProbE - E lower, 2^E the power of two of the largest step
    // seen, so that probability times step times code stays in range; over: the product above which it is moved. ob: 4 bits,
    // sums of p base, row g of the product the group g.
    float nm[NT][2], over[NT][2], l[NT][2], o[NT][kSteps][4], ob[NT][4];
    int step_e = kMinE;
    uint32_t step_over = 0;  // the group (as it is stored) from which on E is moved
#pragma unroll
    for (int a = 0; a < NT; ++a) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            nm[a][i] = FLT_MAX;
            over[a][i] = -INFINITY;
            l[a][i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) ob[a][i] = 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[a][s][i] = 0.f;
    }
    // this lane's keys of a tile: k0 and k0 + 8
    const int k0 = Q4 ? key_of(g) : g;
    const int kw_at = g * L::kRow + t * (D / 8), vw_at = kPagedTile * L::kRow + t * L::kRow + (D == 128 ? (g >> 1 ^ (t & 2)) * 16 + (g & 1) * 8 : g * 4);
    constexpr int kParamsAt = 2 * kPagedTile * L::kRow;
    const int p_at = kParamsAt + k0 * L::kParams, pair_at = kParamsAt + k0 * L::kParams + (D == 128 ? (t & 1) * 8 : 0);
    const int vb_at = kParamsAt + (kPagedTile + t) * L::kParams + (g & (kGroups - 1)) * 4;
    uint32_t at = my_ring;
    int whats = 0;  // of the 32 tiles that the present one is among

#pragma unroll 1
    for (int k = 0; k < n_stages; ++k) {
        if ((k * kTiles & 31) == 0) whats = what;
        copies_wait<L::kStages - 2>();
        __syncwarp();
        issue(k + L::kStages - 1);
        const char *const sp = ring + (at - smem_u32(ring));
        int tile_is[kTiles];
        bool whole = true;
#pragma unroll
        for (int h = 0; h < kTiles; ++h) {
            tile_is[h] = __shfl_sync(kAll, whats, (k * kTiles + h) & 31);
            whole = whole && (tile_is[h] & kWhole);
        }
        // whether no row of this item sees key `key` of tile h
        auto unseen = [&](int h, int key) {
            const int j = (tile_is[h] & ~(kPagedTile - 1)) + key;
            return (tile_is[h] & kNoPage) || !(j < keys.sink || (j >= keys.lo && j < keys.hi));
        };

        // ---------------------------------------------------------- logits
        float z[kTiles][NT][4];
        if constexpr (Q4) {
            constexpr int W = D / 32;  // words of codes: an eighth of a row twice
            uint32_t w0[kTiles][W], w1[kTiles][W], ps0[kTiles][kGroups], ps1[kTiles][kGroups], p0[kTiles][2], p1[kTiles][2];
#pragma unroll
            for (int h = 0; h < kTiles; ++h) {
                lds(w0[h], sp + h * L::kTile + kw_at);
                lds(w1[h], sp + h * L::kTile + kw_at + 8 * L::kRow);
                lds(ps0[h], sp + h * L::kTile + p_at);
                lds(ps1[h], sp + h * L::kTile + p_at + 8 * L::kParams);
                lds(p0[h], sp + h * L::kTile + pair_at);  // this lane's pair of groups
                lds(p1[h], sp + h * L::kTile + pair_at + 8 * L::kParams);
                // base (sum q) - 8 step (sum q), all groups
                const uint32_t ba0 = __byte_perm(p0[h][0], p0[h][1], 0x5410), ba1 = __byte_perm(p1[h][0], p1[h][1], 0x5410);
                const uint32_t sp0 = __byte_perm(p0[h][0], p0[h][1], 0x7632), sp1 = __byte_perm(p1[h][0], p1[h][1], 0x7632);
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    mma_first(z[h][a], ba0, ba1, ba0, ba1, qs[a][0][0], qs[a][0][1]);
                    mma_next(z[h][a], sp0, sp1, sp0, sp1, qs[a][1][0], qs[a][1][1]);
                }
            }
#pragma unroll
            for (int j = 0; j < kGroups; ++j)
#pragma unroll
                for (int h = 0; h < kTiles; ++h) {
                    // half word j of both eighths: channels 8 t + i below, 8 t + 4 + i above
                    const uint32_t sel = j % 2 ? 0x7632 : 0x5410;
                    const uint32_t x0 = __byte_perm(w0[h][j / 2], w0[h][W / 2 + j / 2], sel), x1 = __byte_perm(w1[h][j / 2], w1[h][W / 2 + j / 2], sel);
                    const uint32_t y0 = x0 >> 8, y1 = x1 >> 8;
                    const float st0 = q4_step(ps0[h][j]), st1 = q4_step(ps1[h][j]);
#pragma unroll
                    for (int a = 0; a < NT; ++a) {
                        float d[4];
                        mma_first(d, code(x0), code(x1), code16(x0), code16(x1), qf[a][2 * j][0], qf[a][2 * j][1]);
                        mma_next(d, code(y0), code(y1), code16(y0), code16(y1), qf[a][2 * j + 1][0], qf[a][2 * j + 1][1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) z[h][a][i] = fmaf(i < 2 ? st0 : st1, d[i], z[h][a][i]);
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
                    if (s2 == 0) mma_first(z[0][a], f[0], f[1], f[2], f[3], qf[a][s2][0], qf[a][s2][1]);
                    else mma_next(z[0][a], f[0], f[1], f[2], f[3], qf[a][s2][0], qf[a][s2][1]);
                }
            }
        }

        // --------------------------------------------------------- softmax
        if (!whole) {
#pragma unroll
            for (int h = 0; h < kTiles; ++h)
#pragma unroll
                for (int a = 0; a < NT; ++a)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = (tile_is[h] & ~(kPagedTile - 1)) + k0 + (i < 2 ? 0 : 8);
                        const int r = min(8 * a + 2 * t + (i & 1), nr - 1), pos = sq.p0 + (r0 + r) / p.G;
                        const bool see = j <= pos && j < sq.m && (p.mask.window <= 0 || j < p.mask.n_sink || j > pos - p.mask.window);
                        if (!see || (tile_is[h] & kNoPage)) z[h][a][i] = -INFINITY;
                    }
        }
        uint32_t largest = 0;
        bool move = false;
        if constexpr (Q4) {
            // two words a lane (D = 64: one) are all of V's groups of a tile
#pragma unroll
            for (int h = 0; h < kTiles; ++h) {
                uint32_t v[kGroups / 2];
                lds(v, sp + h * L::kTile + kParamsAt + kPagedTile * L::kParams + lane * (2 * kGroups));
                if (!whole && unseen(h, lane >> 1)) v[0] = v[kGroups / 2 - 1] = 0;  // (a key that no row sees does not count)
#pragma unroll
                for (int i = 0; i < kGroups / 2; ++i) largest = max(largest, v[i]);
            }
            move = largest >= step_over;
        }
        float top[NT][2];
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[a][i] = fmaxf(z[0][a][i], z[0][a][i + 2]);
#pragma unroll
                for (int h = 1; h < kTiles; ++h) top[a][i] = fmaxf(top[a][i], fmaxf(z[h][a][i], z[h][a][i + 2]));
                move = move || top[a][i] > over[a][i];
            }
        if (__any_sync(kAll, move)) {
            float lower = 0.f, rise = 0.f;
            if constexpr (Q4) {
                const uint32_t e = largest & 0x7F800000u;  // (infinities and NaN are no measure)
                const int was = step_e;
                step_e = max(step_e, static_cast<int>(__reduce_max_sync(kAll, e == 0x7F800000u ? 0u : e) >> 23) - 127);
                rise = static_cast<float>(step_e - was);
                step_over = min(static_cast<uint32_t>(step_e + 127 + static_cast<int>(kSlack)), 255u) << 23;
                lower = static_cast<float>(kProbE - step_e);
            }
#pragma unroll
            for (int a = 0; a < NT; ++a)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float mx = top[a][i] * sl2[a][i];
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, w));
                    const float mn = fmaxf(rise - nm[a][i], mx - lower), f = pow2(-nm[a][i] - mn);
                    nm[a][i] = -mn;
                    over[a][i] = mn == -FLT_MAX ? -INFINITY : (mn + lower + kSlack) / sl2[a][i];
                    l[a][i] *= f;
                    ob[a][i] *= f;
                    ob[a][i + 2] *= f;
#pragma unroll
                    for (int s2 = 0; s2 < kSteps; ++s2) {
                        o[a][s2][i] *= f;
                        o[a][s2][i + 2] *= f;
                    }
                }
        }
#pragma unroll
        for (int h = 0; h < kTiles; ++h)
#pragma unroll
            for (int a = 0; a < NT; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    z[h][a][i] = pow2(fmaf(z[h][a][i], sl2[a][i & 1], nm[a][i & 1]));
                    l[a][i & 1] += z[h][a][i];
                }

        // --------------------------------------------------------- outputs
        if constexpr (Q4) {
            constexpr int W = D / 64;  // words of an eighth of a row
            uint32_t w[kTiles][4][W], vs0[kTiles][kGroups], vs1[kTiles][kGroups], vb[kTiles][4][1];
#pragma unroll
            for (int h = 0; h < kTiles; ++h) {
                const char *const tp = sp + h * L::kTile;
#pragma unroll
                for (int i = 0; i < 4; ++i) lds(w[h][i], tp + vw_at + 4 * i * L::kRow);
                lds(vs0[h], tp + p_at + 16 * L::kParams);
                lds(vs1[h], tp + p_at + 24 * L::kParams);
#pragma unroll
                for (int i = 0; i < 4; ++i) lds(vb[h][i], tp + vb_at + 4 * i * L::kParams);  // group g (mod kGroups) of this lane's four keys
                if (!whole) {
                    // a row takes nothing of a key that it does not see, whatever that stands for; one that sees NaN gets it
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!finite_group(vb[h][i][0]) || unseen(h, 4 * i + t)) vb[h][i][0] = 0;
#pragma unroll
                    for (int j = 0; j < kGroups; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t &v = e ? vs1[h][j] : vs0[h][j];
                            const bool none = unseen(h, k0 + 8 * e), nan = !finite_group(v) && !none;
                            if (none || nan) v = 0;
#pragma unroll
                            for (int a = 0; a < NT; ++a)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    // (each row of the product of the bases is a group: the lanes with g = j take it up)
                                    const bool hit = __reduce_or_sync(kAll, nan && z[h][a][2 * e + i] != 0.f ? 1u << t : 0u) >> t & 1;
                                    if (hit && (g & (kGroups - 1)) == j) ob[a][i] = __uint_as_float(0x7FC00000u);
                                }
                        }
                }
                const uint32_t va0 = __byte_perm(vb[h][0][0], vb[h][1][0], 0x5410), va1 = __byte_perm(vb[h][2][0], vb[h][3][0], 0x5410);
#pragma unroll
                for (int a = 0; a < NT; ++a)
                    mma_next(ob[a], va0, 0, va1, 0, transpose8x8(pack_bf16x2(z[h][a][0], z[h][a][1])),
                             transpose8x8(pack_bf16x2(z[h][a][2], z[h][a][3])));
            }
#pragma unroll
            for (int j = 0; j < kGroups; ++j)
#pragma unroll
                for (int h = 0; h < kTiles; ++h) {
                    const uint32_t sel = j % 2 ? 0x7632 : 0x5410;
                    const uint32_t x0 = __byte_perm(w[h][0][j / 2], w[h][1][j / 2], sel), x1 = __byte_perm(w[h][2][j / 2], w[h][3][j / 2], sel);
                    const uint32_t y0 = high_bytes(x0), y1 = high_bytes(x1), v0 = low_bytes(x0), v1 = low_bytes(x1);
                    const float st0 = q4_step(vs0[h][j]), st1 = q4_step(vs1[h][j]);
#pragma unroll
                    for (int a = 0; a < NT; ++a) {
                        const uint32_t b0 = transpose8x8(pack_bf16x2(z[h][a][0] * st0, z[h][a][1] * st0));
                        const uint32_t b1 = transpose8x8(pack_bf16x2(z[h][a][2] * st1, z[h][a][3] * st1));
                        mma_next(o[a][2 * j], less<8>(code(v0)), less<136>(v0), less<8>(code(v1)), less<136>(v1), b0, b1);
                        mma_next(o[a][2 * j + 1], less<8>(code(y0)), less<136>(y0), less<8>(code(y1)), less<136>(y1), b0, b1);
                    }
                }
        } else {
            uint32_t b0[NT], b1[NT], f[4];
#pragma unroll
            for (int a = 0; a < NT; ++a) {
                b0[a] = transpose8x8(pack_bf16x2(z[0][a][0], z[0][a][1]));
                b1[a] = transpose8x8(pack_bf16x2(z[0][a][2], z[0][a][3]));
            }
#pragma unroll
            for (int s2 = 0; s2 < kSteps; ++s2) {
                // matrices, transposed: channels 16 s / 16 s + 8, keys 0-7 / 8-15
                const int r = (lane & 7) + (lane >> 4) * 8, ch = 2 * s2 + (lane >> 3 & 1);
                ldsm_x4_trans(at + kPagedTile * L::kRow + r * L::kRow + ((ch & ~7) | ((ch ^ r) & 7)) * 16, f[0], f[1], f[2], f[3]);
#pragma unroll
                for (int a = 0; a < NT; ++a) mma_next(o[a][s2], f[0], f[1], f[2], f[3], b0[a], b1[a]);
            }
        }
        at += L::kStage;
        if (at == ring_end) at = my_ring;
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
            }
    float obs[NT][kGroups][2];  // every group's
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int j = 0; j < kGroups; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) obs[a][j][i] = Q4 ? __shfl_sync(kAll, ob[a][i], 4 * j + t) : 0.f;
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
                // 4 bits: tile 2 j + h has channel 32 j + 4 g + 2 h, and it with 16 times the next one
                if constexpr (Q4)
                    row[32 * (s2 / 2) + 4 * g + 2 * (s2 % 2) + i / 2] =
                        fmaf((i < 2 ? o[a][s2][i] : (o[a][s2][i] - o[a][s2][i & 1]) * 0.0625f) * exponent_of(66), exponent_of(-kCodeE - 66),
                             obs[a][s2 / 2][i & 1]);
                else row[16 * s2 + g + 8 * (i / 2)] = o[a][s2][i];
            }
            if (g == 0 && i < 2) {
                sm[warp * R + 8 * a + 2 * t + i] = -nm[a][i];
                sl[warp * R + 8 * a + 2 * t + i] = l[a][i];
            }
        }
    __syncthreads();
    float *const cm = sl + kWarps * R, *const cl = cm + R;  // the CTA's maximum and sum of a row
    // the warps' parts of eight channels of a row (e: which), and the CTA's maximum and sum
    auto join_warps = [&](int r, int ch, float(&v)[8], float &big) {
        float total = 0.f;
        big = -FLT_MAX;
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
        return total;
    };
    if (p.clusters) {
        // into the place of the first warp's part, where only this thread reads; then each CTA of the cluster joins a share
        for (int e = threadIdx.x; e < nr * (D / 8); e += kWarps * 32) {
            const int r = e / (D / 8), ch = e % (D / 8) * 8;
            float v[8], big;
            const float total = join_warps(r, ch, v, big);
#pragma unroll
            for (int i = 0; i < 8; ++i) so[r * kPad + ch + i] = v[i];
            if (ch == 0) {
                cm[r] = big;
                cl[r] = total;
            }
        }
        cluster_sync();
    }
    const int share = p.clusters ? p.splits : 1, from = p.clusters ? part : 0;
    for (int e = threadIdx.x * share + from; e < nr * (D / 8); e += kWarps * 32 * share) {
        const int r = e / (D / 8), ch = e % (D / 8) * 8;
        float v[8], big;
        const float total = p.clusters ? paged_join_peers(so + r * kPad + ch, cm + r, cl + r, p.splits, v, big) : join_warps(r, ch, v, big);
        const float inv = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= inv;
        const float lse2 = total == 0.f ? -INFINITY : big + log2f(total);
        const int tk = (r0 + r) / p.G, h = kvh * p.G + r0 + r - tk * p.G;
        const long long row = static_cast<long long>(sq.q0 + tk) * p.Hq + h;
        if (p.splits > 1 && !p.clusters) {
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
    if (p.clusters) cluster_sync();  // no CTA's shared memory goes while another reads it
}

template <int D, bool Q4, int NT> cudaError_t mma_for(const PagedAttnParams &p, cudaStream_t st)
{
    constexpr int bytes = smem_bytes<D, Q4, NT>();
    auto kern = paged_mma_kernel<D, Q4, NT>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, static_cast<unsigned>(p.c.batch) * p.c.Hkv * p.q_tiles * p.splits, kWarps * 32, bytes, st, p,
                            p.clusters ? static_cast<unsigned>(p.splits) : 1u);
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
