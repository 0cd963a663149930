// window_attn_tc.cu -- attention for bf16 on the 5th-generation tensor cores.
//
// One pass over the key tiles a row sees, with a running maximum and sum:
//   S = Q K^T (tcgen05, fp32 in TMEM);  p = 2^(S c - M), c = scale log2(e);
//   l += sum p;  O += P V (P rounded to bf16 in TMEM, fp32 accumulator in TMEM);
//   out = O / l, lse = (M + log2 l) ln 2.
// M is the row's running maximum, but moves (and O and l are rescaled by
// 2^(old - new)) only where the new maximum is more than 8 above it: until
// then p <= 256, which changes nothing in the relative precision of fp32 sums
// or of bf16 probabilities, and the rescaling's pass over O is rare.
//
// A persistent CTA per SM walks items (window_attn.h). It holds two row tiles
// of 128 rows ("subs"), each with its own S/P and O in TMEM (S0 S1 O0 O1: 512
// columns; P overwrites the first half of S) and its own softmax warpgroup, a
// row a thread: while one sub's rows go through the softmax the tensor cores
// work for the other. A K or V tile of 128 keys is loaded once for both subs
// (TMA ring). Where a unit's rows fit one sub ("pair": decoding, short
// chunks), both hold the same rows and take alternate key tiles; their sums
// are joined through TMEM at the end of the item. Rows are (token, group
// head) pairs, so all query heads of a KV head share its tiles.
//
// Warps 0-3, 4-7: softmax and output of sub 0, 1; 8: TMA; 9: MMA issue; 10: the items.
#include <cmath>

#include "tc5_common.cuh"
#include "window_attn.h"
#include "window_attn_common.cuh"

namespace kvevict {

namespace {

constexpr int kBM = kAttnTcRows, kBN = kAttnTcKeys;
constexpr int kSubThreads = 128;
constexpr int kTmaWarp = 8, kMmaWarp = 9, kSchedWarp = 10;
constexpr int kTcThreads = 384;       // warp 11 only completes the third warpgroup, for the register split
// Registers a thread: the launch's 168 (65,536 over 384 threads), of which the
// third warpgroup gives up 80 to the softmax warpgroups, whose threads hold a
// whole row of 128 logits: 2 x 208 + 88 = 3 x 168.
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 208, kIssueRegs = 88;
static_assert(2 * kSoftmaxRegs + kIssueRegs <= 3 * kLaunchRegs, "register split");
constexpr uint32_t kTcTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 * sub
constexpr float kRescale = 8.f;             // log2 units
constexpr float kLn2 = 0.69314718055994531f;

template <int D> struct TcLayout {
    static constexpr int kTile = 128 * D * 2;  // one Q, K or V tile: D / 64 boxes of 128 rows x 128 bytes
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kOffQ = 0;
    static constexpr int kOffKV = 2 * kTile;
    static constexpr int kOffBar = kOffKV + kStages * kTile;
    static constexpr int kOffX = kOffBar + 256;               // [2][128] log2 normalisers of the subs' rows
    static constexpr int kOffItem = kOffX + 2 * kBM * 4;      // posted items
    static constexpr int kBytes = kOffItem + 256 + 1024;  // + slack to align the base to 1 KB
};
static_assert(TcLayout<128>::kBytes <= 232448 && TcLayout<64>::kBytes <= 232448, "shared memory");

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float fmax3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mov.b64 rc, {%6, %7};\n\tfma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Named barrier over nthreads threads that counts those with a true `pred`.
__device__ __forceinline__ int named_bar_count(int id, int nthreads, bool pred)
{
    int n;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.popc.aligned.u32 %0, %1, %2, p;\n\t}"
                 : "=r"(n)
                 : "r"(id), "r"(nthreads), "r"(pred ? 1u : 0u)
                 : "memory");
    return n;
}

// D[tmem] (+)= A[tmem] * B for one K step, A bf16 pairs in TMEM columns.
__device__ __forceinline__ void tc_mma_ts_bf16(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                               bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Shared-memory descriptor of a V tile as the B operand with N (head_dim)
// contiguous: atoms of 8 keys x 64 columns (1 KB, 128-byte swizzle); the
// stride between groups of 8 keys is 1 KB (bits 32-45), between 64-column
// boxes 16 KB (bits 16-29).
__device__ __forceinline__ uint64_t smem_desc_v(uint32_t addr)
{
    uint64_t d = static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(16384u >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, int x, int y, int z, int w, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_5d(void *dst, const void *tmap, int x, int y, int z, int w, int u, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(u), "r"(smem_u32(bar))
        : "memory");
}

// Of 32 logits (keys 0 .. 31 of the chunk), those not seen become -infinity:
// seen is e <= top, and e >= low or e < sink.
__device__ __forceinline__ void tc_mask32(uint32_t (&r)[32], int top, int low, int sink)
{
    uint32_t seen = top >= 31 ? 0xffffffffu : top < 0 ? 0u : (2u << top) - 1u;
    const uint32_t near = low <= 0 ? 0xffffffffu : low >= 32 ? 0u : ~((1u << low) - 1u);
    const uint32_t first = sink >= 32 ? 0xffffffffu : sink <= 0 ? 0u : (1u << sink) - 1u;
    seen &= near | first;
#pragma unroll
    for (int e = 0; e < 32; ++e) r[e] = (seen >> e) & 1u ? r[e] : 0xff800000u;
}

__device__ __forceinline__ float tc_max32(const uint32_t (&r)[32])
{
    float m = fmax3(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[2]));
#pragma unroll
    for (int e = 3; e < 31; e += 2) m = fmax3(m, __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
    return fmaxf(m, __uint_as_float(r[31]));
}

// 2^(r c - m) of 32 logits: their sums in four chains, and as 16 bf16 pairs.
__device__ __forceinline__ void tc_exp32(const uint32_t (&r)[32], float2 c2, float2 nm2, float2 (&sum)[4], uint32_t *pk)
{
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        const float2 z = ffma2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), c2, nm2);
        const float2 pe = make_float2(ex2(z.x), ex2(z.y));
        sum[(e >> 1) & 3] = fadd2(sum[(e >> 1) & 3], pe);
        pk[e / 2] = pack_bf16x2(pe.x, pe.y);
    }
}

// One sub of an item: its tokens, the key tiles they see, how many of them
// are in this part.
struct TcSub {
    int t0, nt;
    int tiles_sink, main0, end;
    int count;
};

// An item as the scheduler warp posts it in shared memory.
struct TcItem {
    int prob;          // -1: no more work
    int part, b, kvh;
    int q0, k0, p0, m; // of its sequence: first rows, position of the first query, keys
    int bad;
    AttnKeys keys;     // of both subs together
    int lo, hi;        // this part of the list of key tiles
    int pair;
    TcSub sub[2];
};
constexpr int kItemSlots = 2;

__device__ __forceinline__ bool tc_active(const TcItem &it, int n, int s)
{
    if (it.pair) return ((n - it.lo) & 1) == s;
    const int t = attn_tile_at(it.keys, n);
    return t < it.sub[s].tiles_sink || (t >= it.sub[s].main0 && t < it.sub[s].end);
}

// Keys of a tile to work on, a multiple of 16: the others are seen by no row.
__device__ __forceinline__ int tc_keys_in(const AttnKeys &keys, bool sink_tile, int tile)
{
    const int j0 = tile * kBN;
    const int last = sink_tile && j0 + kBN <= keys.lo ? min(keys.sink, keys.hi) : keys.hi;
    return min(kBN, (last - j0 + 15) & ~15);
}

__device__ __forceinline__ void tc_make_item(const AttnTcParams &tp, int idx, TcItem &it)
{
    const AttnParams &ap = tp.a;
    it.prob = idx >= ap.pr[0].n_items ? 1 : 0;
    if (it.prob) idx -= ap.pr[0].n_items;
    const AttnProblem &p = ap.pr[it.prob];
    it.part = idx % p.splits;
    idx /= p.splits;
    int tile, unit;
    const int units = p.batch * ap.Hkv;
    if (p.window > 0) {  // equal work: neighbours share the keys in L2
        unit = idx / p.q_tiles;
        tile = idx - unit * p.q_tiles;
    } else {             // the most work first
        tile = p.q_tiles - 1 - idx / units;
        unit = idx % units;
    }
    it.b = unit / ap.Hkv;
    it.kvh = unit - it.b * ap.Hkv;
    const AttnSeq sq = attn_sequence(p, it.b);
    it.q0 = sq.q0;
    it.k0 = sq.k0;
    it.p0 = sq.p0;
    it.m = sq.m;
    it.bad = sq.bad;
    it.pair = p.pair;
    const int per = kBM / ap.G;
    const int t0 = it.pair ? 0 : 2 * tile * per;
    const int n0 = max(0, min(per, sq.n - t0));
    const int t1 = it.pair ? 0 : t0 + per;
    const int n1 = max(0, min(per, sq.n - t1));
    it.keys = AttnKeys{};
    if (n0 > 0) it.keys = attn_keys(p, sq.m, sq.p0 + t0, sq.p0 + (n1 > 0 ? t1 + n1 : t0 + n0) - 1, kBN);
    it.lo = static_cast<int>(static_cast<long long>(it.keys.count) * it.part / p.splits);
    it.hi = static_cast<int>(static_cast<long long>(it.keys.count) * (it.part + 1) / p.splits);
    for (int s = 0; s < 2; ++s) {
        TcSub &u = it.sub[s];
        u.t0 = s ? t1 : t0;
        u.nt = s ? n1 : n0;
        AttnKeys k = {};
        if (u.nt > 0) k = attn_keys(p, sq.m, sq.p0 + u.t0, sq.p0 + u.t0 + u.nt - 1, kBN);
        u.tiles_sink = k.sink_tiles;
        u.main0 = k.main0;
        u.end = k.main0 + k.count - k.sink_tiles;
        u.count = 0;
        if (it.pair) {
            u.count = (it.hi - it.lo + 1 - s) / 2;
        } else {
            for (int n = it.lo; n < it.hi; ++n) u.count += tc_active(it, n, s) ? 1 : 0;
        }
    }
}

// The i-th item of this CTA: the direction alternates, so that with items in
// the order of their work the CTAs' sums stay close.
__device__ __forceinline__ int tc_item_index(int i)
{
    const int c = blockIdx.x, n = gridDim.x;
    return i * n + ((i & 1) ? n - 1 - c : c);
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) attn_tc_kernel(const __grid_constant__ AttnTcParams tp)
{
    using L = TcLayout<D>;
    const AttnParams &ap = tp.a;
    extern __shared__ uint8_t traw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(traw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::kOffBar);
    uint64_t *q_full = bars;                    // [2] a sub's rows landed
    uint64_t *q_empty = q_full + 2;             // [2] its last Q K^T completed
    uint64_t *s_full = q_empty + 2;             // [2] logits ready
    uint64_t *p_full = s_full + 2;              // [2] probabilities written (four warps)
    uint64_t *o_done = p_full + 2;              // [2] P V completed
    uint64_t *kv_full = o_done + 2;             // [kStages]
    uint64_t *kv_empty = kv_full + L::kStages;  // [kStages]
    uint64_t *i_full = kv_empty + L::kStages;   // [kItemSlots] an item is posted
    uint64_t *i_empty = i_full + kItemSlots;    // [kItemSlots] every role is done with it
    uint64_t *fin = i_empty + kItemSlots;       // the MMA warp's last operation completed
    uint32_t *tslot = reinterpret_cast<uint32_t *>(fin + 1);
    TcItem *items = reinterpret_cast<TcItem *>(sm + L::kOffItem);
    float *xl = reinterpret_cast<float *>(sm + L::kOffX);
    static_assert((10 + 2 * L::kStages + 2 * kItemSlots + 1) * 8 + 4 <= 256, "barrier area");

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // warp-uniform to the compiler
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 4);
            mbar_init(&o_done[s], 1);
        }
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
        }
        for (int s = 0; s < kItemSlots; ++s) {
            mbar_init(&i_full[s], 1);
            mbar_init(&i_empty[s], 2 + 8);  // TMA, MMA, the softmax warps
        }
        mbar_init(fin, 1);
        mbar_fence_init();
    }
    if (warp == kTmaWarp) tmem_alloc(tslot, kTcTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(tslot), 0);
    static_assert(kItemSlots * sizeof(TcItem) <= 240, "item area");
    const int n_items = ap.pr[0].n_items + (ap.n_problems > 1 ? ap.pr[1].n_items : 0);

    // The i-th posted item; null where there is none or the wait ran out.
    auto take = [&](int i, bool &ok) -> const TcItem * {
        if (!mbar_wait(&i_full[i % kItemSlots], (i / kItemSlots) & 1)) {
            ok = false;
            return nullptr;
        }
        const TcItem *it = items + i % kItemSlots;
        return *reinterpret_cast<const volatile int *>(&it->prob) < 0 ? nullptr : it;
    };
    // The register split, by whole warpgroups; the host has checked that the kernel was built for kLaunchRegs.
    if (warp >= kTmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == kSchedWarp) {
            // -------------------------------------------------------- scheduler
            if (lane == 0) {
                for (int i = 0, k = 0;; ++k) {
                    const bool end = k * static_cast<int>(gridDim.x) >= n_items;
                    const int idx = tc_item_index(k);
                    if (!end && idx >= n_items) continue;
                    const int slot = i % kItemSlots;
                    if (i >= kItemSlots && !mbar_wait(&i_empty[slot], ((i / kItemSlots) - 1) & 1)) {
                        attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
                        break;
                    }
                    if (end) items[slot].prob = -1;
                    else tc_make_item(tp, idx, items[slot]);
                    mbar_arrive(&i_full[slot]);
                    if (end) break;
                    ++i;
                }
            }
        } else if (warp == kTmaWarp) {
            // ------------------------------------------------------ TMA producer
            if (lane == 0) {
                bool ok = true;
                int ld = 0;              // ring loads issued (K and V tiles alternate)
                int nq0 = 0, nq1 = 0;    // loads of each sub's rows
                const int per = kBM / ap.G;
                for (int i = 0; ok; ++i) {
                    const TcItem *ip = take(i, ok);
                    if (!ip) break;
                    const TcItem &it = *ip;
                    const AttnTcMaps &mp = tp.maps[it.prob];
                    const int qb = ap.pr[it.prob].q_starts ? 0 : it.b;
                    const int loads = 2 * (it.hi - it.lo);
#pragma unroll 1
                    for (int j = 0; j < loads; ++j) {
                        const int st = ld % L::kStages;
                        if (ld >= L::kStages && !mbar_wait(&kv_empty[st], ((ld / L::kStages) - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        const int tile = attn_tile_at(it.keys, it.lo + (j >> 1));
                        const void *map = (j & 1) ? &mp.v : &mp.k;
                        mbar_arrive_expect_tx(&kv_full[st], L::kTile);
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_4d(sm + L::kOffKV + st * L::kTile + c * 16384, map, c * 64, it.k0 + tile * kBN, it.kvh, qb,
                                        &kv_full[st]);
                        ++ld;
                        if (j != 1) continue;
                        // the rows: after the first K and V, which wait for no item's end
#pragma unroll 1
                        for (int s = 0; s < 2; ++s) {
                            if (it.sub[s].count == 0) continue;
                            const int q = s ? nq1++ : nq0++;
                            if (q > 0 && !mbar_wait(&q_empty[s], (q - 1) & 1)) {
                                ok = false;
                                break;
                            }
                            mbar_arrive_expect_tx(&q_full[s], static_cast<uint32_t>(per * ap.G * 128 * (D / 64)));
#pragma unroll
                            for (int c = 0; c < D / 64; ++c)
                                tma_load_5d(sm + L::kOffQ + s * L::kTile + c * 16384, &mp.q, c * 64, 0, it.q0 + it.sub[s].t0,
                                            it.kvh, qb, &q_full[s]);
                        }
                        if (!ok) break;
                    }
                    if (!ok) break;
                    mbar_arrive(&i_empty[i % kItemSlots]);
                }
                if (!ok) attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
                // every copy has landed before the CTA may end
                for (int n = max(0, ld - L::kStages); n < ld; ++n) mbar_wait(&kv_full[n % L::kStages], (n / L::kStages) & 1);
                if (nq0 > 0) mbar_wait(&q_full[0], (nq0 - 1) & 1);
                if (nq1 > 0) mbar_wait(&q_full[1], (nq1 - 1) & 1);
            }
        } else if (warp == kMmaWarp) {
            // -------------------------------------------------------- MMA issuer
            // The whole warp walks the items with warp-uniform values (the instruction takes its
            // descriptors from uniform registers; issued from one lane of divergent code, each MMA
            // cost about 90 cycles of moves); one elected lane issues.
            constexpr uint32_t idesc_pv = idesc_bf16_f32(kBM, D) | (1u << 16);  // B with N contiguous
            const bool leader = elect_one();
            bool ok = true;
            const uint32_t q_addr = smem_u32(sm + L::kOffQ), kv_addr = smem_u32(sm + L::kOffKV);
            uint32_t st = 0, ph = 0;     // ring stage of the next K tile, and its phase's parity
            uint32_t nq = 0, np = 0;     // bit s: parity of the rows' tiles and of the probabilities taken
            // per sub: the pending P V's ring stage (-1: none) with its phase, and its 16-key steps
            int pv[2] = {-1, -1};
            uint32_t vph[2] = {0, 0};
            int psteps[2] = {0, 0};
            bool pfirst[2] = {false, false};
            auto wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0; };
            auto issue_pv = [&](int s) {
                const int v = pv[s];
                if (!wait(&p_full[s], (np >> s) & 1) || !wait(&kv_full[v], vph[s])) return false;
                np ^= 1u << s;
                tc_fence_after();
                const uint64_t vd = smem_desc_v(kv_addr + v * L::kTile);
                const uint32_t d = tmem + kColO + 128u * s, a = tmem + kColS + 128u * s;
                const bool last_use = pv[1 - s] != v;  // the other sub has no use of this V (any more)
                if (leader) {
                    if (psteps[s] == kBN / 16) {
#pragma unroll
                        for (int kk = 0; kk < kBN / 16; ++kk)
                            tc_mma_ts_bf16(d, a + 8u * kk, vd + kk * (2048 >> 4), idesc_pv, kk > 0 || !pfirst[s]);
                    } else {
                        for (int kk = 0; kk < psteps[s]; ++kk)
                            tc_mma_ts_bf16(d, a + 8u * kk, vd + kk * (2048 >> 4), idesc_pv, kk > 0 || !pfirst[s]);
                    }
                    tc_commit(&o_done[s]);
                    if (last_use) tc_commit(&kv_empty[v]);
                }
                __syncwarp();
                pv[s] = -1;
                return true;
            };
            for (int i = 0;; ++i) {
                const TcItem *ip = take(i, ok);
                if (!__all_sync(0xffffffffu, ip != nullptr)) break;
                // the fields a step needs, in registers
                auto get = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
                const int lo = get(ip->lo), hi = get(ip->hi), pair = get(ip->pair);
                const AttnKeys keys = {get(ip->keys.sink), get(ip->keys.lo), get(ip->keys.hi), get(ip->keys.sink_tiles), get(ip->keys.main0), 0};
                int left[2], sink[2], main0[2], end[2];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    left[s] = get(ip->sub[s].count);
                    sink[s] = get(ip->sub[s].tiles_sink);
                    main0[s] = get(ip->sub[s].main0);
                    end[s] = get(ip->sub[s].end);
                }
                __syncwarp();
                if (leader) mbar_arrive(&i_empty[i % kItemSlots]);
                bool first[2] = {true, true};
#pragma unroll 1
                for (int n = lo; n < hi && ok; ++n) {
                    const int t = n < keys.sink_tiles ? n : keys.main0 + n - keys.sink_tiles;
                    const int nk = tc_keys_in(keys, n < keys.sink_tiles, t);
                    bool act[2];
#pragma unroll
                    for (int s = 0; s < 2; ++s)
                        act[s] = pair ? ((n - lo) & 1) == s : t < sink[s] || (t >= main0[s] && t < end[s]);
                    const uint32_t vs = st + 1 == L::kStages ? 0 : st + 1;  // V follows K in the ring
                    const uint32_t vp = st + 1 == L::kStages ? ph ^ 1 : ph;
                    ok = wait(&kv_full[st], ph);
                    // first the subs that see the tile: the pending P V of each, then its Q K^T (S is
                    // overwritten behind the P V that reads P from it, in issue order)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (!ok || !act[s]) continue;
                        if (pv[s] >= 0) ok = issue_pv(s);
                        if (ok && first[s]) {
                            ok = wait(&q_full[s], (nq >> s) & 1);
                            nq ^= 1u << s;
                        }
                        if (!ok) continue;
                        tc_fence_after();
                        const uint32_t idesc = idesc_bf16_f32(kBM, nk);
                        const uint64_t qd = smem_desc_sw128(q_addr + s * L::kTile), kd = smem_desc_sw128(kv_addr + st * L::kTile);
                        --left[s];
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t koff = static_cast<uint32_t>((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                                tc_mma_bf16(tmem + kColS + 128u * s, qd + koff, kd + koff, idesc, kk > 0);
                            }
                            tc_commit(&s_full[s]);
                            if (left[s] == 0) tc_commit(&q_empty[s]);
                        }
                        __syncwarp();
                        pv[s] = static_cast<int>(vs);
                        vph[s] = vp;
                        psteps[s] = nk / 16;
                        pfirst[s] = first[s];
                        first[s] = false;
                    }
                    if (ok && leader) tc_commit(&kv_empty[st]);  // K of this tile has been used
                    __syncwarp();
                    // then the pending P V of those that do not see it
#pragma unroll
                    for (int s = 0; s < 2; ++s)
                        if (ok && !act[s] && pv[s] >= 0) ok = issue_pv(s);
                    st = vs + 1 == L::kStages ? 0 : vs + 1;
                    ph = vs + 1 == L::kStages ? vp ^ 1 : vp;
                }
                // an item without tiles pushes nothing out: what is pending goes now, or the softmax
                // warps, and behind them the scheduler, would wait for it
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (ok && lo == hi && pv[s] >= 0) ok = issue_pv(s);
                if (!ok) break;
            }
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (ok && pv[s] >= 0) ok = issue_pv(s);
            if (leader) {
                if (!ok) attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
                tc_commit(fin);
                mbar_wait(fin, 0);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------ softmax and output
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int s = warp >> 2, quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t tS = tmem + kColS + 128u * s + lanes, tO = tmem + kColO + 128u * s + lanes;
        const float c = ap.scale_log2;
        const int G = ap.G;
        bool ok = true;
        int ld = 0, nt = 0;  // ring loads before this item; tiles of this sub so far
        for (int i = 0;; ++i) {
            bool got = true;
            const TcItem *ip = take(i, got);
            // all 256 threads leave together: they meet at barriers inside
            const int votes = named_bar_count(2, 2 * kSubThreads, ip != nullptr);
            if (votes < 2 * kSubThreads) {
                if ((votes > 0 || !got) && lane == 0) attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
                break;
            }
            const TcItem &it = *ip;
            const AttnProblem &p = ap.pr[it.prob];
            const TcSub u = it.sub[s];
            if (it.bad && tid == 0) attn_flag(ap.err, KVEVICT_DEV_BAD_LENGTH);
            const int nrows = u.nt * G;
            const bool live = quad * 32 < nrows;  // this warp has rows
            // the positions this row sees: j <= top, and j < n_sink or j >= low
            const int pos = p.causal ? it.p0 + u.t0 + min(row, nrows - 1) / G : it.m - 1;
            const int top = pos;
            const int low = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
            // of all the sub's rows: the least top, the greatest low
            const int top_min = p.causal ? it.p0 + u.t0 : it.m - 1;
            const int pos_max = p.causal ? it.p0 + u.t0 + u.nt - 1 : it.m - 1;
            const int low_max = p.window > 0 && pos_max >= p.window ? pos_max - p.window + 1 : 0;
            float m = -INFINITY, l = 0.f;
            int done = 0;  // tiles of this item
            for (int n = it.lo; n < it.hi; ++n) {
                if (!tc_active(it, n, s)) continue;
                if (ok && !__all_sync(0xffffffffu, mbar_wait(&s_full[s], nt & 1))) {
                    ok = false;
                    if (lane == 0) attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
                }
                tc_fence_after();
                const int j0 = attn_tile_at(it.keys, n) * kBN;
                const int keys = tc_keys_in(it.keys, n < it.keys.sink_tiles, j0 / kBN);
                if (ok && live) {
                    const bool masked = j0 + kBN - 1 > top_min || (j0 < low_max && j0 + kBN > p.n_sink);
                    uint32_t r[4][32];
                    const bool small = keys <= 32;
                    tmem_ld32(tS, r[0]);
                    if (!small) {
                        tmem_ld32(tS + 32, r[1]);
                        tmem_ld32(tS + 64, r[2]);
                        tmem_ld32(tS + 96, r[3]);
                    }
                    tc_wait_ld();
                    float mx;
                    if (small) {
                        if (masked) tc_mask32(r[0], top - j0, low - j0, p.n_sink - j0);
                        mx = tc_max32(r[0]);
                    } else {
                        if (masked) {
#pragma unroll
                            for (int g = 0; g < 4; ++g)
                                tc_mask32(r[g], top - j0 - 32 * g, low - j0 - 32 * g, p.n_sink - j0 - 32 * g);
                        }
                        mx = fmaxf(fmaxf(tc_max32(r[0]), tc_max32(r[1])), fmaxf(tc_max32(r[2]), tc_max32(r[3])));
                    }
                    mx *= c;
                    // rescale where the maximum outgrew the one in use (a first finite one included)
                    const bool grow = mx > m + kRescale || (m == -INFINITY && mx != -INFINITY);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float mn = grow ? mx : m;
                        const float f = m == -INFINITY ? 0.f : ex2(m - mn);
                        m = mn;
                        l *= f;
                        if (done > 0) {
                            // O holds tiles before this one: wait for the last of them, then scale it
                            if (!__all_sync(0xffffffffu, mbar_wait(&o_done[s], (nt - 1) & 1))) {
                                ok = false;
                                if (lane == 0) attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
                            } else {
                                tc_fence_after();
#pragma unroll
                                for (int q = 0; q < D; q += 32) {
                                    uint32_t o[32];
                                    tmem_ld32(tO + q, o);
                                    tc_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                    tmem_st32(tO + q, o);
                                }
                            }
                        }
                    }
                    const float ms = m == -INFINITY ? 0.f : m;
                    const float2 c2 = make_float2(c, c), nm2 = make_float2(-ms, -ms);
                    float2 sum[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) sum[g] = make_float2(0.f, 0.f);
                    uint32_t pk[32];  // 64 probabilities
                    tc_exp32(r[0], c2, nm2, sum, pk);
                    if (!small) {
                        tc_exp32(r[1], c2, nm2, sum, pk + 16);
                        tmem_st32(tS, pk);
                        tc_exp32(r[2], c2, nm2, sum, pk);
                        tc_exp32(r[3], c2, nm2, sum, pk + 16);
                        tmem_st32(tS + 32, pk);
                    } else {
#pragma unroll
                        for (int e = 16; e < 32; ++e) pk[e] = 0u;
                        tmem_st32(tS, pk);
                    }
                    const float2 t = fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3]));
                    l += t.x + t.y;
                    tc_wait_st();
                }
                // V rows that no row of the item sees may hold anything: 0 times that must be 0
                const bool edge = j0 + keys > it.keys.hi || (j0 < it.keys.lo && j0 + keys > it.keys.sink);
                if (edge) {
                    const int v = ld + 2 * (n - it.lo) + 1, st = v % L::kStages;
                    if (ok && !__all_sync(0xffffffffu, mbar_wait(&kv_full[st], (v / L::kStages) & 1))) {
                        ok = false;
                        if (lane == 0) attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
                    }
                    const int j = j0 + row;
                    if (ok && row < keys && !(j < it.keys.sink || (j >= it.keys.lo && j < it.keys.hi))) {
                        uint4 *z = reinterpret_cast<uint4 *>(sm + L::kOffKV + st * L::kTile + row * 128);
#pragma unroll
                        for (int e = 0; e < D / 64; ++e)
#pragma unroll
                            for (int w = 0; w < 8; ++w) z[e * 1024 + w] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[s]);
                ++nt;
                ++done;
            }
            ld += 2 * (it.hi - it.lo);

            // -------------------------------------------------------- output
            if (done > 0 && ok && !__all_sync(0xffffffffu, mbar_wait(&o_done[s], (nt - 1) & 1))) {
                ok = false;
                if (lane == 0) attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
            }
            tc_fence_after();
            const int t = it.q0 + u.t0 + row / G, h = it.kvh * G + row % G;
            const long long at = it.b * p.rs[0] + h * p.rs[1] + t * p.rs[2];
            float f0 = l > 0.f ? 1.f / l : l, f1 = 0.f;  // factors on this sub's O and the other's
            float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
            int col0 = 0, cols = D;
            uint32_t tO1 = tO;
            if (it.pair) {
                // both subs hold the same rows: each scales its own O to a normalised one, by
                // weights from the normalisers (shared memory), and writes half of the columns of
                // the sum; the other's O is read through TMEM (the two warpgroups' warps address
                // the same lanes), its factor 1 / l with the weight (shared memory again)
                xl[s * kBM + row] = lse2;
                named_bar_sync(1, 2 * kSubThreads);
                const float other = xl[(1 - s) * kBM + row];
                const float mt = fmaxf(lse2, other), mm = mt == -INFINITY ? 0.f : mt;
                const float w = ex2(lse2 - mm), total = w + ex2(other - mm);
                lse2 = total == 0.f ? -INFINITY : mt + log2f(total);
                f0 = l == 0.f ? 0.f : f0 * (w / total);
                named_bar_sync(1, 2 * kSubThreads);
                xl[s * kBM + row] = f0;
                tc_fence_before();
                named_bar_sync(1, 2 * kSubThreads);
                tc_fence_after();
                f1 = xl[(1 - s) * kBM + row];
                cols = D / 2;
                col0 = s * cols;
                tO1 = tmem + kColO + 128u * (1 - s) + lanes;
            }
            if (ok && live) {
                const bool split = ap.slots > 1;
                const long long slot = (p.slot0 + it.part) * ap.rows + at;
                float *po = split ? ap.part_o + slot * D : nullptr;
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(ap.out) + it.b * p.os[0] + h * p.os[1] + t * p.os[2];
                const bool any0 = f0 != 0.f, any1 = f1 != 0.f;
                for (int q = col0; q < col0 + cols; q += 32) {
                    uint32_t o[32];
                    float v[32];
                    tmem_ld32(tO + q, o);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = any0 ? __uint_as_float(o[e]) * f0 : 0.f;
                    if (it.pair) {
                        tmem_ld32(tO1 + q, o);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] += any1 ? __uint_as_float(o[e]) * f1 : 0.f;
                    }
                    if (row < nrows) {
                        if (split) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                *reinterpret_cast<float4 *>(po + q + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                *reinterpret_cast<uint4 *>(out + q + e) =
                                    make_uint4(pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]),
                                               pack_bf16x2(v[e + 4], v[e + 5]), pack_bf16x2(v[e + 6], v[e + 7]));
                        }
                    }
                }
                if (row < nrows && col0 == 0) {
                    if (split) ap.part_l[slot] = lse2;
                    else if (ap.lse) ap.lse[at] = lse2 * kLn2;
                }
            }
            tc_fence_before();
            if (it.pair) named_bar_sync(1, 2 * kSubThreads);  // the other's O and factors have been read
            __syncwarp();
            if (lane == 0) mbar_arrive(&i_empty[i % kItemSlots]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kTmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTcTmemCols);
    }
}

template <int D> cudaError_t launch_tc(const AttnTcParams &p, int sms, cudaStream_t st)
{
    constexpr int bytes = TcLayout<D>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    static const int regs = [] {
        cudaFuncAttributes at{};
        return cudaFuncGetAttributes(&at, attn_tc_kernel<D>) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs != kLaunchRegs) return cudaErrorInvalidKernelImage;  // the split would wait for registers that are not there
    const int n = p.a.pr[0].n_items + (p.a.n_problems > 1 ? p.a.pr[1].n_items : 0);
    attn_tc_kernel<D><<<n < sms ? n : sms, kTcThreads, bytes, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tc(const AttnTcParams &p, int head_dim, int sms, cudaStream_t st)
{
    return head_dim == 64 ? launch_tc<64>(p, sms, st) : launch_tc<128>(p, sms, st);
}

}  // namespace kvevict
