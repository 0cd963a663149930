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
// A CTA holds two row tiles of 128 rows ("subs"), each with its own S/P and O in
// TMEM (S0 S1 O0 O1: all 512 columns; P overwrites the first half of S) and its
// own softmax warpgroup, a row a thread: while one sub's rows go through the
// softmax the tensor cores work for the other. A K or V tile of 128 keys is
// loaded once for both subs (TMA ring). Where a unit's rows fit one sub ("pair":
// decoding, short chunks), both hold the same rows and take alternate key tiles,
// each a part of its own to the join. Rows are (token, group head) pairs, so all
// query heads of a KV head share its tiles.
//
// The grid has a block for every item (window_attn.h), longest first; a block
// that runs takes over others that have not started, one when the loads of the
// item before begin, so that loads, products, softmax and output of neighbouring
// items overlap and the SMs end together.
//
// Warps 0-3, 4-7: softmax of sub 0, 1; 8-11: output; 12: TMA; 13: the items;
// 14, 15: MMA issue of sub 0, 1. Output has warps of its own because the
// softmax warps, writing it themselves, left the tensor cores idle for 10,000
// cycles an item.
//
// What bounds it: prompts, the chain logits - softmax - P V - next logits of a
// sub (about 3,300 cycles a tile of 128 x 128 for both subs, 2,048 of them MMAs;
// shared memory is read by Q K^T at its full rate meanwhile); decoding, bytes and
// the start and end of items. Causal prompt of 8192, 32 query heads over 8, d
// 128: 396 us, 1,390 TFLOP/s (72% of the cuBLAS rate; 412 us a call, one after
// another); 2 x 32 heads x 4096, 4 sinks and a window of 1021: 150 us; a token of
// 32 sequences over 2,048 keys, 64 query heads over 8: 63 us, 4.2 TB/s with the
// join.
#include <atomic>
#include <climits>
#include <cmath>

#include "launch.h"
#include "tc5_common.cuh"
#include "window_attn.h"
#include "window_attn_common.cuh"

namespace kvevict {

namespace {

constexpr int kBM = kAttnTcRows, kBN = kAttnTcKeys;
constexpr int kSoftmaxWarps = 8;  // then four output warps
constexpr int kTmaWarp = 12, kSchedWarp = 13, kMmaWarp = 14;  // and 15
constexpr int kTcThreads = 512;
// Registers a thread: the launch's 128 (65,536 over 512 threads), moved to the
// two softmax warpgroups, whose threads hold a whole row of 128 logits:
// 2 x 160 + 120 + 72 = 4 x 128.
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 160, kOutRegs = 120, kIssueRegs = 72;
static_assert(2 * kSoftmaxRegs + kOutRegs + kIssueRegs <= 4 * kLaunchRegs, "register split");
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
    static constexpr int kOffX = kOffBar + 384;            // [2 subs][2][128 rows]: log2 normalisers, 1 / l
    static constexpr int kOffItem = kOffX + 4 * kBM * 4;   // posted items
    static constexpr int kOffStep = kOffItem + 544;        // the two subs' steps; a cancelled block's index
    static constexpr int kBytes = kOffStep + 32;
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

// Cluster launch control: asks the hardware for one of the grid's blocks that
// has not started; 16 bytes arrive at `slot`, completing on `bar`.
__device__ __forceinline__ void steal_request(void *slot, uint64_t *bar)
{
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(slot)),
                 "r"(smem_u32(bar))
                 : "memory");
}

// The block that was taken over, or -1: none was left.
__device__ __forceinline__ int steal_result(const void *slot)
{
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\tld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, h;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(smem_u32(slot))
        : "memory");
    return got ? static_cast<int>(x) : -1;
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

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
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
    if (__all_sync(0xffffffffu, seen == 0xffffffffu)) return;  // most chunks of a border tile
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

// Writes 64 bytes of every lane's row. Lane by lane that would be 32 lines an
// instruction, 16 bytes of each; the four lanes of a quad exchange their 16-byte
// pieces (a 4 x 4 transpose in two rounds), so that each store covers 64 bytes
// of eight rows. dst: the quad's four rows, + the lane's piece; null: no row.
struct TcWords {
    uint4 a, b, c, d;
};
__device__ __forceinline__ TcWords tc_words(const uint32_t *w)
{
    return TcWords{make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]), make_uint4(w[8], w[9], w[10], w[11]),
                   make_uint4(w[12], w[13], w[14], w[15])};
}
__device__ __forceinline__ void tc_store_rows(const TcWords &w, uint4 *const (&dst)[4], int at)
{
    const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
    auto swap = [](uint4 &a, uint4 &b, bool up, int mask) {  // a of the upper lane for b of the lower
        const uint4 out = up ? a : b;
        uint4 in;
        in.x = __shfl_xor_sync(0xffffffffu, out.x, mask);
        in.y = __shfl_xor_sync(0xffffffffu, out.y, mask);
        in.z = __shfl_xor_sync(0xffffffffu, out.z, mask);
        in.w = __shfl_xor_sync(0xffffffffu, out.w, mask);
        if (up) a = in;
        else b = in;
    };
    uint4 a = w.a, b = w.b, c = w.c, d = w.d;
    swap(a, b, odd, 1);
    swap(c, d, odd, 1);
    swap(a, c, high, 2);
    swap(b, d, high, 2);
    if (dst[0]) dst[0][at] = a;
    if (dst[1]) dst[1][at] = b;
    if (dst[2]) dst[2][at] = c;
    if (dst[3]) dst[3][at] = d;
}

// One sub of an item: its tokens, the key tiles they see, how many of them
// are in this part.
struct TcSub {
    int t0, nt;
    int tiles_sink, main0, end;
    int count;
    int top_min, low_max;  // of its rows: the least last key seen, the greatest first one of the window
};

// What a softmax warp has to know about the tile whose logits are ready.
struct TcStep {
    int j0;            // first key
    int what;          // keys to work on | kStepMask | kStepEdge | V's ring stage << 16 | its parity << 24
};
constexpr int kStepMask = 256, kStepEdge = 512;

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
constexpr int kItemSlots = 4;
constexpr int kMaxSkipped = 4096;  // empty items in a row that are not posted

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

// `sound`: a packed batch's sequences before the first one that falls.
__device__ __forceinline__ void tc_make_item(const AttnTcParams &tp, int idx, int sound, TcItem &it)
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
    const AttnSeq sq = attn_sequence(p, it.b, it.b < sound);
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
        const int pa = p.causal ? sq.p0 + u.t0 : sq.m - 1, pb = p.causal ? pa + u.nt - 1 : sq.m - 1;
        u.top_min = pa;
        u.low_max = p.window > 0 ? max(0, pb - p.window + 1) : 0;
        AttnKeys k = {};
        if (u.nt > 0) k = attn_keys(p, sq.m, sq.p0 + u.t0, sq.p0 + u.t0 + u.nt - 1, kBN);
        u.tiles_sink = k.sink_tiles;
        u.main0 = k.main0;
        u.end = k.main0 + k.count - k.sink_tiles;
        u.count = 0;
        if (it.pair) {
            u.count = (it.hi - it.lo + 1 - s) / 2;
        } else {
            if (p.splits == 1) u.count = k.count;
            else
                for (int n = it.lo; n < it.hi; ++n) u.count += tc_active(it, n, s) ? 1 : 0;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) attn_tc_kernel(const __grid_constant__ AttnTcParams tp)
{
    using L = TcLayout<D>;
    const AttnParams &ap = tp.a;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::kOffBar);
    uint64_t *q_full = bars;                    // [2] a sub's rows landed
    uint64_t *q_empty = q_full + 2;             // [2] its last Q K^T completed
    uint64_t *s_full = q_empty + 2;             // [2] logits ready
    uint64_t *p_full = s_full + 2;              // [2] probabilities written (four warps)
    uint64_t *o_done = p_full + 2;              // [2] P V completed
    uint64_t *kv_full = o_done + 2;             // [kStages]
    uint64_t *kv_empty = kv_full + L::kStages;  // [kStages]
    uint64_t *l_ready = kv_empty + L::kStages;  // [2] a sub's sums of the item are in shared memory
    uint64_t *l_free = l_ready + 2;             // [2] and have been read there
    uint64_t *o_free = l_free + 2;              // [2] its O has been read (a phase an item with tiles of the sub)
    uint64_t *i_full = o_free + 2;              // [kItemSlots] an item is posted
    uint64_t *i_empty = i_full + kItemSlots;    // [kItemSlots] every role is done with it
    uint64_t *fin = i_empty + kItemSlots;       // [2] an MMA warp's last operation completed
    uint64_t *taken = fin + 2;                  // the TMA warp has taken up an item
    uint64_t *stolen = taken + 1;               // the answer about another block is there
    uint32_t *tslot = reinterpret_cast<uint32_t *>(stolen + 1);
    TcItem *items = reinterpret_cast<TcItem *>(sm + L::kOffItem);
    TcStep *steps = reinterpret_cast<TcStep *>(sm + L::kOffStep);  // [2]
    uint8_t *steal_slot = sm + L::kOffStep + 16;
    float *xl = reinterpret_cast<float *>(sm + L::kOffX);
    static_assert((18 + 2 * L::kStages + 2 * kItemSlots + 2) * 8 + 4 <= 384, "barrier area");
    static_assert(kItemSlots * sizeof(TcItem) <= 544 && L::kOffStep % 16 == 0, "item area");

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // warp-uniform to the compiler
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
            mbar_init(&s_full[s], 2);  // the step is posted; its logits are complete
            mbar_init(&p_full[s], 4);
            mbar_init(&o_done[s], 1);
            mbar_init(&l_ready[s], 4);
            mbar_init(&l_free[s], 4);
            mbar_init(&o_free[s], 4);
            mbar_init(&fin[s], 1);
        }
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 2);
        }
        for (int s = 0; s < kItemSlots; ++s) {
            mbar_init(&i_full[s], 1);
            mbar_init(&i_empty[s], 3 + kSoftmaxWarps + 4);  // TMA, MMA, softmax, output warps
        }
        mbar_init(taken, 1);
        mbar_init(stolen, 1);
        mbar_fence_init();
    }
    if (warp == kTmaWarp) tmem_alloc(tslot, kTcTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(tslot), 0);
    grid_dependency_wait();
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
            // The grid has a block for every item, in the order of tc_make_item; a block that runs
            // takes over one after another of those that have not started.
            const int sound = ap.pr[0].q_starts ? attn_first_fall(ap.pr[0], ap.pr[0].batch - 1, lane) : INT_MAX;
            if (lane == 0) {
                int idx = blockIdx.x;
                uint32_t asked = 0;
                auto next = [&]() {
                    mbar_arrive_expect_tx(stolen, 16);
                    steal_request(steal_slot, stolen);
                    if (!mbar_wait(stolen, asked++ & 1)) {
                        attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
                        return -1;
                    }
                    const int x = steal_result(steal_slot);
                    fence_proxy_async_smem();  // read before the next answer is written
                    return x;
                };
                for (int i = 0;; ++i) {
                    const int slot = i % kItemSlots;
                    // a block is taken over when the loads of the item before it begin: what waits here
                    // could be running elsewhere
                    if ((i >= kItemSlots && !mbar_wait(&i_empty[slot], ((i / kItemSlots) - 1) & 1)) ||
                        (i > 0 && !mbar_wait(taken, (i - 1) & 1))) {
                        // a role gave up: the blocks that have not started are taken and dropped, so that
                        // the launch ends with the ones that run
                        attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
                        while (idx >= 0) idx = next();
                        break;
                    }
                    if (i > 0) idx = next();
                    // (an item whose rows lie behind its sequence's last has nothing to do; at 1.25 us each,
                    // one of kMaxSkipped goes to the other warps all the same, before their waits run out)
                    for (int skipped = 0; idx >= 0; ++skipped) {
                        tc_make_item(tp, idx, sound, items[slot]);
                        if (items[slot].bad) attn_flag(ap.err, KVEVICT_DEV_BAD_LENGTH);
                        if (items[slot].sub[0].nt > 0 || skipped >= kMaxSkipped) break;
                        idx = next();
                    }
                    if (idx < 0) items[slot].prob = -1;
                    mbar_arrive(&i_full[slot]);
                    if (idx < 0) break;
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
                    mbar_arrive(taken);
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
        } else {
            // ------------------------------------------- MMA issue, a warp a sub
            // A sub's products follow one another through its P and S; two warps, because a warp's
            // waits and the issue itself take as long as its MMAs run: meanwhile the other sub's run.
            // The whole warp walks the items with warp-uniform values (the instruction takes its
            // descriptors from uniform registers; issued from one lane of divergent code, each MMA
            // cost about 90 cycles of moves); one elected lane issues.
            constexpr uint32_t idesc_pv = idesc_bf16_f32(kBM, D) | (1u << 16);  // B with N contiguous
            const int s = warp == kMmaWarp ? 0 : 1;
            const bool leader = elect_one();
            bool ok = true;
            const uint32_t q_addr = smem_u32(sm + L::kOffQ + s * L::kTile), kv_addr = smem_u32(sm + L::kOffKV);
            const uint32_t tS = tmem + kColS + 128u * s, tO = tmem + kColO + 128u * s;
            uint32_t st = 0, ph = 0;     // ring stage of the next K tile, and its phase's parity
            uint32_t nq = 0, np = 0;     // parities of the rows' tiles and of the probabilities taken
            int pv = -1;                 // ring stage of the pending P V's tile (-1: none), with
            uint32_t vph = 0;            // its phase's parity,
            int psteps = 0;              // its steps of 16 keys,
            bool pfirst = false;         // and whether it starts the sum
            uint32_t sums = 0;           // items with tiles of this sub before the pending one's
            auto wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0; };
            auto issue_pv = [&]() {
                if (!wait(&kv_full[pv], vph) || !wait(&p_full[s], np)) return false;
                // a sum starts over O once the one before has been read
                if (pfirst && sums++ > 0 && !wait(&o_free[s], sums & 1)) return false;
                np ^= 1;
                tc_fence_after();
                const uint64_t vd = smem_desc_v(kv_addr + pv * L::kTile);
                if (leader) {
                    if (psteps == kBN / 16) {
#pragma unroll
                        for (int kk = 0; kk < kBN / 16; ++kk)
                            tc_mma_ts_bf16(tO, tS + 8u * kk, vd + kk * (2048 >> 4), idesc_pv, kk > 0 || !pfirst);
                    } else {
                        for (int kk = 0; kk < psteps; ++kk)
                            tc_mma_ts_bf16(tO, tS + 8u * kk, vd + kk * (2048 >> 4), idesc_pv, kk > 0 || !pfirst);
                    }
                    tc_commit(&o_done[s]);
                    tc_commit(&kv_empty[pv]);
                }
                __syncwarp();
                pv = -1;
                return true;
            };
            for (int i = 0;; ++i) {
                const TcItem *ip = take(i, ok);
                if (!__all_sync(0xffffffffu, ip != nullptr)) break;
                // the fields a step needs, in registers
                auto get = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
                const int lo = get(ip->lo), hi = get(ip->hi), pair = get(ip->pair);
                const AttnKeys keys = {get(ip->keys.sink), get(ip->keys.lo), get(ip->keys.hi), get(ip->keys.sink_tiles), get(ip->keys.main0), 0};
                const int n_sink = ap.pr[get(ip->prob)].n_sink;
                const TcSub &sub = ip->sub[s];
                int left = get(sub.count);
                const int sink = get(sub.tiles_sink), main0 = get(sub.main0), end = get(sub.end);
                const int top_min = get(sub.top_min), low_max = get(sub.low_max);
                __syncwarp();
                if (leader) mbar_arrive(&i_empty[i % kItemSlots]);
                bool first = true;
#pragma unroll 1
                for (int n = lo; n < hi && ok; ++n) {
                    const int t = n < keys.sink_tiles ? n : keys.main0 + n - keys.sink_tiles;
                    const uint32_t ks = st, kp = ph;
                    const uint32_t vs = ks + 1 == L::kStages ? 0 : ks + 1;  // V follows K in the ring
                    const uint32_t vp = ks + 1 == L::kStages ? kp ^ 1 : kp;
                    st = vs + 1 == L::kStages ? 0 : vs + 1;
                    ph = vs + 1 == L::kStages ? vp ^ 1 : vp;
                    if (pair ? ((n - lo) & 1) != s : !(t < sink || (t >= main0 && t < end))) {
                        // not this sub's: what is pending goes, and the tile is given up (once it is
                        // there: a phase of kv_empty takes one arrival of each sub)
                        if (pv >= 0) ok = issue_pv();
                        ok = ok && wait(&kv_full[ks], kp);
                        if (ok && leader) mbar_arrive(&kv_empty[ks]);
                        ok = ok && wait(&kv_full[vs], vp);
                        if (ok && leader) mbar_arrive(&kv_empty[vs]);
                        __syncwarp();
                        continue;
                    }
                    const int j0 = t * kBN, nk = tc_keys_in(keys, n < keys.sink_tiles, t);
                    const bool edge = j0 + nk > keys.hi || (j0 < keys.lo && j0 + nk > keys.sink);
                    const bool mask = j0 + kBN - 1 > top_min || (j0 < low_max && j0 + kBN > n_sink);
                    const TcStep step = {j0, nk | (mask ? kStepMask : 0) | (edge ? kStepEdge : 0) | static_cast<int>(vs << 16 | vp << 24)};
                    const uint32_t idesc = idesc_bf16_f32(kBM, nk);
                    const uint64_t qd = smem_desc_sw128(q_addr), kd = smem_desc_sw128(kv_addr + ks * L::kTile);
                    ok = wait(&kv_full[ks], kp);
                    if (ok && first) {
                        ok = wait(&q_full[s], nq);
                        nq ^= 1;
                    }
                    // the pending P V, then Q K^T: S is overwritten behind the P V that reads P from it, in issue order
                    if (ok && pv >= 0) ok = issue_pv();
                    if (!ok) break;
                    tc_fence_after();
                    --left;
                    if (leader) {
                        steps[s] = step;  // the softmax warps are done with the last one: they have written its P
                        mbar_arrive(&s_full[s]);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t koff = static_cast<uint32_t>((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                            tc_mma_bf16(tS, qd + koff, kd + koff, idesc, kk > 0);
                        }
                        tc_commit(&s_full[s]);
                        tc_commit(&kv_empty[ks]);
                        if (left == 0) tc_commit(&q_empty[s]);
                    }
                    __syncwarp();
                    pv = static_cast<int>(vs);
                    vph = vp;
                    psteps = nk / 16;
                    pfirst = first;
                    first = false;
                }
                // an item without tiles pushes nothing out: what is pending goes now, or the softmax
                // warps, and behind them the scheduler, would wait for it
                if (ok && lo == hi && pv >= 0) ok = issue_pv();
                if (!ok) break;
            }
            if (ok && pv >= 0) ok = issue_pv();
            if (leader) {
                if (!ok) attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
                tc_commit(&fin[s]);
                mbar_wait(&fin[s], 0);
            }
            __syncwarp();
        }
    } else if (warp < kSoftmaxWarps) {
        // ----------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int s = warp >> 2, quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t tS = tmem + kColS + 128u * s + lanes, tO = tmem + kColO + 128u * s + lanes;
        const float c = ap.scale_log2;
        bool ok = true;
        uint32_t nt = 0;          // parity of this sub's next tile
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok && !__all_sync(0xffffffffu, mbar_wait(bar, parity))) {
                ok = false;
                if (lane == 0) attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
            }
        };
        for (int i = 0; ok; ++i) {
            bool got = true;
            const TcItem *ip = take(i, got);
            if (!__all_sync(0xffffffffu, ip != nullptr)) {
                if (!got && lane == 0) attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
                break;
            }
            const TcItem &it = *ip;
            const AttnProblem &p = ap.pr[it.prob];
            const int n_sink = p.n_sink;
            // the keys this row sees: j <= top, and j < n_sink or j >= low
            int top = it.m - 1, low = 0;
            const int nrows = it.sub[s].nt * ap.G;
            if (p.causal) {
                top = it.sub[s].top_min + min(row, nrows - 1) / ap.G;
                if (p.window > 0) low = max(0, top - p.window + 1);
            }
            const bool live = quad * 32 < nrows;  // this warp has rows
            float m = -INFINITY, l = 0.f;
            const int count = it.sub[s].count;
#pragma unroll 1
            for (int k = 0; k < count; ++k) {
                wait(&s_full[s], nt);
                tc_fence_after();
                const TcStep step = steps[s];
                if (ok && live) {
                    const bool small = (step.what & 255) <= 32;
                    uint32_t r[4][32];
                    tmem_ld32(tS, r[0]);
                    if (!small) {
#pragma unroll
                        for (int g = 1; g < 4; ++g) tmem_ld32(tS + 32u * g, r[g]);
                    }
                    tc_wait_ld();
                    if (step.what & kStepMask) {
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            tc_mask32(r[g], top - step.j0 - 32 * g, low - step.j0 - 32 * g, n_sink - step.j0 - 32 * g);
                    }
                    float mx = tc_max32(r[0]);
                    if (!small) mx = fmaxf(fmaxf(mx, tc_max32(r[1])), fmaxf(tc_max32(r[2]), tc_max32(r[3])));
                    mx *= c;
                    // rescale where the maximum outgrew the one in use (a first finite one included)
                    const bool grow = mx > m + kRescale || (m == -INFINITY && mx != -INFINITY);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float mn = grow ? mx : m;
                        const float f = m == -INFINITY ? 0.f : ex2(m - mn);
                        m = mn;
                        l *= f;
                        if (k > 0) {
                            // O holds tiles before this one: wait for the last of them, then scale it
                            wait(&o_done[s], nt ^ 1);
                            if (ok) {
                                tc_fence_after();
#pragma unroll 1
                                for (int q = 0; q < D; q += 16) {
                                    uint32_t o[16];
                                    tmem_ld16(tO + q, o);
                                    tc_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                    tmem_st16(tO + q, o);
                                }
                            }
                        }
                    }
                    const float ms = m == -INFINITY ? 0.f : m;
                    const float2 c2 = make_float2(c, c), nm2 = make_float2(-ms, -ms);
                    float2 sum[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) sum[g] = make_float2(0.f, 0.f);
                    if (small) {
                        uint32_t pk[16];
                        tc_exp32(r[0], c2, nm2, sum, pk);
                        tmem_st16(tS, pk);
                    } else {
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            uint32_t pk[16];  // 32 probabilities
                            tc_exp32(r[g], c2, nm2, sum, pk);
                            tmem_st16(tS + 16u * g, pk);
                        }
                    }
                    const float2 t2 = fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3]));
                    l += t2.x + t2.y;
                    tc_wait_st();
                }
                if (step.what & kStepEdge) {
                    // V rows that no row of the item sees may hold anything: 0 times that must be 0
                    const int vs = (step.what >> 16) & 255;
                    wait(&kv_full[vs], step.what >> 24);
                    const int j = step.j0 + row;
                    if (ok && row < (step.what & 255) && !(j < it.keys.sink || (j >= it.keys.lo && j < it.keys.hi))) {
#pragma unroll
                        for (int x = 0; x < D / 64; ++x) {
                            uint4 *z = reinterpret_cast<uint4 *>(sm + L::kOffKV + vs * L::kTile + x * 16384 + row * 128);
#pragma unroll
                            for (int w = 0; w < 8; ++w) z[w] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[s]);
                nt ^= 1;
            }
            // the row's sum, for the output warps: they have read the last item's
            if (i > 0) wait(&l_free[s], (i - 1) & 1);
            xl[(s * 2) * kBM + row] = l == 0.f ? -INFINITY : m + log2f(l);
            xl[(s * 2 + 1) * kBM + row] = l > 0.f ? 1.f / l : l;
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&l_ready[s]);
                mbar_arrive(&i_empty[i % kItemSlots]);
            }
        }
    } else {
        // ------------------------------------------------------------ output
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOutRegs));
        const int quad = warp & 3;
        const int row = quad * 32 + lane;
        const uint32_t tO = tmem + kColO + (static_cast<uint32_t>(quad * 32) << 16);
        bool ok = true;
        uint32_t tiles = 0;  // bit s: parity of the sub's tiles so far
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok && !__all_sync(0xffffffffu, mbar_wait(bar, parity))) {
                ok = false;
                if (lane == 0) attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
            }
        };
        for (int i = 0; ok; ++i) {
            bool got = true;
            const TcItem *ip = take(i, got);
            if (!__all_sync(0xffffffffu, ip != nullptr)) {
                if (!got && lane == 0) attn_flag(ap.err, KVEVICT_DEV_WAIT_TIMEOUT);
                break;
            }
            const TcItem &it = *ip;
            const AttnProblem &p = ap.pr[it.prob];
            const bool pair = it.pair != 0, split = ap.slots > 1;
#pragma unroll 1
            for (int s = 0; s < 2; ++s) {
                // the sub's sums are there, and its last P V (the one before it was complete when the
                // softmax warps read their last logits, so the parity is not a phase behind)
                wait(&l_ready[s], i & 1);
                const int count = it.sub[s].count, nrows = it.sub[s].nt * ap.G;
                const float lse2 = xl[s * 2 * kBM + row], f = xl[(s * 2 + 1) * kBM + row];
                __syncwarp();
                if (lane == 0) mbar_arrive(&l_free[s]);
                // where this lane's row goes, in units of 16 bytes
                const int tok = it.q0 + it.sub[s].t0 + row / ap.G, h = it.kvh * ap.G + row % ap.G;
                const long long at = it.b * p.rs[0] + h * p.rs[1] + tok * p.rs[2];
                const long long slot = (p.slot0 + (pair ? 2 * it.part + s : it.part)) * ap.rows + at;
                const bool mine = ok && row < nrows, live = ok && quad * 32 < nrows;
                if (mine) {
                    if (split) ap.part_l[slot] = lse2;
                    else if (ap.lse) ap.lse[at] = lse2 * kLn2;
                }
                tiles ^= (count & 1) << s;
                if (count > 0) wait(&o_done[s], ((tiles >> s) & 1) ^ 1);
                tc_fence_after();
                // O is free for the next item once its last columns are in registers, before their stores
                auto release = [&]() {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0 && count > 0) mbar_arrive(&o_free[s]);
                };
                const bool any = f != 0.f;
                if (!live) {
                    release();
                } else if (split) {
                    // a part of its own: normalised fp32 rows, which the join reads once (nothing to
                    // write where nothing was seen: its weight is 0)
                    float4 *dst = reinterpret_cast<float4 *>(ap.part_o + slot * D);
#pragma unroll 1
                    for (int q = 0; q < D; q += 64) {
                        uint32_t o[2][32];
                        tmem_ld32(tO + 128u * s + q, o[0]);
                        tmem_ld32(tO + 128u * s + q + 32, o[1]);
                        tc_wait_ld();
                        if (q + 64 == D) release();
                        if (mine && any) {
#pragma unroll
                            for (int g = 0; g < 2; ++g)
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    dst[(q + 32 * g + e) / 4] =
                                        make_float4(__uint_as_float(o[g][e]) * f, __uint_as_float(o[g][e + 1]) * f,
                                                    __uint_as_float(o[g][e + 2]) * f, __uint_as_float(o[g][e + 3]) * f);
                        }
                    }
                } else {
                    uint4 *dst[4];
                    const long long base = (it.b * p.os[0] + h * p.os[1] + tok * p.os[2]) / 8;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const long long off = __shfl_sync(0xffffffffu, base, (lane & ~3) + e);
                        dst[e] = static_cast<uint4 *>(ap.out) + off + (lane & 3);
                        if (quad * 32 + (lane & ~3) + e >= nrows) dst[e] = nullptr;
                    }
#pragma unroll 1
                    for (int q = 0; q < D; q += 32) {
                        uint32_t o[32], w[16];
                        tmem_ld32(tO + 128u * s + q, o);
                        tc_wait_ld();
                        if (q + 32 == D) release();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            w[e] = any ? pack_bf16x2(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f) : 0u;
                        tc_store_rows(tc_words(w), dst, q / 8);
                    }
                }
            }
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

template <int D> cudaError_t launch_tc(const AttnTcParams &p, cudaStream_t st)
{
    constexpr int bytes = TcLayout<D>::kBytes;
    // once a device: the shared-memory limit; and that the kernel has the registers that its split counts on
    static std::atomic<uint64_t> ready[4] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev > 255 || !(ready[dev >> 6].load() >> (dev & 63) & 1)) {
        cudaFuncAttributes at{};
        e = cudaFuncSetAttribute(attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, attn_tc_kernel<D>);
        if (e != cudaSuccess) return e;
        if (at.numRegs != kLaunchRegs) return cudaErrorInvalidKernelImage;
        if (dev <= 255) ready[dev >> 6].fetch_or(uint64_t{1} << (dev & 63));
    }
    const int n = p.a.pr[0].n_items + (p.a.n_problems > 1 ? p.a.pr[1].n_items : 0);
    return launch_dependent(attn_tc_kernel<D>, n, kTcThreads, bytes, st, p);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnTcParams &p, int head_dim, cudaStream_t st)
{
    return head_dim == 64 ? launch_tc<64>(p, st) : launch_tc<128>(p, st);
}

}  // namespace kvevict
