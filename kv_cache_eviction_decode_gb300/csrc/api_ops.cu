// api_ops.cu -- host side of the attention operators (include/kvevict_ops.h):
// argument checks, how the work is cut into items, and the launches.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include "api_internal.h"
#include "kvevict_ops.h"
#include "window_attn.h"

using namespace kvevict;

namespace {

constexpr int kSMs = 152;
constexpr int64_t kMaxRows = int64_t{1} << 30;
constexpr int kMaxGroup = 64;
constexpr int kMaxParts = 64;  // parts a unit's keys are split into at most

// The errors of calls that give no word of their own. (The kernels get one in
// any case: with a test for null beside each of their waits a causal prompt of
// 8192, 32 heads over 8, took 404 us, without 396.)
__device__ uint32_t g_errors, g_errors_taken;

__global__ void take_errors_kernel() { g_errors_taken = atomicExch(&g_errors, 0u); }

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The stride of an axis of one entry is not looked at; any other is a positive
// multiple of 16 bytes.
bool strides_ok(const int64_t *s, const int64_t *sizes, int n, int elem)
{
    for (int i = 0; i < n; ++i)
        if (sizes[i] > 1 && (s[i] <= 0 || s[i] >= (int64_t{1} << 38) || (s[i] * elem) % 16)) return false;
    return true;
}

int check_shape(const kvevict_attention_args *a)
{
    if (!a) return KVEVICT_ERR_INVALID_ARG;
    if (a->dtype != KVEVICT_F32 && a->dtype != KVEVICT_BF16) return KVEVICT_ERR_INVALID_ARG;
    if (a->head_dim != 64 && a->head_dim != 128) return KVEVICT_ERR_INVALID_ARG;
    if (a->n_kv_heads < 1 || a->n_kv_heads > 65535 || a->n_q_heads < 1 || a->n_q_heads % a->n_kv_heads ||
        a->n_q_heads / a->n_kv_heads > kMaxGroup)
        return KVEVICT_ERR_INVALID_ARG;
    if (a->batch < 0 || a->batch > (1 << 24) || a->n_sink < 0 || a->window < 0) return KVEVICT_ERR_INVALID_ARG;
    if (a->q_rows < 0 || a->k_rows < 0 || a->q_rows >= kMaxRows || a->k_rows >= kMaxRows) return KVEVICT_ERR_INVALID_ARG;
    if (!(a->scale >= 0.f) || !std::isfinite(a->scale)) return KVEVICT_ERR_INVALID_ARG;
    if (!a->q_starts != !a->k_starts) return KVEVICT_ERR_INVALID_ARG;
    if (a->q_starts) {
        if (a->q_lens || a->kv_lens || a->max_q < 0 || a->max_k < 0) return KVEVICT_ERR_INVALID_ARG;
        if (!aligned(a->q_starts, 4) || !aligned(a->k_starts, 4)) return KVEVICT_ERR_INVALID_ARG;
    }
    const int64_t per = a->q_starts ? 1 : a->batch;
    if (per * a->n_q_heads * a->q_rows >= (int64_t{1} << 40)) return KVEVICT_ERR_INVALID_ARG;
    return KVEVICT_OK;
}

// The keys a tile of rows can see at most, as tiles of `keys`.
int64_t key_tiles(int64_t max_k, int n_sink, int window, int64_t tokens, int keys)
{
    const int64_t all = (max_k + keys - 1) / keys;
    if (!window) return all;
    return std::min(all, (static_cast<int64_t>(n_sink) + keys - 1) / keys + (window + tokens - 1 + keys - 1) / keys + 1);
}

// How a problem is cut into items: tiles of rows, and parts of the key range
// where the tiles alone would leave SMs idle. An SM works on one item after
// another (on the CUDA cores a few side by side). In key tiles: an item of t
// takes t + kItemCost for its start and end (32 sequences, 8 KV heads, window
// 2044: 4.9 us an item of 5.7 tiles that would stream in 2.4), and with several
// parts rows * 4 / (tile keys * element bytes) more for writing and reading its
// part's fp32 output: little for the rows of a decoded token, four tiles for 256
// rows (a causal prompt of 4096, 32 heads over 8: 197 us in two parts, 117 in one).
constexpr double kItemCost = 1.8;

struct Cut {
    int64_t items = 0, tiles = 0;  // tiles of rows over all units; key tiles one sees at most
    double out = 0;
    bool ramp = false;             // a causal prompt: from all keys down to few

    double length(int64_t parts) const
    {
        return static_cast<double>((tiles + parts - 1) / parts) + kItemCost + (parts > 1 ? out : 0);
    }
    int64_t most() const { return items >= 4 * kSMs ? 1 : std::min<int64_t>(kMaxParts, std::max<int64_t>(1, (tiles + 1) / 2)); }
};

Cut cut(AttnProblem &p, int G, int Hkv, int rows, int keys, int elem, int64_t max_k)
{
    Cut c;
    const int per = rows / G;
    p.q_tiles = (p.max_q + per - 1) / per;
    p.splits = 1;
    p.pair = 0;
    c.items = static_cast<int64_t>(p.batch) * Hkv * p.q_tiles;
    c.tiles = key_tiles(max_k, p.n_sink, p.causal ? p.window : 0, std::min(per, p.max_q), keys);
    c.out = std::min<double>(rows, static_cast<double>(p.max_q) * G) * 4 / (keys * elem);
    c.ramp = p.causal && !p.window && p.q_tiles > 1;
    return c;
}

// Parts of a problem alone: items of equal work run in whole waves; those of a
// causal prompt take the longest item, or the work over the SMs, as where they
// start with the longest and one runs on an SM. That is the tensor-core kernel's
// way. The fp32 kernel starts with the shortest and has up to four CTAs an SM:
// for its causal prompts the estimate is too low, more so the fewer the items.
int parts_alone(const Cut &c)
{
    int best = 1;
    double least = 0;
    for (int64_t s = 1; s <= c.most(); ++s) {
        const double all = static_cast<double>(c.items * s), len = c.length(s), cost = kItemCost + (s > 1 ? c.out : 0);
        const double load = c.ramp ? std::max(len, all * (len + cost) / 2 / kSMs) : std::ceil(all / kSMs) * len;
        if (s == 1 || load < least * 0.97) {
            least = load;
            best = static_cast<int>(s);
        }
    }
    return best;
}

// Parts of two problems in one launch, the first one's items first: those take
// whole waves and, for the rest of the last one, `long_sms` SMs; the second one's
// items then fill up. A key tile of the first costs `weight` (its products, where
// both row tiles are full: 3,300 cycles against 2,750 that a streamed tile takes;
// 1.5 fits the measurements that it was chosen by: 64 sequences behind 32768 tokens
// took 154, 135, 141 and 151 us with 4, 6, 8 and 16 parts, 32 behind 8192, whose
// rows fill one row tile, 72, 62, 64 and 73 with 2, 3, 6 and 8). `share`: of the
// second's keys expected. Their lengths are on the device: the caller's 0.8 is an
// assumption, and fuller or emptier suffixes get a plan that may be slower.
void parts_together(const Cut &a, const Cut &b, double weight, double share, int &pa, int &pb)
{
    static constexpr int kTry[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 48, 64};
    double least = 0;
    pa = pb = 1;
    for (const int sb : {1, 2, 3, 4, 6, 8}) {
        if (sb > b.most()) break;
        const double lb = (b.length(sb) - kItemCost) * share + kItemCost;
        const double nb = static_cast<double>(b.items * sb);
        for (const int sa : kTry) {
            if (sa > a.most()) break;
            const double la = a.length(sa) + (weight - 1) * static_cast<double>((a.tiles + sa - 1) / sa);
            const int64_t na = a.items * sa;
            const double base = static_cast<double>(na / kSMs) * la;
            const int64_t long_sms = na % kSMs;
            // the least end at which the SMs have had room for the second's items
            double end = base + (long_sms ? la : 0);
            const double whole = std::ceil(std::max(0.0, (nb * lb - (kSMs * (end - base) - long_sms * la)) / (kSMs * lb)) - 1) * lb;
            for (double t = end + std::max(0.0, whole);; t += lb / 4) {
                const double room = std::floor((t - base) / lb + 1e-9) * (kSMs - long_sms) +
                                    std::floor((t - base - la) / lb + 1e-9) * (t - base >= la ? long_sms : 0);
                if (room >= nb) {
                    end = t;
                    break;
                }
            }
            if (least == 0 || end < least * 0.98) {
                least = end;
                pa = sa;
                pb = sb;
            }
        }
    }
}

struct Plan {
    AttnTcParams tc{};
    AttnParams &p = tc.a;
    bool tensor = false;  // bf16: the tensor-core kernel
    bool few = false;     // fp32: tiles of 16 rows
    int64_t items = 0;
    size_t bytes = 0;  // workspace
};

// fp32: tiles of 16 rows where every unit has that few, or where tiles of 64
// would leave SMs idle (8 heads x 256 rows: 23 us with 32 tiles of 64); else of 64.
bool few_rows(int G, int64_t units, int64_t max_q)
{
    const int64_t per = kAttnF32Rows / G;
    return G <= kAttnF32FewRows && (G * max_q <= kAttnF32FewRows || units * ((max_q + per - 1) / per) < kSMs);
}

// Cuts a problem for the kernel of the plan's type. The tensor cores take two
// tiles of 128 rows an item, or one (with alternate key tiles) where the rows
// fit one.
Cut cut_for(Plan &w, AttnProblem &q, int64_t max_k)
{
    const int G = w.p.G;
    if (!w.tensor)
        return cut(q, G, w.p.Hkv, w.few ? kAttnF32FewRows : kAttnF32Rows, w.few ? kAttnF32FewKeys : kAttnF32Keys, 4, max_k);
    const bool fits = q.max_q <= kAttnTcRows / G;
    const Cut c = cut(q, G, w.p.Hkv, (fits ? 1 : 2) * (kAttnTcRows / G) * G, kAttnTcKeys, 2, max_k);
    // (one key tile at most: nothing to share, the second tile stays without rows)
    q.pair = fits && c.tiles > 1;
    return c;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Slots and workspace of a cut plan; the second problem's slots follow the first's.
int finish(Plan &w, int head_dim)
{
    AttnParams &p = w.p;
    p.slots = 0;
    w.items = 0;
    for (int i = 0; i < p.n_problems; ++i) {
        AttnProblem &q = p.pr[i];
        q.slot0 = p.slots;
        p.slots += q.splits * (q.pair ? 2 : 1);  // both row tiles of a pair write a part
        const int64_t n = static_cast<int64_t>(q.batch) * p.Hkv * q.q_tiles * q.splits;
        if (n >= (int64_t{1} << 30)) return KVEVICT_ERR_INVALID_ARG;
        q.n_items = static_cast<int>(n);
        w.items += n;
    }
    w.bytes = 0;
    if (p.slots > 1)
        w.bytes = up256(static_cast<size_t>(p.slots) * p.rows * head_dim * 4) + up256(static_cast<size_t>(p.slots) * p.rows * 4);
    return KVEVICT_OK;
}

int plan_window(const kvevict_attention_args *a, Plan &w)
{
    AttnParams &p = w.p;
    p.Hq = a->n_q_heads;
    p.Hkv = a->n_kv_heads;
    p.G = p.Hq / p.Hkv;
    p.n_problems = 1;
    AttnProblem &q = p.pr[0];
    const bool packed = a->q_starts != nullptr;
    q.batch = a->batch;
    q.causal = 1;
    q.n_sink = static_cast<int>(std::min<int64_t>(a->n_sink, a->k_rows));
    q.window = a->window >= a->k_rows ? 0 : a->window;  // a window as long as the keys hides nothing
    q.q_rows = static_cast<int>(a->q_rows);
    q.k_rows = static_cast<int>(a->k_rows);
    q.max_q = packed ? static_cast<int>(std::min<int64_t>(a->max_q, a->q_rows)) : q.q_rows;
    const int64_t max_k = packed ? std::min<int64_t>(a->max_k, a->k_rows) : a->k_rows;
    const int64_t N = a->q_rows;
    p.rows = (packed ? 1 : static_cast<int64_t>(a->batch)) * p.Hq * N;
    if (packed) {
        q.rs[0] = 0; q.rs[1] = 1; q.rs[2] = p.Hq;
    } else {
        q.rs[0] = p.Hq * N; q.rs[1] = N; q.rs[2] = 1;
    }
    w.tensor = a->dtype == KVEVICT_BF16;
    w.few = few_rows(p.G, static_cast<int64_t>(q.batch) * p.Hkv, q.max_q);
    q.splits = parts_alone(cut_for(w, q, max_k));
    return finish(w, a->head_dim);
}

// `outside`: the suffixes' part is one that the caller writes.
int plan_shared(const kvevict_shared_prefix_args *s, Plan &w, bool outside)
{
    const kvevict_attention_args *a = &s->a;
    AttnParams &p = w.p;
    p.Hq = a->n_q_heads;
    p.Hkv = a->n_kv_heads;
    p.G = p.Hq / p.Hkv;
    p.n_problems = 2;
    p.rows = static_cast<int64_t>(a->batch) * p.Hq;
    // the prefix: one sequence whose tokens are the batch's sequences
    AttnProblem &x = p.pr[0];
    x.batch = 1;
    x.q_rows = x.max_q = a->batch;
    x.k_rows = static_cast<int>(s->prefix_rows);
    x.rs[0] = 0; x.rs[1] = 1; x.rs[2] = p.Hq;
    // the suffixes: one token each
    AttnProblem &y = p.pr[1];
    y.batch = a->batch;
    y.q_rows = y.max_q = 1;
    y.k_rows = static_cast<int>(a->k_rows);
    y.rs[0] = p.Hq; y.rs[1] = 1; y.rs[2] = 0;
    w.tensor = a->dtype == KVEVICT_BF16;
    w.few = few_rows(p.G, p.Hkv, a->batch);
    const Cut cx = cut_for(w, x, x.k_rows);
    if (outside) {
        x.splits = parts_alone(cx);
        y.splits = 1;  // no items
    } else {
        const Cut cy = cut_for(w, y, y.k_rows);
        parts_together(cx, cy, w.tensor && !x.pair ? 1.5 : 1.0, 0.8, x.splits, y.splits);
    }
    return finish(w, a->head_dim);
}

int check_tensors(const kvevict_attention_args *a, bool needs_k)
{
    const int elem = a->dtype == KVEVICT_F32 ? 4 : 2;
    const int64_t seqs = a->q_starts ? 1 : a->batch;
    const int64_t qn[3] = {seqs, a->n_q_heads, a->q_rows}, kn[3] = {seqs, a->n_kv_heads, a->k_rows};
    if (!a->q || !a->out || !aligned(a->q, 16) || !aligned(a->out, 16) || !strides_ok(a->q_stride, qn, 3, elem) ||
        !strides_ok(a->out_stride, qn, 3, elem))
        return KVEVICT_ERR_INVALID_ARG;
    if (needs_k && (!a->k || !a->v || !aligned(a->k, 16) || !aligned(a->v, 16) || !strides_ok(a->k_stride, kn, 3, elem) ||
                    !strides_ok(a->v_stride, kn, 3, elem)))
        return KVEVICT_ERR_INVALID_ARG;
    if (!aligned(a->lse, 4) || !aligned(a->q_lens, 4) || !aligned(a->kv_lens, 4) || !aligned(a->error_word, 4))
        return KVEVICT_ERR_INVALID_ARG;
    return KVEVICT_OK;
}

// Encodes a bf16 tensor map of `rank` axes, the first (head_dim) contiguous.
// strides: in elements, of axes 1.. ; an axis of one entry takes any valid stride.
int encode_map(AttnTmap *out, const void *base, int rank, const uint64_t *dims, const long long *strides, const uint32_t *box)
{
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn) : nullptr;
    }();
    if (!encode) return KVEVICT_ERR_CUDA;
    cuuint64_t d[5], s[4];
    cuuint32_t b[5], one[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        one[i] = 1;
        if (i) s[i - 1] = static_cast<cuuint64_t>(dims[i] > 1 ? strides[i - 1] : static_cast<long long>(dims[0])) * 2;
    }
    static_assert(sizeof(CUtensorMap) == sizeof(AttnTmap), "tensor map size");
    CUtensorMap m;
    if (encode(&m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void *>(base), d, s, b, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return KVEVICT_ERR_INVALID_ARG;
    std::memcpy(out, &m, sizeof m);
    return KVEVICT_OK;
}

int make_maps(AttnTcMaps &t, const AttnProblem &p, int G, int Hkv, int head_dim)
{
    const uint64_t D = static_cast<uint64_t>(head_dim);
    const uint64_t qseq = p.q_starts ? 1 : p.batch, kseq = p.k_starts ? 1 : p.batch;
    const uint64_t qd[5] = {D, static_cast<uint64_t>(G), static_cast<uint64_t>(p.q_rows), static_cast<uint64_t>(Hkv), qseq};
    const long long qs[4] = {p.qs[1], p.qs[2], G * p.qs[1], p.qs[0]};
    const uint32_t qb[5] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(kAttnTcRows / G), 1, 1};
    int rc = encode_map(&t.q, p.q, 5, qd, qs, qb);
    // without keys nothing is loaded: any address does
    const uint64_t kd[4] = {D, static_cast<uint64_t>(std::max(p.k_rows, 1)), static_cast<uint64_t>(Hkv), kseq};
    const long long ks[3] = {p.ks[2], p.ks[1], p.ks[0]}, vs[3] = {p.vs[2], p.vs[1], p.vs[0]};
    const long long any[3] = {head_dim, head_dim, head_dim};
    const uint32_t kb[4] = {64, kAttnTcKeys, 1, 1};
    const bool none = p.k_rows == 0;
    if (!rc) rc = encode_map(&t.k, none ? p.q : p.k, 4, kd, none ? any : ks, kb);
    if (!rc) rc = encode_map(&t.v, none ? p.q : p.v, 4, kd, none ? any : vs, kb);
    return rc;
}

int bind_workspace(const kvevict_attention_args *a, Plan &w)
{
    AttnParams &p = w.p;
    if (w.bytes) {
        if (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < w.bytes) return KVEVICT_ERR_INVALID_ARG;
        p.part_o = static_cast<float *>(a->workspace);
        p.part_l = reinterpret_cast<float *>(static_cast<uint8_t *>(a->workspace) +
                                             up256(static_cast<size_t>(p.slots) * p.rows * a->head_dim * 4));
    }
    return KVEVICT_OK;
}

int run(const kvevict_attention_args *a, Plan &w, cudaStream_t st)
{
    AttnParams &p = w.p;
    const int rw = bind_workspace(a, w);
    if (rw) return rw;
    const double scale = a->scale > 0.f ? a->scale : 1.0 / std::sqrt(static_cast<double>(a->head_dim));
    p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
    p.out = a->out;
    p.lse = a->lse;
    p.err = a->error_word;
    const bool bf16 = a->dtype == KVEVICT_BF16;
    cudaError_t e = p.err ? cudaSuccess : operator_errors_address(&p.err);
    if (e != cudaSuccess) return KVEVICT_ERR_CUDA;
    if (w.tensor) {
        for (int i = 0; i < p.n_problems; ++i) {
            const int rc = make_maps(w.tc.maps[i], p.pr[i], p.G, p.Hkv, a->head_dim);
            if (rc) return rc;
        }
        e = launch_attn_tc(w.tc, a->head_dim, st);
    } else {
        e = launch_attn_f32(p, a->head_dim, w.few, st);
    }
    if (e == cudaSuccess && p.slots > 1) e = launch_attn_join(p, a->head_dim, bf16, st);
    return e == cudaSuccess ? KVEVICT_OK : KVEVICT_ERR_CUDA;
}

void copy3(long long (&d)[3], const int64_t *s)
{
    for (int i = 0; i < 3; ++i) d[i] = s[i];
}

int check_shared(const kvevict_shared_prefix_args *s)
{
    if (!s) return KVEVICT_ERR_INVALID_ARG;
    const int rc = check_shape(&s->a);
    if (rc) return rc;
    const kvevict_attention_args *a = &s->a;
    if (a->q_starts || a->k_starts || a->q_lens || a->n_sink || a->window || a->q_rows != 1 || s->prefix_rows < 0 ||
        s->prefix_rows >= kMaxRows)
        return KVEVICT_ERR_INVALID_ARG;
    return KVEVICT_OK;
}

}  // namespace

cudaError_t kvevict::operator_errors_address(uint32_t **out)
{
    static std::atomic<uint32_t *> known[256] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    void *p = dev < 256 ? known[dev].load() : nullptr;
    if (!p) {
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        e = cudaThreadExchangeStreamCaptureMode(&mode);
        if (e != cudaSuccess) return e;
        e = cudaGetSymbolAddress(&p, g_errors);
        const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
        if (e == cudaSuccess) e = back;
        if (e != cudaSuccess) return e;
        if (dev < 256) known[dev].store(static_cast<uint32_t *>(p));
    }
    *out = static_cast<uint32_t *>(p);
    return cudaSuccess;
}

extern "C" int kvevict_window_attention_workspace_bytes(const kvevict_attention_args *a, size_t *bytes)
{
    int rc = check_shape(a);
    if (rc) return rc;
    if (!bytes) return KVEVICT_ERR_INVALID_ARG;
    Plan w;
    rc = plan_window(a, w);
    if (rc == KVEVICT_OK) *bytes = w.bytes;
    return rc;
}

extern "C" int kvevict_window_attention(const kvevict_attention_args *a, void *cuda_stream)
{
    int rc = check_shape(a);
    if (rc) return rc;
    Plan w;
    rc = plan_window(a, w);
    if (rc) return rc;
    if (w.items == 0) return KVEVICT_OK;  // no query rows
    rc = check_tensors(a, a->k_rows > 0);
    if (rc) return rc;
    AttnProblem &q = w.p.pr[0];
    q.q = a->q; q.k = a->k; q.v = a->v;
    copy3(q.qs, a->q_stride);
    copy3(q.ks, a->k_stride);
    copy3(q.vs, a->v_stride);
    copy3(q.os, a->out_stride);
    if (a->q_starts) q.os[0] = 0;
    q.q_starts = a->q_starts; q.k_starts = a->k_starts; q.q_lens = a->q_lens; q.k_lens = a->kv_lens;
    return run(a, w, static_cast<cudaStream_t>(cuda_stream));
}

extern "C" int kvevict_operator_errors(uint32_t *device_error)
{
    if (!device_error) return KVEVICT_ERR_INVALID_ARG;
    static std::mutex one;  // (g_errors_taken holds one caller's)
    const std::lock_guard<std::mutex> lock(one);
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return KVEVICT_ERR_CUDA;
    take_errors_kernel<<<1, 1>>>();
    e = cudaGetLastError();
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(device_error, g_errors_taken, sizeof g_errors_taken);
    if (e != cudaSuccess) return KVEVICT_ERR_CUDA;
    return *device_error ? KVEVICT_ERR_DEVICE : KVEVICT_OK;
}

extern "C" int kvevict_shared_prefix_attention_workspace_bytes(const kvevict_shared_prefix_args *s, size_t *bytes)
{
    int rc = check_shared(s);
    if (rc) return rc;
    if (!bytes) return KVEVICT_ERR_INVALID_ARG;
    Plan w;
    rc = plan_shared(s, w, false);
    if (rc == KVEVICT_OK) *bytes = w.bytes;
    return rc;
}

namespace {

// Checks the call's tensors, and fills the plan with them.
int bind_shared(const kvevict_shared_prefix_args *s, Plan &w)
{
    const kvevict_attention_args *a = &s->a;
    const int rc = check_tensors(a, a->k_rows > 0);
    if (rc) return rc;
    const int elem = a->dtype == KVEVICT_F32 ? 4 : 2;
    const int64_t pn[2] = {a->n_kv_heads, s->prefix_rows};
    if (s->prefix_rows > 0 && (!s->k_prefix || !s->v_prefix || !aligned(s->k_prefix, 16) || !aligned(s->v_prefix, 16) ||
                               !strides_ok(s->k_prefix_stride, pn, 2, elem) || !strides_ok(s->v_prefix_stride, pn, 2, elem)))
        return KVEVICT_ERR_INVALID_ARG;
    AttnProblem &x = w.p.pr[0], &y = w.p.pr[1];
    x.q = y.q = a->q;
    x.qs[0] = 0; x.qs[1] = a->q_stride[1]; x.qs[2] = a->q_stride[0];
    y.qs[0] = a->q_stride[0]; y.qs[1] = a->q_stride[1]; y.qs[2] = 0;
    x.os[0] = 0; x.os[1] = a->out_stride[1]; x.os[2] = a->out_stride[0];
    y.os[0] = a->out_stride[0]; y.os[1] = a->out_stride[1]; y.os[2] = 0;
    x.k = s->k_prefix; x.v = s->v_prefix;
    x.ks[0] = x.vs[0] = 0;
    x.ks[1] = s->k_prefix_stride[0]; x.ks[2] = s->k_prefix_stride[1];
    x.vs[1] = s->v_prefix_stride[0]; x.vs[2] = s->v_prefix_stride[1];
    y.k = a->k; y.v = a->v;
    copy3(y.ks, a->k_stride);
    copy3(y.vs, a->v_stride);
    y.k_lens = a->kv_lens;
    return KVEVICT_OK;
}

int shared_call(const kvevict_shared_prefix_args *s, Plan &w, bool outside)
{
    int rc = check_shared(s);
    if (!rc) rc = plan_shared(s, w, outside);
    return rc;
}

}  // namespace

extern "C" int kvevict_shared_prefix_attention(const kvevict_shared_prefix_args *s, void *cuda_stream)
{
    Plan w;
    int rc = shared_call(s, w, false);
    if (rc) return rc;
    if (s->a.batch == 0) return KVEVICT_OK;
    rc = bind_shared(s, w);
    return rc ? rc : run(&s->a, w, static_cast<cudaStream_t>(cuda_stream));
}

extern "C" int kvevict_prefix_bytes(const kvevict_shared_prefix_args *s, size_t *bytes)
{
    Plan w;
    const int rc = shared_call(s, w, true);
    if (rc == KVEVICT_OK) *bytes = w.bytes;
    return rc;
}

extern "C" int kvevict_prefix_part(const kvevict_shared_prefix_args *s, float **part_o, float **part_l)
{
    Plan w;
    int rc = shared_call(s, w, true);
    if (!rc) rc = bind_shared(s, w);
    if (!rc) rc = bind_workspace(&s->a, w);
    if (rc) return rc;
    const AttnParams &p = w.p;
    *part_o = p.part_o + static_cast<size_t>(p.pr[1].slot0) * p.rows * s->a.head_dim;
    *part_l = p.part_l + static_cast<size_t>(p.pr[1].slot0) * p.rows;
    return KVEVICT_OK;
}

extern "C" int kvevict_prefix_run(const kvevict_shared_prefix_args *s, void *cuda_stream)
{
    Plan w;
    int rc = shared_call(s, w, true);
    if (!rc) rc = bind_shared(s, w);
    return rc ? rc : run(&s->a, w, static_cast<cudaStream_t>(cuda_stream));
}
