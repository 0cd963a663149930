// api_paged.cu -- host side of the operators on a paged cache
// (include/kvevict_paged.h): argument checks, how the work is cut, launches.
#include <algorithm>
#include <climits>
#include <cmath>

#include "api_internal.h"
#include "paged_attn.h"
#include "paged_move.h"

using namespace kvevict;

namespace {

constexpr int kSMs = 152;
constexpr int64_t kMaxRows = int64_t{1} << 30;
constexpr int64_t kMaxStride = int64_t{1} << 38;
constexpr int kMaxGroup = 64;
constexpr int kMaxParts = 64;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The stride of an axis of one entry is not looked at.
bool strides_ok(const int64_t *s, const int64_t *sizes, int n, int elem, int64_t least)
{
    for (int i = 0; i < n; ++i)
        if (sizes[i] > 1 && (s[i] < least || s[i] >= kMaxStride || (s[i] * elem) % 16)) return false;
    return true;
}

int elem_of(int dtype) { return dtype == KVEVICT_F32 ? 4 : 2; }

// Shapes only: pointers and strides are looked at where there is work.
int check_cache(const kvevict_paged_cache &c)
{
    if (c.dtype != KVEVICT_F32 && c.dtype != KVEVICT_BF16) return KVEVICT_ERR_INVALID_ARG;
    if (c.page_dtype != c.dtype && c.page_dtype != KVEVICT_Q4) return KVEVICT_ERR_INVALID_ARG;
    if (c.head_dim != 64 && c.head_dim != 128) return KVEVICT_ERR_INVALID_ARG;
    if (c.n_kv_heads < 1 || c.n_kv_heads > 32767) return KVEVICT_ERR_INVALID_ARG;
    if (c.page_size < 16 || c.page_size > 256 || (c.page_size & (c.page_size - 1))) return KVEVICT_ERR_INVALID_ARG;
    if (c.batch < 0 || c.batch > (1 << 24) || c.table_width < 0 || c.n_pages < 0) return KVEVICT_ERR_INVALID_ARG;
    if (static_cast<int64_t>(c.table_width) * c.page_size >= kMaxRows) return KVEVICT_ERR_INVALID_ARG;
    return KVEVICT_OK;
}

int bind_cache(const kvevict_paged_cache &c, PagedCache &p)
{
    const bool q4 = c.page_dtype == KVEVICT_Q4;
    const int elem = q4 ? 1 : elem_of(c.dtype);
    const int64_t sizes[3] = {c.n_pages, c.n_kv_heads, q4 ? 1 : c.page_size};
    if (c.n_pages > 0 && (!c.k_pages || !c.v_pages || !aligned(c.k_pages, 16) || !aligned(c.v_pages, 16) ||
                          !strides_ok(c.k_page_stride, sizes, 3, elem, 1) || !strides_ok(c.v_page_stride, sizes, 3, elem, 1)))
        return KVEVICT_ERR_INVALID_ARG;
    if (!c.kv_lens || !aligned(c.kv_lens, 4) || !aligned(c.error_word, 4)) return KVEVICT_ERR_INVALID_ARG;
    if (c.table_width > 0 && (!c.block_table || !aligned(c.block_table, 4))) return KVEVICT_ERR_INVALID_ARG;
    if (c.table_width > 0 && c.batch > 1 && (c.table_stride < 0 || c.table_stride >= kMaxStride)) return KVEVICT_ERR_INVALID_ARG;
    void *pages[2] = {c.k_pages, c.v_pages};
    const int64_t *strides[2] = {c.k_page_stride, c.v_page_stride};
    for (int i = 0; i < 2; ++i) {
        p.pages[i] = static_cast<char *>(pages[i]);
        p.page_bytes[i] = c.n_pages > 1 ? strides[i][0] * elem : 0;
        p.head_bytes[i] = c.n_kv_heads > 1 ? strides[i][1] * elem : 0;
        p.token_bytes[i] = q4 ? 0 : strides[i][2] * elem;
    }
    p.table = c.block_table;
    p.table_stride = c.batch > 1 ? c.table_stride : 0;
    p.kv_lens = c.kv_lens;
    p.Hkv = c.n_kv_heads;
    p.S = c.page_size;
    p.log2_s = __builtin_ctz(static_cast<unsigned>(c.page_size));
    p.batch = c.batch;
    p.width = c.table_width;
    p.n_pages = c.n_pages;
    p.err = c.error_word;
    if (!p.err && operator_errors_address(&p.err) != cudaSuccess) return KVEVICT_ERR_CUDA;
    return KVEVICT_OK;
}

// New tokens: with starts any number, else the same of every sequence.
int check_tokens(int64_t tokens, const int32_t *starts, int batch)
{
    if (tokens < 0 || tokens >= kMaxRows || !aligned(starts, 4)) return KVEVICT_ERR_INVALID_ARG;
    if (!starts && (batch ? tokens % batch : tokens) != 0) return KVEVICT_ERR_INVALID_ARG;
    return KVEVICT_OK;
}

struct Plan {
    PagedAttnParams p{};
    int rows = 0;  // of an item: with bf16 those of the tensor-core kernel
    int64_t items = 0;
    size_t bytes = 0;
};

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int check_attention(const kvevict_paged_attention_args *a)
{
    if (!a) return KVEVICT_ERR_INVALID_ARG;
    int rc = check_cache(a->c);
    if (!rc) rc = check_tokens(a->tokens, a->q_starts, a->c.batch);
    if (rc) return rc;
    if (a->n_q_heads < 1 || a->n_q_heads % a->c.n_kv_heads || a->n_q_heads / a->c.n_kv_heads > kMaxGroup) return KVEVICT_ERR_INVALID_ARG;
    if (a->n_sink < 0 || a->window < 0 || a->max_q < 0 || a->max_k < 0) return KVEVICT_ERR_INVALID_ARG;
    if (!(a->scale >= 0.f) || !std::isfinite(a->scale)) return KVEVICT_ERR_INVALID_ARG;
    if (a->tokens * a->n_q_heads >= (int64_t{1} << 40)) return KVEVICT_ERR_INVALID_ARG;
    return KVEVICT_OK;
}

// The 16-key tiles that a tile of rows can see at most.
int64_t key_tiles(int64_t max_k, int n_sink, int window, int64_t tokens)
{
    const int64_t all = (max_k + kPagedTile - 1) / kPagedTile;
    if (!window) return all;
    return std::min(all, (static_cast<int64_t>(n_sink) + kPagedTile - 1) / kPagedTile + (window + tokens - 1 + kPagedTile - 1) / kPagedTile + 1);
}

// Parts that the keys of a unit are split into, by a cost in a warp's tiles. An item
// takes kItemCost more for its start and end, joining takes what is below, both times
// `light`: 1 where a tile is 4 bits, less where it is more bytes (bf16 a half, fp32 a
// quarter). Items under a window are of one length and run in waves of `slots` CTAs.
// Without one their lengths are on the device, and taken to be anything from all alike
// to spread around kShare of the longest, where the slots are filled but for half an
// item at the end: the mean of both. (4 bits, 256 units of up to 2048 tiles: 316, 231,
// 221, 224 and 245 us with 1, 4, 7, 10 and 20 parts; bf16, 256 units of up to 640: 167,
// 149, 152 and 164 us with 1, 5, 10 and 16; bf16, 8 units of 2048, all alike: 36, 33, 34
// and 45 us with 16, 24, 38 and 40; 4 bits, 128 units of 130 under a window: 41, 31, 41
// us with 1, 2 and 3.)
// Up to eight parts are joined in clusters where all of them run at once, with some
// room, as clusters do not fill every slot (4 bits, 32 units of 63 tiles: 9.5 us with
// eight parts, 11.4 through the workspace, 12.8 with one; 64 units of 250: 16.4 with
// six, 17.7 with four through the workspace; but 256 units of 2048 in seven: 242,
// through the workspace 213).
constexpr int kMaxCluster = 8;
constexpr double kItemCost = 6, kClusterCost = 3, kJoinCost = 8, kJoinPart = 0.1, kShare = 0.75, kClusterFill = 0.9;

int parts(int64_t units, int64_t tiles, int64_t slots, double light, bool window, int &clusters)
{
    int best = 1;
    double least = 0;
    clusters = 0;
    for (int64_t s = 1; s <= kMaxParts && (s == 1 || s * kPagedMmaWarps <= tiles); ++s) {
        const double load = static_cast<double>(units * s) / static_cast<double>(slots);
        const double item = kItemCost * light, len = std::ceil(static_cast<double>(tiles) / static_cast<double>(s * kPagedMmaWarps)), longest = len + item;
        const bool cluster = s > 1 && s <= kMaxCluster && load <= kClusterFill;
        const double waves = std::ceil(load) * longest, spread = std::max(longest, load * (len * kShare + item) + longest / 2);
        const double cost = (window ? waves : (waves + spread) / 2) +
                            (s == 1 ? 0 : cluster ? kClusterCost : kJoinCost + kJoinPart * static_cast<double>(s)) * light;
        if (s == 1 || cost < least * 0.99) {
            least = cost;
            best = static_cast<int>(s);
            clusters = cluster;
        }
    }
    return best;
}

int plan_attention(const kvevict_paged_attention_args *a, Plan &w)
{
    PagedAttnParams &p = w.p;
    p.Hq = a->n_q_heads;
    p.G = p.Hq / a->c.n_kv_heads;
    p.tokens = static_cast<int>(a->tokens);
    p.per = a->q_starts || !a->c.batch ? 0 : static_cast<int>(a->tokens / a->c.batch);
    p.max_q = a->q_starts ? static_cast<int>(std::min<int64_t>(a->max_q, a->tokens)) : p.per;
    const int64_t room = static_cast<int64_t>(a->c.table_width) * a->c.page_size;
    const int64_t max_k = a->max_k ? std::min<int64_t>(a->max_k, room) : room;
    p.mask.causal = 1;
    p.mask.n_sink = a->n_sink;
    p.mask.window = a->window >= room ? 0 : a->window;  // a window as long as the table hides nothing
    p.mask.q_starts = a->q_starts;
    const bool tensor = a->c.dtype == KVEVICT_BF16, q4 = a->c.page_dtype == KVEVICT_Q4;
    const int64_t rows = static_cast<int64_t>(p.max_q) * p.G;
    if (rows > INT_MAX - 16) return KVEVICT_ERR_INVALID_ARG;  // a unit's rows are ints in the kernels
    w.rows = tensor ? (rows <= 8 ? 8 : 16) : rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : 8;
    p.q_tiles = static_cast<int>((rows + w.rows - 1) / w.rows);
    const int64_t units = static_cast<int64_t>(a->c.batch) * a->c.n_kv_heads * p.q_tiles;
    const int64_t tiles = key_tiles(max_k, p.mask.n_sink, p.mask.window, std::min<int64_t>(p.max_q, (w.rows + p.G - 1) / p.G + 1));
    // (with starts only the mean of the new tokens is known here)
    const int64_t mean = a->c.batch ? (a->tokens + a->c.batch - 1) / a->c.batch * p.G : 0;
    const int64_t busy = static_cast<int64_t>(a->c.batch) * a->c.n_kv_heads * std::min<int64_t>(p.q_tiles, (mean + w.rows - 1) / w.rows);
    const int ctas = tensor ? paged_mma_ctas(q4, w.rows) : paged_simt_ctas(q4, a->c.head_dim, w.rows);
    p.splits = parts(busy, tiles, kSMs * ctas, q4 && tensor ? 1 : tensor || q4 ? 0.5 : 0.25, p.mask.window > 0, p.clusters);
    w.items = units * p.splits;
    if (w.items >= (int64_t{1} << 31)) return KVEVICT_ERR_INVALID_ARG;
    const size_t slots = static_cast<size_t>(p.splits) * a->tokens * p.Hq;
    w.bytes = p.splits > 1 && !p.clusters ? up256(slots * a->c.head_dim * 4) + up256(slots * 4) : 0;
    return KVEVICT_OK;
}

}  // namespace

extern "C" int kvevict_paged_append(const kvevict_paged_append_args *a, void *cuda_stream)
{
    if (!a) return KVEVICT_ERR_INVALID_ARG;
    int rc = check_cache(a->c);
    if (!rc) rc = check_tokens(a->tokens, a->starts, a->c.batch);
    if (rc) return rc;
    if (a->rotary_dim < 0 || a->rotary_dim % 2 || a->rotary_dim > a->c.head_dim) return KVEVICT_ERR_INVALID_ARG;
    if (a->rotary_dim && (((a->interleaved | a->positions_64) & ~1) || !std::isfinite(a->scale) || !a->inv_freq || !aligned(a->inv_freq, 8)))
        return KVEVICT_ERR_INVALID_ARG;
    const bool turns = a->rotary_dim != 0;
    if (turns && a->positions && !aligned(a->positions, a->positions_64 ? 8 : 4)) return KVEVICT_ERR_INVALID_ARG;
    if (a->tokens == 0 || a->c.batch == 0) return KVEVICT_OK;
    const int elem = elem_of(a->c.dtype);
    const int64_t sizes[2] = {a->c.n_kv_heads, a->tokens};
    if (!a->k || !a->v || !aligned(a->k, 16) || !aligned(a->v, 16) || !strides_ok(a->k_stride, sizes, 2, elem, 0) ||
        !strides_ok(a->v_stride, sizes, 2, elem, 0))
        return KVEVICT_ERR_INVALID_ARG;
    AppendParams p{};
    rc = bind_cache(a->c, p.c);
    if (rc) return rc;
    p.x[0] = a->k;
    p.x[1] = a->v;
    for (int i = 0; i < 2; ++i) {
        p.xs[0][i] = a->k_stride[i];
        p.xs[1][i] = a->v_stride[i];
    }
    p.starts = a->starts;
    p.tokens = static_cast<int>(a->tokens);
    p.per = a->starts ? 0 : static_cast<int>(a->tokens / a->c.batch);
    if (turns) {
        p.freq = a->inv_freq;
        p.pos = a->positions;
        p.ps = a->pos_stride;
        p.pos64 = a->positions_64;
        p.R = a->rotary_dim;
        p.inter = a->interleaved;
        p.scale = a->scale;
    }
    // A CTA's heads: a thread's whole batch of loads (4 bits: four of them), or, where that would leave SMs idle, what
    // gives every SM two CTAs, but what its threads take at once at least.
    const bool own = append_own(p, elem, a->c.page_dtype == KVEVICT_Q4);
    const int64_t heads = 2 * a->c.n_kv_heads, once = own ? 2 * kPagedThreads * 16 / (a->c.head_dim * elem) : 8 * kPagedThreads / a->c.head_dim;
    const int64_t want = std::min((own ? kAppendOwnBatch : 16) * once, std::max(once, a->tokens * heads / (2 * kSMs)));
    p.heads_per = static_cast<int>(std::min(heads, want));
    p.head_blocks = static_cast<int>((heads + p.heads_per - 1) / p.heads_per);
    p.tokens_per = p.head_blocks > 1 ? 1 : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kAppendTokens, want / heads)));
    if ((a->tokens + p.tokens_per - 1) / p.tokens_per * p.head_blocks >= (int64_t{1} << 31)) return KVEVICT_ERR_INVALID_ARG;
    const cudaError_t e = launch_append(p, a->c.head_dim, elem, a->c.page_dtype == KVEVICT_Q4, static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? KVEVICT_OK : KVEVICT_ERR_CUDA;
}

extern "C" int kvevict_paged_gather(const kvevict_paged_gather_args *a, void *cuda_stream)
{
    if (!a) return KVEVICT_ERR_INVALID_ARG;
    int rc = check_cache(a->c);
    if (rc) return rc;
    if (a->rows < 0 || a->rows >= kMaxRows || !aligned(a->k_starts, 4)) return KVEVICT_ERR_INVALID_ARG;
    if (a->rows == 0 || a->c.batch == 0) return KVEVICT_OK;
    const int elem = elem_of(a->c.dtype);
    const int64_t sizes[3] = {a->k_starts ? 1 : a->c.batch, a->c.n_kv_heads, a->rows};
    if (!a->k_out || !a->v_out || !aligned(a->k_out, 16) || !aligned(a->v_out, 16) || !strides_ok(a->k_out_stride, sizes, 3, elem, 1) ||
        !strides_ok(a->v_out_stride, sizes, 3, elem, 1))
        return KVEVICT_ERR_INVALID_ARG;
    GatherParams p{};
    rc = bind_cache(a->c, p.c);
    if (rc) return rc;
    p.y[0] = a->k_out;
    p.y[1] = a->v_out;
    for (int i = 0; i < 3; ++i) {
        p.ys[0][i] = a->k_out_stride[i];
        p.ys[1][i] = a->v_out_stride[i];
    }
    p.k_starts = a->k_starts;
    p.rows = static_cast<int>(a->rows);
    p.tiles = (p.rows + kGatherRows - 1) / kGatherRows;
    if (static_cast<int64_t>(p.tiles) * a->c.n_kv_heads * (a->k_starts ? 1 : a->c.batch) >= (int64_t{1} << 31)) return KVEVICT_ERR_INVALID_ARG;
    const cudaError_t e = launch_gather(p, a->c.head_dim, elem, a->c.page_dtype == KVEVICT_Q4, static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? KVEVICT_OK : KVEVICT_ERR_CUDA;
}

extern "C" int kvevict_paged_attention_workspace_bytes(const kvevict_paged_attention_args *a, size_t *bytes)
{
    int rc = check_attention(a);
    if (rc) return rc;
    if (!bytes) return KVEVICT_ERR_INVALID_ARG;
    Plan w;
    rc = plan_attention(a, w);
    if (rc == KVEVICT_OK) *bytes = w.bytes;
    return rc;
}

extern "C" int kvevict_paged_attention(const kvevict_paged_attention_args *a, void *cuda_stream)
{
    int rc = check_attention(a);
    if (rc) return rc;
    Plan w;
    rc = plan_attention(a, w);
    if (rc) return rc;
    if (w.items == 0) return KVEVICT_OK;  // no query rows
    PagedAttnParams &p = w.p;
    const int elem = elem_of(a->c.dtype);
    const int64_t sizes[2] = {a->n_q_heads, a->tokens};
    if (!a->q || !a->out || !aligned(a->q, 16) || !aligned(a->out, 16) || !strides_ok(a->q_stride, sizes, 2, elem, 1) ||
        !strides_ok(a->out_stride, sizes, 2, elem, 1) || !aligned(a->lse, 4))
        return KVEVICT_ERR_INVALID_ARG;
    if (w.bytes) {
        if (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < w.bytes) return KVEVICT_ERR_INVALID_ARG;
        p.part_o = static_cast<float *>(a->workspace);
        p.part_l = reinterpret_cast<float *>(static_cast<char *>(a->workspace) +
                                             up256(static_cast<size_t>(p.splits) * p.tokens * p.Hq * a->c.head_dim * 4));
    }
    rc = bind_cache(a->c, p.c);
    if (rc) return rc;
    if (a->c.n_pages == 0)  // no key is read, but the copies of none of its bytes need an address: a row of q
        for (int i = 0; i < 2; ++i) {
            p.c.pages[i] = const_cast<char *>(static_cast<const char *>(a->q));
            p.c.head_bytes[i] = p.c.token_bytes[i] = 0;
        }
    p.q = a->q;
    p.out = a->out;
    p.lse = a->lse;
    for (int i = 0; i < 2; ++i) {
        p.qs[i] = a->q_stride[i];
        p.os[i] = a->out_stride[i];
    }
    const double scale = a->scale > 0.f ? a->scale : 1.0 / std::sqrt(static_cast<double>(a->c.head_dim));
    p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const bool bf16 = a->c.dtype == KVEVICT_BF16, q4 = a->c.page_dtype == KVEVICT_Q4;
    cudaError_t e = bf16 ? launch_paged_mma(p, a->c.head_dim, q4, w.rows, st) : launch_paged_simt(p, a->c.head_dim, q4, w.rows, st);
    if (e == cudaSuccess && p.splits > 1 && !p.clusters) e = launch_paged_join(p, a->c.head_dim, bf16, st);
    return e == cudaSuccess ? KVEVICT_OK : KVEVICT_ERR_CUDA;
}
