/*
 * kvevict_ops.h -- operators around the decode step, in libkvevict.so: the
 * prompt's attention under the set of tokens a StreamingLLM cache keeps (or
 * plain causal attention), decode attention of a batch that shares a prefix,
 * rotary positions for queries and keys, and norms of their heads before them.
 * (A paged cache and its attention: kvevict_paged.h.)
 *
 * These calls take no handle unless they say so: the arguments come in one
 * struct, the work is queued on the given stream (a cudaStream_t; NULL: the
 * legacy default stream), and the device that holds the tensors must be the
 * current one. As with kvevict.h, argument errors are found on the host
 * before anything is launched and returned as a negative kvevict_status;
 * anomalies found on the GPU set bits of a device error word, here one that
 * the caller may pass, else the device's, which kvevict_operator_errors reads.
 * No call allocates device memory; none but that one waits for the GPU, and each
 * of the others can be captured in a CUDA graph.
 *
 * Tensors have their last axis (head_dim) contiguous; every other axis has a
 * stride of its own, in elements, given in the order sequence, head, token.
 * Base addresses are 16-byte aligned and strides positive multiples of 16 bytes
 * (the inputs of kvevict_rotary: any multiples). The stride of an axis of one
 * entry is not looked at.
 */
#ifndef KVEVICT_OPS_H
#define KVEVICT_OPS_H

#include "kvevict.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A length or start on the device was out of range (negative, decreasing,
 * beyond the tensor, a sequence longer than max_q): it was clamped. Of a
 * sequence with more queries than there are rows, or than max_q, the first ones
 * are computed, at the positions that the given number of queries puts them at;
 * the other rows are left as they were. Where the starts of a packed batch go
 * back, the sequence that would end before it starts and every one behind it
 * were left out. */
#define KVEVICT_DEV_BAD_LENGTH 0x10u

/*
 * Attention in which a query at position p sees the keys j <= p with
 * j < n_sink (the first tokens, which stay visible) or j > p - window (the
 * newest `window` keys, its own included):
 *   out_i = sum_j softmax_j(scale q_i . k_j) v_j,
 *   lse_i = log sum_j exp(scale q_i . k_j)        over the visible keys j.
 * The queries are the last rows of their sequence: query i of a sequence with
 * n queries and m keys sits at position p = m - n + i. So n = m is a prompt,
 * n < m a chunk of one, n = 1 a single decoded token. A row that sees nothing
 * (p < 0, or no keys) gives out 0 and lse -infinity. ("Attention Sinks 与 KV
 * Cache 淘汰策略" section 4.1: sinks plus a sliding window. With window =
 * n_recent + 1 these are the tokens that kvevict_decode_step of a
 * KVEVICT_SINK_WINDOW cache attends to: n_sink, the newest n_recent, and the
 * new one.)
 *   dtype:     KVEVICT_F32 or KVEVICT_BF16, of q, k, v and out. Sums, softmax
 *              statistics and lse are fp32. bf16 products run on the tcgen05
 *              tensor cores, the probabilities rounded to bf16 for the
 *              product with V; fp32 products on the CUDA cores in fp32.
 *   head_dim:  64 or 128. n_q_heads is a multiple of n_kv_heads, at most 64
 *              times it; query heads g*G .. g*G+G-1 share KV head g.
 *   Padded form (q_starts, k_starts NULL): q and out are
 *              [batch][n_q_heads][q_rows], k and v [batch][n_kv_heads][k_rows],
 *              in any strides; q_lens and kv_lens (device int32 [batch], or
 *              NULL: all rows) say how many rows of each sequence are real,
 *              the first ones; out and lse rows beyond q_lens are left as they
 *              were, and k and v rows beyond kv_lens may hold anything. max_q
 *              and max_k are ignored. lse is dense [batch][n_q_heads][q_rows].
 *   Packed form (q_starts and k_starts device int32 [batch + 1], ascending):
 *              sequence b owns the token rows q_starts[b] .. q_starts[b + 1] - 1
 *              of q, out and lse (q_rows of them in all) and k_starts[b] .. of
 *              k and v (k_rows in all); the sequence strides are ignored. No
 *              sequence has more than max_q queries (0: nothing is launched, and
 *              no start looked at); max_k, the most keys, only steers the launch.
 *              Rows outside every sequence are left as they were. lse is dense
 *              [q_rows][n_q_heads].
 *   out and lse must not overlap q, k or v.
 *   V rows that no query of the sequence sees may hold anything, infinities
 *              and NaN included; K likewise. Rows that one query sees and
 *              another does not must be finite for the other's sake.
 *   n_sink >= 0; window >= 1, or 0: no window (every key up to the query's
 *              position). scale > 0, or 0: 1 / sqrt(head_dim).
 *   lse:       NULL where it is not wanted.
 *   workspace: device, 256-byte aligned, at least
 *              kvevict_window_attention_workspace_bytes() bytes (0 for most
 *              prompts: then NULL). It is used when few rows attend to many
 *              keys: the keys are split over CTAs and the parts joined by a
 *              second kernel. Contents need not be kept or cleared; calls that
 *              may overlap on the GPU need one each.
 *   error_word: device uint32 that error bits are OR-ed into (BAD_LENGTH, and
 *              WAIT_TIMEOUT: a pipeline wait gave up, the results are not valid),
 *              or NULL: then into the device's (kvevict_operator_errors).
 */
typedef struct {
    int32_t dtype, head_dim, n_q_heads, n_kv_heads, batch, n_sink, window;
    int32_t max_q, max_k;
    float scale;
    int64_t q_rows, k_rows;
    const void *q, *k, *v;
    void *out;
    float *lse;
    int64_t q_stride[3], k_stride[3], v_stride[3], out_stride[3];
    const int32_t *q_starts, *k_starts, *q_lens, *kv_lens;
    void *workspace;
    size_t workspace_bytes;
    uint32_t *error_word;
} kvevict_attention_args;

/* INVALID_ARG for shapes, strides, pointers or alignments outside the above,
 * a workspace smaller than needed, or 2^30 rows and more. Nothing is launched
 * where there are no query rows. The workspace size does not look at pointers
 * or strides. */
int kvevict_window_attention_workspace_bytes(const kvevict_attention_args *a, size_t *bytes);
int kvevict_window_attention(const kvevict_attention_args *a, void *cuda_stream);

/*
 * The error bits that calls without an error_word have set on the current
 * device since the last time; waits for the device, and clears them. OK,
 * DEVICE where there are any, CUDA; INVALID_ARG for NULL. Not while a stream of
 * the device is being captured. */
int kvevict_operator_errors(uint32_t *device_error);

/*
 * Decode attention, one token of every sequence, over a prefix that all
 * sequences share (stored once) and a suffix of each sequence's own; every
 * query sees its whole prefix and suffix:
 *   out_b = sum over prefix and suffix keys j of softmax_j(scale q_b . k_j) v_j.
 * The prefix is read once for the whole batch (its products run over all
 * sequences' rows), the suffixes once each, in one launch; a second joins the
 * parts by their lse. ("Random Attention" summary, 方法: the prompt is kept
 * whole and only generated tokens are evicted; many traces of one prompt then
 * share it.) From kvevict_attention_args it takes the padded form with
 * q_rows = 1 (q [batch][n_q_heads][head_dim]; the token stride is ignored) and
 * k, v, k_rows, kv_lens as the suffixes (k_rows = 0: none); q_starts,
 * k_starts, q_lens, n_sink and window must be 0 or NULL. lse is dense
 * [batch][n_q_heads].
 *   k_prefix, v_prefix: [n_kv_heads][prefix_rows], strides (head, token) in
 *              elements; prefix_rows >= 0.
 *   workspace: as above, kvevict_shared_prefix_attention_workspace_bytes().
 */
typedef struct {
    kvevict_attention_args a;
    const void *k_prefix, *v_prefix;
    int64_t k_prefix_stride[2], v_prefix_stride[2];
    int64_t prefix_rows;
} kvevict_shared_prefix_args;

int kvevict_shared_prefix_attention_workspace_bytes(const kvevict_shared_prefix_args *a, size_t *bytes);
int kvevict_shared_prefix_attention(const kvevict_shared_prefix_args *a, void *cuda_stream);

/*
 * Rotary positions: every pair (a, b) of a head's first rotary_dim elements
 * turns by the angle t = pos * inv_freq[pair],
 *   a' = scale (a cos t - b sin t),   b' = scale (a sin t + b cos t),
 * and the other head_dim - rotary_dim elements are copied. Half layout: pair i
 * is (x[i], x[i + rotary_dim / 2]); interleaved: (x[2 i], x[2 i + 1]).
 * inverse = 1 turns by -t: with the same scale this is the gradient of the
 * forward call with respect to its input; with scale 1 it undoes it, and a
 * call with the difference of two positions moves a cached key from one to
 * the other.
 *   dtype:     KVEVICT_F32 or KVEVICT_BF16; computed in fp32.
 *   head_dim:  a multiple of 8, at most 1024; rotary_dim even, 2 .. head_dim.
 *   q, q_out:  [batch][n_q_heads][tokens], any strides (q_out's not 0);
 *              q_out may be q itself (with q's strides: in place), else must not
 *              overlap it. k, k_out likewise with n_k_heads; k NULL: queries only.
 *   positions: device, int64 (positions_64 = 1) or int32, element
 *              [b * pos_stride[0] + token * pos_stride[1]]; any value,
 *              negative ones too. NULL: pos_start + token for every sequence.
 *   inv_freq:  device fp64 [rotary_dim / 2], radians per position, finite.
 *              The angle is formed as a 64-bit binary fraction of a turn, the
 *              frequency's (from an fp64 product) times the position modulo 2^64.
 *              Its error is below 2^-52 |inv_freq / 2 pi| + 2^-64 turns times
 *              |pos|: for inv_freq <= 1 less than 2^-54 turns a position.
 */
typedef struct {
    int32_t dtype, head_dim, rotary_dim, interleaved, inverse, positions_64;
    int32_t n_q_heads, n_k_heads;
    int64_t batch, tokens;
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_stride[3], q_out_stride[3], k_stride[3], k_out_stride[3];
    const void *positions;
    int64_t pos_stride[2], pos_start;
    const double *inv_freq;
    float scale;
} kvevict_rotary_args;

int kvevict_rotary(const kvevict_rotary_args *a, void *cuda_stream);

/*
 * The root-mean-square norm of every head, then its rotary positions, in one pass:
 *   y = x / sqrt(mean_i x_i^2 + eps) * weight,   out = y turned as by kvevict_rotary,
 * computed in fp32 and rounded once. The arguments are kvevict_rotary's with
 * inverse = 0; rotary_dim may be 0 (inv_freq and positions then NULL): norms only.
 *   q_weight, k_weight: [head_dim] in dtype, contiguous, 16-byte aligned;
 *              k_weight NULL exactly where k is.
 *   eps:       finite, >= 0. (With eps = 0 a head of zeros gives NaN.)
 */
typedef struct {
    kvevict_rotary_args r;
    const void *q_weight, *k_weight;
    float eps;
} kvevict_norm_rotary_args;

int kvevict_norm_rotary(const kvevict_norm_rotary_args *a, void *cuda_stream);

/*
 * With a handle: the prompt of an empty layer, attended and appended in one
 * call. out (and lse, where not NULL) get the prompt's attention under the
 * tokens that the policy keeps in view -- KVEVICT_SINK_WINDOW: the first n_sink
 * and the newest n_recent + 1, which is what kvevict_decode_step would have
 * attended to token by token; the other policies: every earlier token -- by
 * kvevict_window_attention; then the prompt enters the cache as
 * kvevict_prefill(h, layer, K, V, n_tokens) puts it there.
 *   Q, out: device, [batch][n_q_heads][n_tokens][head_dim]; K, V: device,
 *           [batch][n_kv_heads][n_tokens][head_dim]; lse: fp32
 *           [batch][n_q_heads][n_tokens] or NULL;
 *   workspace: as kvevict_prefill_attend_workspace_bytes() says (NULL where 0).
 * On the handle's stream; error bits in the handle's error word. INVALID_ARG
 * for n_tokens outside 1 .. 2^30 - 1, null or misaligned pointers or a short
 * workspace; STATE if the layer is out of range, already holds tokens or has
 * decoded; CAPACITY for a KVEVICT_RANDOM prompt beyond max_prompt. */
int kvevict_prefill_attend_workspace_bytes(kvevict_t h, int n_tokens, size_t *bytes);
int kvevict_prefill_attend(kvevict_t h, int layer, const void *Q, const void *K, const void *V, int n_tokens, void *out,
                           float *lse, void *workspace, size_t workspace_bytes);

/*
 * kvevict_decode_step over the layer's cache and, in front of it, a prefix that
 * all sequences share: one softmax over prefix, retained tokens and the new
 * token. The cache does what the step always does (it appends, evicts and
 * counts positions as if there were no prefix); only the attention is joined
 * with the prefix's, three launches in all. For the policies that keep no
 * scores (KVEVICT_SINK_WINDOW, KVEVICT_RANDOM): scores would be attention
 * probabilities, which the prefix takes a share of.
 *   q, k_new, v_new, out: as kvevict_decode_step; k_prefix, v_prefix: device,
 *   [n_kv_heads][prefix_rows][head_dim], NULL where prefix_rows is 0;
 *   workspace: kvevict_decode_step_shared_workspace_bytes(), 256-byte aligned;
 *   calls that may overlap on the GPU need one each.
 * INVALID_ARG for other policies, a negative prefix_rows, null or misaligned
 * pointers or a short workspace; STATE as kvevict_decode_step. */
int kvevict_decode_step_shared_workspace_bytes(kvevict_t h, int prefix_rows, size_t *bytes);
int kvevict_decode_step_shared(kvevict_t h, int layer, const void *q, const void *k_new, const void *v_new,
                               const void *k_prefix, const void *v_prefix, int prefix_rows, void *out, void *workspace,
                               size_t workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* KVEVICT_OPS_H */
