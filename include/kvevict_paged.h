/*
 * kvevict_paged.h -- a paged cache of keys and values on plain tensors, in
 * libkvevict.so: new tokens into their sequences' pages (keys turned by their
 * positions on the way), attention of a few tokens of every sequence over its
 * pages, and whole sequences out of their pages for the attention of a prompt's
 * next chunk (kvevict_window_attention). Pages hold the keys' own type or 4 bits
 * a channel.
 *
 * The calls follow kvevict_ops.h: one argument struct, the caller's stream, the
 * tensors' device the current one; argument errors are returned before anything
 * is launched, and what the GPU finds wrong sets bits of an error word. No call
 * allocates device memory or waits for the GPU; each can be captured in a CUDA
 * graph, lengths and tables then being read anew by every replay.
 */
#ifndef KVEVICT_PAGED_H
#define KVEVICT_PAGED_H

#include "kvevict_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Page type: 4 bits a channel. A page holds `page_size` tokens of each KV head.
 * Every 32 channels of a token and head are a group with a base and a step in
 * bf16; channel x of the group stands for base + (code - 8) * step, code 0 .. 15
 * (a group with an infinity or NaN in it stands for NaN).
 *   base = bf16(8/15 hi + 7/15 lo), hi and lo the group's largest and smallest;
 *   step = max((hi - base) / 7, (base - lo) / 8), rounded up to bf16;
 *   code = round((x - base) / step) + 8, ties to even, in 0 .. 15 (8 where step is 0).
 * (The ends of a group that reaches within a 64th of the type's largest number may
 * stand for an infinity, as the step is rounded up.)
 * A page's block for one head, [page_size * 5 head_dim / 8] bytes, contiguous:
 * first the codes [page_size][head_dim / 2], then [page_size][head_dim / 32]
 * groups of (base, step). Channel 32 j + 4 g + i of a row (j the group, g 0 .. 7,
 * i 0 .. 3) is in byte (head_dim / 16) g + 2 j + i / 2, the low half for even i:
 * the four channels of one g in all groups are neighbours, which is what a lane of
 * a matrix instruction takes. */
#define KVEVICT_Q4 2

/* A block table's entry that a token needs is no page (negative, or n_pages and
 * more): the new token was dropped, the page's keys were not seen, its rows left
 * as they were. */
#define KVEVICT_DEV_BAD_PAGE 0x20u

/*
 *   dtype:     KVEVICT_F32 or KVEVICT_BF16, of everything that is not a page.
 *   page_dtype: dtype, or KVEVICT_Q4.
 *   head_dim:  64 or 128. page_size: 16, 32, 64, 128 or 256.
 *   k_pages, v_pages: [n_pages][n_kv_heads][page_size][head_dim], 16-byte
 *              aligned, strides (page, head, token) positive multiples of 16 bytes,
 *              in elements. KVEVICT_Q4: strides (page, head) in bytes, multiples of
 *              16; the token stride is ignored (a head's block is contiguous).
 *   block_table: device int32 [batch][table_width], rows table_stride entries
 *              apart: token i of sequence b is row i % page_size of page
 *              block_table[b][i / page_size]. Entries that no token of a call needs
 *              (behind the length, before the window) may hold anything. A table
 *              row has room for fewer than 2^30 tokens.
 *   kv_lens:   device int32 [batch]: tokens of each sequence, the new ones of
 *              this call included.
 *   New tokens (queries, keys, values) are [tokens][heads][head_dim], strides
 *              (head, token): sequence b owns the rows starts[b] .. starts[b + 1] - 1
 *              (device int32 [batch + 1], ascending), or, starts NULL, tokens /
 *              batch rows each. They are the last of their sequence: token i of n
 *              is at kv_lens[b] - n + i.
 *   error_word: as in kvevict_attention_args.
 */
typedef struct {
    int32_t dtype, page_dtype, head_dim, n_kv_heads, page_size, batch, table_width, n_pages;
    void *k_pages, *v_pages;
    int64_t k_page_stride[3], v_page_stride[3];
    const int32_t *block_table;
    int64_t table_stride;
    const int32_t *kv_lens;
    uint32_t *error_word;
} kvevict_paged_cache;

/*
 * Writes the new tokens' keys and values into their pages; keys with rotary
 * positions as kvevict_rotary gives them (computed in fp32 and rounded once, to
 * the pages' type) where rotary_dim > 0.
 *   k, v:      [tokens][n_kv_heads][head_dim], strides (head, token) multiples of
 *              16 bytes, 0 included.
 *   positions: device int32 or int64 (positions_64), token t at t * pos_stride;
 *              NULL: the token's place in its sequence.
 *   rotary_dim, interleaved, inv_freq, scale: as in kvevict_rotary; rotary_dim 0:
 *              none of them is looked at.
 * Tokens before the first place or behind the table (BAD_LENGTH) and in no page
 * (BAD_PAGE) are dropped, and so is every sequence of starts that go back from the
 * first such on. k and v must not overlap the pages. Two tokens that the tables put
 * in one place, or a call that reads the pages at the same time, give undefined
 * contents there. Other rows of the pages are left as they were.
 */
typedef struct {
    kvevict_paged_cache c;
    const void *k, *v;
    int64_t k_stride[2], v_stride[2];
    int64_t tokens;
    const int32_t *starts;
    const double *inv_freq;
    const void *positions;
    int64_t pos_stride;
    int32_t positions_64, rotary_dim, interleaved;
    float scale;
} kvevict_paged_append_args;

int kvevict_paged_append(const kvevict_paged_append_args *a, void *cuda_stream);

/*
 * Copies whole sequences out of their pages, as values of `dtype` (4 bits: base +
 * (code - 8) * step, rounded once).
 *   k_out, v_out: padded (k_starts NULL) [batch][n_kv_heads][rows][head_dim], or
 *              packed [rows][n_kv_heads][head_dim] with sequence b in the rows
 *              k_starts[b] .. k_starts[b + 1] - 1 (device int32 [batch + 1],
 *              ascending); strides (sequence, head, token) positive multiples of 16
 *              bytes. Rows behind a sequence's kv_lens, or outside the starts, are
 *              left as they were; a sequence longer than its rows or its table is
 *              cut (BAD_LENGTH; rows = 0: nothing is launched, and no length looked at).
 */
typedef struct {
    kvevict_paged_cache c;
    void *k_out, *v_out;
    int64_t k_out_stride[3], v_out_stride[3];
    int64_t rows;
    const int32_t *k_starts;
} kvevict_paged_gather_args;

int kvevict_paged_gather(const kvevict_paged_gather_args *a, void *cuda_stream);

/*
 * Attention of the new tokens over their sequences' pages, the mask that of
 * kvevict_window_attention (n_sink first keys, the newest `window`; 0: all up to
 * the query's own place), which also says what a row without keys gives.
 *   q, out:    [tokens][n_q_heads][head_dim], strides (head, token) positive
 *              multiples of 16 bytes; n_q_heads a multiple of n_kv_heads, at most
 *              64 times it. A sequence's new tokens times n_q_heads / n_kv_heads:
 *              fewer than 2^31 - 16. lse: dense fp32 [tokens][n_q_heads] or NULL.
 *              out and lse must not overlap q or the pages.
 *   Sums, softmax statistics and lse are fp32. bf16 queries take the tensor cores,
 *              the probabilities (4 bits: times the step) rounded to bf16 for the
 *              product with V; over 4 bits steps of V below 2^-50 lose precision,
 *              and bases of V above 2^60 or queries of 2^118 may overflow. fp32 ones
 *              take the CUDA cores, in fp32.
 *   max_q:     with starts: no sequence has more new tokens (0: nothing is launched,
 *              and no start looked at). max_k: the most keys of a sequence, or 0:
 *              as many as the table holds; it only steers the launch.
 *   V rows that no query of the sequence sees may hold anything; of bf16 and fp32
 *              pages, rows that one query sees and another does not must be finite
 *              for the other's sake.
 *   workspace: device, 256-byte aligned, at least
 *              kvevict_paged_attention_workspace_bytes() bytes; it need not be kept
 *              or cleared; calls that may overlap on the GPU need one each.
 * A length beyond the table is clamped to it (BAD_LENGTH).
 */
typedef struct {
    kvevict_paged_cache c;
    int32_t n_q_heads, n_sink, window, max_q, max_k;
    float scale;
    int64_t tokens;
    const void *q;
    void *out;
    float *lse;
    int64_t q_stride[2], out_stride[2];
    const int32_t *q_starts;
    void *workspace;
    size_t workspace_bytes;
} kvevict_paged_attention_args;

int kvevict_paged_attention_workspace_bytes(const kvevict_paged_attention_args *a, size_t *bytes);
int kvevict_paged_attention(const kvevict_paged_attention_args *a, void *cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* KVEVICT_PAGED_H */
