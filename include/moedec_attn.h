/*
 * moedec_attn.h - C ABI of libmoedec, second part: the attention half of a
 * decode layer on the number formats of moedec.h (codes of 8, 4 or 2 bits with
 * one fp32 scale per row), on AMD Instinct MI355X (gfx950).
 *
 *   dense_linear_q4 / _q8 / _q2   product with a packed weight; bias, activation
 *                                 and residual in its epilogue
 *   kv4_append, kv4_read          write / read back the paged cache that holds
 *                                 keys and values in 4 bits
 *   kv4_attention                 attention over that cache: single tokens,
 *                                 drafts verified together, chunks of prompts
 *   kv4_reserve, kv4_fork,        the cache's pages: room for new tokens (with
 *   kv4_truncate, kv4_compact     copy on write), branches, freeing, compaction
 *
 * Conventions are those of moedec.h: device pointers, caller-owned memory,
 * work enqueued on `stream`, nothing allocated, no synchronisation, arguments
 * validated on the host before anything is enqueued, MOEDEC_* status codes.
 * There is no mutable global state.  Every call may be captured into a graph;
 * the page calls read and write their counts on the device, so a captured
 * step may be replayed as the sequences grow.  Results are deterministic.
 */
#ifndef MOEDEC_ATTN_H
#define MOEDEC_ATTN_H

#include <stdint.h>

#include "moedec.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types of activations */
#define MOEDEC_F32 0
#define MOEDEC_F16 1
#define MOEDEC_BF16 2

/* activations of dense_linear_q* (v = the product with its bias) */
#define MOEDEC_ACT_NONE 0   /* v */
#define MOEDEC_ACT_SILU 1   /* v / (1 + e^-v) */
#define MOEDEC_ACT_GELU 2   /* v/2 * (1 + erf(v / sqrt 2)) */
#define MOEDEC_ACT_RELU 3   /* max(v, 0); a NaN stays */

/*
 * y[t][n] = act(scale[n] * sum_k x[t][k] * code[n][k] + bias[n]) + residual[t][n]
 *   x        : [T] rows of K elements of `dtype`, ldx elements apart
 *   w        : uint8 [N, K*bits/8] packed codes in the layout of moe_pack_q*
 *   scale    : fp32 [N]; bias: fp32 [N] or NULL
 *   residual : [T] rows of N elements of `dtype`, ldr apart, or NULL; may be y
 *              itself (with ldr == ldy), else must not overlap it
 *   y        : [T] rows of N elements of `dtype`, ldy apart; must not overlap x
 *   workspace: dense_linear_workspace(...) bytes of device memory,
 *              16-byte aligned (NULL when that is 0); calls that may run at
 *              the same time need separate ones
 * Products with fp16 and bf16 activations are exact (every activation of a row
 * enters as an fp16 multiple of one power of two, so elements smaller than
 * 2^-23 of the row's largest lose bits), fp32 activations enter with about 22
 * bits; sums are fp32 (with 16-bit activations within about 1e-5 of their rms,
 * far below the rounding of y); y is rounded once.  A row of x that holds a NaN
 * or an infinity gives unspecified values in that row of y only.
 * T == 0 is a no-op.  dense_linear_workspace gives -1 for sizes that are refused.
 * Requires K a positive multiple of 128/bits, N >= 1,
 * x and w 16-byte aligned, ldx*element size a multiple of 16, ldx >= K,
 * ldr, ldy >= N, no overlap but the one above (INVALID_ARG; rows of one stride
 * may interleave, as columns of one buffer do); K <= 65536, T and N < 2^24 and T*N/512 < 2^31
 * (UNSUPPORTED).
 */
int64_t dense_linear_workspace(int bits, int dtype, int64_t T, int64_t K, int64_t N);
int dense_linear_q4(const void* x, int dtype, int64_t ldx, const uint8_t* w, const float* scale, const float* bias,
                    int act, const void* residual, int64_t ldr, void* y, int64_t ldy, int64_t T, int64_t K, int64_t N,
                    void* workspace, int64_t workspace_bytes, void* stream);
int dense_linear_q8(const void* x, int dtype, int64_t ldx, const uint8_t* w, const float* scale, const float* bias,
                    int act, const void* residual, int64_t ldr, void* y, int64_t ldy, int64_t T, int64_t K, int64_t N,
                    void* workspace, int64_t workspace_bytes, void* stream);
int dense_linear_q2(const void* x, int dtype, int64_t ldx, const uint8_t* w, const float* scale, const float* bias,
                    int act, const void* residual, int64_t ldr, void* y, int64_t ldy, int64_t T, int64_t K, int64_t N,
                    void* workspace, int64_t workspace_bytes, void* stream);

/*
 * A paged cache of keys and values in 4 bits.  Host struct; pointers are device
 * memory of the caller.
 *   data  : uint8 [layers][n_pages][kv_heads][page_tokens*(head_dim + 8)],
 *           16-byte aligned.  A page holds page_tokens positions of one
 *           sequence (or of several that share them); every (token, head) row of
 *           keys and of values is head_dim codes with one fp32 scale by the rule
 *           of moe_quantize_rows_q4.  The order of the codes inside a page is the
 *           kernels' own: read it with kv4_read.
 *   table : int32 [n_seqs][max_pages]; table[s][i] is the page with positions
 *           i*page_tokens .. of sequence s, defined for i < ceil(len[s] /
 *           page_tokens) only
 *   len   : int32 [n_seqs] tokens held (0: the slot is empty)
 *   ref   : int32 [n_pages] sequences that hold the page (0: free), 16-byte aligned
 * One table serves all layers.  A fresh cache is len = 0 and ref = 0
 * everywhere; data and table need no initial values.  The page calls keep table,
 * len and ref; a caller that keeps pages itself may write them instead.
 * A page index outside [0, n_pages) in the table is taken as positions that are
 * not there: nothing is written to them, no query sees them, kv4_read gives
 * zeros.
 * Limits: page_tokens 32, 64 or 128; head_dim 64, 128, 192 or 256; kv_heads <=
 * 1024; n_seqs <= KV4_MAX_SEQS; n_pages <= 2^24; max_pages*page_tokens <=
 * 2^30 (else UNSUPPORTED).
 */
#define KV4_MAX_SEQS 1024
typedef struct kv4_cache {
    int32_t layers, n_pages, page_tokens, kv_heads, head_dim, n_seqs, max_pages;
    uint8_t* data;
    int32_t* table;
    int32_t* len;
    int32_t* ref;
} kv4_cache;

/*
 * The rows of a call: q_start is int32 [n_seqs + 1], not descending; rows
 * q_start[s] .. q_start[s+1]-1 of the activations belong to sequence s (none:
 * it takes no part).  granted is int32 [n_seqs] or NULL: only the first
 * granted[s] of these rows count (the output of kv4_reserve, so a sequence that
 * got no room is left alone).  With m counting rows, they are the sequence's
 * last m positions, len[s]-m .. len[s]-1: reserve (or set len) first.  Rows
 * outside every sequence are left as they are; a q_start above `rows` is taken
 * as `rows`.
 *
 * kv4_append writes keys and values:
 *   k, v : [rows][kv_heads][head_dim] of `dtype`, row strides ldk, ldv elements
 * The codes are those of moe_quantize_rows_q4 on the rows converted to fp32
 * (bit for bit).  A page written here must belong to one sequence only.
 * kv4_read gives the values back (code * scale, rounded once to dtype):
 *   first : int32 [n_seqs]; row q_start[s]+i is position first[s]+i of sequence
 *           s; positions outside [0, len[s]) give zeros
 * Row strides >= kv_heads*head_dim; pointers 16-byte aligned, row strides a
 * multiple of 16 bytes (INVALID_ARG).  rows == 0 is a no-op; rows < 2^24.
 */
int kv4_append(const kv4_cache* cache, int layer, const void* k, int64_t ldk, const void* v, int64_t ldv, int dtype,
               int64_t rows, const int32_t* q_start, const int32_t* granted, void* stream);
int kv4_read(const kv4_cache* cache, int layer, const int32_t* first, const int32_t* q_start, int64_t rows, void* k,
             int64_t ldk, void* v, int64_t ldv, int dtype, void* stream);

/*
 * out[r][h] = sum_j p_j * v_j, p = softmax_j(scale * q[r][h] . k_j), over the
 * keys j of the row's sequence with j <= pos(r) and, if window > 0, j > pos(r) -
 * window; head h reads key/value head h / (heads / kv_heads).
 *   q, out  : [rows][heads][head_dim] of `dtype`, row strides ldq, ldo; out must
 *             not overlap q (INVALID_ARG; columns of one buffer may interleave)
 *   lse     : fp32 [rows][heads] or NULL; the natural log of sum_j
 *             exp(scale * q . k_j)
 *   max_len : an upper bound of the lengths as far as the caller knows it
 *             (>= 1); it sizes the split of the keys over workgroups only, longer
 *             sequences are still right
 *   workspace : kv4_attention_workspace(...) bytes of device memory, 16-byte
 *             aligned (NULL when that is 0); calls that may run at the same time
 *             need separate ones
 * A row that sees no key (outside its granted count, positions below 0, an empty
 * sequence) gives zeros and lse = -inf.  What masked positions hold (stale codes,
 * infinite or NaN scales) never reaches a result.  Queries enter as for
 * dense_linear_q*, probabilities as fp16 (with fp16 or bf16 queries) or about 22
 * bits (fp32) against the exact codes; scores, softmax and sums are fp32.
 * heads a multiple of kv_heads, heads <= 16384, scale finite, window >= 0.
 * kv4_attention_workspace returns -1 for arguments that kv4_attention refuses.
 */
int64_t kv4_attention_workspace(const kv4_cache* cache, int64_t rows, int heads, int64_t max_len);
int kv4_attention(const kv4_cache* cache, int layer, const void* q, int64_t ldq, int dtype, int64_t rows, int heads,
                  const int32_t* q_start, const int32_t* granted, float scale, int window, int64_t max_len, void* out,
                  int64_t ldo, float* lse, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Room for new tokens: len[s] += n_new[s] (negative counts as 0), with pages for
 * them.  Sequences are served in index order; the new pages are the free ones of
 * lowest index, in order.  If a sequence's last page is partly filled and other
 * sequences hold it too, the sequence first gets a copy of it in all layers (of
 * those that share it and grow in this call, the last one keeps the page).  A
 * sequence that max_pages cannot hold is refused; the first other one that the
 * free pages cannot serve is refused together with every later one that asks.
 * granted[s] = n_new[s], or 0 (and nothing changed) for a refused one.
 *   workspace : int32 [2*n_seqs + 1]
 */
int kv4_reserve(const kv4_cache* cache, const int32_t* n_new, int32_t* granted, int32_t* workspace, void* stream);

/*
 * Branches: slot dst[i] becomes the first n_tokens[i] tokens (NULL: all) of
 * sequence src[i], sharing its pages; n <= KV4_MAX_SEQS.  ok[i] = 1, or 0 with
 * nothing changed if an index is out of range, dst[i] is not empty before the
 * call or stands earlier in the list, or n_tokens[i] is outside [0, len[src[i]]].
 * All entries read the state before the call.
 */
int kv4_fork(const kv4_cache* cache, int n, const int32_t* src, const int32_t* dst, const int32_t* n_tokens,
             int32_t* ok, void* stream);

/*
 * Freeing: sequence s keeps its first new_len[s] tokens (negative, or not below
 * len[s]: left alone; 0 frees the slot); pages that no sequence holds any more
 * become free.
 */
int kv4_truncate(const kv4_cache* cache, const int32_t* new_len, void* stream);

/*
 * Compaction: with n live pages, the live pages of index >= n move, in ascending
 * order, to the free pages of index < n in ascending order (all layers); table
 * and ref follow.  Table entries of held pages outside [0, n_pages) stay.
 *   remap  : int32 [n_pages]; the new index of every page, -1 for free ones
 *   n_live : int32 [1]
 *   workspace : int32 [n_pages + 1]
 */
int kv4_compact(const kv4_cache* cache, int32_t* remap, int32_t* n_live, int32_t* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOEDEC_ATTN_H */
