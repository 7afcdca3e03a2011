/*
 * bsa_seq.h -- C ABI of libbsa.so for token sequences: the attention that a
 * model needs next to its block-sparse video attention when tokens come as
 * packed sequences of different lengths (text, audio and reference
 * conditioning, causal generation clip by clip) or one at a time (serving
 * from a key-value cache).
 *
 *   training, prompts   bsa_packed_attn_fwd, bsa_packed_attn_bwd
 *   serving             bsa_kv_append (rotate, write to the paged cache),
 *                       bsa_paged_attn_decode (one new token over the cache)
 *
 * Conventions are those of bsa.h: device memory is caller-owned, every
 * argument the host can see is validated before anything is launched, calls
 * are asynchronous on `stream` (a cudaStream_t) and run on the current
 * device, device-side errors reach dev_status (or, when it is NULL, the
 * library's own word, bsa_take_default_status), and no call allocates
 * memory.
 *
 * Tensors.  A [rows, heads, head_dim] tensor is given by its pointer
 * (16-byte aligned) and two element strides, stride_n (row) and stride_h
 * (head), multiples of 8; head_dim is contiguous.  A stride of an axis of
 * extent 1 is ignored.  bf16 or fp16, all tensors of a call alike.
 * Query head h uses key-value head h / (heads / kv_heads).
 *
 * Packed sequences.  cu[0..n_seqs] (int32, device) are ascending row
 * offsets: sequence b owns rows cu[b] .. cu[b+1]-1, possibly none.  Rows
 * behind cu[n_seqs] (or in front of cu[0]) are neither read as data nor
 * written and may hold anything, NaN included; rows of a sequence must be
 * finite.  Offsets that descend or leave the tensor are reported as
 * BSA_ERR_INVALID_ARG through the status word and read as an empty sequence;
 * where they make sequences overlap, or among more than 32 sequences, they may
 * leave rows of others unwritten or written twice.  At most 2^30 rows a tensor.
 *
 * Paged cache.  k_cache and v_cache share the strides (stride_page,
 * stride_token, stride_head), element strides that are multiples of 8, of a
 * [n_pages, page_size, kv_heads, head_dim] view, so that token-major and
 * head-major pages both fit.  block_table (int32, device) has n_seqs rows of
 * table_width entries, table_stride apart: position p of sequence b lies in
 * page block_table[b][p / page_size] at token p % page_size.  Entries behind
 * a sequence's last page are not read.  seq_lens (int32, device) holds the
 * cached tokens of each sequence INCLUDING those of the current call.
 */
#ifndef BSA_SEQ_H
#define BSA_SEQ_H

#include "bsa.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum bsa_dtype { BSA_DTYPE_BF16 = 0, BSA_DTYPE_FP16 = 1 } bsa_dtype;

/* What the calls of one attention layer share. */
typedef struct bsa_seq_problem {
  int32_t heads;        /* query heads, 1..65535 */
  int32_t kv_heads;     /* divides heads */
  int32_t head_dim;     /* 64 or 128 */
  int32_t dtype;        /* a bsa_dtype */
  int32_t causal;       /* packed attention: 1 causal, 0 every key is seen */
  float softmax_scale;  /* finite and > 0 */
} bsa_seq_problem;

/* A [rows, heads, head_dim] tensor: its data and element strides. */
typedef struct bsa_rows {
  void* data;
  int64_t stride_n, stride_h;
} bsa_rows;

/* A paged cache and the pages of each sequence. */
typedef struct bsa_paged_cache {
  void *k, *v;
  int64_t stride_page, stride_token, stride_head;
  int64_t n_pages, page_size;
  const int32_t* block_table;
  int64_t table_stride, table_width;
} bsa_paged_cache;

/* Arguments of the packed calls; the forward reads q .. lse. */
typedef struct bsa_packed_args {
  int64_t n_seqs, total_q, total_k;
  bsa_rows q, k, v, o;
  const int32_t *cu_q, *cu_k;
  float* lse;
  bsa_rows dout, dq, dk, dv;
  void* workspace;
  size_t ws_bytes;
} bsa_packed_args;

typedef struct bsa_append_args {
  int64_t n_seqs, n_tokens;
  bsa_rows k, v;
  bsa_paged_cache cache;
  const int32_t *cu_new, *seq_lens;
  const float* rope;
  int64_t rope_n, rot_dim, interleaved;
  const int32_t* rope_rows;
  bsa_rows q, q_out, k_out;
} bsa_append_args;

typedef struct bsa_decode_args {
  int64_t n_seqs;
  bsa_rows q;
  bsa_paged_cache cache;
  const int32_t* seq_lens;
  bsa_rows o;
  void* workspace;
  size_t ws_bytes;
} bsa_decode_args;

/* Attention over packed sequences: row i of sequence b (Lq queries, Lk keys)
 * sees keys j < lim,
 *   causal      lim = min(Lk, max(0, i + 1 + Lk - Lq)): the last query sees
 *               every key, so queries may be the last part of a longer text
 *   otherwise   lim = Lk (cross attention, or an encoder when cu_q == cu_k)
 * and o = sum_j softmax_j(softmax_scale q.k_j) v_j; a row that sees nothing
 * gives 0.
 *   q, o        [total_q, heads, head_dim];  k, v [total_k, kv_heads, head_dim];
 *               the strides of q, k and v must not be 0 (no broadcast views)
 *   cu_q, cu_k  int32 [n_seqs + 1]
 *   o           must not overlap an input
 *   lse         fp32 [heads, total_q] or NULL: each row's log-sum-exp in the
 *               exp2 domain, log2 sum_j exp2(softmax_scale log2(e) q.k_j)
 *               (-inf for a row that sees nothing), for the backward
 * Scores, statistics and outputs accumulate in fp32; the probabilities are
 * rounded to the element type for their product with V. */
bsa_status bsa_packed_attn_fwd(const bsa_seq_problem* prob, const bsa_packed_args* args,
                               int32_t* dev_status, void* stream);

/* Bytes of bsa_packed_attn_bwd's workspace (row statistics, in fp16 the largest
 * norms of each sequence).  Host only. */
bsa_status bsa_query_packed_bwd_workspace(const bsa_seq_problem* prob, int32_t n_seqs,
                                          int64_t total_q, size_t* bytes);

/* Gradients of bsa_packed_attn_fwd:
 *   dV = P^T dO,  dP = dO V^T,  D_i = sum_j P_ij dP_ij,  dS = P * (dP - D),
 *   dQ = softmax_scale dS K,  dK = softmax_scale dS^T Q,
 * (D is rowsum(dO * O), and taken as that from the rounded o for query tiles
 * that see more than 1,024 keys), dK and dV summed over the query heads of
 * their kv head; P is recomputed from lse.  Every row of a sequence is written (0 where nothing was seen),
 * rows no sequence owns are left as they were.  Sums are fp32, in a fixed
 * order without atomics, so gradients do not vary from run to run; P and dS
 * are rounded to the element type for their products (in fp16 with scales
 * that keep them in its range, taken for each sequence from its own rows).
 *   q, k, v, cu_q, cu_k   the forward's
 *   o, lse                its results;  dout the gradient of o, [total_q,
 *                         heads, head_dim], strides not 0
 *   dq, dk, dv            shaped as q, k, v; must not overlap any input
 *   workspace             caller-owned, 16-byte aligned, ws_bytes at least
 *                         bsa_query_packed_bwd_workspace; holds nothing
 *                         between calls.  Calls that overlap on the GPU need
 *                         one each. */
bsa_status bsa_packed_attn_bwd(const bsa_seq_problem* prob, const bsa_packed_args* args,
                               int32_t* dev_status, void* stream);

/* Append new keys and values to a paged cache, rotating keys (and queries)
 * on the way.  Token t of the packed [n_tokens, ...] inputs belongs to the
 * sequence b with cu_new[b] <= t < cu_new[b+1]; its position is
 *   p = seq_lens[b] - (cu_new[b+1] - cu_new[b]) + (t - cu_new[b]).
 * With a rotation table, row r = rope_rows[t] (or p when rope_rows is NULL)
 * of rope holds cos in its first rot_dim/2 entries and sin in the others;
 * channel pairs (x1, x2) of the first rot_dim channels become
 *   (x1 cos - x2 sin, x2 cos + x1 sin),  computed in fp32 and rounded once,
 * pairs being (i, i + rot_dim/2), or (2i, 2i+1) when interleaved.  The other
 * channels and V are copied.
 *   k, v          [n_tokens, kv_heads, head_dim]
 *   cu_new        int32 [n_seqs + 1], seq_lens int32 [n_seqs]
 *   rope          fp32 [rope_n, rot_dim] contiguous, 16-byte aligned, or NULL
 *                 (nothing is rotated); rot_dim a multiple of 16 up to head_dim
 *   rope_rows     int32 [n_tokens] or NULL
 *   q, q_out      [n_tokens, heads, head_dim] or both NULL; q_out may be q
 *   k_out         the rotated keys as a dense [n_tokens, kv_heads, head_dim]
 *                 tensor, for the prompt's own attention, or NULL; may be k
 * A token whose position, table entry or rotation row is out of range is
 * reported as BSA_ERR_INVALID_ARG through the status word and none of its
 * outputs are written.  Two tokens must not share a cache slot (sequences
 * may share pages they do not write). */
bsa_status bsa_kv_append(const bsa_seq_problem* prob, const bsa_append_args* args,
                         int32_t* dev_status, void* stream);

/* Bytes of bsa_paged_attn_decode's workspace; the same for every batch.
 * Host only. */
bsa_status bsa_query_decode_workspace(const bsa_seq_problem* prob, size_t* bytes);

/* Attention of one new token per sequence over the paged cache:
 *   o[b, h] = softmax_p(softmax_scale q[b, h] . K[p]) V[p],  p < seq_lens[b].
 * A sequence of length 0 gives 0.  Cache slots at or behind seq_lens[b] may
 * hold anything.  The keys of the whole batch are dealt evenly over the SMs
 * whatever the lengths; parts of a sequence are joined in a fixed order, so
 * results do not vary from run to run.
 *   q, o          [n_seqs, heads, head_dim]
 *   workspace     caller-owned, 16-byte aligned, ws_bytes at least
 *                 bsa_query_decode_workspace; holds nothing between calls.
 *                 Calls that overlap on the GPU need one each.
 * A length beyond the table's reach (or negative) and a page outside the
 * cache are reported as BSA_ERR_INVALID_ARG through the status word; the
 * length is clamped, such a page's keys are read as zeros, and the
 * sequence's output is then meaningless. */
bsa_status bsa_paged_attn_decode(const bsa_seq_problem* prob, const bsa_decode_args* args,
                                 int32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* BSA_SEQ_H */
