/*
 * mk_ops.h -- operators beside the decode step, over its paged K/V pools and
 * its logits: what a sequence needs to advance by more than one greedy token
 * per step.
 *
 *   mk_kv_append    K and V of any number of new tokens into the pools, with
 *                   the rotation applied on the way (Q rotated alongside)
 *   mk_tree_attn    attention of those tokens over the pools: a tree of
 *                   drafted tokens (a bit mask per token) or a causal run
 *   mk_kv_commit    the accepted path of a drafted tree moved to the head of
 *                   the drafted slots, in every layer
 *   mk_beam_select  one step of beam search: the best continuations over
 *                   beams x vocabulary
 *   mk_beam_reorder the beams' block tables and open pages following their
 *                   parents
 *
 * The conventions are mk.h's: device memory is the caller's, nothing is
 * allocated on the device, calls are asynchronous on `stream` and can be
 * captured into a graph, a bad argument returns MK_ERR_ARG before anything is
 * launched (mk_last_error()).  The tensors, the stream and the current device
 * have to be of one device; an array's address is a multiple of its elements'
 * size.  The arrays and workspaces that a call writes lie apart from its other
 * arguments and from the pools (an overlap is refused, but where q_out is q);
 * the K, V and Q of an append are none of the pool rows that it writes.
 * Workspaces need no initialisation and hold nothing between calls; calls (and
 * replays of captured calls) that can overlap in time need a workspace each.
 *
 * Values in device memory are checked on the device.  A call never reads or
 * writes outside the arrays it was given: what a value out of range would
 * touch is left out (each call says what) and recorded in `status`, device
 * uint32 [8], zeroed by the caller, which keeps the first record until the
 * caller zeroes it again; NULL: not recorded.  mk_check_status reads it.
 *
 * A sequence's slot s is row s % page_size of page block_tables[b][s /
 * page_size].  Two sequences may share pages that no call writes.
 */
#ifndef MK_OPS_H
#define MK_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "mk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MK_BF16 0
#define MK_F32 1

/* The pools as mk_decode_step takes them: bf16 [n_layers][num_pages][n_kv]
 * [page_size][head_dim].  head_dim 64 or 128; page_size a power of two from
 * 16 to 256; the pools 16-byte aligned; num_pages * n_kv * page_size below
 * 2^31.  A block table has at most 2^30 slots.  rope_base > 1: the rotation's base, as in mk_config. */
typedef struct {
  int32_t n_layers, n_kv, page_size, head_dim;
  int64_t num_pages;
  void* k_pool;
  void* v_pool;
  double rope_base;
} mk_kv_config;

typedef struct mk_kv mk_kv;

/* A handle on the pools: the rotation's frequencies, and (made by the first
 * mk_tree_attn) the pools' tensor maps.  Host memory only; it keeps the pool
 * pointers, not their contents.  Calls on one handle may come from several
 * threads.  Freed with mk_kv_free, after the last call on it has returned. */
int mk_kv_open(const mk_kv_config* cfg, mk_kv** out);
void mk_kv_free(mk_kv* kv);

/* The new tokens of a batch, ragged: sequence b has the rows cu_seqlens[b] ..
 * cu_seqlens[b + 1] - 1 of the token arrays; its i-th new token lies (or is
 * put) in slot cache_lens[b] + i.  Rows before cu_seqlens[0] and from
 * cu_seqlens[batch] on are left as they are. */
typedef struct {
  int32_t batch;
  int32_t n_tokens;            /* rows of the token arrays */
  int32_t max_pages;           /* columns of block_tables */
  const int32_t* cu_seqlens;   /* device [batch + 1], ascending, at most n_tokens */
  const int32_t* cache_lens;   /* device [batch]: tokens in the cache before the new ones */
  const int32_t* block_tables; /* device [batch][max_pages] */
  const int32_t* positions;    /* device [n_tokens]: positions of the new tokens (a drafted
                                  tree: the depths); NULL: a token's position is its slot */
} mk_tokens;

/* K and V of the new tokens into layer `layer` of the pools, and Q beside
 * them: elements 2i and 2i + 1 of each head of q and k are turned by position
 * * rope_base^(-2i / head_dim) (angles exact to 2^-24 of a turn up to
 * position 2^31), then rounded to bf16; v is rounded only.
 *  q, k, v   device, dtype MK_BF16 or MK_F32, head_dim elements per head,
 *            heads side by side, *_stride elements from one token to the next
 *            (q [n_tokens][n_q], k and v [n_tokens][n_kv] heads); pointers
 *            and strides multiples of 16 bytes.  q may be NULL (with q_out)
 *  q_out     device bf16, q_out_stride elements from token to token; either
 *            q itself (bf16, the same stride) or apart from q, k and v
 * A token whose slot has no page in [0, num_pages) is not written (q_out is).
 * A sequence with a negative length or rows outside [0, n_tokens) is left
 * out.  A slot that two tokens of a call name holds either's values. */
typedef struct {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int32_t n_q;
  int32_t dtype;
} mk_append_io;
int mk_kv_append(const mk_kv* kv, int32_t layer, const mk_tokens* tok, const mk_append_io* io,
                 uint32_t* status, void* stream);

/* Attention of the new tokens over the cache and over each other, from the
 * pools (their K and V appended before):
 *   out_t = sum_s p_s V_s / sum_s p_s,  p_s = exp(scale * q_t . K_s)
 * over the slots that token t sees: every slot below cache_lens[b], and the
 * new tokens its mask names.
 *  q          device bf16 [n_tokens][n_q][head_dim], rotated, q_stride
 *             elements from token to token; n_q a multiple of n_kv, query
 *             head h reads K/V head h / (n_q / n_kv)
 *  out        device bf16 [n_tokens][n_q][head_dim], out_stride; not q
 *  lse        device fp32 [n_tokens][n_q]: log sum_s p_s, or NULL
 *  tree_mask  device uint64 [n_tokens][mask_words]: bit j of a token's words
 *             (word j / 64) is set if it sees its sequence's j-th new token;
 *             bits past the sequence's count are ignored.  NULL: the tokens
 *             form a run, each sees itself and those before it
 *  window     > 0: token t sees a slot only if position_t - position_slot <
 *             window (a cached slot's position is the slot; new tokens have
 *             mk_tokens.positions, which must lie in [cache_len, cache_len +
 *             count) of their sequence).  0: no limit
 *  scale      > 0; 0 stands for 1 / sqrt(head_dim)
 * A token that sees nothing gets 0 and lse -inf.  What a token does not see
 * (unused rows of a page, masked tokens) does not reach its output, whatever
 * its bits.  Products of bf16 with fp32 sums; the running maximum, the sum
 * and the output are fp32, the probabilities are rounded to bf16 for the
 * product with V.  (mk_decode_step keeps q, the probabilities and the output
 * at fp32 accuracy: where two tokens are closer than bf16 tells, a draft that
 * is verified here need not be the token that the step would have chosen.)
 * Pointers and strides multiples of 16 bytes.  Results do not depend on timing:
 * the same call gives the same bits.
 * A page id out of range is read as page 0; a sequence with a bad length, or
 * with more tokens than mask bits, is left out (its rows stay as they are); a
 * position out of range is moved into it.  All are recorded. */
typedef struct {
  const void* q;
  void* out;
  float* lse;
  const uint64_t* tree_mask;
  int64_t q_stride, out_stride;
  int32_t n_q;
  int32_t mask_words;
  int32_t window;
  float scale;
} mk_attn_io;
/* Bytes of workspace (16-byte aligned) for calls on the current device with
 * these pools, 0 without a device. */
size_t mk_tree_attn_workspace_bytes(const mk_kv* kv);
int mk_tree_attn(mk_kv* kv, int32_t layer, const mk_tokens* tok, const mk_attn_io* io,
                 void* workspace, size_t workspace_bytes, uint32_t* status, void* stream);

/* After drafted tokens were verified: slot cache_lens[b] + k of every layer
 * takes K and V of slot cache_lens[b] + path[b][k], k = 0 .. path_lens[b] -
 * 1.  Each row of path ascends (0 <= path[b][0] < path[b][1] < ...).
 *  path       device int32 [batch][max_path]
 *  new_lens   device int32 [batch], receives cache_lens[b] + path_lens[b];
 *             apart from the inputs; or NULL
 * A sequence whose path does not ascend, is longer than max_path or leaves
 * its pages is left out (its new length is its cache length).  batch <= 65535. */
int mk_kv_commit(const mk_kv* kv, int32_t batch, const int32_t* cache_lens, const int32_t* path,
                 const int32_t* path_lens, int32_t max_path, const int32_t* block_tables,
                 int32_t max_pages, int32_t* new_lens, uint32_t* status, void* stream);

/* One step of beam search for each request: of the beams * vocab
 * continuations (beam w, token v) of score
 *   scores[w] + logits[w][v] - log sum_u exp(logits[w][u])
 * the n_out best, best first; of equal scores the lower w * vocab + v first.
 * The scores are formed and compared in 64 bits (sums of exponentials in 32,
 * joined in 64).  A finished beam has one continuation, the token eos, and
 * its score stays.  A score that is not a number counts as -inf.
 *  logits     device fp32 [requests * beams][vocab], logits_stride elements
 *             from row to row (mk_decode_step's logits: vocab)
 *  scores     device fp32 [requests][beams]
 *  finished   device uint8 [requests][beams], nonzero: finished; or NULL
 *  out_*      device [requests][n_out]: scores fp32, parent beams int32,
 *             tokens int32; apart from the inputs
 * beams <= 64, n_out <= 128, n_out <= beams * vocab <= 2^30, requests * beams
 * <= 65535; with finished, 0 <= eos < vocab.  Bytes of workspace (16-byte
 * aligned): 0 for a shape that the call refuses. */
size_t mk_beam_select_workspace_bytes(int32_t requests, int32_t beams, int32_t vocab, int32_t n_out);
int mk_beam_select(const float* logits, int64_t logits_stride, const float* scores,
                   const uint8_t* finished, int32_t eos, int32_t requests, int32_t beams,
                   int32_t vocab, int32_t n_out, float* out_scores, int32_t* out_parents,
                   int32_t* out_tokens, void* workspace, size_t workspace_bytes, void* stream);

/* The beams' cache after a selection.  Row r * beams + i of the tables is
 * beam i of request r; its sequence so far becomes that of row r * beams +
 * parents[r][i].  With `len` = lens[r] tokens in each beam's cache:
 *  - columns below len / page_size (full pages, only read from now on) are
 *    the parent's;
 *  - if len % page_size > 0, the column len / page_size (the open page, each
 *    beam's own) is passed on: a parent's first child (the lowest i) keeps
 *    it, the k-th of the other children takes the open page of the k-th beam
 *    without children, and the parent's first len % page_size rows are
 *    copied there, in every layer;
 *  - all other columns stay the row's own (pages given to it ahead).
 * So pages are neither allocated nor freed, and each open page keeps one
 * owner.  A request whose open pages are not `beams` different ones must not
 * share them with another.
 *  lens       device int32 [requests]
 *  parents    device int32 [requests][beams]
 *  tables_in, tables_out  device int32 [requests * beams][max_pages], apart
 * beams <= 64.  A request with a parent outside [0, beams) or a length
 * outside [0, max_pages * page_size] keeps its tables and pages; a copy from
 * or to a page out of range is left out. */
int mk_beam_reorder(const mk_kv* kv, int32_t requests, int32_t beams, const int32_t* lens,
                    const int32_t* parents, const int32_t* tables_in, int32_t* tables_out,
                    int32_t max_pages, uint32_t* status, void* stream);

/* Waits for `stream` and reads a status record: MK_OK, MK_ERR_TIMEOUT (a
 * device-side wait gave up) or MK_ERR_DEVICE (a value out of range; the
 * operator, the sequence and the value in mk_last_error()). */
int mk_check_status(const uint32_t* status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MK_OPS_H */
