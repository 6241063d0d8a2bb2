/*
 * jf_serving.h -- C ABI of libjf.so for serving several sampled continuations of one prompt: token
 * sampling from given random numbers, the acceptance walk under sampling, and tree attention whose
 * sequences share a long prefix.  The conventions of jf.h hold for every call here: caller-owned
 * device memory, nothing allocated, stream-ordered and graph-capturable, host-checkable problems
 * returned with nothing launched, data-dependent ones written to `*dev_status`.
 *
 * The pages describe greedy verification only [JF section 1] and one continuation a prompt; these
 * calls extend the same path to sampled decoding.
 */
#ifndef JF_SERVING_H_
#define JF_SERVING_H_

#include "jf.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------------------
 * jf_tree_attention_shared -- tree attention of a batch whose sequences share long prefixes.
 *
 * The attention of jf_tree_attention, for a batch that consists of groups of consecutive sequences
 * (several continuations of one prompt): the sequences of group g hold the same first
 * shared_lens[g] tokens, so their K/V up to there is the same, and with S = shared_lens[g] rounded
 * down to whole pages the slots [0, S) of every sequence of the group are read through the block
 * table row of the group's FIRST sequence, once for all nodes of the group.  Slots from S on are
 * each sequence's own.  Block tables that agree on their first S / 16 entries, as prefix sharing
 * gives them, therefore yield jf_tree_attention's result; the entries before S / 16 of the other
 * rows are not read.  A group of one sequence, or one that shares nothing (shared_lens[g] = 0), is
 * allowed; sequences without nodes are too.  For query rows the two parts' softmax states are joined
 * in float32 before the one rounding to bf16.
 *
 * Layouts: as jf_tree_attention, and group_offsets int32 [num_groups+1], group_offsets[0] = 0,
 *          non-decreasing, group_offsets[num_groups] = batch; shared_lens int32 [num_groups], >= 0.
 * Limits: as jf_tree_attention, and batch + num_groups <= 1024, 1 <= num_groups <= batch,
 *          max_pages_per_seq <= 2^27 - 16.
 * Device checks (JF_ERR_DEVICE_CHECK): those of jf_tree_attention; a sequence whose prefix is
 *          shorter than its group's shared_lens is left unwritten; a page id out of range among the
 *          shared ones, or more of them than the block table holds, leaves the whole group unwritten;
 *          malformed group_offsets or a negative shared_lens leave the batch unwritten.
 * workspace: jf_tree_attention_shared_workspace_size(total_nodes, num_q_heads) bytes, 256-byte
 *          aligned, no initialisation; reusable by consecutive calls on one stream, also by calls of
 *          fewer nodes and heads.
 * ------------------------------------------------------------------------------------------ */
JF_API size_t jf_tree_attention_shared_workspace_size(int total_nodes, int num_q_heads);

JF_API jf_status jf_tree_attention_shared(const void* q, const void* k_cache, const void* v_cache,
                                          const int32_t* block_table, int max_pages_per_seq,
                                          const int32_t* prefix_lens, const int32_t* tree_offsets,
                                          const int32_t* parent, const int32_t* group_offsets,
                                          const int32_t* shared_lens, int num_groups, int batch, int total_nodes,
                                          int num_q_heads, int num_kv_heads, int head_dim, int page_size,
                                          int num_pages, float sm_scale, void* out, float* lse, void* workspace,
                                          size_t workspace_bytes, int32_t* dev_status, jf_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * jf_tree_attention_shared_fp8 -- jf_tree_attention_shared over an 8-bit (E4M3) cache, as
 * jf_tree_attention_fp8 stands to jf_tree_attention: uint8 caches, one scale > 0 for each.
 * ------------------------------------------------------------------------------------------ */
JF_API jf_status jf_tree_attention_shared_fp8(const void* q, const void* k_cache, const void* v_cache, float k_scale,
                                              float v_scale, const int32_t* block_table, int max_pages_per_seq,
                                              const int32_t* prefix_lens, const int32_t* tree_offsets,
                                              const int32_t* parent, const int32_t* group_offsets,
                                              const int32_t* shared_lens, int num_groups, int batch,
                                              int total_nodes, int num_q_heads, int num_kv_heads, int head_dim,
                                              int page_size, int num_pages, float sm_scale, void* out, float* lse,
                                              void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                              jf_stream_t stream);

typedef enum {
  JF_LOGITS_F32 = 0,
  JF_LOGITS_BF16 = 1
} jf_logits_type;

/* ------------------------------------------------------------------------------------------
 * jf_sample -- draws one token per row of logits from a given random number.
 *
 * For row r with logits x, m = max_v x_v and temperature T = temperature[r] > 0:
 *   1. weights w_v = exp((x_v - m) / T); the candidates are all v with w_v >= min_p[r], that is
 *      x_v - m >= T ln(min_p[r]), in the order (x descending, token id ascending);
 *   2. of these only the first top_k[r] are kept (0 = all of them);
 *   3. of these only the shortest non-empty prefix whose weights sum to at least top_p[r] of the
 *      weight that step 2 kept (1 = all of them);
 *   4. with W the weight kept, token[r] is the lowest kept id at which the running sum of the kept
 *      weights, taken in id order, exceeds u[r] * W; logprob[r] = ln(w_token / W).
 * T = 0 is greedy: the lowest id that attains m, logprob 0, whatever u[r] and the other parameters
 * are.
 * Weights are computed in float64 (relative error below 2^-45) and summed as integers of 2^-f of the
 * row's largest (f = min(48, 62 - ceil(log2 vocab)), at least 43), so that every sum is exact and a
 * result does not depend on the order of the additions, the size of the batch or the device's
 * schedule; a token lighter than 2^-(f+1) of the heaviest is never drawn.
 * logprob is off by at most vocab * 2^-(f+1) (2^-25 for the largest vocabulary), beside its own
 * rounding to float32.
 * -inf logits (masked tokens) and NaN are no candidates.  A row without any candidate gives
 * token -1 and logprob -inf.  +inf logits share the weight equally among themselves.
 *
 * Layouts: logits float32 or bf16 (logits_type) [rows, vocab], consecutive rows `row_stride`
 *          entries apart; u, temperature float32 [rows]; top_k int32 [rows], top_p, min_p float32
 *          [rows], each may be NULL (off); token int32 [rows]; logprob float32 [rows] or NULL.
 * Limits: 1 <= vocab <= 524288, row_stride >= vocab, rows <= 2^24, logits 16-byte aligned.
 * Device checks (JF_ERR_DEVICE_CHECK; the row's outputs are left unwritten): temperature negative
 *          or not finite; with temperature > 0 also top_k < 0, top_p or min_p outside [0, 1], u outside
 *          [0, 1).
 * ------------------------------------------------------------------------------------------ */
JF_API jf_status jf_sample(const void* logits, int logits_type, long long row_stride, int rows, int vocab,
                           const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                           const float* min_p, int32_t* token, float* logprob, int32_t* dev_status,
                           jf_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * jf_accept_sampled -- the acceptance walk of jf_accept under sampling.
 *
 * As jf_accept, with step 4 of jf_sample in place of the argmax: cur = 0 (root), L = 0; loop:
 * a = the token that jf_sample draws from target_logits[b, cur] with u[b, L] and sequence b's
 * parameters; stop if L == max_depth; otherwise look for a child c of cur (parent[c] == cur) with
 * token[c] == a (lowest c if several); if found, L += 1, path[L] = c, cur = c, repeat; else stop.
 * bonus_token = a from the last iteration.  Every token so accepted, and the bonus token, is drawn
 * from the target's own (filtered) distribution given its path, whatever the draft tree proposed,
 * so the text is distributed as if it had been sampled token by token.
 * A row without any candidate ends the walk with bonus_token -1.
 *
 * Layouts: token, parent, accepted_len, path, bonus_token as jf_accept; target_logits float32 or
 *          bf16 (logits_type) [batch, num_nodes, vocab]; u float32 [batch, max_depth+1];
 *          temperature float32 [batch]; top_k int32, top_p, min_p float32 [batch] or NULL (off);
 *          logprob float32 [batch, max_depth+1] or NULL: entry i is that of the token drawn in step
 *          i (i = 0 .. L), 0 behind them.
 * Limits: 1 <= num_nodes <= 1024, 0 <= max_depth <= 1023, 1 <= vocab <= 524288, target_logits
 *         16-byte aligned.
 * Device checks (JF_ERR_DEVICE_CHECK; the sequence's outputs are left unwritten): parent[i] outside
 *         [-1, i-1]; the parameters as jf_sample's, and with temperature > 0 the random numbers that the
 *         walk comes to.
 * ------------------------------------------------------------------------------------------ */
JF_API jf_status jf_accept_sampled(const int32_t* token, const int32_t* parent, const void* target_logits,
                                   int logits_type, const float* u, const float* temperature, const int32_t* top_k,
                                   const float* top_p, const float* min_p, int batch, int num_nodes, int vocab,
                                   int max_depth, int32_t* accepted_len, int32_t* path, int32_t* bonus_token,
                                   float* logprob, int32_t* dev_status, jf_stream_t stream);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* JF_SERVING_H_ */
