/*
 * mla_kv_ops.h -- the KV-pool steps on either side of tree verification for
 * DDTree speculative decoding over a page_size=1 MLA latent pool.
 *
 * Same pool, slot-table and sequence conventions as mla_verify.h: the pool is
 * bf16 [slots][576] (1152-byte rows); slot_table is int32 [num_seqs][stride];
 * sequence b has a prefix of L_b = seq_lens[b] tokens at slot_table[b][0, L_b)
 * and its T = num_nodes tree nodes at slot_table[b][L_b, L_b + T); a seq_lens
 * entry outside [0, max_seq_len] is clamped (and reported under `debug`).
 *
 * All functions enqueue on `stream`, allocate nothing, never synchronise and
 * are graph-capturable. They return MLA_OK, MLA_ERR_INVALID_ARGUMENT (null or
 * misaligned pointer, bad size) or MLA_ERR_CUDA (launch failure). With a
 * non-NULL dev_status and debug != 0, device-side checks OR MLA_CHECK_* bits
 * into *dev_status (which the caller zeroes); offending entries are skipped,
 * never dereferenced.
 */
#ifndef MLA_KV_OPS_H
#define MLA_KV_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "mla_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * mla_tree_kv_append -- write the tree nodes' latent rows into the slots the
 * slot table gives them, before verification (the tree KV lives in the pool:
 * "The Moment of Certainty", The Final Piece, on accepted nodes being scattered
 * across the cache):
 *   for b < num_seqs, j < num_nodes:
 *     pool[slot_table[b][L_b + j]] = tree_kv[b * num_nodes + j]
 *   pool     device bf16 [num_slots][576], 16-byte aligned (written).
 *   tree_kv  device bf16 [num_seqs * num_nodes][576], 16-byte aligned.
 * A slot outside [0, num_slots) is skipped (MLA_CHECK_BAD_SLOT under debug).
 * Two nodes sharing a slot leave one of the two rows there (unspecified which).
 */
int mla_tree_kv_append(void *pool, int64_t num_slots, const void *tree_kv, const int32_t *slot_table,
                       const int32_t *seq_lens, int32_t num_seqs, int32_t num_nodes, int32_t stride,
                       int32_t max_seq_len, int32_t debug, int32_t *dev_status, mla_stream_t stream);

/*
 * mla_tree_accept_commit -- after verification, make the accepted path part of
 * the prefix (accepted nodes are non-contiguous in the verify block: "The
 * Moment of Certainty", The Final Piece). For each sequence b with
 * n = num_accepted[b] and path a = accepted[b][0, n) (node indices, root first):
 *   slot_table[b][L_b + k]     = old slot of node a[k]          for k < n
 *   slot_table[b][L_b + n + i] = old slot of the i-th rejected node, in node order
 *   seq_lens[b]                = L_b + n
 * so the tree block stays a permutation of its old slots (the rejected nodes'
 * slots can be reused by the next tree). The path is validated: 0 <= n <= T,
 * parent[a[0]] == -1 and parent[a[k]] == a[k-1]; an invalid path leaves the
 * sequence unchanged (MLA_CHECK_BAD_PARENT under debug), as does a prefix
 * length that would exceed max_seq_len (MLA_CHECK_BAD_LENGTH).
 *   slot_table   device int32 [num_seqs][stride] (updated in place).
 *   seq_lens     device int32 [num_seqs] (updated in place).
 *   tree_parent  device int32 [num_seqs][num_nodes], as for mla_verify_attn.
 *   accepted     device int32 [num_seqs][num_nodes]; entries past n are ignored.
 *   num_accepted device int32 [num_seqs].
 * num_nodes must be in [1, 64] and stride >= max_seq_len + num_nodes.
 */
int mla_tree_accept_commit(int32_t *slot_table, int32_t *seq_lens, const int32_t *tree_parent,
                           const int32_t *accepted, const int32_t *num_accepted, int32_t num_seqs,
                           int32_t num_nodes, int32_t stride, int32_t max_seq_len, int32_t debug,
                           int32_t *dev_status, mla_stream_t stream);

/*
 * mla_kv_compact -- Tier-0 KV defragmentation: keep each request's KV
 * contiguous in the pool ("The Moment of Reckoning (User Challenge...)",
 * Output, item 4). Copies each sequence's visible rows, in logical order, into
 * one contiguous range of a destination pool and points the slot table there:
 *   for b < num_seqs, t < n_b = L_b + num_nodes:
 *     dst_pool[dst_base[b] + t] = src_pool[slot_table[b][t]]
 *     new_slot_table[b][t]      = dst_base[b] + t     (when new_slot_table != NULL)
 *   src_pool        device bf16 [src_slots][576]; dst_pool device bf16 [dst_slots][576];
 *                   both 16-byte aligned; they must not overlap.
 *   dst_base        device int64 [num_seqs]: first destination slot of each sequence;
 *                   [dst_base[b], dst_base[b] + n_b) must lie in [0, dst_slots) and the
 *                   ranges of different sequences must not overlap.
 *   new_slot_table  device int32 [num_seqs][stride] or NULL; it may be slot_table itself
 *                   (each entry is read before it is rewritten). dst_slots <= 2^31 - 1.
 * A source slot outside [0, src_slots) or a destination row outside [0, dst_slots)
 * is skipped (MLA_CHECK_BAD_SLOT under debug). After it, mla_verify_attn over
 * (dst_pool, new_slot_table) returns exactly what it returned over
 * (src_pool, slot_table).
 */
int mla_kv_compact(const void *src_pool, int64_t src_slots, void *dst_pool, int64_t dst_slots,
                   const int32_t *slot_table, int32_t *new_slot_table, const int32_t *seq_lens,
                   const int64_t *dst_base, int32_t num_seqs, int32_t num_nodes, int32_t stride,
                   int32_t max_seq_len, int32_t debug, int32_t *dev_status, mla_stream_t stream);

/*
 * mla_slot_map_build -- block tables and slot maps from the requests' lengths, on the device:
 * gives every new token of a step its slot (a prompt's tokens, or a draft tree's nodes) and takes
 * the pages that this needs from a free list. For sequence b the step's tokens are the positions
 * [L_b, L_b + n_b), L_b = seq_lens[b], n_b = new_lens[b]; h_b = held_lens[b] >= L_b positions have
 * a slot already (after mla_tree_accept_commit the rejected nodes' slots behind the prefix are
 * held), and a page is page_size consecutive slots:
 *   have_b = ceil(h_b / page_size),  end_b = max(h_b, L_b + n_b),
 *   take_b = ceil(end_b / page_size) - have_b,  first_b = sum_{c < b} take_c
 *   block_table[b][have_b + k] = free_pages[free_count - 1 - (first_b + k)]      for k < take_b
 *   slot_table[b][t] = block_table[b][t / page_size] * page_size + t % page_size  for h_b <= t < end_b
 *   cu_new[b] = sum_{c < b} n_c  (cu_new[num_seqs] is the sum of all)
 *   slot_map[cu_new[b] + j] = slot_table[b][L_b + j]  for j < n_b,  and -1 from cu_new[num_seqs] on
 *   held_out[b] = end_b,  *free_left = *free_count - sum_b take_b
 * slot_map is what mla_kv4_append takes; its length is fixed on the host, so a captured step
 * serves any lengths (the padding rows are skipped). The rest of both tables is left as it was.
 *
 * All or nothing: when the free pages or the map's capacity do not suffice, no table is changed,
 * slot_map is all -1, cu_new all 0, held_out = held_lens, *free_left = *free_count
 * (MLA_CHECK_NO_PAGES under debug). A sequence with L_b < 0, n_b < 0, h_b < L_b or more positions
 * than its table rows hold is taken as n_b = 0 and end_b = h_b (MLA_CHECK_BAD_LENGTH), and a free_count outside
 * [0, free_capacity] as too few pages. A page outside [0, num_pages), or a held slot outside
 * [0, num_pages * page_size), gives the slot -1 to its tokens (MLA_CHECK_BAD_SLOT).
 *   seq_lens, new_lens  device int32 [num_seqs]; 1 <= num_seqs <= 8192.
 *   held_lens           device int32 [num_seqs] or NULL (= seq_lens).
 *   free_pages          device int32 [free_capacity], taken from the end; free_count: device int32.
 *   block_table         device int32 [num_seqs][block_stride]; NULL only when page_size is 1.
 *   slot_table          device int32 [num_seqs][slot_stride].
 *   slot_map            device int32 [map_capacity].
 *   cu_new              device int32 [num_seqs + 1].
 *   held_out, free_left device int32 [num_seqs] and [1].
 * Inputs are not written, and no array that is written (the tables, the outputs, dev_status under debug) may
 * overlap another array of the call: MLA_ERR_INVALID_ARGUMENT. Inputs may be the same array as one another, and with
 * page_size 1 block_table may be slot_table itself (they hold the same numbers then).
 * page_size >= 1 and num_pages * page_size <= 2^31 - 1; map_capacity <= 2^31 - 1.
 */
int mla_slot_map_build(const int32_t *seq_lens, const int32_t *new_lens, const int32_t *held_lens, int32_t num_seqs,
                       int32_t page_size, int32_t num_pages, const int32_t *free_pages, int32_t free_capacity,
                       const int32_t *free_count, int32_t *block_table, int32_t block_stride, int32_t *slot_table,
                       int32_t slot_stride, int32_t *slot_map, int64_t map_capacity, int32_t *cu_new,
                       int32_t *held_out, int32_t *free_left, int32_t debug, int32_t *dev_status,
                       mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_KV_OPS_H */
