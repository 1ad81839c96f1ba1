/*
 * mla_kv4.h -- the latent pool held in 4 bits: rows into it, rows out of it, and
 * tree-verify attention over it.
 *
 * Long contexts are bound by the pool (about 13 GB of KV per step at 185k,
 * "The Moment of Doubt", subject message); a 4-bit row is 2.77 times smaller than a
 * bf16 row. The pool is page_size=1 like the bf16 one: the slot table, the sequence
 * lengths and the tree conventions are those of mla_verify.h, and mla_slot_map_build
 * and mla_tree_accept_commit (mla_kv_ops.h) serve both pools.
 *
 * A row is MLA_KV4_ROW_BYTES = 416 bytes:
 *   bytes [0, 256)    512 codes of the latent dims in e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 with a
 *                     sign in bit 3); dim 2i in the low four bits of byte i, dim 2i+1 in the high
 *   bytes [256, 288)  32 scales in e4m3; scale g belongs to dims [16g, 16g + 16)
 *   bytes [288, 416)  the 64 RoPE dims in bf16, unchanged
 * Latent dim d stands for code_d * scale_{d/16}. The product has at most six significant
 * bits, so it is exact in bf16 (and in fp16): a 4-bit pool means exactly the bf16 pool that
 * mla_kv4_gather reads out of it.
 *
 * Functions enqueue on `stream`, allocate nothing, never synchronise (but for
 * MLA_FLAG_DEBUG_CHECKS in mla_verify_attn_kv4) and are graph-capturable. They return
 * MLA_OK or a negative MLA_ERR_* code; nothing is launched when a host-side check fails.
 */
#ifndef MLA_KV4_H
#define MLA_KV4_H

#include <stddef.h>
#include <stdint.h>

#include "mla_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_KV4_ROW_BYTES 416

/*
 * mla_kv4_append -- quantise bf16 latent rows into their slots of a 4-bit pool:
 *   for i < num_rows with slot_map[i] != -1:  pool[slot_map[i]] = row format of rows[i]
 * For each block of 16 latent dims: scale = max|x| / 6 rounded to e4m3 (nearest even, at most
 * 448), code = x / scale rounded to e2m1 (nearest, ties to the even code, at most 6, with x's sign
 * also where it rounds to 0). Both are the roundings of the exact quotients. A block whose scale rounds to 0 (max|x| <= 6 * 2^-10)
 * has codes 0; magnitudes over 6 * 448 are held as 2688. A block with a NaN or an infinity gets
 * the scale NaN, so all its dims read as NaN. RoPE dims are copied.
 *   pool      device [num_slots][416] bytes, 32-byte aligned (written).
 *   rows      device bf16, row i at rows + i * row_stride elements; 16-byte aligned; row_stride
 *             >= 576 and a multiple of 8 (rows may be a slice of a wider projection's output).
 *   slot_map  device int32 [num_rows]; -1 skips the row (padding). Another value outside
 *             [0, num_slots) is skipped and reported (MLA_CHECK_BAD_SLOT under debug).
 * Two rows with the same slot leave that slot's contents unspecified. num_rows may be 0.
 */
int mla_kv4_append(void *pool, int64_t num_slots, const void *rows, int64_t row_stride, const int32_t *slot_map,
                   int64_t num_rows, int32_t debug, int32_t *dev_status, mla_stream_t stream);

/*
 * mla_kv4_gather -- rows of a 4-bit pool as bf16:  out[i] = the values of pool[slots[i]], exactly.
 *   slots  device int32 [num_rows], the same slot any number of times; -1 gives a row of zeros, as does
 *          another value outside [0, num_slots) (reported, MLA_CHECK_BAD_SLOT under debug).
 *   out    device bf16 [num_rows][576], 16-byte aligned; it must not overlap the pool.
 * Use it to hand a prefix to a step that takes bf16 rows (mla_verify_attn's pool, mla_kv_compact).
 */
int mla_kv4_gather(const void *pool, int64_t num_slots, const int32_t *slots, int64_t num_rows, void *out,
                   int32_t debug, int32_t *dev_status, mla_stream_t stream);

/*
 * mla_verify_attn_kv4 -- mla_verify_attn over a 4-bit pool (absorbed latent attention): the same
 * operation, with key row t the 576 values that pool[slot_table[b][t]] stands for and value row t
 * their first 512. num_nodes = 1 with tree_parent -1 is single-token decode.
 *   desc        as for mla_verify_attn; num_slots counts pool rows. MLA_FLAG_PREFIX_STABLE is
 *               accepted and changes nothing; MLA_FLAG_SIMT runs the plain reference kernel.
 *   pool        device [num_slots][416] bytes, 32-byte aligned.
 *   tree_sizes  NULL (every tree has desc->num_nodes nodes), or device int32 [B] as for
 *               mla_verify_attn_ragged: rows of nodes >= tree_sizes[b] give out = 0, lse = -inf.
 *   workspace   device, >= mla_verify_kv4_workspace_size bytes, 256-byte aligned.
 * Other arguments, checks and return codes are those of mla_verify_attn. A key row with a NaN
 * scale makes exactly the rows that see it NaN. The result does not depend on which physical
 * slots hold the rows. Scores, maxima, sums and the output's sums are float32 (finite q and RoPE dims of any
 * size may be used as long as the scores are float32 numbers); each weight and each part's output is rounded to float16 once (2^-11 of the largest
 * value that the row sees, each), also with out_dtype float32 and with one part.
 * Give total_tokens_hint where several sequences, or one of more than 128 query rows, are shorter than max_seq_len:
 * work is shared out by it (mla_verify_kv4_plan). 32 sequences of 301 k positions in all, 128 rows: 96 us with
 * the hint; without it 251 us when max_seq_len is the longest of them and 1.28 ms when it is 184,320, where the hint
 * takes 98 us and a workspace of 202 MB instead of 17.
 */
int mla_verify_attn_kv4(const mla_verify_desc *desc, const void *q, const void *pool, const int32_t *slot_table,
                        const int32_t *seq_lens, const int32_t *tree_sizes, const int32_t *tree_parent, void *out,
                        float *lse, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                        mla_stream_t stream);

/*
 * mla_verify_kv4_plan, mla_verify_kv4_workspace_size -- the launch plan and the workspace bytes of
 * mla_verify_attn_kv4 (mla_verify_plan and mla_verify_workspace_size describe the bf16 kernels).
 * The plan is a pure host function of its arguments; the workspace has the layout given there.
 * plan->kernel is 2 for the kernel that calls with at most 16 query rows a sequence and many sequences of
 * fairly even lengths (max_seq_len against total_tokens_hint) take; its chunks are fixed, as in the SIMT plan.
 * In the tcgen05 plan (0) chunk_tokens is the least that a pair of CTAs takes at a time: the pairs share
 * the positions of all sequences and row tiles evenly, as the lengths on the device turn out, so a
 * sequence may be cut anywhere, into at most num_splits parts. One sequence of at most 128 query
 * rows is shared evenly whatever its length; otherwise a total_tokens_hint far above the actual
 * lengths (or none, which stands for num_seqs * max_seq_len) leaves pairs without work, and one below them only
 * makes the workspace larger: it has room for num_splits parts of every row, and the hint divides the parts.
 */
int mla_verify_kv4_plan(const mla_verify_desc *desc, int32_t num_sms, mla_verify_plan_t *plan);
int mla_verify_kv4_workspace_size(const mla_verify_desc *desc, size_t *bytes);

#ifdef __cplusplus
}
#endif
#endif /* MLA_KV4_H */
