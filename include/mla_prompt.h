/*
 * mla_prompt.h -- what comes before tree verification: a layer's projections made ready for the latent
 * pool and its attention, and the attention of the prompt itself.
 *
 * mla_rope_append takes the latent rows and the query heads of a layer as the projections leave them, normalises and
 * rotates both and writes the rows into the pool (bf16, or the 4 bits of mla_kv4.h) in one launch; the
 * pool, the slot maps (mla_slot_map_build) and the rows are those of mla_verify.h. mla_prompt_attn is the attention of
 * whole prompts, or of their next chunks, in the form that is cheaper for many queries: keys and values expanded
 * to heads, K of 128 dims a head and the 64 RoPE dims that all heads share, V of 128 dims a head. Its
 * result is that of the absorbed attention over the latent rows (mla_verify_attn on a chain), up to the rounding of the expanded
 * keys and values. A step of a layer:
 *   prompt:  mla_rope_append(rows, q) -> rows_out, q_out, pool;  kv = rows_out[:, :512] x W (the caller's product,
 *            128 + 128 dims a head);  mla_prompt_attn(q_out, kv's keys, rows_out[:, 512:], kv's values)
 *   decode:  mla_rope_append(rows, q's RoPE dims -> dims 512.. of the absorbed queries);  mla_verify_attn / _kv4
 *
 * Functions enqueue on `stream`, allocate nothing, never synchronise (but for MLA_FLAG_DEBUG_CHECKS in
 * mla_prompt_attn) and are graph-capturable. They return MLA_OK or a negative MLA_ERR_* code; nothing is launched when a
 * host-side check fails. "Device" pointers belong to the current device. Strides are in elements.
 */
#ifndef MLA_PROMPT_H
#define MLA_PROMPT_H

#include <stddef.h>
#include <stdint.h>

#include "mla_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A further bit of *dev_status. */
enum mla_prompt_device_check { MLA_CHECK_BAD_POSITION = 1 << 5 };  /* positions[i] outside [-1, num_positions) */

/* Formats of the pool that mla_rope_append writes. */
enum mla_pool_format { MLA_POOL_NONE = 0, MLA_POOL_BF16 = 1, MLA_POOL_KV4 = 2 };
/* Which dims of the 64 RoPE dims turn together. */
enum mla_rope_pairs { MLA_ROPE_ADJACENT = 0 /* 2k, 2k + 1 */, MLA_ROPE_HALVES = 1 /* k, k + 32 */ };

typedef struct mla_rope_desc {
  int64_t num_rows;            /* tokens, 0 or more */
  int64_t row_stride;          /* of rows; >= 576 and a multiple of 8 */
  int64_t num_slots;           /* rows of the pool, 1 .. 2^31 - 1 (unread without a pool) */
  int64_t q_token_stride, q_head_stride;          /* multiples of 8 */
  int64_t q_out_token_stride, q_out_head_stride;  /* multiples of 8 */
  int32_t pool_format;         /* MLA_POOL_* */
  int32_t num_heads;           /* query heads a token (unread without q) */
  int32_t head_dim;            /* dims of a query head: 64 .. 256, a multiple of 8; its last 64 are the RoPE dims */
  int32_t num_positions;       /* rows of cos_sin, >= 1 */
  int32_t pairs;               /* MLA_ROPE_* */
  float eps;                   /* finite and >= 0, added to the mean of squares */
} mla_rope_desc;

/*
 * mla_rope_append -- for token i < num_rows at position p = positions[i], with c_k = cos_sin[p][k] and
 * s_k = cos_sin[p][32 + k] for k < 32, the pair of dims (x, y) number k of a vector's 64 RoPE dims turned into
 * (x c_k - y s_k, y c_k + x s_k):
 *   y[0:512]   = weight * x / sqrt(mean(x^2) + eps), x = rows[i][0:512]   (x itself when weight is NULL)
 *   y[512:576] = turned rows[i][512:576]
 *   rows_out[i] = y   (when rows_out is not NULL)
 *   pool[slot_map[i]] = y, or for MLA_POOL_KV4 the 4-bit row that mla_kv4_append makes of the bf16 y
 * and for each query head h
 *   z = q_weight * q / sqrt(mean(q^2) + eps) over all head_dim dims   (q itself when q_weight is NULL)
 *   q_out[i][h] = z with its last 64 dims turned
 * All of it is computed in float32 and rounded to bf16 once (sums of squares have to be float32 numbers). cos_sin may
 * hold any numbers, a scale of long contexts among them.
 *   rows       device bf16, row i at rows + i * row_stride, 16-byte aligned; NULL: only the queries.
 *   weight     device bf16 [512] or NULL, 16-byte aligned.
 *   q          device bf16, head h of token i at q + i * q_token_stride + h * q_head_stride, 16-byte aligned; or NULL.
 *   q_weight   device bf16 [head_dim] or NULL, 16-byte aligned.
 *   positions  device int32 [num_rows]. -1: a padding row, for which nothing is written. Another value outside
 *              [0, num_positions) is treated the same and reported (MLA_CHECK_BAD_POSITION under debug).
 *   cos_sin    device float32 [num_positions][64], 16-byte aligned.
 *   slot_map   device int32 [num_rows], with a pool. -1: the row is not put into the pool (rows_out and q_out are written).
 *              Another value outside [0, num_slots) is treated the same and reported (MLA_CHECK_BAD_SLOT under debug).
 *   pool       device bf16 [num_slots][576], 16-byte aligned, or [num_slots][416] bytes, 32-byte aligned (written).
 *   rows_out   device bf16 [num_rows][576], 16-byte aligned, or NULL. It may be rows itself when row_stride is 576.
 *   q_out      device bf16, laid out by its own strides, 16-byte aligned. It may be q itself, with q's strides.
 *   dev_status device int32, needed when debug is not 0 (bits are OR-ed in; the caller zeroes it).
 * Beyond these two, what is written may overlap nothing else of the call. Heads of q_out may not overlap one another. Two rows
 * with the same slot leave that slot's contents unspecified. With rows NULL there is no pool, slot_map, weight or
 * rows_out; one of rows and q is needed, and with rows one of pool and rows_out.
 */
int mla_rope_append(const mla_rope_desc *desc, const void *rows, const void *weight, const void *q,
                    const void *q_weight, const int32_t *positions, const float *cos_sin, const int32_t *slot_map,
                    void *pool, void *rows_out, void *q_out, int32_t debug, int32_t *dev_status, mla_stream_t stream);

/* Shapes of one mla_prompt_attn call. The launch is a pure function of this struct and of the SM count. */
typedef struct mla_prompt_desc {
  int32_t num_seqs;        /* B, 1 .. 2^30 */
  int32_t num_heads;       /* H >= 1, query heads */
  int32_t num_kv_heads;    /* >= 1, divides H: query head h reads key head h / (H / num_kv_heads) */
  int32_t max_q_len;       /* host-known upper bound of a sequence's queries, >= 0 */
  int32_t max_k_len;       /* host-known upper bound of a sequence's keys, >= 0 */
  int32_t causal;          /* 1: query i sees keys up to its own place; 0: all keys of its sequence */
  int32_t out_dtype;       /* MLA_DTYPE_BF16 or MLA_DTYPE_F32 */
  int32_t flags;           /* MLA_FLAG_DEBUG_CHECKS, MLA_FLAG_SIMT */
  int32_t num_ctas;        /* 0: planner decides; > 0: the work is shared out evenly over this many CTAs (at most 1024) */
  float softmax_scale;     /* > 0 and at most 2^127 */
  int64_t num_q, num_k;    /* rows of q (and out, lse), and of k_nope, k_rope and v; 0 .. 2^30 */
  int64_t q_token_stride, q_head_stride;  /* all strides: multiples of 8, from 8 to 2^38 */
  int64_t k_token_stride, k_head_stride;
  int64_t k_rope_token_stride;
  int64_t v_token_stride, v_head_stride;
} mla_prompt_desc;

/* The launch plan chosen for a desc (for introspection and tests). */
typedef struct mla_prompt_plan_t {
  int32_t kernel;          /* 0: tcgen05 kernel, 1: SIMT reference kernel */
  int32_t rows_per_unit;   /* rows (query and head) that a CTA works on at a time: 256, or 128 when no sequence has more */
  int32_t pack;            /* query heads of one key head that share a unit's rows: H / num_kv_heads, or 1 */
  int32_t shared;          /* 1: the CTAs share all tiles of keys evenly, and parts of a unit are merged; 0: whole units */
  int32_t listed;          /* 1: a first kernel lists the units of a batch, longest first (with shared 0) */
  int32_t reserved;
  int64_t ctas;            /* CTAs launched: with shared 0, an upper bound of the units */
  int64_t workspace_bytes; /* 0 when none is needed */
} mla_prompt_plan_t;

/*
 * mla_prompt_plan, mla_prompt_workspace_size -- the plan (a pure host function) and the workspace bytes of
 * mla_prompt_attn on the current device. MLA_OK, MLA_ERR_INVALID_ARGUMENT, MLA_ERR_UNSUPPORTED or MLA_ERR_NO_DEVICE.
 */
int mla_prompt_plan(const mla_prompt_desc *desc, int32_t num_sms, mla_prompt_plan_t *plan);
int mla_prompt_workspace_size(const mla_prompt_desc *desc, size_t *bytes);

/*
 * mla_prompt_attn -- attention of packed prompts. Sequence b has the query rows [cu_q[b], cu_q[b + 1]) and the keys
 * [cu_k[b], cu_k[b + 1]) (m and n of them); its queries are the last m of its n places, so query i sees, when causal, the
 * keys t <= i + n - m (a chunk of a prompt over all keys up to its end; m = n for a whole prompt, m = 1 for one
 * new token), else all n. For head h, key head g = h / (H / num_kv_heads), with the visible t of the sequence:
 *   s_t = softmax_scale * (<q[i][h][0:128], k_nope[t][g]> + <q[i][h][128:192], k_rope[t]>)
 *   out[i][h] = sum_t softmax(s)_t v[t][g],   lse[i][h] = ln sum_t exp(s_t)
 * A query that sees no key gives out = 0 and lse = -inf. Rows of out and lse outside [cu_q[0], cu_q[B]) are left as
 * they were. Keys and values that a query does not see do not reach its result, whatever they hold (NaN among them).
 *   q        device bf16, row i head h at q + i * q_token_stride + h * q_head_stride; 192 dims.
 *   k_nope   device bf16, 128 dims a key head; v the same: both may be slices of one [num_k][Hk][256] tensor.
 *   k_rope   device bf16 [num_k][64], e.g. the RoPE dims of mla_rope_append's rows_out.
 *            These four are 16-byte aligned; a tensor without rows may be NULL.
 *   cu_q, cu_k  device int32 [B + 1], not falling, within [0, num_q] and [0, num_k]; cu_k may be cu_q itself. Values outside, and
 *            lengths outside [0, max_q_len] or [0, max_k_len], are clamped (MLA_CHECK_BAD_LENGTH under debug checks).
 *   out      device [num_q][H][128], bf16 or float32, 16-byte aligned;  lse  device float32 [num_q][H].
 *   workspace  device, >= mla_prompt_workspace_size bytes, 256-byte aligned (NULL where that is 0). Nothing is kept in it: calls
 *            that run one after the other may share it, captured ones too; calls that run at once may not.
 *   dev_status as for mla_verify_attn.
 * Weights are rounded to bf16 for the product with V; scores, maxima, sums and outputs are float32, and
 * where a row's keys are cut into parts (calls with few units, by the lengths on the device) these are merged in float32. out, lse and
 * workspace may overlap nothing else of the call.
 */
int mla_prompt_attn(const mla_prompt_desc *desc, const void *q, const void *k_nope, const void *k_rope, const void *v,
                    const int32_t *cu_q, const int32_t *cu_k, void *out, float *lse, void *workspace,
                    size_t workspace_bytes, int32_t *dev_status, mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_PROMPT_H */
