// C ABI of the prompt attention: checks, planner and dispatch (include/mla_prompt.h).
#include <math.h>
#include <string.h>

#include "prompt.cuh"

namespace mla {
namespace {

constexpr int64_t kMaxRows = 1ll << 30;
constexpr int64_t kGroupBytes = 48ll << 20;  // keys and values of the heads that run at a time, in L2

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool good_stride(int64_t s) { return s >= 8 && s % 8 == 0 && s <= (1ll << 38); }

int check_prompt(const mla_prompt_desc* d) {
  if (!d || d->num_seqs < 1 || d->num_heads < 1 || d->num_kv_heads < 1 || d->num_heads % d->num_kv_heads != 0)
    return MLA_ERR_INVALID_ARGUMENT;
  if (d->max_q_len < 0 || d->max_k_len < 0 || d->num_q < 0 || d->num_k < 0) return MLA_ERR_INVALID_ARGUMENT;
  if (d->num_q > kMaxRows || d->num_k > kMaxRows || d->num_q * d->num_heads > (1ll << 40)) return MLA_ERR_UNSUPPORTED;
  if (d->causal != 0 && d->causal != 1) return MLA_ERR_INVALID_ARGUMENT;
  if (d->out_dtype != MLA_DTYPE_BF16 && d->out_dtype != MLA_DTYPE_F32) return MLA_ERR_INVALID_ARGUMENT;
  if (d->flags & ~(MLA_FLAG_DEBUG_CHECKS | MLA_FLAG_SIMT)) return MLA_ERR_INVALID_ARGUMENT;
  if (d->num_splits < 0 || d->num_splits > kMaxPromptSplits) return MLA_ERR_INVALID_ARGUMENT;
  if (!isfinite(d->softmax_scale) || !(d->softmax_scale > 0.f)) return MLA_ERR_INVALID_ARGUMENT;
  // the stride of a dim with one element is not used
  if ((d->num_q > 1 && !good_stride(d->q_token_stride)) || (d->num_heads > 1 && !good_stride(d->q_head_stride)))
    return MLA_ERR_INVALID_ARGUMENT;
  if (d->num_k > 1 && (!good_stride(d->k_token_stride) || !good_stride(d->k_rope_token_stride) || !good_stride(d->v_token_stride)))
    return MLA_ERR_INVALID_ARGUMENT;
  if (d->num_kv_heads > 1 && (!good_stride(d->k_head_stride) || !good_stride(d->v_head_stride))) return MLA_ERR_INVALID_ARGUMENT;
  return MLA_OK;
}

// Row tiles of all sequences, at most.
int64_t entries_of(const mla_prompt_desc& d, int64_t rows) {
  const int64_t most = d.max_q_len < d.num_q ? d.max_q_len : d.num_q, a = d.num_seqs * cdiv(most, rows), b = d.num_q / rows + d.num_seqs;
  return a < b ? a : b;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_prompt_plan(const mla_prompt_desc* d, int32_t num_sms, mla_prompt_plan_t* plan) {
  int rc = check_prompt(d);
  if (rc) return rc;
  if (!plan || num_sms < 1) return MLA_ERR_INVALID_ARGUMENT;
  mla_prompt_plan_t p;
  memset(&p, 0, sizeof p);
  const int64_t rows = d->num_q * d->num_heads;
  const int64_t most_k = d->max_k_len < d->num_k ? d->max_k_len : d->num_k, tiles = cdiv(most_k, kPromptTile);
  if (d->flags & MLA_FLAG_SIMT) {
    p.kernel = 1;
    p.rows_per_unit = 1;
    p.num_splits = d->num_splits > 0 ? d->num_splits : 1;
    p.units = rows * p.num_splits;
  } else {
    // Units of 256 rows keep the tensor cores busy with one half while the softmax of the other runs; of 128 there are more. Parts
    // of the keys make more units still, for the price of writing and merging them. Estimated in us: a tile of keys takes 1.4
    // (256 rows) or 1.1 (128), a unit 3 more, a merge 3 and its partials 1 per 4 MB; the call as long as its longest unit, or all of
    // them over the SMs.
    const int64_t most_q = d->max_q_len < d->num_q ? d->max_q_len : d->num_q;
    const double mean = d->causal && most_k > 0 ? (double)tiles * (1.0 - 0.5 * (most_q < most_k ? most_q : most_k) / most_k) : (double)tiles;
    double best = 1e300;
    for (int half = 0; half < 2; ++half) {
      const int64_t per = half ? kPromptTile : 2 * kPromptTile, units = entries_of(*d, per) * d->num_heads;
      const int64_t most = d->num_splits > 0 ? d->num_splits : tiles < 64 ? (tiles > 1 ? tiles : 1) : 64;
      for (int64_t s = d->num_splits > 0 ? d->num_splits : 1; s <= most; ++s) {
        const double tile_us = half || most_q <= kPromptTile ? 1.1 : 1.4;
        const double longest = 3 + tile_us * cdiv(tiles, s), all = units * s * (3 + tile_us * (mean / s < 1 ? 1 : mean / s)) / num_sms;
        const double merge = s > 1 ? 3 + (double)rows * s * kHeadV * 4 / 4e6 : 0;
        const double us = (longest > all ? longest : all) + merge;
        if (us < best - 1e-9) {
          best = us;
          p.rows_per_unit = (int32_t)per;
          p.num_splits = (int32_t)s;
          p.units = units * s;
        }
      }
    }
    p.listed = d->num_seqs > 1;
  }
  if (p.units > 0x7fffffff) return MLA_ERR_UNSUPPORTED;
  if (p.num_splits > 1) p.workspace_bytes = cdiv(rows * p.num_splits * kHeadV * 4, 256) * 256 + cdiv(rows * p.num_splits * 4, 256) * 256;
  if (p.listed) p.workspace_bytes += cdiv(entries_of(*d, p.rows_per_unit) * (int64_t)sizeof(int2), 256) * 256;
  *plan = p;
  return MLA_OK;
}

extern "C" int mla_prompt_workspace_size(const mla_prompt_desc* d, size_t* bytes) {
  if (!bytes) return MLA_ERR_INVALID_ARGUMENT;
  int rc = check_prompt(d);
  if (rc) return rc;
  int32_t sms = 0;
  rc = current_sms(&sms);
  if (rc) return rc;
  mla_prompt_plan_t p;
  rc = mla_prompt_plan(d, sms, &p);
  if (rc) return rc;
  *bytes = (size_t)p.workspace_bytes;
  return MLA_OK;
}

extern "C" int mla_prompt_attn(const mla_prompt_desc* d, const void* q, const void* k_nope, const void* k_rope, const void* v,
                               const int32_t* cu_q, const int32_t* cu_k, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, int32_t* dev_status, mla_stream_t stream) {
  int rc = check_prompt(d);
  if (rc) return rc;
  if (!cu_q || !cu_k || (d->num_q > 0 && (!q || !out || !lse)) || (d->num_k > 0 && (!k_nope || !k_rope || !v)))
    return MLA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k_nope, 16) || !aligned(k_rope, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(workspace, 256))
    return MLA_ERR_INVALID_ARGUMENT;
  const bool debug = (d->flags & MLA_FLAG_DEBUG_CHECKS) != 0;
  if (debug && !dev_status) return MLA_ERR_INVALID_ARGUMENT;
  int32_t sms = 0;
  rc = current_sms(&sms);
  if (rc) return rc;
  mla_prompt_plan_t p;
  rc = mla_prompt_plan(d, sms, &p);
  if (rc) return rc;
  if (p.workspace_bytes > 0 && (!workspace || workspace_bytes < (size_t)p.workspace_bytes)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (p.kernel == 0 && !tc_kernel_supported()) return MLA_ERR_UNSUPPORTED;

  PromptArgs a;
  memset(&a, 0, sizeof a);
  const int64_t rows = d->num_q * d->num_heads;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k_nope);
  a.kr = static_cast<const __nv_bfloat16*>(k_rope);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.out = out;
  a.lse = lse;
  char* ws = static_cast<char*>(workspace);
  if (p.num_splits > 1) {
    a.part_o = reinterpret_cast<float*>(ws);
    ws += cdiv(rows * p.num_splits * kHeadV * 4, 256) * 256;
    a.part_lse = reinterpret_cast<float*>(ws);
    ws += cdiv(rows * p.num_splits * 4, 256) * 256;
  }
  a.list = reinterpret_cast<int2*>(ws);
  a.dev_status = dev_status;
  a.num_q = d->num_q;
  a.num_k = d->num_k;
  a.q_ts = d->q_token_stride;
  a.q_hs = d->q_head_stride;
  a.k_ts = d->k_token_stride;
  a.k_hs = d->k_head_stride;
  a.kr_ts = d->k_rope_token_stride;
  a.v_ts = d->v_token_stride;
  a.v_hs = d->v_head_stride;
  a.B = d->num_seqs;
  a.H = d->num_heads;
  a.group = d->num_heads / d->num_kv_heads;
  a.max_q = d->max_q_len;
  a.max_k = d->max_k_len;
  a.causal = d->causal;
  a.splits = p.num_splits;
  a.rows_per_unit = p.rows_per_unit;
  a.entries = p.kernel == 0 ? entries_of(*d, p.rows_per_unit) : 0;
  a.listed = p.listed;
  const int64_t in_l2 = kGroupBytes / ((d->num_k > 0 ? d->num_k : 1) * 2 * (kNope + kHeadV));
  const int64_t heads = (in_l2 > 1 ? in_l2 : 1) * a.group;
  a.head_group = (int32_t)(heads < a.H ? heads : a.H);
  a.out_f32 = d->out_dtype == MLA_DTYPE_F32;
  a.debug = debug ? 1 : 0;
  a.scale = d->softmax_scale;
  a.scale_log2 = d->softmax_scale * 1.4426950408889634f;

  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (debug && cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess) return MLA_ERR_CUDA;
  if (p.units > 0) {
    if ((p.kernel == 1 ? launch_prompt_simt(a, s) : launch_prompt_tc(a, s)) != cudaSuccess) return MLA_ERR_CUDA;
    if (p.num_splits > 1 && launch_prompt_merge(a, s) != cudaSuccess) return MLA_ERR_CUDA;
  }
  if (!debug) return MLA_OK;
  mla_verify_desc checks = {};
  checks.flags = d->flags;
  return finish_debug(&checks, dev_status, s);
}
