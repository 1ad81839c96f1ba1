// C ABI of the prompt attention: checks, planner and dispatch (include/mla_prompt.h).
#include <math.h>
#include <string.h>

#include "prompt.cuh"

// Cycles after which a wait of the attention kernel gives up: about 2 s, and ten times what a tile takes (3000 to 4300) for each tile of a
// sequence's keys, since a role without work in a unit waits for the end of that unit. (A build may name others, to see what a call leaves
// behind whose waits run out.)
#ifndef MLA_PROMPT_WAIT_CYCLES
#define MLA_PROMPT_WAIT_CYCLES 4000000000ll
#endif
#ifndef MLA_PROMPT_WAIT_CYCLES_A_TILE
#define MLA_PROMPT_WAIT_CYCLES_A_TILE 32768
#endif

namespace mla {
namespace {

constexpr int64_t kMaxRows = 1ll << 30;
// Keys and values of the heads that run at a time, to stay in L2. With 1, 12, 24, 48, 96 MB and without groups, us: 8192 tokens of 64 heads 904,
// 908, 892, 890, 875, 918; 16,384 of 64 heads 3371, 3420, 3396, 3410, 3404, 3651; 24 prompts of 61 to 2048 tokens of 64 heads 371, 371, 368,
// 368, 366, 385, of 16 heads 118, 118, 115, 110, 120, 99 (their keys and values fit L2 whole).
constexpr int64_t kGroupBytes = 48ll << 20;
// Calls with fewer units than so many times the SMs share their tiles evenly, if there are more than kLeastShare tiles of keys. Whole units / shared,
// us, at so many units an SM:
//   4096 tokens, causal       0.5: 58 / 38   1.05: 62 / 56    1.7: 80 / 76     2.0: 87 / 89     3.4: 145 / 139   4.2: 163 / 168   6.7: 256 / 267
//   4096 tokens, not causal   0.5: 58 / 51   1.05: 113 / 84   1.7: 118 / 125   2.5: 179 / 180   3.4: 236 / 236   4.2: 299 / 308   6.7: 429 / 490
//   512 after 16 Ki           0.2: 222 / 76  0.8: 236 / 260   1.7: 471 / 497   3.4: 948 / 979
//   single tokens, 2 Ki       0.8: 31 / 27   1.6: 50 / 39     3.2: 68 / 61     6.7: 121 / 122
//   1024 tokens, causal       0.6: 22 / 29   1.7: 34 / 44     3.4: 56 / 64     5.3: 83 / 90
// So 4 is the limit of calls of one lane (single tokens); those of two lanes would gain by one between 1 and 2, and those of few tiles a unit by none.
constexpr int64_t kSharedUnits = 4;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool good_stride(int64_t s) { return s >= 8 && s % 8 == 0 && s <= (1ll << 38); }

int check_prompt(const mla_prompt_desc* d) {
  if (!d || d->num_seqs < 1 || d->num_heads < 1 || d->num_kv_heads < 1 || d->num_heads % d->num_kv_heads != 0)
    return MLA_ERR_INVALID_ARGUMENT;
  if (d->max_q_len < 0 || d->max_k_len < 0 || d->num_q < 0 || d->num_k < 0) return MLA_ERR_INVALID_ARGUMENT;
  if (d->num_seqs > kMaxRows || d->num_q > kMaxRows || d->num_k > kMaxRows || d->num_q * d->num_heads > 0x7fffff00ll) return MLA_ERR_UNSUPPORTED;
  if (d->causal != 0 && d->causal != 1) return MLA_ERR_INVALID_ARGUMENT;
  if (d->out_dtype != MLA_DTYPE_BF16 && d->out_dtype != MLA_DTYPE_F32) return MLA_ERR_INVALID_ARGUMENT;
  if (d->flags & ~(MLA_FLAG_DEBUG_CHECKS | MLA_FLAG_SIMT)) return MLA_ERR_INVALID_ARGUMENT;
  if (d->num_ctas < 0 || d->num_ctas > kMaxPromptCtas) return MLA_ERR_INVALID_ARGUMENT;
  // (the kernel works with the scale times log2 e, which has to be finite too)
  if (!(d->softmax_scale > 0.f) || !(d->softmax_scale <= 0x1p127f)) return MLA_ERR_INVALID_ARGUMENT;
  // the stride of a dim with one element is not used
  if ((d->num_q > 1 && !good_stride(d->q_token_stride)) || (d->num_heads > 1 && !good_stride(d->q_head_stride)))
    return MLA_ERR_INVALID_ARGUMENT;
  if (d->num_k > 1 && (!good_stride(d->k_token_stride) || !good_stride(d->k_rope_token_stride) || !good_stride(d->v_token_stride)))
    return MLA_ERR_INVALID_ARGUMENT;
  if (d->num_kv_heads > 1 && (!good_stride(d->k_head_stride) || !good_stride(d->v_head_stride))) return MLA_ERR_INVALID_ARGUMENT;
  return MLA_OK;
}

// Query heads of a key head that share a unit's rows: all of them, if the tile can be divided among them.
int32_t pack_of(const mla_prompt_desc& d) {
  const int32_t group = d.num_heads / d.num_kv_heads;
  return group <= kPromptTile && (group & (group - 1)) == 0 ? group : 1;
}
int64_t longest_q(const mla_prompt_desc& d) { return d.max_q_len < d.num_q ? d.max_q_len : d.num_q; }
// Row tiles of all sequences, at most: whatever the ends in memory are, and where they do not fall.
int64_t any_entries(const mla_prompt_desc& d, int64_t rows) { return d.num_seqs * cdiv(longest_q(d) * pack_of(d), rows); }
int64_t entries_of(const mla_prompt_desc& d, int64_t rows) {
  const int64_t a = any_entries(d, rows), b = d.num_q * pack_of(d) / rows + d.num_seqs;
  return a < b ? a : b;
}
// Tiles of a sequence's keys, at most.
int64_t key_tiles(const mla_prompt_desc& d) { return cdiv(d.max_k_len < d.num_k ? d.max_k_len : d.num_k, kPromptTile); }
int64_t pad(int64_t bytes) { return cdiv(bytes, 256) * 256; }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_prompt_plan(const mla_prompt_desc* d, int32_t num_sms, mla_prompt_plan_t* plan) {
  int rc = check_prompt(d);
  if (rc) return rc;
  if (!plan || num_sms < 1) return MLA_ERR_INVALID_ARGUMENT;
  mla_prompt_plan_t p;
  memset(&p, 0, sizeof p);
  const int64_t tiles = key_tiles(*d);
  p.pack = pack_of(*d);
  if (d->flags & MLA_FLAG_SIMT) {
    p.kernel = 1;
    p.rows_per_unit = p.pack = 1;
    p.ctas = d->num_q * d->num_heads;
  } else {
    p.rows_per_unit = longest_q(*d) * p.pack <= kPromptTile ? kPromptTile : kMaxUnitRows;
    const int64_t heads = d->num_heads / p.pack, units = entries_of(*d, p.rows_per_unit) * heads;
    // (the kernels count the work of shared calls in 32 bits)
    const int64_t most = any_entries(*d, p.rows_per_unit);
    const bool fits = most < 0x40000000 && most * heads < 0x40000000 && most * heads * (tiles + 1 + kUnitCost) < 0x40000000;
    if (d->num_ctas > 0 && !fits) return MLA_ERR_UNSUPPORTED;
    p.shared = units > 0 && fits && (d->num_ctas > 0 || (units < kSharedUnits * num_sms && tiles > kLeastShare));
    p.listed = d->num_seqs > 1 && !p.shared;
    p.ctas = !p.shared ? units : d->num_ctas > 0 ? d->num_ctas : num_sms;
    if (p.shared && p.ctas > kMaxPromptCtas) p.ctas = kMaxPromptCtas;
    if (p.shared)
      p.workspace_bytes = pad(p.ctas * 2 * p.rows_per_unit * kHeadV * 4) + pad(p.ctas * 2 * p.rows_per_unit * 4) +
                          pad(p.ctas * (int64_t)sizeof(PromptMerge));
    if (p.listed) p.workspace_bytes += pad(entries_of(*d, p.rows_per_unit) * (int64_t)sizeof(int2));
  }
  if (p.ctas > 0x7fffffff) return MLA_ERR_UNSUPPORTED;
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
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k_nope);
  a.kr = static_cast<const __nv_bfloat16*>(k_rope);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.out = out;
  a.lse = lse;
  char* ws = static_cast<char*>(workspace);
  const auto take = [&](int64_t bytes) {
    char* at = ws;
    ws += pad(bytes);
    return at;
  };
  if (p.shared) {
    a.part_o = reinterpret_cast<float*>(take(p.ctas * 2 * p.rows_per_unit * kHeadV * 4));
    a.part_lse = reinterpret_cast<float*>(take(p.ctas * 2 * p.rows_per_unit * 4));
    a.merges = reinterpret_cast<PromptMerge*>(take(p.ctas * (int64_t)sizeof(PromptMerge)));
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
  a.pack = p.pack;
  while ((1 << a.pack_log) < a.pack) ++a.pack_log;
  a.virtual_heads = a.H / a.pack;
  a.shared = p.shared;
  a.ctas = (int32_t)p.ctas;
  a.rows_per_unit = p.rows_per_unit;
  a.entries = p.kernel == 0 ? entries_of(*d, p.rows_per_unit) : 0;
  a.listed = p.listed;
  const int64_t in_l2 = kGroupBytes / ((d->num_k > 0 ? d->num_k : 1) * 2 * (kNope + kHeadV));
  const int64_t heads = (in_l2 > 1 ? in_l2 : 1) * (a.group / a.pack);  // virtual heads
  a.head_group = (int32_t)(heads < a.virtual_heads ? heads : a.virtual_heads);
  a.out_32 = aligned(out, 32);
  a.out_f32 = d->out_dtype == MLA_DTYPE_F32;
  a.debug = debug ? 1 : 0;
  a.scale = d->softmax_scale;
  a.scale_log2 = d->softmax_scale * 1.4426950408889634f;
  a.wait_cycles = MLA_PROMPT_WAIT_CYCLES + (int64_t)MLA_PROMPT_WAIT_CYCLES_A_TILE * key_tiles(*d);

  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (debug && cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess) return MLA_ERR_CUDA;
  if (p.ctas > 0) {
    if ((p.kernel == 1 ? launch_prompt_simt(a, s) : launch_prompt_tc(a, s)) != cudaSuccess) return MLA_ERR_CUDA;
    if (p.shared && launch_prompt_merge(a, s) != cudaSuccess) return MLA_ERR_CUDA;
  }
  if (!debug) return MLA_OK;
  // the tcgen05 kernels look at every sequence, the SIMT kernel at those that a row belongs to
  if ((p.kernel == 1 || p.ctas == 0) && launch_prompt_check(a, s) != cudaSuccess) return MLA_ERR_CUDA;
  mla_verify_desc checks = {};
  checks.flags = d->flags;
  return finish_debug(&checks, dev_status, s);
}
