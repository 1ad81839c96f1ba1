// What the prompt attention kernels share (include/mla_prompt.h).
#pragma once

#include "common.cuh"
#include "mla_prompt.h"

namespace mla {

constexpr int kNope = 128;                  // a head's own dims of a key
constexpr int kHeadQ = kNope + kDRope;      // 192 dims of a query head
constexpr int kHeadV = 128;                 // dims of a value
constexpr int kPromptTile = 128;            // keys to a tile, and query rows to an MMA
constexpr int kMaxPromptCtas = 1024;
constexpr int kMaxUnitRows = 2 * kPromptTile;
// What starting and ending a run of tiles costs, in tiles, and the least that a CTA takes in shared calls. Costs of 0, 1, 2, 3, 4, us: 16 heads
// of 4096 tokens 114, 88, 76, 79, 79; 61 single tokens 63.3, 59.5, 59.4, 59.4, 60.1; 17 tokens after 16 Ki 94.9, 93.8, 97.1, 94.5, 93.7; 16 heads of 512
// tokens after 16 Ki 77.9, 76.6, 75.5, 76.3, 75.6. Leasts of 2, 3, 4, 6, 8: 8 heads of 1024 tokens 22.5, 24.6, 25.7, 27.9, 19.9, no other of these
// calls by more than 1%.
constexpr int kUnitCost = 2, kLeastShare = 4;

// A unit whose last part CTA number c computed, with the first one's CTA: parts first .. c, to be merged.
struct PromptMerge {
  int32_t live, first, slot;  // slot of the first part (the others have slot 0)
  int32_t row0, rows;         // the unit's rows in its sequence, and how many there are
  int32_t q0, head;
  int32_t reserved;
};

struct PromptArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* kr;
  const __nv_bfloat16* v;
  const int32_t* cu_q;
  const int32_t* cu_k;
  void* out;
  float* lse;
  float* part_o;      // shared: [ctas][2][rows_per_unit][128], parts of units, each normalised over its own keys
  float* part_lse;    // [ctas][2][rows_per_unit]
  PromptMerge* merges;  // [ctas]
  int2* list;         // listed: (sequence, row tile) of every entry, longest first, then (-1, 0)
  int32_t* dev_status;
  int64_t num_q, num_k;
  int64_t q_ts, q_hs, k_ts, k_hs, kr_ts, v_ts, v_hs;
  int64_t entries;    // row tiles of all sequences, at most
  int32_t B, H, group, max_q, max_k;
  int32_t pack, pack_log, virtual_heads;  // rows of a unit: pack heads a query; H / pack of such groups
  int32_t causal, shared, ctas, rows_per_unit, listed, head_group, out_f32, debug;
  int32_t out_32;     // out is aligned to 32 bytes
  float scale, scale_log2;
  int64_t wait_cycles;  // after which a wait of the attention kernel gives up
};

cudaError_t launch_prompt_simt(const PromptArgs& a, cudaStream_t stream);
cudaError_t launch_prompt_tc(const PromptArgs& a, cudaStream_t stream);
cudaError_t launch_prompt_merge(const PromptArgs& a, cudaStream_t stream);
cudaError_t launch_prompt_check(const PromptArgs& a, cudaStream_t stream);  // under debug: reports bad ends of any sequence

// A sequence's queries [q0, q0 + m) and keys [k0, k0 + n), clamped into the tensors and the host's bounds.
struct PromptSeq {
  int32_t q0, m, k0, n;
};
__device__ __forceinline__ void clamp_range(const PromptArgs& a, int32_t lo, int32_t hi, int64_t rows, int32_t most, int32_t& at, int32_t& len) {
  const int64_t l = lo < 0 ? 0 : lo > rows ? rows : lo;
  int64_t h = hi < l ? l : hi > rows ? rows : hi;
  if (h > l + most) h = l + most;
  if (l != lo || h != hi) report(a.dev_status, a.debug, MLA_CHECK_BAD_LENGTH);
  at = (int32_t)l;
  len = (int32_t)(h - l);
}
__device__ __forceinline__ PromptSeq clamp_seq(const PromptArgs& a, int32_t q0, int32_t q1, int32_t k0, int32_t k1) {
  PromptSeq s;
  clamp_range(a, q0, q1, a.num_q, a.max_q, s.q0, s.m);
  clamp_range(a, k0, k1, a.num_k, a.max_k, s.k0, s.n);
  return s;
}
__device__ __forceinline__ PromptSeq load_seq(const PromptArgs& a, int b) { return clamp_seq(a, a.cu_q[b], a.cu_q[b + 1], a.cu_k[b], a.cu_k[b + 1]); }
// How many keys query i of a sequence sees (the first so many).
__device__ __forceinline__ int32_t visible(const PromptArgs& a, const PromptSeq& s, int32_t i) {
  return a.causal ? max(0, i - s.m + 1 + s.n) : s.n;  // (i < m)
}
// The sequence of a row of q, and its place there; -1 outside the sequences (or behind a clamped one).
__device__ __forceinline__ int sequence_of(const PromptArgs& a, int64_t row, PromptSeq& s) {
  int lo = 0, hi = a.B;  // cu_q[lo] <= row < cu_q[hi], if there is such a sequence
  if (row < a.cu_q[0] || row >= a.cu_q[a.B]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_q[mid] <= row) lo = mid;
    else hi = mid;
  }
  s = load_seq(a, lo);
  return row >= s.q0 && row < (int64_t)s.q0 + s.m ? lo : -1;
}
// Tiles of keys that a unit's rows [row0, row1) of a sequence see.
__device__ __forceinline__ int32_t tiles_of(const PromptArgs& a, const PromptSeq& s, int64_t row1) {
  return (int32_t)(((int64_t)visible(a, s, (int32_t)((row1 - 1) >> a.pack_log)) + kPromptTile - 1) / kPromptTile);
}
// Units that so many rows make (of 128 or 256 rows).
__device__ __forceinline__ int32_t units_in(const PromptArgs& a, int64_t rows) {
  return (int32_t)((rows + a.rows_per_unit - 1) >> (a.rows_per_unit > kPromptTile ? 8 : 7));
}
// Units of work of an entry and virtual head: its tiles, at least one, and what a run costs besides.
__device__ __forceinline__ int32_t cost_of(int32_t tiles) { return max(1, tiles) + kUnitCost; }

// total + low += x, x >= 0: low keeps what total's rounding loses (exactly, as long as total is not below x; each time it is, total at
// least doubles, so that those errors stay within 2^-22 of the end's total). A softmax sum that takes weights of about 1 one by one
// rounds each to the last place of the total, equal ones always the same way: off by 2^-12 after 2^17 of them.
__device__ __forceinline__ void add_keeping(float& total, float& low, float x) {
  const float s = __fadd_rn(total, x);
  low = __fadd_rn(low, __fsub_rn(x, __fsub_rn(s, total)));
  total = s;
}

}  // namespace mla
