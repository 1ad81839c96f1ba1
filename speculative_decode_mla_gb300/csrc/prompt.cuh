// What the prompt attention kernels share (include/mla_prompt.h).
#pragma once

#include "common.cuh"
#include "mla_prompt.h"

namespace mla {

constexpr int kNope = 128;                  // a head's own dims of a key
constexpr int kHeadQ = kNope + kDRope;      // 192 dims of a query head
constexpr int kHeadV = 128;                 // dims of a value
constexpr int kPromptTile = 128;            // keys to a tile, and query rows to an MMA
constexpr int kMaxPromptSplits = 1024;

struct PromptArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* kr;
  const __nv_bfloat16* v;
  const int32_t* cu_q;
  const int32_t* cu_k;
  void* out;
  float* lse;
  float* part_o;      // splits > 1: [splits][num_q * H][128], each part normalised over its own keys
  float* part_lse;    // [splits][num_q * H]
  int2* list;         // listed: (sequence, row tile) of every entry, longest first, then (-1, 0)
  int32_t* dev_status;
  int64_t num_q, num_k;
  int64_t q_ts, q_hs, k_ts, k_hs, kr_ts, v_ts, v_hs;
  int64_t entries;    // row tiles of all sequences, at most
  int32_t B, H, group, max_q, max_k;
  int32_t causal, splits, rows_per_unit, listed, head_group, out_f32, debug;
  float scale, scale_log2;
};

cudaError_t launch_prompt_simt(const PromptArgs& a, cudaStream_t stream);
cudaError_t launch_prompt_tc(const PromptArgs& a, cudaStream_t stream);
cudaError_t launch_prompt_merge(const PromptArgs& a, cudaStream_t stream);

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
__device__ __forceinline__ PromptSeq load_seq(const PromptArgs& a, int b) {
  PromptSeq s;
  clamp_range(a, a.cu_q[b], a.cu_q[b + 1], a.num_q, a.max_q, s.q0, s.m);
  clamp_range(a, a.cu_k[b], a.cu_k[b + 1], a.num_k, a.max_k, s.k0, s.n);
  return s;
}
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
// The tiles [t0, t1) of part `split` when `tiles` tiles are cut into a.splits parts of one size.
__device__ __forceinline__ void part_of(const PromptArgs& a, int32_t tiles, int32_t split, int32_t& t0, int32_t& t1) {
  const int32_t each = (tiles + a.splits - 1) / a.splits;
  t0 = (int32_t)min((int64_t)tiles, (int64_t)each * split);
  t1 = min(tiles, t0 + each);
}

}  // namespace mla
