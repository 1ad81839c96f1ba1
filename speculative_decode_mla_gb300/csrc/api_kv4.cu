// C ABI of tree-verify attention over the 4-bit pool: planner and dispatch (include/mla_kv4.h).
#include <string.h>

#include "kv4.cuh"

namespace mla {
namespace {

constexpr int kTcRowsPerTile = 128;  // query rows of a pair of CTAs
constexpr int kSimtRowsPerTile = 8;  // one warp per row, 8 warps per CTA
constexpr int kFewRows = 16;         // the rows of one MMA of the kernel for few rows
constexpr int kMaxSplits = 65535;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

int64_t part_o_bytes(const mla_verify_plan_t& p, int64_t rows) {
  return cdiv((int64_t)p.num_splits * rows * kDLatent * 2, 256) * 256;
}

// One row tile in all: the pairs may share any length evenly, since it has no more splits than there are pairs, and as
// many at its greatest length. (A captured call of 128 rows with room for 180 Ki positions
// takes 19 us at 16 Ki, not 50, and 29 at 64 Ki, not 50.)
bool shares_any_length(const mla_verify_desc& d, const mla_verify_plan_t& p, int64_t row_tiles) {
  return p.kernel == 0 && row_tiles == 1 && d.num_splits == 0;
}

// The kernel for few rows: at most 16 a sequence, and enough sequences and positions to keep three small CTAs on every SM
// busy (a lone CTA waits on itself). 16 rows, equal lengths, tcgen05 kernel against this one, us: 4096 sequences of 300 positions
// 827, 433; 1024 of 300: 210, 123; 256 of 1000: 97, 83; 32 of 8192: 75, 65; 16 of up to 1000: 16.5, 15.0; 4 of 65,536: 70, 61;
// but 4 of 16,384: 26, 29; 8 of 2000: 15, 18; 1 of 65,536: 27, 37.
// Its chunks are fixed and walked by one CTA each, on a grid that has room for every sequence at the greatest length, where the
// tcgen05 kernel's pairs share all positions. So the lengths have to be even, as far as the hint tells: the longest at most 2.25
// times the mean, or chunks of at most 1.5 times an even share of all positions and at most four CTAs for every place on the SMs.
// One of 131,072 among 1000 of 300: 238, 5461 us; one of 16,384: 209, 764; one of 32,000 among 64 of 1000: 43, 96 (chunks of 1.2 times
// the share, 18 CTAs a place); 512 between 300 and 9600: 380, 482 (2.3 times the share); 4 between 16,384 and 65,536: 45, 55 (1.8). On the
// other side 128 between 300 and 9600: 103, 89; 16 of 65,536 with room for 184,320: 249, 190; 1024 of up to 8000: 1041, 954.
bool takes_few_rows(const mla_verify_desc& d, int64_t total, int64_t uniform, int64_t max_tiles, int64_t tiles, int64_t slots) {
  if ((int64_t)d.num_nodes * d.num_heads > kFewRows || (d.flags & MLA_FLAG_SIMT)) return false;
  if (d.num_seqs < 4 || (d.num_seqs < 16 && total < 131072)) return false;
  if (d.num_seqs >= 8 && 4 * uniform <= 9 * total) return true;
  return 2 * tiles * slots <= 3 * cdiv(total, kTileTokens) && d.num_seqs * cdiv(max_tiles, tiles) <= 4 * slots;
}

// Tiles of 64 positions to a chunk of the kernel for few rows: one wave of CTAs (a sequence's last chunk is half empty on average);
// the merge reads every split, so at most 128 of them, and four tiles a CTA but for short calls.
int64_t few_rows_tiles(const mla_verify_desc& d, int64_t total, int64_t max_tiles, int64_t slots) {
  if (d.num_splits > 0) return cdiv(max_tiles, d.num_splits);
  const int64_t room = slots - d.num_seqs / 2 > 1 ? slots - d.num_seqs / 2 : 1;
  const int64_t few_tiles = cdiv(max_tiles, 16) < 4 ? cdiv(max_tiles, 16) : 4, few_splits = cdiv(max_tiles, 128);
  int64_t tiles = cdiv(cdiv(total, kTileTokens), room);
  tiles = tiles > few_tiles ? tiles : few_tiles;
  tiles = tiles > few_splits ? tiles : few_splits;
  return tiles > max_tiles ? max_tiles : tiles;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_verify_kv4_plan(const mla_verify_desc* d, int32_t num_sms, mla_verify_plan_t* plan) {
  int rc = check_desc(d);
  if (rc) return rc;
  if (!plan || num_sms < 1) return MLA_ERR_INVALID_ARGUMENT;
  mla_verify_plan_t p;
  memset(&p, 0, sizeof p);
  const bool simt = (d->flags & MLA_FLAG_SIMT) != 0;
  const int64_t R = (int64_t)d->num_nodes * d->num_heads;
  const int64_t max_n = (int64_t)d->max_seq_len + d->num_nodes;
  const int64_t uniform = (int64_t)d->num_seqs * max_n;
  const int64_t total = d->total_tokens_hint > 0 && d->total_tokens_hint < uniform ? d->total_tokens_hint : uniform;
  const int64_t few_slots = (int64_t)num_sms * 3, few_max = cdiv(max_n, kTileTokens);
  const int64_t few_tiles = few_rows_tiles(*d, total, few_max, few_slots);
  const bool few = takes_few_rows(*d, total, uniform, few_max, few_tiles, few_slots), tc = !simt && !few;
  p.kernel = simt ? 1 : few ? 2 : 0;
  p.rows_per_tile = simt ? kSimtRowsPerTile : few ? kFewRows : kTcRowsPerTile;
  p.row_tiles = (int32_t)cdiv(R, p.rows_per_tile);
  const int64_t tile = tc ? kKv4TileTokens : kTileTokens;
  const int64_t max_tiles = cdiv(max_n, tile);
  const int64_t row_tiles = (int64_t)d->num_seqs * p.row_tiles;
  // (the kernels count tiles, and positions of a segment, in 32 bits)
  if (max_n > 0x7fffff00 || (max_tiles + kKv4SegmentUnits) * row_tiles > 0x3fffffff) return MLA_ERR_UNSUPPORTED;
  // SIMT and few rows: units of (sequence, row tile, chunk), small CTAs, several per SM. tcgen05: one cluster per pair of SMs; the
  // clusters share all tiles equally, at least chunk_tokens / 128 each. That least share only bounds the number of
  // splits that the workspace has room for: the kernel takes the even share of the lengths that it finds.
  const int64_t slots = simt ? (int64_t)num_sms * 8 : few ? few_slots : (num_sms / 2 > 0 ? num_sms / 2 : 1);
  int64_t tiles = few               ? few_tiles
                  : d->num_splits > 0 ? cdiv(max_tiles, d->num_splits)
                                      : cdiv(cdiv(total, tile) * p.row_tiles, slots);
  tiles = tiles < 1 ? 1 : tiles > max_tiles ? max_tiles : tiles;
  if (cdiv(max_tiles, tiles) + 1 > kMaxSplits) tiles = cdiv(max_tiles, kMaxSplits - 1);
  p.chunk_tokens = (int32_t)(tiles * tile);
  if (shares_any_length(*d, p, row_tiles)) p.num_splits = (int32_t)(max_tiles < slots ? max_tiles : slots);
  else if (!tc || row_tiles == 1) p.num_splits = (int32_t)cdiv(max_tiles, tiles);
  else p.num_splits = (int32_t)((max_tiles + tiles - 2) / tiles + 1);  // a row tile may begin inside a share
  if (!tc && row_tiles * p.num_splits > 0x7fffffff) return MLA_ERR_UNSUPPORTED;
  const int64_t all = row_tiles * (max_tiles + kKv4SegmentUnits) - kKv4SegmentUnits;
  p.ctas = (int32_t)(!tc ? row_tiles * p.num_splits : 2 * (all < slots ? all : slots));
  const int64_t rows = (int64_t)d->num_seqs * R;
  p.workspace_bytes = part_o_bytes(p, rows) + cdiv((int64_t)p.num_splits * rows * 4, 256) * 256;
  *plan = p;
  return MLA_OK;
}

extern "C" int mla_verify_kv4_workspace_size(const mla_verify_desc* d, size_t* bytes) {
  if (!bytes) return MLA_ERR_INVALID_ARGUMENT;
  int rc = check_desc(d);
  if (rc) return rc;
  int32_t sms = 0;
  rc = current_sms(&sms);
  if (rc) return rc;
  mla_verify_plan_t p;
  rc = mla_verify_kv4_plan(d, sms, &p);
  if (rc) return rc;
  *bytes = (size_t)p.workspace_bytes;
  return MLA_OK;
}

extern "C" int mla_verify_attn_kv4(const mla_verify_desc* d, const void* q, const void* pool,
                                   const int32_t* slot_table, const int32_t* seq_lens, const int32_t* tree_sizes,
                                   const int32_t* tree_parent, void* out, float* lse, void* workspace,
                                   size_t workspace_bytes, int32_t* dev_status, mla_stream_t stream) {
  int rc = check_desc(d);
  if (rc) return rc;
  if (!q || !pool || !slot_table || !seq_lens || !tree_parent || !out || !lse || !workspace)
    return MLA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(pool, 32) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 256) ||
      !aligned(slot_table, 4) || !aligned(seq_lens, 4) || !aligned(tree_sizes, 4) || !aligned(tree_parent, 4))
    return MLA_ERR_INVALID_ARGUMENT;
  const bool debug = (d->flags & MLA_FLAG_DEBUG_CHECKS) != 0;
  if (debug && !dev_status) return MLA_ERR_INVALID_ARGUMENT;
  int32_t sms = 0;
  rc = current_sms(&sms);
  if (rc) return rc;
  mla_verify_plan_t p;
  rc = mla_verify_kv4_plan(d, sms, &p);
  if (rc) return rc;
  if (workspace_bytes < (size_t)p.workspace_bytes) return MLA_ERR_WORKSPACE_TOO_SMALL;

  VerifyArgs a;
  memset(&a, 0, sizeof a);
  a.rows = (int64_t)d->num_seqs * d->num_nodes * d->num_heads;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.kv = static_cast<const __nv_bfloat16*>(pool);
  a.slot_table = slot_table;
  a.tree_sizes = tree_sizes;
  a.seq_lens = seq_lens;
  a.tree_parent = tree_parent;
  a.part_o = static_cast<__half*>(workspace);
  a.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + part_o_bytes(p, a.rows));
  a.dev_status = dev_status;
  a.num_slots = d->num_slots;
  a.B = d->num_seqs;
  a.T = d->num_nodes;
  a.H = d->num_heads;
  a.stride = d->slot_table_stride;
  a.max_seq_len = d->max_seq_len;
  a.chunk = shares_any_length(*d, p, (int64_t)d->num_seqs * p.row_tiles) ? kKv4TileTokens : p.chunk_tokens;
  a.splits = p.num_splits;
  a.row_tiles = p.row_tiles;
  a.rows_per_tile = p.rows_per_tile;
  a.debug = debug ? 1 : 0;
  a.scale = d->softmax_scale;
  a.scale_log2 = d->softmax_scale * 1.4426950408889634f;

  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (debug && cudaMemsetAsync(dev_status, 0, sizeof(int32_t), s) != cudaSuccess) return MLA_ERR_CUDA;
  if ((p.kernel == 1   ? launch_verify_kv4_simt(a, s)
       : p.kernel == 2 ? launch_verify_kv4_rows(a, s)
                       : launch_verify_kv4_tc(a, p.ctas, s)) != cudaSuccess)
    return MLA_ERR_CUDA;
  if (launch_combine(p.num_splits, a.rows, kDLatent, a.part_o, MLA_DTYPE_F16, a.part_lse, out, lse, d->out_dtype,
                     /*dependent=*/true, s) != cudaSuccess)
    return MLA_ERR_CUDA;
  return finish_debug(d, dev_status, s);
}
