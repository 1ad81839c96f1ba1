// A layer's latent rows and query heads: norm, rotation of the RoPE dims, and the rows' way into the pool
// (declared in include/mla_prompt.h).
//
// Bound by memory, or, for a decode step, by the latency of one launch; so both parts run in one launch: the first blocks take
// rows, the others query heads. A warp takes a row: 16 latent dims and one adjacent pair of RoPE dims a lane, the sum
// of squares over the warp. A group of 8, 16 or 32 lanes takes a query head, 16 bytes a lane, so that heads of 64
// dims (the RoPE dims alone) fill the warp too. Loads of kRowsPerWarp rows, or of kHeadsInFlight heads, are out before one is used.
#include <math.h>

#include "kv4.cuh"
#include "mla_prompt.h"

namespace mla {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kWarps = kRopeThreads / 32;
constexpr int kPairs = kDRope / 2;
constexpr int kMaxHeadDim = 256;
constexpr int kHeadsInFlight = 4;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct RopeArgs {
  const __nv_bfloat16* rows;
  const __nv_bfloat16* weight;
  const __nv_bfloat16* q;
  const __nv_bfloat16* q_weight;
  const int32_t* positions;
  const float* cos_sin;
  const int32_t* slot_map;
  void* pool;
  __nv_bfloat16* rows_out;
  __nv_bfloat16* q_out;
  int32_t* dev_status;
  int64_t num_rows, row_stride, num_slots;
  int64_t q_ts, q_hs, qo_ts, qo_hs;
  int64_t row_blocks;
  int32_t pool_format, num_heads, head_dim, num_positions, halves, debug;
  int32_t copy;  // the dims before the RoPE dims are written too
  float eps;
};

// (not through the read-only path: rows_out may be rows, q_out may be q)
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// The position of a token, -1 where there is nothing to do. Every lane of the warp has the same token or, with `one`,
// reports for itself.
__device__ __forceinline__ int32_t load_position(const RopeArgs& a, int64_t token, bool one) {
  int32_t p = a.positions[token];
  if (p < -1 || p >= a.num_positions) {
    if (one) report(a.dev_status, a.debug, MLA_CHECK_BAD_POSITION);
    p = -1;
  }
  return p;
}

// N rows of a warp, from row0 on.
template <int N>
__device__ __forceinline__ void do_rows(const RopeArgs& a, int64_t row0) {
  const int lane = threadIdx.x & 31;
  int32_t pos[N];
  int64_t slot[N];
  uint4 v[N][2];
  uint32_t rope[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t row = row0 + i;
    pos[i] = row < a.num_rows ? load_position(a, row, lane == 0) : -1;
    slot[i] = a.pool_format != MLA_POOL_NONE && row < a.num_rows ? a.slot_map[row] : -1;
    if (row < a.num_rows) {  // (the row is in range whatever its position is)
      const __nv_bfloat16* src = a.rows + row * a.row_stride;
      v[i][0] = ld16(src + 8 * lane);
      v[i][1] = ld16(src + 256 + 8 * lane);
      rope[i] = *(reinterpret_cast<const uint32_t*>(src + kDLatent) + lane);
    }
  }
  uint4 w[2];
  if (a.weight) {
    w[0] = __ldg(reinterpret_cast<const uint4*>(a.weight) + lane);
    w[1] = __ldg(reinterpret_cast<const uint4*>(a.weight) + 32 + lane);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (pos[i] < 0) continue;  // (the same for the whole warp)
    const int64_t row = row0 + i;
    if (slot[i] != -1 && (slot[i] < 0 || slot[i] >= a.num_slots)) {
      if (lane == 0) report(a.dev_status, a.debug, MLA_CHECK_BAD_SLOT);
      slot[i] = -1;
    }
    const float* t = a.cos_sin + (int64_t)pos[i] * kDRope;
    float x = bf16_lo(rope[i]), y = bf16_hi(rope[i]);
    if (a.halves) {  // lane l has dims 2l, 2l + 1; their partners are 32 dims away, on lane l ^ 16
      const int k = (2 * lane) & 31;
      const float2 c = __ldg(reinterpret_cast<const float2*>(t + k)), s = __ldg(reinterpret_cast<const float2*>(t + kPairs + k));
      const float px = __shfl_xor_sync(0xffffffffu, x, 16), py = __shfl_xor_sync(0xffffffffu, y, 16);
      const float sx = lane < 16 ? -s.x : s.x, sy = lane < 16 ? -s.y : s.y;
      x = fmaf(px, sx, x * c.x);
      y = fmaf(py, sy, y * c.y);
    } else {
      const float c = __ldg(t + lane), s = __ldg(t + kPairs + lane), x0 = x;
      x = fmaf(-y, s, x0 * c);
      y = fmaf(x0, s, y * c);
    }
    rope[i] = pack_bf16(x, y);
    if (a.weight) {
      float f[2][8], ss = 0.f;
      unpack8(v[i][0], f[0]);
      unpack8(v[i][1], f[1]);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[0][j], f[0][j], fmaf(f[1][j], f[1][j], ss));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
      const float r = rsqrtf(fmaf(ss, 1.f / kDLatent, a.eps));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float g[8];
        unpack8(w[h], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[h][j] = f[h][j] * r * g[j];
        v[i][h] = pack8(f[h]);
      }
    }
    if (a.rows_out) {
      __nv_bfloat16* dst = a.rows_out + row * kDK;
      reinterpret_cast<uint4*>(dst)[lane] = v[i][0];
      reinterpret_cast<uint4*>(dst)[32 + lane] = v[i][1];
      reinterpret_cast<uint32_t*>(dst + kDLatent)[lane] = rope[i];
    }
    if (slot[i] < 0) continue;
    if (a.pool_format == MLA_POOL_BF16) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.pool) + slot[i] * kDK;
      reinterpret_cast<uint4*>(dst)[lane] = v[i][0];
      reinterpret_cast<uint4*>(dst)[32 + lane] = v[i][1];
      reinterpret_cast<uint32_t*>(dst + kDLatent)[lane] = rope[i];
    } else {  // as mla_kv4_append: two lanes share a block of 16 dims
      uint8_t* dst = static_cast<uint8_t*>(a.pool) + slot[i] * kKv4Row;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t top = top_of(v[i][h]);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        const uint32_t s = block_scale(top);
        reinterpret_cast<uint32_t*>(dst)[32 * h + lane] = block_codes(v[i][h], s);
        if ((lane & 1) == 0) dst[kKv4Codes + 16 * h + (lane >> 1)] = (uint8_t)s;
      }
      reinterpret_cast<uint32_t*>(dst + kKv4Rope)[lane] = rope[i];
    }
  }
}

// N heads of a group of G lanes, 32 / G groups a warp; item0 is the first head of the warp, counted over tokens and heads.
template <int G, int N>
__device__ __forceinline__ void do_heads(const RopeArgs& a, uint32_t item0, uint32_t items) {
  const int lane = threadIdx.x & 31, at = lane & (G - 1), chunks = a.head_dim >> 3, rope0 = chunks - 8;
  const int part = at - rope0;  // 0..7: the lane holds RoPE dims 8 part ..
  const bool turns = part >= 0 && part < 8, active = at < chunks && (a.copy || turns);
  int32_t pos[N];
  int64_t out_at[N];
  uint4 v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t item = item0 + i * (32 / G) + lane / G;
    const bool real = item < items;
    const uint32_t token = real ? item / (uint32_t)a.num_heads : 0, head = real ? item - token * (uint32_t)a.num_heads : 0;
    pos[i] = real ? load_position(a, token, at == 0 && head == 0 && !a.rows) : -1;
    out_at[i] = token * a.qo_ts + head * a.qo_hs + 8 * at;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (real && active) v[i] = ld16(a.q + token * a.q_ts + head * a.q_hs + 8 * at);
  }
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if (a.q_weight && active) w = __ldg(reinterpret_cast<const uint4*>(a.q_weight) + at);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float x[8];
    unpack8(v[i], x);
    if (a.q_weight) {
      float ss = 0.f, g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
      for (int d = G / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
      const float r = rsqrtf(ss / (float)a.head_dim + a.eps);
      unpack8(w, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] * r * g[j];
    }
    const float* t = a.cos_sin + (int64_t)max(pos[i], 0) * kDRope;
    if (a.halves) {  // dim k's partner is 32 dims, four lanes, away
      float p[8];
      const int from = (lane & ~(G - 1)) + rope0 + ((part & 7) ^ 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = __shfl_sync(0xffffffffu, x[j], from);
      if (turns) {
        const float4* c = reinterpret_cast<const float4*>(t + 8 * (part & 3));
        const float4* s = reinterpret_cast<const float4*>(t + kPairs + 8 * (part & 3));
        const float4 c0 = __ldg(c), c1 = __ldg(c + 1), s0 = __ldg(s), s1 = __ldg(s + 1);
        const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaf(p[j], part < 4 ? -sv[j] : sv[j], x[j] * cc[j]);
      }
    } else if (turns) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(t) + part), s = __ldg(reinterpret_cast<const float4*>(t + kPairs) + part);
      const float cc[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x0 = x[2 * j], y0 = x[2 * j + 1];
        x[2 * j] = fmaf(-y0, sv[j], x0 * cc[j]);
        x[2 * j + 1] = fmaf(x0, sv[j], y0 * cc[j]);
      }
    }
    if (pos[i] >= 0 && active) *reinterpret_cast<uint4*>(a.q_out + out_at[i]) = pack8(x);
  }
}

// ROWS rows a warp and HEADS heads a group of G lanes.
template <int G, int ROWS, int HEADS>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs a) {
  const int warp = threadIdx.x >> 5;
  if ((int64_t)blockIdx.x < a.row_blocks) {
    do_rows<ROWS>(a, ((int64_t)blockIdx.x * kWarps + warp) * ROWS);
  } else {
    const uint32_t items = (uint32_t)(a.num_rows * a.num_heads);
    const uint64_t item0 = ((uint64_t)(blockIdx.x - a.row_blocks) * kWarps + warp) * (32 / G * HEADS);
    if (item0 < items) do_heads<G, HEADS>(a, (uint32_t)item0, items);
  }
}

template <int ROWS, int HEADS>
cudaError_t launch(RopeArgs a, cudaStream_t stream) {
  const int G = a.head_dim <= 64 ? 8 : a.head_dim <= 128 ? 16 : 32;
  const int64_t per_row = kWarps * ROWS, per_head = (int64_t)kWarps * (32 / G) * HEADS;
  a.row_blocks = a.rows ? (a.num_rows + per_row - 1) / per_row : 0;
  const int64_t blocks = a.row_blocks + (a.q ? (a.num_rows * a.num_heads + per_head - 1) / per_head : 0);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  if (G == 8) rope_append_kernel<8, ROWS, HEADS><<<(unsigned)blocks, kRopeThreads, 0, stream>>>(a);
  else if (G == 16) rope_append_kernel<16, ROWS, HEADS><<<(unsigned)blocks, kRopeThreads, 0, stream>>>(a);
  else rope_append_kernel<32, ROWS, HEADS><<<(unsigned)blocks, kRopeThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

bool good_stride(int64_t s) { return s >= 0 && s % 8 == 0 && s <= (1ll << 38); }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_rope_append(const mla_rope_desc* d, const void* rows, const void* weight, const void* q,
                               const void* q_weight, const int32_t* positions, const float* cos_sin,
                               const int32_t* slot_map, void* pool, void* rows_out, void* q_out, int32_t debug,
                               int32_t* dev_status, mla_stream_t stream) {
  if (!d || d->num_rows < 0 || d->num_rows > 0x7fffffff || d->num_positions < 1) return MLA_ERR_INVALID_ARGUMENT;
  if (!isfinite(d->eps) || d->eps < 0.f || (d->pairs != MLA_ROPE_ADJACENT && d->pairs != MLA_ROPE_HALVES))
    return MLA_ERR_INVALID_ARGUMENT;
  if (!rows && !q) return d->num_rows == 0 ? MLA_OK : MLA_ERR_INVALID_ARGUMENT;
  if (!positions || !cos_sin || !aligned(positions, 4) || !aligned(cos_sin, 16)) return MLA_ERR_INVALID_ARGUMENT;
  if (debug && !dev_status) return MLA_ERR_INVALID_ARGUMENT;
  if (rows) {
    if (d->pool_format < MLA_POOL_NONE || d->pool_format > MLA_POOL_KV4) return MLA_ERR_INVALID_ARGUMENT;
    if (!aligned(rows, 16) || d->row_stride < kDK || !good_stride(d->row_stride) || !aligned(weight, 16) || !aligned(rows_out, 16))
      return MLA_ERR_INVALID_ARGUMENT;
    if (d->pool_format == MLA_POOL_NONE ? (pool || slot_map || !rows_out) : (!pool || !slot_map)) return MLA_ERR_INVALID_ARGUMENT;
    if (!aligned(pool, d->pool_format == MLA_POOL_KV4 ? 32 : 16) || !aligned(slot_map, 4)) return MLA_ERR_INVALID_ARGUMENT;
    if (pool && (d->num_slots < 1 || d->num_slots > 0x7fffffff)) return MLA_ERR_INVALID_ARGUMENT;
    if (rows == rows_out && d->row_stride != kDK) return MLA_ERR_INVALID_ARGUMENT;
  } else if (weight || pool || slot_map || rows_out) {
    return MLA_ERR_INVALID_ARGUMENT;
  }
  if (q) {
    if (!q_out || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(q_weight, 16)) return MLA_ERR_INVALID_ARGUMENT;
    if (d->num_heads < 1 || d->head_dim < kDRope || d->head_dim % 8 != 0) return MLA_ERR_INVALID_ARGUMENT;
    if (d->head_dim > kMaxHeadDim || d->num_rows * d->num_heads > 0xffffffffll) return MLA_ERR_UNSUPPORTED;
    if (!good_stride(d->q_token_stride) || !good_stride(d->q_head_stride) || !good_stride(d->q_out_token_stride) ||
        !good_stride(d->q_out_head_stride))
      return MLA_ERR_INVALID_ARGUMENT;
    // heads of q_out that would overlap: neither all heads of a token nor all tokens of a head fit between two of the others
    const int64_t token_span = (d->num_heads - 1) * d->q_out_head_stride + d->head_dim;
    const int64_t head_span = (d->num_rows - 1) * d->q_out_token_stride + d->head_dim;
    if (d->num_heads > 1 && d->q_out_head_stride < d->head_dim) return MLA_ERR_INVALID_ARGUMENT;
    if (d->num_rows > 1 && d->q_out_token_stride < (d->num_heads > 1 && d->q_out_head_stride >= head_span ? d->head_dim : token_span))
      return MLA_ERR_INVALID_ARGUMENT;
    if (q == q_out && ((d->num_rows > 1 && d->q_token_stride != d->q_out_token_stride) ||
                       (d->num_heads > 1 && d->q_head_stride != d->q_out_head_stride)))
      return MLA_ERR_INVALID_ARGUMENT;
  } else if (q_weight || q_out) {
    return MLA_ERR_INVALID_ARGUMENT;
  }
  if (d->num_rows == 0) return MLA_OK;
  RopeArgs a = {};
  a.rows = static_cast<const __nv_bfloat16*>(rows);
  a.weight = static_cast<const __nv_bfloat16*>(weight);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.slot_map = slot_map;
  a.pool = pool;
  a.rows_out = static_cast<__nv_bfloat16*>(rows_out);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.dev_status = dev_status;
  a.num_rows = d->num_rows;
  a.row_stride = d->row_stride;
  a.num_slots = d->num_slots;
  a.q_ts = d->q_token_stride;
  a.q_hs = d->q_head_stride;
  a.qo_ts = d->q_out_token_stride;
  a.qo_hs = d->q_out_head_stride;
  a.pool_format = rows ? d->pool_format : MLA_POOL_NONE;
  a.num_heads = q ? d->num_heads : 1;
  a.head_dim = q ? d->head_dim : kDRope;
  a.num_positions = d->num_positions;
  a.halves = d->pairs == MLA_ROPE_HALVES;
  a.debug = debug;
  a.copy = q_weight || q != q_out;
  a.eps = d->eps;
  return launch<2, kHeadsInFlight>(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
