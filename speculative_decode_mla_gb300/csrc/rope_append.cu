// A layer's latent rows and query heads: norm, rotation of the RoPE dims, and the rows' way into the pool
// (declared in include/mla_prompt.h).
//
// Bound by memory, or, for a decode step, by the latency of one launch; so both parts run in one launch: the first blocks take
// rows, the others query heads. A warp takes a row: 16 latent dims and one adjacent pair of RoPE dims a lane, the sum
// of squares over the warp. A group of 8 lanes (16 or 32 for uneven head sizes) takes a query head, so that heads of 64 dims, the
// RoPE dims alone, fill the warp too. All loads of a row, or of the heads of a warp, are out before one is used.
//   16,384 tokens with 64 heads of 192 dims, norms, rows and pool: 137 us, 6.3 TB/s (93% of the copy rate)
//   65,536 rows into the 4-bit pool: 34 us; 61 tokens with 64 heads of 64 dims, a decode step: 3 us
#include <math.h>

#include "kv4.cuh"
#include "mla_prompt.h"
#include "tc.cuh"

namespace mla {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kWarps = kRopeThreads / 32;
constexpr int kPairs = kDRope / 2;
constexpr int kMaxHeadDim = 256;

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
  int32_t head_units;  // warps that a token's heads take
  float eps, inv_dim;
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

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 ra, rb, rd;\nmov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %5};\nmul.rn.f32x2 rd, ra, rb;\nmov.b64 {%0, %1}, rd;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
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

// One row of a warp.
__device__ __forceinline__ void do_row(const RopeArgs& a, int64_t row) {
  if (row >= a.num_rows) return;
  const int lane = threadIdx.x & 31;
  const __nv_bfloat16* src = a.rows + row * a.row_stride;
  const int32_t pos = load_position(a, row, lane == 0);
  int64_t slot = a.pool_format != MLA_POOL_NONE ? a.slot_map[row] : -1;
  uint4 v[2] = {ld16(src + 8 * lane), ld16(src + 256 + 8 * lane)};
  uint32_t rope = *(reinterpret_cast<const uint32_t*>(src + kDLatent) + lane);
  if (pos < 0) return;
  if (slot != -1 && (slot < 0 || slot >= a.num_slots)) {
    if (lane == 0) report(a.dev_status, a.debug, MLA_CHECK_BAD_SLOT);
    slot = -1;
  }
  const float* t = a.cos_sin + (int64_t)pos * kDRope;
  float x = bf16_lo(rope), y = bf16_hi(rope);
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
  rope = pack_bf16(x, y);
  if (a.weight) {
    const uint4 w[2] = {__ldg(reinterpret_cast<const uint4*>(a.weight) + lane), __ldg(reinterpret_cast<const uint4*>(a.weight) + 32 + lane)};
    float f[2][8], ss = 0.f;
    unpack8(v[0], f[0]);
    unpack8(v[1], f[1]);
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
      v[h] = pack8(f[h]);
    }
  }
  if (a.rows_out) {
    __nv_bfloat16* dst = a.rows_out + row * kDK;
    reinterpret_cast<uint4*>(dst)[lane] = v[0];
    reinterpret_cast<uint4*>(dst)[32 + lane] = v[1];
    reinterpret_cast<uint32_t*>(dst + kDLatent)[lane] = rope;
  }
  if (slot < 0) return;
  if (a.pool_format == MLA_POOL_BF16) {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.pool) + slot * kDK;
    reinterpret_cast<uint4*>(dst)[lane] = v[0];
    reinterpret_cast<uint4*>(dst)[32 + lane] = v[1];
    reinterpret_cast<uint32_t*>(dst + kDLatent)[lane] = rope;
  } else {  // as mla_kv4_append: two lanes share a block of 16 dims
    uint8_t* dst = static_cast<uint8_t*>(a.pool) + slot * kKv4Row;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t top = top_of(v[h]);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      const uint32_t s = block_scale(top);
      reinterpret_cast<uint32_t*>(dst)[32 * h + lane] = block_codes(v[h], s);
      if ((lane & 1) == 0) dst[kKv4Codes + 16 * h + (lane >> 1)] = (uint8_t)s;
    }
    reinterpret_cast<uint32_t*>(dst + kKv4Rope)[lane] = rope;
  }
}

// N heads for each group of G lanes, 32 / G groups a warp, all of one token: its angles are loaded once. A lane holds K pieces
// of 16 bytes, G pieces apart. Heads of 64, 128, 192 and 256 dims take eight lanes, so that every lane holds one piece of the RoPE
// dims and none is idle (16,384 tokens, 64 heads of 192 dims: 137 us; with 32 lanes a head and one piece a lane 157, the issue
// slots 72% in use); others 16 or 32 and one piece.
template <int G, int K, int N, bool HALVES, bool NORM>
__device__ __forceinline__ void do_heads(const RopeArgs& a, uint32_t unit) {
  const int lane = threadIdx.x & 31, at = lane & (G - 1), chunks = a.head_dim >> 3, rope0 = chunks - 8;
  const int part = at + G * (K - 1) - rope0;  // 0..7: the lane's last piece holds RoPE dims 8 part ..
  const bool turns = K > 1 || G == 8 || (part >= 0 && part < 8), last = K > 1 || G == 8 || (at < chunks && (a.copy || turns));
  const uint32_t token = unit / (uint32_t)a.head_units;
  const int head0 = (int)(unit - token * (uint32_t)a.head_units) * (32 / G * N) + lane / G;
  const int32_t pos = load_position(a, token, lane == 0 && head0 == 0 && !a.rows);
  const __nv_bfloat16* src = a.q + (int64_t)token * a.q_ts + (int64_t)head0 * a.q_hs + 8 * at;
  uint4 v[N][K];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[i][k] = make_uint4(0u, 0u, 0u, 0u);
      if ((k < K - 1 ? a.copy != 0 : last) && head0 + i * (32 / G) < a.num_heads)
        v[i][k] = ld16(src + (int64_t)(i * (32 / G)) * a.q_hs + 8 * G * k);
    }
  if (pos < 0) return;  // (the whole warp)
  uint4 w[NORM ? K : 1];
#pragma unroll
  for (int k = 0; k < (NORM ? K : 0); ++k) {
    w[k] = make_uint4(0u, 0u, 0u, 0u);
    if (k < K - 1 || last) w[k] = __ldg(reinterpret_cast<const uint4*>(a.q_weight) + at + G * k);
  }
  // the angles: of adjacent pairs 4 part .. 4 part + 3, or of the dims 8 part .. 8 part + 7 (mod 32)
  float4 c[HALVES ? 2 : 1] = {}, s[HALVES ? 2 : 1] = {};
  if (turns) {
    const float4* t = reinterpret_cast<const float4*>(a.cos_sin + (int64_t)pos * kDRope);
#pragma unroll
    for (int j = 0; j < (HALVES ? 2 : 1); ++j) {
      c[j] = __ldg(t + (HALVES ? 2 * (part & 3) + j : part));
      s[j] = __ldg(t + kPairs / 4 + (HALVES ? 2 * (part & 3) + j : part));
    }
  }
  __nv_bfloat16* dst = a.q_out + (int64_t)token * a.qo_ts + (int64_t)head0 * a.qo_hs + 8 * at;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float2 scale = make_float2(1.f, 1.f);
    if (NORM) {
      float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float x[8];
        unpack8(v[i][k], x);
#pragma unroll
        for (int j = 0; j < 8; j += 2) s2 = fma2(make_float2(x[j], x[j + 1]), make_float2(x[j], x[j + 1]), s2);
      }
      float ss = s2.x + s2.y;
#pragma unroll
      for (int d = G / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
      scale.x = scale.y = rsqrtf(fmaf(ss, a.inv_dim, a.eps));
    }
    const bool real = head0 + i * (32 / G) < a.num_heads;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool mine = real && (k < K - 1 ? a.copy != 0 : last);
      if (k < K - 1 && !NORM) {
        if (mine) *reinterpret_cast<uint4*>(dst + (int64_t)(i * (32 / G)) * a.qo_hs + 8 * G * k) = v[i][k];
        continue;
      }
      float x[8];
      unpack8(v[i][k], x);
      if (NORM) {
        float g[8];
        unpack8(w[k], g);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float2 y = mul2(mul2(make_float2(x[j], x[j + 1]), scale), make_float2(g[j], g[j + 1]));
          x[j] = y.x;
          x[j + 1] = y.y;
        }
      }
      if (k == K - 1 && HALVES) {  // dim j's partner is 32 dims, four lanes, away
        float p[8];
        const int from = (lane & ~(G - 1)) + rope0 - G * (K - 1) + ((part & 7) ^ 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = __shfl_sync(0xffffffffu, x[j], from);
        const float cc[8] = {c[0].x, c[0].y, c[0].z, c[0].w, c[HALVES].x, c[HALVES].y, c[HALVES].z, c[HALVES].w};
        const float sv[8] = {s[0].x, s[0].y, s[0].z, s[0].w, s[HALVES].x, s[HALVES].y, s[HALVES].z, s[HALVES].w};
        if (turns)
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = fmaf(p[j], part < 4 ? -sv[j] : sv[j], x[j] * cc[j]);
      } else if (k == K - 1 && turns) {
        const float cc[4] = {c[0].x, c[0].y, c[0].z, c[0].w}, sv[4] = {s[0].x, s[0].y, s[0].z, s[0].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = x[2 * j], y0 = x[2 * j + 1];
          x[2 * j] = fmaf(-y0, sv[j], x0 * cc[j]);
          x[2 * j + 1] = fmaf(x0, sv[j], y0 * cc[j]);
        }
      }
      if (mine) *reinterpret_cast<uint4*>(dst + (int64_t)(i * (32 / G)) * a.qo_hs + 8 * G * k) = pack8(x);
    }
  }
}

// Blocks on an SM and heads in flight: enough bytes under way, with no more than a few registers spilled (40 bytes with norms of 192 dims, 8 with norms
// and halves of 256, none elsewhere). 16,384 tokens, 64 heads of 192 dims,
// adjacent pairs, norms, us: one head a group and 4, 5, 6 blocks 153, 143, 143; two and 4, 5, 6 blocks 137, 203, 252 (spills). Pairs half a
// head apart take more registers: 2111 tokens of 5 heads 5.5 with one head a group, 6.8 with two. Rows alone, 65,536 into the
// 4-bit pool and read back: 60.5 with 4 blocks, 54.7 with 6, 51.2 with 8.
__host__ __device__ constexpr int blocks_on_sm(int heads) { return heads == 0 ? 8 : 4; }

// A row a warp, and HEADS heads (0: rows alone) a group of G lanes, K pieces a lane.
template <int G, int K, int HEADS, bool HALVES, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, blocks_on_sm(HEADS)) rope_append_kernel(const RopeArgs a) {
  const int warp = threadIdx.x >> 5;
  if (HEADS == 0 || (int64_t)blockIdx.x < a.row_blocks) {
    do_row(a, (int64_t)blockIdx.x * kWarps + warp);
  } else if constexpr (HEADS > 0) {
    const uint64_t unit = (uint64_t)(blockIdx.x - a.row_blocks) * kWarps + warp;
    if (unit < (uint64_t)a.num_rows * a.head_units) do_heads<G, K, HEADS, HALVES, NORM>(a, (uint32_t)unit);
  }
}

template <int G, int K, int HEADS, bool HALVES, bool NORM>
cudaError_t launch(RopeArgs a, cudaStream_t stream) {
  constexpr int per_warp = HEADS ? 32 / G * HEADS : 1;
  a.head_units = HEADS ? (a.num_heads + per_warp - 1) / per_warp : 0;
  a.row_blocks = a.rows ? (a.num_rows + kWarps - 1) / kWarps : 0;
  const int64_t blocks = a.row_blocks + (a.num_rows * a.head_units + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  rope_append_kernel<G, K, HEADS, HALVES, NORM><<<(unsigned)blocks, kRopeThreads, 0, stream>>>(a);
  return cudaGetLastError();
}
// HEADS: heads in flight of adjacent pairs, half as many of pairs half a head apart.
template <int G, int K, int HEADS>
cudaError_t launch_heads(const RopeArgs& a, cudaStream_t stream) {
  if (a.halves) return a.q_weight ? launch<G, K, (HEADS + 1) / 2, true, true>(a, stream) : launch<G, K, (HEADS + 1) / 2, true, false>(a, stream);
  return a.q_weight ? launch<G, K, HEADS, false, true>(a, stream) : launch<G, K, HEADS, false, false>(a, stream);
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
  a.inv_dim = 1.f / (float)a.head_dim;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = !q                       ? launch<8, 1, 0, false, false>(a, s)
                        : a.head_dim == 64       ? launch_heads<8, 1, 4>(a, s)
                        : a.head_dim == 128      ? launch_heads<8, 2, 2>(a, s)
                        : a.head_dim == 192      ? launch_heads<8, 3, 2>(a, s)
                        : a.head_dim == 256      ? launch_heads<8, 4, 1>(a, s)
                        : a.head_dim <= 128      ? launch_heads<16, 1, 4>(a, s)
                                                 : launch_heads<32, 1, 4>(a, s);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
