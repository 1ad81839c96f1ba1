// Plain SIMT reference kernel for tree-verify attention over the 4-bit pool (fp32 FMA, no tensor
// cores): the work split and partial layout of verify_simt.cu, one warp per query row, one position
// at a time. Lane l holds dims [16l, 16l + 16) of a row (one scale block) and the RoPE dims 2l, 2l + 1.
#include "kv4.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32) verify_kv4_simt_kernel(VerifyArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.y;
  const int b = blockIdx.x / a.row_tiles;
  const int tile = blockIdx.x % a.row_tiles;
  const int R = a.T * a.H;
  const int local_row = tile * a.rows_per_tile + warp;
  if (local_row >= R) return;
  const int i = local_row / a.H;
  const int64_t row = (int64_t)b * R + local_row;

  const int32_t L = load_len(a, b);
  const int32_t Tb = load_tree_size(a, b);
  const int64_t N = (int64_t)L + Tb;
  const int64_t t0 = (int64_t)s * a.chunk;
  const int64_t t1 = min(N, t0 + a.chunk);
  __half* po = a.part_o + ((int64_t)s * a.rows + row) * kDLatent;
  if (t0 >= t1 || i >= Tb) {  // nothing in this chunk, or a padding row of a smaller tree
    if (lane == 0) a.part_lse[(int64_t)s * a.rows + row] = -INFINITY;
    return;
  }
  const uint64_t anc = ancestor_mask(a, b, i);

  float q[16];
  const __nv_bfloat162* q2 = reinterpret_cast<const __nv_bfloat162*>(a.q + row * kDK);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = __bfloat1622float2(q2[8 * lane + j]);
    q[2 * j] = f.x;
    q[2 * j + 1] = f.y;
  }
  const float2 qr = __bfloat1622float2(q2[kDLatent / 2 + lane]);

  const uint8_t* pool = reinterpret_cast<const uint8_t*>(a.kv);
  float m = -INFINITY, l = 0.f;
  float o[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j] = 0.f;

  for (int64_t t = t0; t < t1; ++t) {
    if (t >= L && !((anc >> (t - L)) & 1ull)) continue;
    const uint8_t* src = pool + load_slot(a, b, L, t) * kKv4Row;
    const uint2 code = reinterpret_cast<const uint2*>(src)[lane];
    const float sc8 = __half2float(
        __ushort_as_half((unsigned short)(e4m3x2_to_f16x2(src[kKv4Codes + lane]) & 0xffffu)));
    const float2 kr = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(src + kKv4Rope)[lane]);
    float k[16];
    float dot = fmaf(qr.x, kr.x, qr.y * kr.y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t h = e2m1x2_to_f16x2((j < 4 ? code.x >> (8 * j) : code.y >> (8 * (j - 4))) & 0xffu);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      k[2 * j] = f.x * sc8;
      k[2 * j + 1] = f.y * sc8;
      dot = fmaf(q[2 * j], k[2 * j], fmaf(q[2 * j + 1], k[2 * j + 1], dot));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    const float sc = dot * a.scale;
    if (sc == -INFINITY) continue;               // weight 0
    const float m_new = sc > m ? sc : m;         // (a NaN score does not become the maximum: it reaches l and o)
    const float m_ref = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = expf(m - m_ref);         // 0 on the first visible position (m = -inf)
    const float p = expf(sc - m_ref);
    l = l * alpha + p;
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = fmaf(p, k[j], o[j] * alpha);
    m = m_new;
  }
  if (m == -INFINITY && l == 0.f) {  // nothing visible to this row in this chunk
    if (lane == 0) a.part_lse[(int64_t)s * a.rows + row] = -INFINITY;
    return;
  }
  const float inv = 1.f / l;
  __half2* po2 = reinterpret_cast<__half2*>(po) + 8 * lane;
#pragma unroll
  for (int j = 0; j < 8; ++j) po2[j] = __floats2half2_rn(o[2 * j] * inv, o[2 * j + 1] * inv);
  if (lane == 0) a.part_lse[(int64_t)s * a.rows + row] = l == l ? m + logf(l) : l;
}

}  // namespace

cudaError_t launch_verify_kv4_simt(const VerifyArgs& a, cudaStream_t stream) {
  dim3 grid((unsigned)(a.B * a.row_tiles), (unsigned)a.splits);
  verify_kv4_simt_kernel<<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
