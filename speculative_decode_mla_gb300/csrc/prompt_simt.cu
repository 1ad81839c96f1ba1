// Prompt attention, plain fp32 reference kernel (one warp a query row and head), and the merge of parts.
#include "prompt.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Lane l holds dims l, l + 32, ... of the query, the key (192 dims) and the output (128 dims).
__global__ void __launch_bounds__(kThreads) prompt_simt_kernel(const PromptArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), rows = a.num_q * a.H;
  if (unit >= rows) return;
  const int64_t rh = unit, row = rh / a.H;
  const int h = (int)(rh % a.H), g = h / a.group;
  PromptSeq s;
  if (sequence_of(a, row, s) < 0) return;
  const int32_t vis = visible(a, s, (int32_t)(row - s.q0));
  float q[6], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < 6; ++j) q[j] = __bfloat162float(a.q[row * a.q_ts + h * a.q_hs + lane + 32 * j]);
  for (int64_t t = 0; t < vis; ++t) {
    const __nv_bfloat16* k = a.k + (s.k0 + t) * a.k_ts + g * a.k_hs;
    const __nv_bfloat16* kr = a.kr + (s.k0 + t) * a.kr_ts;
    const __nv_bfloat16* v = a.v + (s.k0 + t) * a.v_ts + g * a.v_hs;
    float x = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) x = fmaf(q[j], __bfloat162float(k[lane + 32 * j]), x);
#pragma unroll
    for (int j = 0; j < 2; ++j) x = fmaf(q[4 + j], __bfloat162float(kr[lane + 32 * j]), x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= a.scale;
    const float top = fmaxf(m, x);
    const float keep = m == top ? 1.f : expf(m - top), p = expf(x - (top == -INFINITY ? 0.f : top));
    m = top;
    l = fmaf(l, keep, p);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = fmaf(o[j], keep, p * __bfloat162float(v[lane + 32 * j]));
  }
  const float inv = l == 0.f ? 0.f : 1.f / l, lse = l == 0.f ? -INFINITY : m + logf(l);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t at = rh * kHeadV + lane + 32 * j;
    if (a.out_f32) static_cast<float*>(a.out)[at] = o[j] * inv;
    else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(o[j] * inv);
  }
  if (lane == 0) a.lse[rh] = lse;
}

// One warp a row of a unit that CTAs share, four dims a lane: the sum of the parts weighted by exp(lse - largest lse). Bound
// by reading the parts once (they mostly lie in L2). Block (c, y): rows of the unit that ends with CTA c's part.
__global__ void __launch_bounds__(kThreads) prompt_merge_kernel(const PromptArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, row = blockIdx.y * kWarps + (threadIdx.x >> 5), last = blockIdx.x;
  const PromptMerge u = a.merges[last];
  if (!u.live || row >= u.rows) return;
  const auto part = [&](int c) { return ((int64_t)c * 2 + (c == u.first ? u.slot : 0)) * a.rows_per_unit + row; };
  float top = -INFINITY, bad = 0.f;
  for (int c = u.first + lane; c <= last; c += 32) {
    const float x = a.part_lse[part(c)];
    bad += x != x ? 1.f : 0.f;
    top = fmaxf(top, x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    bad += __shfl_xor_sync(0xffffffffu, bad, d);
  }
  if (bad > 0.f) top = NAN;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float z = 0.f;
#pragma unroll 4
  for (int c = u.first; c <= last; ++c) {
    const float x = a.part_lse[part(c)];
    if (x == -INFINITY) continue;  // (the same for the whole warp)
    const float w = expf(x - top);
    const float4 v = *reinterpret_cast<const float4*>(a.part_o + part(c) * kHeadV + 4 * lane);
    z += w;
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
  const float inv = z == 0.f ? 0.f : 1.f / z;
  const int at = u.row0 + row;
  const int64_t rh = (int64_t)(u.q0 + (at >> a.pack_log)) * a.H + u.head + (at & (a.pack - 1));
  if (a.out_f32) {
    reinterpret_cast<float4*>(static_cast<float*>(a.out) + rh * kHeadV)[lane] = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + rh * kHeadV)[lane] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
  if (lane == 0) a.lse[rh] = z == 0.f ? -INFINITY : top + logf(z);
}

}  // namespace

cudaError_t launch_prompt_simt(const PromptArgs& a, cudaStream_t stream) {
  const int64_t blocks = (a.num_q * a.H + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  prompt_simt_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_prompt_merge(const PromptArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.ctas, (unsigned)(a.rows_per_unit / kWarps));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_merge_kernel, a);
}

}  // namespace mla
