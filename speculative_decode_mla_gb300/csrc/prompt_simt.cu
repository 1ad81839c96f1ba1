// Prompt attention, plain fp32 reference kernel (one warp a query row and head), and the merge of parts.
#include "prompt.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Lane l holds dims l, l + 32, ... of the query, the key (192 dims) and the output (128 dims). Sums are taken over 128 keys first and then
// over these, so that a total of many keys does not round each of them to its own last place (as add_keeping says).
__global__ void __launch_bounds__(kThreads) prompt_simt_kernel(const PromptArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), rows = a.num_q * a.H;
  if (unit >= rows) return;
  const int64_t rh = unit, row = rh / a.H;
  const int h = (int)(rh % a.H), g = h / a.group;
  PromptSeq s;
  if (sequence_of(a, row, s) < 0) return;
  const int32_t vis = visible(a, s, (int32_t)(row - s.q0));
  float q[6], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f, l_low = 0.f;
  float part_o[4] = {0.f, 0.f, 0.f, 0.f}, part_l = 0.f;  // of the keys since the last whole 128
  const auto add_part = [&] {
    add_keeping(l, l_low, part_l);
    part_l = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[j] += part_o[j];
      part_o[j] = 0.f;
    }
  };
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
    l *= keep;
    l_low *= keep;
    part_l = fmaf(part_l, keep, p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[j] *= keep;
      part_o[j] = fmaf(part_o[j], keep, p * __bfloat162float(v[lane + 32 * j]));
    }
    if (t % 128 == 127) add_part();
  }
  add_part();
  l += l_low;
  const float inv = l == 0.f ? 0.f : 1.f / l, lse = l == 0.f ? -INFINITY : m + logf(l);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t at = rh * kHeadV + lane + 32 * j;
    if (a.out_f32) static_cast<float*>(a.out)[at] = o[j] * inv;
    else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(o[j] * inv);
  }
  if (lane == 0) a.lse[rh] = lse;
}

// The rows of units that CTAs share: the sum of the parts weighted by exp(lse - largest lse). Block (c, y): rows of the unit that ends
// with CTA c's part. A warp takes kRows rows, four dims a lane, and reads kAhead of their parts at a time. Reads that wait for each
// other are what this kernel is made of, so it takes two rows and two parts together where units are of 256 rows in few parts (16 heads
// of 4096 rows and keys: the call takes 125.1 us, 127.7 with a row and four parts), a row and four parts where they are of 128 rows at
// most and a sequence's keys can be in many parts (8 heads, 100 rows against 30100 keys: 38.7 us, 44.3 with two and two).
template <int kRows, int kAhead>
__global__ void __launch_bounds__(kThreads) prompt_merge_kernel(const PromptArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, last = blockIdx.x;
  const PromptMerge u = a.merges[last];
  const int row0 = (blockIdx.y * kWarps + (threadIdx.x >> 5)) * kRows, rows = min(kRows, u.rows - row0);
  if (!u.live || rows <= 0) return;
  float top[kRows], z[kRows];
  float4 o[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    top[i] = -INFINITY;
    z[i] = 0.f;
    o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll 1
  for (int c0 = u.first; c0 <= last; c0 += kAhead) {
    float x[kAhead][kRows];
    float4 v[kAhead][kRows];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int c = min(c0 + j, last);
      const int64_t part = ((int64_t)c * 2 + (c == u.first ? u.slot : 0)) * a.rows_per_unit + row0;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int64_t at = part + min(i, rows - 1);
        x[j][i] = c0 + j <= last ? a.part_lse[at] : -INFINITY;
        v[j][i] = *reinterpret_cast<const float4*>(a.part_o + at * kHeadV + 4 * lane);
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (x[j][i] == -INFINITY) continue;
        // (a NaN part: the row is NaN)
        const float most = x[j][i] > top[i] || x[j][i] != x[j][i] ? x[j][i] : top[i];
        const float w = expf(x[j][i] - most), keep = top[i] == -INFINITY ? 0.f : expf(top[i] - most);
        top[i] = most;
        z[i] = fmaf(z[i], keep, w);
        o[i].x = fmaf(w, v[j][i].x, o[i].x * keep);
        o[i].y = fmaf(w, v[j][i].y, o[i].y * keep);
        o[i].z = fmaf(w, v[j][i].z, o[i].z * keep);
        o[i].w = fmaf(w, v[j][i].w, o[i].w * keep);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (i >= rows) break;
    const float inv = z[i] == 0.f ? 0.f : 1.f / z[i];
    const int at = u.row0 + row0 + i;
    const int64_t rh = (int64_t)(u.q0 + (at >> a.pack_log)) * a.H + u.head + (at & (a.pack - 1));
    if (a.out_f32) {
      reinterpret_cast<float4*>(static_cast<float*>(a.out) + rh * kHeadV)[lane] = make_float4(o[i].x * inv, o[i].y * inv, o[i].z * inv, o[i].w * inv);
    } else {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(o[i].x * inv, o[i].y * inv), hi = __floats2bfloat162_rn(o[i].z * inv, o[i].w * inv);
      reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + rh * kHeadV)[lane] =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    if (lane == 0) a.lse[rh] = z[i] == 0.f ? -INFINITY : top[i] + logf(z[i]);
  }
}

__global__ void __launch_bounds__(kThreads) prompt_check_kernel(const PromptArgs a) {
  const int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (b < a.B) load_seq(a, (int)b);
}

}  // namespace

cudaError_t launch_prompt_check(const PromptArgs& a, cudaStream_t stream) {
  prompt_check_kernel<<<(unsigned)(((int64_t)a.B + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

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
  const bool large = a.rows_per_unit > kPromptTile;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.ctas, (unsigned)(a.rows_per_unit / (kWarps * (large ? 2 : 1))));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return large ? cudaLaunchKernelEx(&cfg, prompt_merge_kernel<2, 2>, a) : cudaLaunchKernelEx(&cfg, prompt_merge_kernel<1, 4>, a);
}

}  // namespace mla
