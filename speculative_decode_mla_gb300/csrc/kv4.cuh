// The 4-bit row format (include/mla_kv4.h) on the device.
#pragma once

#include "common.cuh"
#include "mla_kv4.h"

namespace mla {

constexpr int kKv4Block = 16;                              // latent dims to a scale
constexpr int kKv4Codes = kDLatent / 2;                    // 256 bytes of codes
constexpr int kKv4Scales = kDLatent / kKv4Block;           // 32 bytes of scales
constexpr int kKv4Rope = kKv4Codes + kKv4Scales;           // the RoPE dims start here
constexpr int kKv4Row = kKv4Rope + 2 * kDRope;             // 416 bytes
static_assert(kKv4Row == MLA_KV4_ROW_BYTES && kKv4Row % 16 == 0, "row format");

constexpr int kKv4TileTokens = 128;  // positions per tile of the tcgen05 kernel
// What starting and ending a run of tiles costs, in tiles. At 0, 1, 2, 3, 4 a batch of 32 sequences took 118, 116, 111,
// 114, 114 us, one of 61 took 119, 104, 101, 104, 106 (in the state of the kernel in which this was compared).
constexpr int kKv4SegmentUnits = 2;

// The two values of a code byte (dim 2i low, dim 2i+1 high) as packed fp16, exact.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte) {
  uint32_t h;
  asm("{\n.reg .b8 b0, b1, b2, b3;\nmov.b32 {b0, b1, b2, b3}, %1;\ncvt.rn.f16x2.e2m1x2 %0, b0;\n}" : "=r"(h) : "r"(byte));
  return h;
}
// Keys go into the score MMAs as fp16 times 2^-kKeyShift, still exact (a code times a scale is a multiple of 2^-10 below
// 2^12, fp16 holds multiples of 2^-24 of that many bits), so that the RoPE part of the scores, which lie in the same sum, has
// room: a query row is scaled by a power of two to [2^7, 2^8) at its largest, its RoPE dims in bf16 by 2^-kKeyShift more, below 2^-6,
// and 64 products with any finite bf16 keys then stay within fp32. Latent dims of Q are exact in fp16 down to 2^-24 of the row's
// largest and off by at most 2^-32 of it below that (the fp32 sum is off by 2^-24 of that largest one's product).
constexpr int kKeyShift = 14;
// k of the factor 2^k for a query row, given its largest magnitude as bf16 bits: rows with infinities or NaN stay as they are, and
// the two limits keep the factors and their inverses normal fp32 numbers (a row of 2^121 and more gets up to [2^14, 2^15)).
__device__ __forceinline__ int query_shift(uint32_t top) {
  const int e = (int)(top >> 7);
  return e == 255 ? 0 : max(-113, min(110, 134 - e));
}
__device__ __forceinline__ float exp2i(int k) { return __int_as_float((127 + k) << 23); }  // 2^k, -126 <= k <= 127
// What the row's sums are multiplied by to give scores in powers of two (never 0 or infinite: masked scores are).
__device__ __forceinline__ float score_scale(int query_shift, float scale_log2) {
  return fminf(fmaxf(exp2i(kKeyShift - query_shift) * scale_log2, 1.17549435e-38f), 3.402823466e38f);
}
// Two e4m3 scales as packed fp16, exact (a NaN stays one).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
  return h;
}
__device__ __forceinline__ uint32_t key_scales(uint32_t scales) {  // fp16 pairs times 2^-kKeyShift
  const uint32_t down = 0x04000400u;
  static_assert(kKeyShift == 14, "2^-14 in fp16");
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&scales), *reinterpret_cast<const __half2*>(&down));
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace mla
