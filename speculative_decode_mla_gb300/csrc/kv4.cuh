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
// Two e4m3 scales as packed fp16, exact (a NaN stays one).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pair));
  return h;
}

}  // namespace mla
