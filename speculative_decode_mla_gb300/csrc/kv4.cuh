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

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The e4m3 scale of a block: max|x| / 6, the exact quotient rounded to nearest even and at most
// 448; NaN (0x7f) when the block holds a NaN or an infinity. `top`: the largest bf16 magnitude as bits.
// top times fp32's 1/6 serves as the quotient: fp32's 1/6 is off by 2^-25 of itself. If top / 6 is a midpoint m of e4m3
// (at most 5 significant bits), the product lies within m * 2^-25 of m, under half an ulp, and rounds to m; if not, it
// is off every midpoint by 2^-8 of its size (top has 8 significant bits, 6 m has 7), so rounding twice is harmless.
__device__ __forceinline__ uint32_t block_scale(uint32_t top) {
  uint16_t s;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s) : "f"(0.f), "f"(__uint_as_float(top << 16) * (1.f / 6.f)));
  return top >= 0x7f80u ? 0x7fu : s & 0xffu;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
// Codes of eight values (four words of bf16 pairs) under the scale byte. y = x / s is taken as x * r, r = 1 / s within
// 2^-23 of itself, and rounded to a multiple of 2^-11 by adding and taking away 1.5 * 2^12: a quotient on one
// of e2m1's midpoints (0.25 .. 5) comes out exactly on it, and any other stays off it, since x has 8
// significant bits and s * midpoint at most 7, so they differ by 2^-8 of their size or not at all.
__device__ __forceinline__ uint32_t block_codes(const uint4& w, uint32_t scale) {
  const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(scale) & 0xffffu)));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));  // (s is 0, NaN or a normal fp32 number)
  const uint64_t rr = pack2(r, r), magic = pack2(6144.f, 6144.f), minus = pack2(-6144.f, -6144.f);
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t v = pack2(bf16_lo(x[i]), bf16_hi(x[i]));
    asm("{\n.reg .b64 y;\n.reg .f32 lo, hi;\n.reg .b8 d;\n"
        "fma.rn.f32x2 y, %1, %2, %3;\nadd.rn.f32x2 y, y, %4;\nmov.b64 {lo, hi}, y;\n"
        "cvt.rn.satfinite.e2m1x2.f32 d, hi, lo;\nmov.b32 %0, {d, 0, 0, 0};\n}"
        : "=r"(c[i])
        : "l"(v), "l"(rr), "l"(magic), "l"(minus));
    const uint32_t sign = x[i] & 0x80008000u;  // a negative value that rounds to zero has lost its sign by now
    c[i] |= (sign >> 12) | (sign >> 24);       // (only the low byte is used)
  }
  const uint32_t out = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  return s > 0.f ? out : 0u;  // (scale 0 or NaN: codes 0)
}

__device__ __forceinline__ uint32_t top_of(const uint4& w) {
  uint32_t t = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
  return max(t & 0xffffu, t >> 16);
}

}  // namespace mla
