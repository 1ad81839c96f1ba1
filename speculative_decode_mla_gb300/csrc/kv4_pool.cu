// Rows into and out of the 4-bit latent pool (declared in include/mla_kv4.h).
//
// Both kernels are bound by memory: append reads 1152 + 4 bytes and writes 416 per row, gather the
// other way round. One warp takes a row at a time, kRowsPerWarp rows in flight, so every access is a run
// of 128 to 512 consecutive bytes and a warp has its loads out before it waits on one. Append and then gather
// of 65,536 rows (one in seven skipped): 34 us, 82% of the copy rate; gather of 184,320: 46.8 us, 92%. Append, whose issue
// slots are 61% in use, does without true divisions (see below): with two a row and lane the pair took 35.2 us, then 33.5.
#include "kv4.cuh"

namespace mla {
namespace {

constexpr int kPoolThreads = 256;
constexpr int kRowsPerWarp = 2;
constexpr int kRowsPerBlock = kPoolThreads / 32 * kRowsPerWarp;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
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

// Lane l quantises dims [8l, 8l + 8) and [256 + 8l, 256 + 8l + 8) of its warp's row: two lanes share a block.
__global__ void __launch_bounds__(kPoolThreads) kv4_append_kernel(uint8_t* __restrict__ pool, int64_t num_slots,
                                                                  const __nv_bfloat16* __restrict__ rows,
                                                                  int64_t row_stride,
                                                                  const int32_t* __restrict__ slot_map,
                                                                  int64_t num_rows, int32_t debug,
                                                                  int32_t* dev_status) {
  const int lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5) * kRowsPerWarp;
  int64_t slot[kRowsPerWarp];
  uint4 v[kRowsPerWarp][2];
  uint32_t rope[kRowsPerWarp];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    const int64_t row = row0 + i;
    slot[i] = row < num_rows ? slot_map[row] : -1;
    if (slot[i] != -1 && (slot[i] < 0 || slot[i] >= num_slots)) {
      if (lane == 0) report(dev_status, debug, MLA_CHECK_BAD_SLOT);
      slot[i] = -1;
    }
    if (slot[i] >= 0) {
      const __nv_bfloat16* src = rows + row * row_stride;
      v[i][0] = ld_stream16(src + 8 * lane);
      v[i][1] = ld_stream16(src + 256 + 8 * lane);
      rope[i] = __ldg(reinterpret_cast<const uint32_t*>(src + kDLatent) + lane);
    }
  }
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    if (slot[i] < 0) continue;  // (the same for the whole warp)
    uint8_t* dst = pool + slot[i] * kKv4Row;
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

// Lane l reads out block l (dims [16l, 16l + 16)) and the RoPE dims 2l, 2l + 1 of its warp's row.
__global__ void __launch_bounds__(kPoolThreads) kv4_gather_kernel(const uint8_t* __restrict__ pool,
                                                                  int64_t num_slots,
                                                                  const int32_t* __restrict__ slots,
                                                                  int64_t num_rows, __nv_bfloat16* __restrict__ out,
                                                                  int32_t debug, int32_t* dev_status) {
  const int lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5) * kRowsPerWarp;
  uint2 code[kRowsPerWarp];
  uint32_t scale[kRowsPerWarp], rope[kRowsPerWarp];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    const int64_t row = row0 + i;
    int64_t slot = row < num_rows ? slots[row] : -1;
    if (slot != -1 && (slot < 0 || slot >= num_slots)) {
      if (lane == 0) report(dev_status, debug, MLA_CHECK_BAD_SLOT);
      slot = -1;
    }
    code[i] = make_uint2(0u, 0u);
    scale[i] = rope[i] = 0u;
    if (slot >= 0) {
      const uint8_t* src = pool + slot * kKv4Row;
      code[i] = __ldg(reinterpret_cast<const uint2*>(src) + lane);
      scale[i] = __ldg(src + kKv4Codes + lane);
      rope[i] = __ldg(reinterpret_cast<const uint32_t*>(src + kKv4Rope) + lane);
    }
  }
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    const int64_t row = row0 + i;
    if (row >= num_rows) continue;
    const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(scale[i]) & 0xffffu)));
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t h = e2m1x2_to_f16x2((j < 4 ? code[i].x >> (8 * j) : code[i].y >> (8 * (j - 4))) & 0xffu);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);  // exact
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    uint4* dst = reinterpret_cast<uint4*>(out + row * kDK) + 2 * lane;
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    reinterpret_cast<uint32_t*>(out + row * kDK + kDLatent)[lane] = rope[i];
  }
}

int check_rows(const void* pool, int64_t num_slots, const int32_t* slots, int64_t num_rows, int32_t debug,
               const int32_t* dev_status) {
  if (num_slots < 1 || num_slots > 0x7fffffff || num_rows < 0) return MLA_ERR_INVALID_ARGUMENT;
  if ((num_rows + kRowsPerBlock - 1) / kRowsPerBlock > 0x7fffffff) return MLA_ERR_INVALID_ARGUMENT;
  if (num_rows > 0 && (!pool || !slots)) return MLA_ERR_INVALID_ARGUMENT;
  if (!aligned(pool, 32) || !aligned(slots, 4)) return MLA_ERR_INVALID_ARGUMENT;
  if (debug && !dev_status) return MLA_ERR_INVALID_ARGUMENT;
  return MLA_OK;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_kv4_append(void* pool, int64_t num_slots, const void* rows, int64_t row_stride,
                              const int32_t* slot_map, int64_t num_rows, int32_t debug, int32_t* dev_status,
                              mla_stream_t stream) {
  int rc = check_rows(pool, num_slots, slot_map, num_rows, debug, dev_status);
  if (rc) return rc;
  if ((num_rows > 0 && !rows) || !aligned(rows, 16) || row_stride < kDK || row_stride % 8 != 0)
    return MLA_ERR_INVALID_ARGUMENT;
  if (num_rows == 0) return MLA_OK;
  const unsigned blocks = (unsigned)((num_rows + kRowsPerBlock - 1) / kRowsPerBlock);
  kv4_append_kernel<<<blocks, kPoolThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<uint8_t*>(pool), num_slots, static_cast<const __nv_bfloat16*>(rows), row_stride, slot_map, num_rows,
      debug, dev_status);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

extern "C" int mla_kv4_gather(const void* pool, int64_t num_slots, const int32_t* slots, int64_t num_rows, void* out,
                              int32_t debug, int32_t* dev_status, mla_stream_t stream) {
  int rc = check_rows(pool, num_slots, slots, num_rows, debug, dev_status);
  if (rc) return rc;
  if ((num_rows > 0 && !out) || !aligned(out, 16)) return MLA_ERR_INVALID_ARGUMENT;
  if (num_rows == 0) return MLA_OK;
  const unsigned blocks = (unsigned)((num_rows + kRowsPerBlock - 1) / kRowsPerBlock);
  kv4_gather_kernel<<<blocks, kPoolThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(pool), num_slots, slots, num_rows, static_cast<__nv_bfloat16*>(out), debug,
      dev_status);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
