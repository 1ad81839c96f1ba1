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
