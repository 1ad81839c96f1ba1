// Tree-verify attention over the 4-bit latent pool for calls of at most 16 query rows a sequence, for sm_103a.
//
// verify_kv4_tc.cu works on 128 query rows and takes as long for one; what it pays for is codes turned into fp16 operands
// in shared memory. With so few rows the operands go from the codes straight into the registers of m16n8k16
// MMAs, and a CTA is small enough for three on an SM, which hide one another's latency.
//   grid (sequence, split); 4 warps; warp w owns the dims [128w, 128w + 128) and the RoPE dims [16w, 16w + 16).
// Per tile of 32 positions each warp copies its part of the rows to its own shared memory (cp.async, three stages), sums
// its dims' share of S = Q K^T, and exchanges it for the others'; every warp then does the same softmax and its dims of
// O += P V, with P taken from the S registers (one block barrier a tile).
//   K operand: thread (g, t) = (lane / 4, lane % 4) reads 16 bytes, the dims [32t, 32t + 32), of key g: four of them a step of
//   16 dims, in Q's order too.  V operand: 8 bytes, the dims [16g, 16g + 16), of the keys 2t, 2t + 1, 2t + 8, 2t + 9; column
//   g of MMA j is dim 16g + j, so a thread ends with 32 dims in a row of its two rows.
// Codes lie as 128-byte lines of two keys, 16-byte chunk c at c ^ 2 (line % 4): conflict-free for both reads.
// What bounds it: the chain of a tile (copies, S, exchange, softmax, PV: about 2700 cycles for a CTA alone, 5000 with three on
// an SM, 1870 a tile of the SM) and the issue slots (48% of the active cycles, 32 sequences of 8192 positions); tensor pipe
// 29%, DRAM 26%. MMAs of one key after another instead of interleaved took 5 to 8% longer, two CTAs on an SM without spills
// 25% (here: 8 bytes spilled).
//   16 rows: 32 sequences of 8192 positions 64 us, 1024 of 300 123 us, 4096 of 300 433 us (8 rows: 335), merge included
// Rounding as in verify_kv4_tc.cu: Q's rows and the keys scaled by powers of two (kv4.cuh), P = 2^(s - m + 7) in fp16, l from
// unrounded weights.
#include <atomic>

#include "kv4.cuh"
#include "tc.cuh"

namespace mla {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 32, kStages = 3;
constexpr int kCodes = kKeys * 64, kScales = kKeys * 8, kRope = kKeys * 32;
constexpr int kWarpStage = kCodes + kScales + kRope;
constexpr int kXch = kWarps * (kKeys / 8) * 512;  // partial scores of one tile
constexpr int kSmemBytes = kWarps * kStages * kWarpStage + 2 * kXch;
constexpr float kBias = 7.f;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Eight values (a word of codes) times a scale.
__device__ __forceinline__ void dequant8(uint32_t w, uint32_t scale2, uint32_t (&h)[4]) {
  asm("{\n.reg .b8 b0, b1, b2, b3;\nmov.b32 {b0, b1, b2, b3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\ncvt.rn.f16x2.e2m1x2 %1, b1;\n"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\ncvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int k = 0; k < 4; ++k) h[k] = mul2(h[k], scale2);
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__global__ void __launch_bounds__(kWarps * 32, 3) verify_kv4_rows_kernel(const VerifyArgs a) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ uint32_t s_top[kWarps][16];
  __shared__ uint64_t s_anc[16];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int b = blockIdx.x, s = blockIdx.y, R = a.T * a.H;
  const int32_t L = load_len(a, b), Tb = load_tree_size(a, b);
  const int64_t N = (int64_t)L + Tb, t0 = (int64_t)s * a.chunk, t1 = min(N, t0 + a.chunk);
  const int64_t out_row = (int64_t)s * a.rows + (int64_t)b * R;
  if (t0 >= t1) {
    if (threadIdx.x < R) a.part_lse[out_row + threadIdx.x] = -INFINITY;
    return;
  }
  const int rows_here = Tb * a.H, ntiles = (int)((t1 - t0 + kKeys - 1) / kKeys);

  // ---- loads of the pool's rows: lane l holds the slot of the tile's key l
  const int32_t* table = a.slot_table + (int64_t)b * a.stride;
  const uint8_t* pool = reinterpret_cast<const uint8_t*>(a.kv);
  uint8_t* mine = sm + warp * kStages * kWarpStage;
  auto slot_of = [&](int tile) -> int32_t {
    const int64_t at = t0 + (int64_t)tile * kKeys + lane;
    return at < t1 ? table[at] : 0;
  };
  auto load = [&](int tile, int32_t slot) {
    if (slot < 0 || slot >= a.num_slots) {
      report(a.dev_status, a.debug, MLA_CHECK_BAD_SLOT);
      slot = slot < 0 ? 0 : (int32_t)(a.num_slots - 1);
    }
    const uint32_t to = smem_u32(mine + (tile % kStages) * kWarpStage);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = 8 * i + g;
      const uint8_t* row = pool + (int64_t)__shfl_sync(0xffffffffu, slot, key) * kKv4Row;
      cp_async16(to + (key >> 1) * 128 + ((((key & 1) * 4 + t) ^ (((key >> 1) & 3) << 1)) << 4), row + 64 * warp + 16 * t);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = 16 * i + (lane >> 1);
      const uint8_t* row = pool + (int64_t)__shfl_sync(0xffffffffu, slot, key) * kKv4Row;
      cp_async16(to + kCodes + kScales + key * 32 + (lane & 1) * 16, row + kKv4Rope + 32 * warp + 16 * (lane & 1));
    }
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to + kCodes + lane * 8),
                 "l"(pool + (int64_t)slot * kKv4Row + kKv4Codes + 8 * warp)
                 : "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (i < ntiles) load(i, slot_of(i));
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  int32_t slot_next = kStages - 1 < ntiles ? slot_of(kStages - 1) : 0;

  // ---- Q: rows g and g + 8, in the order of K's operand
  uint32_t q[9][4];
  float unscale[2];
  uint64_t anc[2];
  {
    uint32_t top[2] = {0u, 0u};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = g + 8 * h;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + ((int64_t)b * R + (row < rows_here ? row : 0)) * kDK);
#pragma unroll
      for (int k = 0; k < 16; ++k) q[k >> 1][h + 2 * (k & 1)] = row < rows_here ? __ldg(src + 64 * warp + 16 * t + k) : 0u;
#pragma unroll
      for (int k = 0; k < 2; ++k) q[8][h + 2 * k] = row < rows_here ? __ldg(src + kDLatent / 2 + 8 * warp + 2 * t + k) : 0u;
#pragma unroll
      for (int k = 0; k < 9; ++k) {
        const uint32_t x = __vmaxu2(q[k][h] & 0x7fff7fffu, q[k][h + 2] & 0x7fff7fffu);
        top[h] = max(top[h], max(x & 0xffffu, x >> 16));
      }
      top[h] = max(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
      top[h] = max(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
      if (t == 0) s_top[warp][row] = top[h];
    }
    if (threadIdx.x < 16) s_anc[threadIdx.x] = threadIdx.x < rows_here ? ancestor_mask(a, b, threadIdx.x / a.H) : 0ull;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = g + 8 * h;
      anc[h] = s_anc[row];
      uint32_t x = 0u;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) x = max(x, s_top[w][row]);
      const int k2 = query_shift(x);
      const float up = exp2i(k2);
      unscale[h] = score_scale(k2, a.scale_log2);
#pragma unroll
      for (int k = 0; k < 9; ++k)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float f = k < 8 ? up : up * exp2i(-kKeyShift);
          const float lo = __uint_as_float(q[k][h + i] << 16) * f, hi = __uint_as_float(q[k][h + i] & 0xffff0000u) * f;
          if (k < 8) {
            q[k][h + i] = pack_half2(lo, hi);
          } else {
            const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
            q[k][h + i] = *reinterpret_cast<const uint32_t*>(&v);
          }
        }
    }
  }

  float o[16][4];
#pragma unroll
  for (int j = 0; j < 16; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[j][k] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float4* xch = reinterpret_cast<float4*>(sm + kWarps * kStages * kWarpStage);

#pragma unroll 1
  for (int tile = 0; tile < ntiles; ++tile) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();
    const uint8_t* st = mine + (tile % kStages) * kWarpStage;
    float4* x = xch + (tile & 1) * (kXch / 16);
    // ---- this warp's share of S
    uint4 w[kKeys / 8];
    uint32_t sc[kKeys / 8];
    float c[kKeys / 8][4];
#pragma unroll
    for (int j = 0; j < kKeys / 8; ++j) {
      const int key = 8 * j + g;
      w[j] = *reinterpret_cast<const uint4*>(st + (key >> 1) * 128 + ((((key & 1) * 4 + t) ^ (((key >> 1) & 3) << 1)) << 4));
      sc[j] = key_scales(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(st + kCodes + key * 8 + 2 * t)));
      const uint2 r = *reinterpret_cast<const uint2*>(st + kCodes + kScales + key * 32 + 8 * t);
#pragma unroll
      for (int k = 0; k < 4; ++k) c[j][k] = 0.f;
      mma_bf16(c[j], q[8], r.x, r.y);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)  // (the MMAs of different keys do not wait on one another)
#pragma unroll
      for (int j = 0; j < kKeys / 8; ++j) {
        uint32_t h[4];
        dequant8(k == 0 ? w[j].x : k == 1 ? w[j].y : k == 2 ? w[j].z : w[j].w, __byte_perm(sc[j], 0, k < 2 ? 0x1010 : 0x3232), h);
        mma_f16(c[j], q[2 * k], h[0], h[1]);
        mma_f16(c[j], q[2 * k + 1], h[2], h[3]);
      }
#pragma unroll
    for (int j = 0; j < kKeys / 8; ++j)
      x[(warp * (kKeys / 8) + j) * 32 + lane] = make_float4(c[j][0], c[j][1], c[j][2], c[j][3]);
    __syncthreads();  // (the next write to these places comes after the next barrier)
    if (tile + kStages - 1 < ntiles) load(tile + kStages - 1, slot_next);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (tile + kStages < ntiles) slot_next = slot_of(tile + kStages);

    // ---- softmax, the same in every warp
    float p[kKeys / 8][4], mt[2] = {-INFINITY, -INFINITY};
    const int ahead = (int)(L - t0) - tile * kKeys;  // prefix positions from the tile's first one on
#pragma unroll
    for (int j = 0; j < kKeys / 8; ++j) {
      const float4 c0 = x[j * 32 + lane], c1 = x[(kKeys / 8 + j) * 32 + lane], c2 = x[(2 * (kKeys / 8) + j) * 32 + lane],
                   c3 = x[(3 * (kKeys / 8) + j) * 32 + lane];
      p[j][0] = ((c0.x + c1.x) + (c2.x + c3.x)) * unscale[0];
      p[j][1] = ((c0.y + c1.y) + (c2.y + c3.y)) * unscale[0];
      p[j][2] = ((c0.z + c1.z) + (c2.z + c3.z)) * unscale[1];
      p[j][3] = ((c0.w + c1.w) + (c2.w + c3.w)) * unscale[1];
      if (ahead < kKeys) {  // some positions past the prefix: the tree's bitmask
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int node = 8 * j + 2 * t + (k & 1) - ahead;
          if (node >= 0 && (node >= 64 || !((anc[k >> 1] >> node) & 1ull))) p[j][k] = -INFINITY;
        }
      }
      mt[0] = fmaxf(mt[0], fmaxf(p[j][0], p[j][1]));
      mt[1] = fmaxf(mt[1], fmaxf(p[j][2], p[j][3]));
    }
    float alpha[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mt[h] = fmaxf(mt[h], __shfl_xor_sync(0xffffffffu, mt[h], 1));
      mt[h] = fmaxf(mt[h], __shfl_xor_sync(0xffffffffu, mt[h], 2));
      const float m_new = fmaxf(m[h], mt[h]);
      alpha[h] = m_new == m[h] ? 1.f : ex2(m[h] - m_new);  // 0 on the first visible position
      m[h] = m_new;
      const float base = m_new == -INFINITY ? 0.f : m_new - kBias;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          p[j][2 * h + k] = ex2(p[j][2 * h + k] - base);
          sum += p[j][2 * h + k];
        }
      l[h] = l[h] * alpha[h] + sum;
    }
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        o[j][0] *= alpha[0];
        o[j][1] *= alpha[0];
        o[j][2] *= alpha[1];
        o[j][3] *= alpha[1];
      }
    }

    // ---- this warp's dims of O
#pragma unroll
    for (int i = 0; i < kKeys / 16; ++i) {
      const uint32_t pa[4] = {pack_half2(p[2 * i][0], p[2 * i][1]), pack_half2(p[2 * i][2], p[2 * i][3]),
                              pack_half2(p[2 * i + 1][0], p[2 * i + 1][1]), pack_half2(p[2 * i + 1][2], p[2 * i + 1][3])};
      uint2 w[4];
      uint32_t sc[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = 16 * i + 2 * t + (k & 1) + 8 * (k >> 1);
        w[k] = *reinterpret_cast<const uint2*>(st + (key >> 1) * 128 +
                                               ((((key & 1) * 4 + (g >> 1)) ^ (((key >> 1) & 3) << 1)) << 4) + (g & 1) * 8);
        uint32_t e = st[kCodes + key * 8 + g];
        if ((e & 0x7fu) == 0x7fu) e = 0u;  // NaN: the key's score is NaN already, and rows that do not see it stay clean
        sc[k] = __byte_perm(e4m3x2_to_f16x2(e), 0, 0x1010);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t h[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) dequant8(half ? w[k].y : w[k].x, sc[k], h[k]);
#pragma unroll
        for (int d = 0; d < 4; ++d) {  // dims 8 half + 2d and + 1
          mma_f16(o[8 * half + 2 * d], pa, __byte_perm(h[0][d], h[1][d], 0x5410), __byte_perm(h[2][d], h[3][d], 0x5410));
          mma_f16(o[8 * half + 2 * d + 1], pa, __byte_perm(h[0][d], h[1][d], 0x7632), __byte_perm(h[2][d], h[3][d], 0x7632));
        }
      }
    }
    __syncwarp();  // (this stage is loaded over in the next step)
  }

#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = g + 8 * h;
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if (row >= R) continue;
    const bool valid = row < rows_here && l[h] != 0.f;
    if (warp == 0 && t == 0) a.part_lse[out_row + row] = valid ? (m[h] + (log2f(l[h]) - kBias)) * 0.6931471805599453f : -INFINITY;
    if (!valid) continue;
    const float inv = 1.f / l[h];
    uint4* dst = reinterpret_cast<uint4*>(a.part_o + (out_row + row) * kDLatent + 128 * warp + 32 * t);
#pragma unroll
    for (int v = 0; v < 4; ++v) {  // dims 16 (v / 2) + 8 (v % 2) .. + 7 of the thread's 32
      uint32_t y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        y[k] = pack_half2(o[8 * (v & 1) + 2 * k][2 * h + (v >> 1)] * inv, o[8 * (v & 1) + 2 * k + 1][2 * h + (v >> 1)] * inv);
      dst[v] = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
}

}  // namespace

cudaError_t launch_verify_kv4_rows(const VerifyArgs& a, cudaStream_t stream) {
  static std::atomic<bool> configured[64];  // the smem opt-in, set once per device (setting it twice is harmless)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(verify_kv4_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.B, (unsigned)a.splits);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // programmatic dependent launch: inputs are read after griddepcontrol.wait
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kv4_rows_kernel, a);
}

}  // namespace mla
