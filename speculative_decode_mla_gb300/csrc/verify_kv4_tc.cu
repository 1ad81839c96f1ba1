// tcgen05 split-KV tree-verify kernel over the 4-bit latent pool, for sm_103a.
//
// One work unit = (sequence b, 128-row tile of its T*H query rows, KV chunk s), on a cluster of two
// CTAs whose tensor cores work as a pair (cta_group::2, M = 128: CTA r holds query rows
// [64r, 64r + 64) of the tile, all 128 TMEM lanes in use). A 64-row share of the fp32 output over 512
// value dims is 256 TMEM columns, so a pair holds whole rows and no partial scores travel between the
// CTAs. Per 128-position tile:
//
//   S = Q K^T   N = 128: CTA r supplies the keys of positions [64r, 64r + 64), all 576 dims
//   O += P V    N = 256, twice: CTA r supplies value dims [128r, 128r + 128) of each half, all positions
//
// so CTA r dequantises its own 64 rows whole and of the partner's 64 rows the 256 value dims
// that it supplies. Codes x scales are exact in fp16, so K, V and Q are fp16 operands; the RoPE dims
// stay bf16 (kind::f16 takes either, and both accumulate into the same fp32 scores). A query row is
// scaled by a power of two so that its largest magnitude lies in [2^14, 2^15): its bf16 values are then exact
// in fp16 down to 2^-29 of the largest, and the scale is taken out of the scores.
//
//   warps 0-7    gather and dequantise: four threads a key. Codes go from global memory through registers
//                (loads of a tile are out before the one before it is used), cvt e2m1x2 -> f16x2, times the block's
//                scale, to 128B-swizzled shared memory: K into a ring of 16 KB sub-stages (128 dims of 64
//                keys), then, one tile later, V. A value's codes are read once for both.
//   warps 8-11   softmax, two threads a row (64 keys each): S from TMEM, ancestor bitmask on tree positions, row
//                maximum over the two threads through shared memory, exp2, P (fp16) to shared memory; O is
//                rescaled only when the running maximum grows by more than 2^8. Epilogue: O / l to the workspace.
//   warp 12, 13  one thread each: CTA 0 issues S and PV for the pair; CTA 1 tells CTA 0 what is ready
//                (local barriers, then one remote arrive each: a cluster-scope release is slow, so the
//                working warps stay off it).
//
// P is kept as 2^(s - m + 7): under the lazy maximum it is at most 2^15, and weights down to 2^-32 of a
// row's largest still count in fp16. l is the fp32 sum of the unrounded weights.
//
// TMEM (512 columns): O [0, 256), S [256, 320), Q's dims 0..383 [320, 512) (both lane halves hold the
// CTA's 64 rows); Q's dims 384..511 and RoPE dims are in shared memory.
//
// Positions past a chunk's end read slot 0's row and are masked; values whose scale is NaN are 0
// in V (their K is NaN, so every row that sees the key is NaN through its weight, and no other).
// Every wait is bounded (about 2 s); on timeout the kernel stops issuing work, drains what it
// started, reports MLA_CHECK_TIMEOUT in dev_status when given, writes NaN lse for its rows and exits.
#include <atomic>

#include "kv4.cuh"
#include "tc.cuh"

namespace mla {
namespace {

constexpr int kRows = 128;     // query rows of a pair (MMA M)
constexpr int kCtaRows = 64;   // of them on each CTA
constexpr int kKeys = kKv4TileTokens;  // 128 positions per tile (S MMA N)
constexpr int kOwn = 64;       // of them supplied by each CTA
constexpr int kBlock = kOwn * 128;       // 64 keys (or rows) x 64 dims, 128B swizzle
constexpr int kKSlots = 6;               // K ring: sub-stages of 128 dims (two blocks) of the own 64 keys
constexpr int kKSlotBytes = 2 * kBlock;
constexpr int kVBlock = kKeys * 128;     // 128 keys x 64 dims
constexpr int kVHalfBytes = 2 * kVBlock; // 128 value dims
constexpr int kSmemK = 0;
constexpr int kSmemR = kSmemK + kKSlots * kKSlotBytes;  // RoPE dims of the own keys, two tiles
constexpr int kSmemV = kSmemR + 2 * kBlock;
constexpr int kSmemP = kSmemV + 2 * kVHalfBytes;        // two blocks of 64 rows x 64 keys
constexpr int kSmemQ = kSmemP + 2 * kBlock;             // dims 384..447, 448..511, RoPE
constexpr int kSmemX = kSmemQ + 3 * kBlock;             // exchange between the two threads of a row: [2][128] floats
constexpr int kSmemBar = kSmemX + 1024;
constexpr int kSmemBytes = kSmemBar + 512 + 1024;       // barriers, TMEM slot, tree parents + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory");
// Q's rows pass through V and P on their way in (64 rows x 1152 bytes)
static_assert(2 * kVHalfBytes + 2 * kBlock >= kCtaRows * kDK * 2, "Q staging");

constexpr int kDequantWarps = 8;
constexpr int kSWarp = 12, kPVWarp = 13;  // 8..11: softmax, TMEM lane quarters 0..3; 14 and 15 only fill the warpgroup
constexpr int kThreads = 16 * 32;
// Registers a thread: 128 at launch (4 warpgroups x 128 x 128 = 65,536); the issuers' warpgroup hands 72 of its
// own to the softmax warpgroup (128 + 128 + 200 + 56 = 4 x 128).
constexpr int kSoftmaxRegs = 200, kIssuerRegs = 56;
constexpr int kParentThread0 = kSWarp * 32;  // 64 threads read the tree parents

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 320;
constexpr int kQTmemDims = 384;
constexpr float kPBias = 7.f;

constexpr int kBarKFull = 0, kBarKEmpty = kKSlots, kBarVFull = 2 * kKSlots /*2*/, kBarVEmpty = kBarVFull + 2 /*2*/,
              kBarSFull = kBarVEmpty + 2, kBarSEmpty = kBarSFull + 1, kBarPFull = kBarSFull + 2,
              kBarPEmpty = kBarSFull + 3, kBarQFull = kBarSFull + 4, kBarDrainS = kBarSFull + 5,
              kBarDrainP = kBarSFull + 6, kNumBars = kBarSFull + 7;
static_assert(8 * kNumBars + 8 + 4 * kMaxNodes <= 512, "barrier area");

// Instruction descriptor for kind::f16 with fp32 D: A and B both fp16 or both bf16.
__host__ __device__ constexpr uint32_t instr_desc(int N, bool bf16, bool b_mn_major) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(kRows >> 4) << 24);
}
__device__ __forceinline__ void mma2_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma2_smem_a(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the MMAs issued so far have completed.
__device__ __forceinline__ void commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void commit_own(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)1)
      : "memory");
}
__device__ __forceinline__ uint4 ld16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld2(const uint8_t* p) {
  uint16_t v;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}
// Two threads a row: warps w and w + 2 of the softmax warps.
__device__ __forceinline__ void row_pair_sync(int softmax_warp) {
  if (softmax_warp & 1) asm volatile("bar.sync 2, 64;" ::: "memory");
  else asm volatile("bar.sync 1, 64;" ::: "memory");
}

// 32 values (a 16-byte piece of a row's codes, its two scales as fp16) into four 16-byte chunks, c0 .. c0 + 3
// of the 128-byte row at `row_addr` (128B swizzle: chunk c lies at c ^ (row & 7)).
__device__ __forceinline__ void dequant_piece(uint4 code, uint32_t scales, uint32_t row_addr, uint32_t c0, uint32_t r7) {
  const uint32_t s0 = __byte_perm(scales, 0, 0x1010), s1 = __byte_perm(scales, 0, 0x3232);
  const uint32_t w[4] = {code.x, code.y, code.z, code.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t h[4];
    asm("{\n.reg .b8 b0, b1, b2, b3;\nmov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\ncvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\ncvt.rn.f16x2.e2m1x2 %3, b3;\n}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w[j]));
    const uint32_t s = j < 2 ? s0 : s1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h[k]), *reinterpret_cast<const __half2*>(&s));
      h[k] = *reinterpret_cast<const uint32_t*>(&v);
    }
    st_shared_v4(row_addr + (((c0 + (uint32_t)j) ^ r7) << 4), h);
  }
}
// Scales that are NaN become 0 (for V; see the top).
__device__ __forceinline__ uint32_t without_nan(uint32_t scales) {
  return scales & ~__vcmpgtu2(scales & 0x7fff7fffu, 0x7c007c00u);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) verify_kv4_tc_kernel(const VerifyArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_addr);
  const uint32_t bar0 = base + kSmemBar;
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSmemBar + 8 * kNumBars);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  int32_t* s_parent = reinterpret_cast<int32_t*>(smem + kSmemBar + 8 * kNumBars + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));

  const int unit = blockIdx.x >> 1;
  int s, tile_idx, b;
  if (a.lpt) {
    tile_idx = unit % a.row_tiles;
    s = b = 0;
  } else {
    s = unit % a.splits;
    const int bt = unit / a.splits;
    tile_idx = bt % a.row_tiles;
    b = bt / a.row_tiles;
  }
  const int R = a.T * a.H;
  const int row0 = tile_idx * kRows + (int)rank * kCtaRows;  // this CTA's first row of the sequence
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (a.lpt) lpt_unit(a, unit / a.row_tiles, lane, b, s);
  const int64_t t0 = (int64_t)s * a.chunk;
  const int32_t L = load_len(a, b);
  const int32_t Tb = load_tree_size(a, b);
  const int64_t N = (int64_t)L + Tb;
  const int64_t t1 = min(N, t0 + a.chunk);
  if (t0 >= t1) {  // nothing of this sequence falls in this chunk: an empty partial (both CTAs agree)
    if (threadIdx.x < kCtaRows && row0 + (int)threadIdx.x < R)
      a.part_lse[(int64_t)s * a.rows + (int64_t)b * R + row0 + threadIdx.x] = -INFINITY;
    return;
  }
  const int ntiles = (int)((t1 - t0 + kKeys - 1) / kKeys);

  if (threadIdx.x == 0) {
    const uint32_t relay = rank == 0 ? 1u : 0u;  // CTA 0 also waits for the word of CTA 1
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(bar(kBarKFull + i), kDequantWarps + relay);
      mbar_init(bar(kBarKEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarVFull + i), kDequantWarps + relay);
      mbar_init(bar(kBarVEmpty + i), 1);
    }
    mbar_init(bar(kBarSFull), 1);
    mbar_init(bar(kBarSEmpty), 4 + relay);
    mbar_init(bar(kBarPFull), 4 + relay);
    mbar_init(bar(kBarPEmpty), 1);
    mbar_init(bar(kBarQFull), 4 + relay);
    mbar_init(bar(kBarDrainS), 1);
    mbar_init(bar(kBarDrainP), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const int pidx = (int)threadIdx.x - kParentThread0;
  if (pidx >= 0 && pidx < a.T) {  // tree parents of this sequence, validated
    int p = a.tree_parent[(int64_t)b * a.T + pidx];
    if (pidx >= Tb) {
      p = -1;
    } else if (p < -1 || p >= pidx) {
      report(a.dev_status, a.debug, MLA_CHECK_BAD_PARENT);
      p = -1;
    }
    s_parent[pidx] = p;
  }
  if (warp == kSWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }

  // ------------------------------------------------------------------ what the gather needs first
  // Thread (key, qd): lane = 8 qd + key % 8, warp = key / 8; pieces 4i + qd (32 dims each) of a row, i < 4.
  const int key = warp * 8 + (lane & 7), qd = lane >> 3;
  const uint8_t* pool = reinterpret_cast<const uint8_t*>(a.kv);
  const int32_t* tab = a.slot_table + (int64_t)b * a.stride;
  auto row_at = [&](int t, uint32_t of_rank) -> const uint8_t* {  // the row of position `key` of a CTA's share of tile t
    const int64_t pos = t0 + (int64_t)t * kKeys + (int)of_rank * kOwn + key;
    int64_t slot = 0;
    if (pos < t1) {
      slot = tab[pos];
      if (slot < 0 || slot >= a.num_slots) {
        report(a.dev_status, a.debug, MLA_CHECK_BAD_SLOT);
        slot = slot < 0 ? 0 : a.num_slots - 1;
      }
    }
    return pool + slot * kKv4Row;
  };
  uint4 kc[4], kr[2], pc[2];
  uint32_t ks[4], ps[2];
  auto load_own = [&](const uint8_t* row) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      kc[i] = ld16(row + 16 * (4 * i + qd));
      ks[i] = ld2(row + kKv4Codes + 2 * (4 * i + qd));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) kr[i] = ld16(row + kKv4Rope + 32 * qd + 16 * i);
  };
  auto load_peer = [&](const uint8_t* row) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int piece = 4 * ((int)rank + 2 * j) + qd;
      pc[j] = ld16(row + 16 * piece);
      ps[j] = ld2(row + kKv4Codes + 2 * piece);
    }
  };
  const uint8_t *own_next = pool, *peer_next = pool;
  if (warp < kDequantWarps) {
    const uint8_t* own = row_at(0, rank);
    const uint8_t* peer = row_at(0, rank ^ 1u);
    load_own(own);
    load_peer(peer);
    own_next = row_at(1, rank);
    peer_next = row_at(1, rank ^ 1u);
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barrier inits visible to the partner before any remote operation
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < kDequantWarps) {
    // ---------------------------------------------------------------- gather and dequantise
    const uint32_t r7 = (uint32_t)key & 7u, c0 = (uint32_t)(qd & 1) * 4u;
    const uint32_t blk = (uint32_t)(qd >> 1);
    uint4 vc[2] = {}, vc_next[2];
    uint32_t vs[2] = {}, vs_next[2];
    bool ok = true;
    for (int it = 0; it <= ntiles && ok; ++it) {
      if (it < ntiles) {
        // K(it): four sub-stages of 128 dims; the RoPE dims go with the last one. (Its buffer, it & 1, is
        // free: the slot of this sub-stage was last read by S(it - 1), after S(it - 2).)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int sub = 4 * it + i, slot = sub % kKSlots;
          if (sub >= kKSlots && !wait_warp(bar(kBarKEmpty + slot), (sub / kKSlots - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          dequant_piece(kc[i], e4m3x2_to_f16x2(ks[i]), base + kSmemK + slot * kKSlotBytes + blk * kBlock + key * 128, c0, r7);
          if (i == 3) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t w[4] = {kr[k].x, kr[k].y, kr[k].z, kr[k].w};
              st_shared_v4(base + kSmemR + (it & 1) * kBlock + key * 128 + (((uint32_t)(2 * qd + k) ^ r7) << 4), w);
            }
          }
          fence_proxy_async();  // generic-proxy stores, read by the MMA (async proxy)
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarKFull + slot));
        }
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // the pieces of the value dims that this CTA supplies
          vc_next[j] = rank ? kc[1 + 2 * j] : kc[2 * j];
          vs_next[j] = rank ? ks[1 + 2 * j] : ks[2 * j];
        }
        if (it + 1 < ntiles) {
          load_own(own_next);
          own_next = row_at(it + 2, rank);
        }
      }
      if (it > 0) {
        // V(it - 1), once PV(it - 2) has read the buffer (for the first tile: once Q has passed through it)
        const int t = it - 1;
        if (t == 0 && !wait_warp(bar(kBarQFull), 0, abort_flag, rank == 0)) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (t > 0 && !wait_warp(bar(kBarVEmpty + j), (t - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t vb = base + kSmemV + j * kVHalfBytes + blk * kVBlock;
          dequant_piece(vc[j], without_nan(e4m3x2_to_f16x2(vs[j])), vb + (rank * kOwn + key) * 128, c0, r7);
          dequant_piece(pc[j], without_nan(e4m3x2_to_f16x2(ps[j])), vb + ((rank ^ 1u) * kOwn + key) * 128, c0, r7);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarVFull + j));
        }
        if (!ok) break;
        if (it < ntiles) {
          load_peer(peer_next);
          peer_next = row_at(it + 1, rank ^ 1u);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        vc[j] = vc_next[j];
        vs[j] = vs_next[j];
      }
    }
  } else if (warp >= kSWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssuerRegs));
    if (warp == kSWarp && lane == 0) {
      if (rank == 0) {
        // -------------------------------------------------------------- S issuer
        constexpr uint32_t idesc_h = instr_desc(kKeys, false, false), idesc_b = instr_desc(kKeys, true, false);
        bool ok = wait_bar(bar(kBarQFull), 0, abort_flag, true);
        for (int t = 0; t < ntiles && ok; ++t) {
          if (t > 0) ok = wait_bar(bar(kBarSEmpty), (t - 1) & 1, abort_flag, true);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int sub = 4 * t + i, slot = sub % kKSlots;
            if (ok) ok = wait_bar(bar(kBarKFull + slot), (sub / kKSlots) & 1, abort_flag, true);
            if (!ok) break;
            tc_fence_after();
            const uint32_t kb = base + kSmemK + slot * kKSlotBytes;
#pragma unroll
            for (int k = 0; k < 8; ++k) {  // 16 dims each
              const uint64_t bd = smem_desc(kb + (k >> 2) * kBlock + (k & 3) * 32, 16, 1024);
              if (i < 3)
                mma2_tmem_a(tmem + kColS, tmem + kColQ + (i * 8 + k) * 8, bd, idesc_h, (i | k) ? 1u : 0u);
              else
                mma2_smem_a(tmem + kColS, smem_desc(base + kSmemQ + (k >> 2) * kBlock + (k & 3) * 32, 16, 1024), bd,
                            idesc_h, 1u);
            }
            if (i == 3) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma2_smem_a(tmem + kColS, smem_desc(base + kSmemQ + 2 * kBlock + k * 32, 16, 1024),
                            smem_desc(base + kSmemR + (t & 1) * kBlock + k * 32, 16, 1024), idesc_b, 1u);
            }
            commit_both(bar(kBarKEmpty + slot));
          }
          if (ok) commit_both(bar(kBarSFull));
        }
        // drain: every MMA this thread issued has completed once this barrier flips
        commit_own(bar(kBarDrainS));
        const long long st = clock64();
        while (!mbar_test(bar(kBarDrainS), 0) && clock64() - st < kTimeoutCycles) {
        }
      } else {
        // -------------------------------------------------------------- CTA 1: what S waits for, to CTA 0
        const uint32_t remote = map_to_cta(bar0, 0);
        bool ok = wait_bar(bar(kBarQFull), 0, abort_flag);
        if (ok) mbar_arrive_remote(remote + 8u * kBarQFull);
        for (int t = 0; t < ntiles && ok; ++t) {
          if (t > 0) {
            ok = wait_bar(bar(kBarSEmpty), (t - 1) & 1, abort_flag);
            if (ok) mbar_arrive_remote(remote + 8u * kBarSEmpty);
          }
          for (int i = 0; i < 4 && ok; ++i) {
            const int sub = 4 * t + i, slot = sub % kKSlots;
            ok = wait_bar(bar(kBarKFull + slot), (sub / kKSlots) & 1, abort_flag);
            if (ok) mbar_arrive_remote(remote + 8u * (uint32_t)(kBarKFull + slot));
          }
        }
      }
    }
    if (warp == kPVWarp && lane == 0) {
      if (rank == 0) {
        // -------------------------------------------------------------- PV issuer
        constexpr uint32_t idesc_pv = instr_desc(256, false, true);
        bool ok = true;
        for (int t = 0; t < ntiles && ok; ++t) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            ok = ok && wait_bar(bar(kBarVFull + j), t & 1, abort_flag, true);
            if (j == 0) ok = ok && wait_bar(bar(kBarPFull), t & 1, abort_flag, true);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 8; ++k)  // 16 positions each; V is read MN-major
              mma2_smem_a(tmem + kColO + j * 128, smem_desc(base + kSmemP + (k >> 2) * kBlock + (k & 3) * 32, 16, 1024),
                          smem_desc(base + kSmemV + j * kVHalfBytes + k * 2048, kVBlock, 1024), idesc_pv,
                          (t | k) ? 1u : 0u);
            commit_both(bar(kBarVEmpty + j));
          }
          if (ok) commit_both(bar(kBarPEmpty));
        }
        commit_own(bar(kBarDrainP));
        const long long st = clock64();
        while (!mbar_test(bar(kBarDrainP), 0) && clock64() - st < kTimeoutCycles) {
        }
      } else {
        const uint32_t remote = map_to_cta(bar0, 0);
        bool ok = true;
        for (int t = 0; t < ntiles && ok; ++t) {
          ok = wait_bar(bar(kBarVFull), t & 1, abort_flag);
          if (ok) mbar_arrive_remote(remote + 8u * kBarVFull);
          ok = ok && wait_bar(bar(kBarPFull), t & 1, abort_flag);
          if (ok) mbar_arrive_remote(remote + 8u * kBarPFull);
          ok = ok && wait_bar(bar(kBarVFull + 1), t & 1, abort_flag);
          if (ok) mbar_arrive_remote(remote + 8u * (kBarVFull + 1));
        }
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax, two threads a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int q4 = warp & 3;
    const int l128 = q4 * 32 + lane;         // TMEM lane
    const int r = l128 & 63, half = l128 >> 6;
    const uint32_t lane_addr = tmem + ((uint32_t)(q4 * 32) << 16);
    const int local_row = row0 + r;
    const bool valid = local_row < R && local_row / a.H < Tb;
    float* xch = reinterpret_cast<float*>(smem + kSmemX);
    const uint32_t r7 = (uint32_t)r & 7u;

    // Q: each of the two threads brings half of the row (288 dims) into the staging rows and finds its
    // largest magnitude; then the row, times 2^k, as fp16 into TMEM (both lanes of a row hold all of it)
    // and shared memory. Row r's 16-byte chunk c lies at c ^ (r & 7) in the staging rows.
    float unscale;
    {
      uint32_t top = 0;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(a.q + ((int64_t)b * R + (valid ? local_row : 0)) * kDK) + half * 576;
      const uint32_t stage = base + kSmemV + r * (kDK * 2);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint4 v[18];
#pragma unroll
        for (int i = 0; i < 18; ++i) v[i] = valid ? ld16(src + (18 * g + i) * 16) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 18; ++i) {
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) top = __vmaxu2(top, w[k] & 0x7fff7fffu);
          st_shared_v4(stage + (((uint32_t)(half * 36 + 18 * g + i) ^ r7) << 4), w);
        }
      }
      top = max(top & 0xffffu, top >> 16);
      reinterpret_cast<uint32_t*>(xch)[l128] = top;
      row_pair_sync(q4);
      top = max(top, reinterpret_cast<uint32_t*>(xch)[l128 ^ 64]);
      // top is in [2^(e - 127), 2^(e - 126)): k = 14 - (e - 127); rows of zeros, infinities or NaN stay as they are
      const int e = (int)(top >> 7);
      int k = (e == 0 || e == 255) ? 0 : 141 - e;
      k = min(110, k);  // (2^-k stays a normal fp32 number)
      const float up = __int_as_float((127 + k) << 23);
      unscale = __int_as_float((127 - k) << 23) * a.scale_log2;
      auto staged = [&](int c) {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(stage + (((uint32_t)c ^ r7) << 4)));
        return v;
      };
      auto f16_of = [&](uint32_t w) {
        const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
        return *reinterpret_cast<const uint32_t*>(&h);
      };
#pragma unroll 2
      for (int g = 0; g < kQTmemDims / 32; ++g) {  // 32 dims: 16 columns
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = staged(4 * g + i);
          w[4 * i] = f16_of(v.x);
          w[4 * i + 1] = f16_of(v.y);
          w[4 * i + 2] = f16_of(v.z);
          w[4 * i + 3] = f16_of(v.w);
        }
        TMEM_ST16(lane_addr + kColQ + g * 16, w);
      }
      // chunks 48..63 (dims 384..511) and 64..71 (RoPE): this thread takes every other one
#pragma unroll
      for (int i = 0; i < 12; ++i) {
        const int c = 2 * i + half;
        const uint4 v = staged(48 + c);
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k2 = 0; k2 < 4; ++k2) {
          if (i < 8) {
            w[k2] = f16_of(w[k2]);
          } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(w[k2] << 16) * up,
                                                           __uint_as_float(w[k2] & 0xffff0000u) * up);
            w[k2] = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
        st_shared_v4(base + kSmemQ + (c >> 3) * kBlock + r * 128 + (((uint32_t)(c & 7) ^ r7) << 4), w);
      }
      fence_proxy_async();
      tmem_wait_st();
      tc_fence_before();
      row_pair_sync(q4);  // the staging rows (and xch) have been read by both
      if (lane == 0) mbar_arrive(bar(kBarQFull));
    }

    uint64_t anc = 0;  // anc*(node): the tree positions this row can see
    if (valid)
      for (int j = local_row / a.H, step = 0; j >= 0 && step < kMaxNodes; j = s_parent[j], ++step) anc |= 1ull << j;

    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;  // (the row pairs' barriers are passed whether or not a wait has failed)
    for (int t = 0; t < ntiles; ++t) {
      float sc[64];
      float mt = -INFINITY;
      if (ok) ok = wait_warp(bar(kBarSFull), t & 1, abort_flag);
      if (ok) {
        tc_fence_after();
        uint32_t(&su)[64] = reinterpret_cast<uint32_t(&)[64]>(sc);
#pragma unroll
        for (int c = 0; c < 4; ++c) TMEM_LD16(lane_addr + kColS + c * 16, (su + c * 16));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarSEmpty));
        const int64_t p0 = t0 + (int64_t)t * kKeys + half * 64;  // this thread's first position
        if (p0 + 64 > L) {  // some of them past the prefix: the tree's bitmask
          uint64_t vis = 0;
          if (p0 < L) {
            const int n = (int)(L - p0);
            vis = ((1ull << n) - 1) | (anc << n);
          } else if (p0 - L < 64) {
            vis = anc >> (int)(p0 - L);
          }
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (!((vis >> k) & 1ull)) sc[k] = -INFINITY;
        }
        float m[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          m[u] = max3(sc[u], sc[8 + u], sc[16 + u]);
          m[u] = max3(m[u], sc[24 + u], sc[32 + u]);
          m[u] = max3(m[u], sc[40 + u], sc[48 + u]);
          m[u] = fmaxf(m[u], sc[56 + u]);
        }
        mt = max3(max3(m[0], m[1], m[2]), max3(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
      }
      xch[(t & 1) * 128 + l128] = mt;
      row_pair_sync(q4);
      if (!ok) continue;
      mt = fmaxf(mt, xch[(t & 1) * 128 + (l128 ^ 64)]) * unscale;
      bool rescale = false;
      float alpha = 1.f;
      if (mt > m_run + 8.f || m_run == -INFINITY) {
        alpha = m_run == -INFINITY ? 0.f : ex2(m_run - mt);
        rescale = t > 0 && m_run != mt;
        l_run *= alpha;
        m_run = mt;
      }
      const float neg_m = m_run == -INFINITY ? 0.f : kPBias - m_run;
      uint32_t pk[32];
      float2 ls0 = make_float2(0.f, 0.f), ls1 = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 64; k += 4) {
        const float2 x0 = fma2(make_float2(sc[k], sc[k + 1]), make_float2(unscale, unscale), make_float2(neg_m, neg_m));
        const float2 x1 = fma2(make_float2(sc[k + 2], sc[k + 3]), make_float2(unscale, unscale), make_float2(neg_m, neg_m));
        const float2 e0 = make_float2(ex2(x0.x), ex2(x0.y)), e1 = make_float2(ex2(x1.x), ex2(x1.y));
        const __half2 h0 = __floats2half2_rn(e0.x, e0.y), h1 = __floats2half2_rn(e1.x, e1.y);
        pk[k / 2] = *reinterpret_cast<const uint32_t*>(&h0);
        pk[k / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
        ls0 = add2(ls0, e0);
        ls1 = add2(ls1, e1);
      }
      l_run += (ls0.x + ls0.y) + (ls1.x + ls1.y);

      // P and O once PV of the previous tile has finished with them
      if (t > 0) {
        ok = wait_warp(bar(kBarPEmpty), (t - 1) & 1, abort_flag);
        if (!ok) continue;
        tc_fence_after();
      }
      if (__any_sync(0xffffffffu, rescale)) {  // (tcgen05.ld/st are warp-collective: other rows multiply by 1)
        const float f = rescale ? alpha : 1.f;
#pragma unroll 1
        for (int c = 0; c < 16; ++c) {
          uint32_t o[16];
          TMEM_LD16(lane_addr + kColO + c * 16, o);
          tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
          TMEM_ST16(lane_addr + kColO + c * 16, o);
        }
      }
#pragma unroll
      for (int c = 0; c < 8; ++c)
        st_shared_v4(base + kSmemP + half * kBlock + r * 128 + (((uint32_t)c ^ r7) << 4), pk + 4 * c);
      fence_proxy_async();
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarPFull));
    }

    // epilogue: O / l as fp16 partials, 256 dims a thread in runs of 128; lse
    xch[(ntiles & 1) * 128 + l128] = l_run;
    row_pair_sync(q4);
    const float l = l_run + xch[(ntiles & 1) * 128 + (l128 ^ 64)];
    if (ok) ok = wait_warp(bar(kBarPEmpty), (ntiles - 1) & 1, abort_flag);
    if (ok) {
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
      const int64_t grow = (int64_t)b * R + local_row;
      __half* po = a.part_o + ((int64_t)s * a.rows + (valid ? grow : 0)) * kDLatent + half * 128;
#pragma unroll 2
      for (int c = 0; c < 16; ++c) {
        uint32_t o[16], w[8];
        TMEM_LD16(lane_addr + kColO + c * 16, o);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const __half2 h = __floats2half2_rn(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
          w[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        if (valid)
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(po + (c >> 3) * 256 + (c & 7) * 16),
                       "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                       : "memory");
      }
      if (half == 0 && local_row < R)
        a.part_lse[(int64_t)s * a.rows + grow] =
            !valid || l == 0.f ? -INFINITY : (m_run + (log2f(l) - kPBias)) * 0.6931471805599453f;
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    report(a.dev_status, 1, MLA_CHECK_TIMEOUT);
    if (threadIdx.x < kCtaRows && row0 + (int)threadIdx.x < R)
      a.part_lse[(int64_t)s * a.rows + (int64_t)b * R + row0 + threadIdx.x] = __int_as_float(0x7fc00000);
  }
  cluster_sync();  // neither CTA's tensor memory or shared memory is in the partner's use any more
  tc_fence_after();
  if (warp == kSWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  cluster_sync();
}

}  // namespace

cudaError_t launch_verify_kv4_tc(const VerifyArgs& a, cudaStream_t stream) {
  static std::atomic<bool> configured[64];  // the smem opt-in, set once per device (setting it twice is harmless)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(verify_kv4_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
  }
  const int64_t units = (int64_t)a.B * a.row_tiles * a.splits;
  if (units * 2 > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // programmatic dependent launch: inputs are read after griddepcontrol.wait
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kv4_tc_kernel, a);
}

}  // namespace mla
