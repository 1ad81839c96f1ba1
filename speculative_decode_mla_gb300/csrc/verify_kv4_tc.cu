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
//   warps 0-15   gather and dequantise: eight threads a key. Codes go from global memory through registers
//                (loads of a tile are out before the one before it is used), cvt e2m1x2 -> f16x2, times the block's
//                scale, to 128B-swizzled shared memory: K into a ring of 32 KB half tiles (256 dims of 64
//                keys), then, one tile later, V. A value's codes are read once for both.
//   warps 16-19  softmax, two threads a row (64 keys each): S from TMEM, ancestor bitmask on tree positions, row
//                maximum over the two threads through shared memory, exp2, P (fp16) to shared memory; O is
//                rescaled only when the running maximum grows by more than 2^8. The dequantising warps write O / l.
//   warp 20, 21  one thread each: CTA 0 issues S and PV for the pair; CTA 1 tells CTA 0 what is ready
//                (local barriers, then one remote arrive each: a cluster-scope release is slow, so the
//                working warps stay off it).
//
// P is kept as 2^(s - m + 7): under the lazy maximum it is at most 2^15, and weights down to 2^-32 of a
// row's largest still count in fp16. l is the fp32 sum of the unrounded weights.
//
// TMEM (512 columns): O [0, 256), two S buffers [256, 384), Q's dims 0..255 [384, 512) (both lane halves hold the
// CTA's 64 rows); Q's dims 256..511 and RoPE dims are in shared memory.
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
constexpr int kKSlots = 3;               // K ring: half tiles, 256 dims (four blocks) of the own 64 keys
constexpr int kKSlotBytes = 4 * kBlock;
constexpr int kVBlock = kKeys * 128;     // 128 keys x 64 dims
constexpr int kVHalfBytes = 2 * kVBlock; // 128 value dims
constexpr int kSmemK = 0;
constexpr int kSmemR = kSmemK + kKSlots * kKSlotBytes;  // RoPE dims of the own keys
constexpr int kSmemV = kSmemR + kBlock;
constexpr int kSmemP = kSmemV + 2 * kVHalfBytes;        // two blocks of 64 rows x 64 keys
constexpr int kSmemQ = kSmemP + 2 * kBlock;             // dims 256..511 (four blocks), RoPE
constexpr int kSmemX = kSmemQ + 5 * kBlock;             // exchange between the two threads of a row: [2][128] floats
constexpr int kSmemBar = kSmemX + 1024;
constexpr int kSmemBytes = kSmemBar + 512 + 1024;       // barriers, TMEM slot, tree parents + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory");

constexpr int kDequantWarps = 16;
constexpr int kSWarp = 20, kPVWarp = 21;  // 16..19: softmax, TMEM lane quarters 0..3; 22 and 23 only fill the warpgroup
constexpr int kThreads = 24 * 32;
// Registers a thread: 80 at launch (768 threads); the other warpgroups hand some of theirs to the softmax
// warpgroup: 4 x 64 + 168 + 56 = 6 x 80.
constexpr int kDequantRegs = 64, kSoftmaxRegs = 168, kIssuerRegs = 56;
constexpr int kParentThread0 = kSWarp * 32;  // 64 threads read the tree parents

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256 /* two buffers of 64 */, kColQ = 384;
constexpr int kQTmemDims = 256;
static_assert(2 * kVHalfBytes >= kCtaRows * kQTmemDims * 2, "half of Q passes through V's place");
constexpr float kPBias = 7.f;

constexpr int kBarKFull = 0, kBarKEmpty = kKSlots, kBarVFull = 2 * kKSlots /*2*/, kBarVEmpty = kBarVFull + 2 /*2*/,
              kBarSFull = kBarVEmpty + 2 /*2*/, kBarSEmpty = kBarSFull + 2 /*2*/, kBarPFull = kBarSEmpty + 2,
              kBarPEmpty = kBarPFull + 1, kBarQFull = kBarPFull + 2, kBarDrainS = kBarPFull + 3,
              kBarDrainP = kBarPFull + 4, kNumBars = kBarPFull + 5;
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
// A row's 64 dims as a thread takes them: 32 bytes of codes (two pieces of 32 dims) and their four scales.
struct Codes {
  uint32_t c[8];
  uint32_t s;
};
// v = the codes and scales at *p and *q where `on`, else v = other. The registers are read and written by one
// predicated instruction each: a load that reaches the next iteration through a branch gets a copy at the
// branch's end, and the copy waits for the load (about 1700 cycles a tile).
__device__ __forceinline__ void load_codes_or(Codes& v, const uint8_t* p, const uint8_t* q, bool on, const Codes& other) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %11, 0;\n"
      "@!p mov.b32 %0, %12;\n@!p mov.b32 %1, %13;\n@!p mov.b32 %2, %14;\n@!p mov.b32 %3, %15;\n"
      "@!p mov.b32 %4, %16;\n@!p mov.b32 %5, %17;\n@!p mov.b32 %6, %18;\n@!p mov.b32 %7, %19;\n"
      "@!p mov.b32 %8, %20;\n"
      "@p ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%9];\n"
      "@p ld.global.nc.b32 %8, [%10];\n}"
      : "+r"(v.c[0]), "+r"(v.c[1]), "+r"(v.c[2]), "+r"(v.c[3]), "+r"(v.c[4]), "+r"(v.c[5]), "+r"(v.c[6]), "+r"(v.c[7]),
        "+r"(v.s)
      : "l"(p), "l"(q), "r"((int)on), "r"(other.c[0]), "r"(other.c[1]), "r"(other.c[2]), "r"(other.c[3]), "r"(other.c[4]),
        "r"(other.c[5]), "r"(other.c[6]), "r"(other.c[7]), "r"(other.s));
}
__device__ __forceinline__ void load_codes_if(Codes& v, const uint8_t* p, const uint8_t* q, bool on) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %11, 0;\n"
      "@p ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%9];\n"
      "@p ld.global.nc.b32 %8, [%10];\n}"
      : "+r"(v.c[0]), "+r"(v.c[1]), "+r"(v.c[2]), "+r"(v.c[3]), "+r"(v.c[4]), "+r"(v.c[5]), "+r"(v.c[6]), "+r"(v.c[7]),
        "+r"(v.s)
      : "l"(p), "l"(q), "r"((int)on));
}
__device__ __forceinline__ void ld16_if(uint32_t (&v)[4], const uint8_t* p, bool on) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %5, 0;\n"
      "@p ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n}"
      : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3])
      : "l"(p), "r"((int)on));
}
// Arrives on a barrier of the partner CTA. What this thread has acquired from its own CTA's barriers is shared
// memory, so the release is restricted to that; a full cluster-scope release took about 1500 cycles.
__device__ __forceinline__ void arrive_partner(uint32_t cluster_bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// Two threads a row: warps w and w + 2 of the softmax warps.
__device__ __forceinline__ void row_pair_sync(int softmax_warp) {
  if (softmax_warp & 1) asm volatile("bar.sync 2, 64;" ::: "memory");
  else asm volatile("bar.sync 1, 64;" ::: "memory");
}

// 32 values (a 16-byte piece of a row's codes, its two scales as fp16; word j = 8 values) into four 16-byte chunks of
// a 128-byte row: word j at `at` ^ 16 j, where `at` is the place of word 0 (128B swizzle: chunk c lies at c ^ (row & 7)).
// `swap`: the words come in the order 2, 3, 0, 1, so the scales change places.
__device__ __forceinline__ void dequant_piece(const uint32_t* w, uint32_t scales, bool swap, uint32_t at) {
  const uint32_t s0 = __byte_perm(scales, 0, swap ? 0x3232 : 0x1010), s1 = __byte_perm(scales, 0, swap ? 0x1010 : 0x3232);
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
    st_shared_v4(at ^ (uint32_t)(16 * j), h);
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
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarSEmpty + i), 4 + relay);
    }
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
  // Eight threads a key: thread (key, pc) with key = 4 warp + lane / 8, pc = lane % 8 takes 32 bytes of its own key's
  // codes: the pieces (32 dims) 2 pc + i, i < 2, of K's half i. For V (CTA r supplies the dims 256 r .. 256 r + 255, of
  // half j the pieces 8 r + 2x + j) the threads with pc / 4 == rank use the same codes again, the others take the
  // partner's key.
  const int key = warp * 4 + (lane >> 3), pc = lane & 7;
  const bool v_own = (pc >> 2) == (int)rank;
  const uint8_t* pool = reinterpret_cast<const uint8_t*>(a.kv);
  const int32_t* tab = a.slot_table + (int64_t)b * a.stride;
  // The slot of position `key` of a CTA's share of tile t (positions past the end: 0), and its row. The slot is
  // loaded two tiles before its row is, and looked at only then.
  auto slot_at = [&](int t, uint32_t of_rank) -> int32_t {
    const int64_t pos = t0 + (int64_t)t * kKeys + (int)of_rank * kOwn + key;
    return pos < t1 ? tab[pos] : 0;
  };
  auto row_of = [&](int32_t slot) -> const uint8_t* {
    if (slot < 0 || slot >= a.num_slots) {
      report(a.dev_status, a.debug, MLA_CHECK_BAD_SLOT);
      slot = slot < 0 ? 0 : (int32_t)(a.num_slots - 1);
    }
    return pool + (int64_t)slot * kKv4Row;
  };
  Codes kc = {};
  uint32_t kr[4] = {};
  auto load_own = [&](const uint8_t* row, bool on) {
    load_codes_if(kc, row + 32 * pc, row + kKv4Codes + 4 * pc, on);
    ld16_if(kr, row + kKv4Rope + 16 * pc, on);
  };
  int32_t own_next = 0, peer_next = 0;
  if (warp < kDequantWarps) {
    const int32_t own = slot_at(0, rank);
    own_next = slot_at(1, rank);
    if (!v_own) peer_next = slot_at(0, rank ^ 1u);
    // Q: the same eight threads take query row `key`, 16-byte chunks pc + 8m (rows of padding nodes and past the
    // sequence: zeros). Their largest magnitude gives the row's power of two; times it, the dims of K's half 0 go
    // as fp16 to staging rows in V's place (the softmax warps put them into TMEM), those of half 1 and the RoPE dims
    // to their places.
    const bool q_valid = row0 + key < min(R, Tb * a.H);
    const uint8_t* q = reinterpret_cast<const uint8_t*>(a.q + ((int64_t)b * R + (q_valid ? row0 + key : 0)) * kDK) + 16 * pc;
    uint32_t qv[9][4] = {};
#pragma unroll
    for (int m = 0; m < 9; ++m) ld16_if(qv[m], q + 128 * m, q_valid);
    load_own(row_of(own), true);
    __nv_bfloat162 tops = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int m = 0; m < 9; ++m)
#pragma unroll
      for (int k = 0; k < 4; ++k) tops = __hmax2(tops, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&qv[m][k])));
    uint32_t top = *reinterpret_cast<const uint32_t*>(&tops);
    top = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    // top is in [2^(e - 127), 2^(e - 126)): k = 14 - (e - 127); rows of zeros, infinities or NaN stay as they are
    const int e = (int)(top >> 7);
    const int k2 = min(110, (e == 0 || e == 255) ? 0 : 141 - e);  // (2^-k2 stays a normal fp32 number)
    const float up = __int_as_float((127 + k2) << 23);
    if (pc == 0) reinterpret_cast<float*>(smem + kSmemX)[key] = __int_as_float((127 - k2) << 23) * a.scale_log2;
    const uint32_t r7 = (uint32_t)key & 7u, jj = (uint32_t)pc & 3u;
#pragma unroll
    for (int m = 0; m < 9; ++m) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float lo = __uint_as_float(qv[m][k] << 16) * up, hi = __uint_as_float(qv[m][k] & 0xffff0000u) * up;
        if (m < 8) {
          const __half2 h = __floats2half2_rn(lo, hi);
          w[k] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
          w[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      // chunk pc + 8m is word jj of piece 2m + pc / 4: half pc / 4, block m / 2, half row m % 2
      const uint32_t c = jj ^ (uint32_t)(m >> 1);
      uint32_t at = base + kSmemV + key * 512 + (((uint32_t)(4 * m) + c) ^ r7) * 16;
      if (pc >= 4) at = base + kSmemQ + (m >> 1) * kBlock + key * 128 + (((uint32_t)(4 * (m & 1)) + c) ^ r7) * 16;
      if (m == 8) at = base + kSmemQ + 4 * kBlock + key * 128 + ((uint32_t)pc ^ r7) * 16;
      st_shared_v4(at, w);
    }
    fence_proxy_async();  // generic-proxy stores, read by the MMA (async proxy)
  }

  tc_fence_before();
  __syncthreads();
  // Barrier inits (released by the fence after them) visible to the partner before any remote operation; the arrival is
  // relaxed, so it does not wait for the loads in flight.
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < kDequantWarps) {
    // ---------------------------------------------------------------- gather and dequantise
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDequantRegs));
    // Within a row's 64-dim block, word j of a piece goes to chunk j ^ (the block's number mod 4) of its half row, so that
    // the eight threads of a key store to eight different chunks at a time; Q's dims are laid out the same way. In V the
    // two blocks have the numbers 0 and 1 (the epilogue undoes it), and the partner's keys' words are stored two later.
    const uint32_t r7 = (uint32_t)key & 7u, h4 = (uint32_t)(pc & 1) * 4u, v_blk = (uint32_t)(pc & 3) >> 1;
    const uint32_t k_at = base + kSmemK + (uint32_t)(pc >> 1) * kBlock + key * 128 + (((h4 | (uint32_t)(pc >> 1)) ^ r7) << 4);
    const uint32_t v_at = base + kSmemV + v_blk * kVBlock + ((v_own ? rank : rank ^ 1u) * kOwn + key) * 128 +
                          (((h4 | (v_blk ^ (v_own ? 0u : 2u))) ^ r7) << 4);
    const uint32_t r_at = base + kSmemR + key * 128 + (((uint32_t)pc ^ r7) << 4);
    const uint32_t zero = (uint32_t)a.T >> 16;
    // Step `it`: K(it), the loads of K(it + 1) and of V(it), then V(it - 1). False at the end or after a failed wait. All
    // loads go out in one place and are used a step later (two sets of V's codes, so that none is copied).
    auto step = [&](const int it, Codes& next, Codes& now) -> bool {
      if (it < ntiles) {
        // K(it): two halves of 256 dims; the RoPE dims go with the second one, once S(it - 1), which reads its own
        // second half and RoPE dims last, is done.
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int sub = 2 * it + i, slot = sub % kKSlots;
          if (sub >= kKSlots && !wait_warp(bar(kBarKEmpty + slot), (sub / kKSlots - 1) & 1, abort_flag)) return false;
          dequant_piece(kc.c + 4 * i, e4m3x2_to_f16x2(i ? kc.s >> 16 : kc.s), false, k_at + slot * kKSlotBytes);
          if (i == 1) {
            const int before = sub - 2;
            if (it > 0 && !wait_warp(bar(kBarKEmpty + before % kKSlots), (before / kKSlots) & 1, abort_flag)) return false;
            st_shared_v4(r_at, kr);
          }
          fence_proxy_async();  // generic-proxy stores, read by the MMA (async proxy)
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarKFull + slot));
        }
        // Take delivery of the loads of `now` before the next ones go out: waiting for a load also waits for later
        // ones that share its scoreboard. (`zero` is 0, which the compiler does not know.)
#pragma unroll
        for (int j = 0; j < 8; ++j) now.c[j] ^= zero;
        now.s ^= zero;
        const uint8_t* peer = row_of(peer_next);  // V(it)'s codes: of the partner's row, or this thread's own once more
        load_codes_or(next, peer + 32 * (4 * (int)rank + (pc & 3)), peer + kKv4Codes + 4 * (4 * (int)rank + (pc & 3)), !v_own, kc);
        load_own(row_of(own_next), it + 1 < ntiles);
        own_next = slot_at(it + 2, rank);
        if (!v_own) peer_next = slot_at(it + 1, rank ^ 1u);
      }
      if (it > 0) {
        // V(it - 1), once PV(it - 2) has read the buffer (for the first tile: once Q has passed through it)
        const int t = it - 1;
        if (t == 0 && !wait_warp(bar(kBarQFull), 0, abort_flag, rank == 0)) return false;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (t > 0 && !wait_warp(bar(kBarVEmpty + j), (t - 1) & 1, abort_flag)) return false;
          const uint32_t* c = now.c + 4 * j;
          const uint32_t w[4] = {v_own ? c[0] : c[2], v_own ? c[1] : c[3], v_own ? c[2] : c[0], v_own ? c[3] : c[1]};
          dequant_piece(w, without_nan(e4m3x2_to_f16x2(j ? now.s >> 16 : now.s)), !v_own, v_at + j * kVHalfBytes);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarVFull + j));
        }
      }
      return it < ntiles;
    };
    Codes even = {}, odd = {};
    for (int it = 0; step(it, even, odd) && step(it + 1, odd, even); it += 2) {
    }

    // Epilogue: O / l as fp16 partials. Warp w reads TMEM lanes 32 (w % 4) .. (rows lane & 63) and the 64-dim block
    // w / 4 % 2 of half w / 8; lanes from 64 on hold the dims of CTA 1's V.
    const bool done = wait_warp(bar(kBarPEmpty), (ntiles - 1) & 1, abort_flag);
    asm volatile("bar.sync 3, %0;" ::"n"(32 * (kDequantWarps + 4)) : "memory");
    if (done) {
      tc_fence_after();
      const int l128 = (warp & 3) * 32 + lane, r = l128 & 63, local_row = row0 + r, hf = warp >> 3, blk = (warp >> 2) & 1;
      const bool valid = local_row < R && local_row / a.H < Tb;
      const float inv = reinterpret_cast<const float*>(smem + kSmemX)[(~ntiles & 1) * 128 + r];
      __half* po = a.part_o + ((int64_t)s * a.rows + (valid ? (int64_t)b * R + local_row : 0)) * kDLatent +
                   (l128 >> 6) * 256 + 128 * blk + 32 * hf;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // piece 2 (2 blk + h) + hf of this half's 256 dims
        uint32_t o[32];
        TMEM_LD16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColO + hf * 128 + blk * 64 + h * 32, o);
        TMEM_LD16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColO + hf * 128 + blk * 64 + h * 32 + 16, (o + 16));
        tmem_wait_ld();
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const __half2 v = __floats2half2_rn(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
          w[k] = *reinterpret_cast<const uint32_t*>(&v);
        }
        if (valid) {
#pragma unroll
          for (int k = 0; k < 16; k += 8) {  // chunk j of block 1 lies at j ^ 1
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(po + 64 * h + 2 * k),
                         "r"(blk ? w[k + 4] : w[k]), "r"(blk ? w[k + 5] : w[k + 1]), "r"(blk ? w[k + 6] : w[k + 2]),
                         "r"(blk ? w[k + 7] : w[k + 3]), "r"(blk ? w[k] : w[k + 4]), "r"(blk ? w[k + 1] : w[k + 5]),
                         "r"(blk ? w[k + 2] : w[k + 6]), "r"(blk ? w[k + 3] : w[k + 7])
                         : "memory");
          }
        }
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
          const int sb = t & 1;  // S buffer of tile t
          if (t > 1) ok = wait_bar(bar(kBarSEmpty + sb), ((t >> 1) - 1) & 1, abort_flag, true);
          const uint32_t d_s = tmem + kColS + (uint32_t)sb * 64u;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int sub = 2 * t + i, slot = sub % kKSlots;
            if (ok) ok = wait_bar(bar(kBarKFull + slot), (sub / kKSlots) & 1, abort_flag, true);
            if (!ok) break;
            tc_fence_after();
            const uint32_t kb = base + kSmemK + slot * kKSlotBytes;
#pragma unroll
            for (int k = 0; k < 16; ++k) {  // 16 dims each
              const uint64_t bd = smem_desc(kb + (k >> 2) * kBlock + (k & 3) * 32, 16, 1024);
              const int step = 16 * i + k;
              if (step < kQTmemDims / 16)
                mma2_tmem_a(d_s, tmem + kColQ + step * 8, bd, idesc_h, step ? 1u : 0u);
              else
                mma2_smem_a(d_s, smem_desc(base + kSmemQ + ((step >> 2) - 4) * kBlock + (step & 3) * 32, 16, 1024),
                            bd, idesc_h, 1u);
            }
            if (i == 1) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma2_smem_a(d_s, smem_desc(base + kSmemQ + 4 * kBlock + k * 32, 16, 1024),
                            smem_desc(base + kSmemR + k * 32, 16, 1024), idesc_b, 1u);
            }
            commit_both(bar(kBarKEmpty + slot));
          }
          if (ok) commit_both(bar(kBarSFull + sb));
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
        if (ok) arrive_partner(remote + 8u * kBarQFull);
        for (int t = 0; t < ntiles && ok; ++t) {
          if (t > 1) {
            ok = wait_bar(bar(kBarSEmpty + (t & 1)), ((t >> 1) - 1) & 1, abort_flag);
            if (ok) arrive_partner(remote + 8u * (uint32_t)(kBarSEmpty + (t & 1)));
          }
          for (int i = 0; i < 2 && ok; ++i) {
            const int sub = 2 * t + i, slot = sub % kKSlots;
            ok = wait_bar(bar(kBarKFull + slot), (sub / kKSlots) & 1, abort_flag);
            if (ok) arrive_partner(remote + 8u * (uint32_t)(kBarKFull + slot));
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
          if (ok) arrive_partner(remote + 8u * kBarVFull);
          ok = ok && wait_bar(bar(kBarPFull), t & 1, abort_flag);
          if (ok) arrive_partner(remote + 8u * kBarPFull);
          ok = ok && wait_bar(bar(kBarVFull + 1), t & 1, abort_flag);
          if (ok) arrive_partner(remote + 8u * (kBarVFull + 1));
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

    // Q's half 0 into TMEM, from the staging rows (both lanes of a row hold all of it)
    const float unscale = xch[r];
#pragma unroll 4
    for (int g = 0; g < kQTmemDims / 32; ++g) {  // 32 dims: 16 columns
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                     : "r"(base + kSmemV + r * 512 + (((uint32_t)(4 * g + i) ^ r7) << 4)));
      TMEM_ST16(lane_addr + kColQ + g * 16, w);
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarQFull));

    uint64_t anc = 0;  // anc*(node): the tree positions this row can see
    if (valid)
      for (int j = local_row / a.H, step = 0; j >= 0 && step < kMaxNodes; j = s_parent[j], ++step) anc |= 1ull << j;

    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;  // (the row pairs' barriers are passed whether or not a wait has failed)
    for (int t = 0; t < ntiles; ++t) {
      float sc[64];
      float mt = -INFINITY;
      if (ok) ok = wait_warp(bar(kBarSFull + (t & 1)), (t >> 1) & 1, abort_flag);
      if (ok) {
        tc_fence_after();
        uint32_t(&su)[64] = reinterpret_cast<uint32_t(&)[64]>(sc);
#pragma unroll
        for (int c = 0; c < 4; ++c) TMEM_LD16(lane_addr + kColS + (t & 1) * 64 + c * 16, (su + c * 16));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarSEmpty + (t & 1)));
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

    // l of the row from its two threads; 1 / l for the warps that write O, lse to the workspace
    xch[(ntiles & 1) * 128 + l128] = l_run;
    row_pair_sync(q4);
    const float l = l_run + xch[(ntiles & 1) * 128 + (l128 ^ 64)];
    if (half == 0) {
      xch[(~ntiles & 1) * 128 + r] = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
      if (ok && local_row < R)
        a.part_lse[(int64_t)s * a.rows + (int64_t)b * R + local_row] =
            !valid || l == 0.f ? -INFINITY : (m_run + (log2f(l) - kPBias)) * 0.6931471805599453f;
    }
    __syncwarp();
    asm volatile("bar.arrive 3, %0;" ::"n"(32 * (kDequantWarps + 4)) : "memory");
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
