// tcgen05 split-KV tree-verify kernel over the 4-bit latent pool, for sm_103a.
//
// Work is counted in tiles of 128 positions of one 128-row tile of a sequence's T*H query rows, in the order of
// the sequences and their row tiles, with kKv4SegmentUnits more after each row tile for what starting and ending a
// segment costs. Each cluster of two CTAs takes an equal, consecutive share of that (one cluster per pair of SMs), so
// that all SMs are busy for about the same time whatever the lengths are, and works through its segments: runs of
// tiles of one sequence and row tile. A cluster's segment is a split of its row tile, numbered from the row tile's
// first cluster on. The two CTAs' tensor cores work as a pair (cta_group::2, M = 128: CTA r holds query rows
// [64r, 64r + 64) of the row tile, all 128 TMEM lanes in use). A 64-row share of the fp32 output over 512
// value dims is 256 TMEM columns, so a pair holds whole rows and no partial scores travel between the
// CTAs. Per tile:
//
//   S = Q K^T   N = 128: CTA r supplies the keys of positions [64r, 64r + 64), all 576 dims
//   O += P V    N = 256, twice: CTA r supplies value dims [128r, 128r + 128) of each half, all positions
//
// so CTA r dequantises its own 64 rows whole and of the partner's 64 rows the 256 value dims
// that it supplies. Codes x scales are exact in fp16, so K, V and Q are fp16 operands; the RoPE dims
// stay bf16 (kind::f16 takes either, and both accumulate into the same fp32 scores). A query row is
// scaled by a power of two, the keys by another (kv4.cuh), and both are taken out of the scores.
//
//   warps 0-15   gather and dequantise: eight threads a key. Codes go from global memory through registers
//                (loads of a tile are out before the one before it is used), cvt e2m1x2 -> f16x2, times the block's
//                scale, to 128B-swizzled shared memory: K into a ring of 32 KB half tiles (256 dims of 64
//                keys), then, one tile later, V (a thread uses its own key's codes for both). At a segment's end they
//                write O / l: TMEM, rows in the K ring, one bulk copy of 1 KB a row.
//   warps 16-19  softmax, two threads a row (64 keys each): S from TMEM, ancestor bitmask on tree positions, row
//                maximum over the two threads through shared memory, exp2, P (fp16) to shared memory; O is
//                rescaled only when the running maximum grows by more than 2^8.
//   warp 20, 21  CTA 0's issue S and PV for the pair, one elected thread each; CTA 1's tell CTA 0 what is ready
//                (local barriers, then one remote arrive each: a cluster-scope release is slow, so the
//                working warps stay off it).
//   warp 22      finds the next segment and prefetches its query rows and first keys into L2.
//
// P is kept as 2^(s - m + 7): under the lazy maximum it is at most 2^15, and weights down to 2^-32 of a
// row's largest still count in fp16. l is the fp32 sum of the unrounded weights.
//
// TMEM (512 columns): O [0, 256), two S buffers [256, 384), Q's dims 0..255 [384, 512) (both lane halves hold the
// CTA's 64 rows); Q's dims 256..511 and RoPE dims are in shared memory.
//
// What bounds it: the L1 data path. Per tile and SM its counters show (256 rows x 180 Ki positions) 2830 wavefronts of
// loads and stores (152 KB of K, V, RoPE dims and P stored: 1220 at least, 1440 with the barriers; the gathered rows,
// 40 KB, in and out to registers: 1160) and 1660 of MMA operands (S: 72 KB of K, 40 of Q; PV: 64 of V, P twice), together
// as many as the SM has active cycles; the tensor cores need 2200 a tile (64 rows on each SM are half
// their rate). A segment costs about three tiles more (O out, Q in, and the
// first tile's K and V before the first PV), launch and merge about 10 us. 36 bytes are spilled in all (none before the
// maximum was taken away ahead of the product, at the same speed); the gather at 64 registers instead of 72, with 24 bytes
// spilled there, took 918 us for 4096 rows x 128 Ki instead of 867.
//   rows x positions (sequences): 64 x 1 Ki 13.3 us, 128 x 64 Ki 27.8, 256 x 180 Ki 94, 128 x 301 k (32) 93,
//   64 x 250 k (61) 86, 4096 x 128 Ki 859 (1.36 PFLOP/s); merge included
// One unit (sequence, row tile, chunk) a cluster, without the shares: 12.7, 28.5, 95, 118, 105, 938 (95.5 us then for 180 Ki).
//
// Positions past a sequence's end read slot 0's row and are masked; values whose scale is NaN are 0
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
constexpr int kSmemScale = kSmemX + 1024;               // what a row's scores are multiplied by: 64 floats
constexpr int kSmemInv = kSmemScale + 256;              // 1 / l of a row: 64 floats
constexpr int kSmemBar = kSmemInv + 256;
constexpr int kSmemBytes = kSmemBar + 512 + 1024;       // barriers, TMEM slot, tree parents + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory");

constexpr int kGatherWarps = 16;
constexpr int kSWarp = 20, kPVWarp = 21, kSegWarp = 22;  // 16..19: softmax, TMEM lane quarters 0..3; 23 only fills the warpgroup
constexpr int kThreads = 24 * 32;
// Registers a thread: 80 at launch (768 threads); the other warpgroups hand some of theirs to the softmax
// warpgroup: 4 x 72 + 152 + 40 = 6 x 80.
constexpr int kGatherRegs = 72, kSoftmaxRegs = 152, kIssuerRegs = 40;

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256 /* two buffers of 64 */, kColQ = 384;
constexpr int kQTmemDims = 256;
static_assert(2 * kVHalfBytes >= kCtaRows * kQTmemDims * 2, "half of Q passes through V's place");
constexpr int kOutRow = kDLatent * 2 + 16;  // a row of the output on its way out: 8 rows' chunks lie in different banks
static_assert(kCtaRows * kOutRow <= kKSlots * kKSlotBytes, "output rows");
constexpr int kPrefetchTiles = 3;  // of the next segment, to L2: 4096 sequences of 300 positions, 16 rows, took 911 us with 1, 878 with 3 then
constexpr float kPBias = 7.f;

constexpr int kBarKFull = 0, kBarKEmpty = kKSlots, kBarVFull = 2 * kKSlots /*2*/, kBarVEmpty = kBarVFull + 2 /*2*/,
              kBarSFull = kBarVEmpty + 2 /*2*/, kBarSEmpty = kBarSFull + 2 /*2*/, kBarPFull = kBarSEmpty + 2,
              kBarPEmpty = kBarPFull + 1, kBarQFull = kBarPFull + 2, kBarDrainS = kBarPFull + 3,
              kBarDrainP = kBarPFull + 4, kBarOEmpty = kBarPFull + 5, kBarSeg = kBarPFull + 6 /*2*/, kNumBars = kBarPFull + 8;
static_assert(8 * kNumBars + 8 + 4 * kMaxNodes + 64 <= 512, "barrier area");

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
__device__ __forceinline__ Codes copy_of(const Codes& v) {  // (an opaque copy: it is made before v is loaded again)
  Codes c;
#pragma unroll
  for (int j = 0; j < 8; ++j) asm volatile("mov.b32 %0, %1;" : "=r"(c.c[j]) : "r"(v.c[j]));
  asm volatile("mov.b32 %0, %1;" : "=r"(c.s) : "r"(v.s));
  return c;
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
__device__ __forceinline__ void prefetch_l2(const void* p, int bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.b32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
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

// The lengths of 32 sequences, one a lane: those from b0 on (no tiles past the last one).
struct Lengths {
  int32_t L, Tb;
  int ntiles;
};
__device__ __forceinline__ Lengths lengths_from(const VerifyArgs& a, int lane, int b0) {
  Lengths x = {0, 0, 0};
  if (b0 + lane < a.B) {
    x.L = load_len(a, b0 + lane);
    x.Tb = load_tree_size(a, b0 + lane);
    x.ntiles = (int)(((int64_t)x.L + x.Tb + kKeys - 1) / kKeys);
  }
  return x;
}
// The units of a sequence's row tiles: their tiles, and kKv4SegmentUnits after each for starting and ending a segment.
__device__ __forceinline__ int units_of(const VerifyArgs& a, int ntiles) {
  return ntiles ? (ntiles + kKv4SegmentUnits) * a.row_tiles : 0;
}
// The units of all sequences and row tiles (every lane of the warp calls it; `head`: the first 32 sequences).
__device__ __forceinline__ int all_units(const VerifyArgs& a, int lane, const Lengths& head) {
  int n = units_of(a, head.ntiles);
  for (int b0 = 32; b0 < a.B; b0 += 32) n += units_of(a, lengths_from(a, lane, b0).ntiles);
  return max(0, __reduce_add_sync(0xffffffffu, n) - kKv4SegmentUnits);  // (nothing follows the last tile)
}
struct Segment {
  int b, row_tile;
  int split, used;    // which split of its row tile it is, and how many that row tile has
  int tile0, ntiles;  // its tiles
  int32_t L, Tb;
};
// The segment that begins at unit w, for a cluster whose share ends at w_end; w goes to the next row tile first where
// it lies behind the last tile of one. The search begins at the 32 sequences from b0 on, with `base` units before them and
// the lengths x, and leaves the place where it ended (warp-collective).
__device__ __forceinline__ Segment segment_at(const VerifyArgs& a, int lane, Lengths x, int& b0, int& base, int& w, int w_end,
                                              int share) {
  Segment g = {};
#pragma unroll 1
  while (b0 < a.B) {
    const int own = units_of(a, x.ntiles);
    int inc = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += u;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, own > 0 && base + inc - kKv4SegmentUnits > w);
    if (past) {
      const int l = __ffs(past) - 1;
      const int ntiles = __shfl_sync(0xffffffffu, x.ntiles, l), per_row_tile = ntiles + kKv4SegmentUnits;
      const int start = base + __shfl_sync(0xffffffffu, inc - own, l);
      w = max(w, start);
      int row_tile = a.row_tiles == 1 ? 0 : (w - start) / per_row_tile;
      if (w - start - row_tile * per_row_tile >= ntiles) w = start + ++row_tile * per_row_tile;
      const int first = start + row_tile * per_row_tile, before = first / share;
      g.b = b0 + l;
      g.row_tile = row_tile;
      g.tile0 = w - first;
      g.ntiles = min(ntiles - g.tile0, w_end - w);
      g.split = w / share - before;
      g.used = (first + ntiles - 1) / share - before + 1;
      g.L = __shfl_sync(0xffffffffu, x.L, l);
      g.Tb = __shfl_sync(0xffffffffu, x.Tb, l);
      return g;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
    b0 += 32;
    x = lengths_from(a, lane, b0);
  }
  return g;
}

// The segments of a cluster, one after the other (every lane of the warp calls these).
struct Walk {
  int share, w, w_end, b0 = 0, base = 0;
  __device__ __forceinline__ Walk(const VerifyArgs& a, int lane, const Lengths& head) {
    const int clusters = (int)(gridDim.x >> 1), total = all_units(a, lane, head);
    share = max(a.chunk / kKeys, (total + clusters - 1) / clusters);
    w = (int)min((int64_t)total, (int64_t)(blockIdx.x >> 1) * share);
    w_end = min(total, w + share);
  }
  // The next one, if w < w_end says that the share goes on; no tiles: there is none.
  __device__ __forceinline__ Segment next(const VerifyArgs& a, int lane, const Lengths& head) {
    Segment g = segment_at(a, lane, head, b0, base, w, w_end, share);
    if (w >= w_end) g.ntiles = 0;
    w += g.ntiles + kKv4SegmentUnits;
    return g;
  }
};
// The cluster's segment number n once more, for use after a failed wait.
__device__ __forceinline__ Segment segment_number(const VerifyArgs& a, int lane, int n, bool& more) {
  const Lengths head = lengths_from(a, lane, 0);
  Walk walk(a, lane, head);
  Segment g = {};
  for (int i = 0; i <= n; ++i) {
    walk.b0 = walk.base = 0;
    g = walk.next(a, lane, head);
  }
  more = walk.w < walk.w_end;
  return g;
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
  volatile int32_t* s_seg = s_parent + kMaxNodes;  // the segments with odd and even numbers, the current and the next one
  float* xch = reinterpret_cast<float*>(smem + kSmemX);
  float* s_scale = reinterpret_cast<float*>(smem + kSmemScale);
  float* s_inv = reinterpret_cast<float*>(smem + kSmemInv);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int R = a.T * a.H;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const Lengths head = lengths_from(a, lane, 0);
  Walk walk(a, lane, head);
  if (walk.w >= walk.w_end) return;  // (both CTAs agree, here and below)
  Segment first = walk.next(a, lane, head);
  if (first.ntiles == 0) return;
  auto put_segment = [&](int n, const Segment& g, bool more) {  // (one thread)
    volatile int32_t* s = s_seg + 8 * (n & 1);
    s[0] = g.b;
    s[1] = g.row_tile;
    s[2] = g.split;
    s[3] = g.used;
    s[4] = g.tile0;
    s[5] = more ? g.ntiles : -g.ntiles;
    s[6] = g.L;
    s[7] = g.Tb;
  };
  // Segment n, from warp kSegWarp (after a failed wait from the lengths: every warp has to pass its named barriers).
  auto get_segment = [&](int n, bool& more, bool& ok) {
    if (n > 0 && !wait_warp(bar(kBarSeg + (n & 1)), ((n - 1) >> 1) & 1, abort_flag)) {
      ok = false;
      return segment_number(a, lane, n, more);
    }
    volatile int32_t* s = s_seg + 8 * (n & 1);
    const int tiles = s[5];
    more = tiles > 0;
    return Segment{s[0], s[1], s[2], s[3], s[4], abs(tiles), s[6], s[7]};
  };

  if (threadIdx.x == 0) {
    const uint32_t relay = rank == 0 ? 1u : 0u;  // CTA 0 also waits for the word of CTA 1
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(bar(kBarKFull + i), kGatherWarps + relay);
      mbar_init(bar(kBarKEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarVFull + i), kGatherWarps + relay);
      mbar_init(bar(kBarVEmpty + i), 1);
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarSEmpty + i), 4 + relay);
    }
    mbar_init(bar(kBarPFull), 4 + relay);
    mbar_init(bar(kBarPEmpty), 1);
    mbar_init(bar(kBarQFull), 4 + relay);
    mbar_init(bar(kBarOEmpty), kGatherWarps + relay);
    for (int i = 0; i < 2; ++i) mbar_init(bar(kBarSeg + i), 1);
    mbar_init(bar(kBarDrainS), 1);
    mbar_init(bar(kBarDrainP), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kSegWarp && lane == 0) put_segment(0, first, walk.w < walk.w_end);
  if (warp == kSWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  // Barrier inits (released by the fence after them) visible to the partner before any remote operation.
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Every role walks the same segments; `t` counts a segment's tiles, `gt` all tiles of the cluster (barrier phases go by
  // it). After a failed wait a role skips its work but passes every named barrier.
  if (warp < kGatherWarps) {
    // ---------------------------------------------------------------- gather and dequantise
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGatherRegs));
    // Eight threads a key: thread (key, pc) with key = 4 warp + lane / 8, pc = lane % 8 takes 32 bytes of its own key's
    // codes: the pieces (32 dims) 2 pc + i, i < 2, of K's half i. For V (CTA r supplies the dims 256 r .. 256 r + 255, of
    // half j the pieces 8 r + 2x + j) the threads with pc / 4 == rank use the same codes again, the others take the
    // partner's key.
    // Within a row's 64-dim block, word j of a piece goes to chunk j ^ (the block's number mod 4) of its half row, so that
    // the eight threads of a key store to eight different chunks at a time; Q's dims are laid out the same way. In V the
    // two blocks have the numbers 0 and 1 (the epilogue undoes it), and the partner's keys' words are stored two later.
    const int key = warp * 4 + (lane >> 3), pc = lane & 7;
    const bool v_own = (pc >> 2) == (int)rank;
    const uint32_t r7 = (uint32_t)key & 7u, h4 = (uint32_t)(pc & 1) * 4u, v_blk = (uint32_t)(pc & 3) >> 1;
    const uint32_t k_at = base + kSmemK + (uint32_t)(pc >> 1) * kBlock + key * 128 + (((h4 | (uint32_t)(pc >> 1)) ^ r7) << 4);
    const uint32_t v_at = base + kSmemV + v_blk * kVBlock + ((v_own ? rank : rank ^ 1u) * kOwn + key) * 128 +
                          (((h4 | (v_blk ^ (v_own ? 0u : 2u))) ^ r7) << 4);
    const uint32_t r_at = base + kSmemR + key * 128 + (((uint32_t)pc ^ r7) << 4);
    const uint32_t zero = (uint32_t)a.T >> 16;
    const uint8_t* pool = reinterpret_cast<const uint8_t*>(a.kv);
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
    bool ok = true;
    // K ring: the next slot, the parity of its uses so far; the parity of the tiles so far. (A wait for the phase before a
    // barrier's first one, parity 1, returns at once.)
    uint32_t k_slot = 0, k_par = 0, t_par = 0;
    int nseg = 0, ntiles = 0;
    for (bool more = true; more; ++nseg) {
      const Segment sg = get_segment(nseg, more, ok);
      ntiles = sg.ntiles;
      const int32_t* tab = a.slot_table + (int64_t)sg.b * a.stride + (int64_t)sg.tile0 * kKeys + key;
      const int past = (int)min((int64_t)ntiles * kKeys, (int64_t)sg.L + sg.Tb - (int64_t)sg.tile0 * kKeys) - key;
      // The slot of position `key` of a CTA's share of tile t (past the end: 0). It is loaded a tile or two before
      // its row is, and looked at only then.
      auto slot_at = [&](int t, uint32_t of_rank) -> int32_t {
        const int at = t * kKeys + (int)of_rank * kOwn;
        return at < past ? tab[at] : 0;
      };
      const int32_t own = slot_at(0, rank);
      int32_t own_next = slot_at(1, rank), peer_next = v_own ? 0 : slot_at(0, rank ^ 1u);
      if (ok) {
        const int row0 = sg.row_tile * kRows + (int)rank * kCtaRows;  // this CTA's first row of the sequence
        const int rows_here = min(kCtaRows, min(R, sg.Tb * a.H) - row0);
        // Q: the same eight threads take query row `key`, 16-byte chunks pc + 8m (rows of padding nodes and past the
        // sequence: zeros). Their largest magnitude gives the row's power of two; times it, the dims of K's half 0 go
        // as fp16 to staging rows in V's place (the softmax warps put them into TMEM), those of half 1 and the RoPE dims
        // to their places. All of these are free: the segment before has been written out.
        const uint8_t* q =
            reinterpret_cast<const uint8_t*>(a.q + ((int64_t)sg.b * R + (key < rows_here ? row0 + key : 0)) * kDK) + 16 * pc;
        uint32_t qv[9][4] = {};
#pragma unroll
        for (int m = 0; m < 9; ++m) ld16_if(qv[m], q + 128 * m, key < rows_here);
        __nv_bfloat162 tops = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
        for (int m = 0; m < 9; ++m)
#pragma unroll
          for (int k = 0; k < 4; ++k) tops = __hmax2(tops, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&qv[m][k])));
        uint32_t top = *reinterpret_cast<const uint32_t*>(&tops);
        top = max(top & 0xffffu, top >> 16);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        load_own(row_of(own), true);
        const int k2 = query_shift(top);
        const float up = exp2i(k2);
        if (pc == 0) s_scale[key] = score_scale(k2, a.scale_log2);
        const uint32_t jj = (uint32_t)pc & 3u;
#pragma unroll
        for (int m = 0; m < 9; ++m) {
          uint32_t x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float f = m < 8 ? up : up * exp2i(-kKeyShift);
            const float lo = __uint_as_float(qv[m][k] << 16) * f, hi = __uint_as_float(qv[m][k] & 0xffff0000u) * f;
            if (m < 8) {
              const __half2 h = __floats2half2_rn(lo, hi);
              x[k] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
              const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
              x[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
          }
          // chunk pc + 8m is word jj of piece 2m + pc / 4: half pc / 4, block m / 2, half row m % 2
          const uint32_t c = jj ^ (uint32_t)(m >> 1);
          uint32_t at = base + kSmemV + key * 512 + (((uint32_t)(4 * m) + c) ^ r7) * 16;
          if (pc >= 4) at = base + kSmemQ + (m >> 1) * kBlock + key * 128 + (((uint32_t)(4 * (m & 1)) + c) ^ r7) * 16;
          if (m == 8) at = base + kSmemQ + 4 * kBlock + key * 128 + ((uint32_t)pc ^ r7) * 16;
          st_shared_v4(at, x);
        }
        fence_proxy_async();  // generic-proxy stores, read by the MMA (async proxy)
      }
      __syncwarp();
      asm volatile("bar.arrive 4, %0;" ::"n"(32 * (kGatherWarps + 4)) : "memory");
      if (nseg > 0) {  // the output of the segment before has been read out of the K ring
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        asm volatile("bar.sync 6, %0;" ::"n"(32 * kGatherWarps) : "memory");
      }

      // Step `it`: K(it), the loads of K(it + 1), V(it - 1), then V(it)'s codes. (One copy of this code: all roles' loops
      // together have to stay in the instruction cache.)
      Codes vc = {};
      for (int it = 0; it <= ntiles && ok; ++it) {
        Codes again = {};
        if (it < ntiles) {
          // K(it): two halves of 256 dims; the RoPE dims go with the second one, once the S before, which reads its own
          // second half and RoPE dims last, is done.
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            ok = ok && wait_warp(bar(kBarKEmpty + k_slot), k_par ^ 1u, abort_flag);
            if (!ok) break;
            dequant_piece(kc.c + 4 * i, key_scales(e4m3x2_to_f16x2(i ? kc.s >> 16 : kc.s)), false, k_at + k_slot * kKSlotBytes);
            if (i == 1) {
              // (the slot of the S before's second half is two back, or one on)
              ok = wait_warp(bar(kBarKEmpty + (k_slot == 2 ? 0 : k_slot + 1)), k_slot == 2 ? k_par : k_par ^ 1u, abort_flag);
              if (!ok) break;
              st_shared_v4(r_at, kr);
            }
            fence_proxy_async();  // generic-proxy stores, read by the MMA (async proxy)
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarKFull + k_slot));
            if (++k_slot == kKSlots) {
              k_slot = 0;
              k_par ^= 1u;
            }
          }
          if (!ok) break;
          again = copy_of(kc);
          load_own(row_of(own_next), it + 1 < ntiles);
          own_next = slot_at(it + 2, rank);
        }
        if (it > 0) {
          // V(it - 1), once the PV before has read the buffer (the first one: once Q has passed through it)
          if (it == 1) ok = wait_warp(bar(kBarQFull), nseg & 1, abort_flag, rank == 0);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            ok = ok && wait_warp(bar(kBarVEmpty + j), t_par ^ 1u, abort_flag);
            if (!ok) break;
            const uint32_t* c = vc.c + 4 * j;
            const uint32_t x[4] = {v_own ? c[0] : c[2], v_own ? c[1] : c[3], v_own ? c[2] : c[0], v_own ? c[3] : c[1]};
            dequant_piece(x, without_nan(e4m3x2_to_f16x2(j ? vc.s >> 16 : vc.s)), !v_own, v_at + j * kVHalfBytes);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarVFull + j));
          }
          if (!ok) break;
          t_par ^= 1u;
        }
        // Take delivery of K(it + 1)'s codes before the next loads go out: waiting for a load also waits for later ones
        // that share its scoreboard. (`zero` is 0, which the compiler does not know.)
#pragma unroll
        for (int j = 0; j < 8; ++j) kc.c[j] ^= zero;
        kc.s ^= zero;
        const uint8_t* peer = row_of(peer_next);  // V(it)'s codes: of the partner's row, or this thread's own once more
        load_codes_or(vc, peer + 32 * (4 * (int)rank + (pc & 3)), peer + kKv4Codes + 4 * (4 * (int)rank + (pc & 3)),
                      !v_own && it < ntiles, again);
        if (!v_own) peer_next = slot_at(it + 1, rank ^ 1u);
      }

      // Epilogue: O / l as fp16 partials. Warp w reads TMEM lanes 32 (w % 4) .. (rows lane & 63) and the 64-dim block
      // w / 4 % 2 of half w / 8; lanes from 64 on hold the dims of CTA 1's V.
      ok = ok && wait_warp(bar(kBarPEmpty), t_par ^ 1u, abort_flag);
      asm volatile("bar.sync 3, %0;" ::"n"(32 * (kGatherWarps + 4)) : "memory");
      if (ok) {
        tc_fence_after();
        const int l128 = (warp & 3) * 32 + lane, r = l128 & 63, hf = warp >> 3, blk = (warp >> 2) & 1;
        const float inv = s_inv[r];
        const uint32_t src = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColO + hf * 128 + blk * 64;
        uint32_t x[32];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t o[16];
          TMEM_LD16(src + h * 16, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const __half2 v = __floats2half2_rn(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
            x[8 * h + k] = *reinterpret_cast<const uint32_t*>(&v);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarOEmpty));
        // Half h % 2 of piece 2 (2 blk + h / 2) + hf of this CTA half's 256 dims; chunk j of block 1 lies at j ^ 1. Through
        // rows in the K ring, whose last S is done, since a row of the partials is 1 KB in one piece.
        const uint32_t to = base + kSmemK + r * kOutRow + ((l128 >> 6) * 256 + 128 * blk + 32 * hf) * 2;
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = blk ? x[8 * h + 4 * (c ^ 1) + k] : x[8 * h + 4 * c + k];
            st_shared_v4(to + 128 * (h >> 1) + 32 * (h & 1) + 16 * c, y);
          }
        fence_proxy_async();  // read by the bulk copies
      }
      asm volatile("bar.sync 6, %0;" ::"n"(32 * kGatherWarps) : "memory");
      if (ok && lane < 4) {
        volatile int32_t* s = s_seg + 8 * (nseg & 1);  // (read once more rather than kept through the tiles)
        const int r = 4 * warp + lane, row = s[1] * kRows + (int)rank * kCtaRows + r;
        if (row < min(R, s[7] * a.H))
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                           a.part_o + ((int64_t)s[2] * a.rows + (int64_t)s[0] * R + row) * kDLatent),
                       "r"(base + kSmemK + r * kOutRow), "n"(kDLatent * 2)
                       : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else if (warp >= kSWarp) {
    // The whole warp walks the loops, so that the operands of its MMAs stay uniform; one elected thread issues them.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssuerRegs));
    const uint32_t remote = map_to_cta(bar0, 0);
    const bool leader = elect_one();
    bool ok = true;
    int gt = 0, nseg = 0;
    if (warp == kSWarp) {
      int k_slot = 0, k_round = 0;
      auto next_slot = [&]() {
        if (++k_slot == kKSlots) {
          k_slot = 0;
          ++k_round;
        }
      };
      for (bool more = true; more && ok; ++nseg) {
        ok = wait_warp(bar(kBarQFull), nseg & 1, abort_flag, rank == 0);
        if (!ok) break;
        const int tiles = s_seg[8 * (nseg & 1) + 5], end = gt + abs(tiles);
        more = tiles > 0;
        if (rank == 0) {
          // ------------------------------------------------------------ S issuer
          constexpr uint32_t idesc_h = instr_desc(kKeys, false, false), idesc_b = instr_desc(kKeys, true, false);
          for (; gt < end && ok; ++gt) {
            const int sb = gt & 1;  // S buffer
            if (gt > 1) ok = wait_warp(bar(kBarSEmpty + sb), ((gt >> 1) - 1) & 1, abort_flag, true);
            const uint32_t d_s = tmem + kColS + (uint32_t)sb * 64u;
            // dims of half 0, A = Q from TMEM, then of half 1 and the RoPE dims, A = Q from shared memory: 16 dims a
            // step, a block of 64 dims at a time
            ok = ok && wait_warp(bar(kBarKFull + k_slot), k_round & 1, abort_flag, true);
            if (!ok) break;
            tc_fence_after();
            if (leader) {
              const uint64_t kd = smem_desc(base + kSmemK + k_slot * kKSlotBytes, 16, 1024);
#pragma unroll 1
              for (int x = 0; x < 4; ++x) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma2_tmem_a(d_s, tmem + kColQ + (4 * x + k) * 8, desc_at(kd, x * kBlock + k * 32), idesc_h,
                              (x | k) ? 1u : 0u);
              }
              commit_both(bar(kBarKEmpty + k_slot));
            }
            next_slot();
            ok = wait_warp(bar(kBarKFull + k_slot), k_round & 1, abort_flag, true);
            if (!ok) break;
            tc_fence_after();
            if (leader) {
              const uint64_t kd = smem_desc(base + kSmemK + k_slot * kKSlotBytes, 16, 1024);
              const uint64_t qd = smem_desc(base + kSmemQ, 16, 1024), rd = smem_desc(base + kSmemR, 16, 1024);
#pragma unroll 1
              for (int x = 0; x < 5; ++x) {
                const uint64_t bb = x < 4 ? desc_at(kd, x * kBlock) : rd;
                const uint32_t idesc = x < 4 ? idesc_h : idesc_b;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma2_smem_a(d_s, desc_at(qd, x * kBlock + k * 32), desc_at(bb, k * 32), idesc, 1u);
              }
              commit_both(bar(kBarKEmpty + k_slot));
              commit_both(bar(kBarSFull + sb));
            }
            next_slot();
          }
        } else {
          // ------------------------------------------------------------ CTA 1: what S waits for, to CTA 0
          if (leader) arrive_partner(remote + 8u * kBarQFull);
          for (; gt < end && ok; ++gt) {
            if (gt > 1) {
              ok = wait_warp(bar(kBarSEmpty + (gt & 1)), ((gt >> 1) - 1) & 1, abort_flag);
              if (ok && leader) arrive_partner(remote + 8u * (uint32_t)(kBarSEmpty + (gt & 1)));
            }
            for (int i = 0; i < 2 && ok; ++i) {
              ok = wait_warp(bar(kBarKFull + k_slot), k_round & 1, abort_flag);
              if (ok && leader) arrive_partner(remote + 8u * (uint32_t)(kBarKFull + k_slot));
              next_slot();
            }
          }
        }
      }
    } else if (warp == kPVWarp) {
      for (bool more = true; more && ok; ++nseg) {
        ok = wait_warp(bar(kBarQFull), nseg & 1, abort_flag, rank == 0);
        if (!ok) break;
        const int tiles = s_seg[8 * (nseg & 1) + 5], ntiles = abs(tiles);
        more = tiles > 0;
        if (rank == 0) {
          // ------------------------------------------------------------ PV issuer
          constexpr uint32_t idesc_pv = instr_desc(256, false, true);
          if (nseg > 0) ok = ok && wait_warp(bar(kBarOEmpty), (nseg - 1) & 1, abort_flag, true);
          for (int t = 0; t < ntiles && ok; ++t, ++gt) {
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
              ok = ok && wait_warp(bar(kBarVFull + j), gt & 1, abort_flag, true);
              if (j == 0) ok = ok && wait_warp(bar(kBarPFull), gt & 1, abort_flag, true);
              if (!ok) break;
              tc_fence_after();
              if (leader) {
                const uint64_t pd = smem_desc(base + kSmemP, 16, 1024), vd = smem_desc(base + kSmemV, kVBlock, 1024);
#pragma unroll 1
                for (int x = 0; x < 2; ++x)
#pragma unroll
                  for (int k = 0; k < 4; ++k)  // 16 positions each; V is read MN-major
                    mma2_smem_a(tmem + kColO + j * 128, desc_at(pd, x * kBlock + k * 32),
                                desc_at(vd, j * kVHalfBytes + (4 * x + k) * 2048), idesc_pv,
                                (t | x | k) ? 1u : 0u);
                commit_both(bar(kBarVEmpty + j));
                if (j == 1) commit_both(bar(kBarPEmpty));
              }
            }
          }
        } else {
          if (nseg > 0) {
            ok = ok && wait_warp(bar(kBarOEmpty), (nseg - 1) & 1, abort_flag);
            if (ok && leader) arrive_partner(remote + 8u * kBarOEmpty);
          }
          for (int t = 0; t < ntiles && ok; ++t, ++gt) {
            ok = wait_warp(bar(kBarVFull), gt & 1, abort_flag);
            if (ok && leader) arrive_partner(remote + 8u * kBarVFull);
            ok = ok && wait_warp(bar(kBarPFull), gt & 1, abort_flag);
            if (ok && leader) arrive_partner(remote + 8u * kBarPFull);
            ok = ok && wait_warp(bar(kBarVFull + 1), gt & 1, abort_flag);
            if (ok && leader) arrive_partner(remote + 8u * (kBarVFull + 1));
          }
        }
      }
    }
    if (warp == kSegWarp) {
      // ------------------------------------------------------------ the segments to come, and their first data to L2
      // This CTA's rows of Q, and its keys of the first tiles: later ones are loaded a tile ahead, which hides the latency.
      auto prefetch = [&](const Segment& sg) {
        const int row0 = sg.row_tile * kRows + (int)rank * kCtaRows;
        const int rows_here = min(kCtaRows, min(R, sg.Tb * a.H) - row0);
        if (lane == 0 && rows_here > 0) prefetch_l2(a.q + ((int64_t)sg.b * R + row0) * kDK, rows_here * kDK * 2);
        const int32_t* tab = a.slot_table + (int64_t)sg.b * a.stride;
        const int64_t first = (int64_t)sg.tile0 * kKeys + (int)rank * kOwn + lane, end = (int64_t)sg.L + sg.Tb;
#pragma unroll 1
        for (int t = 0; t < min(sg.ntiles, kPrefetchTiles); ++t)
#pragma unroll
          for (int i = 0; i < kOwn; i += 32) {
            const int64_t at = first + t * kKeys + i;
            const int32_t slot = at < end ? tab[at] : -1;
            if (slot >= 0 && slot < a.num_slots)
              prefetch_l2(reinterpret_cast<const uint8_t*>(a.kv) + (int64_t)slot * kKv4Row, kKv4Row);
          }
        __syncwarp();
      };
      for (int n = 1; walk.w < walk.w_end; ++n) {
        // the place of segment n - 2 is free once Q of segment n - 1 is in place: every role has read that one
        // (after all of segment n - 2, which may take longer than other waits do: several times its tiles' time on top)
        const long long start = clock64(), limit = kTimeoutCycles + (n > 1 ? 32768ll * abs(s_seg[8 * (n & 1) + 5]) : 0);
        bool ready = mbar_test(bar(kBarQFull), (n - 1) & 1);
        while (!ready && !*abort_flag && clock64() - start <= limit) ready = mbar_test(bar(kBarQFull), (n - 1) & 1);
        if (!ready) *abort_flag = 1;
        if (!__all_sync(0xffffffffu, ready)) break;
        const Segment sg = walk.next(a, lane, lengths_from(a, lane, walk.b0));
        if (lane == 0) {
          put_segment(n, sg, walk.w < walk.w_end);
          mbar_arrive(bar(kBarSeg + (n & 1)));
        }
        __syncwarp();
        prefetch(sg);
      }
    }
    if (rank == 0 && warp <= kPVWarp) {  // drain: every MMA that the elected thread issued has completed once this flips
      const int drain = warp == kSWarp ? kBarDrainS : kBarDrainP;
      if (leader) commit_own(bar(drain));
      const long long st = clock64();
      while (!mbar_test(bar(drain), 0) && clock64() - st < kTimeoutCycles) {
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax, two threads a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int q4 = warp & 3;
    const int l128 = q4 * 32 + lane;  // TMEM lane
    const int r = l128 & 63, half = l128 >> 6;
    const uint32_t lane_addr = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t r7 = (uint32_t)r & 7u;
    bool ok = true;
    int g0 = 0, nseg = 0, ntiles = 0;
    for (bool more = true; more; g0 += ntiles, ++nseg) {
      const Segment sg = get_segment(nseg, more, ok);
      ntiles = sg.ntiles;
      // prefix positions from this thread's first one on
      const int ahead = (int)(sg.L - (int64_t)sg.tile0 * kKeys) - half * 64;
      const int local_row = sg.row_tile * kRows + (int)rank * kCtaRows + r;
      const bool valid = local_row < min(R, sg.Tb * a.H);
      if (l128 < a.T) {  // tree parents of this sequence, validated
        int p = a.tree_parent[(int64_t)sg.b * a.T + l128];
        if (l128 >= sg.Tb) {
          p = -1;
        } else if (p < -1 || p >= l128) {
          report(a.dev_status, a.debug, MLA_CHECK_BAD_PARENT);
          p = -1;
        }
        s_parent[l128] = p;
      }
      if (sg.split == 0 && half == 1 && local_row < R)  // the splits that this row tile does not have
        for (int x = sg.used; x < a.splits; ++x) a.part_lse[(int64_t)x * a.rows + (int64_t)sg.b * R + local_row] = -INFINITY;
      asm volatile("bar.sync 5, 128;" ::: "memory");
      uint64_t anc = 0;  // anc*(node): the tree positions this row can see
      if (valid)
        for (int j = local_row / a.H, step = 0; j >= 0 && step < kMaxNodes; j = s_parent[j], ++step) anc |= 1ull << j;
      asm volatile("bar.sync 4, %0;" ::"n"(32 * (kGatherWarps + 4)) : "memory");
      tc_fence_after();

      // Q's half 0 into TMEM, from the staging rows (both lanes of a row hold all of it)
      const float unscale = s_scale[r];
#pragma unroll 4
      for (int g = 0; g < kQTmemDims / 32; ++g) {  // 32 dims: 16 columns
        uint32_t x[16];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[4 * i]), "=r"(x[4 * i + 1]), "=r"(x[4 * i + 2]), "=r"(x[4 * i + 3])
                       : "r"(base + kSmemV + r * 512 + (((uint32_t)(4 * g + i) ^ r7) << 4)));
        TMEM_ST16(lane_addr + kColQ + g * 16, x);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarQFull));

      float m_run = -INFINITY, l_run = 0.f;
      for (int t = 0; t < ntiles; ++t) {
        const int gt = g0 + t;
        float sc[64];
        float mt = -INFINITY;
        if (ok) ok = wait_warp(bar(kBarSFull + (gt & 1)), (gt >> 1) & 1, abort_flag);
        if (ok) {
          tc_fence_after();
          uint32_t(&su)[64] = reinterpret_cast<uint32_t(&)[64]>(sc);
#pragma unroll
          for (int c = 0; c < 4; ++c) TMEM_LD16(lane_addr + kColS + (gt & 1) * 64 + c * 16, (su + c * 16));
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarSEmpty + (gt & 1)));
          const int n = ahead - t * kKeys;  // how many of this thread's 64 positions are in the prefix
          if (n < 64) {                     // the others: the tree's bitmask
            uint64_t vis = 0;
            if (n > 0) vis = ((1ull << n) - 1) | (anc << n);
            else if (n > -64) vis = anc >> -n;
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
        xch[(gt & 1) * 128 + l128] = mt;
        row_pair_sync(q4);
        if (!ok) continue;
        // The running maximum is kept as the scores come, before their scale, and taken away before the product: the key that
        // set it weighs 2^kPBias to the bit however large the scores are. (One fma, the exact product less the rounded
        // product of the maximum, is off by half an ulp of it: from 2^27 on that put weights anywhere from 0 to infinity.)
        mt = fmaxf(mt, xch[(gt & 1) * 128 + (l128 ^ 64)]);
        bool rescale = false;
        float alpha = 1.f;
        if ((mt - m_run) * unscale > 8.f || m_run == -INFINITY) {
          alpha = m_run == -INFINITY ? 0.f : ex2((m_run - mt) * unscale);
          rescale = t > 0 && m_run != mt;
          l_run *= alpha;
          m_run = mt;
        }
        const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
        uint32_t pk[32];
        float2 ls0 = make_float2(0.f, 0.f), ls1 = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 64; k += 4) {
          const float2 d0 = add2(make_float2(sc[k], sc[k + 1]), make_float2(neg_m, neg_m));
          const float2 d1 = add2(make_float2(sc[k + 2], sc[k + 3]), make_float2(neg_m, neg_m));
          const float2 x0 = fma2(d0, make_float2(unscale, unscale), make_float2(kPBias, kPBias));
          const float2 x1 = fma2(d1, make_float2(unscale, unscale), make_float2(kPBias, kPBias));
          const float2 e0 = make_float2(ex2(x0.x), ex2(x0.y)), e1 = make_float2(ex2(x1.x), ex2(x1.y));
          const __half2 h0 = __floats2half2_rn(e0.x, e0.y), h1 = __floats2half2_rn(e1.x, e1.y);
          pk[k / 2] = *reinterpret_cast<const uint32_t*>(&h0);
          pk[k / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
          ls0 = add2(ls0, e0);
          ls1 = add2(ls1, e1);
        }
        l_run += (ls0.x + ls0.y) + (ls1.x + ls1.y);

        // P (and O) once the PV before has finished with them
        if (gt > 0) {
          ok = wait_warp(bar(kBarPEmpty), (gt - 1) & 1, abort_flag);
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
      xch[((g0 + ntiles) & 1) * 128 + l128] = l_run;
      row_pair_sync(q4);
      const float l = l_run + xch[((g0 + ntiles) & 1) * 128 + (l128 ^ 64)];
      if (half == 0) {
        s_inv[r] = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
        volatile int32_t* s = s_seg + 8 * (nseg & 1);
        const int row = s[1] * kRows + (int)rank * kCtaRows + r;
        if (ok && row < R)
          a.part_lse[(int64_t)s[2] * a.rows + (int64_t)s[0] * R + row] =
              row >= s[7] * a.H || l == 0.f ? -INFINITY : (m_run * unscale + (log2f(l) - kPBias)) * 0.6931471805599453f;
      }
      __syncwarp();
      asm volatile("bar.arrive 3, %0;" ::"n"(32 * (kGatherWarps + 4)) : "memory");
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    report(a.dev_status, 1, MLA_CHECK_TIMEOUT);
    bool more = true;
    for (int n = 0; more; ++n) {
      const Segment sg = segment_number(a, lane, n, more);
      const int local_row = sg.row_tile * kRows + (int)rank * kCtaRows + (int)threadIdx.x;
      if (threadIdx.x < kCtaRows && local_row < R)
        a.part_lse[(int64_t)sg.split * a.rows + (int64_t)sg.b * R + local_row] = __int_as_float(0x7fc00000);
    }
  }
  cluster_sync();  // neither CTA's tensor memory or shared memory is in the partner's use any more
  tc_fence_after();
  if (warp == kSWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  cluster_sync();
}

}  // namespace

cudaError_t launch_verify_kv4_tc(const VerifyArgs& a, int32_t ctas, cudaStream_t stream) {
  static std::atomic<bool> configured[64];  // the smem opt-in, set once per device (setting it twice is harmless)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(verify_kv4_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
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
