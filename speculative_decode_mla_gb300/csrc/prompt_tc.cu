// tcgen05 prompt attention for sm_103a (include/mla_prompt.h).
//
// A unit is up to 256 rows (two lanes of 128) of one sequence; a row is a query and a head, and the heads that share a key
// head lie side by side (pack). A CTA works through units, or, in calls with few of them, through an equal share of all units'
// tiles of 128 keys (a share may begin and end inside a unit; prompt_merge_kernel joins such parts). In calls of many units the
// next one's number comes from cancelling a CTA that has not started (clusterlaunchcontrol), so units go, in index
// order (heads in groups whose keys and values stay in L2; inside a group longest first), to whichever SM is free, with no
// counter in memory. Per tile and lane:
//
//   S = Q K^T   M = 128, N = 128, 12 K-steps: 8 over the head's own dims, 4 over the shared RoPE dims
//   P = 2^((S - m) scale log2 e) as bf16, in S's place in TMEM; the running maximum is kept in the sums' own units and
//       taken away before the scale, so that large scores lose nothing; O is rescaled only when it grows by more than 2^8
//   O += P V    M = 128, N = 128, 8 K-steps, P from TMEM
//
// While one lane's softmax runs, the tensor cores work for the other lane. When no sequence has more than 128 rows (ONE), there
// is one lane with two S buffers: S of the next tile is ready when the softmax has done with this one, and the other lane's
// shared memory makes the ring longer, since such calls wait for keys and values.
//
//   warps 0-3 (, 4-7)  softmax of lane 0 (, 1): a thread a row; they also write O / l out
//   next warp          TMA loads, and the units
//   the one after it   MMA issue
//
// TMEM (512 columns): two S [0, 256), two O [256, 512). Shared memory: Q, 48 KB a lane, and a ring of 16 KB blocks (8, with ONE
// 11) which a tile's keys (three blocks of 64 dims) and values (two blocks of 64 keys) go through in the order
// K(0) V(0) K(1) V(1) ..., each block free for the next load as soon as all MMAs are done with it.
//
// A key that a row does not see has a score of -inf there. Values in tiles that some row of the unit does not see whole
// (on the diagonal, behind the sequence's end) are looked through first: rows behind the end become 0, and
// infinities and NaN become 0 and are added to the rows that do see them when O is written, so that they reach no other row.
//
// Bound by the tensor cores in long prompts: 8192 tokens of 64 heads 0.88 to 0.94 ms, 1.5 PFLOP/s, 80% of a large library product's rate (a tile
// and both lanes take 3014 cycles, the MMAs 2560; the rest are beginnings and ends of units). By memory where few queries meet many keys: 17
// tokens after 16 Ki, 64 heads, 95 to 98 us, 5.6 TB/s. By beginnings and ends of units in batches of short prompts: 24 of 61 to 2048
// tokens, 16 heads, 110 us, 0.74 PFLOP/s. The kernel of two lanes spills 92 bytes a thread, that of one none.
//
// Every wait is bounded (about 2 s, and more for many keys). When one runs out its CTA stops issuing work, drains what is in flight, reports MLA_CHECK_TIMEOUT,
// gives a NaN lse to the rows of its last two units and of those that it had claimed, or had as its share, and not begun, and exits; a
// row that is merged from such a part is NaN. Rows of units before those are as they should be, and other CTAs go on.
#include <atomic>

#include "prompt.cuh"
#include "tc.cuh"

namespace mla {
namespace {

constexpr int kRows = kPromptTile, kKeys = kPromptTile;
constexpr int kBlock = 16384;                 // 128 rows x 64 dims (Q, K) or 64 keys x 128 dims (V), 128B swizzle
constexpr int kQBytes = 3 * kBlock;           // a lane's queries
constexpr int kTileBlocks = 5;
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;
constexpr int kMaxSpecial = 3;                // tiles that some row of a unit does not see whole, and another does in part
constexpr int kUnitWords = 24;
constexpr int kAlone = 4;                     // a thread deals with a sequence of so many row tiles alone, a warp with a longer one

template <bool ONE>
struct Layout {
  static constexpr int lanes = ONE ? 1 : 2, slots = ONE ? 11 : 8;
  static constexpr int load_warp = 4 * lanes, mma_warp = load_warp + 1;
  // Registers: two lanes take 168 a thread at launch with a third warpgroup (loads, MMAs, two warps that only fill it), which hands
  // 80 of its own to the others: 2 x 208 + 88 = 3 x 168.
  static constexpr int threads = ONE ? 32 * (mma_warp + 1) : 384;
  static constexpr int softmax_regs = 208, other_regs = 88;
  static constexpr int ring = lanes * kQBytes, bars = ring + slots * kBlock;
  // barriers: keys and values landed (by tile, mod 4: with ONE, blocks of three tiles may be under way), freed (group
  // 2 t: the keys of tile t, group 2 t + 1: its values; mod 8), ...
  static constexpr int keys = 0 /*4*/, vals = 4 /*4*/, freed = 8 /*8*/, q_full = 16 /*2*/, q_empty = q_full + 2 /*2*/, s = q_empty + 2 /*2*/,
                       p = s + 2 /*[half][buffer]*/, o = p + 4 /*2*/, unit = o + 2 /*2*/, unit_empty = unit + 2 /*2*/, next = unit_empty + 2,
                       drain = next + 1, num_bars = drain + 1;
  static constexpr int bar_bytes = (8 * num_bars + 15) / 16 * 16;
  static constexpr int answer = bars + bar_bytes;              // 16 bytes: the answer to a cancel request
  static constexpr int units = answer + 16;                    // two unit descriptions
  static constexpr int bad = units + 2 * kUnitWords * 4;       // [2][kMaxSpecial][4] words: keys whose values are not all finite
  static constexpr int flags = bad + 2 * kMaxSpecial * 16;     // TMEM address, abort flag
  static constexpr int bytes = flags + 16;
  static_assert(bytes <= 232448 && answer % 16 == 0, "shared memory");
};

#define TMEM_LD32(addr, r)                                                                                              \
  asm volatile(                                                                                                         \
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"  \
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"                                                        \
      : "=r"((r)[0]), "=r"((r)[1]), "=r"((r)[2]), "=r"((r)[3]), "=r"((r)[4]), "=r"((r)[5]), "=r"((r)[6]),               \
        "=r"((r)[7]), "=r"((r)[8]), "=r"((r)[9]), "=r"((r)[10]), "=r"((r)[11]), "=r"((r)[12]), "=r"((r)[13]),           \
        "=r"((r)[14]), "=r"((r)[15]), "=r"((r)[16]), "=r"((r)[17]), "=r"((r)[18]), "=r"((r)[19]), "=r"((r)[20]),        \
        "=r"((r)[21]), "=r"((r)[22]), "=r"((r)[23]), "=r"((r)[24]), "=r"((r)[25]), "=r"((r)[26]), "=r"((r)[27]),        \
        "=r"((r)[28]), "=r"((r)[29]), "=r"((r)[30]), "=r"((r)[31])                                                      \
      : "r"(addr))
#define TMEM_ST32(addr, r)                                                                                              \
  asm volatile(                                                                                                         \
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"   \
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),                                          \
      "r"((r)[0]), "r"((r)[1]), "r"((r)[2]), "r"((r)[3]), "r"((r)[4]), "r"((r)[5]), "r"((r)[6]), "r"((r)[7]),           \
      "r"((r)[8]), "r"((r)[9]), "r"((r)[10]), "r"((r)[11]), "r"((r)[12]), "r"((r)[13]), "r"((r)[14]), "r"((r)[15]),     \
      "r"((r)[16]), "r"((r)[17]), "r"((r)[18]), "r"((r)[19]), "r"((r)[20]), "r"((r)[21]), "r"((r)[22]), "r"((r)[23]),   \
      "r"((r)[24]), "r"((r)[25]), "r"((r)[26]), "r"((r)[27]), "r"((r)[28]), "r"((r)[29]), "r"((r)[30]), "r"((r)[31])    \
      : "memory")

// Instruction descriptor for kind::f16: bf16 A and B, fp32 D, B K-major (0) or MN-major (1).
__host__ __device__ constexpr uint32_t instr_desc(int N, int b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(kRows >> 4) << 24);
}
// Shared-memory descriptors with 128-byte swizzle and 1024 bytes from one group of eight rows to the next, as their low words (the
// address, and for B read MN-major the 8 KB from one block of 64 dims to the next); the high words are all the same.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); }
__device__ __forceinline__ void mma_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 b;\nmov.b64 b, {%2, %5};\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_low), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_smem_a(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 a, b;\nmov.b64 a, {%1, %5};\nmov.b64 b, {%2, %5};\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
// Takes bytes that a barrier was told of and that nobody will load off its phase.
__device__ __forceinline__ void mbar_forget_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.b32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Three-input maximum that is NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 32 bytes, in one piece where the place is aligned to 32.
__device__ __forceinline__ void store32(void* dst, const uint32_t* v, bool whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}
// Four barriers asked together, which takes the time of one: bit i, phase i is over.
__device__ __forceinline__ uint32_t probe4(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, uint32_t b2, uint32_t p2, uint32_t b3, uint32_t p3) {
  uint32_t r0, r1, r2, r3;
  asm volatile(
      "{\n.reg .pred p, q, r, s;\n"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%4], %5;\nmbarrier.test_wait.parity.shared::cta.b64 q, [%6], %7;\n"
      "mbarrier.test_wait.parity.shared::cta.b64 r, [%8], %9;\nmbarrier.test_wait.parity.shared::cta.b64 s, [%10], %11;\n"
      "selp.u32 %0, 1, 0, p;\nselp.u32 %1, 2, 0, q;\nselp.u32 %2, 4, 0, r;\nselp.u32 %3, 8, 0, s;\n}"
      : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
      : "r"(b0), "r"(p0), "r"(b1), "r"(p1), "r"(b2), "r"(p2), "r"(b3), "r"(p3)
      : "memory");
  return r0 | r1 | r2 | r3;
}
// A wait that gives up after so many cycles, or when another role has: false then. (The first probe goes out before the clock is read.)
__device__ __forceinline__ bool wait_until(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, long long limit) {
  if (mbar_test(bar, parity)) return true;
  const long long start = clock64();
  while (true) {
    if (mbar_test(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - start > limit) {
      *abort_flag = 1;
      return false;
    }
  }
}
// A wait of one thread. Its loop is a function where there are two lanes: one at each place would fill the instruction cache. (16 heads
// of 4096 rows and keys: 122.6 us, 123.9 with a loop at each place. Calls of one lane lose 0.3 us by the call's time.)
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, long long limit) {
  return wait_until(bar, parity, abort_flag, limit);
}
template <bool ONE>
__device__ __forceinline__ bool wait_thread(const PromptArgs& a, uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
  return ONE ? wait_until(bar, parity, abort_flag, a.wait_cycles) : mbar_test(bar, parity) || wait_on(bar, parity, abort_flag, a.wait_cycles);
}
// The same of every lane of a warp; the result is uniform across the warp.
__device__ __forceinline__ bool wait_warp(const PromptArgs& a, uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
  return __all_sync(0xffffffffu, wait_until(bar, parity, abort_flag, a.wait_cycles));
}
// A wait for copies and MMAs that are in flight when a thread is done or gives up: bounded by its own clock.
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity) {
  const long long start = clock64();
  while (!mbar_test(bar, parity) && clock64() - start < kTimeoutCycles) {
  }
}

// What every role needs to know of a unit, or of a part of one. Lane r's rows are [row0 + 128 r, row0 + 128 r + 128) of the
// sequence, of which those below `rows` exist; it works on the tiles [t0, t0 + tiles[r]). `special`: the first tile that some row does
// not see whole. `part`: where its result goes in part_o, -1: to out.
struct Unit {
  int32_t live;      // 0: there is no further unit
  int32_t row0, rows, h, g, part;
  PromptSeq s;
  int32_t all;       // tiles of the whole unit
  int32_t t0, special;
  int32_t tiles[2];
};
static_assert(sizeof(Unit) <= kUnitWords * 4, "unit description");

// Row tile `tile` of sequence s, heads of virtual head vh, all tiles.
__device__ __forceinline__ Unit unit_of(const PromptArgs& a, const PromptSeq& s, int tile, int vh) {
  Unit x;
  x.live = 1;
  x.part = -1;
  x.h = vh * a.pack;
  x.g = x.h / a.group;
  x.t0 = x.special = x.tiles[0] = x.tiles[1] = x.row0 = x.rows = x.all = 0;
  x.s = s;
  const int64_t rows = (int64_t)x.s.m << a.pack_log, row0 = (int64_t)tile * a.rows_per_unit;
  if (row0 >= rows) return x;
  x.row0 = (int32_t)row0;
  x.rows = (int32_t)rows;
  x.all = tiles_of(a, x.s, min(rows, row0 + a.rows_per_unit));
  x.special = visible(a, x.s, x.row0 >> a.pack_log) / kKeys;
  return x;
}
// Its tiles [t0, t1).
__device__ __forceinline__ void cut(const PromptArgs& a, Unit& x, int32_t t0, int32_t t1) {
  const int64_t mid = (int64_t)x.row0 + kRows;
  x.t0 = t0;
  x.tiles[0] = x.all ? max(0, min(t1, tiles_of(a, x.s, min((int64_t)x.rows, mid))) - t0) : 0;
  x.tiles[1] = a.rows_per_unit > kRows && x.rows > mid ? t1 - t0 : 0;
}
// Where row i of a unit, or of its part, has its lse.
__device__ __forceinline__ float* lse_at(const PromptArgs& a, const Unit& x, int i) {
  const int at = x.row0 + i;
  return x.part >= 0 ? a.part_lse + (int64_t)x.part * a.rows_per_unit + i
                     : a.lse + (int64_t)(x.s.q0 + (at >> a.pack_log)) * a.H + x.h + (at & (a.pack - 1));
}
// Says of a unit's rows that they were not computed: a NaN lse (and, of parts, NaN rows when they are merged). Rows first, first + step, ...
__device__ __forceinline__ void give_up(const PromptArgs& a, const Unit& x, int first, int step) {
  const int rows = min(a.rows_per_unit, x.rows - x.row0);
#pragma unroll 1
  for (int i = first; i < rows; i += step) *lse_at(a, x, i) = NAN;
}
// Unit number u of a call that is not shared (virtual heads in groups of a.head_group; in a group by row tile, then head), found in
// steps whose reads of memory wait for each other: a step's results are used by the next one, some tiles later.
struct Place {
  int b, tile, vh;          // sequence (-1: none)
  int32_t q0, q1, k0, k1;   // its ends, as they are in memory
};
__device__ __forceinline__ Place place_of(const PromptArgs& a, uint32_t u) {
  const uint32_t full = (uint32_t)a.entries * (uint32_t)a.head_group, group = u / full;  // (all units together are below 2^31)
  const uint32_t heads = min(a.head_group, a.virtual_heads - (int)group * a.head_group);
  const uint32_t rest = u - group * full, e = rest / heads;
  Place at = {};
  at.vh = (int)(group * a.head_group + (rest - e * heads));
  at.tile = (int)((uint32_t)a.entries - 1 - e);
  if (a.listed) {
    const int2 entry = a.list[e];
    at.b = entry.x;
    at.tile = entry.y;
  }
  return at;
}
__device__ __forceinline__ void read_ends(const PromptArgs& a, Place& at) {
  if (at.b < 0) return;
  at.q0 = a.cu_q[at.b];
  at.q1 = a.cu_q[at.b + 1];
  at.k0 = a.cu_k[at.b];
  at.k1 = a.cu_k[at.b + 1];
}
__device__ __forceinline__ Unit unit_at(const PromptArgs& a, const Place& at) {
  PromptSeq s = {0, 0, 0, 0};
  if (at.b >= 0) s = clamp_seq(a, at.q0, at.q1, at.k0, at.k1);
  Unit x = unit_of(a, s, at.tile, at.vh);
  cut(a, x, 0, x.all);
  return x;
}

// What a CTA of a shared call takes.
__device__ __forceinline__ int32_t share_of(const PromptArgs& a, int32_t total) {
  return max(kLeastShare + kUnitCost, total / a.ctas + (total % a.ctas ? 1 : 0));
}
// Cost of row tile t of a sequence, for one virtual head.
__device__ __forceinline__ int32_t entry_cost(const PromptArgs& a, const PromptSeq& s, int32_t t) {
  return cost_of(tiles_of(a, s, min((int64_t)s.m << a.pack_log, ((int64_t)t + 1) * a.rows_per_unit)));
}
// Cost of all n row tiles of a lane's sequence; every lane of the warp calls it. A lane deals with a short sequence alone, the warp with a
// longer one.
__device__ __forceinline__ int32_t sequence_cost(const PromptArgs& a, const PromptSeq& s, int32_t n, int lane) {
  int32_t own = 0;
  if (n <= kAlone)
#pragma unroll 1
    for (int32_t t = 0; t < n; ++t) own += entry_cost(a, s, t);
#pragma unroll 1
  for (uint32_t left = __ballot_sync(0xffffffffu, n > kAlone); left; left &= left - 1) {
    const int l = __ffs(left) - 1;
    PromptSeq o = {0, 0, 0, 0};
    o.m = __shfl_sync(0xffffffffu, s.m, l);
    o.n = __shfl_sync(0xffffffffu, s.n, l);
    const int32_t o_n = __shfl_sync(0xffffffffu, n, l);
    int32_t sum = 0;
#pragma unroll 1
    for (int32_t t = lane; t < o_n; t += 32) sum += entry_cost(a, o, t);
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == l) own = sum;
  }
  return own;
}
// Where in the lanes' work (own each, `before` before them) place w lies: the lane, or -1; what lies before that lane is left in `before`.
__device__ __forceinline__ int lane_at(int32_t own, int32_t w, int32_t& before, int lane) {
  int32_t inc = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t up = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += up;
  }
  const uint32_t past = __ballot_sync(0xffffffffu, before + inc > w);
  const int l = past ? __ffs(past) - 1 : 31;
  before += __shfl_sync(0xffffffffu, past ? inc - own : inc, l);
  return past ? l : -1;
}
// A CTA's way through its share of a shared call: sequences in order, their row tiles in order, the virtual heads of a row tile one
// after the other, each cost_of(its tiles) units of work, of which the last kUnitCost stand for starting and ending it.
struct Walk {
  int32_t w, w_end, offset, share;  // offset: of w in the unit (all work together is below 2^31: mla_prompt_plan)
  int32_t b, tile, num_tiles, head;
  PromptSeq s;
  bool first;
};
// Where share number c begins (every lane of the warp calls it). Every CTA goes through all sequences for itself: such calls have few
// units. (61 single tokens: 58.2 us, 59.6 and one launch more with a kernel before this one that shares out; one sequence alone loses 0.3 us.)
__device__ __forceinline__ Walk walk_from(const PromptArgs& a, int c, int lane) {
  Walk k = {};
  k.first = true;
  k.b = a.B;
  PromptSeq s = {0, 0, 0, 0};
  int32_t n = 0, own = 0, total = 0, before = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {  // all work; then the sequence where the share begins
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      if (pass == 0 || a.B > 32) {
        s.m = s.n = 0;
        if (b0 + lane < a.B) s = load_seq(a, b0 + lane);
        n = units_in(a, (int64_t)s.m << a.pack_log);
        own = sequence_cost(a, s, n, lane);
      }
      if (pass == 0) {
        total += own;
        continue;
      }
      const int l = lane_at(own * a.virtual_heads, k.w, before, lane);
      if (l < 0) continue;
      k.b = b0 + l;
      k.s.q0 = __shfl_sync(0xffffffffu, s.q0, l);
      k.s.m = __shfl_sync(0xffffffffu, s.m, l);
      k.s.k0 = __shfl_sync(0xffffffffu, s.k0, l);
      k.s.n = __shfl_sync(0xffffffffu, s.n, l);
      k.num_tiles = __shfl_sync(0xffffffffu, n, l);
      break;
    }
    if (pass == 0) {
      total = __reduce_add_sync(0xffffffffu, total) * a.virtual_heads;
      k.share = share_of(a, total);
      k.w = (int32_t)min((int64_t)total, (int64_t)c * k.share);
      k.w_end = k.w + min(k.share, total - k.w);
      if (k.w >= k.w_end) return k;
    }
  }
#pragma unroll 1
  for (int32_t t0 = 0; t0 < k.num_tiles; t0 += 32) {
    const int32_t cost = t0 + lane < k.num_tiles ? entry_cost(a, k.s, t0 + lane) : 0;
    const int l = lane_at(cost * a.virtual_heads, k.w, before, lane);
    if (l < 0) continue;
    const int32_t per = __shfl_sync(0xffffffffu, cost, l);
    k.tile = t0 + l;
    k.head = (k.w - before) / per;
    k.offset = k.w - before - k.head * per;
    break;
  }
  return k;
}
// The next part of the share; not live when it is done. The unit that ends with a part of this share, but began before it, is
// the first one, if any: *merge says so.
__device__ __forceinline__ Unit next_part(const PromptArgs& a, Walk& k, int c, PromptMerge* merge) {
  Unit x;
  x.live = 0;
#pragma unroll 1
  while (k.w < k.w_end && k.b < a.B) {
    x = unit_of(a, k.s, k.tile, k.head);
    const int32_t len = max(1, x.all), off = k.offset, take = min(len - off, k.w_end - k.w);
    if (off < len) {
      cut(a, x, off, min(x.all, off + take));
      if (off > 0 || take < len) x.part = 2 * c + (k.first ? 0 : 1);
      if (off > 0 && off + take == len) {
        const int32_t begin = k.w - off;
        merge->first = begin / k.share;
        merge->slot = begin % k.share ? 1 : 0;
        merge->row0 = x.row0;
        merge->rows = min(a.rows_per_unit, x.rows - x.row0);
        merge->q0 = x.s.q0;
        merge->head = x.h;
        merge->live = 1;
      }
    }
    k.first = false;
    // on to the next unit
    k.w += min(len + kUnitCost - off, k.w_end - k.w);
    k.offset = 0;
    if (++k.head == a.virtual_heads) {
      k.head = 0;
      ++k.tile;
    }
#pragma unroll 1
    while (k.tile == k.num_tiles && ++k.b < a.B) {
      k.s = load_seq(a, k.b);
      k.num_tiles = units_in(a, (int64_t)k.s.m << a.pack_log);
      k.tile = 0;
    }
    if (off < len) return x;
    x.live = 0;
  }
  return x;
}

// What a CTA gives up when a wait has run out: the rest of its share; a unit that it has claimed; the units that its roles were told of last,
// which may not be done (the loader waits for all others' end of the one before those). Functions, since code that is hardly ever run costs
// the calls of one lane 1% where it stands in the kernel (64 single tokens of 16 heads: 114.1 us, 115.6 so).
__device__ __noinline__ void give_up_share(const PromptArgs& a, Walk walk, int c) {
  PromptMerge merge;
#pragma unroll 1
  while (true) {
    const Unit x = next_part(a, walk, c, &merge);
    if (!x.live) break;
    give_up(a, x, 0, 1);
  }
}
__device__ __noinline__ void give_up_unit(const PromptArgs& a, Place place) {
  read_ends(a, place);
  give_up(a, unit_at(a, place), 0, 1);
}
__device__ __noinline__ void give_up_last(const PromptArgs& a, const uint32_t* units, int threads) {
  if (threadIdx.x == 0) report(a.dev_status, a.dev_status != nullptr, MLA_CHECK_TIMEOUT);
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const Unit& x = *reinterpret_cast<const Unit*>(units + i * kUnitWords);
    if (x.live) give_up(a, x, threadIdx.x, threads);
  }
}

template <bool ONE>
__global__ void __launch_bounds__(Layout<ONE>::threads, 1)
    prompt_tc_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_kr, const __grid_constant__ CUtensorMap map_v) {
  using L = Layout<ONE>;
  constexpr uint32_t kSlots = L::slots;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const auto bar = [&](int i) { return base + L::bars + 8u * (uint32_t)i; };
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L::flags);
  volatile uint32_t* const abort_flag = tmem_slot + 1;
  const auto unit_slot = [&](int i) { return reinterpret_cast<Unit*>(smem + L::units + i * kUnitWords * 4); };
  uint32_t* const bad = reinterpret_cast<uint32_t*>(smem + L::bad);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) mbar_init(bar(L::freed + i), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(L::keys + i), 1);
      mbar_init(bar(L::vals + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::q_full + i), 1);
      mbar_init(bar(L::q_empty + i), 1);
      mbar_init(bar(L::s + i), 1);
      mbar_init(bar(L::p + i), 4);
      mbar_init(bar(L::p + 2 + i), 4);
      mbar_init(bar(L::o + i), 1);
      mbar_init(bar(L::unit + i), 1);
      mbar_init(bar(L::unit_empty + i), 1 + 4 * L::lanes);
    }
    mbar_init(bar(L::next), 1);
    mbar_init(bar(L::drain), 1);
    *abort_flag = 0;
    unit_slot(0)->live = unit_slot(1)->live = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == L::load_warp && elect_one()) {
    for (const CUtensorMap* map : {&map_q, &map_k, &map_kr, &map_v})
      asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
  }
  if (warp == L::mma_warp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // everything above read no global memory
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (a.shared) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge, which waits for this kernel's end

  const auto fewer_registers = [&] {
    if (!ONE) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::other_regs));
  };
  if (warp == L::load_warp) {
    // ------------------------------------------------------------------------------ loads and units
    fewer_registers();
    Walk walk = {};
    if (a.shared) walk = walk_from(a, blockIdx.x, lane);
    if (elect_one()) {
      uint32_t blocks = 0, q_loads[2] = {0, 0};  // ring blocks and query tiles loaded so far
      uint32_t tiles = 0, freed = 0;             // tiles, and groups of blocks known to be free again
      // The next block of the ring, once the block that was there before is done with.
      const auto load_block = [&](const CUtensorMap* map, int x, int y, int z, int landed, bool value) {
        if (blocks >= kSlots) {
          const uint32_t old = blocks - kSlots, group = 2 * (old / kTileBlocks) + (old % kTileBlocks >= 3);
          for (; freed <= group; ++freed)
            if (!wait_thread<ONE>(a, bar(L::freed + (freed & 7)), (freed >> 3) & 1, abort_flag)) return false;
        }
        const uint32_t dst = base + L::ring + (blocks % kSlots) * kBlock;
        tma_load3(dst, map, x, y, z, bar(landed));
        if (value) tma_load3(dst + kBlock / 2, map, x + 64, y, z, bar(landed));
        ++blocks;
        return true;
      };
      bool next_asked = false;
      uint32_t n_unit = 0, n_asked = 0;
      bool ok = true, more = true;  // more: there is a next unit, at `place`, which no other role has heard of
      Place place = {};
      if (!a.shared) {
        place = place_of(a, blockIdx.x);
        read_ends(a, place);
      }
      const auto take_answer = [&] {
        uint32_t got, id;
        asm volatile(
            "{\n.reg .b128 h;\n.reg .pred p;\n.reg .b64 lo, hi;\n"
            "ld.shared.v2.b64 {lo, hi}, [%2];\nmov.b128 h, {lo, hi};\n"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\nselp.u32 %0, 1, 0, p;\nmov.u32 %1, 0;\n"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n}"
            : "=r"(got), "=r"(id)
            : "r"(base + L::answer)
            : "memory");
        more = got != 0;
        if (more) place = place_of(a, id);
      };
      PromptMerge merge = {};
      while (ok) {
        const int slot = n_unit & 1;
        if (n_unit >= 2 && !wait_thread<ONE>(a, bar(L::unit_empty + slot), ((n_unit >> 1) - 1) & 1, abort_flag)) break;
        Unit x;
        x.live = 0;
        if (a.shared) {
          x = next_part(a, walk, blockIdx.x, &merge);
          if (n_unit == 0) a.merges[blockIdx.x] = merge;
        } else if (more) {
          x = unit_at(a, place);
          more = false;
        }
        // (a unit without rows, where the lengths leave fewer than the call has room for, is passed over)
        const bool none = !a.shared && x.live && x.rows == 0;
        if (!none) {
          *unit_slot(slot) = x;
          mbar_arrive(bar(L::unit + slot));
        }
        if (!x.live) break;
        if (!a.shared) {  // ask for the unit after this one
          mbar_arrive_expect_tx(bar(L::next), 16);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                           base + L::answer),
                       "r"(bar(L::next))
                       : "memory");
          next_asked = true;
        }
        const int n = max(x.tiles[0], x.tiles[1]);
        const auto load_q = [&](int r) {
          if (x.tiles[r] == 0) return true;
          if (q_loads[r] > 0 && !wait_thread<ONE>(a, bar(L::q_empty + r), (q_loads[r] - 1) & 1, abort_flag)) return false;
          const uint32_t full = bar(L::q_full + r);
          mbar_arrive_expect_tx(full, kQBytes);
          for (int i = 0; i < 3; ++i)
            tma_load3(base + r * kQBytes + i * kBlock, &map_q, 64 * i, x.h, x.s.q0 + ((x.row0 + r * kRows) >> a.pack_log), full);
          ++q_loads[r];
          return true;
        };
        for (int j = 0; j < max(n, 2) && ok; ++j) {
          if (j < n) {
            const int at = x.s.k0 + (x.t0 + j) * kKeys, keys = L::keys + (tiles & 3), vals = L::vals + (tiles & 3);
            if (!ONE && j == 0) ok = load_q(0);  // (free before the ring's blocks are)
            if (!ok) break;
            mbar_arrive_expect_tx(bar(keys), 3 * kBlock);
            ok = load_block(&map_k, 0, x.g, at, keys, false) && load_block(&map_k, 64, x.g, at, keys, false) &&
                 load_block(&map_kr, 0, 0, at, keys, false);
            if (ok && j == 0) ok = load_q(ONE ? 0 : 1);
            if (!ok) break;
            mbar_arrive_expect_tx(bar(vals), 2 * kBlock);
            ok = load_block(&map_v, 0, x.g, at, vals, true) && load_block(&map_v, 0, x.g, at + 64, vals, true);
            if (ok) ++tiles;
          }
          if (a.shared || !ok) continue;
          if (j == 0) {
            ok = wait_thread<ONE>(a, bar(L::next), n_asked & 1, abort_flag);
            if (!ok) break;
            ++n_asked;
            next_asked = false;
            take_answer();
          } else if (j == 1 && more) {
            read_ends(a, place);
          }
        }
        if (!none) ++n_unit;
      }
      // What is in flight lands before the CTA ends, also where another role gives up after this one has left.
      if (next_asked) drain_bar(bar(L::next), n_asked & 1);
      const uint32_t begun = blocks - kTileBlocks * tiles;  // blocks of a tile that was not loaded whole
      if (begun > 0) {
        if (begun != 3) mbar_forget_tx(bar((begun < 3 ? L::keys : L::vals) + (tiles & 3)), ((begun < 3 ? 3 : 5) - begun) * kBlock);
        drain_bar(bar(L::keys + (tiles & 3)), (tiles >> 2) & 1);
        if (begun > 3) drain_bar(bar(L::vals + (tiles & 3)), (tiles >> 2) & 1);
      }
      for (uint32_t i = tiles > 2 ? tiles - 3 : 0; i < tiles; ++i) {
        drain_bar(bar(L::keys + (i & 3)), (i >> 2) & 1);
        drain_bar(bar(L::vals + (i & 3)), (i >> 2) & 1);
      }
      for (int r = 0; r < 2; ++r)
        if (q_loads[r]) drain_bar(bar(L::q_full + r), (q_loads[r] - 1) & 1);
      if (*abort_flag) {  // what this CTA was to compute and no other role has heard of
        if (a.shared) {
          give_up_share(a, walk, blockIdx.x);
        } else {
          if (next_asked && mbar_test(bar(L::next), n_asked & 1)) take_answer();
          if (more) give_up_unit(a, place);
        }
      }
    }
    __syncwarp();
  } else if (warp == L::mma_warp) {
    // ------------------------------------------------------------------------------ MMA issue
    // One thread. The tensor cores hold about four MMAs (256 cycles) that have been issued and not begun, and an issue waits for room, so
    // what this thread does between the last MMA of one step and the first of the next has to take less: a probe of a barrier takes
    // 55 cycles (80 for a warp, with its vote), a commit about 50. So the next step's barriers are asked, all together, before the last
    // four MMAs of a step, and O is committed only where nothing later tells the same. (A tile and a lane, all barriers long done, where
    // the MMAs take 1280 cycles: every wait at its place, a warp, 1720; one thread, 1418; with the early probes 1398; and without O's
    // commit the calls of one long prompt are 2% faster than with it and without the probes: 126.5 us against 129.7 at 16 heads of 4096
    // rows and keys, not causal.)
    fewer_registers();
    if (elect_one()) {
      constexpr uint32_t idesc_s = instr_desc(kKeys, 0), idesc_pv = instr_desc(kHeadV, 1);
      uint32_t tiles = 0, p_uses = 0, q_uses = 0;  // (p_uses, q_uses: bit i is the parity of S buffer or lane i)
      uint32_t keys_seen = 0, vals_seen = 0;       // tiles whose keys, values are known to have landed
      uint32_t p_seen = 0;                         // bits of the next step's halves of P that are known to be there
      bool issued = false;
      const auto wait = [&](int b, uint32_t parity) { return wait_thread<ONE>(a, bar(b), parity, abort_flag); };
      const auto block_at = [&](uint32_t tile, int i) { return base + L::ring + (tile * kTileBlocks + i) % kSlots * kBlock; };
      // S buffer s = Q of lane r times the keys of a tile; `ask` asks for what comes next.
      const auto scores = [&](int r, int s, uint32_t tile, bool last, auto ask) {
        if (tile >= keys_seen) {
          if (!wait(L::keys + (tile & 3), (tile >> 2) & 1)) return false;
          keys_seen = tile + 1;
        }
        const uint32_t d = tmem + kColS + 128 * s;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const uint32_t qa = desc_low(base + r * kQBytes + i * kBlock, 16), kb = desc_low(block_at(tile, i), 16);
          if (i == 2) ask();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_smem_a(d, qa + 2 * kk, kb + 2 * kk, idesc_s, i > 0 || kk > 0);
        }
        mma_commit(bar(L::s + s));
        if (last) mma_commit(bar(L::q_empty + r));
        issued = true;
        return true;
      };
      // O of lane r += P (in S buffer s) V of a tile
      const auto values = [&](int r, int s, uint32_t tile, bool begins, bool ends) {
        const uint32_t d = tmem + kColO + 128 * r, w = tmem + kColS + 128 * s;
        if (tile >= vals_seen) {
          if (!wait(L::vals + (tile & 3), (tile >> 2) & 1)) return false;
          vals_seen = tile + 1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t vb = desc_low(block_at(tile, 3 + i), kBlock / 2);
          if (!(p_seen >> i & 1) && !wait(L::p + 2 * i + s, p_uses >> s & 1)) return false;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_tmem_a(d, w + 32 * i + kk * 8, vb + 128 * kk, idesc_pv, !begins || i > 0 || kk > 0);
        }
        p_seen = 0;
        p_uses ^= 1u << s;
        if (ends) mma_commit(bar(L::o + r));  // (with two lanes the lane's next scores tell that the tiles before the last are in)
        issued = true;
        return true;
      };
      // P in S buffer s, the values of tile v and the keys of tile k, as far as they are there. (A barrier may be asked for a phase only
      // when the one before it is over: P's was waited for, the tiles' was four tiles ago.)
      const auto look = [&](int s, uint32_t v, uint32_t k) {
        const uint32_t got = probe4(bar(L::p + s), p_uses >> s & 1, bar(L::p + 2 + s), p_uses >> s & 1, bar(L::vals + (v & 3)), (v >> 2) & 1,
                                    bar(L::keys + (k & 3)), (k >> 2) & 1);
        p_seen = got & 3;
        if ((got & 4) && v == vals_seen) vals_seen = v + 1;
        if ((got & 8) && k == keys_seen) keys_seen = k + 1;
      };
      // Group 2 t is the keys of tile t, group 2 t + 1 its values: done with.
      const auto free_group = [&](uint32_t g) { mma_commit(bar(L::freed + (g & 7))); };
      const auto queries = [&](int r) {
        const bool ok = wait(L::q_full + r, q_uses >> r & 1);
        q_uses ^= 1u << r;
        return ok;
      };
      for (uint32_t n_unit = 0;; ++n_unit) {
        if (!wait(L::unit + (n_unit & 1), (n_unit >> 1) & 1)) break;
        const Unit* const x = unit_slot(n_unit & 1);
        const int live = x->live, n0 = x->tiles[0], n1 = x->tiles[1], n = max(n0, n1);
        mbar_arrive(bar(L::unit_empty + (n_unit & 1)));
        if (!live) break;
        bool ok = true;
        if (ONE) {  // tiles take the S buffers in turn, across units too
#pragma unroll 1
          for (int j = -2; j < n && ok; ++j) {
            const uint32_t here = tiles + j;
            if (j >= 0) {
              ok = values(0, here & 1, here, j == 0, true);
              if (ok) free_group(2 * here + 1);
            }
            if (ok && j + 2 < n) {
              if (j == -2) ok = queries(0);
              ok = ok && scores(0, here & 1, here + 2, j + 3 == n, [&] {
                if (j >= -1) look((here + 1) & 1, here + 1, here + 3);
              });
              if (ok) free_group(2 * (here + 2));
            }
          }
        } else {
#pragma unroll 1
          for (int j = -1; j < n && ok; ++j) {
            const uint32_t here = tiles + j;
            // (one body for both lanes: at 83 to 93% hits the instruction cache is what every unit's beginning and end wait for. 24
            // sequences of 61 to 2048 rows: 113 us, with a body for each lane 117)
#pragma unroll 1
            for (int r = 0; r < 2; ++r) {
              const int of_lane = r ? n1 : n0;
              if (ok && j >= 0 && j < of_lane) ok = values(r, r, here, j == 0, j + 1 == of_lane);
              if (ok && j >= 0 && r == 1) free_group(2 * here + 1);
              if (ok && j + 1 < of_lane) {
                if (j < 0) ok = queries(r);
                ok = ok && scores(r, r, here + 1, j + 2 == of_lane, [&] {
                  // the step after this one: lane 1's with this tile, or lane 0's with the next
                  if (r == 0 ? j >= 0 && j < n1 : j + 1 < n0) look(r ^ 1, here + r, here + r + 1);
                });
              }
            }
            if (ok && j + 1 < n) free_group(2 * (here + 1));
          }
        }
        if (!ok) break;
        tiles += n;
      }
      if (issued) {  // (also where another role gives up after this one has left)
        mma_commit(bar(L::drain));
        drain_bar(bar(L::drain), 0);
      }
    }
    __syncwarp();
  } else if (warp < L::load_warp) {
    // ------------------------------------------------------------------------------ softmax and output
    if (!ONE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::softmax_regs));
    const int r = warp >> 2, in_warp = (warp & 3) * 32, row = in_warp + lane;  // lane of the unit, row of the lane
    const uint32_t lanes = (uint32_t)in_warp << 16, tO = tmem + lanes + kColO + 128 * r;
    uint32_t tiles = 0, tile_uses = 0, units_done = 0;  // tiles of the units before; tiles, and units with any, of this lane so far
    bool ok = true;
    for (uint32_t n_unit = 0; ok; ++n_unit) {
      const int slot = n_unit & 1;
      if (!wait_warp(a, bar(L::unit + slot), (n_unit >> 1) & 1, abort_flag)) break;
      const Unit& x = *unit_slot(slot);
      if (!x.live) break;
      const int n = r ? x.tiles[1] : x.tiles[0], unit_tiles = max(x.tiles[0], x.tiles[1]), other = r ? x.tiles[0] : x.tiles[1];
      const int at = x.row0 + r * kRows + row;  // this thread's row
      const bool real = at < x.rows;
      const int32_t vis = real ? visible(a, x.s, at >> a.pack_log) : 0;
      const int t0 = x.t0, special = x.special;
      float m = -INFINITY;
      float l = 0.f, l_low = 0.f;
      for (int j = 0; j < n; ++j) {
        const int buf = ONE ? (int)(tile_uses & 1) : r, tile = t0 + j;
        const uint32_t tS = tmem + lanes + kColS + 128 * buf;
        const auto scores_there = [&] { return wait_warp(a, bar(L::s + buf), (ONE ? tile_uses >> 1 : tile_uses) & 1, abort_flag); };
        if (tile >= special && (r == 0 || j >= other)) {
          // the first lane that uses the tile looks through its values: thread `row` has key `row`
          // (A barrier may be asked for a phase only when the one before it is over: here that of four tiles ago, whose block the tile
          // after it has taken by now.)
          const uint32_t here = tiles + j, block = kTileBlocks * here + 3 + (row >> 6);
          if ((j == 0 && !scores_there()) || !wait_warp(a, bar(L::vals + (here & 3)), (here >> 2) & 1, abort_flag)) {
            ok = false;
            break;
          }
          uint4* const values = reinterpret_cast<uint4*>(smem + L::ring + (block % kSlots) * kBlock + (row & 63) * 128);
          const auto piece = [&](int c) { return values + (c >> 3) * (kBlock / 32) + ((c + row) & 7); };
          const bool behind = (int64_t)tile * kKeys + row >= x.s.n;
          uint32_t top = 0;  // bits 15 and 31: some exponent is all ones
#pragma unroll 4
          for (int c = 0; c < 16; ++c) {
            const uint4 d = *piece(c);
            top |= ((d.x & 0x7f807f80u) + 0x00800080u) | ((d.y & 0x7f807f80u) + 0x00800080u) | ((d.z & 0x7f807f80u) + 0x00800080u) |
                   ((d.w & 0x7f807f80u) + 0x00800080u);
          }
          const bool odd = !behind && (top & 0x80008000u);
          const uint32_t found = __ballot_sync(0xffffffffu, odd);
          if (lane == 0) bad[(slot * kMaxSpecial + (tile - special)) * 4 + (warp & 3)] = found;
          if (behind || odd) {
#pragma unroll 1
            for (int c = 0; c < 16; ++c) {
              const auto keep = [&](uint32_t w) { return behind ? 0u : w & ~__vcmpeq2(w & 0x7f807f80u, 0x7f807f80u); };
              const uint4 d = *piece(c);
              *piece(c) = make_uint4(keep(d.x), keep(d.y), keep(d.z), keep(d.w));
            }
          }
          fence_proxy_async();
        }
        if (!scores_there()) {
          ok = false;
          break;
        }
        tc_fence_after();
        float p[kKeys];
        {
          uint32_t* u = reinterpret_cast<uint32_t*>(p);
          TMEM_LD32(tS, u);
          TMEM_LD32(tS + 32, u + 32);
          TMEM_LD32(tS + 64, u + 64);
          TMEM_LD32(tS + 96, u + 96);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < kKeys; ++k) asm volatile("" : "+f"(p[k]));
        }
        if (tile >= special) {
          const int64_t left = (int64_t)vis - (int64_t)tile * kKeys;
          const int seen = (int)(left < 0 ? 0 : left > kKeys ? kKeys : left);
          if (__any_sync(0xffffffffu, seen < kKeys)) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {  // (by bits of a word: one instruction sets seven predicates)
              const int in = seen - 32 * c;
              const uint32_t bits = in >= 32 ? 0xffffffffu : in <= 0 ? 0u : (1u << in) - 1u;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(bits >> k & 1u)) p[32 * c + k] = -INFINITY;
            }
          }
        }
        float top;  // NaN if a score is, so that the row becomes NaN
        {
          float t[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            t[c] = max3_nan(p[c], p[8 + c], p[16 + c]);
#pragma unroll
            for (int k = 24; k + 8 < kKeys; k += 16) t[c] = max3_nan(t[c], p[k + c], p[k + 8 + c]);
            t[c] = max3_nan(t[c], p[120 + c], p[120 + c]);
          }
          top = max3_nan(max3_nan(t[0], t[1], t[2]), max3_nan(t[3], t[4], t[5]), max3_nan(t[6], t[7], t[7]));
        }
        const bool grows = (top - m) * a.scale_log2 > 8.f || top != top;
        if (__any_sync(0xffffffffu, grows)) {
          const float keep = grows ? ex2((m - top) * a.scale_log2) : 1.f;
          m = grows ? top : m;
          l *= keep;
          l_low *= keep;
          if (j > 0) {
            // (with two lanes these scores were issued after the product before, so that it is over)
            if (ONE && !wait_warp(a, bar(L::o + r), (tile_uses - 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              TMEM_LD16(tO + 16 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
              TMEM_ST16(tO + 16 * c, o);
            }
          }
        }
        // (an infinite score: all weights NaN)
        const float ref = m == -INFINITY ? 0.f : m == INFINITY ? NAN : m;
        float ref_log2 = ref * a.scale_log2;
        // One fma a weight, its addend the rounded maximum: where that is large its rounding error (2^-24 of it) would be one of
        // the exponent, so there the maximum is taken away first. At 2^10 the two differ by 2^-14, less than the scores' own rounding.
        if (__any_sync(0xffffffffu, !(fabsf(ref_log2) <= 1024.f))) {
#pragma unroll
          for (int k = 0; k < kKeys; k += 2) {
            const float2 s = add2(make_float2(p[k], p[k + 1]), make_float2(-ref, -ref));
            p[k] = s.x;
            p[k + 1] = s.y;
          }
          ref_log2 = 0.f;
        }
        const float2 scale2 = make_float2(a.scale_log2, a.scale_log2), off2 = make_float2(-ref_log2, -ref_log2);
        // The tile's sums begin with its own first weights, not with zeros or the sum so far. (Two registers more here and the compiler
        // spills in the loop: 24 sequences of 61 to 2048 rows 110 us so, 113 from zeros, 122 with a sum of two numbers that needs no order.)
        float2 sum[2];
        const auto announce = [&](int half) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::p + 2 * half + buf));
        };
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t w[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            float2 v = fma2(make_float2(p[64 * half + 2 * k], p[64 * half + 2 * k + 1]), scale2, off2);
            v.x = ex2(v.x);
            v.y = ex2(v.y);
            sum[k & 1] = half == 0 && k < 2 ? v : add2(sum[k & 1], v);
            // (bf16 as the values are, which an MMA's two operands have to share: 2^-8 of a weight at most. fp16 weights would take values
            // in fp16, which has not their range. The sum takes them unrounded, so that the roundings do not add up in it.)
            w[k] = pack_bf16(v.x, v.y);
          }
          TMEM_ST32(tS + 32 * half, w);
          // With two S buffers the product before the last may not be over when the last one's weights are there. It has to be before
          // these are announced: afterwards the parity could not tell whether one more, two more or none has ended.
          if (ONE && half == 1 && j == n - 1 && j > 0) ok = wait_warp(a, bar(L::o + r), (tile_uses - 1) & 1, abort_flag);
          announce(half);
        }
        if (!ok) break;
        sum[0] = add2(sum[0], sum[1]);
        add_keeping(l, l_low, sum[0].x + sum[0].y);
        ++tile_uses;
      }
      // the last product of this lane, then O / l
      if (ok && n > 0) ok = wait_warp(a, bar(L::o + r), (ONE ? tile_uses - 1 : units_done) & 1, abort_flag);
      units_done += n > 0;
      const int64_t rh = (int64_t)(x.s.q0 + (at >> a.pack_log)) * a.H + x.h + (at & (a.pack - 1));
      const int64_t part = (int64_t)x.part * a.rows_per_unit + r * kRows + row;
      if (!ok) break;
      tc_fence_after();
      const float sum = l + l_low, inv = sum == 0.f ? 0.f : 1.f / sum;
      if (real) *(x.part >= 0 ? a.part_lse + part : a.lse + rh) = sum == 0.f ? -INFINITY : m * a.scale + __logf(sum);
      if (x.part >= 0 || a.out_f32) {
        float* const dst = x.part >= 0 ? a.part_o + part * kHeadV : static_cast<float*>(a.out) + rh * kHeadV;
#pragma unroll 1
        for (int c = 0; c < kHeadV; c += 16) {
          uint32_t o[16];
          if (n > 0) {
            TMEM_LD16(tO + c, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = n > 0 ? __float_as_uint(__uint_as_float(o[k]) * inv) : 0u;
          if (real) {
            store32(dst + c, o, x.part >= 0 || a.out_32);
            store32(dst + c + 8, o + 8, x.part >= 0 || a.out_32);
          }
        }
      } else {
        __nv_bfloat16* const dst = static_cast<__nv_bfloat16*>(a.out) + rh * kHeadV;
#pragma unroll 1
        for (int c = 0; c < kHeadV; c += 32) {
          uint32_t o[32], w[16];
          if (n > 0) {
            TMEM_LD32(tO + c, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) w[k] = n > 0 ? pack_bf16(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv) : 0u;
          if (real) {
            store32(dst + c, w, a.out_32);
            store32(dst + c + 16, w + 8, a.out_32);
          }
        }
      }
      // the keys among this lane's tiles whose values are not all finite (the other lane's tiles may not have been looked through)
      const int specials = max(0, t0 + n - max(t0, special));
      const uint32_t* const odd_at = bad + (slot * kMaxSpecial + max(t0 - special, 0)) * 4;
      uint32_t odd = 0;
#pragma unroll 1
      for (int k = 0; k < specials; ++k) {
        const uint4 of_tile = reinterpret_cast<const uint4*>(odd_at)[k];
        odd |= of_tile.x | of_tile.y | of_tile.z | of_tile.w;
      }
      if (odd && real) {
#pragma unroll 1
        for (int t = 0; t < specials * kKeys; ++t) {
          const int64_t key = (int64_t)max(t0, special) * kKeys + t;
          if (!(odd_at[t >> 5] >> (t & 31) & 1) || key >= vis) continue;
          const __nv_bfloat16* const v = a.v + (x.s.k0 + key) * a.v_ts + x.g * a.v_hs;
#pragma unroll 1
          for (int d = 0; d < kHeadV; ++d) {
            const float f = __bfloat162float(v[d]);
            if (isfinite(f)) continue;
            if (x.part >= 0) a.part_o[part * kHeadV + d] += f;
            else if (a.out_f32) static_cast<float*>(a.out)[rh * kHeadV + d] += f;
            else static_cast<__nv_bfloat16*>(a.out)[rh * kHeadV + d] = __float2bfloat16_rn(__bfloat162float(static_cast<__nv_bfloat16*>(a.out)[rh * kHeadV + d]) + f);
          }
        }
      }
      tiles += unit_tiles;
      tc_fence_before();  // (the reads of O are done before the next unit's first P is announced)
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::unit_empty + slot));
    }
    __syncwarp();
  } else {
    fewer_registers();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_flag) give_up_last(a, reinterpret_cast<const uint32_t*>(unit_slot(0)), L::threads);
  if (warp == L::mma_warp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// The (sequence, row tile) entries of a batch, by one CTA.
constexpr int kListThreads = 1024, kBins = 2048;

// Calls use(sequence, row tile, tiles of keys) for every entry.
template <class Use>
__device__ __forceinline__ void each_entry(const PromptArgs& a, Use use) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int b0 = threadIdx.x - lane; b0 < a.B; b0 += kListThreads) {
    PromptSeq s = {0, 0, 0, 0};
    if (b0 + lane < a.B) s = load_seq(a, b0 + lane);
    const int64_t rows = (int64_t)s.m << a.pack_log;
    const int32_t n = units_in(a, rows);
    if (n <= kAlone)
#pragma unroll 1
      for (int32_t t = 0; t < n; ++t) use(b0 + lane, t, tiles_of(a, s, min(rows, ((int64_t)t + 1) * a.rows_per_unit)));
#pragma unroll 1
    for (uint32_t left = __ballot_sync(0xffffffffu, n > kAlone); left; left &= left - 1) {
      const int l = __ffs(left) - 1;
      PromptSeq o;
      o.q0 = o.k0 = 0;
      o.m = __shfl_sync(0xffffffffu, s.m, l);
      o.n = __shfl_sync(0xffffffffu, s.n, l);
      const int64_t o_rows = (int64_t)o.m << a.pack_log;
      const int32_t o_n = units_in(a, o_rows);
#pragma unroll 1
      for (int32_t t = lane; t < o_n; t += 32) use(b0 + l, t, tiles_of(a, o, min(o_rows, ((int64_t)t + 1) * a.rows_per_unit)));
    }
  }
}
// Exclusive prefix sum over the block's threads, and the sum of all (sums: 32 numbers of shared memory).
template <class T>
__device__ __forceinline__ T block_scan(T v, T* sums, T& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  T inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T up = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += up;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    T x = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const T up = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += up;
    }
    sums[lane] = x;
  }
  __syncthreads();
  all = sums[31];
  return inc - v + (warp ? sums[warp - 1] : 0);
}

// Longest first: a counting sort by tiles of keys.
__global__ void __launch_bounds__(kListThreads) prompt_list_kernel(const PromptArgs a) {
  __shared__ int32_t bins[kBins];
  __shared__ int32_t sums[32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the attention, which sets itself up and waits for this kernel's end
  const int64_t most = ((int64_t)a.max_k + kKeys - 1) / kKeys;
  int shift = 0;
  while ((most >> shift) >= kBins) ++shift;
#pragma unroll 1
  for (int i = threadIdx.x; i < kBins; i += kListThreads) bins[i] = 0;
  __syncthreads();
  each_entry(a, [&](int, int, int32_t tiles) { atomicAdd(&bins[kBins - 1 - (tiles >> shift)], 1); });
  __syncthreads();
  const int32_t c0 = bins[2 * threadIdx.x], c1 = bins[2 * threadIdx.x + 1];
  int32_t all;
  const int32_t before = block_scan(c0 + c1, sums, all);
  bins[2 * threadIdx.x] = before;
  bins[2 * threadIdx.x + 1] = before + c0;
  __syncthreads();
  each_entry(a, [&](int b, int t, int32_t tiles) {
    const int32_t at = atomicAdd(&bins[kBins - 1 - (tiles >> shift)], 1);
    if (at < a.entries) a.list[at] = make_int2(b, t);
  });
#pragma unroll 1
  for (int64_t i = all + threadIdx.x; i < a.entries; i += kListThreads) a.list[i] = make_int2(-1, 0);
}
static_assert(kBins == 2 * kListThreads, "two bins a thread");

bool encode(EncodeTiledFn enc, CUtensorMap* map, const void* p, int64_t dims, int64_t heads, int64_t head_stride, int64_t rows,
            int64_t row_stride, int box_heads, int box_rows) {
  // (a dim of one element may have any stride in the caller's tensor)
  const cuuint64_t size[3] = {(cuuint64_t)dims, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t stride[2] = {(cuuint64_t)(heads > 1 ? head_stride : dims) * 2, (cuuint64_t)(rows > 1 ? row_stride : dims) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), size, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool ONE>
cudaError_t launch(const PromptArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& kr, const CUtensorMap& v,
                   cudaStream_t stream) {
  using L = Layout<ONE>;
  // once a device (a racing second time does no harm)
  static std::atomic<bool> set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  if (dev < 0 || dev >= 64 || !set[dev].load(std::memory_order_relaxed)) {
    const cudaError_t e = cudaFuncSetAttribute(prompt_tc_kernel<ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) set[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.ctas);
  cfg.blockDim = dim3(L::threads);
  cfg.dynamicSmemBytes = L::bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_tc_kernel<ONE>, a, q, k, kr, v);
}

}  // namespace

cudaError_t launch_prompt_tc(const PromptArgs& a, cudaStream_t stream) {
  EncodeTiledFn enc = tensor_map_encoder();
  CUtensorMap q, k, kr, v;
  const int64_t hk = a.H / a.group;
  // without keys nothing is loaded through these three: the queries' tensor stands in for them
  const bool keys = a.num_k > 0;
  if (!enc || !encode(enc, &q, a.q, kHeadQ, a.H, a.q_hs, a.num_q, a.q_ts, a.pack, kRows / a.pack) ||
      !(keys ? encode(enc, &k, a.k, kNope, hk, a.k_hs, a.num_k, a.k_ts, 1, kKeys) : (k = q, true)) ||
      !(keys ? encode(enc, &kr, a.kr, kDRope, 1, 0, a.num_k, a.kr_ts, 1, kKeys) : (kr = q, true)) ||
      !(keys ? encode(enc, &v, a.v, kHeadV, hk, a.v_hs, a.num_k, a.v_ts, 1, kKeys / 2) : (v = q, true)))
    return cudaErrorInvalidValue;
  if (a.listed) {
    prompt_list_kernel<<<1, kListThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return a.rows_per_unit > kRows ? launch<false>(a, q, k, kr, v, stream) : launch<true>(a, q, k, kr, v, stream);
}

}  // namespace mla
