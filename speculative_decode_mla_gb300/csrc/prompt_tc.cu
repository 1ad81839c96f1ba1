// tcgen05 prompt attention for sm_103a (include/mla_prompt.h).
//
// A unit is up to 256 query rows (two lanes of 128) of one head and a part of the keys that they see. A CTA works
// through units; the next one's number comes from cancelling a CTA that has not started (clusterlaunchcontrol),
// so units go, in index order (heads in groups whose keys and values stay in L2; inside a group longest first),
// to whichever SM is free, with no counter in memory. Per tile of 128 keys and lane:
//
//   S = Q K^T   M = 128, N = 128, 12 K-steps: 8 over the head's own dims, 4 over the shared RoPE dims
//   P = 2^((S - m) scale log2 e) as bf16, in S's place in TMEM; the running maximum is kept in the sums' own units and
//       taken away before the scale, so that large scores lose nothing; O is rescaled only when it grows by more than 2^8
//   O += P V    M = 128, N = 128, 8 K-steps, P from TMEM
//
// While one lane's softmax runs, the tensor cores work for the other lane.
//
//   warps 0-3, 4-7  softmax of lane 0, 1: a thread a row; they also write O / l out
//   warp 8          TMA loads, and the units
//   warp 9          MMA issue, one thread
//
// TMEM (512 columns): S of lane 0, 1 [0, 256), O of lane 0, 1 [256, 512). Shared memory: Q 96 KB, and a ring of eight
// 16 KB blocks which a tile's keys (three blocks of 64 dims) and values (two blocks of 64 keys) go through in the order
// of their use, K(0) V(0) K(1) V(1) ..., each block free for the next load as soon as both lanes' MMAs are done with it.
//
// A key that a row does not see has a score of -inf there. Values in tiles that some row of the unit does not see whole
// (on the diagonal, behind the sequence's end) are looked through first: rows behind the end become 0, and
// infinities and NaN become 0 and are added to the rows that do see them when O is written, so that they reach no other row.
//
// Every wait is bounded (about 2 s). On a timeout the kernel stops issuing work, drains what is in flight, reports
// MLA_CHECK_TIMEOUT, gives its rows a NaN lse and exits.
#include "prompt.cuh"
#include "tc.cuh"

namespace mla {
namespace {

constexpr int kRows = kPromptTile, kKeys = kPromptTile;
constexpr int kBlock = 16384;                 // 128 rows x 64 dims (Q, K) or 64 keys x 128 dims (V), 128B swizzle
constexpr int kQBytes = 3 * kBlock;           // a lane's queries
constexpr int kSlots = 8;
constexpr int kTileBlocks = 5;
constexpr int kSmemQ = 0;
constexpr int kSmemRing = 2 * kQBytes;
constexpr int kSmemBar = kSmemRing + kSlots * kBlock;
constexpr int kThreads = 320;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;

constexpr int kBarFull = 0, kBarEmpty = kSlots, kBarQFull = 2 * kSlots /*2*/, kBarQEmpty = kBarQFull + 2 /*2*/,
              kBarS = kBarQEmpty + 2 /*2*/, kBarP = kBarS + 2 /*2*/, kBarO = kBarP + 2 /*2*/, kBarUnit = kBarO + 2 /*2*/,
              kBarUnitEmpty = kBarUnit + 2 /*2*/, kBarNext = kBarUnitEmpty + 2, kBarDrain = kBarNext + 1, kNumBars = kBarDrain + 1;
constexpr int kSmemNext = kSmemBar + 512;     // 16 bytes: the answer to a cancel request
constexpr int kSmemUnit = kSmemNext + 16;     // two unit descriptions
constexpr int kUnitWords = 24;
constexpr int kSmemBad = kSmemUnit + 2 * kUnitWords * 4;  // [2][kMaxSpecial][4] words: keys whose values are not all finite
constexpr int kMaxSpecial = 3;
constexpr int kSmemFlags = kSmemBad + 2 * kMaxSpecial * 16;  // TMEM address, abort flag
constexpr int kSmemBytes = kSmemFlags + 16 + 1024;
static_assert(8 * kNumBars <= 512 && kSmemBytes <= 232448, "shared memory");

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
__device__ __forceinline__ void mma_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_smem_a(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
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
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 ra, rb, rd;\nmov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %5};\nmul.rn.f32x2 rd, ra, rb;\nmov.b64 {%0, %1}, rd;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// A wait after an abort, for copies and MMAs that are in flight: bounded by its own clock.
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity) {
  const long long start = clock64();
  while (!mbar_test(bar, parity) && clock64() - start < kTimeoutCycles) {
  }
}

// What every role needs to know of a unit. Lane r's rows are [row0 + 128 r, row0 + 128 r + 128) of the sequence, of which
// those below m exist; it works on the tiles [t0, t0 + tiles[r]). `special`: the first tile that some row does not see whole.
struct Unit {
  int32_t live;      // 0: there is no further unit
  int32_t row0, h, g, split;
  PromptSeq s;
  int32_t t0, special;
  int32_t tiles[2];
};
static_assert(sizeof(Unit) <= kUnitWords * 4, "unit description");

// Unit number u (heads in groups of a.head_group; in a group by row tile, then part, then head).
__device__ __forceinline__ Unit unit_at(const PromptArgs& a, int64_t u) {
  Unit x;
  const int64_t full = a.entries * a.splits * a.head_group, group = u / full;
  const int heads = min(a.head_group, a.H - (int)group * a.head_group);
  const int64_t rest = u - group * full, per = (int64_t)a.splits * heads, e = rest / per;
  const int in = (int)(rest - e * per);
  x.split = in / heads;
  x.h = (int)group * a.head_group + in % heads;
  x.g = x.h / a.group;
  x.live = 1;
  x.t0 = x.special = x.tiles[0] = x.tiles[1] = x.row0 = 0;
  int b = 0, tile = (int)(a.entries - 1 - e);
  if (a.listed) {
    const int2 at = a.list[e];
    b = at.x;
    tile = at.y;
  }
  if (b < 0) {
    x.s.q0 = x.s.m = x.s.k0 = x.s.n = 0;
    return x;
  }
  x.s = load_seq(a, b);
  x.row0 = tile * a.rows_per_unit;
  if (x.row0 >= x.s.m) {
    x.s.m = 0;
    return x;
  }
  const int last = min(x.s.m, x.row0 + a.rows_per_unit) - 1;
  const auto tiles_of = [&](int row) { return (int)(((int64_t)visible(a, x.s, row) + kKeys - 1) / kKeys); };
  int32_t t1;
  part_of(a, tiles_of(last), x.split, x.t0, t1);
  x.tiles[0] = max(0, min(t1, tiles_of(min(last, x.row0 + kRows - 1))) - x.t0);
  x.tiles[1] = last - x.row0 >= kRows ? max(0, t1 - x.t0) : 0;
  x.special = visible(a, x.s, x.row0) / kKeys;
  return x;
}

__global__ void __launch_bounds__(kThreads, 1)
    prompt_tc_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_kr, const __grid_constant__ CUtensorMap map_v) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw), base = (raw_addr + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw_addr);
  const auto bar = [&](int i) { return base + kSmemBar + 8u * (uint32_t)i; };
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + kSmemFlags);
  volatile uint32_t* const abort_flag = tmem_slot + 1;
  Unit* const units = reinterpret_cast<Unit*>(smem + kSmemUnit);
  const auto unit_slot = [&](int i) { return reinterpret_cast<Unit*>(smem + kSmemUnit + i * kUnitWords * 4); };
  (void)units;
  uint32_t* const bad = reinterpret_cast<uint32_t*>(smem + kSmemBad);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar(kBarFull + i), 1);
      mbar_init(bar(kBarEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarQFull + i), 1);
      mbar_init(bar(kBarQEmpty + i), 1);
      mbar_init(bar(kBarS + i), 1);
      mbar_init(bar(kBarP + i), 4);
      mbar_init(bar(kBarO + i), 1);
      mbar_init(bar(kBarUnit + i), 1);
      mbar_init(bar(kBarUnitEmpty + i), 9);
    }
    mbar_init(bar(kBarNext), 1);
    mbar_init(bar(kBarDrain), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
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

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------------------------ loads and units
    if (elect_one()) {
      uint32_t blocks = 0, q_loads[2] = {0, 0};  // ring blocks and query tiles loaded so far
      const auto load_block = [&](const CUtensorMap* map, int x, int y, int z, bool value) {
        const uint32_t slot = blocks % kSlots, use = blocks / kSlots;
        if (use > 0 && !wait_bar(bar(kBarEmpty + slot), (use - 1) & 1, abort_flag)) return false;
        const uint32_t dst = base + kSmemRing + slot * kBlock, full = bar(kBarFull + slot);
        mbar_arrive_expect_tx(full, kBlock);
        tma_load3(dst, map, x, y, z, full);
        if (value) tma_load3(dst + kBlock / 2, map, x + 64, y, z, full);
        ++blocks;
        return true;
      };
      bool next_asked = false;
      uint32_t n_unit = 0;
      int64_t u = blockIdx.x;
      bool ok = true;
      while (ok) {
        const int slot = n_unit & 1;
        if (n_unit >= 2 && !wait_bar(bar(kBarUnitEmpty + slot), ((n_unit >> 1) - 1) & 1, abort_flag)) break;
        Unit x;
        if (u >= 0) x = unit_at(a, u);
        else x.live = 0;
        *unit_slot(slot) = x;
        mbar_arrive(bar(kBarUnit + slot));
        if (!x.live) break;
        // ask for the unit after this one
        mbar_arrive_expect_tx(bar(kBarNext), 16);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                         base + kSmemNext),
                     "r"(bar(kBarNext))
                     : "memory");
        next_asked = true;
        const int n = max(x.tiles[0], x.tiles[1]);
        const auto load_q = [&](int r) {
          if (x.tiles[r] == 0) return true;
          if (q_loads[r] > 0 && !wait_bar(bar(kBarQEmpty + r), (q_loads[r] - 1) & 1, abort_flag)) return false;
          const uint32_t full = bar(kBarQFull + r);
          mbar_arrive_expect_tx(full, kQBytes);
          for (int i = 0; i < 3; ++i)
            tma_load3(base + kSmemQ + r * kQBytes + i * kBlock, &map_q, 64 * i, x.h, x.s.q0 + x.row0 + r * kRows, full);
          ++q_loads[r];
          return true;
        };
        for (int j = 0; j < n && ok; ++j) {
          const int at = x.s.k0 + (x.t0 + j) * kKeys;
          ok = load_block(&map_k, 0, x.g, at, false) && load_block(&map_k, 64, x.g, at, false) && load_block(&map_kr, 0, 0, at, false);
          if (ok && j == 0) ok = load_q(0) && load_q(1);
          ok = ok && load_block(&map_v, 0, x.g, at, true) && load_block(&map_v, 0, x.g, at + 64, true);
        }
        if (!ok || !wait_bar(bar(kBarNext), n_unit & 1, abort_flag)) break;
        next_asked = false;
        uint32_t got, id;
        asm volatile(
            "{\n.reg .b128 h;\n.reg .pred p;\n.reg .b64 lo, hi;\n"
            "ld.shared.v2.b64 {lo, hi}, [%2];\nmov.b128 h, {lo, hi};\n"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\nselp.u32 %0, 1, 0, p;\nmov.u32 %1, 0;\n"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n}"
            : "=r"(got), "=r"(id)
            : "r"(base + kSmemNext)
            : "memory");
        u = got ? (int64_t)id : -1;
        ++n_unit;
      }
      if (*abort_flag) {  // what is in flight lands before the CTA ends
        if (next_asked) drain_bar(bar(kBarNext), n_unit & 1);
        for (uint32_t i = blocks > kSlots ? blocks - kSlots : 0; i < blocks; ++i) drain_bar(bar(kBarFull + i % kSlots), (i / kSlots) & 1);
        for (int r = 0; r < 2; ++r)
          if (q_loads[r]) drain_bar(bar(kBarQFull + r), (q_loads[r] - 1) & 1);
        report(a.dev_status, a.dev_status != nullptr, MLA_CHECK_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------------------ MMA issue
    if (elect_one()) {
      constexpr uint32_t idesc_s = instr_desc(kKeys, 0), idesc_pv = instr_desc(kHeadV, 1);
      uint32_t blocks = 0, p_uses[2] = {0, 0}, q_uses[2] = {0, 0};
      bool issued = false;
      const auto landed = [&](uint32_t i) { return wait_bar(bar(kBarFull + i % kSlots), (i / kSlots) & 1, abort_flag); };
      const auto block_at = [&](uint32_t i) { return base + kSmemRing + (i % kSlots) * kBlock; };
      // S of lane r over the tile whose first block is `first`
      const auto scores = [&](int r, uint32_t first, bool last) {
        for (int i = 0; i < 3; ++i) {
          if (!landed(first + i)) return false;
          const uint32_t qa = base + kSmemQ + r * kQBytes + i * kBlock, kb = block_at(first + i);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_smem_a(tmem + kColS + 128 * r, smem_desc(qa + kk * 32, 16, 1024), smem_desc(kb + kk * 32, 16, 1024), idesc_s,
                       i > 0 || kk > 0);
        }
        issued = true;
        mma_commit(bar(kBarS + r));
        if (last) mma_commit(bar(kBarQEmpty + r));
        return true;
      };
      // O of lane r += P V
      const auto values = [&](int r, uint32_t first, bool begins) {
        if (!wait_bar(bar(kBarP + r), p_uses[r] & 1, abort_flag)) return false;
        ++p_uses[r];
        tc_fence_after();
        for (int i = 0; i < 2; ++i) {
          if (!landed(first + 3 + i)) return false;
          const uint32_t vb = block_at(first + 3 + i);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_tmem_a(tmem + kColO + 128 * r, tmem + kColS + 128 * r + (i * 4 + kk) * 8, smem_desc(vb + kk * 2048, kBlock / 2, 1024),
                       idesc_pv, !begins || i > 0 || kk > 0);
        }
        issued = true;
        mma_commit(bar(kBarO + r));
        return true;
      };
      const auto free_blocks = [&](uint32_t first, int n) {
        for (int i = 0; i < n; ++i) mma_commit(bar(kBarEmpty + (first + i) % kSlots));
      };
      for (uint32_t n_unit = 0;; ++n_unit) {
        const int slot = n_unit & 1;
        if (!wait_bar(bar(kBarUnit + slot), (n_unit >> 1) & 1, abort_flag)) break;
        const Unit x = *unit_slot(slot);
        mbar_arrive(bar(kBarUnitEmpty + slot));
        if (!x.live) break;
        const int n0 = x.tiles[0], n1 = x.tiles[1], n = max(n0, n1);
        if (n == 0) continue;
        bool ok = true;
        if (n0) ok = wait_bar(bar(kBarQFull + 0), q_uses[0]++ & 1, abort_flag) && scores(0, blocks, n0 == 1);
        if (ok && n1) ok = wait_bar(bar(kBarQFull + 1), q_uses[1]++ & 1, abort_flag) && scores(1, blocks, n1 == 1);
        if (ok) free_blocks(blocks, 3);
        for (int j = 0; j < n && ok; ++j) {
          const uint32_t here = blocks + kTileBlocks * j, next = here + kTileBlocks;
          if (j < n0) ok = values(0, here, j == 0);
          if (ok && j + 1 < n0) ok = scores(0, next, j + 2 == n0);
          if (ok && j < n1) ok = values(1, here, j == 0);
          if (ok) free_blocks(here + 3, 2);
          if (ok && j + 1 < n1) ok = scores(1, next, j + 2 == n1);
          if (ok && j + 1 < n) free_blocks(next, 3);
        }
        if (!ok) break;
        blocks += kTileBlocks * n;
      }
      if (*abort_flag && issued) {
        mma_commit(bar(kBarDrain));
        drain_bar(bar(kBarDrain), 0);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------------------ softmax and output
    const int r = warp >> 2, in_warp = (warp & 3) * 32, row = in_warp + lane;  // lane of the unit, row of the lane
    const uint32_t tS = tmem + ((uint32_t)in_warp << 16) + kColS + 128 * r, tO = tmem + ((uint32_t)in_warp << 16) + kColO + 128 * r;
    uint32_t blocks = 0, tile_uses = 0;  // ring blocks of the units before; tiles of this lane so far
    bool ok = true;
    for (uint32_t n_unit = 0; ok; ++n_unit) {
      const int slot = n_unit & 1;
      if (!wait_warp(bar(kBarUnit + slot), (n_unit >> 1) & 1, abort_flag)) break;
      const Unit x = *unit_slot(slot);
      if (!x.live) break;
      const int n = x.tiles[r], unit_tiles = max(x.tiles[0], x.tiles[1]), other = x.tiles[r ^ 1];
      const int i = x.row0 + r * kRows + row;  // this thread's query
      const bool real = i < x.s.m && r * kRows < a.rows_per_unit;
      const int32_t vis = real ? visible(a, x.s, i) : 0;
      float m = -INFINITY;
      float2 l = make_float2(0.f, 0.f);
      for (int j = 0; j < n; ++j) {
        if (!wait_warp(bar(kBarS + r), tile_uses & 1, abort_flag)) {
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
        const int tile = x.t0 + j;
        if (tile >= x.special) {
          const int64_t left = (int64_t)vis - (int64_t)tile * kKeys;
          const int seen = (int)(left < 0 ? 0 : left > kKeys ? kKeys : left);
#pragma unroll
          for (int k = 0; k < kKeys; ++k) p[k] = k < seen ? p[k] : -INFINITY;
        }
        float top;
        {
          float t[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            t[c] = max3(p[c], p[8 + c], p[16 + c]);
#pragma unroll
            for (int k = 24; k + 8 < kKeys; k += 16) t[c] = max3(t[c], p[k + c], p[k + 8 + c]);
            t[c] = fmaxf(t[c], p[120 + c]);
          }
          top = max3(max3(t[0], t[1], t[2]), max3(t[3], t[4], t[5]), fmaxf(t[6], t[7]));
        }
        const bool grows = (top - m) * a.scale_log2 > 8.f;
        if (__any_sync(0xffffffffu, grows)) {
          const float keep = grows ? ex2((m - top) * a.scale_log2) : 1.f;
          m = grows ? top : m;
          l.x *= keep;
          l.y *= keep;
          if (j > 0) {
            if (!wait_warp(bar(kBarO + r), (tile_uses - 1) & 1, abort_flag)) {
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
        const float off = m == -INFINITY ? 0.f : -m;
        const float2 off2 = make_float2(off, off), scale2 = make_float2(a.scale_log2, a.scale_log2);
        float2 sum[2] = {l, make_float2(0.f, 0.f)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t w[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            float2 v = mul2(add2(make_float2(p[64 * half + 2 * k], p[64 * half + 2 * k + 1]), off2), scale2);
            v.x = ex2(v.x);
            v.y = ex2(v.y);
            sum[k & 1] = add2(sum[k & 1], v);
            w[k] = pack_bf16(v.x, v.y);
          }
          TMEM_ST32(tS + 32 * half, w);
        }
        l = add2(sum[0], sum[1]);
        if (tile >= x.special && (r == 0 || j >= other)) {
          // the first lane that uses the tile looks through its values: thread `row` has key `row`
          const uint32_t block = blocks + kTileBlocks * j + 3 + (row >> 6);
          if (!wait_warp(bar(kBarFull + block % kSlots), (block / kSlots) & 1, abort_flag)) {
            ok = false;
            break;
          }
          uint4* const at = reinterpret_cast<uint4*>(smem + kSmemRing + (block % kSlots) * kBlock + (row & 63) * 128);
          const bool behind = (int64_t)tile * kKeys + row >= x.s.n;
          bool odd = false;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            uint4* const v = at + (c >> 3) * (kBlock / 32) + ((c + row) & 7);
            uint4 d = *v;
            const auto mask = [](uint32_t t) { return __vcmpeq2(t & 0x7f807f80u, 0x7f807f80u); };
            const uint4 f = make_uint4(mask(d.x), mask(d.y), mask(d.z), mask(d.w));
            if (behind) {
              *v = make_uint4(0u, 0u, 0u, 0u);
            } else if (f.x | f.y | f.z | f.w) {
              odd = true;
              *v = make_uint4(d.x & ~f.x, d.y & ~f.y, d.z & ~f.z, d.w & ~f.w);
            }
          }
          const uint32_t found = __ballot_sync(0xffffffffu, odd);
          if (lane == 0) bad[(slot * kMaxSpecial + (tile - x.special)) * 4 + (warp & 3)] = found;
          fence_proxy_async();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarP + r));
        ++tile_uses;
      }
      // the last product of this lane, then O / l
      if (ok && n > 0 && !wait_warp(bar(kBarO + r), (tile_uses - 1) & 1, abort_flag)) ok = false;
      const int64_t rh = (int64_t)(x.s.q0 + (int64_t)i) * a.H + x.h, rows = a.num_q * a.H;
      float* const lse_at = a.splits > 1 ? a.part_lse + x.split * rows + rh : a.lse + rh;
      if (!ok) {
        if (real) *lse_at = NAN;
        break;
      }
      tc_fence_after();
      const float sum = l.x + l.y, inv = sum == 0.f ? 0.f : 1.f / sum;
      if (real) *lse_at = sum == 0.f ? -INFINITY : m * a.scale + logf(sum);
      uint32_t odd = 0;  // does the unit have values that are not finite?
      const int specials = max(0, x.t0 + unit_tiles - max(x.t0, x.special));
      for (int k = 0; k < specials * 4; ++k) odd |= bad[(slot * kMaxSpecial + max(x.t0 - x.special, 0)) * 4 + k];
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float o[32];
        if (n > 0) {
          TMEM_LD32(tO + 32 * c, reinterpret_cast<uint32_t*>(o));
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            asm volatile("" : "+f"(o[k]));
            o[k] *= inv;
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
        if (odd && n > 0) {
#pragma unroll 1
          for (int t = 0; t < specials * kKeys; ++t) {
            const int64_t key = (int64_t)max(x.t0, x.special) * kKeys + t;
            if (!(bad[(slot * kMaxSpecial + max(x.t0 - x.special, 0)) * 4 + (t >> 5)] >> (t & 31) & 1) || key >= vis) continue;
            const __nv_bfloat16* v = a.v + (x.s.k0 + key) * a.v_ts + x.g * a.v_hs + 32 * c;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float f = __bfloat162float(v[k]);
              if (!isfinite(f)) o[k] += f;
            }
          }
        }
        if (!real) continue;
        if (a.splits > 1 || a.out_f32) {
          float4* dst = reinterpret_cast<float4*>((a.splits > 1 ? a.part_o + (x.split * rows + rh) * kHeadV : static_cast<float*>(a.out) + rh * kHeadV) + 32 * c);
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + rh * kHeadV + 32 * c);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dst[k] = make_uint4(pack_bf16(o[8 * k], o[8 * k + 1]), pack_bf16(o[8 * k + 2], o[8 * k + 3]),
                                pack_bf16(o[8 * k + 4], o[8 * k + 5]), pack_bf16(o[8 * k + 6], o[8 * k + 7]));
        }
      }
      blocks += kTileBlocks * unit_tiles;
      tc_fence_before();  // (the reads of O are done before the next unit's first P is announced)
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarUnitEmpty + slot));
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// The (sequence, row tile) entries of a batch in the order of their tiles of keys, most first: a counting sort by one CTA.
constexpr int kListThreads = 1024, kBins = 2048;
__global__ void __launch_bounds__(kListThreads) prompt_list_kernel(const PromptArgs a) {
  __shared__ int32_t bins[kBins];
  __shared__ int32_t sums[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t most = (int32_t)(((int64_t)a.max_k + kKeys - 1) / kKeys);
  int shift = 0;
  while ((most >> shift) >= kBins) ++shift;
  const auto each = [&](auto use) {
    for (int b = warp; b < a.B; b += kListThreads / 32) {
      const PromptSeq s = load_seq(a, b);
      const int32_t tiles = (int32_t)(((int64_t)s.m + a.rows_per_unit - 1) / a.rows_per_unit);
      for (int32_t t = lane; t < tiles; t += 32) {
        const int32_t last = min((int64_t)s.m, ((int64_t)t + 1) * a.rows_per_unit) - 1;
        const int32_t cost = (int32_t)(((int64_t)visible(a, s, last) + kKeys - 1) / kKeys);
        use(b, t, kBins - 1 - (cost >> shift));
      }
    }
  };
  for (int i = threadIdx.x; i < kBins; i += kListThreads) bins[i] = 0;
  __syncthreads();
  each([&](int, int, int bin) { atomicAdd(&bins[bin], 1); });
  __syncthreads();
  // exclusive prefix sums of the bins, two a thread
  const int32_t c0 = bins[2 * threadIdx.x], c1 = bins[2 * threadIdx.x + 1];
  int32_t inc = c0 + c1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t up = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += up;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int32_t v = sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t up = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += up;
    }
    sums[lane] = v;
  }
  __syncthreads();
  const int32_t before = inc - c0 - c1 + (warp ? sums[warp - 1] : 0), all = sums[31];
  bins[2 * threadIdx.x] = before;
  bins[2 * threadIdx.x + 1] = before + c0;
  __syncthreads();
  each([&](int b, int t, int bin) {
    const int32_t at = atomicAdd(&bins[bin], 1);
    if (at < a.entries) a.list[at] = make_int2(b, t);
  });
  for (int64_t i = all + threadIdx.x; i < a.entries; i += kListThreads) a.list[i] = make_int2(-1, 0);
}

bool encode(EncodeTiledFn enc, CUtensorMap* map, const void* p, int64_t dims, int64_t heads, int64_t head_stride, int64_t rows,
            int64_t row_stride, int box_rows) {
  // (a dim of one element may have any stride in the caller's tensor)
  const cuuint64_t size[3] = {(cuuint64_t)dims, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t stride[2] = {(cuuint64_t)(heads > 1 ? head_stride : dims) * 2, (cuuint64_t)(rows > 1 ? row_stride : dims) * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows}, one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), size, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_prompt_tc(const PromptArgs& a, cudaStream_t stream) {
  EncodeTiledFn enc = tensor_map_encoder();
  CUtensorMap q, k, kr, v;
  const int64_t hk = a.H / a.group;
  // without keys nothing is loaded through these three: the queries' tensor stands in for them
  const bool keys = a.num_k > 0;
  if (!enc || !encode(enc, &q, a.q, kHeadQ, a.H, a.q_hs, a.num_q, a.q_ts, kRows) ||
      !(keys ? encode(enc, &k, a.k, kNope, hk, a.k_hs, a.num_k, a.k_ts, kKeys) : (k = q, true)) ||
      !(keys ? encode(enc, &kr, a.kr, kDRope, 1, 0, a.num_k, a.kr_ts, kKeys) : (kr = q, true)) ||
      !(keys ? encode(enc, &v, a.v, kHeadV, hk, a.v_hs, a.num_k, a.v_ts, kKeys / 2) : (v = q, true)))
    return cudaErrorInvalidValue;
  const int64_t units = a.entries * a.splits * a.H;
  if (units > 0x7fffffff) return cudaErrorInvalidValue;
  if (a.listed) {
    prompt_list_kernel<<<1, kListThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = cudaFuncSetAttribute(prompt_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)units);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_tc_kernel, a, q, k, kr, v);
}

}  // namespace mla
