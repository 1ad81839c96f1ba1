// What the tcgen05 attention kernels share: PTX wrappers (mbarriers with bounded waits, fences, TMEM
// loads and stores, shared-memory descriptors) and the longest-first order of a batch's work units.
#pragma once

#include "common.cuh"

namespace mla {

constexpr long long kTimeoutCycles = 4000000000ll;  // ~2 s at 2 GHz

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_test_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait: false when another role aborted or the wait timed out (then it aborts).
// cluster_scope: the phase is completed from the partner CTA (st.async bytes, remote arrive), a
// release at cluster scope; it is polled relaxed and, once seen, acquired by one fence restricted
// to shared::cluster memory, which is cheaper than an acquiring poll.
// A probe of an mbarrier costs over a hundred cycles even when the phase has completed, and
// reading the clock costs some too: the first probe goes out before the clock is read.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                         bool cluster_scope = false) {
  if (cluster_scope) {
    if (mbar_test_cluster(bar, parity)) {
      asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
      return true;
    }
  } else if (mbar_test(bar, parity)) {
    return true;
  }
  const long long start = clock64();
  while (true) {
    if (cluster_scope) {
      if (mbar_test_cluster(bar, parity)) {
        asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
        return true;
      }
    } else if (mbar_test(bar, parity)) {
      return true;
    }
    if (*abort_flag) return false;
    if (clock64() - start > kTimeoutCycles) {
      *abort_flag = 1;
      return false;
    }
  }
}
// The same wait taken by every lane of a warp; the result is uniform across the warp.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          bool cluster_scope = false) {
  const bool ok = wait_bar(bar, parity, abort_flag, cluster_scope);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, uint32_t cta) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
  return r;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 2^x on the MUFU unit (flushes subnormal results to zero; P below 2^-126 is dropped).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// UMMA shared-memory descriptor, descriptor version 1; layout 2 = 128-byte swizzle, 4 = 64-byte swizzle.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t layout = 2) {
  uint64_t d = (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= 1ull << 46;
  d |= (uint64_t)layout << 61;
  return d;
}
// Three-input maximum (one instruction on this architecture; max is exact in any order).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two fp32 lanes per instruction (the packed f32x2 forms); each lane rounds exactly as fmaf / +.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n.reg .b64 ra, rb, rc, rd;\n"
      "mov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %5};\nmov.b64 rc, {%6, %7};\n"
      "fma.rn.f32x2 rd, ra, rb, rc;\nmov.b64 {%0, %1}, rd;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 ra, rb, rd;\n"
      "mov.b64 ra, {%2, %3};\nmov.b64 rb, {%4, %5};\n"
      "add.rn.f32x2 rd, ra, rb;\nmov.b64 {%0, %1}, rd;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
#define TMEM_LD16(addr, r)                                                                                       \
  asm volatile(                                                                                                  \
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];" \
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),       \
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])   \
      : "r"(addr))
#define TMEM_ST16(addr, r)                                                                                        \
  asm volatile(                                                                                                   \
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" \
      ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),     \
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])            \
      : "memory")
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Inclusive prefix sum over the 64 values v0 (sequences 0..31, one per lane) and v1 (32..63).
__device__ __forceinline__ void warp_scan64(int v0, int v1, int lane, int& inc0, int& inc1) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u0 = __shfl_up_sync(0xffffffffu, v0, d), u1 = __shfl_up_sync(0xffffffffu, v1, d);
    if (lane >= d) {
      v0 += u0;
      v1 += u1;
    }
  }
  inc0 = v0;
  inc1 = v1 + __shfl_sync(0xffffffffu, v0, 31);
}
// The first sequence whose inclusive prefix exceeds idx (-1 if none), and that prefix.
__device__ __forceinline__ int first_above(int inc0, int inc1, int idx, int& inc_at) {
  uint32_t m = __ballot_sync(0xffffffffu, inc0 > idx);
  if (m) {
    const int l = __ffs(m) - 1;
    inc_at = __shfl_sync(0xffffffffu, inc0, l);
    return l;
  }
  m = __ballot_sync(0xffffffffu, inc1 > idx);
  const int l = m ? __ffs(m) - 1 : 0;
  inc_at = __shfl_sync(0xffffffffu, inc1, l);
  return m ? 32 + l : -1;
}
// Longest-first order of the work units of a batch of 2..64 sequences of different lengths, for
// unit idx in [0, B x splits): every sequence's full chunks first (sequence by sequence), then
// the partial last chunks from the longest down (equal lengths by sequence), then the (sequence,
// split) pairs past a sequence's end, which only mark their partial empty. Clusters start in index
// order, so the long units start first and the short ones fill the gaps at the end. Every lane of
// the warp calls it; the result (sequence, split) is uniform across the warp.
__device__ __forceinline__ void lpt_unit(const VerifyArgs& a, int idx, int lane, int& b_out, int& s_out) {
  int full[2], part[2], nsp[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int bb = lane + 32 * i;
    const int64_t n = bb < a.B ? (int64_t)load_len(a, bb) + load_tree_size(a, bb) : 0;
    full[i] = (int)(n / a.chunk);
    part[i] = (int)(n % a.chunk);
    nsp[i] = full[i] + (part[i] > 0);
  }
  int inc0, inc1, at;
  // 1. full chunks
  warp_scan64(full[0], full[1], lane, inc0, inc1);
  const int nfull = __shfl_sync(0xffffffffu, inc1, 31);
  if (idx < nfull) {
    const int bb = first_above(inc0, inc1, idx, at);
    b_out = bb;
    s_out = idx - (at - __shfl_sync(0xffffffffu, (bb >> 5) ? full[1] : full[0], bb & 31));
    return;
  }
  idx -= nfull;
  // 2. partial chunks, longest first: the one whose rank among the partial chunks is idx
  const int npart = __popc(__ballot_sync(0xffffffffu, part[0] > 0)) + __popc(__ballot_sync(0xffffffffu, part[1] > 0));
  if (idx < npart) {
    int rank[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll 4
      for (int j = 0; j < 32; ++j) {
        const int pj = __shfl_sync(0xffffffffu, part[h], j);
        const int bj = 32 * h + j;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int bi = lane + 32 * i;
          rank[i] += (pj > part[i] || (pj == part[i] && bj < bi)) && pj > 0;
        }
      }
    }
    const uint32_t m0 = __ballot_sync(0xffffffffu, part[0] > 0 && rank[0] == idx);
    const uint32_t m1 = __ballot_sync(0xffffffffu, part[1] > 0 && rank[1] == idx);
    const int bb = m0 ? __ffs(m0) - 1 : 32 + __ffs(m1) - 1;
    b_out = bb;
    s_out = __shfl_sync(0xffffffffu, (bb >> 5) ? full[1] : full[0], bb & 31);
    return;
  }
  idx -= npart;
  // 3. splits past each sequence's end
  warp_scan64(lane < a.B ? a.splits - nsp[0] : 0, lane + 32 < a.B ? a.splits - nsp[1] : 0, lane, inc0, inc1);
  const int bb = first_above(inc0, inc1, idx, at);
  const int bsafe = bb < 0 ? 0 : bb;  // (idx < B x splits always finds one)
  const int emp = a.splits - __shfl_sync(0xffffffffu, (bsafe >> 5) ? nsp[1] : nsp[0], bsafe & 31);
  b_out = bsafe;
  s_out = a.splits - emp + (idx - (at - emp));
}

}  // namespace mla
