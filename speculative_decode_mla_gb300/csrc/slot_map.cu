// Block tables and slot maps from request lengths (declared in include/mla_kv_ops.h).
//
// One launch. The work is small (four bytes written to the map and to the slot table per token), so
// what counts is the latency of one kernel: every CTA sums the lengths of all sequences for itself
// (num_seqs <= 8192, from L2) instead of waiting for another kernel's sums, then takes its share of
// the tokens. Nothing that a CTA reads is written by another one: held_out and free_left are separate
// outputs (overlapping arrays are refused), the block table is read below have_b and written from there on, the slot
// table read below h_b and written from there on. 64 draft trees of 8 nodes with page_size 1 take 4.6 us, 32 prompts of 301 k tokens
// in pages of 64 take 4.8: launch, then four reads that wait on one another (lengths, the sequence's numbers, block table or
// free list, slots). With 64-bit divisions it was 5.0 and 5.2.
#include <atomic>

#include "mla_kv_ops.h"

#include "common.cuh"

namespace mla {
namespace {

constexpr int kMapThreads = 512;
constexpr int kMapMaxSeqs = 8192;
constexpr int kMapTokens = 4;  // consecutive tokens a thread takes at a time (one 16-byte store to the map)

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Span {  // an array of int32
  const int32_t* p;
  int64_t n;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.n > 0 && b.n > 0 && x < y + 4 * (uintptr_t)b.n && y < x + 4 * (uintptr_t)a.n;
}

struct MapArgs {
  const int32_t *seq_lens, *new_lens, *held_lens, *free_pages, *free_count;
  int32_t *block_table, *slot_table, *slot_map, *cu_new, *held_out, *free_left, *dev_status;
  int64_t map_capacity;
  int32_t B, page_size, num_pages, free_capacity, block_stride, slot_stride, debug;
};

// Pages of x >= 0 positions (32-bit division: a 64-bit one takes several times as long, and there are few warps to hide it).
__device__ __forceinline__ int32_t pages_of(int32_t x, int32_t page_size) {
  return x == 0 ? 0 : (int32_t)((uint32_t)(x - 1) / (uint32_t)page_size) + 1;
}

// What sequence b asks for: n new tokens from position L on, h positions held in `have` pages, `take` pages more.
struct Wish {
  int32_t L, h, n, have, take, end;
  bool ok;
};
__device__ __forceinline__ Wish wish_of(const MapArgs& a, int b) {
  Wish w;
  w.L = a.seq_lens[b];
  w.n = a.new_lens[b];
  w.h = a.held_lens ? a.held_lens[b] : w.L;
  const int64_t end = max((int64_t)w.h, (int64_t)w.L + w.n);
  w.ok = w.L >= 0 && w.n >= 0 && w.h >= w.L && end <= a.slot_stride;
  w.have = w.take = 0;
  w.end = w.h;
  if (w.ok) {
    const int32_t pages = pages_of((int32_t)end, a.page_size);
    w.ok = !a.block_table || pages <= a.block_stride;
    if (w.ok) {
      w.have = pages_of(w.h, a.page_size);
      w.take = pages - w.have;
      w.end = (int32_t)end;
    }
  }
  if (!w.ok) w.n = 0;
  return w;
}

__device__ __forceinline__ longlong2 warp_inclusive(longlong2 v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v.x, d), y = __shfl_up_sync(0xffffffffu, v.y, d);
    if (lane >= d) {
      v.x += x;
      v.y += y;
    }
  }
  return v;
}

__global__ void __launch_bounds__(kMapThreads) slot_map_kernel(const MapArgs a) {
  extern __shared__ int32_t s_sum[];  // [B + 1] first token of each sequence, [B] pages taken before it
  __shared__ longlong2 s_warp[kMapThreads / 32];
  int32_t* s_cu = s_sum;
  int32_t* s_first = s_sum + a.B + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first_cta = blockIdx.x == 0;

  // the sums over the sequences before each one: a thread takes `per` consecutive sequences
  const int per = (a.B + kMapThreads - 1) / kMapThreads;
  const int b0 = tid * per, b1 = min(a.B, b0 + per);
  const int32_t fc = *a.free_count;
  longlong2 own = {0, 0};
  Wish w = {};  // (of the last one; with one sequence a thread, the only one)
  for (int b = b0; b < b1; ++b) {
    w = wish_of(a, b);
    if (!w.ok && first_cta) report(a.dev_status, a.debug, MLA_CHECK_BAD_LENGTH);
    own.x += w.n;
    own.y += w.take;
  }
  const longlong2 inc = warp_inclusive(own, lane);
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  longlong2 base = {0, 0}, total = {0, 0};
#pragma unroll
  for (int i = 0; i < kMapThreads / 32; ++i) {
    if (i < warp) {
      base.x += s_warp[i].x;
      base.y += s_warp[i].y;
    }
    total.x += s_warp[i].x;
    total.y += s_warp[i].y;
  }
  const bool granted = total.x <= a.map_capacity && fc >= 0 && fc <= a.free_capacity && total.y <= fc;
  long long cu = base.x + inc.x - own.x, pages = base.y + inc.y - own.y;
  for (int b = b0; b < b1; ++b) {
    if (per > 1) w = wish_of(a, b);
    s_cu[b] = granted ? (int32_t)cu : 0;
    s_first[b] = granted ? (int32_t)pages : 0;
    if (first_cta) {
      a.cu_new[b] = s_cu[b];
      a.held_out[b] = granted ? w.end : w.h;
    }
    cu += w.n;
    pages += w.take;
  }
  const int32_t tokens = granted ? (int32_t)total.x : 0;
  if (tid == 0) {
    s_cu[a.B] = tokens;
    if (first_cta) {
      a.cu_new[a.B] = tokens;
      *a.free_left = granted ? fc - (int32_t)total.y : fc;
      if (!granted) report(a.dev_status, a.debug, MLA_CHECK_NO_PAGES);
    }
  }
  __syncthreads();

  const int64_t step = (int64_t)gridDim.x * kMapThreads * kMapTokens;
  const bool wide = (reinterpret_cast<uintptr_t>(a.slot_map) & 15) == 0;
  const int64_t num_slots = (int64_t)a.num_pages * a.page_size;
  for (int64_t i0 = ((int64_t)blockIdx.x * kMapThreads + tid) * kMapTokens; i0 < a.map_capacity; i0 += step) {
    int32_t out[kMapTokens];
    int b = -1;
    int32_t next = 0;
#pragma unroll
    for (int k = 0; k < kMapTokens; ++k) {
      const int64_t i = i0 + k;
      out[k] = -1;
      if (i >= tokens) continue;
      if (b < 0 || i >= next) {  // the sequence of token i: the last one that starts at or before it
        int lo = b < 0 ? 0 : b + 1, hi = a.B - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_cu[mid] <= i) lo = mid;
          else hi = mid - 1;
        }
        b = lo;
        next = s_cu[b + 1];
        w = wish_of(a, b);
      }
      const int32_t t = w.L + (int32_t)(i - s_cu[b]);
      int32_t* place = a.slot_table + (int64_t)b * a.slot_stride + t;
      int64_t slot;
      if (t < w.h) {
        slot = *place;
        if (slot < 0 || slot >= num_slots) {
          report(a.dev_status, a.debug, MLA_CHECK_BAD_SLOT);
          slot = -1;
        }
      } else {
        const int32_t k_page = (int32_t)((uint32_t)t / (uint32_t)a.page_size), in_page = t - k_page * a.page_size;
        int32_t page;
        if (k_page >= w.have) {
          page = a.free_pages[fc - 1 - (s_first[b] + (k_page - w.have))];
          if (in_page == 0 && a.block_table) a.block_table[(int64_t)b * a.block_stride + k_page] = page;
        } else {
          page = a.block_table[(int64_t)b * a.block_stride + k_page];
        }
        slot = (int64_t)page * a.page_size + in_page;
        if (page < 0 || page >= a.num_pages) {
          report(a.dev_status, a.debug, MLA_CHECK_BAD_SLOT);
          slot = -1;
        }
        *place = (int32_t)slot;
      }
      out[k] = (int32_t)slot;
    }
    if (wide && i0 + kMapTokens <= a.map_capacity) {
      *reinterpret_cast<int4*>(a.slot_map + i0) = make_int4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kMapTokens; ++k)
        if (i0 + k < a.map_capacity) a.slot_map[i0 + k] = out[k];
    }
  }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_slot_map_build(const int32_t* seq_lens, const int32_t* new_lens, const int32_t* held_lens,
                                  int32_t num_seqs, int32_t page_size, int32_t num_pages, const int32_t* free_pages,
                                  int32_t free_capacity, const int32_t* free_count, int32_t* block_table,
                                  int32_t block_stride, int32_t* slot_table, int32_t slot_stride, int32_t* slot_map,
                                  int64_t map_capacity, int32_t* cu_new, int32_t* held_out, int32_t* free_left,
                                  int32_t debug, int32_t* dev_status, mla_stream_t stream) {
  if (num_seqs < 1 || num_seqs > kMapMaxSeqs) return num_seqs < 1 ? MLA_ERR_INVALID_ARGUMENT : MLA_ERR_UNSUPPORTED;
  if (page_size < 1 || num_pages < 1 || (int64_t)page_size * num_pages > 0x7fffffff) return MLA_ERR_INVALID_ARGUMENT;
  if (free_capacity < 0 || slot_stride < 1 || map_capacity < 0 || map_capacity > 0x7fffffff)
    return MLA_ERR_INVALID_ARGUMENT;
  if (!seq_lens || !new_lens || !free_count || !slot_table || !cu_new || !held_out || !free_left ||
      (free_capacity > 0 && !free_pages) || (map_capacity > 0 && !slot_map))
    return MLA_ERR_INVALID_ARGUMENT;
  if (block_table ? block_stride < 1 : page_size != 1) return MLA_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {seq_lens, new_lens, held_lens, free_pages, free_count, block_table, slot_table,
                        slot_map, cu_new,   held_out,  free_left,  dev_status};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return MLA_ERR_INVALID_ARGUMENT;
  if (debug && !dev_status) return MLA_ERR_INVALID_ARGUMENT;
  // What is written (the tables too) lies over nothing else: CTAs read the inputs, and the tables' old parts, at any time.
  // (With pages of one slot both tables hold the same numbers, and one array may serve as both: a thread writes its
  // place twice, the slot last.)
  const int64_t B = num_seqs;
  const bool one_table = page_size == 1 && block_table == slot_table && block_stride == slot_stride;
  const Span spans[] = {{block_table, block_table && !one_table ? B * block_stride : 0}, {slot_table, B * slot_stride},
                        {slot_map, map_capacity}, {cu_new, B + 1}, {held_out, B}, {free_left, 1},
                        {dev_status, debug ? 1 : 0},  // the first seven are written
                        {seq_lens, B}, {new_lens, B}, {held_lens, held_lens ? B : 0}, {free_pages, free_capacity},
                        {free_count, 1}};
  for (int i = 0; i < 7; ++i)
    for (const Span& other : spans)
      if (&other != &spans[i] && overlap(spans[i], other)) return MLA_ERR_INVALID_ARGUMENT;

  // The opt-in to more than the default limit (48 KB of dynamic and static bytes together, from 6112 sequences on), set
  // once per device whatever this call needs (setting it twice is harmless).
  static std::atomic<bool> configured[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MLA_ERR_NO_DEVICE;
  if (dev < 0 || dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(slot_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (2 * kMapMaxSeqs + 1) * (int)sizeof(int32_t)) != cudaSuccess)
      return MLA_ERR_CUDA;
    if (dev >= 0 && dev < 64) configured[dev].store(true, std::memory_order_release);
  }
  const size_t smem = ((size_t)2 * num_seqs + 1) * sizeof(int32_t);
  const int64_t per_cta = (int64_t)kMapThreads * kMapTokens;
  const int64_t want = (map_capacity + per_cta - 1) / per_cta;
  const unsigned ctas = (unsigned)(want < 1 ? 1 : want > 608 ? 608 : want);
  MapArgs a = {seq_lens,  new_lens, held_lens, free_pages, free_count,   block_table, slot_table, slot_map,
               cu_new,    held_out, free_left, dev_status, map_capacity, num_seqs,    page_size,  num_pages,
               free_capacity, block_stride, slot_stride, debug};
  slot_map_kernel<<<ctas, kMapThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
