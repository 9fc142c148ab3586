// move.cuh -- tokens moved inside a paged cache: copies of pages, and the kept
// tokens of a sequence moved together (see include/ovc.h).
#pragma once

#include <cstdint>

#include "pages.cuh"
#include "paged.cuh"

namespace ovc {

// ---------------------------------------------------------------------------
// Copy: a warp takes 32 tokens of one head of K or V of one copy: 8 rows of 16
// bytes a lane, all read before the first is written, and a scale byte a lane.
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;

struct CopyParams {
  CacheView to, from;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* tokens;    // or nullptr: whole pages
  int32_t n, groups;        // copies; warps' groups of 32 tokens a page
  FastDiv by_groups, by_heads;
  unsigned int* status;
};

__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(CopyParams P) {
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);   // of one copy: kv, head, group
  const int i = blockIdx.y + blockIdx.z * 65535;
  const int hk = unit / P.by_groups, t0 = (unit - hk * P.groups) * 32;
  const int kv = hk / P.by_heads, h = hk - kv * P.to.heads;
  if (i >= P.n || kv > 1) return;
  const int s = P.src[i], d = P.dst[i];
  if (s < 0 || d < 0) return;
  const int page = P.to.page, n = P.tokens ? P.tokens[i] : page;
  if (s >= P.from.pages || d >= P.to.pages || n < 0 || n > page) {
    if (unit == 0 && lane == 0) atomicOr(P.status, kPagedBadIndex);
    return;
  }
  const int64_t a = (static_cast<int64_t>(s) * P.to.heads + h) * page + t0;
  const int64_t b = (static_cast<int64_t>(d) * P.to.heads + h) * page + t0;
  const uint4* from = reinterpret_cast<const uint4*>((kv ? P.from.v : P.from.k) + a * 128) + lane;
  uint4* to = reinterpret_cast<uint4*>((kv ? P.to.v : P.to.k) + b * 128) + lane;
  const uint8_t* from_scale = (kv ? P.from.vs : P.from.ks) + a;
  uint8_t* to_scale = (kv ? P.to.vs : P.to.ks) + b;
  const int rows = n - t0, mine = lane >> 3;
  uint4 x[8];
  uint8_t e = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (4 * j + mine < rows) x[j] = __ldcs(from + 32 * j);
  if (lane < rows) e = from_scale[lane];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (4 * j + mine < rows) __stcs(to + 32 * j, x[j]);
  if (lane < rows) to_scale[lane] = e;
}

// ---------------------------------------------------------------------------
// Compact, in place: position i of a sequence takes token keep[i] >= i.  A cluster
// takes one head of K or V of one sequence and goes over the positions upwards,
// a chunk of 256 for each of its CTAs at a time.  The tokens of later chunks lie
// behind what a chunk writes (keep ascends, so keep[j] >= j), so they may be read
// at any time; those of the same and earlier chunks have been read when the
// cluster passes its barrier, and then the chunk is written.
//
// A warp moves 32 positions of a chunk through its own part of shared memory:
// list, page table, and tokens of the chunks ahead are on their way while one is
// written.
// ---------------------------------------------------------------------------
constexpr int kCompactThreads = 256;
constexpr int kCompactChunk = 256;                // positions of a CTA at a time: 32 a warp, 8 x 16 bytes a lane
constexpr int kCompactStages = 3;                 // chunks in shared memory
constexpr int kCompactSmem = kCompactStages * kCompactChunk * 128;

struct CompactParams {
  CacheView c;
  PagesView P;
  const int32_t* keep;
  int64_t keep_stride;      // 0: one list for all heads
  const int32_t* cu;
  int32_t n;                // kept tokens in all
};

__device__ __forceinline__ void copy_async16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

__global__ void __launch_bounds__(kCompactThreads, 2) kv_compact_kernel(CompactParams C) {
  extern __shared__ __align__(128) uint8_t tokens[];
  __shared__ uint8_t scale_of[kCompactThreads];
  __shared__ int found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = cluster_size(), rank = cluster_rank();
  const int h = blockIdx.y >> 1, kv = blockIdx.y & 1, b = blockIdx.z;
  const int a0 = C.cu[b], a1 = C.cu[b + 1];
  const int len = row_len(C.P, b), n = a1 - a0;
  if (a0 < 0 || a1 > C.n || n < 0 || len < 0 || n > len) {
    if (tid == 0 && (len >= 0 || n != 0)) atomicOr(C.P.status, kPagedBadIndex);
    return;                                       // all CTAs of the cluster
  }
  const int32_t* keep = C.keep + h * C.keep_stride + a0;
  const int32_t* table = C.P.table + static_cast<int64_t>(b) * C.P.width;

  // The first position that does not stay: keep[i] - i never falls.
  int lo = 0, hi = n;                             // it lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + kCompactThreads - 1) / kCompactThreads;
    if (tid == 0) found = hi;
    __syncthreads();
    const int i = lo + (tid + 1) * step - 1;      // the last of this thread's part
    if (i < hi && __ldg(keep + i) != i) atomicMin(&found, i);
    __syncthreads();
    const int f = found;
    __syncthreads();
    const int part = f == hi ? (hi - lo) / step * step : f - step + 1 - lo;
    lo += part;
    hi = f;
    if (step == 1) {
      lo = f;
      break;
    }
  }
  // Pages that would be written must be this row's own.
  int bad = 0;
  for (int c = lo / C.P.by_page + tid; lo < n && c <= (n - 1) / C.P.by_page; c += kCompactThreads) {
    const int p = table[c];
    bad |= p < 0 || p >= C.c.pages || C.P.refs[p] > 1;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) atomicOr(C.P.status, kPagedBadIndex);
    return;                                       // all CTAs of the cluster see the same
  }
  uint8_t* codes = kv ? C.c.v : C.c.k;
  uint8_t* scales = kv ? C.c.vs : C.c.ks;

  // The same number of steps in every CTA; step s is this lane's position lo + s * stride + ...
  const int stride = kCompactChunk * ctas, steps = (n - lo + stride - 1) / stride;
  const int first = lo + rank * kCompactChunk + tid;
  struct Ahead {            // of one position: its token and the one before it, the pages of both
    int t, before, from, to;
  };
  // Each of the three uses what the one before it loaded a step earlier: a value
  // looked at in the step that loads it would make the warp wait for it.
  auto listed = [&](int s, Ahead& x) {            // its token
    const int64_t i = first + static_cast<int64_t>(s) * stride;
    x.t = i < n ? __ldg(keep + i) : -1;
    x.before = lane == 0 && i > 0 && i < n ? __ldg(keep + i - 1) : -1;
  };
  auto paged = [&](int s, Ahead& x) {             // its pages
    const int64_t i = first + static_cast<int64_t>(s) * stride;
    const int up = __shfl_up_sync(0xFFFFFFFFu, x.t, 1);
    const bool ok = i < n && x.t >= i && x.t > (lane ? up : x.before) && x.t < len;
    if (!ok && i < n) atomicOr(C.P.status, kPagedBadIndex);
    if (!ok) x.t = -1;
    x.from = ok ? __ldg(table + x.t / C.P.by_page) : -1;
    x.to = ok ? __ldg(table + static_cast<int>(i) / C.P.by_page) : -1;
  };
  auto row_of = [&](int t, int p) { return (p * C.c.heads + h) * C.c.page + (t - t / C.P.by_page * C.c.page); };
  const uint32_t mine = smem_addr(tokens) + warp * (32 * 128) + lane * 16;
  int to[kCompactStages], scale[kCompactStages];
  auto fetch = [&](int s, int stage, const Ahead& x) {            // its token's codes and scale on their way
    int from = -1;
    to[stage] = -1;
    if (x.t >= 0) {
      if (x.from >= 0 && x.from < C.c.pages && x.to >= 0 && x.to < C.c.pages) {
        from = row_of(x.t, x.from);
        to[stage] = row_of(first + s * stride, x.to);
      } else {
        atomicOr(C.P.status, kPagedBadIndex);
      }
    }
    scale[stage] = from >= 0 ? __ldcg(scales + from) : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = __shfl_sync(0xFFFFFFFFu, from, 4 * j + (lane >> 3));
      if (row >= 0) copy_async16(mine + stage * (kCompactChunk * 128) + j * 512, codes + static_cast<int64_t>(row) * 128 + (lane & 7) * 16);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  Ahead x0, x1, x2;
  listed(0, x0);
  listed(1, x1);
  listed(2, x2);
  paged(0, x0);
  paged(1, x1);
  fetch(0, 0, x0);
  fetch(1, 1, x1);
  x0 = x2;
  paged(2, x0);
  listed(3, x1);
  int s = 0;
  while (s < steps) {
#pragma unroll
    for (int stage = 0; stage < kCompactStages; ++stage, ++s) {   // step s is in `stage`
      if (s >= steps) break;
      fetch(s + 2, (stage + 2) % kCompactStages, x0);
      x0 = x1;
      paged(s + 3, x0);
      listed(s + 4, x1);
      asm volatile("cp.async.wait_group 2;" ::: "memory");
      scale_of[tid] = scale[stage];               // what this thread reads has arrived
      __syncwarp();
      if (ctas > 1) {
        // Only reads have to be over, and those are: no fence for what was written.
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        cluster_wait();
      } else {
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = __shfl_sync(0xFFFFFFFFu, to[stage], 4 * j + (lane >> 3));
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(mine + stage * (kCompactChunk * 128) + j * 512));
        if (row >= 0) *reinterpret_cast<uint4*>(codes + static_cast<int64_t>(row) * 128 + (lane & 7) * 16) = v;
      }
      if (to[stage] >= 0) scales[to[stage]] = scale_of[tid];
      __syncwarp();
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace ovc
