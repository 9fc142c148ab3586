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
// behind what a chunk writes (keep ascends, so keep[j] >= j), and those of the same
// and earlier chunks have been read when the cluster passes its barrier: between
// it and the next the chunk is written, while the next one is being read already.
// ---------------------------------------------------------------------------
constexpr int kCompactThreads = 256;
constexpr int kCompactChunk = 256;                // positions of a CTA at a time: 32 a warp, 8 x 16 bytes a lane

struct CompactParams {
  CacheView c;
  PagesView P;
  const int32_t* keep;
  int64_t keep_stride;      // 0: one list for all heads
  const int32_t* cu;
  int32_t n;                // kept tokens in all
};

struct Kept {               // what a warp moves at once
  uint4 x[8];
  uint8_t e;
  int64_t to;               // this lane's position's row, -1: none
};

// Row of the cache that holds position t of a sequence, or -1.
__device__ __forceinline__ int64_t token_row(const CompactParams& C, const int32_t* table, int t, int h) {
  const int col = t / C.P.by_page, p = table[col];
  if (p < 0 || p >= C.c.pages) return -1;
  return (static_cast<int64_t>(p) * C.c.heads + h) * C.c.page + (t - col * C.c.page);
}

__global__ void __launch_bounds__(kCompactThreads) kv_compact_kernel(CompactParams C) {
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

  auto read = [&](int i0, Kept& r) {              // the warp's 32 positions from i0 on
    const int i = i0 + lane;
    int64_t from = -1;
    r.to = -1;
    if (i < n) {
      const int t = __ldg(keep + i), before = i ? __ldg(keep + i - 1) : -1;
      if (t >= i && t > before && t < len) {
        from = token_row(C, table, t, h);
        r.to = token_row(C, table, i, h);
      }
      if (from < 0) {
        r.to = -1;
        atomicOr(C.P.status, kPagedBadIndex);
      }
    }
    r.e = r.to >= 0 ? __ldcg(scales + from) : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t row = __shfl_sync(0xFFFFFFFFu, from, 4 * j + (lane >> 3));
      if (row >= 0) r.x[j] = __ldcg(reinterpret_cast<const uint4*>(codes + row * 128) + (lane & 7));
    }
  };
  auto write = [&](const Kept& r) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t row = __shfl_sync(0xFFFFFFFFu, r.to, 4 * j + (lane >> 3));
      if (row >= 0) reinterpret_cast<uint4*>(codes + row * 128)[lane & 7] = r.x[j];
    }
    if (r.to >= 0) scales[r.to] = r.e;
  };
  // The same number of steps in every CTA.
  const int stride = kCompactChunk * ctas, steps = (n - lo + stride - 1) / stride;
  int i0 = lo + rank * kCompactChunk + warp * 32;
  Kept r;
  for (int s = 0; s < steps; ++s, i0 += stride) {
    read(i0, r);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    write(r);
    __syncwarp();
  }
}

}  // namespace ovc
