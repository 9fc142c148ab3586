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
// Bound by memory: 2048 pages of 64 tokens x 8 heads, 541 MB read and written, in
// 82 us, 98% of the measured copy rate; 32 page tails in 3 us, a launch.
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
// takes one head of K or V of one sequence (or half of its channels) and goes over
// the positions upwards, a chunk of 256 (512) for each of its CTAs at a time.  The
// tokens of later chunks lie behind what a chunk writes (keep ascends, so keep[j]
// >= j), so they may be read at any time; those of the same and earlier chunks
// have been read when all CTAs of the cluster have said so, and then the chunk is
// written.
//
// A warp moves 32 (64) positions of a chunk through its own part of shared memory:
// list, page table, and tokens of the chunks ahead are on their way while one is
// written.  That a chunk has been read is told with release at the cluster's scope,
// which also waits for what was written before; so the warps tell it to one warp of
// their CTA, by a barrier of the CTA, and that one tells the other CTAs and waits.
// Told by each warp itself, for the two cases below: 47 and 44 us.
//
// Reads and writes 258 bytes a token and head: 49152 tokens of one sequence x 8
// heads, 203 MB, in 42 us (4.9 TB/s, 73% of the measured copy rate), of which the
// chunks take 35 and the chain of lookups before the first token 6; half of 8 ragged
// sequences up to 32768 x 8 heads, 161 MB, in 38 us.  A few tokens at the sequences'
// ends: 7.5 us, that chain.
// Tried: a hardware barrier of the cluster for each chunk instead of the counting
// ones 55 and 47 us; values held in registers, not in shared memory 99 and 70 us.
// ---------------------------------------------------------------------------
constexpr int kCompactThreads = 256;                    // that move tokens
constexpr int kCompactTeller = kCompactThreads / 32;    // the warp behind them, which tells the other CTAs
constexpr int kCompactCtas = 2;                         // of an SM
constexpr int kCompactSorted = 64;                      // most sequences that are put in order
constexpr int kCompactClusters = 8;                     // most CTAs of a cluster
// Chunks in shared memory.  Two, three (a CTA less an SM) and four (two less): 8
// sequences of 16384, half kept, 56, 54 and 69 us, three quarters of 32 of 4096 73, 71
// and 88 us, the ragged ones above 40, 38 and 50 us.
constexpr int kCompactStages = 3;
constexpr uint64_t kCompactTimeoutNs = 4000000000ull;   // of a wait
constexpr unsigned kStatusTimeoutBit = 1u;              // of the device status word

template <int kRow>         // bytes of a token's codes: 128, or 64
struct CompactShape {
  static constexpr int kEach = 128 / kRow;              // positions a lane
  static constexpr int kLanes = kRow / 16;              // of a token's codes
  static constexpr int kChunk = kCompactThreads * kEach;
  static constexpr int kCodes = kChunk * kRow;
  static constexpr int kStage = kCodes + kChunk * 9;    // and words that hold the scales, rows to write, bytes of the words
  static constexpr int kSmem = kCompactStages * kStage;
};

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
__device__ __forceinline__ void copy_async4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}

// As paged_wait, of a barrier that other CTAs of the cluster arrive at.
__device__ __forceinline__ bool told_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool told_wait(uint32_t bar, uint32_t parity, const volatile int* abort) {
  if (__builtin_expect(told_try(bar, parity), 1)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!told_try(bar, parity))
    if (*abort || globaltimer_ns() - t0 > kCompactTimeoutNs) return false;
  return true;
}

template <int kRow>
__global__ void __launch_bounds__(kCompactThreads + 32, kCompactCtas) kv_compact_kernel(CompactParams C) {
  using Shape = CompactShape<kRow>;
  constexpr int kEach = Shape::kEach, kLanes = Shape::kLanes;
  extern __shared__ __align__(128) uint8_t tokens[];
  __shared__ __align__(8) uint64_t bars[kCompactStages], landed[kCompactStages];
  __shared__ int found, abort, kept[kCompactSorted];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = cluster_size(), rank = cluster_rank();
  const int part = blockIdx.y & (kEach - 1), kv = blockIdx.y / kEach & 1, h = blockIdx.y / (2 * kEach);
  // The longest sequences go first, so that they are not what remains at the end:
  // 32 ragged sequences up to 16384, half kept, 95 us without, 83 us with it, the 8
  // ragged ones 43 and 38 us; a few tokens of 16 sequences 6.8 and 7.5 us.
  int b = blockIdx.z;
  if (C.P.rows > 1 && C.P.rows <= kCompactSorted) {
    if (tid < C.P.rows) kept[tid] = C.cu[tid + 1] - C.cu[tid];
    __syncthreads();
    if (tid < C.P.rows) {
      int before = 0;
      for (int j = 0; j < C.P.rows; ++j) before += kept[j] > kept[tid] || (kept[j] == kept[tid] && j < tid);
      if (before == b) found = tid;
    }
    __syncthreads();
    b = found;
    __syncthreads();
  }
  const int a0 = C.cu[b], a1 = C.cu[b + 1];
  const int len = row_len(C.P, b);
  // A stage's barriers: the warps of this CTA that have read its chunk, and the
  // CTAs that have.
  if (tid < kCompactStages) {
    mbar_init(smem_addr(&landed[tid]), kCompactThreads / 32);
    mbar_init(smem_addr(&bars[tid]), ctas);
  }
  if (tid == 0) abort = 0;
  fence_mbar_init();
  __syncthreads();
  cluster_arrive();
  // No CTA leaves before the last barrier, whatever it finds: others may still tell
  // it something.
  bool bad = a0 < 0 || a1 < a0 || a1 > C.n || len < 0 || a1 - a0 > len;
  if (bad && tid == 0) atomicOr(C.P.status, kPagedBadIndex);
  const int n = bad ? 0 : a1 - a0;
  const int32_t* keep = C.keep + h * C.keep_stride + a0;
  const int32_t* table = C.P.table + static_cast<int64_t>(b) * C.P.width;

  uint8_t* codes = (kv ? C.c.v : C.c.k) + part * kRow;
  uint8_t* scales = kv ? C.c.vs : C.c.ks;

  // The CTAs take the same number of steps; a lane's positions in step s are first +
  // s * stride, and 32 more.
  const int stride = Shape::kChunk * ctas, mine = warp < kCompactTeller ? n : 0;
  int first = rank * Shape::kChunk + warp * (32 * kEach) + lane;
  int lo = 0;               // the first position that does not stay, once it is found
  struct Ahead {            // of some positions: their tokens and the one before them, the pages of both
    int t[kEach], before, from[kEach], to[kEach];
  };
  // Each of the three uses what the one before it loaded a step earlier: a value
  // looked at in the step that loads it would make the warp wait for it.
  auto listed = [&](int s, Ahead& x) {            // the tokens
    const int64_t i = first + static_cast<int64_t>(s) * stride;
#pragma unroll
    for (int k = 0; k < kEach; ++k) x.t[k] = i + 32 * k < mine ? __ldg(keep + i + 32 * k) : -1;
    x.before = lane == 0 && i > 0 && i < mine ? __ldg(keep + i - 1) : -1;
  };
  auto paged = [&](int s, Ahead& x) {             // their pages
    const int64_t i = first + static_cast<int64_t>(s) * stride;
    int before = x.before;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, x.t[k], 1), last = __shfl_sync(0xFFFFFFFFu, x.t[k], 31);
      const bool there = i + 32 * k < mine, ok = there && x.t[k] >= i + 32 * k && x.t[k] > (lane ? up : before) && x.t[k] < len;
      if (!ok && there) atomicOr(C.P.status, kPagedBadIndex);
      const bool moves = ok && x.t[k] != i + 32 * k;
      if (!moves) x.t[k] = -1;
      x.from[k] = moves ? __ldg(table + x.t[k] / C.P.by_page) : -1;
      x.to[k] = moves ? __ldg(table + static_cast<int>(i + 32 * k) / C.P.by_page) : -1;
      before = last;
    }
  };
  auto row_of = [&](int t, int p) { return (p * C.c.heads + h) * C.c.page + (t - t / C.P.by_page * C.c.page); };
  const uint32_t base = smem_addr(tokens);
  auto codes_at = [&](int stage) { return base + stage * Shape::kStage + warp * 4096 + lane * 16; };
  auto scale_at = [&](int stage) { return base + stage * Shape::kStage + Shape::kCodes + tid * 4; };
  auto row_at = [&](int stage) { return scale_at(stage) + Shape::kChunk * 4; };
  auto byte_at = [&](int stage) { return base + stage * Shape::kStage + Shape::kCodes + Shape::kChunk * 8 + tid; };
  auto fetch = [&](int s, int stage, const Ahead& x) {            // the tokens' codes and scales on their way
    const uint32_t at = codes_at(stage);
    int from[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      int to = -1;
      from[k] = -1;
      if (x.t[k] >= 0) {
        // (before lo: of a list that does not ascend; its page has not been looked at)
        if (first + s * stride + 32 * k >= lo && x.from[k] >= 0 && x.from[k] < C.c.pages && x.to[k] >= 0 && x.to[k] < C.c.pages) {
          from[k] = row_of(x.t[k], x.from[k]);
          to = row_of(first + s * stride + 32 * k, x.to[k]);
        } else {
          atomicOr(C.P.status, kPagedBadIndex);
        }
      }
      // (the word's other bytes may be written meanwhile: memory keeps bytes apart)
      if (part == 0 && from[k] >= 0) copy_async4(scale_at(stage) + k * (kCompactThreads * 4), scales + (from[k] & ~3));
      // the row to write, and which byte of its scale's word is meant
      asm volatile("st.shared.s32 [%0], %1;" ::"r"(row_at(stage) + k * (kCompactThreads * 4)), "r"(to) : "memory");
      if (part == 0) asm volatile("st.shared.u8 [%0], %1;" ::"r"(byte_at(stage) + k * kCompactThreads), "r"(from[k] & 3) : "memory");
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = __shfl_sync(0xFFFFFFFFu, from[j * kEach / 8], (j * (32 / kLanes) + lane / kLanes) & 31);
      if (row >= 0) copy_async16(at + j * 512, codes + static_cast<int64_t>(row) * 128 + (lane & (kLanes - 1)) * 16);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Where the work begins: at the first position that does not stay, which a search
  // by 256 narrows down (keep[i] - i never falls), or a little before it.  The first
  // lookups of the search, and of the work as if it began at 0, are on their way
  // together: list; the rest of the search, and pages; refs, and tokens.
  Ahead x[kCompactStages + 1];
#pragma unroll
  for (int s = 0; s <= kCompactStages; ++s) listed(s, x[s]);
  int hi = n, step = 0, probe = 0, seen = 0;             // it lies in [lo, hi], and is lo in the end
  auto look = [&] {
    step = (hi - lo + kCompactThreads - 1) / kCompactThreads;
    probe = lo + (min(tid, kCompactThreads - 1) + 1) * step - 1;   // the last of this thread's part
    seen = probe < hi ? __ldg(keep + probe) : probe;
  };
  auto narrow = [&] {
    if (tid == 0) found = hi;
    __syncthreads();
    if (seen != probe) atomicMin(&found, probe);
    __syncthreads();
    const int f = found;
    __syncthreads();
    lo = step == 1 ? f : f == hi ? lo + (hi - lo) / step * step : f - step + 1;
    hi = f;
  };
  if (lo < hi) {
    look();
    narrow();
  }
  const int start = lo;
  if (start > 0) {
    first += start;
#pragma unroll
    for (int s = 0; s <= kCompactStages; ++s) listed(s, x[s]);
  }
  if (lo < hi) look();
  const int columns = n > 0 ? (n - 1) / C.P.by_page + 1 : 0;
  // Where the pages are looked at from: no head moves a token before it.  With a list
  // a head, all clusters of a sequence decide alike whether it is left alone, each by
  // every head's list: `from` lies a few of the search's steps before this head's
  // start, so that most often the others begin to move behind it too.
  const bool lists = C.keep_stride > 0;
  int from = lists ? max(0, start - n / 64) : start;
  bool before = false;
  if (lists && from > 0)
#pragma unroll 1
    for (int k = tid; k < C.c.heads; k += blockDim.x) before |= __ldg(C.keep + k * C.keep_stride + a0 + from - 1) != from - 1;
  int column = from / C.P.by_page + tid, page = column < columns ? __ldg(table + column) : -1;
#pragma unroll
  for (int s = 0; s < kCompactStages; ++s) paged(s, x[s]);
  while (lo < hi) {
    narrow();
    if (lo < hi) look();
  }
  // Pages that will be written must be this row's own.
  if (lists && from > 0 && __syncthreads_or(before)) {
    column = tid;
    page = column < columns ? __ldg(table + column) : -1;
  }
  int last = -1;                                  // of this thread's columns, with a page that is not
  for (; column < columns; column += kCompactThreads, page = column < columns ? __ldg(table + column) : -1)
    if (page < 0 || page >= C.c.pages || __ldg(C.P.refs + page) > 1) last = column;
#pragma unroll
  for (int s = 0; s < kCompactStages - 1; ++s)
    if (mine) fetch(s, s, x[s]);
  Ahead x0 = x[kCompactStages - 1], x1 = x[kCompactStages];
  if (__builtin_expect(__syncthreads_or(last >= 0), 0)) {
    if (tid == 0) found = -1;
    __syncthreads();
    if (last >= 0) atomicMax(&found, last);
    __syncthreads();
    // Positions ascend, so a head writes to a column up to that one exactly if the
    // last position of it does not stay.  (A list that does not ascend may say
    // otherwise: this head's own first that moves counts too.)
    const int end = min(n, (found + 1) * C.c.page);
    bad = lo < end;
    if (lists)
#pragma unroll 1
      for (int k = tid; k < C.c.heads; k += blockDim.x) bad |= __ldg(C.keep + k * C.keep_stride + a0 + end - 1) != end - 1;
    bad = __syncthreads_or(bad);
  }
  if (bad && tid == 0) atomicOr(C.P.status, kPagedBadIndex);
  const int steps = bad || lo >= n ? 0 : (n - start - 1) / stride + 1;
  cluster_wait();
  // A warp's part of a chunk has arrived in shared memory: its CTA is told, before
  // the warp writes the chunk ahead of it, and by the last warp all CTAs are.  One CTA
  // alone needs no more than its own barrier.
  if (warp == kCompactTeller) {
    uint32_t parity = 0;
#pragma unroll 1
    for (int s = 0, stage = 0; ctas > 1 && s < steps; ++s) {
      const bool ok = paged_wait(smem_addr(&landed[stage]), parity, kCompactTimeoutNs, &abort);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      if (lane < ctas)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(&bars[stage], lane)) : "memory");
      __syncwarp();
      if (++stage == kCompactStages) stage = 0, parity ^= 1u;
    }
  }
  auto has_read = [&](int stage) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&landed[stage]));
  };
  uint64_t* const all = ctas > 1 ? bars : landed;
  asm volatile("cp.async.wait_group %0;" ::"n"(kCompactStages - 2) : "memory");
  if (steps > 0 && mine) has_read(0);                     // all that is told is waited for
  int stage = 0;                                  // of chunk s
  uint32_t parity = 0;
#pragma unroll 1
  for (int s = 0; s < steps && mine; ++s) {
    fetch(s + kCompactStages - 1, stage ? stage - 1 : kCompactStages - 1, x0);
    x0 = x1;
    paged(s + kCompactStages, x0);
    listed(s + kCompactStages + 1, x1);
    bool ok = told_wait(smem_addr(&all[stage]), parity, &abort);
    ok = __all_sync(0xFFFFFFFFu, ok);
    if (!ok) {
      abort = 1;
      atomicOr(C.P.status, kStatusTimeoutBit);
      break;
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kCompactStages - 2) : "memory");
    const int next = stage + 1 < kCompactStages ? stage + 1 : 0;
    if (s + 1 < steps) has_read(next);
    const uint32_t at = codes_at(stage);
    int to[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      asm volatile("ld.shared.s32 %0, [%1];" : "=r"(to[k]) : "r"(row_at(stage) + k * (kCompactThreads * 4)));
      if (part == 0 && to[k] >= 0) {
        uint32_t byte, e;
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(byte) : "r"(byte_at(stage) + k * kCompactThreads));
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(e) : "r"(scale_at(stage) + k * (kCompactThreads * 4) + byte));
        scales[to[k]] = static_cast<uint8_t>(e);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = __shfl_sync(0xFFFFFFFFu, to[j * kEach / 8], (j * (32 / kLanes) + lane / kLanes) & 31);
      uint4 v;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at + j * 512));
      if (row >= 0) *reinterpret_cast<uint4*>(codes + static_cast<int64_t>(row) * 128 + (lane & (kLanes - 1)) * 16) = v;
    }
    __syncwarp();
    if (next == 0) parity ^= 1u;
    stage = next;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  // No CTA leaves while others may still tell it something: the barrier's release
  // orders what was told before it (a relaxed one does not, and an arrival at a CTA
  // that has left faults).
  cluster_arrive();
  cluster_wait();
}

}  // namespace ovc
