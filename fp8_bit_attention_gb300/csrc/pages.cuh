// pages.cuh -- who holds which page of a paged cache: rows of a page table that
// take free pages, give them back, and share them (see include/ovc.h).
//
// State: page_table [rows, width], kv_lens [rows], refs [pages].  Row b holds
// ceil(kv_lens[b] / page) pages; refs[p] = 0 says that page p is free.
#pragma once

#include <cstdint>

#include "paged.cuh"

namespace ovc {

struct PagesView {
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  int32_t rows, width, pages, page;
  FastDiv by_page;
  unsigned int* status;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The address of `p`, in shared memory, in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}

__device__ __forceinline__ int pages_of(const PagesView& P, int tokens) { return (tokens + P.page - 1) / P.by_page; }

// Length of row b; -1, reported, where it is none that the table can hold.
__device__ __forceinline__ int row_len(const PagesView& P, int b) {
  const int n = P.lens[b];
  if (n >= 0 && n <= P.width * P.page) return n;
  atomicOr(P.status, kPagedBadIndex);
  return -1;
}

// ---------------------------------------------------------------------------
// Release: a CTA a row
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(1024) pages_release_kernel(PagesView P, const int32_t* __restrict__ lens) {
  const int b = blockIdx.x;
  const int to = lens[b], len = row_len(P, b);
  if (to < 0 || to >= len) return;                   // uniform over the CTA
  const int end = pages_of(P, len);
  int32_t* row = P.table + static_cast<int64_t>(b) * P.width;
  for (int c = pages_of(P, to) + threadIdx.x; c < end; c += blockDim.x) {
    const int p = row[c];
    row[c] = -1;
    bool ok = p >= 0 && p < P.pages;
    if (ok && atomicSub(P.refs + p, 1) <= 0) {       // nobody held it: as it was
      atomicAdd(P.refs + p, 1);
      ok = false;
    }
    if (!ok) atomicOr(P.status, kPagedBadIndex);
  }
  __syncthreads();
  if (threadIdx.x == 0) P.lens[b] = to;
}

// ---------------------------------------------------------------------------
// Fork: a CTA a child
// ---------------------------------------------------------------------------
constexpr int kForkThreads = 256;

__global__ void __launch_bounds__(kForkThreads) pages_fork_kernel(PagesView P, const int32_t* __restrict__ parents,
                                                                  const int32_t* __restrict__ children, int32_t n) {
  const int i = blockIdx.x;
  const int a = parents[i], b = children[i];
  if (a < 0 && b < 0) return;                        // padding
  bool bad = a < 0 || a >= P.rows || b < 0 || b >= P.rows;
  // A child that another entry names, as child or as parent, would change under it.
  for (int j = threadIdx.x; j < n; j += kForkThreads) bad |= parents[j] == b || (j != i && children[j] == b);
  bad = __syncthreads_or(bad);
  const int len = bad ? -1 : row_len(P, a);
  if (len < 0 || P.lens[b] != 0) {
    if (threadIdx.x == 0) atomicOr(P.status, kPagedBadIndex);
    return;
  }
  const int32_t* from = P.table + static_cast<int64_t>(a) * P.width;
  int32_t* row = P.table + static_cast<int64_t>(b) * P.width;
  const int end = pages_of(P, len);
  for (int c = threadIdx.x; c < end; c += kForkThreads) {
    const int p = from[c];
    row[c] = p;
    if (p >= 0 && p < P.pages) atomicAdd(P.refs + p, 1);
    else atomicOr(P.status, kPagedBadIndex);
  }
  __syncthreads();
  if (threadIdx.x == 0) P.lens[b] = len;
}

// ---------------------------------------------------------------------------
// Reserve: one cluster.  Every CTA works out for itself how many pages each row
// needs, and counts the free pages of its own part of refs; the counts are
// exchanged once, and then each free page knows its rank among all, and by it the
// row and column that it goes to.
// ---------------------------------------------------------------------------
constexpr int kReserveThreads = 1024;
constexpr int kReserveWarps = kReserveThreads / 32;
constexpr int kReserveRows = 8192;             // most rows of a call: their sums are held in shared memory
constexpr int kReserveClusters = 8;            // most CTAs
constexpr uint32_t kMoves = 0x80000000u;       // in `first`: the row's last page is replaced

struct ReserveSmem {
  uint32_t* start;      // [rows + 1] pages that the rows before need
  uint32_t* first;      // [rows] the column of its first new page
  uint16_t* slot;       // [rows] where `key` holds its last page, or kNoSlot
  int32_t* key;         // [hash] pages that rows want to write to and others hold too
  uint32_t* val;        // [hash] how many such rows << 16 | the highest of them + 1, if those are all holders
  uint32_t hash;
};
constexpr uint32_t kNoSlot = 0xFFFFu;

__host__ __device__ inline uint32_t reserve_hash(int rows) {
  uint32_t h = 64;
  while (h < 2u * static_cast<uint32_t>(rows)) h *= 2;
  return h;
}
__host__ __device__ inline size_t reserve_smem(int rows) {
  const size_t r = (static_cast<size_t>(rows) + 8) / 8 * 8;      // rows + 1 fit
  return r * 10 + reserve_hash(rows) * 8;
}

__global__ void __launch_bounds__(kReserveThreads) pages_reserve_kernel(PagesView P, const int32_t* __restrict__ lens,
                                                                        int32_t* __restrict__ copies) {
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ uint32_t warp_free[kReserveWarps], cta_free[kReserveClusters], scan[kReserveWarps], carry, granted;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  cluster_arrive();                                  // every CTA has begun before another writes to it

  ReserveSmem S;
  S.hash = reserve_hash(P.rows);
  const size_t r8 = (static_cast<size_t>(P.rows) + 8) / 8 * 8;
  S.start = reinterpret_cast<uint32_t*>(raw);
  S.first = S.start + r8;
  S.key = reinterpret_cast<int32_t*>(S.first + r8);
  S.val = reinterpret_cast<uint32_t*>(S.key + S.hash);
  S.slot = reinterpret_cast<uint16_t*>(S.val + S.hash);
  for (uint32_t i = tid; i < S.hash; i += kReserveThreads) {
    S.key[i] = -1;
    S.val[i] = 0;
  }
  if (tid == 0) carry = granted = 0;

  // Free pages of this warp's part.
  const int per_cta = static_cast<int>((static_cast<int64_t>(P.pages) + ctas - 1) / ctas);
  const int per_warp = ((per_cta + kReserveWarps - 1) / kReserveWarps + 31) / 32 * 32;
  const int64_t lo64 = static_cast<int64_t>(rank) * per_warp * kReserveWarps + static_cast<int64_t>(warp) * per_warp;
  const int lo = static_cast<int>(lo64 < P.pages ? lo64 : P.pages), hi = P.pages - lo < per_warp ? P.pages : lo + per_warp;
  uint32_t mine = 0;
#pragma unroll 8
  for (int p = lo + lane; p < hi; p += 32) mine += P.refs[p] == 0;
  mine = __reduce_add_sync(0xFFFFFFFFu, mine);
  if (lane == 0) warp_free[warp] = mine;
  __syncthreads();

  // What each row needs, its last page apart.
  for (int b = tid; b < P.rows; b += kReserveThreads) {
    const int to = lens[b];
    uint32_t fresh = 0, first = 0, slot = kNoSlot;
    int len = to < 0 ? 0 : row_len(P, b);
    bool bad = to > P.width * P.page;
    if (to >= 0 && len >= 0 && to > len && !bad) {
      const int have = pages_of(P, len);
      fresh = pages_of(P, to) - have;
      first = have;
      if (len % P.page) {
        const int last = P.table[static_cast<int64_t>(b) * P.width + have - 1];
        if (last < 0 || last >= P.pages) {
          bad = true;
        } else if (P.refs[last] > 1) {
          uint32_t h = (static_cast<uint32_t>(last) * 2654435761u >> 16) & (S.hash - 1);
          for (;; h = (h + 1) & (S.hash - 1)) {      // at most half of the places are taken
            const int was = atomicCAS(S.key + h, -1, last);
            if (was == -1 || was == last) break;
          }
          atomicAdd(S.val + h, 1u << 16);
          slot = h;
        }
      }
    }
    if (bad) {
      atomicOr(P.status, kPagedBadIndex);
      fresh = 0, first = 0, slot = kNoSlot;
    }
    S.start[b] = fresh;
    S.first[b] = first;
    S.slot[b] = static_cast<uint16_t>(slot);
  }
  __syncthreads();
  // The highest row keeps a page all of whose holders grow.
  for (int b = tid; b < P.rows; b += kReserveThreads) {
    const uint32_t h = S.slot[b];
    if (h == kNoSlot) continue;
    const uint32_t count = S.val[h] >> 16;
    if (static_cast<int>(count) == P.refs[S.key[h]]) atomicMax(S.val + h, count << 16 | (b + 1));
  }
  __syncthreads();
  // Sums over the rows, in order.
  for (int b0 = 0; b0 < P.rows; b0 += kReserveThreads) {
    const int b = b0 + tid;
    uint32_t fresh = 0;
    if (b < P.rows) {
      fresh = S.start[b];
      const uint32_t h = S.slot[b];
      if (h != kNoSlot && (S.val[h] & 0xFFFFu) != static_cast<uint32_t>(b + 1)) {
        ++fresh;
        S.first[b] = (S.first[b] - 1) | kMoves;
      }
      fresh = min(fresh, static_cast<uint32_t>(P.pages) + 1u);
    }
    // Sums stop at 2^31, more than any cache's pages.
    uint32_t x = fresh;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
      if (lane >= d) x = min(x + y, 0x80000000u);
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    uint32_t before = carry;
    for (int w = 0; w < warp; ++w) before = min(before + scan[w], 0x80000000u);
    const uint32_t upto = min(before + x, 0x80000000u);
    __syncthreads();
    if (b < P.rows) S.start[b] = upto - fresh;       // exact up to 2^31, and beyond it nothing is granted
    if (tid == kReserveThreads - 1) {
      carry = upto;
      if (b0 + kReserveThreads >= P.rows) S.start[P.rows] = upto;
    }
    __syncthreads();
  }

  // The free pages before this CTA's, and all of them.
  cluster_wait();
  if (tid < ctas) {
    uint32_t sum = 0;
    for (int w = 0; w < kReserveWarps; ++w) sum += warp_free[w];
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(&cta_free[rank], tid)), "r"(sum) : "memory");
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();                                    // and no CTA reads the rows' state any more
  uint32_t base = 0, total = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    if (c < rank) base += cta_free[c];
    total += cta_free[c];
  }
  for (int w = 0; w < warp; ++w) base += warp_free[w];

  uint32_t most = 0;                                 // pages given out
  for (int b = tid; b < P.rows; b += kReserveThreads) {
    const uint32_t upto = S.start[b + 1];
    if (upto <= total) most = max(most, upto);
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (lane == 0) atomicMax(&granted, most);
  __syncthreads();
  most = granted;

  int32_t* src = copies;
  int32_t* dst = copies + P.rows;
  int32_t* tokens = dst + P.rows;
  for (int p0 = lo; p0 < hi && base < most; p0 += 32) {
    const int p = p0 + lane;
    const bool free = p < hi && P.refs[p] == 0;
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, free);
    const uint32_t r = base + __popc(mask & ((1u << lane) - 1u));
    base += __popc(mask);
    if (!free || r >= most) continue;
    int b = 0, e = P.rows;                           // start[b] <= r < start[e]
    while (e - b > 1) {
      const int m = (b + e) >> 1;
      if (S.start[m] <= r) b = m;
      else e = m;
    }
    const uint32_t first = S.first[b], at = r - S.start[b];
    P.table[static_cast<int64_t>(b) * P.width + (first & ~kMoves) + at] = p;
    P.refs[p] = 1;
    if ((first & kMoves) && at == 0) dst[b] = p;
  }
  for (int b = rank * kReserveThreads + tid; b < P.rows; b += ctas * kReserveThreads) {
    const int to = lens[b], len = P.lens[b];
    const bool fits = S.start[b + 1] <= total;
    const bool moves = fits && (S.first[b] & kMoves);
    const bool grows = fits && to > len && len >= 0 && to <= P.width * P.page;
    int from = -1, n = 0;
    if (moves) {
      from = S.key[S.slot[b]];
      n = len % P.page;
      atomicSub(P.refs + from, 1);
    } else {
      dst[b] = -1;
    }
    src[b] = from;
    tokens[b] = n;
    if (grows && (S.first[b] || S.start[b + 1] > S.start[b])) P.lens[b] = to;
  }
}

}  // namespace ovc
