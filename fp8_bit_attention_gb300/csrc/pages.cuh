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
// For a later cluster_wait() that only asks whether the other CTAs have come here.
__device__ __forceinline__ void cluster_begun() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
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
// Release: a CTA a row.  Bound by latency (length, entry, its count): 3.2 us for a
// page or none a row, 256 rows dropping up to 2048 pages 4.6 us; 960 rows x 450 pages,
// 15 rows to a page, 7.2 us.  (Counts looked at before they are taken down, and not
// waited for then: 3.0, 4.1 and 7.5 us.)
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(1024) pages_release_kernel(PagesView P, const int32_t* __restrict__ lens) {
  const int b = blockIdx.x;
  const int to = lens[b];
  const int len = to < 0 ? -1 : row_len(P, b);
  if (to >= len || to < 0) return;                   // uniform over the CTA
  const int end = pages_of(P, len);
  int32_t* row = P.table + static_cast<int64_t>(b) * P.width;
  for (int c0 = pages_of(P, to) + threadIdx.x; c0 < end; c0 += 4 * blockDim.x) {
    int p[4], held[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = c0 + j * blockDim.x < end ? row[c0 + j * blockDim.x] : -1;
    // By what the count was, as others may give the page back at the same time.
#pragma unroll
    for (int j = 0; j < 4; ++j) held[j] = p[j] >= 0 && p[j] < P.pages ? atomicSub(P.refs + p[j], 1) : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c0 + j * blockDim.x >= end) break;
      row[c0 + j * blockDim.x] = -1;
      if (held[j] > 0) continue;
      if (p[j] >= 0 && p[j] < P.pages) atomicAdd(P.refs + p[j], 1);
      atomicOr(P.status, kPagedBadIndex);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) P.lens[b] = to;
}

// ---------------------------------------------------------------------------
// Fork: a CTA a child, which also looks for itself in both lists (at most 8192
// entries each).  960 children of 450 pages each 5.9 us (128 and 512 threads: 6.2
// and 7.4), 32 children 3 us.
// ---------------------------------------------------------------------------
constexpr int kForkThreads = 256;

__global__ void __launch_bounds__(kForkThreads) pages_fork_kernel(PagesView P, const int32_t* __restrict__ parents,
                                                                  const int32_t* __restrict__ children, int32_t n) {
  const int i = blockIdx.x;
  const int a = parents[i], b = children[i];
  if (a < 0 && b < 0) return;                        // padding
  bool bad = a < 0 || a >= P.rows || b < 0 || b >= P.rows;
  // A child that another entry names, as child or as parent, would change under it.
#pragma unroll 4
  for (int j = threadIdx.x; j < n; j += kForkThreads) bad |= (parents[j] == b) | ((j != i) & (children[j] == b));
  bad = __syncthreads_or(bad);
  const int len = bad ? -1 : row_len(P, a);
  if (len < 0 || P.lens[b] != 0) {
    if (threadIdx.x == 0) atomicOr(P.status, kPagedBadIndex);
    return;
  }
  const int32_t* from = P.table + static_cast<int64_t>(a) * P.width;
  int32_t* row = P.table + static_cast<int64_t>(b) * P.width;
  const int end = pages_of(P, len);
  for (int c0 = threadIdx.x; c0 < end; c0 += 4 * kForkThreads) {
    int p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = c0 + j * kForkThreads < end ? from[c0 + j * kForkThreads] : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c0 + j * kForkThreads >= end) break;
      row[c0 + j * kForkThreads] = p[j];
      if (p[j] >= 0 && p[j] < P.pages) atomicAdd(P.refs + p[j], 1);
      else atomicOr(P.status, kPagedBadIndex);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) P.lens[b] = len;
}

// ---------------------------------------------------------------------------
// Reserve: one cluster.  Every CTA works out for itself how many pages each row
// needs.  The pages are cut into chunks, dealt out to the CTAs in turn, so that
// the lowest ones, where the free pages are taken, are spread over all of them;
// the chunks' numbers of free pages are exchanged once, and then each free page
// knows its rank among all, and by it the row and column that it goes to.
//
// Bound by its chain of steps, each a latency or a barrier: 40 rows, 8192 pages
// 6.4 us, 64 rows, 32768 pages 7.3 us; 1024 rows that all copy, 131072 pages 11 us; 93000 pages given out of
// 600000 16 us (2.4 MB of refs read at least once: 0.4 us).
// Tried: pages dealt out in contiguous parts, 57 us for the last (the lowest pages,
// which are the ones given out, all in one CTA); a search in shared memory for each
// free page's row 26 us for the 1024 rows.
// ---------------------------------------------------------------------------
constexpr int kReserveThreads = 1024;
constexpr int kReserveWarps = kReserveThreads / 32;
constexpr int kReserveRows = 8192;             // most rows of a state: their sums are held in shared memory
constexpr int kReserveClusters = 16;           // most CTAs
constexpr int kReserveWords = 4;               // words of 32 pages of a warp in a block
constexpr int kReserveBlock = kReserveWarps * kReserveWords * 32;  // pages that a CTA deals out together
constexpr int kReserveAhead = 4;               // blocks on their way at a time where they are counted
constexpr int kReserveChunks = 1024;           // most chunks: blocks, or a power of two of them each
constexpr uint32_t kMoves = 0x80000000u;       // in `first`: the row's last page is replaced

struct ReserveOut {       // [rows] each: what has to be copied
  int32_t* src;
  int32_t* dst;
  int32_t* tokens;
};

struct ReserveSmem {
  uint32_t* start;      // [rows + 1] pages that the rows before need
  uint32_t* first;      // [rows] the column of its first new page
  uint16_t* slot;       // [rows] where `key` holds its last page, or kNoSlot
  int32_t* key;         // [hash] pages that rows want to write to and others hold too
  uint32_t* val;        // [hash] how many such rows << 16 | the highest of them + 1, if those are all holders
};
constexpr uint32_t kNoSlot = 0xFFFFu;

// Places for the pages of `rows` rows, at most half of them taken.
__host__ inline uint32_t reserve_hash(int rows) {
  uint32_t h = 64;
  while (h < 2u * static_cast<uint32_t>(rows)) h *= 2;
  return h;
}
__host__ __device__ inline int reserve_room(int rows) { return (rows + 8) / 8 * 8; }     // rows + 1 fit
__host__ inline size_t reserve_smem(int rows) { return static_cast<size_t>(reserve_room(rows)) * 10 + reserve_hash(rows) * 8; }

// refs of a block of pages from p0 on.  Word m of 32 pages is word m / 32 of warp
// m % 32, so that the lowest free pages are spread over the warps.
struct Block {
  int32_t x[kReserveWords];
  __device__ __forceinline__ void load(const PagesView& P, int p0, int end) {
    const int p = p0 + static_cast<int>(threadIdx.x);
#pragma unroll
    for (int j = 0; j < kReserveWords; ++j) x[j] = p + kReserveThreads * j < end ? P.refs[p + kReserveThreads * j] : 1;
  }
  // Free ones among this lane's.
  __device__ __forceinline__ uint32_t count() const {
    uint32_t n = 0;
#pragma unroll
    for (int j = 0; j < kReserveWords; ++j) n += x[j] == 0;
    return n;
  }
  // In lane j < kReserveWords: which pages of the warp's word j are free.
  __device__ __forceinline__ uint32_t free() const {
    uint32_t f = 0;
#pragma unroll
    for (int j = 0; j < kReserveWords; ++j) {
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, x[j] == 0);
      if (static_cast<int>(threadIdx.x & 31) == j) f = m;
    }
    return f;
  }
};

// The last row with start <= r, from row b on that fulfils it, for ascending r
// over the lanes: among the next 32 rows by exchanging their starts, which takes
// a third of the time of a search in shared memory.
__device__ __forceinline__ int row_of_rank(const uint32_t* start, int b, int rows, uint32_t r) {
  const int next = b + 1 + static_cast<int>(threadIdx.x & 31);
  const uint32_t s = next < rows ? start[next] : 0xFFFFFFFFu;
  int n = 0;
#pragma unroll
  for (int step = 16; step; step >>= 1)
    if (__shfl_sync(0xFFFFFFFFu, s, n + step - 1) <= r) n += step;
  if (__shfl_sync(0xFFFFFFFFu, s, n) <= r) ++n;
  if (n < 32) return b + n;
  int e = rows;
  b += 32;
  while (e - b > 1) {
    const int m = (b + e) >> 1;
    if (start[m] <= r) b = m;
    else e = m;
  }
  return b;
}

__device__ __forceinline__ uint32_t capped_sum(uint32_t a, uint32_t b) { return min(a + b, 0x7FFFFFFFu); }

__global__ void __launch_bounds__(kReserveThreads, 1) pages_reserve_kernel(PagesView P, const int32_t* __restrict__ lens,
                                                                        ReserveOut out, int chunk_shift, uint32_t hash) {
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ uint32_t word_base[kReserveWarps * kReserveWords], free_in[kReserveChunks], scan[kReserveWarps], granted;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_rank(), ctas = cluster_size();
  // The first row of each thread, and the CTA's first pages, are on their way
  // while shared memory is set up.
  int to = -1, len = 0;
  if (tid < P.rows) to = lens[tid], len = P.lens[tid];
  const int chunk = kReserveBlock << chunk_shift, chunks = (P.pages - 1) / chunk + 1;
  const int blocks = ((chunks - rank + ctas - 1) / ctas) << chunk_shift;           // the CTA's, of all its chunks
  const auto chunk_of = [&](int i) { return rank + (i >> chunk_shift) * ctas; };   // of its block i
  Block ahead[kReserveAhead];
  const auto fetch = [&](int i) {
#pragma unroll
    for (int j = 0; j < kReserveAhead; ++j)
      ahead[j].load(P, chunk_of(i + j) * chunk + ((i + j) & ((1 << chunk_shift) - 1)) * kReserveBlock, i + j < blocks ? P.pages : 0);
  };
  fetch(0);

  ReserveSmem S;
  const int room = reserve_room(P.rows);
  S.start = reinterpret_cast<uint32_t*>(raw);
  S.first = S.start + room;
  S.key = reinterpret_cast<int32_t*>(S.first + room);
  S.val = reinterpret_cast<uint32_t*>(S.key + hash);
  S.slot = reinterpret_cast<uint16_t*>(S.val + hash);
  for (uint32_t i = tid; i < hash; i += kReserveThreads) {
    S.key[i] = -1;
    S.val[i] = 0;
  }
  if (tid == 0) granted = 0;
  for (int k = tid; k < chunks; k += kReserveThreads) free_in[k] = 0;
  __syncthreads();
  if (ctas > 1) cluster_arrive();                    // others may write to free_in from here on

  // What each row needs, its last page apart.
  for (int b = tid; b < P.rows; b += kReserveThreads) {
    if (b != tid) to = lens[b], len = P.lens[b];
    uint32_t fresh = 0, first = 0, slot = kNoSlot;
    if (to >= 0) {
      const int most = P.width * P.page;
      bool bad = to > most || len < 0 || len > most;
      if (!bad && to > len) {
        const int have = pages_of(P, len);
        fresh = pages_of(P, to) - have;
        first = have;
        if (len != have * P.page) {
          const int last = P.table[static_cast<int64_t>(b) * P.width + have - 1];
          if (last < 0 || last >= P.pages) {
            bad = true;
          } else if (P.refs[last] > 1) {
            uint32_t h = (static_cast<uint32_t>(last) * 2654435761u >> 16) & (hash - 1);
            for (;; h = (h + 1) & (hash - 1)) {
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
        fresh = 0, first = 0;
      }
    }
    S.start[b] = fresh;
    S.first[b] = first;
    S.slot[b] = static_cast<uint16_t>(slot);
  }

  // The free pages of this CTA's chunks; of the first block each warp keeps which.
  const uint32_t mine = ahead[0].free();
  for (int i = 0; i < blocks; i += kReserveAhead) {
    if (i) fetch(i);
#pragma unroll
    for (int j = 0; j < kReserveAhead; ++j) {
      const uint32_t n = __reduce_add_sync(0xFFFFFFFFu, ahead[j].count());
      if (lane == 0 && n) atomicAdd(&free_in[chunk_of(i + j)], n);
    }
  }
  __syncthreads();
  // The highest row keeps a page all of whose holders grow.
  for (int b = tid; b < P.rows; b += kReserveThreads) {
    const uint32_t h = S.slot[b];
    if (h == kNoSlot) continue;
    const int count = S.val[h] >> 16, refs = P.refs[S.key[h]];
    if (count == refs) atomicMax(S.val + h, static_cast<uint32_t>(count) << 16 | (b + 1));
    if (count > refs) {                              // more rows than it has holders: they stay
      atomicOr(P.status, kPagedBadIndex);
      S.start[b] = 0, S.first[b] = 0, S.slot[b] = static_cast<uint16_t>(kNoSlot);
    }
  }
  __syncthreads();
  // Sums over the rows, in order.  They stop at 2^31 - 1, more than any cache's pages
  // (2^27), and two of them fit 32 bits: a start is exact below that, and beyond it
  // nothing is granted.
  uint32_t carry = 0;
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
    uint32_t x = fresh;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
      if (lane >= d) x = capped_sum(x, y);
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    uint32_t w = scan[lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, w, d);
      if (lane >= d) w = capped_sum(w, y);
    }
    const uint32_t all = __shfl_sync(0xFFFFFFFFu, w, 31), before = __shfl_sync(0xFFFFFFFFu, w, (warp + 31) & 31);
    x = capped_sum(capped_sum(carry, warp ? before : 0u), x);
    carry = capped_sum(carry, all);
    if (b < P.rows) S.start[b] = x - fresh;
    if (b == P.rows - 1) S.start[P.rows] = x;
    __syncthreads();
  }

  // The other CTAs' counts.
  if (ctas > 1) {
    cluster_wait();
    for (int i = tid; i < chunks * ctas; i += kReserveThreads) {
      const int k = i / ctas, other = i - k * ctas;
      if (k % ctas == rank && other != rank)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(&free_in[k], other)), "r"(free_in[k]) : "memory");
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();                                  // and no CTA reads the rows' state any more
  }
  auto free_below = [&](int k) {                     // in the chunks before k
    uint32_t sum = 0;
    for (int i = lane; i < k; i += 32) sum += free_in[i];
    return __reduce_add_sync(0xFFFFFFFFu, sum);
  };
  const uint32_t total = free_below(chunks);

  uint32_t most = 0;                                 // pages given out
  for (int b = tid; b < P.rows; b += kReserveThreads) {
    const uint32_t upto = S.start[b + 1];
    if (upto <= total) most = max(most, upto);
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (lane == 0) atomicMax(&granted, most);
  __syncthreads();
  most = granted;

  // The rows: which page is copied, and the lengths.
  for (int b = rank * kReserveThreads + tid; b < P.rows; b += ctas * kReserveThreads) {
    const bool fits = S.start[b + 1] <= total;
    const uint32_t first = S.first[b];
    int from = -1, n = 0;
    if (first || S.start[b + 1] > S.start[b]) {      // it wants to grow
      if (fits && (first & kMoves)) {
        from = S.key[S.slot[b]];
        n = P.lens[b] - static_cast<int>(first & ~kMoves) * P.page;
        atomicSub(P.refs + from, 1);
      }
      if (fits) P.lens[b] = lens[b];
    }
    out.src[b] = from;
    out.tokens[b] = n;
    if (from < 0) out.dst[b] = -1;
  }
  // The pages.
  for (int k = rank; k < chunks; k += ctas) {
    uint32_t base = free_below(k);
    if (base >= most) break;                         // the whole CTA
    const int end = min(P.pages, (k + 1) * chunk);
    for (int p0 = k * chunk; p0 < end && base < most; p0 += kReserveBlock) {
      uint32_t f = mine;
      if (p0 != rank * chunk) {
        Block x;
        x.load(P, p0, P.pages);
        f = x.free();
      }
      // Ranks of the words: sums over all of the block's, in their order.
      __syncthreads();
      if (lane < kReserveWords) word_base[lane * kReserveWarps + warp] = __popc(f);
      __syncthreads();
      uint32_t x = tid < kReserveWarps * kReserveWords ? word_base[tid] : 0u;
      const uint32_t own = x;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
        if (lane >= d) x += y;
      }
      if (lane == 31) scan[warp] = x;
      __syncthreads();
      x += base + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? scan[lane] : 0u);
      base += __reduce_add_sync(0xFFFFFFFFu, scan[lane]);
      if (tid < kReserveWarps * kReserveWords) word_base[tid] = x - own;
      __syncthreads();
      const uint32_t at = word_base[(lane & (kReserveWords - 1)) * kReserveWarps + warp];
      int row = 0;                                   // start[row] <= ranks to come
#pragma unroll 1
      for (uint32_t words = __ballot_sync(0xFFFFFFFFu, f && at < most); words; words &= words - 1) {
        const int j = __ffs(words) - 1;
        const uint32_t w = __shfl_sync(0xFFFFFFFFu, f, j);
        const uint32_t r = __shfl_sync(0xFFFFFFFFu, at, j) + __popc(w & ((1u << lane) - 1u));
        // Most often the whole word goes to one row.
        const bool one = row + 1 >= P.rows || __shfl_sync(0xFFFFFFFFu, r, 31) < S.start[row + 1];
        const int b = one ? row : row_of_rank(S.start, row, P.rows, r);
        if (w >> lane & 1u && r < most) {
          const int p = p0 + 32 * (j * kReserveWarps + warp) + lane;
          const uint32_t first = S.first[b], col = r - S.start[b];
          P.table[static_cast<int64_t>(b) * P.width + (first & ~kMoves) + col] = p;
          P.refs[p] = 1;
          if ((first & kMoves) && col == 0) out.dst[b] = p;
        }
        row = __shfl_sync(0xFFFFFFFFu, b, 0);
      }
    }
  }
}

}  // namespace ovc
