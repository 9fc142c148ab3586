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
  for (int c0 = pages_of(P, to) + threadIdx.x; c0 < end; c0 += 4 * blockDim.x) {
    int p[4];
    bool ok[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = c0 + j * blockDim.x < end ? row[c0 + j * blockDim.x] : -2;
#pragma unroll
    for (int j = 0; j < 4; ++j) ok[j] = p[j] >= 0 && p[j] < P.pages && P.refs[p[j]] > 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c0 + j * blockDim.x >= end) break;
      row[c0 + j * blockDim.x] = -1;
      if (ok[j]) atomicSub(P.refs + p[j], 1);        // (a use of what it returns would be waited for)
      else atomicOr(P.status, kPagedBadIndex);
    }
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
// ---------------------------------------------------------------------------
constexpr int kReserveThreads = 1024;
constexpr int kReserveWarps = kReserveThreads / 32;
constexpr int kReserveRows = 8192;             // most rows of a call: their sums are held in shared memory
constexpr int kReserveClusters = 8;            // most CTAs
constexpr int kReserveBatch = 4;               // loads of 16 bytes a lane at a time
constexpr int kReserveChunk = kReserveThreads * 4 * kReserveBatch;   // pages, or a power of two times that
constexpr int kReserveChunks = 1024;           // most of them
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

// The last row b with start[b] <= r, from one on that fulfils it; rows give way
// slowly as ranks rise.
__device__ __forceinline__ int row_of_rank(const uint32_t* start, int b, int rows, uint32_t r) {
  if (b + 1 >= rows || r < start[b + 1]) return b;
  int e = rows;
  while (e - b > 1) {
    const int m = (b + e) >> 1;
    if (start[m] <= r) b = m;
    else e = m;
  }
  return b;
}

// Bits k of f[j]: page p0 + 128 j + 4 lane + k, of those below hi, is free.
__device__ __forceinline__ void free_of(const PagesView& P, int p0, int hi, uint32_t (&f)[kReserveBatch]) {
  int4 x[kReserveBatch];
#pragma unroll
  for (int j = 0; j < kReserveBatch; ++j) {
    const int p = p0 + 128 * j + 4 * (threadIdx.x & 31);
    x[j] = make_int4(1, 1, 1, 1);
    if (p + 3 < hi) {
      x[j] = *reinterpret_cast<const int4*>(P.refs + p);
    } else {
      if (p < hi) x[j].x = P.refs[p];
      if (p + 1 < hi) x[j].y = P.refs[p + 1];
      if (p + 2 < hi) x[j].z = P.refs[p + 2];
    }
  }
#pragma unroll
  for (int j = 0; j < kReserveBatch; ++j)
    f[j] = (x[j].x == 0) | (x[j].y == 0) << 1 | (x[j].z == 0) << 2 | (x[j].w == 0) << 3;
}

__global__ void __launch_bounds__(kReserveThreads) pages_reserve_kernel(PagesView P, const int32_t* __restrict__ lens,
                                                                        int32_t* __restrict__ copies, int chunk_shift) {
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ uint32_t warp_free[kReserveWarps], free_in[kReserveChunks], scan[kReserveWarps], carry, granted;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
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

  const int chunk = kReserveChunk << chunk_shift, part = chunk / kReserveWarps;    // of a CTA, of a warp
  const int chunks = static_cast<int>((static_cast<int64_t>(P.pages) + chunk - 1) / chunk);
  for (int k = tid; k < chunks; k += kReserveThreads) free_in[k] = 0;
  __syncthreads();
  cluster_arrive();                                  // others may write to free_in from here on
  // The free pages of this CTA's chunks.
  auto count = [&](int lo, int hi) {                 // of a warp's pages
    uint32_t n = 0, f[kReserveBatch];
    for (int p = lo; p < hi; p += 128 * kReserveBatch) {
      free_of(P, p, hi, f);
#pragma unroll
      for (int j = 0; j < kReserveBatch; ++j) n += __popc(f[j]);
    }
    return __reduce_add_sync(0xFFFFFFFFu, n);
  };
  auto place = [&](int k, int& lo, int& hi) {        // a warp's pages of chunk k
    lo = k * chunk + warp * part;                    // below 2^27 + 2^15 << 10
    hi = min(P.pages, lo + part);
  };
  for (int k = rank; k < chunks; k += ctas) {
    int lo, hi;
    place(k, lo, hi);
    const uint32_t n = count(lo, hi);
    if (lane == 0 && n) atomicAdd(&free_in[k], n);
  }

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

  // The other CTAs' counts.
  cluster_wait();
  for (int i = tid; i < chunks * static_cast<int>(ctas); i += kReserveThreads) {
    const uint32_t k = i / ctas, to = i - k * ctas;
    if (k % ctas == rank && to != rank)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(&free_in[k], to)), "r"(free_in[k]) : "memory");
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();                                    // and no CTA reads the rows' state any more
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

  int32_t* src = copies;
  int32_t* dst = copies + P.rows;
  int32_t* tokens = dst + P.rows;
  for (int k = rank; k < chunks; k += ctas) {
    uint32_t base = free_below(k);
    if (base >= most) break;                         // the whole CTA
    int lo, hi;
    place(k, lo, hi);
    const uint32_t n = count(lo, hi);
    if (lane == 0) warp_free[warp] = n;
    __syncthreads();
    base += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? warp_free[lane] : 0u);
    __syncthreads();
    int row = 0;                                     // start[row] <= base
    for (int p0 = lo; p0 < hi && base < most; p0 += 128 * kReserveBatch) {
      uint32_t f[kReserveBatch];
      free_of(P, p0, hi, f);
#pragma unroll
      for (int j = 0; j < kReserveBatch; ++j) {
        if (base >= most) break;
        row = row_of_rank(S.start, row, P.rows, base);
        uint32_t r = base;                           // rank of this lane's first free page
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t mask = __ballot_sync(0xFFFFFFFFu, f[j] >> i & 1u);
          r += __popc(mask & ((1u << lane) - 1u));
          base += __popc(mask);
        }
        int b = row;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if ((f[j] >> i & 1u) && r < most) {
            const int p = p0 + 128 * j + 4 * lane + i;
            b = row_of_rank(S.start, b, P.rows, r);
            const uint32_t first = S.first[b], at = r - S.start[b];
            P.table[static_cast<int64_t>(b) * P.width + (first & ~kMoves) + at] = p;
            P.refs[p] = 1;
            if ((first & kMoves) && at == 0) dst[b] = p;
          }
          r += f[j] >> i & 1u;
        }
        __syncwarp();
      }
    }
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
