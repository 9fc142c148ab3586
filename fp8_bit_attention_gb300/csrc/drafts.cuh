// drafts.cuh -- which drafted tokens stay, and the token drawn after them, from
// the target's and the draft's probabilities and given random numbers (see
// include/ovc.h).
#pragma once

#include <cstdint>

#include "pages.cuh"

namespace ovc {

constexpr int kDraftThreads = 256;
constexpr int kDraftWarps = kDraftThreads / 32;
constexpr int kDraftTile = 1024;                 // probabilities whose weights a warp sums at a time, or a power of two times that
constexpr int kDraftTiles = 1024;                // most tiles of a CTA
constexpr int kDraftClusters = 8;

struct DraftParams {
  const int32_t* cu;        // or nullptr: each drafts
  int32_t each, B, N, V;
  const int32_t* drafts;
  const void* target;
  const void* draft;        // or nullptr
  int64_t target_stride, draft_stride;
  const float* accept_u;
  const float* sample_u;
  int32_t* tokens;
  int32_t* accepted;
  int32_t tile_shift;       // a tile is kDraftTile << tile_shift
  unsigned int* status;
};

template <int kType>
__device__ __forceinline__ float prob(const void* p, int64_t i) {
  if (kType == 2) return __ldg(static_cast<const float*>(p) + i);
  const uint32_t w = __ldg(static_cast<const uint16_t*>(p) + i);
  if (kType == 0) return __uint_as_float(w << 16);
  return __half2float(__ushort_as_half(static_cast<uint16_t>(w)));
}

// A sum of 24-bit numbers in 48 bits: hi + lo.  (Sums of a vocabulary in FP32
// would move the borders between tokens by more than the least of them are wide;
// the FP64 units are too few for one addition a probability.)
struct Sum2 {
  float hi = 0.0f, lo = 0.0f;

  // + max(p - q, 0), for p, q >= 0.  d + e = p - q without error where p >= q
  // (Dekker, "A floating-point technique for extending the available precision",
  // 1971), and s + e = hi + d always (Knuth's sum).
  __device__ __forceinline__ void add(float p, float q) {
    const float d = p - q;
    if (!(d > 0.0f)) return;                     // a NaN counts as nothing
    const float e = (p - d) - q;
    const float s = hi + d, t = s - hi;
    lo += ((hi - (s - t)) + (d - t)) + e;
    hi = s;
  }
  __device__ __forceinline__ double value() const { return static_cast<double>(hi) + static_cast<double>(lo); }
};

__device__ __forceinline__ double weight(float p, float q) { return p > q ? static_cast<double>(p) - static_cast<double>(q) : 0.0; }

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
  return x;
}

// Inclusive sum over the block's threads, in their order; `part` has a place for
// each warp, and the block's sum is returned in `all`.
__device__ __forceinline__ double block_scan(double x, double* part, double* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const double y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  double before = 0.0, sum = 0.0;
#pragma unroll
  for (int w = 0; w < kDraftWarps; ++w) {
    if (w == warp) before = sum;
    sum += part[w];
  }
  __syncthreads();
  *all = sum;
  return before + x;
}

template <int kType>
__global__ void __launch_bounds__(kDraftThreads) verify_drafts_kernel(DraftParams P) {
  __shared__ double tile_own[kDraftTiles], tile_sum[kDraftTiles], part[kDraftWarps], cta_sum[kDraftClusters];
  __shared__ uint32_t stop;
  __shared__ int first_over, last_some;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const int b = blockIdx.x / ctas;
  cluster_arrive();

  const int a0 = P.cu ? P.cu[b] : b * P.each, a1 = P.cu ? P.cu[b + 1] : a0 + P.each;
  if (a0 < 0 || a1 < a0 || a1 > P.N) {                // all CTAs of the cluster
    if (rank == 0 && tid == 0) {
      P.accepted[b] = 0;
      atomicOr(P.status, kPagedBadIndex);
    }
    cluster_wait();
    return;
  }
  const int n = a1 - a0;
  const int64_t row0 = static_cast<int64_t>(a0) + b;  // of the target's probabilities

  // The first draft that does not stay: 2 i, or 2 i + 1 where there is none at i.
  if (tid == 0) stop = 2u * n + 1u;
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += kDraftThreads) {
    const int i = i0 + tid;
    if (i < n) {
      const int x = P.drafts[a0 + i];
      if (x < 0 || x >= P.V) {
        atomicMin(&stop, 2u * i + 1u);
        if (x >= P.V) atomicOr(P.status, kPagedBadIndex);
      } else {
        const float p = prob<kType>(P.target, (row0 + i) * P.target_stride + x);
        const float q = P.draft ? prob<kType>(P.draft, static_cast<int64_t>(a0 + i) * P.draft_stride + x) : 1.0f;
        // 24 by 24 bits: exact in 64
        if (!(static_cast<double>(P.accept_u[a0 + i]) * q < p)) atomicMin(&stop, 2u * i);
      }
    }
    __syncthreads();
    if (stop < 2u * (i0 + kDraftThreads)) break;
    __syncthreads();
  }
  const int kept = stop >> 1;
  const bool rejected = !(stop & 1u);
  if (rank == 0) {
    for (int i = tid; i <= n; i += kDraftThreads)
      if (i != kept) P.tokens[row0 + i] = i < kept ? P.drafts[a0 + i] : -1;
    if (tid == 0) P.accepted[b] = kept;
  }

  // Sums of the weights of this CTA's part of the vocabulary, tile by tile.
  const uint8_t* pr = static_cast<const uint8_t*>(P.target) + (row0 + kept) * P.target_stride * (kType == 2 ? 4 : 2);
  const uint8_t* qr = nullptr;
  int out = -1;                                       // a token that counts for nothing
  if (rejected) {
    if (P.draft) qr = static_cast<const uint8_t*>(P.draft) + static_cast<int64_t>(a0 + kept) * P.draft_stride * (kType == 2 ? 4 : 2);
    else out = P.drafts[a0 + kept];
  }
  const int tile = kDraftTile << P.tile_shift;
  const int all_tiles = (P.V + tile - 1) / tile, per = (all_tiles + ctas - 1) / ctas;
  const int t0 = min(static_cast<int>(rank) * per, all_tiles), tiles = min(per, all_tiles - t0);
  double mine = 0.0, total = 0.0;
  for (int pass = 0;; ++pass) {
    for (int t = warp; t < tiles; t += kDraftWarps) {
      Sum2 s;
      const int64_t v0 = static_cast<int64_t>(t0 + t) * tile;
      const int64_t v1 = v0 + tile < P.V ? v0 + tile : P.V;
#pragma unroll 8
      for (int64_t v = v0 + lane; v < v1; v += 32) {
        const float q = qr ? prob<kType>(qr, v) : v == out ? INFINITY : 0.0f;
        s.add(prob<kType>(pr, v), q);
      }
      const double w = warp_sum(s.value());
      if (lane == 0) tile_own[t] = w;
    }
    __syncthreads();
    mine = 0.0;
    for (int k = 0; k < kDraftTiles; k += kDraftThreads) {       // running sums over the tiles
      if (k >= tiles) break;
      const int t = k + tid;
      double all;
      const double x = block_scan(t < tiles ? tile_own[t] : 0.0, part, &all);
      if (t < tiles) tile_sum[t] = mine + x;
      mine += all;
    }
    cluster_wait();
    if (tid < ctas)
      asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(cluster_addr(&cta_sum[rank], tid)), "d"(mine) : "memory");
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    total = 0.0;
    for (uint32_t c = 0; c < ctas; ++c) total += cta_sum[c];
    if (total > 0.0 || (!qr && out < 0) || pass) break;
    // Nothing is left of p - q: p itself.
    cluster_arrive();
    qr = nullptr;
    out = -1;
  }

  // The CTA within whose part the running sum first exceeds u * total, or, where
  // rounding (or u >= 1) leaves none, the last that holds any weight.
  const double goal = static_cast<double>(P.sample_u[b]) * total;
  int owner = -1, last = 0;
  double before = 0.0, sum = 0.0;
  for (uint32_t c = 0; c < ctas; ++c) {
    if (cta_sum[c] > 0.0) last = c;
    sum += cta_sum[c];
    if (owner < 0 && cta_sum[c] > 0.0 && sum > goal) owner = c;
    if (owner < 0 && c < rank) before = sum;
  }
  if (!(total > 0.0)) {
    if (rank == 0 && tid == 0) P.tokens[row0 + kept] = -1;
    return;
  }
  if (static_cast<int>(rank) != (owner < 0 ? last : owner)) return;
  if (owner < 0) {
    before = 0.0;
    for (uint32_t c = 0; c < rank; ++c) before += cta_sum[c];
  }
  if (tid == 0) {
    first_over = kDraftTiles;
    last_some = 0;
  }
  __syncthreads();
  for (int t = tid; t < tiles; t += kDraftThreads) {
    if (tile_own[t] > 0.0) {
      atomicMax(&last_some, t);
      if (before + tile_sum[t] > goal) atomicMin(&first_over, t);
    }
  }
  __syncthreads();
  const int t = first_over < kDraftTiles ? first_over : last_some;
  if (t) before += tile_sum[t - 1];
  __syncthreads();
  if (tid == 0) {
    first_over = 0x7FFFFFFF;
    last_some = -1;
  }
  __syncthreads();
  // Its probabilities in order, a few consecutive ones a thread.
  const int64_t v0 = static_cast<int64_t>(t0 + t) * tile;
  const int64_t v1 = v0 + tile < P.V ? v0 + tile : P.V;
  for (int64_t k = v0; k < v1; k += 4 * kDraftThreads) {
    double w[4], own = 0.0, all;
    const int64_t v = k + 4 * tid;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = 0.0;
      if (v + j < v1) w[j] = weight(prob<kType>(pr, v + j), qr ? prob<kType>(qr, v + j) : v + j == out ? INFINITY : 0.0f);
      own += w[j];
    }
    double x = before + (block_scan(own, part, &all) - own);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x += w[j];
      if (w[j] > 0.0) {
        atomicMax(&last_some, static_cast<int>(v + j));
        if (x > goal) {
          atomicMin(&first_over, static_cast<int>(v + j));
          break;
        }
      }
    }
    __syncthreads();
    if (first_over != 0x7FFFFFFF) break;
    before += all;
  }
  if (tid == 0) P.tokens[row0 + kept] = first_over != 0x7FFFFFFF ? first_over : last_some;
}

}  // namespace ovc
