// drafts.cuh -- which drafted tokens stay, and the token drawn after them, from
// the target's and the draft's probabilities and given random numbers (see
// include/ovc.h).
#pragma once

#include <cstdint>

#include "pages.cuh"

namespace ovc {

// Threads of a CTA: without the draft's probabilities a thread holds half as much.
template <bool kDraft>
constexpr int kDraftThreads = kDraft ? 256 : 512;
constexpr int kDraftLoads = 8;                   // of 16 bytes a lane and row
template <int kType>
constexpr int kDraftTile = 32 * kDraftLoads * (kType == 2 ? 4 : 8);   // probabilities whose weights a warp sums into one, or a power of two times that
constexpr int kDraftTiles = 1024;                // most tiles of a CTA
constexpr int kDraftClusters = 8;                // most CTAs of a sequence
constexpr int kDraftCtas = 2;                    // of an SM

struct DraftParams {
  const int32_t* cu;        // or nullptr: each drafts
  int32_t each, N, V;
  const int32_t* drafts;
  const void* target;
  const void* draft;        // or nullptr
  int64_t target_stride, draft_stride;
  const float* accept_u;
  const float* sample_u;
  int32_t* tokens;
  int32_t* accepted;
  int32_t tile_shift;       // a tile is kDraftTile<type> << tile_shift
  unsigned int* status;
};

template <int kType>
__device__ __forceinline__ float prob(const void* p, int64_t i) {
  if (kType == 2) return __ldg(static_cast<const float*>(p) + i);
  const uint32_t w = __ldg(static_cast<const uint16_t*>(p) + i);
  if (kType == 0) return __uint_as_float(w << 16);
  return __half2float(__ushort_as_half(static_cast<uint16_t>(w)));
}

// Sums are pairs hi + lo of FP32 numbers, 48 bits: sums of a vocabulary in FP32
// would move the borders between tokens by more than the least of them are wide,
// and the FP64 units (2 additions a cycle and SM) would take several times as long
// as the memory.
//
// What sums are off by at most, in units of 2^-48 (half a step, squared) of the total:
// a lane's K weights in each of its four sums K^2 / 2 + 4 K (the lower part grows by a
// step's half with each, and is rounded each time); the 7 merges up to a tile's sum
// 14 (K + 8); its place among the tiles and CTAs 2 K + 45, and 3 for every 32 tiles; the
// last search 66.  A running sum against u times the total: K^2 + 40 K + 380.  K = 2 j + 1
// where a lane loads j times 16 bytes of 16-bit weights (V > 256 (j - 1) - 8), j + 1 of
// FP32 (V > 128 (j - 1) - 4), 16 * 2^s + 1 at most in tiles of 2^s lines (V > 2^19 *
// 2^s): less than 4 (V + 128) for every V.
struct FF {
  float hi, lo;
};

// hi + lo = a + b without error (Knuth, "The Art of Computer Programming" 2, 4.2.2).
__device__ __forceinline__ FF two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ FF operator+(const FF& a, const FF& b) {
  FF s = two_sum(a.hi, b.hi);
  s.lo += a.lo + b.lo;
  const float hi = s.hi + s.lo;                  // |lo| <= half a step of hi again
  return {hi, s.lo - (hi - s.hi)};
}
// The same with a lower part that may have grown to a few steps of the upper one.
__device__ __forceinline__ FF near_sum(const FF& a, const FF& b) {
  FF s = two_sum(a.hi, b.hi);
  s.lo += a.lo + b.lo;
  return s;
}
__device__ __forceinline__ bool above(const FF& a, const FF& b) { return (a.hi - b.hi) + (a.lo - b.lo) > 0.0f; }

// max(p - q, 0), NaN: 0.  Where p >= q >= 0 the lower part makes it exact (Dekker,
// "A floating-point technique for extending the available precision", 1971).
__device__ __forceinline__ FF weight(float p, float q) {
  const float d = p - q;
  return d > 0.0f ? FF{d, (p - d) - q} : FF{0.0f, 0.0f};
}

__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t add_pairs(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub_pairs(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Two sums, of every other weight, by instructions that add two FP32 numbers at once.
struct Sums {
  uint64_t hi = 0, lo = 0;

  __device__ __forceinline__ void add(uint64_t d) {
    const uint64_t s = add_pairs(hi, d), t = sub_pairs(s, hi);
    lo = add_pairs(lo, add_pairs(sub_pairs(hi, sub_pairs(s, t)), sub_pairs(d, t)));
    hi = s;
  }
  // max(p - q, 0): fmaxf drops a NaN.
  __device__ __forceinline__ void add(uint64_t p, uint64_t q) {
    const uint64_t c = sub_pairs(p, q);
    const float2 x = unpair(c), y = unpair(sub_pairs(sub_pairs(p, c), q));
    const uint64_t d = pair(fmaxf(x.x, 0.0f), fmaxf(x.y, 0.0f));
    const uint64_t e = pair(x.x > 0.0f ? y.x : 0.0f, x.y > 0.0f ? y.y : 0.0f);
    const uint64_t s = add_pairs(hi, d), t = sub_pairs(s, hi);
    lo = add_pairs(lo, add_pairs(add_pairs(sub_pairs(hi, sub_pairs(s, t)), sub_pairs(d, t)), e));
    hi = s;
  }
  // Both sums and those of c.
  __device__ __forceinline__ FF sum(const Sums& c) const {
    const uint64_t s = add_pairs(hi, c.hi), t = sub_pairs(s, hi);
    const float2 h = unpair(s);
    const float2 l = unpair(add_pairs(add_pairs(lo, c.lo), add_pairs(sub_pairs(hi, sub_pairs(s, t)), sub_pairs(c.hi, t))));
    return near_sum({h.x, l.x}, {h.y, l.y});
  }
};

// The probabilities of a tile that a lane holds, kEach consecutive ones a load.
// Tiles begin at multiples of 16 bytes of the target's row, wherever that begins;
// a row of the draft's that lies otherwise is shifted into place.
template <int kType>
struct Line {
  static constexpr int kEach = kType == 2 ? 4 : 8;
  static constexpr int kTile = kDraftTile<kType>;
  uint32_t w[4 * kDraftLoads];

  // Where value i of this lane lies in a tile from v0 on.
  __device__ __forceinline__ static int64_t place(int64_t v0, int i) {
    return v0 + i / kEach * (32 * kEach) + static_cast<int>(threadIdx.x & 31) * kEach + i % kEach;
  }
  __device__ __forceinline__ void set(int i, const void* p, int64_t v) {
    if (kType == 2) w[i] = __ldg(static_cast<const uint32_t*>(p) + v);
    else w[i / 2] |= static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p) + v)) << 16 * (i & 1);
  }
  // The value of token v, if it is in the tile from v0 on and this lane's, as nothing.
  __device__ __forceinline__ void clear(int64_t v0, int64_t v) {
    const int i = static_cast<int>(v - v0), at = i / kEach;
    if (i < 0 || i >= kTile || (at & 31) != static_cast<int>(threadIdx.x & 31)) return;
    const uint32_t keep = kType == 2 ? 0u : i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
    const int word = at / 32 * 4 + (kType == 2 ? i & 3 : (i & 7) / 2);
#pragma unroll
    for (int k = 0; k < 4 * kDraftLoads; ++k)
      if (k == word) w[k] &= keep;
  }
  // Values 2 i and 2 i + 1.
  __device__ __forceinline__ uint64_t two(int i) const {
    if (kType == 2) return pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    const float2 f = unpack2<kType == 1>(w[i]);
    return pair(f.x, f.y);
  }
  // The same, NaN and what is negative as 0.
  __device__ __forceinline__ uint64_t two_weights(int i) const {
    if (kType == 2) return pair(fmaxf(__uint_as_float(w[2 * i]), 0.0f), fmaxf(__uint_as_float(w[2 * i + 1]), 0.0f));
    uint32_t x;
    if (kType == 1) asm("max.f16x2 %0, %1, %2;" : "=r"(x) : "r"(w[i]), "r"(0u));
    else asm("max.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w[i]), "r"(0u));
    const float2 f = unpack2<kType == 1>(x);
    return pair(f.x, f.y);
  }
  // Row p of V probabilities, from v0 on, where p + v0 is a multiple of 16 bytes;
  // what does not fill 16 bytes at the row's ends is left out (edge()).
  __device__ __forceinline__ void load(const uint8_t* p, int64_t v0, int64_t V) {
    const uint4* at = reinterpret_cast<const uint4*>(p + place(v0, 0) * (16 / kEach));
    if (v0 >= 0 && v0 + kTile <= V) {
#pragma unroll
      for (int j = 0; j < kDraftLoads; ++j) {
        const uint4 x = __ldcs(at + 32 * j);
        w[4 * j] = x.x, w[4 * j + 1] = x.y, w[4 * j + 2] = x.z, w[4 * j + 3] = x.w;
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < kDraftLoads; ++j) {
      const int64_t v = place(v0, j * kEach);
      const uint4 x = v >= 0 && v + kEach <= V ? __ldcs(at + 32 * j) : make_uint4(0u, 0u, 0u, 0u);
      w[4 * j] = x.x, w[4 * j + 1] = x.y, w[4 * j + 2] = x.z, w[4 * j + 3] = x.w;
    }
  }
  // The token of this lane among those that load() leaves out of a tile, or -1.
  __device__ __forceinline__ static int64_t edge(int64_t v0, int64_t V) {
    const int lane = threadIdx.x & 31;
    const int64_t first = v0 < 0 ? v0 + kEach : 0;                       // of the row's first whole 16 bytes (-kEach < v0)
    if (lane < kEach) return lane < first && lane < V ? lane : -1;
    const int64_t tail = V - (V - v0) % kEach, v = tail + lane - kEach;  // behind the last
    return v0 + kTile > V && tail >= first && lane < 2 * kEach && v < V ? v : -1;
  }
  // The same, of a row that lies otherwise: p + v0 lies `off` values behind a
  // multiple of 16 bytes (uniform over the warp, not 0).  Nothing is left out.
  __device__ __forceinline__ void load_shifted(const uint8_t* p, int64_t v0, int64_t V, int off) {
    constexpr int kBytes = 16 / kEach;
    if (v0 >= off && v0 + kTile + kEach <= V) {
      const uint4* at = reinterpret_cast<const uint4*>(p + (place(v0, 0) - off) * kBytes);
#pragma unroll
      for (int j = 0; j < kDraftLoads; ++j) {
        const uint4 x = __ldcs(at + 32 * j);
        w[4 * j] = x.x, w[4 * j + 1] = x.y, w[4 * j + 2] = x.z, w[4 * j + 3] = x.w;
      }
      // What follows a lane's 16 bytes is the next lane's, and the next load's first after the last.
      const uint4 end = __ldg(at + 32 * (kDraftLoads - 1) + 1);
      const int words = off * kBytes / 4, bits = off * kBytes % 4 * 8;
#pragma unroll
      for (int j = 0; j < kDraftLoads; ++j) {
        uint32_t c[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          c[k] = w[4 * j + k];
          const uint32_t mine = (threadIdx.x & 31) == 0 && j + 1 < kDraftLoads ? w[(4 * j + 4 + k) % (4 * kDraftLoads)] : c[k];
          c[4 + k] = __shfl_sync(0xFFFFFFFFu, mine, (threadIdx.x + 1) & 31);
        }
        if (j + 1 == kDraftLoads && (threadIdx.x & 31) == 31) c[4] = end.x, c[5] = end.y, c[6] = end.z, c[7] = end.w;
#pragma unroll
        for (int k = 0; k < 6; ++k) c[k] = words & 2 ? c[k + 2] : c[k];
#pragma unroll
        for (int k = 0; k < 5; ++k) c[k] = words & 1 ? c[k + 1] : c[k];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[4 * j + k] = __funnelshift_r(c[k], c[k + 1], bits);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 4 * kDraftLoads; ++i) w[i] = 0u;
#pragma unroll
    for (int i = 0; i < kEach * kDraftLoads; ++i) {
      const int64_t v = place(v0, i);
      if (v >= 0 && v < V) set(i, p, v);
    }
  }
};

// Inclusive sum over the warp's lanes, of the first kLanes of them.
template <int kLanes>
__device__ __forceinline__ FF warp_scan(FF x) {
#pragma unroll
  for (int d = 1; d < kLanes; d *= 2) {
    const FF y = {__shfl_up_sync(0xFFFFFFFFu, x.hi, d), __shfl_up_sync(0xFFFFFFFFu, x.lo, d)};
    if (static_cast<int>(threadIdx.x & 31) >= d) x = y + x;
  }
  return x;
}
__device__ __forceinline__ FF from_lane(const FF& x, int lane) {
  return {__shfl_sync(0xFFFFFFFFu, x.hi, lane), __shfl_sync(0xFFFFFFFFu, x.lo, lane)};
}

// Whether sequence b's starts are sound.
__device__ __forceinline__ bool starts_ok(const DraftParams& P, int a0, int a1) { return a0 >= 0 && a1 >= a0 && a1 <= P.N; }

// -1 for the rows of no sequence, by the first CTA of sequence b: those before the
// first sequence, those behind the last, and what a run of sequences whose starts are
// not sound leaves between its neighbours, by the first of the run.
__device__ __forceinline__ void leave_unnamed(const DraftParams& P, int b, int batch, int a0, int a1, int* next) {
  const int tid = threadIdx.x, threads = blockDim.x, rows = P.N + batch;
  const bool ok = starts_ok(P, a0, a1);
  int from = b ? a0 + b : 0, to = ok ? a0 + b : rows;
  if (!ok) {
    if (b && !starts_ok(P, P.cu[b - 1], a0)) return;
    if (tid == 0) *next = batch;
    __syncthreads();
    for (int k = b + 1; k < batch; k += threads) {
      if (k + tid < batch && starts_ok(P, P.cu[k + tid], P.cu[k + tid + 1])) atomicMin(next, k + tid);
      if (__syncthreads_or(*next < batch)) break;
    }
    if (*next < batch) to = P.cu[*next] + *next;
  }
  for (int i = from + tid; i < to; i += threads) P.tokens[i] = -1;
  if (ok && b == batch - 1)
    for (int i = a1 + batch + tid; i < rows; i += threads) P.tokens[i] = -1;
}

// One cluster a sequence.  Every CTA finds the first draft that does not stay, sums
// the weights of its part of that row tile by tile, and learns the other parts'
// sums; the one whose part holds the drawn place looks for it in one tile again.
// Bound by memory where rows are many and long: 64 x 131072 FP32 with the draft's
// rows, 67 MB, 17.2 us, of which the sums take 10 to 11 (the memory's rate); before
// them a chain of lookups (starts, draft, its probabilities, 2.5 us), after them the
// exchange and the last tile (3 us).  256 x 100003 BF16 without them, 51 MB, 20 us:
// 104 of 152 SMs have two CTAs, the others one.  1 x 32000: 6.5 us, the chain alone.
// Tried: one 16-bit probability a load where rows are not aligned 28 us for the
// latter; the running sums in FP64 30 and 41 us.
template <int kType, bool kDraft>
__global__ void __launch_bounds__(kDraftThreads<kDraft>, kDraftCtas) verify_drafts_kernel(DraftParams P) {
  constexpr int kThreads = kDraftThreads<kDraft>, kWarps = kThreads / 32;
  constexpr int kBytes = kType == 2 ? 4 : 2;
  __shared__ FF tile_own[kDraftTiles], tile_sum[kDraftTiles], part[kWarps], cta_sum[kDraftClusters];
  __shared__ int again;
  __shared__ uint32_t stop;
  __shared__ int first_over, last_some, owner_tile;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const int b = blockIdx.x / ctas;
  if (ctas > 1) cluster_begun();

  const float u = __ldg(P.sample_u + b);              // here, so that nothing waits for it later
  const int a0 = P.cu ? P.cu[b] : b * P.each, a1 = P.cu ? P.cu[b + 1] : a0 + P.each;
  // No CTA leaves before the last barrier, whatever it finds: others write to it.
  const bool bad = !starts_ok(P, a0, a1);
  const int n = bad ? 0 : a1 - a0;
  const int64_t row0 = bad ? 0 : static_cast<int64_t>(a0) + b;         // of the target's probabilities

  if (rank == 0 && P.cu) {
    const int batch = gridDim.x / ctas;
    if (bad || (b == 0 && a0 > 0) || (b == batch - 1 && a1 < P.N)) leave_unnamed(P, b, batch, a0, a1, &again);
  }

  // The first draft that does not stay: 2 i, or 2 i + 1 where there is none at i.
  if (tid == 0) stop = 2u * n + 1u;
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    if (i < n) {
      const int x = P.drafts[a0 + i];
      const float luck = P.accept_u[a0 + i];
      if (x < 0 || x >= P.V) {
        atomicMin(&stop, 2u * i + 1u);
        if (x >= P.V) atomicOr(P.status, kPagedBadIndex);
      } else {
        const float p = prob<kType>(P.target, (row0 + i) * P.target_stride + x);
        const float q = kDraft ? prob<kType>(P.draft, static_cast<int64_t>(a0 + i) * P.draft_stride + x) : 1.0f;
        // 24 by 24 bits: exact in 64
        if (!(static_cast<double>(luck) * q < p)) atomicMin(&stop, 2u * i);
      }
    }
    __syncthreads();
    if (stop < 2u * (i0 + kThreads)) break;
    __syncthreads();
  }
  const int kept = stop >> 1;
  const bool rejected = !(stop & 1u);
  if (rank == 0) {
    for (int i = tid; i <= n; i += kThreads)
      if (i != kept) P.tokens[row0 + i] = i < kept ? P.drafts[a0 + i] : -1;
    if (tid == 0) {
      P.accepted[b] = kept;
      if (bad) atomicOr(P.status, kPagedBadIndex);
    }
  }

  // Sums of the weights of this CTA's part of the vocabulary, tile by tile.
  const uint8_t* pr = static_cast<const uint8_t*>(P.target) + (row0 + kept) * P.target_stride * kBytes;
  const uint8_t* qr = nullptr;
  int64_t out = -1;                                   // a token that counts for nothing
  if (rejected) {
    if (kDraft) qr = static_cast<const uint8_t*>(P.draft) + static_cast<int64_t>(a0 + kept) * P.draft_stride * kBytes;
    else out = P.drafts[a0 + kept];
  }
  using L = Line<kType>;
  const auto behind = [](const uint8_t* p) { return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) / kBytes; };
  const int skip = behind(pr), tile = L::kTile << P.tile_shift;       // tile t begins at token t * tile - skip
  const int all_tiles = static_cast<int>((static_cast<int64_t>(P.V) + skip + tile - 1) / tile), per = (all_tiles + ctas - 1) / ctas;
  const int t0 = min(static_cast<int>(rank) * per, all_tiles), tiles = bad ? 0 : min(per, all_tiles - t0);
  FF mine, total, upto;                               // upto: of the CTAs up to the one with this lane's rank
  for (int pass = 0;; ++pass) {
    const int off = kDraft && qr ? (behind(qr) - skip) & (L::kEach - 1) : 0;
    for (int t = warp; t < tiles; t += kWarps) {
      Sums a, c;
      int64_t v0 = static_cast<int64_t>(t0 + t) * tile - skip;
#pragma unroll 1
      for (int k = 0; k < 1 << P.tile_shift && v0 < P.V; ++k, v0 += L::kTile) {
        L p;
        p.load(pr, v0, P.V);
        if (v0 < 0 || v0 + L::kTile > P.V) {
          const int64_t v = L::edge(v0, P.V);
          if (v >= 0 && v != out) a.add(pair(prob<kType>(pr, v), 0.0f), pair(kDraft && qr ? prob<kType>(qr, v) : 0.0f, 0.0f));
        }
        if (kDraft && qr) {
          L q;
          if (off) q.load_shifted(qr, v0, P.V, off);
          else q.load(qr, v0, P.V);
#pragma unroll
          for (int i = 0; i < L::kEach * kDraftLoads / 2; i += 2) {
            a.add(p.two(i), q.two(i));
            c.add(p.two(i + 1), q.two(i + 1));
          }
        } else {
          if (!kDraft && out >= v0 && out < v0 + L::kTile) p.clear(v0, out);
#pragma unroll
          for (int i = 0; i < L::kEach * kDraftLoads / 2; i += 2) {
            a.add(p.two_weights(i));
            c.add(p.two_weights(i + 1));
          }
        }
      }
      FF w = a.sum(c);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1)
        w = near_sum(w, FF{__shfl_xor_sync(0xFFFFFFFFu, w.hi, d), __shfl_xor_sync(0xFFFFFFFFu, w.lo, d)});
      if (lane == 0) tile_own[t] = w;
    }
    __syncthreads();
    // Running sums over the tiles, and those of the CTAs exchanged.
    mine = {0.0f, 0.0f};
    if (warp == 0) {
      for (int k = 0; k < tiles; k += 32) {
        const int t = k + lane;
        const FF x = mine + warp_scan<32>(t < tiles ? tile_own[t] : FF{0.0f, 0.0f});
        if (t < tiles) tile_sum[t] = x;
        mine = from_lane(x, 31);
      }
      __syncwarp();
    }
    if (ctas > 1) cluster_wait();
    if (warp == 0) {
      if (lane < ctas)
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(cluster_addr(&cta_sum[rank], lane)), "f"(mine.hi), "f"(mine.lo)
                     : "memory");
      if (rank == 0 && lane < ctas)                   // whether there is another row to draw from
        asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(cluster_addr(&again, lane)), "r"(static_cast<int>(!pass && (qr || out >= 0))) : "memory");
      __syncwarp();
    }
    if (ctas > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    upto = warp_scan<kDraftClusters>(lane < ctas ? cta_sum[lane] : FF{0.0f, 0.0f});
    total = from_lane(upto, kDraftClusters - 1);
    if (total.hi > 0.0f || !again) break;
    // Nothing is left of p - q: p itself.
    if (ctas > 1) {
      __syncwarp();
      cluster_arrive();
    } else {
      __syncthreads();
    }
    qr = nullptr;
    out = -1;
  }
  if (!(total.hi > 0.0f)) {
    if (rank == 0 && tid == 0 && !bad) P.tokens[row0 + kept] = -1;
    return;
  }

  // The part of the vocabulary, tile and thread within which the running sum first
  // exceeds u * total, or, where rounding (or u >= 1) leaves none, the last that
  // holds any weight.
  FF goal = {u * total.hi, 0.0f};
  goal.lo = fmaf(u, total.hi, -goal.hi) + u * total.lo;
  const bool some = lane < ctas && cta_sum[lane].hi > 0.0f;
  const uint32_t any = __ballot_sync(0xFFFFFFFFu, some), over = __ballot_sync(0xFFFFFFFFu, some && above(upto, goal));
  if (static_cast<int>(rank) != (over ? __ffs(over) - 1 : 31 - __clz(any))) return;
  FF before = rank ? from_lane(upto, rank - 1) : FF{0.0f, 0.0f};
  if (warp == 0) {
    int first = -1, last = 0;
    for (int k = 0; k < tiles && first < 0; k += 32) {
      const int t = k + lane;
      const bool holds = t < tiles && tile_own[t].hi > 0.0f;
      const uint32_t h = __ballot_sync(0xFFFFFFFFu, holds);
      const uint32_t o = __ballot_sync(0xFFFFFFFFu, holds && above(before + tile_sum[t < tiles ? t : 0], goal));
      if (h) last = k + 31 - __clz(h);
      if (o) first = k + __ffs(o) - 1;
    }
    if (lane == 0) {
      owner_tile = first >= 0 ? first : last;
      first_over = 0x7FFFFFFF;
      last_some = -1;
    }
  }
  __syncthreads();
  const int t = owner_tile;
  if (t) before = before + tile_sum[t - 1];
  // Its probabilities in order, a few consecutive ones a thread.
  const int64_t v0 = static_cast<int64_t>(t0 + t) * tile - skip;
  const int64_t v1 = v0 + tile < P.V ? v0 + tile : P.V;
  for (int64_t k = v0; k < v1; k += 4 * kThreads) {
    FF w[4], own = {0.0f, 0.0f};
    const int64_t v = k + 4 * tid;
    float p[4], q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool there = v + j >= 0 && v + j < v1 && v + j != out;
      p[j] = there ? prob<kType>(pr, v + j) : 0.0f;
      q[j] = kDraft && there && qr ? prob<kType>(qr, v + j) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = weight(p[j], q[j]);
      own = own + w[j];
    }
    const FF in_warp = warp_scan<32>(own);
    if (lane == 31) part[warp] = in_warp;
    __syncthreads();
    const FF parts = warp_scan<kWarps>(lane < kWarps ? part[lane] : FF{0.0f, 0.0f});
    const FF ahead = from_lane(parts, warp ? warp - 1 : 0);
    const FF up = warp ? before + ahead + in_warp : before + in_warp;
    // A thread within whose numbers it may exceed goes through them once more.
    if (own.hi > 0.0f) {
      int has = -1, hit = -1;
      FF x = up + FF{-own.hi, -own.lo};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x = x + w[j];
        if (w[j].hi > 0.0f) {
          has = static_cast<int>(v + j);
          if (hit < 0 && above(x, goal)) hit = has;
        }
      }
      atomicMax(&last_some, has);
      if (hit >= 0) atomicMin(&first_over, hit);
    }
    __syncthreads();
    if (first_over != 0x7FFFFFFF) break;
    before = before + from_lane(parts, kWarps - 1);
  }
  if (tid == 0) P.tokens[row0 + kept] = first_over != 0x7FFFFFFF ? first_over : last_some;
}

}  // namespace ovc
