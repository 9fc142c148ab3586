// paged_plan.cuh -- how attention over the paged cache is shared out.
//
// The query rows of a sequence that use one KV head (its new tokens times the
// group of query heads) are packed token by token and cut into tiles of R
// rows; a tile has to see the key blocks from its first row's first key to its
// last row's last one.  All tiles' blocks, in the order (sequence, tile, head,
// block), form one line, which the CTAs of a persistent grid cut into equal
// shares: lengths that differ, or a single long sequence, load every SM alike.
// A tile that lies in one share is finished by its CTA.  A tile cut by a share's
// end leaves partial results (each normalised, with its maximum and sum) in the
// workspace, at most two a CTA, which paged_join_kernel joins.  Every CTA
// derives its share from the lengths on the device, so that lengths may change
// under a captured graph and no other launch has to plan.
#pragma once

#include "paged.cuh"

namespace ovc {

// Programmatic launch: the join is launched while the attention kernel still
// runs (allow) and waits here for its end and its memory (wait), so that its own
// launch costs nothing.
__device__ __forceinline__ void grid_dependency_allow() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A cut tile, written by the second CTA that works on it (c0 + 1).
struct CutTile {
  int32_t c0, c1;             // the CTAs that work on it; c1 < 0: none
  int32_t q0, p0, rows, h;    // its first row is packed row p0 of the sequence whose rows start at q0
};

// Workspace of one call.
struct PagedWork {
  float* o;         // [ctas][2][R][128] normalised partial outputs
  float2* ml;       // [ctas][2][R] their largest scores (log2 units) and their sums against those
  CutTile* cut;     // [ctas]
};

// Key blocks [k0, k1) of tile i of a sequence: at least one, so that a tile
// whose rows see no key is visited too and its output written.
template <int R, int BK>
__device__ __forceinline__ void tile_blocks(const PagedParams& P, const Seq& s, int i, int& k0, int& k1) {
  const int rows = s.ql * P.group;
  int lo, hi, x;
  row_range(P, s, i * R / P.by_group, lo, x);
  row_range(P, s, (min(rows, i * R + R) - 1) / P.by_group, x, hi);
  k0 = 0;
  k1 = 1;
  if (hi >= lo) {
    k0 = lo / BK;
    k1 = hi / BK + 1;
  }
}

template <int R>
__device__ __forceinline__ int tiles_of(const PagedParams& P, const Seq& s) {
  return static_cast<int>((static_cast<int64_t>(s.ql) * P.group + R - 1) / R);
}

// What a tile costs beside its key blocks (query rows in, the warps' join, rows
// out), in blocks: each tile stands for so many more blocks on the line, behind
// its own, where there is nothing to do.  (3, 4 and 5 for blocks of 128 keys: 8
// ragged sequences of up to 500 tokens with a window of 4096 89, 82, 88 us; 16 x 4
// tokens over 8192 keys 27, 25, 27 us; a prompt of 1024 tokens, 56 heads, 53, 53, 57 us.  4, 8
// and 16 for blocks of 16: 32 single tokens over ragged contexts 43, 35, 35 us; 256
// sequences of 256 keys, 16 rows, 75, 71, 72 us.)
template <int BK>
constexpr int kTileCost = BK < 128 ? 8 : 4;

// A cut so near a tile's start or end is moved there: so few blocks are not worth
// a part of their own, with its partial results and their join.  (0, 2, 3 and 4 for
// blocks of 128 keys: 8 prompts of 512 tokens 64, 55, 55, 55 us; 8 ragged sequences
// with a window 84, 83, 82, 82 us; 16 x 4 tokens over 8192 keys 25, 25, 25, 29 us.
// 0 and 4 for blocks of 16: 256 sequences of 256 keys, 16 rows, 74 and 71 us.)
template <int BK>
constexpr int kSnap = BK < 128 ? 4 : 3;

// Where a cut behind `off` of a tile's n blocks falls.  The CTA that ends and
// the one that begins there both ask.
template <int BK>
__device__ __forceinline__ int cut_at(const PagedParams& P, int off, int n) {
  if (off <= 0) return 0;
  if (off >= n || (P.unit == 0 && n - off <= kSnap<BK>)) return n;
  return P.unit == 0 && off <= kSnap<BK> ? 0 : off;
}

// The line is cut at places 2^unit blocks apart; the host takes unit = 0 unless
// the line could then pass 31 bits.
template <int BK>
__device__ __forceinline__ int tile_places(const PagedParams& P, int t0, int t1) {
  return (t1 - t0 + kTileCost<BK> - 1 >> P.unit) + 1;
}

// A CTA's share: it starts at place `off` of tile (b, i, h), whose key blocks
// are [t0, t1), and is `len` places of the line long.
struct Share {
  Seq s;
  int b, h, i, off, t0, t1;
  int len, share;
};

struct PlanSmem {
  int places[160];           // of each sequence of a chunk, one head
  int sums[8];
  int rem;
  Share found;
};

// Inclusive sum of w over threads 0 .. N - 1 of the CTA, and all of it; `any`
// becomes true if it is so in any thread.
template <int N>
__device__ __forceinline__ int cta_scan(int w, PlanSmem& sm, int& all, bool& any) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = w;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += u;
  }
  if (lane == 31 && warp < N / 32) sm.sums[warp] = v;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int k = 0; k < N / 32; ++k) {
    const int x = sm.sums[k];
    if (k < warp) v += x;
    all += x;
  }
  any = __syncthreads_or(any);
  return v;
}

// Computed by the whole CTA, N sequences at a time; kLanes threads add up one
// sequence's tiles (1 where sequences have a tile or two, 32 where many).
// min_share: the least places worth a CTA.
template <int R, int BK, int kThreads, int kLanes>
__device__ Share plan_share(const PagedParams& P, PlanSmem& sm, int min_share) {
  constexpr int N = kThreads < 160 ? kThreads : 160;
  const int tid = threadIdx.x, lane = tid & 31;
  // Places of sequence b0 + tid, all heads.
  bool descends = false;
  auto places = [&](int b0, bool first) {
    const int n = min(N, P.B - b0);
    int w = 0;
    if (kLanes == 1) {
      if (tid < n) {
        const Seq s = load_seq(P, b0 + tid);
        if (s.bad && first && blockIdx.x == 0) atomicOr(P.status, kPagedBadIndex);
        descends |= s.bad == 2;
        const int nt = tiles_of<R>(P, s);
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
          int t0, t1;
          tile_blocks<R, BK>(P, s, i, t0, t1);
          w += tile_places<BK>(P, t0, t1);
        }
      }
    } else {
#pragma unroll 1
      for (int j = tid / 32; j < n; j += kThreads / 32) {
        const Seq s = load_seq(P, b0 + j);
        if (s.bad && first && blockIdx.x == 0 && lane == 0) atomicOr(P.status, kPagedBadIndex);
        descends |= s.bad == 2;
        const int nt = tiles_of<R>(P, s);
        int x = 0;
#pragma unroll 1
        for (int i = lane; i < nt; i += 32) {
          int t0, t1;
          tile_blocks<R, BK>(P, s, i, t0, t1);
          x += tile_places<BK>(P, t0, t1);
        }
        x = __reduce_add_sync(0xFFFFFFFFu, x);
        if (lane == 0) sm.places[j] = x;
      }
      __syncthreads();
      if (tid < n) w = sm.places[tid];
      // the next chunk's sums are written behind cta_scan's barriers
    }
    return w * P.c.heads;
  };

  int total = 0, w = 0, v = 0, all = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < P.B; b0 += N) {
    w = places(b0, true);
    v = cta_scan<N>(w, sm, all, descends);
    total += all;
  }
  // Where cu_q descends its sequences overlap, and their places may pass the 31
  // bits that the host saw to: nothing of the batch is done then.
  if (descends) total = 0;
  const int share = max(min_share, static_cast<int>((static_cast<unsigned>(total) + gridDim.x - 1) / gridDim.x));
  const long long at = static_cast<long long>(share) * blockIdx.x;
  if (at >= total) {
    Share none{};
    return none;                                       // the whole CTA
  }
  // The sequence that the share starts in: a batch of one chunk has its sums at
  // hand, a longer one adds them up again.
  auto found = [&](const Seq& s, int b, int i, int rem, int t0, int t1) {
    const int n = tile_places<BK>(P, t0, t1), h = static_cast<unsigned>(rem) / static_cast<unsigned>(n);
    sm.found = Share{s, b, h, i, rem - h * n, t0, t1, min(share, total - static_cast<int>(at)), share};
  };
  int base = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < P.B; b0 += N) {
    if (P.B > N) {
      w = places(b0, false);
      v = cta_scan<N>(w, sm, all, descends);
    }
    const int rem = static_cast<int>(at) - (base + v - w);
    if (tid < N && rem >= 0 && rem < w) {              // one thread of one chunk
      const Seq s = load_seq(P, b0 + tid);
      sm.found.b = b0 + tid;
      sm.rem = -1;
      if (tiles_of<R>(P, s) == 1) {
        int t0, t1;
        tile_blocks<R, BK>(P, s, 0, t0, t1);
        found(s, b0 + tid, 0, rem, t0, t1);
      } else {
        sm.rem = rem;
      }
    }
    base += all;
  }
  __syncthreads();
  if (sm.rem >= 0) {
    // A sequence of several tiles: 32 tiles at a time.
    const int b = sm.found.b;
    int rem = sm.rem;
    __syncthreads();
    if (tid < 32) {
      const Seq s = load_seq(P, b);
      const int nt = tiles_of<R>(P, s);
#pragma unroll 1
      for (int i0 = 0; i0 < nt; i0 += 32) {
        int t0 = 0, t1 = 0, x = 0;
        if (i0 + lane < nt) {
          tile_blocks<R, BK>(P, s, i0 + lane, t0, t1);
          x = tile_places<BK>(P, t0, t1) * P.c.heads;
        }
        int y = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int u = __shfl_up_sync(0xFFFFFFFFu, y, d);
          if (lane >= d) y += u;
        }
        const unsigned past = __ballot_sync(0xFFFFFFFFu, y > rem);
        if (past) {
          if (lane == __ffs(past) - 1) found(s, b, i0 + lane, rem - (y - x), t0, t1);
          break;
        }
        rem -= __shfl_sync(0xFFFFFFFFu, y, 31);
      }
    }
    __syncthreads();
  }
  return sm.found;
}

// The parts of tiles in a share, one after another: heads fastest, so that
// what depends on the sequence and the tile alone is computed once for all
// heads.
template <int R, int BK>
struct Walk {
  Seq s;
  int b, i, h;       // the tile
  int t0, t1;        // its key blocks
  int k0, k1;        // those in this share
  bool whole;        // the tile lies in this share alone
  int slot;          // else: which of the CTA's two partial results
  int nt;
  int len;           // places left

  __device__ __forceinline__ void part(const PagedParams& P, int off) {
    const int places = tile_places<BK>(P, t0, t1);
    k0 = t0 + cut_at<BK>(P, off << P.unit, t1 - t0);
    k1 = off + len < places ? t0 + cut_at<BK>(P, off + len << P.unit, t1 - t0) : t1;
    whole = k0 == t0 && k1 == t1;
    slot = k0 > t0 ? 0 : 1;
    len -= places - off;
  }

  int off;           // the place that the next part starts at; negative: in the next tile

  __device__ __forceinline__ Walk(const PagedParams& P, const Share& sh)
      : s(sh.s), b(sh.b), i(sh.i), h(sh.h), t0(sh.t0), t1(sh.t1), nt(tiles_of<R>(P, sh.s)), len(sh.len), off(sh.off) {}

  // Goes to the next part (the first, after construction) that has blocks; false
  // if there is none.
  __device__ __forceinline__ bool step(const PagedParams& P) {
    do {
      if (off < 0) {
        if (len <= 0) return false;
        if (++h >= P.c.heads) {
          h = 0;
          if (++i >= nt) {
            i = 0;
            do {
              if (++b >= P.B) return false;            // not reached: len ends first
              s = load_seq(P, b);
              nt = tiles_of<R>(P, s);
            } while (nt == 0);
          }
          tile_blocks<R, BK>(P, s, i, t0, t1);
        }
        off = 0;
      }
      part(P, off);
      off = -1;
    } while (k0 >= k1);                                // a last part too short to be one
    return true;
  }
};

// Says which tile, if any, the join of this CTA's number puts together: the one
// its share starts within, unless an earlier CTA's does too.
template <int R, int BK>
__device__ __forceinline__ void write_cut(const PagedParams& P, const Share& sh, const PagedWork& w) {
  CutTile c{0, -1, 0, 0, 0, 0};
  const int n = sh.t1 - sh.t0;
  auto cut = [&](int off) {                            // is the tile cut behind place `off`?
    const int k = cut_at<BK>(P, off << P.unit, n);
    return k > 0 && k < n;
  };
  if (sh.len > 0 && sh.off > 0 && cut(sh.off) && !(sh.off > sh.share && cut(sh.off - sh.share))) {
    c.c0 = blockIdx.x - 1;
    c.c1 = blockIdx.x;
    // The last cut: behind the last place that leaves more than kSnap blocks.
    const int most = P.unit == 0 ? n - 1 - kSnap<BK> : (n - 1) >> P.unit;
    c.c1 += static_cast<unsigned>(most - sh.off) / static_cast<unsigned>(sh.share);
    c.q0 = sh.s.q0;
    c.p0 = sh.i * R;
    c.rows = min(R, sh.s.ql * P.group - c.p0);
    c.h = sh.h;
  }
  w.cut[blockIdx.x] = c;
}

// ---------------------------------------------------------------------------
// Join of a cut tile's partial results: with m_c and l_c the maximum and sum of
// part c, M = max m_c and l = sum_c 2^(m_c - M) l_c, O = sum_c 2^(m_c - M) l_c O_c / l.
// (A log-sum in one number would lose log2 l_c beside a large m_c.)  Part c0 is in its CTA's
// second slot, the others in their CTA's first.  kWarps warps per row share the
// parts (4 where few rows are cut into many parts), four channels a lane.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

template <int R, int kWarps>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedParams P, PagedWork w) {
  constexpr int kRows = kJoinThreads / 32 / kWarps;     // rows at a time
  __shared__ float4 part[kJoinThreads / 32][32];
  grid_dependency_wait();
  const CutTile c = w.cut[blockIdx.x];
  if (c.c1 < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % kWarps;
  const int rows = c.rows;
  for (int r0 = blockIdx.y * kRows; r0 < rows; r0 += gridDim.y * kRows) {
    const int r = r0 + warp / kWarps;
    const bool here = r < rows;
    const int n = c.c1 - c.c0 + 1;
    float top = kNegInf, total = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (here) {
      auto at = [&](int k) { return (static_cast<int64_t>(c.c0 + k) * 2 + (k == 0)) * R + r; };
      for (int k = lane; k < n; k += 32) top = fmaxf(top, w.ml[at(k)].x);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      const float ref = top == kNegInf ? 0.0f : top;
      auto weight = [&](int k) {
        const float2 x = w.ml[at(k)];
        return exp2f(x.x - ref) * x.y;
      };
      for (int k = lane; k < n; k += 32) total += weight(k);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
#pragma unroll 8
      for (int k = sub; k < n; k += kWarps) {
        const float f = weight(k);
        const float4 x = reinterpret_cast<const float4*>(w.o + at(k) * 128)[lane];
        acc.x += f * x.x;
        acc.y += f * x.y;
        acc.z += f * x.z;
        acc.w += f * x.w;
      }
      top = ref;
    }
    if (kWarps > 1) {
      part[warp][lane] = acc;
      __syncthreads();
      if (sub == 0) {
#pragma unroll
        for (int k = 1; k < kWarps; ++k) {
          const float4 x = part[warp + k][lane];
          acc.x += x.x;
          acc.y += x.y;
          acc.z += x.z;
          acc.w += x.w;
        }
      }
      __syncthreads();
    }
    if (here && sub == 0) {
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;
      const int p = c.p0 + r, tok = p / P.by_group, t = c.q0 + tok, hq = c.h * P.group + p - tok * P.group;
      reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.o.ptr) + t * P.o.st + hq * P.o.sh)[lane] =
          make_uint2(pack2<false>(acc.x * inv, acc.y * inv), pack2<false>(acc.z * inv, acc.w * inv));
      if (P.lse && lane == 0)
        P.lse[static_cast<int64_t>(t) * P.Hq + hq] = total == 0.0f ? kNegInf : (top + log2f(total)) * 0.69314718055994531f;
    }
  }
}

}  // namespace ovc
