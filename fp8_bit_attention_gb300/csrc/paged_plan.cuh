// paged_plan.cuh -- how attention over the paged cache is shared out.
//
// The query rows of a sequence that use one KV head (its new tokens times the
// group of query heads) are packed token by token and cut into tiles of R
// rows; a tile has to see the key blocks from its first row's first key to its
// last row's last one.  All tiles' blocks, in the order (sequence, tile, head,
// block), form one line, which the CTAs of a persistent grid cut into equal
// shares: lengths that differ, or a single long sequence, load every SM alike.
// A tile that lies in one share is finished by its CTA.  A tile cut by a share's
// end leaves partial results (each normalised, with its log-sum) in the
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
  int32_t b, h, i, c0, c1;    // c1 < 0: none
};

// Workspace of one call.
struct PagedWork {
  float* o;         // [ctas][2][R][128] normalised partial outputs
  float* lse;       // [ctas][2][R] their log2-sums
  CutTile* cut;     // [ctas]
};

// Key blocks [k0, k1) of tile i of a sequence: at least one, so that a tile
// whose rows see no key is visited too and its output written.
template <int R, int BK>
__device__ __forceinline__ void tile_blocks(const PagedParams& P, const Seq& s, int i, int& k0, int& k1) {
  const int rows = s.ql * P.group;
  int lo, hi, x;
  row_range(P, s, i * R / P.group, lo, x);
  row_range(P, s, (min(rows, i * R + R) - 1) / P.group, x, hi);
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
// its own, where there is nothing to do.
template <int BK>
constexpr int kTileCost = BK == 32 ? 8 : 2;

constexpr int kPlanSeqs = 256;

struct PlanSmem {
  long long blocks[kPlanSeqs];     // of each sequence of a chunk, one head
  long long sums[kPlanSeqs / 32];
  long long total;
  int b, h, i, off;
};

// A CTA's share: it starts at place `off` of tile (b, i, h) and is `len` places
// of the line long.
struct Share {
  int b, h, i, off;
  long long len, at, share;
};

// Computed by the whole CTA (kThreads >= kPlanSeqs); kLanes threads add up one
// sequence's tiles (1 where sequences have a tile or two, 32 where many).
// min_share: the least places worth a CTA.
template <int R, int BK, int kThreads, int kLanes>
__device__ Share plan_share(const PagedParams& P, PlanSmem& sm, int min_share) {
  const int tid = threadIdx.x, lane = tid & 31;
  Share out{};
  long long base = 0;
  // Pass 0 adds up the line; pass 1 finds the share's start.  A batch of one
  // chunk keeps its sums between the passes.
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    base = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < P.B; b0 += kPlanSeqs) {
      const int n = min(kPlanSeqs, P.B - b0);
      if (pass == 0 || P.B > kPlanSeqs) {
        __syncthreads();
        for (int j = tid / kLanes; j < n; j += kThreads / kLanes) {
          const Seq s = load_seq(P, b0 + j);
          const int nt = tiles_of<R>(P, s);
          long long w = 0;
          for (int i = tid % kLanes; i < nt; i += kLanes) {
            int k0, k1;
            tile_blocks<R, BK>(P, s, i, k0, k1);
            w += k1 - k0 + kTileCost<BK>;
          }
          if (kLanes == 32) {
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) w += __shfl_xor_sync(0xFFFFFFFFu, w, d);
          }
          if (tid % kLanes == 0) {
            sm.blocks[j] = w;
            if (s.bad && pass == 0 && blockIdx.x == 0) atomicOr(P.status, kPagedBadIndex);
          }
        }
        __syncthreads();
      }
      // Inclusive sums over the chunk's sequences (all heads).
      long long w = 0, v = 0;
      if (tid < kPlanSeqs) {
        w = tid < n ? sm.blocks[tid] * P.c.heads : 0;
        v = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long u = __shfl_up_sync(0xFFFFFFFFu, v, d);
          if (lane >= d) v += u;
        }
        if (lane == 31) sm.sums[tid >> 5] = v;
      }
      __syncthreads();
      if (tid < kPlanSeqs) {
        for (int k = 0; k < (tid >> 5); ++k) v += sm.sums[k];
        if (pass == 1) {
          const long long lo = base + v - w;
          if (out.at >= lo && out.at < lo + w) {       // one thread of one chunk
            sm.b = b0 + tid;
            sm.total = out.at - lo;                    // place within the sequence
          }
        }
        if (pass == 0 && tid == n - 1) sm.total = base + v;
      }
      __syncthreads();
      if (pass == 0) base = sm.total;
      else if (P.B > kPlanSeqs) {
        long long all = 0;
        for (int k = 0; k < n; ++k) all += sm.blocks[k] * P.c.heads;
        base += all;
      }
    }
    if (pass == 0) {
      const long long total = base;
      out.share = max(static_cast<long long>(min_share), (total + gridDim.x - 1) / gridDim.x);
      out.at = out.share * blockIdx.x;
      out.len = min(out.share, total - out.at);
      if (out.len <= 0) {
        out.len = 0;
        return out;                                    // the whole CTA
      }
    }
  }
  // The tile and head within the sequence, 32 tiles at a time.
  if (tid < 32) {
    const Seq s = load_seq(P, sm.b);
    const int nt = tiles_of<R>(P, s);
    long long rem = sm.total;
    for (int i0 = 0; i0 < nt; i0 += 32) {
      int len = 0;
      if (i0 + lane < nt) {
        int k0, k1;
        tile_blocks<R, BK>(P, s, i0 + lane, k0, k1);
        len = k1 - k0 + kTileCost<BK>;
      }
      const long long w = static_cast<long long>(len) * P.c.heads;
      long long v = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v += u;
      }
      const unsigned past = __ballot_sync(0xFFFFFFFFu, v > rem);
      if (past) {
        if (lane == __ffs(past) - 1) {
          const long long r = rem - (v - w);
          sm.i = i0 + lane;
          sm.h = static_cast<int>(r / len);
          sm.off = static_cast<int>(r - static_cast<long long>(sm.h) * len);
        }
        break;
      }
      rem -= __shfl_sync(0xFFFFFFFFu, v, 31);
    }
  }
  __syncthreads();
  out.b = sm.b;
  out.h = sm.h;
  out.i = sm.i;
  out.off = sm.off;
  return out;
}

// The parts of tiles in a share, one after another: heads fastest, so that
// what depends on the sequence and the tile alone is computed once for all
// heads.  Every role of a CTA walks its own.
template <int R, int BK>
struct Walk {
  Seq s;
  int b, i, h;       // the tile
  int t0, t1;        // its key blocks
  int k0, k1;        // those in this share
  bool fresh;        // b or i changed with the last step
  bool whole;        // the tile lies in this share alone
  int slot;          // else: which of the CTA's two partial results
  int nt;
  long long len;     // places left

  __device__ __forceinline__ void part(int off) {
    const int places = t1 - t0 + kTileCost<BK>;
    k0 = min(t0 + off, t1);
    k1 = static_cast<int>(min(static_cast<long long>(t1), t0 + off + len));
    whole = k0 == t0 && k1 == t1;
    slot = off > 0 ? 0 : 1;
    len -= places - off;
  }

  // Stands on the first part that has blocks; false if there is none.
  __device__ __forceinline__ bool start(const PagedParams& P, const Share& sh) {
    b = sh.b;
    i = sh.i;
    h = sh.h;
    len = sh.len;
    s = load_seq(P, b);
    nt = tiles_of<R>(P, s);
    tile_blocks<R, BK>(P, s, i, t0, t1);
    part(sh.off);
    if (k0 >= k1 && !step(P)) return false;
    fresh = true;
    return true;
  }

  __device__ __forceinline__ bool step(const PagedParams& P) {
    if (len <= 0) return false;
    fresh = false;
    if (++h >= P.c.heads) {
      h = 0;
      fresh = true;
      if (++i >= nt) {
        i = 0;
        do {
          if (++b >= P.B) return false;                // not reached: len ends first
          s = load_seq(P, b);
          nt = tiles_of<R>(P, s);
        } while (nt == 0);
      }
      tile_blocks<R, BK>(P, s, i, t0, t1);
    }
    part(0);
    return true;                                       // at least one block: places begin with them
  }
};

// Says which tile, if any, the join of this CTA's number puts together: the one
// its share starts within, unless an earlier CTA's does too.
template <int R, int BK>
__device__ __forceinline__ void write_cut(const PagedParams& P, const Share& sh, const PagedWork& w) {
  CutTile c{0, 0, 0, 0, -1};
  if (sh.len > 0 && sh.off > 0) {
    int k0, k1;
    tile_blocks<R, BK>(P, load_seq(P, sh.b), sh.i, k0, k1);
    const long long a = sh.at - sh.off;
    const int c0 = static_cast<int>(a / sh.share), c1 = static_cast<int>((a + (k1 - k0) - 1) / sh.share);
    if (sh.off < k1 - k0 && c0 + 1 == static_cast<int>(blockIdx.x)) c = CutTile{sh.b, sh.h, sh.i, c0, c1};
  }
  w.cut[blockIdx.x] = c;
}

// ---------------------------------------------------------------------------
// Join of a cut tile's partial results: with L_c the log2-sum of part c,
// O = sum_c 2^(L_c - L) O_c, L = log2 sum_c 2^L_c.  Part c0 is in its CTA's
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
  const Seq s = load_seq(P, c.b);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % kWarps;
  const int rows = min(R, s.ql * P.group - c.i * R);
  for (int r0 = blockIdx.y * kRows; r0 < rows; r0 += gridDim.y * kRows) {
    const int r = r0 + warp / kWarps;
    const bool here = r < rows;
    const int n = c.c1 - c.c0 + 1;
    float top = kNegInf, total = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (here) {
      auto at = [&](int k) { return (static_cast<int64_t>(c.c0 + k) * 2 + (k == 0)) * R + r; };
      for (int k = lane; k < n; k += 32) top = fmaxf(top, w.lse[at(k)]);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      const float ref = top == kNegInf ? 0.0f : top;
      for (int k = lane; k < n; k += 32) total += exp2f(w.lse[at(k)] - ref);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
#pragma unroll 8
      for (int k = sub; k < n; k += kWarps) {
        const float f = exp2f(w.lse[at(k)] - ref);
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
      const int p = c.i * R + r, t = s.q0 + p / P.group, hq = c.h * P.group + p % P.group;
      reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.o.ptr) + t * P.o.st + hq * P.o.sh)[lane] =
          make_uint2(pack2<false>(acc.x * inv, acc.y * inv), pack2<false>(acc.z * inv, acc.w * inv));
      if (P.lse && lane == 0)
        P.lse[static_cast<int64_t>(t) * P.Hq + hq] = total == 0.0f ? kNegInf : (top + log2f(total)) * 0.69314718055994531f;
    }
  }
}

}  // namespace ovc
