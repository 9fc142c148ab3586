// paged_decode.cuh -- attention over the paged cache for few query rows per KV
// head: single tokens, drafted tokens, groups of query heads.
//
// Bound by memory: every key costs 258 bytes a head and each of them meets at
// most 16 query rows.  8 sequences of 131072 keys, 8 heads, group 4: 320 us,
// 99% of the rate of a plain copy; 32 ragged sequences of up to 16384 keys, 8
// heads, group 7: 35 us, 56%, the rest being the start, the tiles' ends and the
// join.  Short calls (1024 keys: 12 us) are bound by their two launches and the
// latency of a chain of loads.  With 9 to 16 rows (kTiles = 2) the products and
// conversions of two tiles bound it: 8 x 65536 keys, 8 heads: 249 us with BF16
// queries (64%), whose kernel spills some registers, 202 us with FP16 (79%).
//
// A CTA is a loading warp and four computing ones.  The
// loading warp walks the CTA's share, looks up pages, and streams 16-key blocks
// (2 KB of K, 2 KB of V) by TMA into a ring for each computing warp, which keeps
// its own running maximum, sum and output in registers; no barrier joins the
// warps until a tile's part ends.  Several such CTAs share an SM, so that one's
// ends and starts lie under the others' streams: 3 CTAs of 3 stages, against 4
// of 2 stages 319 and 323 us, 34.7 and 36.4 us for the two calls above.
//
// The products run transposed, S^T = K Q^T and O^T = V^T P^T, with
// mma.m16n8k16: keys and channels fill the 16 rows of the instruction, and the
// query rows its 8 columns (kTiles tiles of 8), so that a group of 8 query
// heads wastes nothing.  (tcgen05 has M = 64 or 128, and its 8-bit operands
// would need P in 8 bits; here each code is converted once to FP16, exactly,
// in registers.)
//   S^T: K's fragment wants two channels per register and any order of the 128,
//     as long as Q has the same.  Lane (g, t) takes the 32 channels from 32 t on
//     of keys g and g + 8: two 16-byte loads each, and Q's registers are its
//     32 channels in memory order.
//   O^T: V's fragment wants two keys per register.  Lane (g, t) takes channels
//     16 g .. 16 g + 15 of keys 2t, 2t+1, 2t+8, 2t+9 and interleaves the bytes of
//     two keys; it ends up with 16 neighbouring channels of rows 2t and 2t+1.
//   The tiles have TMA's 128-byte swizzle (16-byte chunk c of row r lies at
//   c ^ (r & 7)), which frees both kinds of loads of bank conflicts.
//   P^T goes from the first product's layout to the second's by movmatrix.
//
// Numbers: Q enters as FP16 (BF16 rows scaled by a power of two: exact but for
// elements below 2^-29 of the row's largest); scores, maxima, sums and outputs
// are FP32; a weight is rounded to FP16 once, as 2^14 p 2^(e - E) with e the
// token's V scale and E the largest so far: what is lost of it is below 2^-39 of
// 2^E.  E is the same for all rows as long as the scales spread over at most
// 2^kDecSpread.  Beyond that ("wide") every row has its own, of the largest
// p 2^e that it sees, so that a token counts by its term and one that is masked
// not at all.  Either way no more than 2^-20 of a row's largest term is lost.
// (All blocks wide: the first call above 368 us, 16 rows 380.)
#pragma once

#include <cuda.h>

#include <type_traits>

#include "paged_plan.cuh"

namespace ovc {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * (kDecWarps + 1);
constexpr int kDecKeys = 16;                       // keys of a block: a page is a multiple of them
constexpr int kDecStages = 3;
constexpr uint32_t kDecCodes = kDecKeys * 128;     // bytes of a block's K (or V) codes
constexpr int kDecPBias = 14;
// Scales of V that spread further have units by row.  A block is looked at closely
// where a scale is above E or more than kDecNear below it.
constexpr int kDecSpread = 19, kDecNear = 9;
constexpr int kDecParts = 4;                       // descriptions of parts in flight

// A tile's part, as the computing warps need it.
struct DecodePart {
  int more;                 // 0: the share is done
  int q0, ql, kv;           // the sequence
  int p0, rows, h;          // the tile: its first packed row, its rows, its KV head
  int t0, k0, k1;           // the tile's first key block; the part's blocks
  int all_lo, all_hi;       // blocks within these keys need no mask
  int slot;                 // of the partial result; negative: the tile is whole
};

struct DecodeSmem {
  uint8_t kv[kDecWarps][kDecStages][2][kDecCodes];
  union {
    float o[kDecWarps][8][128];                    // the warps' outputs of 8 rows; 16-byte chunks swizzled by the row
    PlanSmem plan;                                 // before the first of them
  };
  uint8_t scale[kDecWarps][kDecStages][2][kDecKeys];
  float m[kDecWarps][8], l[kDecWarps][8];
  int e[kDecWarps][16];                            // the rows' E
  DecodePart part[kDecParts];
  uint64_t full[kDecWarps][kDecStages], empty[kDecWarps][kDecStages];
  uint64_t part_full[kDecParts], part_empty[kDecParts];
  int abort;
  int zero;
};

// CTAs per SM: what the registers of kTiles tiles (1 or 2) leave room for.
template <int kTiles>
constexpr int kDecodeCtas = kTiles == 1 ? 3 : 2;
static_assert((sizeof(DecodeSmem) + 1024) * 3 <= 233472, "shared memory per SM");

struct PagedMaps {
  CUtensorMap k, v;     // boxes of `box` rows, which divides the page and the key block
  int32_t box;
  int32_t rows;         // rows of the cache: a box from there on reads zeros
  int32_t min_share;
  uint64_t timeout_ns;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(__cvta_generic_to_global(src)) : "memory");
}

// An arrival (one of the barrier's count) once this thread's cp.async copies
// so far are complete.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint4 lds128(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

// 2^x for an integer x, 0 below FP32's normal range.
__device__ __forceinline__ float exp2i(int x) { return x < -126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(x + 127) << 23); }

// Bit 2 i: row i of the 16 of a tile of codes is a vector of zeros, of either sign.
__device__ __forceinline__ uint32_t zero_rows(const uint8_t* codes) {
  const uint8_t* half = codes + (threadIdx.x & 31) * 64;
  uint32_t any = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint4 x = lds128(half + 16 * c);
    any |= x.x | x.y | x.z | x.w;
  }
  const uint32_t b = __ballot_sync(0xFFFFFFFFu, (any & 0x7F7F7F7Fu) != 0);
  return ~(b | b >> 1);
}

// The computing warps' own barrier: the loading warp is past them.
__device__ __forceinline__ void decode_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kDecWarps) : "memory"); }

// The same, and whether all of them say yes: the warps end together.
__device__ __forceinline__ bool decode_sync_and(bool x) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, %2, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(x)), "n"(32 * kDecWarps)
      : "memory");
  return r != 0;
}

template <bool kHalf, int kTiles>
__global__ void __launch_bounds__(kDecThreads, kDecodeCtas<kTiles>)
    paged_decode_kernel(const __grid_constant__ PagedParams P, const __grid_constant__ PagedMaps M, PagedWork work) {
  constexpr int R = 8 * kTiles;
  extern __shared__ __align__(1024) uint8_t raw[];
  DecodeSmem& sm = *reinterpret_cast<DecodeSmem*>(raw);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    sm.abort = 0;
    sm.zero = 0;
    for (int i = 0; i < kDecWarps * kDecStages; ++i) {
      mbar_init(smem_addr(&sm.full[0][0] + i), 2);
      mbar_init(smem_addr(&sm.empty[0][0] + i), 1);
    }
    for (int i = 0; i < kDecParts; ++i) {
      mbar_init(smem_addr(&sm.part_full[i]), 1);
      mbar_init(smem_addr(&sm.part_empty[i]), kDecWarps);
    }
    fence_mbar_init();
  }
  if (threadIdx.x == 32 * kDecWarps) {
    tma_prefetch_map(&M.k);
    tma_prefetch_map(&M.v);
  }
  grid_dependency_allow();
  const Share share = plan_share<R, kDecKeys, kDecThreads, 1>(P, sm.plan, M.min_share);
  volatile int* const abort_flag = &sm.abort;
  // A wait that ran out: every role goes on without waiting or loading, works on
  // whatever is there, and ends.
  auto wait = [&](uint64_t& bar, uint32_t parity) -> bool {
    if (paged_wait(smem_addr(&bar), parity, M.timeout_ns, abort_flag)) return true;
    if (!*abort_flag) atomicOr(P.status, 1u);
    *abort_flag = 1;
    return false;
  };
  if (share.len == 0) {
    if (threadIdx.x == 0) write_cut<R, kDecKeys>(P, share, work);
    return;
  }
  __syncthreads();                                 // the plan's memory is free

  if (warp == kDecWarps) {
    // -------------------------------------------------------------- loading
    Walk<R, kDecKeys> w(P, share);
    uint32_t parts = 0;
    uint32_t issued = 0;                           // blocks of lane's ring (lanes 0 .. kDecWarps - 1)
    while (true) {
      const bool more = w.step(P);
      // Describe the part.
      const uint32_t d = parts % kDecParts;
      if (parts >= kDecParts && !__all_sync(0xFFFFFFFFu, wait(sm.part_empty[d], (parts / kDecParts - 1) & 1))) break;
      if (lane == 0) {
        DecodePart& x = sm.part[d];
        x.more = more;
        if (more) {
          int y;
          x.q0 = w.s.q0;
          x.ql = w.s.ql;
          x.kv = w.s.kv;
          x.p0 = w.i * R;
          x.rows = min(R, w.s.ql * P.group - x.p0);
          x.h = w.h;
          x.t0 = w.t0;
          x.k0 = w.k0;
          x.k1 = w.k1;
          x.slot = w.whole ? -1 : w.slot;
          row_range(P, w.s, (x.p0 + x.rows - 1) / P.by_group, x.all_lo, y);
          row_range(P, w.s, x.p0 / P.by_group, y, x.all_hi);
        }
        mbar_arrive(smem_addr(&sm.part_full[d]));
      }
      ++parts;
      if (!more || __any_sync(0xFFFFFFFFu, *abort_flag)) break;
      // Block kb goes to warp (kb - t0) mod 4.  32 blocks at a time are looked up
      // in the page table, a lane each, and issued four at a time, a lane each.
      for (int base = w.k0 - ((w.k0 - w.t0) & (kDecWarps - 1)); base < w.k1; base += 32) {
        const int mine = base + lane, key = mine * kDecKeys;
        int row = M.rows;                          // past the cache's end: reads zeros
        if (mine >= w.k0 && mine < w.k1 && key < w.s.kv) {
          const int n = key / P.by_page;
          const int p = __ldg(P.table + w.b * P.table_stride + n);
          if (p >= 0 && p < P.c.pages) row = (p * P.c.heads + w.h) * P.c.page + key - n * P.c.page;
          else atomicOr(P.status, kPagedBadIndex);
        }
#pragma unroll 1
        for (int j = 0; j < 32 && base + j < w.k1; j += kDecWarps) {
          const int at = __shfl_sync(0xFFFFFFFFu, row, j + (lane & (kDecWarps - 1))), kb = base + j + lane;
          if (lane < kDecWarps && kb >= w.k0 && kb < w.k1) {
            const uint32_t stage = issued % kDecStages;
            if (issued >= kDecStages) wait(sm.empty[lane][stage], (issued / kDecStages - 1) & 1);
            if (!*abort_flag) {
              const uint32_t bar = smem_addr(&sm.full[lane][stage]);
              mbar_arrive_expect_tx(bar, 2 * kDecCodes);
              tma_load_2d(smem_addr(sm.kv[lane][stage][0]), &M.k, bar, 0, at);
              tma_load_2d(smem_addr(sm.kv[lane][stage][1]), &M.v, bar, 0, at);
              if (at < M.rows) {
                // (By cp.async: as two more bulk copies of 16 bytes the scales
                // keep the copy engine busier than the codes do, 361 against 350
                // us for 8 x 131072 keys at the time.)
                cp_async16(smem_addr(sm.scale[lane][stage][0]), P.c.ks + at);
                cp_async16(smem_addr(sm.scale[lane][stage][1]), P.c.vs + at);
              }
              cp_async_arrive(bar);
              ++issued;
            }
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) write_cut<R, kDecKeys>(P, share, work);
    // The CTA's shared memory must outlive the copies in flight, also where the
    // computing warps give up on them after this warp's last look at the flag.
    if (lane < kDecWarps)
      for (uint32_t n = issued > kDecStages ? issued - kDecStages : 0; n < issued; ++n)
        paged_wait(smem_addr(&sm.full[lane][n % kDecStages]), (n / kDecStages) & 1, 4000000000ull, &sm.zero);
    return;
  }

  // ---------------------------------------------------------------- computing
  const int g = lane >> 2, t = lane & 3;
  // Row g of each tile, channels 32 t .. 32 t + 31: loaded before the part
  // begins, so that the latency lies under other work.
  uint4 x[kTiles][4];
  auto load_q = [&](const DecodePart& d) {
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const int r = 8 * n + g, p = d.p0 + r;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[n][i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < d.rows) {
        const int tok = p / P.by_group;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.q.ptr) + (d.q0 + tok) * P.q.st +
                                                          (d.h * P.group + p - tok * P.group) * P.q.sh + 32 * t);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = __ldg(src + i);
      }
    }
  };
  uint32_t used = 0, parts = 0;
  bool more = wait(sm.part_full[0], 0) && sm.part[0].more;
  if (more) load_q(sm.part[0]);
  more = decode_sync_and(more);
  while (more) {
    const DecodePart& d = sm.part[parts % kDecParts];
    Seq s;
    s.q0 = d.q0;
    s.ql = d.ql;
    s.kv = d.kv;
    const int p0 = d.p0, all_lo = d.all_lo, all_hi = d.all_hi, k1 = d.k1;
    // Q's fragments: lane (g, t) holds row g of each tile, channels 32 t ..
    // 32 t + 31; and the factor of rows 2t, 2t+1 to log2 units.
    uint32_t qf[kTiles][8][2];
    float rowf[kTiles][2];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      float f = P.c2;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qf[n][2 * i][0] = x[n][i].x;
        qf[n][2 * i][1] = x[n][i].y;
        qf[n][2 * i + 1][0] = x[n][i].z;
        qf[n][2 * i + 1][1] = x[n][i].w;
      }
      float amax = largest_of<kHalf, 16>(&qf[n][0][0]);
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      if (!kHalf) {
        // BF16 to FP16: the row's largest magnitude goes to [2^14, 2^15).
        const uint32_t up = min(268u - (__float_as_uint(amax) >> 23), 254u);       // 2^(up - 127)
        const float mul = __uint_as_float(up << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 a = unpack2<false>(qf[n][i / 2][i % 2]);
          qf[n][i / 2][i % 2] = pack2<true>(a.x * mul, a.y * mul);
        }
        f *= inverse_scale(up);
      }
      if (amax == INFINITY) f = __uint_as_float(0x7FFFFFFFu);      // a row that is not finite: NaN, whatever its scores
#pragma unroll
      for (int j = 0; j < 2; ++j) rowf[n][j] = __shfl_sync(0xFFFFFFFFu, f, (2 * t + j) * 4);
    }

    float m[kTiles][2], l[kTiles][2], o[kTiles][8][4];
    int E = -1, low = 255;                         // the scales of V so far: the largest, none below
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[n][j] = kNegInf;
        l[n][j] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][i][j] = 0.0f;
    }

    // A block; with a true tag the rows have an E each (in shared memory).  False, with
    // nothing done, if they have to have from this block on.  (Two loops: with both
    // ways in one, 9 to 16 rows took 5% more.)
    bool first = true;
    auto block = [&](int kb, auto tag) __attribute__((always_inline)) -> bool {
      constexpr bool rows_apart = decltype(tag)::value;
      const uint32_t stage = used % kDecStages;
      wait(sm.full[warp][stage], (used / kDecStages) & 1);
      const uint8_t* K = sm.kv[warp][stage][0];
      const uint8_t* V = sm.kv[warp][stage][1];
      const uint8_t* ks = sm.scale[warp][stage][0];
      const uint8_t* vs = sm.scale[warp][stage][1];
      const int key0 = kb * kDecKeys;
      const bool masked = key0 < all_lo || key0 + kDecKeys - 1 > all_hi;

      // S^T; a single tile's eight products in two chains, which are then added.
      float z[kTiles][4], z2[kTiles][4];
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) z[n][j] = z2[n][j] = 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t chunk = static_cast<uint32_t>((2 * t + j) ^ g) * 16;
        const uint4 a = lds128(K + g * 128 + chunk), b = lds128(K + (8 + g) * 128 + chunk);
        const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t f[4];
          cvt_e4m3x4_to_f16x2x2(wa[w], f[0], f[2]);
          cvt_e4m3x4_to_f16x2x2(wb[w], f[1], f[3]);
#pragma unroll
          for (int n = 0; n < kTiles; ++n) mma_f16(kTiles == 1 && j ? z2[n] : z[n], f, qf[n][4 * j + w]);
        }
      }
      // Scores in log2 units; z[n][2 i + j]: key 8 i + g, row 2t + j.
      float top[kTiles][2];
#pragma unroll
      for (int n = 0; n < kTiles; ++n) top[n][0] = top[n][1] = kNegInf;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int kk = 8 * i + g;
        const float sk = scale_value(ks[kk]);
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float& y = z[n][2 * i + j];
            // (The factors first: y * sk may pass FP32's range.  A rounded product:
            // fused with the subtraction of the maximum it would differ from that by
            // the maximum's rounding, which can be large.)
            y = __fmul_rn(kTiles == 1 ? y + z2[n][2 * i + j] : y, sk * rowf[n][j]);
            top[n][j] = fmaxf(top[n][j], y);
          }
      }
      if (masked) {
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            int lo, hi;
            row_range(P, s, (p0 + 8 * n + 2 * t + j) / P.by_group, lo, hi);
            top[n][j] = kNegInf;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float& y = z[n][2 * i + j];
              const int key = key0 + 8 * i + g;
              if (key < lo || key > hi) y = kNegInf;
              top[n][j] = fmaxf(top[n][j], y);
            }
          }
      }
      // V's scales among the sequence's keys.
      int ev = vs[lane & 15];
      if (key0 + (lane & 15) >= s.kv || ev == 255) ev = -1;
      bool close = ev > E || (ev >= 0 && ev < E - kDecNear) || rows_apart;
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) top[n][j] = fmaxf(top[n][j], __shfl_xor_sync(0xFFFFFFFFu, top[n][j], d));
          close |= top[n][j] > m[n][j];
        }
      int En = E;
      close = __any_sync(0xFFFFFFFFu, close);
      if (close) {
        // A vector of zeros has 127 by the format and counts for nothing.
        if (__any_sync(0xFFFFFFFFu, ev == 127)) {
          const bool zero = zero_rows(V) >> (2 * (lane & 15)) & 1u;
          if (zero && ev == 127) ev = -1;
        }
        const int hi = __reduce_max_sync(0xFFFFFFFFu, ev), lo = __reduce_min_sync(0xFFFFFFFFu, ev < 0 ? 255 : ev);
        if (hi >= 0 && !rows_apart) {
          low = min(low, E < 0 ? min(lo, hi - kDecNear) : lo);
          En = max(E, hi);
          if (En - low > kDecSpread) return false;
        }
      }
      uint32_t pf[kTiles][2];
      if constexpr (!rows_apart) {
        if (close) {
          const float fe = exp2i(E - En);
          E = En;
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            float f[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float mn = fmaxf(m[n][j], top[n][j]);
              f[j] = m[n][j] == kNegInf ? 0.0f : ex2(m[n][j] - mn);
              m[n][j] = mn;
              l[n][j] *= f[j];
              f[j] *= fe;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[n][i][0] *= f[0];
              o[n][i][1] *= f[1];
              o[n][i][2] *= f[0];
              o[n][i][3] *= f[1];
            }
          }
        }
        // Weights: their sum in FP32, then rounded with the token's V scale.
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int kk = 8 * i + g;
          const uint32_t e = vs[kk];
          const float sv = e == 255u ? __uint_as_float(0x7FFFFFFFu) : exp2i(min(static_cast<int>(e) - E, 0) + kDecPBias);
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            float w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float y = z[n][2 * i + j];
              const float p = ex2(y - (m[n][j] == kNegInf ? 0.0f : m[n][j]));
              l[n][j] += p;
              w[j] = masked && y == kNegInf ? 0.0f : p * sv;
            }
            pf[n][i] = transpose8x8(pack2<true>(w[0], w[1]));
          }
        }
      } else {
        // The same with units by row.  E of a row follows its maximum down, and the
        // largest p 2^e of the block up.
        const uint32_t counts = __ballot_sync(0xFFFFFFFFu, ev >= 0);
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          float w[2][2];
          int Er[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float mn = fmaxf(m[n][j], top[n][j]), ref = mn == kNegInf ? 0.0f : mn, down = m[n][j] - ref;
            float x[2], most = kNegInf;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int kk = 8 * i + g;
              x[i] = z[n][2 * i + j] - ref + (counts >> kk & 1u ? static_cast<float>(vs[kk]) : 0.0f);
              most = fmaxf(most, x[i]);
            }
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
            const int Eo = first ? E : sm.e[warp][8 * n + 2 * t + j];
            Er[j] = max(0, max(__float2int_rd(static_cast<float>(Eo) + down), __float2int_rd(most)));
            const float f = m[n][j] == kNegInf ? 0.0f : ex2(down + static_cast<float>(Eo - Er[j]));
            l[n][j] *= ex2(down);
            m[n][j] = mn;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[n][i][j] *= f;
              o[n][i][2 + j] *= f;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float y = z[n][2 * i + j];
              l[n][j] += ex2(y - ref);
              w[i][j] = masked && y == kNegInf ? 0.0f
                        : vs[8 * i + g] == 255u ? __uint_as_float(0x7FFFFFFFu)
                                                : ex2(x[i] + static_cast<float>(kDecPBias - Er[j]));
            }
          }
          __syncwarp();                              // every lane has read its rows' E
          if (g == 0) {
            sm.e[warp][8 * n + 2 * t] = Er[0];
            sm.e[warp][8 * n + 2 * t + 1] = Er[1];
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) pf[n][i] = transpose8x8(pack2<true>(w[i][0], w[i][1]));
        }
        first = false;
      }
      // O^T += V^T P^T.
      const int left = s.kv - key0;                  // keys of the sequence from here on
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int kk = 2 * t + (i & 1) + 8 * (i >> 1);
        v[i] = lds128(V + kk * 128 + ((g ^ (kk & 7)) * 16));
        // Slots behind the sequence's end hold anything, NaN codes too.
        if (kk >= left) v[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&v[0]);
      const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&v[1]);
      const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&v[2]);
      const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&v[3]);
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t sel = y ? 0x7362u : 0x5140u;
          uint32_t f[4];
          cvt_e4m3x4_to_f16x2x2(__byte_perm(w0[w], w1[w], sel), f[0], f[1]);
          cvt_e4m3x4_to_f16x2x2(__byte_perm(w2[w], w3[w], sel), f[2], f[3]);
#pragma unroll
          for (int n = 0; n < kTiles; ++n) mma_f16(o[n][2 * w + y], f, pf[n]);
        }
      __syncwarp();                                  // every lane is done with the stage
      if (lane == 0) mbar_arrive(smem_addr(&sm.empty[warp][stage]));
      ++used;
      return true;
    };
    int kb = d.k0 + ((warp - (d.k0 - d.t0)) & (kDecWarps - 1));
#pragma unroll 1
    for (; kb < k1; kb += kDecWarps)
      if (!block(kb, std::false_type())) break;
#pragma unroll 1
    for (; kb < k1; kb += kDecWarps) block(kb, std::true_type());
    // The next part's rows, while this one ends.
    const int rows = d.rows, h = d.h, slot = d.slot;
    ++parts;
    {
      const DecodePart& after = sm.part[parts % kDecParts];
      more = wait(sm.part_full[parts % kDecParts], (parts / kDecParts) & 1) && after.more;
      if (more) load_q(after);
    }

    // Join the warps, 8 rows at a time, and write them: warp w takes rows w and
    // w + 4.  o[n][i][2 c + j]: channel 16 g + 2 i + c of row 2t + j.
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) l[n][j] += __shfl_xor_sync(0xFFFFFFFFu, l[n][j], d);
        const int r = 2 * t + j;
        if (g == 0) {
          sm.m[warp][r] = m[n][j];
          sm.l[warp][r] = l[n][j];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          reinterpret_cast<float4*>(sm.o[warp][r])[(4 * g + q) ^ r] =
              make_float4(o[n][2 * q][j], o[n][2 * q][2 + j], o[n][2 * q + 1][j], o[n][2 * q + 1][2 + j]);
      }
      if (n == 0 && first && lane < 16) sm.e[warp][lane] = max(E, 0);
      decode_sync();
#pragma unroll
      for (int r = warp; r < 8; r += kDecWarps) {
        if (8 * n + r >= rows) break;
        float top = kNegInf, total = 0.0f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) top = fmaxf(top, sm.m[w][r]);
        const float ref = top == kNegInf ? 0.0f : top;
        // The row's unit: a warp's is 2^(m + E).
        int Et = 0;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) Et = max(Et, sm.e[w][8 * n + r] + __float2int_rd(sm.m[w][r] - ref));
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
          const float d = sm.m[w][r] - ref, f = ex2(d), fe = ex2(d + static_cast<float>(sm.e[w][8 * n + r] - Et));
          total += sm.l[w][r] * f;
          const float4 y = reinterpret_cast<const float4*>(sm.o[w][r])[lane ^ r];
          acc.x += fe * y.x;
          acc.y += fe * y.y;
          acc.z += fe * y.z;
          acc.w += fe * y.w;
        }
        // 2^(E-127) and the weights' 2^-14; a row that saw no key has total 0.
        const float inv = total == 0.0f ? 0.0f : exp2i(-kDecPBias) / total, se = scale_value(Et);
        acc.x = acc.x * inv * se;
        acc.y = acc.y * inv * se;
        acc.z = acc.z * inv * se;
        acc.w = acc.w * inv * se;
        if (slot < 0) {
          const int p = p0 + 8 * n + r, tok = p / P.by_group, hq = h * P.group + p - tok * P.group;
          reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.o.ptr) + (s.q0 + tok) * P.o.st + hq * P.o.sh)[lane] =
              make_uint2(pack2<false>(acc.x, acc.y), pack2<false>(acc.z, acc.w));
          if (P.lse && lane == 0) P.lse[static_cast<int64_t>(s.q0 + tok) * P.Hq + hq] = total == 0.0f ? kNegInf : (top + log2f(total)) * 0.69314718055994531f;
        } else {
          const int64_t place = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * R + 8 * n + r;
          reinterpret_cast<float4*>(work.o + place * 128)[lane] = acc;
          if (lane == 0) work.ml[place] = make_float2(top, total);
        }
      }
      if (n + 1 < kTiles) decode_sync();
    }
    if (lane == 0) mbar_arrive(smem_addr(&sm.part_empty[(parts - 1) % kDecParts]));
    more = decode_sync_and(more);
  }
}

}  // namespace ovc
