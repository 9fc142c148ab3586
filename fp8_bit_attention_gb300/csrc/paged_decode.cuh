// paged_decode.cuh -- attention over the paged cache for few query rows per KV
// head: single tokens, drafted tokens, groups of query heads.
//
// Bound by memory: every key costs 258 bytes a head and each of them meets at
// most 32 query rows.  A CTA is eight warps; each streams its own 32-key blocks
// (4 KB of K, 4 KB of V) through a private ring of TMA tiles and keeps its own
// running maximum, sum and output in registers; no barrier joins the warps
// until the segment ends.
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
// token's V scale and E the largest so far, so that what is flushed is below
// 2^-39 of the largest possible term.
#pragma once

#include <cuda.h>

#include "paged_plan.cuh"

namespace ovc {

constexpr int kDecWarps = 8;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDecKeys = 32;                       // keys of a block
constexpr int kDecStages = 3;
constexpr uint32_t kDecCodes = kDecKeys * 128;     // bytes of a block's K (or V) codes
constexpr int kDecPBias = 14;

struct DecodeSmem {
  uint8_t kv[kDecWarps][kDecStages][2][kDecCodes];
  union {
    float o[kDecWarps][8][128];                    // the warps' outputs of 8 rows; 16-byte chunks swizzled by the row
    PlanSmem plan;                                 // before the first of them
  };
  uint8_t scale[kDecWarps][kDecStages][2][kDecKeys];
  float m[kDecWarps][8], l[kDecWarps][8];
  int e[kDecWarps];
  uint64_t full[kDecWarps][kDecStages];
  int abort;
  int zero;
};

static_assert(sizeof(DecodeSmem) <= 232448, "shared memory per CTA");

struct PagedMaps {
  CUtensorMap k, v;
  int32_t box;          // rows of a TMA box (divides the page and the key block)
  int32_t rows;         // rows of the cache: a box from there on reads zeros
  int32_t min_share;
  uint64_t timeout_ns;
};

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
               : "memory");
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

// A warp's loads: its blocks of the share (of each tile those w, w + 8, ...
// from the tile's first one on), in order, kDecStages ahead of its products.
template <int R>
struct DecodeLoader {
  Walk<R, kDecKeys> w;
  int kb;                 // next block of the part for this warp
  int seq, first;         // the lanes' rows belong to this sequence's blocks from `first` on (first < 0: none)
  int32_t row;            // lane n: box n % boxes of the warp's (n / boxes)-th block from `first` on, as the
                          // cache row of head 0; negative where the sequence has none
  bool more;

  // The warp's first block of the part at hand, or of the next part that has one.
  __device__ __forceinline__ void own(const PagedParams& P, int warp) {
    while (more) {
      kb = w.k0 + ((warp - (w.k0 - w.t0)) & (kDecWarps - 1));
      if (kb < w.k1) break;
      more = w.step(P);
    }
  }
};

template <bool kHalf, int kTiles>
__global__ void __launch_bounds__(kDecThreads, 1)
    paged_decode_kernel(const __grid_constant__ PagedParams P, const __grid_constant__ PagedMaps M, PagedWork work) {
  constexpr int R = 8 * kTiles;
  extern __shared__ __align__(1024) uint8_t raw[];
  DecodeSmem& sm = *reinterpret_cast<DecodeSmem*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) {
    sm.abort = 0;
    sm.zero = 0;
  }
  if (lane == 0) {
    for (int i = 0; i < kDecStages; ++i) mbar_init(smem_addr(&sm.full[warp][i]), 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    tma_prefetch_map(&M.k);
    tma_prefetch_map(&M.v);
  }
  __syncthreads();
  grid_dependency_allow();
  const Share share = plan_share<R, kDecKeys, kDecThreads, 1>(P, sm.plan, M.min_share);
  if (threadIdx.x == 0) write_cut<R, kDecKeys>(P, share, work);
  if (share.len == 0) return;
  __syncthreads();                                 // the plan's memory is free

  volatile int* const abort_flag = &sm.abort;
  const int boxes = kDecKeys / M.box;              // of a block: 1 or 2
  Walk<R, kDecKeys> at;
  bool more = at.start(P, share);
  DecodeLoader<R> ld;
  ld.w = at;
  ld.more = more;
  ld.first = -1;
  ld.seq = -1;
  ld.own(P, warp);
  uint32_t issued = 0, used = 0;

  // Issues the warp's next block into its ring.
  auto issue = [&]() {
    if (!ld.more || __any_sync(0xFFFFFFFFu, *abort_flag)) return;
    int entry = (ld.kb - ld.first) / kDecWarps * boxes;
    if (ld.first < 0 || ld.seq != ld.w.b || ld.kb < ld.first || entry >= 32 || ((ld.kb - ld.first) & (kDecWarps - 1))) {
      // The rows of the warp's next blocks: one page table look-up a lane.
      ld.first = ld.kb;
      ld.seq = ld.w.b;
      entry = 0;
      const int key = (ld.kb + lane / boxes * kDecWarps) * kDecKeys + lane % boxes * M.box;
      ld.row = -1;
      if (key < ld.w.s.kv && key < ld.w.t1 * kDecKeys) {
        const int n = key / P.c.page;
        const int p = __ldg(P.table + ld.w.b * P.table_stride + n);
        if (p >= 0 && p < P.c.pages) ld.row = p * P.c.heads * P.c.page + key - n * P.c.page;
        else atomicOr(P.status, kPagedBadIndex);
      }
    }
    const uint32_t stage = issued % kDecStages;
    const uint32_t bar = smem_addr(&sm.full[warp][stage]);
    int row = __shfl_sync(0xFFFFFFFFu, ld.row, entry + (lane < boxes ? lane : 0));
    row = row < 0 ? M.rows : row + ld.w.h * P.c.page;
    const unsigned in = __ballot_sync(0xFFFFFFFFu, lane < boxes && row < M.rows);
    if (lane == 0) mbar_arrive_expect_tx(bar, 2 * kDecCodes + __popc(in) * 2 * M.box);
    __syncwarp();
    if (lane < boxes) {
      const uint32_t at = lane * M.box;
      tma_load_2d(smem_addr(sm.kv[warp][stage][0]) + at * 128, &M.k, bar, 0, row);
      tma_load_2d(smem_addr(sm.kv[warp][stage][1]) + at * 128, &M.v, bar, 0, row);
      if (row < M.rows) {
        bulk_copy(smem_addr(sm.scale[warp][stage][0]) + at, P.c.ks + row, M.box, bar);
        bulk_copy(smem_addr(sm.scale[warp][stage][1]) + at, P.c.vs + row, M.box, bar);
      }
    }
    ++issued;
    ld.kb += kDecWarps;
    if (ld.kb >= ld.w.k1) {
      ld.more = ld.w.step(P);
      ld.own(P, warp);
    }
  };
#pragma unroll 1
  for (int i = 0; i < kDecStages; ++i) issue();

  // What the tile's rows need, the same for all heads: row g's place in q, and
  // of rows 2t, 2t+1, whose scores this lane will hold, the keys they see.
  const Seq& s = at.s;
  int rows = 0, lo[kTiles][2], hi[kTiles][2], all_lo = 0, all_hi = 0, join_t[kTiles], join_h[kTiles];
  const uint16_t* qrow[kTiles];
  for (; more; more = at.step(P)) {
    if (at.fresh) {
      const int p0 = at.i * R;
      rows = min(R, s.ql * P.group - p0);
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        const int p = p0 + 8 * n + g, tok = p / P.group;
        qrow[n] = static_cast<const uint16_t*>(P.q.ptr) + (s.q0 + tok) * P.q.st + (p - tok * P.group) * P.q.sh + 32 * t;
        const int pj = p0 + 8 * n + warp;
        join_t[n] = pj / P.group;
        join_h[n] = pj - join_t[n] * P.group;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int token = __shfl_sync(0xFFFFFFFFu, tok, (2 * t + j) * 4);
          lo[n][j] = 0;
          hi[n][j] = -1;
          if (8 * n + 2 * t + j < rows) row_range(P, s, token, lo[n][j], hi[n][j]);
        }
      }
      // Blocks within [all_lo, all_hi] need no mask.
      int x;
      row_range(P, s, (p0 + rows - 1) / P.group, all_lo, x);
      row_range(P, s, p0 / P.group, x, all_hi);
    }
    // Q's fragments: lane (g, t) holds row g of each tile, channels 32 t ..
    // 32 t + 31; and the factor of rows 2t, 2t+1 to log2 units.
    uint32_t qf[kTiles][8][2];
    float rowf[kTiles][2];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      uint4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (8 * n + g < rows) {
        const uint4* src = reinterpret_cast<const uint4*>(qrow[n] + at.h * (P.group * P.q.sh));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __ldg(src + i);
      }
      float f = P.c2;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qf[n][2 * i][0] = x[i].x;
        qf[n][2 * i][1] = x[i].y;
        qf[n][2 * i + 1][0] = x[i].z;
        qf[n][2 * i + 1][1] = x[i].w;
      }
      if (!kHalf) {
        // BF16 to FP16: the row's largest magnitude goes to [2^14, 2^15).
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 a = unpack2<false>(qf[n][i / 2][i % 2]);
          amax = fmaxf(amax, fmaxf(fabsf(a.x), fabsf(a.y)));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        const float mul = __uint_as_float(min(268u - (__float_as_uint(amax) >> 23), 254u) << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 a = unpack2<false>(qf[n][i / 2][i % 2]);
          qf[n][i / 2][i % 2] = pack2<true>(a.x * mul, a.y * mul);
        }
        f /= mul;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) rowf[n][j] = __shfl_sync(0xFFFFFFFFu, f, (2 * t + j) * 4);
    }

    float m[kTiles][2], l[kTiles][2], o[kTiles][8][4];
    int E = 0;
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

#pragma unroll 1
    for (int kb = at.k0 + ((warp - (at.k0 - at.t0)) & (kDecWarps - 1)); kb < at.k1; kb += kDecWarps) {
      const uint32_t stage = used % kDecStages;
      if (!mbar_wait(smem_addr(&sm.full[warp][stage]), (used / kDecStages) & 1, M.timeout_ns, abort_flag)) {
        // Give up: what follows works on whatever the ring holds, and no wait or
        // load is begun any more.
        if (lane == 0 && !*abort_flag) atomicOr(P.status, 1u);
        *abort_flag = 1;
      }
      ++used;
      const uint8_t* K = sm.kv[warp][stage][0];
      const uint8_t* V = sm.kv[warp][stage][1];
      const uint8_t* ks = sm.scale[warp][stage][0];
      const uint8_t* vs = sm.scale[warp][stage][1];
      const int key0 = kb * kDecKeys;
      const bool masked = key0 < all_lo || key0 + kDecKeys - 1 > all_hi;

      float z[kTiles][2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) z[n][u][j] = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t chunk = static_cast<uint32_t>((2 * t + j) ^ g) * 16;
          const uint4 a = lds128(K + (16 * u + g) * 128 + chunk), b = lds128(K + (16 * u + 8 + g) * 128 + chunk);
          const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t f[4];
            cvt_e4m3x4_to_f16x2x2(wa[w], f[0], f[2]);
            cvt_e4m3x4_to_f16x2x2(wb[w], f[1], f[3]);
#pragma unroll
            for (int n = 0; n < kTiles; ++n) mma_f16(z[n][u], f, qf[n][4 * j + w]);
          }
        }
      }
      // Scores in log2 units; z[n][u][2 i + j]: key 16 u + 8 i + g, row 2t + j.
      float top[kTiles][2];
#pragma unroll
      for (int n = 0; n < kTiles; ++n) top[n][0] = top[n][1] = kNegInf;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int kk = 16 * u + 8 * i + g;
          const float sk = scale_value(ks[kk]);
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float& y = z[n][u][2 * i + j];
              y = y * sk * rowf[n][j];
              if (masked && (key0 + kk < lo[n][j] || key0 + kk > hi[n][j])) y = kNegInf;
              top[n][j] = fmaxf(top[n][j], y);
            }
        }
      // The block's largest V scale among the sequence's keys.
      const uint32_t ev = vs[lane];
      const int Eb = __reduce_max_sync(0xFFFFFFFFu, key0 + lane < s.kv && ev != 255u ? static_cast<int>(ev) : 0);
      bool grown = Eb > E;
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) top[n][j] = fmaxf(top[n][j], __shfl_xor_sync(0xFFFFFFFFu, top[n][j], d));
          grown |= top[n][j] > m[n][j];
        }
      if (__any_sync(0xFFFFFFFFu, grown)) {
        const int En = max(E, Eb);
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
      uint32_t pf[kTiles][2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int kk = 16 * u + 8 * i + g;
          const uint32_t e = vs[kk];
          const float sv = e == 255u ? __uint_as_float(0x7FFFFFFFu) : exp2i(static_cast<int>(e) - E + kDecPBias);
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            float w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float y = z[n][u][2 * i + j];
              const float p = ex2(y - (m[n][j] == kNegInf ? 0.0f : m[n][j]));
              l[n][j] += p;
              w[j] = masked && y == kNegInf ? 0.0f : p * sv;
            }
            pf[n][u][i] = transpose8x8(pack2<true>(w[0], w[1]));
          }
        }
      // O^T += V^T P^T.
      const int left = s.kv - key0;                  // keys of the sequence from here on
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kk = 16 * u + 2 * t + (i & 1) + 8 * (i >> 1);
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
            for (int n = 0; n < kTiles; ++n) mma_f16(o[n][2 * w + y], f, pf[n][u]);
          }
      }
      __syncwarp();                                  // every lane is done with the stage
      issue();
    }

    // Join the warps, 8 rows at a time, and write them: warp w takes row w.
    // o[n][i][2 c + j]: channel 16 g + 2 i + c of row 2t + j.
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
      if (n == 0 && lane == 0) sm.e[warp] = E;
      __syncthreads();
      const int r = warp;
      float top = kNegInf, total = 0.0f;
      int Et = 0;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        top = fmaxf(top, sm.m[w][r]);
        Et = max(Et, sm.e[w]);
      }
      const float ref = top == kNegInf ? 0.0f : top;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float f = ex2(sm.m[w][r] - ref), fe = f * exp2i(sm.e[w] - Et);
        total += sm.l[w][r] * f;
        const float4 y = reinterpret_cast<const float4*>(sm.o[w][r])[lane ^ r];
        acc.x += fe * y.x;
        acc.y += fe * y.y;
        acc.z += fe * y.z;
        acc.w += fe * y.w;
      }
      if (8 * n + r < rows) {
        // 2^(E-127) and the weights' 2^-14; a row that saw no key has total 0.
        const float inv = total == 0.0f ? 0.0f : exp2i(-kDecPBias) / total, se = scale_value(Et);
        acc.x = acc.x * inv * se;
        acc.y = acc.y * inv * se;
        acc.z = acc.z * inv * se;
        acc.w = acc.w * inv * se;
        const float L = total == 0.0f ? kNegInf : top + log2f(total);
        if (at.whole) {
          const int tok = s.q0 + join_t[n], hq = at.h * P.group + join_h[n];
          reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.o.ptr) + tok * P.o.st + hq * P.o.sh)[lane] =
              make_uint2(pack2<false>(acc.x, acc.y), pack2<false>(acc.z, acc.w));
          if (P.lse && lane == 0) P.lse[static_cast<int64_t>(tok) * P.Hq + hq] = L * 0.69314718055994531f;
        } else {
          const int64_t place = (static_cast<int64_t>(blockIdx.x) * 2 + at.slot) * R + 8 * n + r;
          reinterpret_cast<float4*>(work.o + place * 128)[lane] = acc;
          if (lane == 0) work.lse[place] = L;
        }
      }
      __syncthreads();
    }
  }
  // After a timeout copies may still be in flight: they end by themselves, and
  // the CTA's shared memory must outlive them.
  if (*abort_flag)
    for (; used < issued; ++used)
      mbar_wait(smem_addr(&sm.full[warp][used % kDecStages]), (used / kDecStages) & 1, 4000000000ull, &sm.zero);
}

}  // namespace ovc
