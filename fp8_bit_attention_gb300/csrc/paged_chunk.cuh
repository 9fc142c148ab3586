// paged_chunk.cuh -- attention over the paged cache for many query rows per KV
// head: chunks of new tokens, on the tensor cores (tcgen05).
//
// A tile is 256 query rows (tokens times query heads of one KV head) in two
// halves of 128; a turn is one half's work on a block of 128 keys, whose softmax
// takes two steps of 64 keys.  Halves t = 0, 1:
//   S_t = Q_t K^T          kind::f8f6f4.  K's codes go in as they lie in the
//                          cache (TMA tiles, K-major); Q enters as a sum of
//                          E4M3 parts, each the rounding error of the ones
//                          before it: two parts hold a BF16 row (8 bits), three
//                          an FP16 row (11 bits), but for what lies below 2^-18
//                          of the row's largest element.  Two 8-bit products
//                          cost what one 16-bit product costs, and K needs no
//                          conversion.
//   O_t += P_t V           kind::f16.  P is FP16 and read from tensor memory,
//                          where it overwrites S_t; V's codes are converted to
//                          FP16 (exactly) by four warps, once per block for all
//                          256 rows, with the token's scale: V 2^(e - E + 7), E
//                          the largest scale so far.
// While one half's softmax runs, the tensor core works on the other half.  The
// softmax hands over P one step at a time, so that the first step's product runs
// beside the second step's softmax.  A tile of at most 128 rows keeps the overlap
// by giving the blocks to the halves in turn, both on the same rows, and joining
// the two results at the end ("solo").
//
// What bounds it: long calls, the softmax beside the products.  4096 tokens x 32
// heads over 65536 keys take 3.05 ms, 1390 TFLOP/s, 72% of a library product's
// rate; a turn's 16 MMA instructions take 1026 cycles of the tensor core, its
// softmax 1500 to 1870 of its four warps while the others run (900 alone), and
// two turns in step 2900.  Calls of many tiles with few keys, what a tile costs
// beside its blocks: 8 us (Q's rows in, their conversion, the first scores, O's
// rows out; one CTA fills the SM, so nothing covers them): 8 prompts of 512 tokens,
// 32 heads, 55 us, one of 1024 tokens 39 us, a batch of chunks and short sequences
// 81 us.
// Few rows over many keys ("solo"): 8 x 65536 keys x 8 heads for 32 rows 237 us, 67%
// of a copy's rate.  Without V's conversion and softmax such a call took 200 of 232
// us, so more than half of the gap lies elsewhere, and FP16, with one stage of V's
// codes and two of K's, takes 360: too few bytes are on their way.  Instructions
// are a resource: every warp role runs its own code at once, and waiting for
// instructions was the second largest stall, so what is not in the inner loop is
// kept in loops of little code, or of its own.
//
// Measured and left out (ms for 4096 over 65536; the kernel of the time in
// brackets): scores of 64 keys in two buffers a half 3.5 (3.1); 16 softmax warps,
// two threads a row, 3.7 (3.1); a warp issuing products for each half 3.9 (3.1);
// O through shared memory, for stores of whole rows, 3.6 (3.1); the next tile's Q
// in registers before the end of the one before 3.35 (3.06); scores 32 at a time,
// the next ones on their way, 3.22 (3.05); warps without a row hand over at once,
// 1% slower where all have some, 3% faster for 32 rows.
//
// Warps: 0-3 and 4-7 softmax of the halves, a thread per row; 8-11 convert V; 12
// walks the share, looks up pages and loads K and V; 13 issues the products; 14
// loads the scales; 15 idles.  All waits are bounded.
//
// Numbers: scores, references, sums and outputs are FP32.  Weights are 2^7 p
// relative to a reference, the row's maximum when it was last looked for: that is
// when the weights of a step add up to 2^15.5, so that none passes FP16's
// largest value (O is then rescaled in tensor memory).  What is lost of a weight
// is below 2^-32 of the one at the reference.  V's values are exact as long as its
// scales spread over at most 2^kChSpread.  Beyond that ("wide") V goes in without
// its scales and they go into the weights, which are then 2^7 p 2^(e - E) with an E
// of each row's own, of the largest p 2^e that it sees: a token counts by its term
// and one that is masked not at all.  Either way no more than 2^-20 of a row's
// largest term is lost.  (All blocks wide: 4096 over 65536 9.1 ms, 32 rows 648 us.)
#pragma once

#include "paged_decode.cuh"

namespace ovc {

constexpr int kChRows = 256;
constexpr int kChKeys = 128;
constexpr int kChStep = 64;                        // keys of a softmax step
constexpr int kChThreads = 512;
// Registers: 512 threads of 128 at launch; 256 x 184 + 256 x 72 = 512 x 128.
constexpr int kChSoftmaxRegs = 184;
constexpr int kChOtherRegs = 72;
static_assert(256 * kChSoftmaxRegs + 256 * kChOtherRegs <= kChThreads * 128, "register split");
constexpr uint32_t kChTile = 128 * 128;            // bytes of an E4M3 tile
constexpr uint32_t kChTile16 = 2 * kChTile;        // bytes of V in FP16
constexpr float kChPBias = 7.0f;                   // log2 of the weight at the reference
constexpr float kChSumLimit = 46341.0f;            // 2^15.5: a row's weights in a step stay below FP16's largest value
constexpr int kChVBias = 7;
// Scales of V that spread further go into the weights.  A block is looked at
// closely where a scale is above E or more than kChNear below it.
constexpr int kChSpread = 12, kChNear = 6;
constexpr int kChParts = 4;

template <bool kHalf>
struct ChunkShape {
  static constexpr int kQParts = kHalf ? 3 : 2;
  static constexpr int kK = kHalf ? 2 : 3;         // stages of K
  static constexpr int kV = kHalf ? 1 : 2;         // stages of V's codes
  static constexpr int kScales = 4;
};

// A block's scales: those of K times the scores' factor to log2 units (the row's
// factor is then a power of two, and a score less the row's maximum one exact
// subtraction, however large both are) over kmul, those of V as FP16 pairs 2^(e-E+7), or
// 2^7 where they go into the weights.
struct alignas(16) ChunkScales {
  float k[kChKeys];
  uint32_t v[kChKeys];
  uint8_t nan[kChKeys];                            // 1: K's scale is NaN, 2: V's (their values above are 1 and 0)
  uint8_t ve[kChKeys];                             // wide: V's e, 0 for vectors of zeros
  int e;                                           // E, from the first wide block on unchanged
  int rare;                                        // 1: any such NaN, 2: wide
  float kmul;                                      // 1, or what brings the largest scale of K down to k_most
};

// A tile's part.
struct ChunkPart {
  int more;
  int b, q0, ql, kv;
  int p0, rows, h;
  int k0, nblk;
  int all_lo, all_hi;
  int slot;                                        // negative: the tile is whole
};

template <bool kHalf>
struct ChunkSmem {
  using Sh = ChunkShape<kHalf>;
  uint8_t q[Sh::kQParts][2][kChTile];
  uint8_t k[Sh::kK][kChTile];
  uint8_t v8[Sh::kV][kChTile];
  uint8_t v16[2][kChTile16];                       // [64-channel half][key][128 bytes]
  union {
    ChunkScales sc[Sh::kScales];
    PlanSmem plan;
  };
  float2 ml[128];                                  // solo: the second half's reference and sum
  int e1[128];                                     // and its E
  ChunkPart part[kChParts];
  uint64_t k_full[Sh::kK], k_empty[Sh::kK];
  uint64_t v8_full[Sh::kV], v8_empty[Sh::kV];
  uint64_t v16_full[2], v16_empty[2];
  uint64_t sc_full[Sh::kScales], sc_empty[Sh::kScales];
  uint64_t s_full[2], p_full[2][2];                // [half], [half][step of a block]
  uint64_t o_done[2], o_full[2];                   // the products of a block's first step, of a part are complete
  uint64_t q_full, x_full, x_empty;
  uint64_t part_full[kChParts], part_empty[kChParts];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int zero;
};
static_assert(sizeof(ChunkSmem<false>) <= 232448 && sizeof(ChunkSmem<true>) <= 232448, "shared memory per CTA");

// Descriptor of V in FP16: MN-major (channels contiguous), 128-byte swizzle;
// 64-channel halves 16 KB apart, groups of 8 keys 1024 bytes apart.
__device__ __forceinline__ uint64_t v16_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(kChTile >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

// kind::f16 with FP16 operands, FP32 result, A K-major, B MN-major (bit 16).
constexpr uint32_t kChIdescPV = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kChIdescQK = idesc_e4m3_f32(128, 128);

// D[tmem] (+)= A[tmem] B[smem], 16-bit operands, by a converged warp.
__device__ __forceinline__ void mma_16_ts_w(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint64_t pack_f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack_f2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// One column of this thread's lane of tensor memory.
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t x;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(x)
      : "r"(taddr)
      : "memory");
  return x;
}

// 2^x as an FP16 pair, x <= 15.
__device__ __forceinline__ uint32_t exp2h2(int x) {
  const uint32_t h = x >= -14 ? static_cast<uint32_t>(x + 15) << 10 : x >= -24 ? 1u << (x + 24) : 0u;
  return h | (h << 16);
}

// E4M3 pair -> the values as floats.
__device__ __forceinline__ float2 e4m3x2_values(uint32_t pair) {
  uint32_t h;
  asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(h) : "r"(pair));
  return unpack2<true>(h);
}

// 32 bytes in one load or store (a whole sector): the address is a multiple of 32.
__device__ __forceinline__ void load8(uint32_t* w, const void* from) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(__cvta_generic_to_global(from)));
}
__device__ __forceinline__ void store8(void* to, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(__cvta_generic_to_global(to)), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(__cvta_generic_to_global(p)));
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Two FP16 pairs -> four E4M3 bytes in order (nearest even, saturating).
__device__ __forceinline__ uint32_t e4m3x4_of_f16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("{\n\t.reg .b16 x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 x, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 y, %2;\n\t"
      "mov.b32 %0, {x, y};\n\t}"
      : "=r"(d)
      : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ ChunkPart uniform(const ChunkPart& x) {
  return {uniform(x.more), uniform(x.b),    uniform(x.q0),   uniform(x.ql),     uniform(x.kv),     uniform(x.p0),  uniform(x.rows),
          uniform(x.h),    uniform(x.k0),   uniform(x.nblk), uniform(x.all_lo), uniform(x.all_hi), uniform(x.slot)};
}

template <bool kHalf>
__global__ void __launch_bounds__(kChThreads, 1)
    paged_chunk_kernel(const __grid_constant__ PagedParams P, const __grid_constant__ PagedMaps M, PagedWork work) {
  using Sh = ChunkShape<kHalf>;
  extern __shared__ __align__(1024) uint8_t raw[];
  ChunkSmem<kHalf>& sm = *reinterpret_cast<ChunkSmem<kHalf>*>(raw);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile int* const abort_flag = &sm.abort;
  constexpr int kReaders = 4 + 1 + 1 + 8;          // warps that read a part's description: V, products, scales, softmax
  if (threadIdx.x == 0) {
    sm.abort = 0;
    sm.zero = 0;
    for (int i = 0; i < Sh::kK; ++i) {
      mbar_init(smem_addr(&sm.k_full[i]), 1);
      mbar_init(smem_addr(&sm.k_empty[i]), 1);
    }
    for (int i = 0; i < Sh::kV; ++i) {
      mbar_init(smem_addr(&sm.v8_full[i]), 1);
      mbar_init(smem_addr(&sm.v8_empty[i]), 4);
    }
    for (int i = 0; i < Sh::kScales; ++i) {
      mbar_init(smem_addr(&sm.sc_full[i]), 1);
      mbar_init(smem_addr(&sm.sc_empty[i]), 12);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sm.v16_full[i]), 128);
      mbar_init(smem_addr(&sm.v16_empty[i]), 1);
      mbar_init(smem_addr(&sm.s_full[i]), 1);
      for (int j = 0; j < 2; ++j) mbar_init(smem_addr(&sm.p_full[i][j]), 128);
      mbar_init(smem_addr(&sm.o_done[i]), 1);
      mbar_init(smem_addr(&sm.o_full[i]), 1);
    }
    for (int i = 0; i < kChParts; ++i) {
      mbar_init(smem_addr(&sm.part_full[i]), 1);
      mbar_init(smem_addr(&sm.part_empty[i]), kReaders);
    }
    mbar_init(smem_addr(&sm.q_full), 256);
    mbar_init(smem_addr(&sm.x_full), 128);
    mbar_init(smem_addr(&sm.x_empty), 128);
    mbar_init(smem_addr(&sm.drain), 1);
    fence_mbar_init();
    tma_prefetch_map(&M.k);
    tma_prefetch_map(&M.v);
  }
  grid_dependency_allow();
  __syncthreads();
  const Share share = plan_share<kChRows, kChKeys, kChThreads, 32>(P, sm.plan, M.min_share);
  if (share.len == 0) {
    if (threadIdx.x == 0) write_cut<kChRows, kChKeys>(P, share, work);
    return;
  }
  if (warp == 13) {
    tmem_alloc(smem_addr(&sm.tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();                                 // also: the plan's memory is free
  tc_fence_after();
  const uint32_t tmem = uniform(sm.tmem_base);

  auto wait = [&](uint64_t& bar, uint32_t parity) -> bool { return paged_wait(smem_addr(&bar), parity, M.timeout_ns, abort_flag); };
  auto give_up = [&]() {
    if (!*abort_flag) atomicOr(P.status, 1u);
    *abort_flag = 1;
  };

  if (warp >= 8) {
    regs_dec<kChOtherRegs>();
    if (warp == 12) {
      // -------------------------------------------------- the share, K and V
      Walk<kChRows, kChKeys> w(P, share);
      uint32_t parts = 0, n = 0, nv = 0;           // blocks whose K, V were loaded
      bool ok = true;
      const int boxes = kChKeys / M.box;
      while (true) {
        const bool more = w.step(P);
        const uint32_t d = parts % kChParts;
        if (parts >= kChParts) ok = __all_sync(0xFFFFFFFFu, wait(sm.part_empty[d], (parts / kChParts - 1) & 1));
        if (!ok) break;
        if (lane == 0) {
          ChunkPart& x = sm.part[d];
          x.more = more;
          if (more) {
            int y;
            x.b = w.b;
            x.q0 = w.s.q0;
            x.ql = w.s.ql;
            x.kv = w.s.kv;
            x.p0 = w.i * kChRows;
            x.rows = min(kChRows, w.s.ql * P.group - x.p0);
            x.h = w.h;
            x.k0 = w.k0;
            x.nblk = w.k1 - w.k0;
            x.slot = w.whole ? -1 : w.slot;
            row_range(P, w.s, (x.p0 + x.rows - 1) / P.by_group, x.all_lo, y);
            row_range(P, w.s, x.p0 / P.by_group, y, x.all_hi);
          }
          mbar_arrive(smem_addr(&sm.part_full[d]));
        }
        ++parts;
        if (!more) break;
        // Its query rows go to L2 while the part before it still runs.
        if (parts > 1) {
          const int p0 = w.i * kChRows, rows = min(kChRows, w.s.ql * P.group - p0);
          for (int i = lane; i < rows; i += 32) {
            const int tok = (p0 + i) / P.by_group;
            const uint16_t* src = static_cast<const uint16_t*>(P.q.ptr) + (w.s.q0 + tok) * P.q.st + (w.h * P.group + p0 + i - tok * P.group) * P.q.sh;
            prefetch_l2(src);
            prefetch_l2(src + 64);
          }
        }
        auto lookup = [&](int kb) {
          const int key = kb * kChKeys + lane * M.box;
          int row = M.rows;                        // past the cache's end: reads zeros
          if (lane < boxes && kb < w.k1 && key < w.s.kv) {
            const int i = key / P.by_page;
            const int p = __ldg(P.table + w.b * P.table_stride + i);
            if (p >= 0 && p < P.c.pages) row = (p * P.c.heads + w.h) * P.c.page + key - i * P.c.page;
            else atomicOr(P.status, kPagedBadIndex);
          }
          return row;
        };
        int row = lookup(w.k0);
        for (int kb = w.k0; kb < w.k1; ++kb) {
          const int next = lookup(kb + 1);
          const uint32_t ks = n % Sh::kK, vs = nv % Sh::kV;
          if (n >= Sh::kK) ok = __all_sync(0xFFFFFFFFu, wait(sm.k_empty[ks], (n / Sh::kK - 1) & 1));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(smem_addr(&sm.k_full[ks]), kChTile);
          __syncwarp();
          if (lane < boxes) tma_load_2d(smem_addr(sm.k[ks]) + lane * M.box * 128, &M.k, smem_addr(&sm.k_full[ks]), 0, row);
          ++n;
          if (nv >= Sh::kV) ok = __all_sync(0xFFFFFFFFu, wait(sm.v8_empty[vs], (nv / Sh::kV - 1) & 1));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(smem_addr(&sm.v8_full[vs]), kChTile);
          __syncwarp();
          if (lane < boxes) tma_load_2d(smem_addr(sm.v8[vs]) + lane * M.box * 128, &M.v, smem_addr(&sm.v8_full[vs]), 0, row);
          ++nv;
          row = next;
        }
        if (!ok) break;
      }
      if (lane == 0) write_cut<kChRows, kChKeys>(P, share, work);
      if (!ok) give_up();
      // The CTA's shared memory must outlive the copies in flight, also where others
      // give up on them after this warp's last wait.
      for (uint32_t i = n > Sh::kK ? n - Sh::kK : 0; i < n; ++i)
        paged_wait(smem_addr(&sm.k_full[i % Sh::kK]), (i / Sh::kK) & 1, 4000000000ull, &sm.zero);
      for (uint32_t i = nv > Sh::kV ? nv - Sh::kV : 0; i < nv; ++i)
        paged_wait(smem_addr(&sm.v8_full[i % Sh::kV]), (i / Sh::kV) & 1, 4000000000ull, &sm.zero);
    } else if (warp == 13) {
      // --------------------------------------------------------- the products
      // By one warp, the halves in turn: with a warp for each the two fall into
      // step, and both softmaxes wait for both halves' products (3.9 against 3.1
      // ms for 4096 tokens x 32 heads over 65536 keys).  What the products are
      // told must be in uniform registers: computed per lane, each costs the warp
      // several times its 64 cycles (3.7 ms).
      uint32_t parts = 0, n = 0, phase = 0;          // bit t: parity of half t's weights
      bool ok = true, issued = false;
      const uint64_t qd = sw128_desc(smem_addr(sm.q[0][0]));
      while (true) {
        const uint32_t d = parts % kChParts;
        ok = __all_sync(0xFFFFFFFFu, wait(sm.part_full[d], (parts / kChParts) & 1));
        if (!ok || !sm.part[d].more) break;
        const int nblk = uniform(sm.part[d].nblk);
        const bool solo = uniform(sm.part[d].rows) <= 128;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.part_empty[d]));
        ok = __all_sync(0xFFFFFFFFu, wait(sm.q_full, parts & 1));
        if (!ok) break;
        ++parts;
        tc_fence_after();
        // Turn i: half i & 1 on block i / 2, in solo on block i.
        const int total = solo ? nblk : 2 * nblk;
        auto wait_k = [&](int i) {
          const uint32_t blk = n + (solo ? i : i >> 1);
          ok = __all_sync(0xFFFFFFFFu, wait(sm.k_full[blk % Sh::kK], (blk / Sh::kK) & 1));
        };
        auto scores = [&](int i) {
          const int t = i & 1;
          const uint32_t blk = n + (solo ? i : i >> 1), ks = blk % Sh::kK;
          const uint64_t kd = sw128_desc(smem_addr(sm.k[ks]));
#pragma unroll
          for (int part = 0; part < Sh::kQParts; ++part)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f8_ss_w(tmem + t * 128, qd + (part * 2 + (solo ? 0 : t)) * (kChTile >> 4) + 2 * kk, kd + 2 * kk, kChIdescQK,
                          part > 0 || kk > 0);
          tc_commit_w(smem_addr(&sm.s_full[t]));
          if (solo || t == 1) tc_commit_w(smem_addr(&sm.k_empty[ks]));
          issued = true;
        };
#pragma unroll 1
        for (int i = 0; i < 2 && i < total; ++i) {
          wait_k(i);
          if (!ok) break;
          tc_fence_after();
          scores(i);
        }
        for (int i = 0; i < total && ok; ++i) {
          const int t = i & 1;
          const uint32_t blk = n + (solo ? i : i >> 1), vs = blk & 1;
          const uint64_t vd = v16_desc(smem_addr(sm.v16[vs]));
          // The waits for what has long been there come first: even a wait for a
          // completed barrier takes a round trip.
          if (i + 2 < total && (solo || t == 0)) wait_k(i + 2);
          if (ok && (solo || t == 0)) ok = __all_sync(0xFFFFFFFFu, wait(sm.v16_full[vs], (blk >> 1) & 1));
          if (!ok) break;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = __all_sync(0xFFFFFFFFu, wait(sm.p_full[t][half], phase >> t & 1));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
              mma_16_ts_w(tmem + 256 + t * 128, tmem + t * 128 + 8 * kk, vd + kk * (2048 >> 4), kChIdescPV, i > 1 || kk > 0);
            if (half == 0) tc_commit_w(smem_addr(&sm.o_done[t]));
          }
          if (!ok) break;
          phase ^= 1u << t;
          if (solo || t == 1) tc_commit_w(smem_addr(&sm.v16_empty[vs]));
          if (i + 2 < total) scores(i + 2);
          else tc_commit_w(smem_addr(&sm.o_full[t]));
        }
        if (!ok) break;
        n += nblk;
      }
      if (!ok) give_up();
      if (issued) {
        // Every product issued so far has completed once this barrier flips.
        tc_commit_w(smem_addr(&sm.drain));
        paged_wait(smem_addr(&sm.drain), 0, 4000000000ull, &sm.zero);
      }
    } else if (warp == 14) {
      // ----------------------------------------------------------- the scales
      uint32_t parts = 0, n = 0;
      bool ok = true;
      while (true) {
        const uint32_t d = parts % kChParts;
        ok = __all_sync(0xFFFFFFFFu, wait(sm.part_full[d], (parts / kChParts) & 1));
        if (!ok || !sm.part[d].more) break;
        const ChunkPart x = uniform(sm.part[d]);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.part_empty[d]));
        ++parts;
        // Lane i takes keys 4 i .. 4 i + 3 (one page holds them), from `row` of the
        // cache on.
        auto load = [&](int i, uint32_t& kw, uint32_t& vw, int& row) {
          const int key = (x.k0 + i) * kChKeys + 4 * lane;
          kw = vw = 0;
          row = 0;
          if (i < x.nblk && key < x.kv) {
            const int j = key / P.by_page;
            const int p = __ldg(P.table + x.b * P.table_stride + j);
            if (p >= 0 && p < P.c.pages) {
              row = (p * P.c.heads + x.h) * P.c.page + key - j * P.c.page;
              kw = *reinterpret_cast<const uint32_t*>(P.c.ks + row);
              vw = *reinterpret_cast<const uint32_t*>(P.c.vs + row);
            }
          }
        };
        uint32_t kw, vw;
        int row;
        load(0, kw, vw, row);
        int E = -1, low = 255;                     // the scales of V so far: the largest, none below
        int wide = 0;
        for (int i = 0; i < x.nblk; ++i, ++n) {
          uint32_t kn, vn;
          int rown;
          load(i + 1, kn, vn, rown);
          const uint32_t s = n % Sh::kScales;
          const int left = x.kv - ((x.k0 + i) * kChKeys + 4 * lane);
          int most = -1, least = 255, kmost = 0;     // V's scales, the largest of K
          uint32_t nan = 0, zeros = 0;
          bool poison = false;
          float kmul = 1.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < left) {
              const int ev = (vw >> (8 * j)) & 255u;
              most = max(most, ev);
              least = min(least, ev);
              kmost = max(kmost, static_cast<int>((kw >> (8 * j)) & 255u));
            }
          if (__any_sync(0xFFFFFFFFu, most > E || least < E - kChNear || kmost > P.k_most || wide)) {
            most = -1;
            least = 255;
            kmost = 0;
#pragma unroll 1
            for (int j = 0; j < 4 && j < left; ++j) {
              const int ev = (vw >> (8 * j)) & 255u, ek = (kw >> (8 * j)) & 255u;
              if (ek == 255) nan |= 1u << (8 * j);
              else kmost = max(kmost, ek);
              // A vector of zeros has 127 by the format and counts for nothing.
              uint32_t any = 1;
              if (ev == 127) {
                const uint4* codes = reinterpret_cast<const uint4*>(P.c.v + static_cast<int64_t>(row + j) * 128);
                any = 0;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  const uint4 y = codes[c];
                  any |= y.x | y.y | y.z | y.w;
                }
                any &= 0x7F7F7F7Fu;
              }
              if (ev == 255) nan |= 2u << (8 * j);
              if (ev == 255 || any == 0) {
                zeros |= 255u << (8 * j);
              } else {
                most = max(most, ev);
                least = min(least, ev);
              }
            }
            most = __reduce_max_sync(0xFFFFFFFFu, most);
            least = __reduce_min_sync(0xFFFFFFFFu, least);
            if (most >= 0) {
              low = min(low, E < 0 ? min(least, most - kChNear) : least);
              if (max(E, most) - low > kChSpread) wide = 2;      // and stays so
              if (!wide) E = max(E, most);
            }
            poison = __any_sync(0xFFFFFFFFu, nan != 0);
            kmul = exp2i(min(max(__reduce_max_sync(0xFFFFFFFFu, kmost) - P.k_most, 0), 127));
          }
          if (n >= Sh::kScales) ok = __all_sync(0xFFFFFFFFu, wait(sm.sc_empty[s], (n / Sh::kScales - 1) & 1));
          if (!ok) break;
          ChunkScales& sc = sm.sc[s];
          float4 f;
          uint4 h;
          // Never 0, which would make a hidden key's score NaN.
          const float c2 = kmul == 1.0f ? P.c2 : P.c2 / kmul;
          auto kscale = [&](uint32_t ek) { return ek == 255u ? 1.0f : fmaxf(c2 * scale_value(ek), __uint_as_float(1u)); };
          f.x = kscale(kw & 255u);
          f.y = kscale((kw >> 8) & 255u);
          f.z = kscale((kw >> 16) & 255u);
          f.w = kscale(kw >> 24);
          const int to = wide ? 0 : E;
          auto vscale = [&](uint32_t ev) { return ev == 255u ? 0u : exp2h2(min(static_cast<int>(ev) - to, 0) + kChVBias); };
          h.x = vscale(vw & 255u);
          h.y = vscale((vw >> 8) & 255u);
          h.z = vscale((vw >> 16) & 255u);
          h.w = vscale(vw >> 24);
          reinterpret_cast<float4*>(sc.k)[lane] = f;
          reinterpret_cast<uint4*>(sc.v)[lane] = h;
          reinterpret_cast<uint32_t*>(sc.nan)[lane] = nan;
          if (wide) reinterpret_cast<uint32_t*>(sc.ve)[lane] = vw & ~zeros;
          if (lane == 0) {
            sc.e = max(E, 0);
            sc.rare = poison | wide;
            sc.kmul = kmul;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sm.sc_full[s]));
          kw = kn;
          vw = vn;
          row = rown;
        }
        if (!ok) break;
      }
      if (!ok) give_up();
    } else if (warp < 12) {
      // ------------------------------------------------- V's codes to FP16
      const int w = warp - 8;
      uint32_t parts = 0, n = 0;
      bool ok = true;
      while (true) {
        const uint32_t d = parts % kChParts;
        ok = __all_sync(0xFFFFFFFFu, wait(sm.part_full[d], (parts / kChParts) & 1));
        if (!ok || !sm.part[d].more) break;
        const int nblk = uniform(sm.part[d].nblk), k0 = uniform(sm.part[d].k0), kv = uniform(sm.part[d].kv);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.part_empty[d]));
        ++parts;
        for (int i = 0; i < nblk; ++i, ++n) {
          const uint32_t vs = n % Sh::kV, ss = n % Sh::kScales, os = n & 1;
          ok = wait(sm.v8_full[vs], (n / Sh::kV) & 1) && wait(sm.sc_full[ss], (n / Sh::kScales) & 1);
          if (ok && n >= 2) ok = wait(sm.v16_empty[os], ((n >> 1) - 1) & 1);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          // Eight lanes take a key's 128 channels, 16 each: 16 bytes in, 2 x 16
          // out.  The lanes of the upper 64 channels work on the neighbouring key
          // (r ^ 1), so that the eight lanes of a load or store meet all banks.
          const int c = lane & 7, half = c >> 2, c0 = 2 * (c & 3);
          const int left = kv - (k0 + i) * kChKeys;
          const uint8_t* src = sm.v8[vs];
          uint8_t* dst = sm.v16[os] + half * kChTile;
          const uint32_t* sv = sm.sc[ss].v;
#pragma unroll 2
          for (int j = 0; j < 8; ++j) {
            const int r = 32 * w + 4 * j + ((lane >> 3) ^ half), x7 = (4 * (j & 1) + ((lane >> 3) ^ half)) & 7;
            uint4 x = lds128(src + r * 128 + ((c ^ x7) << 4));
            if (left < kChKeys && r >= left) x = make_uint4(0u, 0u, 0u, 0u);     // behind the sequence's end: anything
            const uint32_t f = sv[r];
            uint4 a, b;
            cvt_e4m3x4_to_f16x2x2(x.x, a.x, a.y);
            cvt_e4m3x4_to_f16x2x2(x.y, a.z, a.w);
            cvt_e4m3x4_to_f16x2x2(x.z, b.x, b.y);
            cvt_e4m3x4_to_f16x2x2(x.w, b.z, b.w);
            uint8_t* row = dst + r * 128;
            *reinterpret_cast<uint4*>(row + ((c0 ^ x7) << 4)) = make_uint4(hmul2(a.x, f), hmul2(a.y, f), hmul2(a.z, f), hmul2(a.w, f));
            *reinterpret_cast<uint4*>(row + (((c0 + 1) ^ x7) << 4)) = make_uint4(hmul2(b.x, f), hmul2(b.y, f), hmul2(b.z, f), hmul2(b.w, f));
          }
          fence_proxy_async_smem();
          mbar_arrive(smem_addr(&sm.v16_full[os]));
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_addr(&sm.v8_empty[vs]));
            mbar_arrive(smem_addr(&sm.sc_empty[ss]));
          }
        }
        if (!ok) break;
      }
      if (!ok) give_up();
    }
  } else {
    regs_inc<kChSoftmaxRegs>();
    // -------------------------------------------------------------- softmax
    const int t = warp >> 2;                       // the half
    const int r = threadIdx.x & 127;               // the row in it
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lanes + 256 + t * 128;
    uint32_t parts = 0, n = 0, steps = 0, ends = 0, solos = 0;
    bool ok = true;
    while (true) {
      const uint32_t d = parts % kChParts;
      ok = __all_sync(0xFFFFFFFFu, wait(sm.part_full[d], (parts / kChParts) & 1));
      if (!ok || !sm.part[d].more) break;
      const ChunkPart x = uniform(sm.part[d]);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sm.part_empty[d]));
      ++parts;
      const bool solo = x.rows <= 128;
      const int row = solo ? r : t * 128 + r;      // of the tile
      const bool here = row < x.rows;
      const int p = x.p0 + row, tok = p / P.by_group, hq = x.h * P.group + p - tok * P.group;
      Seq s;
      s.q0 = x.q0;
      s.ql = x.ql;
      s.kv = x.kv;
      int lo = 0, hi = -1;
      if (here) row_range(P, s, tok, lo, hi);

      // Q's row in E4M3 parts, scaled by a power of two to at most 448.
      float rowf = 1.0f;
      if (!solo || t == 0) {
        uint32_t w[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) w[i] = 0u;
        if (here) {
          const uint16_t* src = static_cast<const uint16_t*>(P.q.ptr) + (s.q0 + tok) * P.q.st + hq * P.q.sh;
          if (P.q32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) load8(w + 8 * i, src + 16 * i);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint4 y = __ldg(reinterpret_cast<const uint4*>(src) + i);
              w[4 * i] = y.x;
              w[4 * i + 1] = y.y;
              w[4 * i + 2] = y.z;
              w[4 * i + 3] = y.w;
            }
          }
        }
        const uint32_t e = scale_byte(largest_of<kHalf, 64>(w));
        const float mul = e == 255u ? 0.0f : inverse_scale(e);
        const uint64_t mul2 = pack_f2(mul, mul);
        // NaN for a row that is not finite: so are its results, if it sees a key.
        if (e != 255u || lo <= hi) rowf *= scale_value(e);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t out[Sh::kQParts][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // As FP16 pairs: exact where E4M3's range reaches, and so is what a
            // part leaves over.
            float2 f = unpack2<kHalf>(w[8 * c + 2 * i]), g = unpack2<kHalf>(w[8 * c + 2 * i + 1]);
            f = unpack_f2(mul_f2(pack_f2(f.x, f.y), mul2));
            g = unpack_f2(mul_f2(pack_f2(g.x, g.y), mul2));
            uint32_t a = pack2<true>(f.x, f.y), b = pack2<true>(g.x, g.y);
#pragma unroll
            for (int k = 0; k < Sh::kQParts; ++k) {
              out[k][i] = e4m3x4_of_f16(a, b);
              if (k + 1 < Sh::kQParts) {
                uint32_t va, vb;
                cvt_e4m3x4_to_f16x2x2(out[k][i], va, vb);
                a = hsub2(a, va);
                b = hsub2(b, vb);
              }
            }
          }
#pragma unroll
          for (int k = 0; k < Sh::kQParts; ++k)
            *reinterpret_cast<uint4*>(sm.q[k][t] + r * 128 + ((c ^ (r & 7)) << 4)) = make_uint4(out[k][0], out[k][1], out[k][2], out[k][3]);
        }
        if (solo) sm.ml[r] = make_float2(rowf, 0.0f);
        fence_proxy_async_smem();
      }
      mbar_arrive(smem_addr(&sm.q_full));
      if (solo && t == 1) {
        // The rows' factor comes from the first half's threads.
        ok = __all_sync(0xFFFFFFFFu, wait(sm.q_full, (parts - 1) & 1));
        if (!ok) break;
        rowf = sm.ml[r].x;
      }

      float m = kNegInf, l = 0.0f;
      int E = 0;
      bool begun = false;
      // Keys that the row does not see: -inf in tensor memory, before the scores are
      // read, by a loop that stays out of the common path.
      auto hide = [&](uint32_t tS, int a, int b) {
#pragma unroll 1
        for (int c = 0; c < kChStep; c += 32) {
          uint32_t y[32];
          tmem_ld32(tS + c, y);
          tmem_wait_ld32(y);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (c + k < a || c + k > b) y[k] = 0xFF800000u;
          tmem_st32(tS + c, y);
        }
        tmem_wait_st();
      };
      // The factor that is left of a score: a power of two, finite, so that a score of
      // 0 stays 0; a NaN stays NaN.
      auto row_factor = [&](const ChunkScales& sc) {
        float y;
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(rowf * sc.kmul), "f"(1.7014118e38f));
        return y;
      };
      // The row's largest score of a step, in log2 units.
      auto largest = [&](uint32_t tS, const float* sk, float rk) {
        float top = kNegInf;
#pragma unroll 1
        for (int c = 0; c < kChStep; c += 32) {
          uint32_t y[32];
          tmem_ld32(tS + c, y);
          tmem_wait_ld32(y);
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 k4 = *reinterpret_cast<const float4*>(sk + c + k);
            top = fmax3(top, __uint_as_float(y[k]) * k4.x, __uint_as_float(y[k + 1]) * k4.y);
            top = fmax3(top, __uint_as_float(y[k + 2]) * k4.z, __uint_as_float(y[k + 3]) * k4.w);
          }
        }
        return top * rk;
      };
      auto rescale = [&](float f) {
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          uint32_t o[32];
          tmem_ld32(tO + c, o);
          tmem_wait_ld32(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
          tmem_st32(tO + c, o);
        }
      };
      // Tokens whose K or V is NaN: a NaN weight in the rows that see them, and for K
      // a NaN sum.  (In tensor memory: picked out of registers by a loop, the weights
      // would live in local memory.)
      auto poison = [&](const ChunkScales& sc, int half, uint32_t tP, int a, int b) {
        tmem_wait_st();
#pragma unroll 1
        for (int c = 0; c < kChStep; c += 2) {
          const uint32_t bad0 = sc.nan[half * kChStep + c], bad1 = sc.nan[half * kChStep + c + 1];
          if (bad0 | bad1) {
            uint32_t y = tmem_ld1(tP + c / 2);
            const uint32_t see0 = c >= a && c <= b ? bad0 : 0u, see1 = c + 1 >= a && c + 1 <= b ? bad1 : 0u;
            if (see0) y |= 0x7FFFu;
            if (see1) y |= 0x7FFF0000u;
            if ((see0 | see1) & 1u) l = __uint_as_float(0x7FFFFFFFu);
            tmem_st1(tP + c / 2, y);
          }
        }
      };
      int i = 0;
      for (; i < x.nblk; ++i) {
        const uint32_t blk = n + i, ss = blk % Sh::kScales;
        ok = __all_sync(0xFFFFFFFFu, wait(sm.sc_full[ss], (blk / Sh::kScales) & 1));
        if (!ok) break;
        if (solo && (i & 1) != t) {                // the other half's block
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sm.sc_empty[ss]));
          continue;
        }
        const ChunkScales& sc = sm.sc[ss];
        if (sc.rare & 2) break;                    // wide: the loop below
        const float rk = row_factor(sc);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
        // Two steps a block: scores in columns 64 half .., weights in 32 half ..
        const uint32_t tS = tmem + lanes + t * 128 + half * kChStep, tP = tmem + lanes + t * 128 + half * (kChStep / 2);
        if (half == 0) {
          ok = __all_sync(0xFFFFFFFFu, wait(sm.s_full[t], steps & 1));
          if (!ok) break;
          tc_fence_after();
        }
        const float* sk = sc.k + half * kChStep;
        const int key0 = (x.k0 + i) * kChKeys + half * kChStep, a = lo - key0, b = hi - key0;
        const bool masked = key0 < x.all_lo || key0 + kChStep - 1 > x.all_hi;
        if (masked) hide(tS, a, b);
        // Weights against the reference at hand.  Their sum tells whether it is
        // still good: only when that reaches kChSumLimit (and in the first
        // blocks, without a reference) is the maximum looked for and are the
        // weights computed again.  P stays in registers until then, since it
        // overwrites S.
        const uint64_t f2 = pack_f2(rk, rk);
        const int Eb = sc.e;
        uint32_t w[32];
        float sum;
        if (!begun && half == 0) m = largest(tS, sk, rk);      // a part's first step has no reference to try
#pragma unroll 1
        for (int attempt = 0; attempt < 2; ++attempt) {
          const float shift = kChPBias - (m == kNegInf ? 0.0f : m);
          const uint64_t s2 = pack_f2(shift, shift);
          uint64_t la = 0, lb = 0;
          uint32_t z[kChStep];
          tmem_ld32(tS, z);
          tmem_ld32(tS + 32, z + 32);
          tmem_wait_ld32(z);
          tmem_wait_ld32(z + 32);
#pragma unroll
          for (int c = 0; c < kChStep; c += 4) {
            const float4 k4 = *reinterpret_cast<const float4*>(sk + c);
            const uint64_t u = mul_f2(pack_f2(__uint_as_float(z[c]), __uint_as_float(z[c + 1])), pack_f2(k4.x, k4.y));
            const uint64_t v = mul_f2(pack_f2(__uint_as_float(z[c + 2]), __uint_as_float(z[c + 3])), pack_f2(k4.z, k4.w));
            const float2 e = unpack_f2(fma_f2(u, f2, s2)), f = unpack_f2(fma_f2(v, f2, s2));
            const float p0 = ex2(e.x), p1 = ex2(e.y), p2 = ex2(f.x), p3 = ex2(f.y);
            la = add_f2(la, pack_f2(p0, p1));
            lb = add_f2(lb, pack_f2(p2, p3));
            w[c / 2] = pack2<true>(p0, p1);
            w[c / 2 + 1] = pack2<true>(p2, p3);
          }
          const float2 y = unpack_f2(add_f2(la, lb));
          sum = y.x + y.y;
          const bool again = attempt == 0 && __any_sync(0xFFFFFFFFu, here && (m == kNegInf || sum >= kChSumLimit));
          if (!again && Eb == E) break;
          float f = 1.0f;
          if (again) {
            const float mn = fmaxf(m, largest(tS, sk, rk));
            f = m == kNegInf ? 0.0f : ex2(m - mn);
            m = mn;
            l *= f;
          }
          f *= exp2i(E - Eb);
          E = Eb;
          if (begun || half == 1) {
            // O is at rest in a block's first step (its scores came after all
            // earlier products), in the second once the first one's are complete.
            if (half == 1) ok = __all_sync(0xFFFFFFFFu, wait(sm.o_done[t], steps & 1));
            if (!ok) break;
            tc_fence_after();
            rescale(f);
          }
          if (!again) break;
        }
        if (!ok) break;
        l += sum;
        tmem_st32(tP, w);
        if (sc.rare) poison(sc, half, tP, a, b);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_addr(&sm.p_full[t][half]));
        }
        if (!ok) break;
        ++steps;
        begun = true;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.sc_empty[ss]));
      }
      // Wide blocks (in a loop of their own: as a branch of the one above they slowed
      // it down by 3%).  O's unit is 2^(m + E) with m the row's maximum; E follows
      // that down, and the largest p 2^e of a step up.
      for (; ok && i < x.nblk; ++i) {
        const uint32_t blk = n + i, ss = blk % Sh::kScales;
        ok = __all_sync(0xFFFFFFFFu, wait(sm.sc_full[ss], (blk / Sh::kScales) & 1));
        if (!ok) break;
        if (solo && (i & 1) != t) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sm.sc_empty[ss]));
          continue;
        }
        const ChunkScales& sc = sm.sc[ss];
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const uint32_t tS = tmem + lanes + t * 128 + half * kChStep, tP = tmem + lanes + t * 128 + half * (kChStep / 2);
          // O is at rest as above.
          ok = __all_sync(0xFFFFFFFFu, half ? wait(sm.o_done[t], steps & 1) : wait(sm.s_full[t], steps & 1));
          if (!ok) break;
          tc_fence_after();
          const float* sk = sc.k + half * kChStep;
          const uint8_t* ve = sc.ve + half * kChStep;
          const int key0 = (x.k0 + i) * kChKeys + half * kChStep, a = lo - key0, b = hi - key0;
          if (key0 < x.all_lo || key0 + kChStep - 1 > x.all_hi) hide(tS, a, b);
          const float rk = row_factor(sc), mn = fmaxf(m, largest(tS, sk, rk)), ref = mn == kNegInf ? 0.0f : mn, down = m - ref;
          float most = kNegInf;
#pragma unroll 1
          for (int c = 0; c < kChStep; c += 32) {
            uint32_t y[32];
            tmem_ld32(tS + c, y);
            tmem_wait_ld32(y);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              most = fmaxf(most, fmaf(__uint_as_float(y[k]) * sk[c + k], rk, -ref) + static_cast<float>(ve[c + k]));
          }
          const int En = max(0, max(__float2int_rd(static_cast<float>(E) + down), __float2int_rd(most)));
          if (begun || half == 1) rescale(m == kNegInf ? 0.0f : ex2(down + static_cast<float>(E - En)));
          l *= ex2(down);
          m = mn;
          E = En;
#pragma unroll 1
          for (int c = 0; c < kChStep; c += 32) {      // P lies before the scores that are still to be read
            uint32_t y[32], w[16];
            tmem_ld32(tS + c, y);
            tmem_wait_ld32(y);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float z = fmaf(__uint_as_float(y[k]) * sk[c + k], rk, kChPBias - ref);
              l += ex2(z);
              y[k] = __float_as_uint(ex2(z + static_cast<float>(ve[c + k] - E)));
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = pack2<true>(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1]));
            tmem_st16(tP + c / 2, w);
          }
          if (sc.rare & 1) poison(sc, half, tP, a, b);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(smem_addr(&sm.p_full[t][half]));
        }
        if (!ok) break;
        ++steps;
        begun = true;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.sc_empty[ss]));
      }
      if (!ok) break;
      n += x.nblk;

      // The end of the part: O / l, and the halves' results joined in solo.
      if (begun) {
        ok = __all_sync(0xFFFFFFFFu, wait(sm.o_full[t], ends & 1));
        if (!ok) break;
        ++ends;
        tc_fence_after();
      }
      if (solo && t == 1) {
        sm.ml[r] = make_float2(m, l);
        sm.e1[r] = E;
        mbar_arrive(smem_addr(&sm.x_full));
        // The first half reads this half's O.
        ok = __all_sync(0xFFFFFFFFu, wait(sm.x_empty, solos & 1));
        ++solos;
        if (!ok) break;
        continue;
      }
      float f0 = 1.0f, f1 = 0.0f;
      if (solo) {
        ok = __all_sync(0xFFFFFFFFu, wait(sm.x_full, solos & 1));
        ++solos;
        if (!ok) break;
        tc_fence_after();
        // A half's unit is 2^(m + E).
        const float2 y = sm.ml[r];
        const int e1 = sm.e1[r];
        const float mj = fmaxf(m, y.x), ref = mj == kNegInf ? 0.0f : mj, d0 = m - ref, d1 = y.x - ref;
        const int Ej = max(0, max(E + __float2int_rd(d0), e1 + __float2int_rd(d1)));
        l = l * ex2(d0) + y.y * ex2(d1);
        f0 = ex2(d0 + static_cast<float>(E - Ej));
        f1 = x.nblk > 1 ? ex2(d1 + static_cast<float>(e1 - Ej)) : 0.0f;
        m = mj;
        E = Ej;
      }
      // 2^(E-127) and V's 2^7; the weights' 2^7 is in l.
      const float inv = l == 0.0f ? 0.0f : exp2i(-kChVBias) / l, se = scale_value(E);
      f0 *= inv;
      f1 *= inv;
      uint16_t* orow = static_cast<uint16_t*>(P.o.ptr) + (s.q0 + tok) * P.o.st + hq * P.o.sh;
      const int64_t place = (static_cast<int64_t>(blockIdx.x) * 2 + x.slot) * kChRows + row;
      const bool two = solo && x.nblk > 1;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        uint32_t o[32];
        float y[32];
        tmem_ld32(tO + c, o);
        tmem_wait_ld32(o);
#pragma unroll
        for (int k = 0; k < 32; ++k) y[k] = __uint_as_float(o[k]) * f0;
        if (two) {
          tmem_ld32(tO + 128 + c, o);
          tmem_wait_ld32(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) y[k] += __uint_as_float(o[k]) * f1;
        }
        if (here) {
          if (x.slot < 0) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = pack2<false>(y[2 * k] * se, y[2 * k + 1] * se);
            if (P.o32) {
              store8(orow + c, w);
              store8(orow + c + 16, w + 8);
            } else {
#pragma unroll
              for (int k = 0; k < 16; k += 4) *reinterpret_cast<uint4*>(orow + c + 2 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
#pragma unroll
              for (int j = 0; j < 8; ++j) o[k + j] = __float_as_uint(y[k + j] * se);
              store8(work.o + place * 128 + c + k, o + k);
            }
          }
        }
      }
      tc_fence_before();
      if (here) {
        if (x.slot >= 0) work.ml[place] = make_float2(m, l * exp2i(-static_cast<int>(kChPBias)));
        else if (P.lse) P.lse[static_cast<int64_t>(s.q0 + tok) * P.Hq + hq] = l == 0.0f ? kNegInf : (m + log2f(l) - kChPBias) * 0.69314718055994531f;
      }
      if (solo) mbar_arrive(smem_addr(&sm.x_empty));
    }
    if (!ok) give_up();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace ovc
