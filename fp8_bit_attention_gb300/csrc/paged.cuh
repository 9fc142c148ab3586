// paged.cuh -- the paged FP8 KV cache: its format, its write and read kernels,
// and what the attention kernels over it share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx.cuh"

namespace ovc {

constexpr unsigned kPagedBadIndex = 2u;   // device status bit (host.cuh: kStatusBadIndex)
constexpr float kNegInf = -INFINITY;

// ---------------------------------------------------------------------------
// Format
// ---------------------------------------------------------------------------
// E8M0 byte of a vector whose largest magnitude is amax: the least e with
// amax <= 448 * 2^(e-127).  With amax = 1.f * 2^(E-127), 448 = 1.75 * 2^8 and
// so e = E - 8, one more where the fraction exceeds .75.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0u) return 127u;
  if (u >= 0x7F800000u) return 255u;
  const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 0));
}

// 2^(e-127), NaN for 255 (e = 0 is a subnormal of FP32).
__device__ __forceinline__ float scale_value(uint32_t e) {
  const uint32_t u = e == 255u ? 0x7FFFFFFFu : e == 0u ? 0x00400000u : e << 23;
  return __uint_as_float(u);
}

// 2^(127-e) for e <= 254: exponent field 254 - e (e = 254 gives the subnormal 2^-127).
__device__ __forceinline__ float inverse_scale(uint32_t e) {
  return __uint_as_float(e == 254u ? 0x00400000u : (254u - e) << 23);
}

template <bool kHalf>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (kHalf) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (kHalf) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Largest magnitude of N BF16 or FP16 pairs; infinity if one is a NaN.
template <bool kHalf, int N>
__device__ __forceinline__ float largest_of(const uint32_t* w) {
  uint32_t m[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t x = w[i] & 0x7FFF7FFFu;
    if (kHalf) asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m[i & 3]) : "r"(x));
    else asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m[i & 3]) : "r"(x));
  }
  float best = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack2<kHalf>(m[i]);
    best = fmaxf(best, fmaxf(a.x == a.x ? a.x : INFINITY, a.y == a.y ? a.y : INFINITY));
  }
  return best;
}

// A value that is the same in all lanes, by a shuffle: the compiler then keeps it,
// and what is computed from it alone, in uniform registers.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

// mbar_wait (ptx.cuh) in little code: the attention kernels wait in many places,
// their warps run through different code at the same time, and what does not fit
// the instruction caches is what they wait for most.
__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns, const volatile int* abort) {
  if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity))
    if (*abort || globaltimer_ns() - t0 > timeout_ns) return false;
  return true;
}

struct CacheView {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ks;
  uint8_t* vs;
  int32_t pages, heads, page;
};

struct RowsView {
  void* ptr;
  int64_t st, sh;   // element strides
};

// Division of 0 <= n < 2^31 by a number known at the launch (Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994): with 2^(s-1) < d <=
// 2^s and m = floor(2^32 (2^s - d) / d) + 1, n / d = (m n / 2^32 + n) >> s.  (A
// division by a register is about 20 dependent instructions, and a CTA does a
// dozen of them before its first load.)
struct FastDiv {
  uint32_t m, s;
  int32_t d;
};

__host__ inline FastDiv fast_div(int32_t d) {
  FastDiv f{0, 0, d};
  while ((int64_t{1} << f.s) < d) ++f.s;
  f.m = static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{1} << f.s) - d)) / d + 1);
  return f;
}

__device__ __forceinline__ int operator/(int n, const FastDiv& f) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(n), f.m) + static_cast<uint32_t>(n)) >> f.s);
}

// ---------------------------------------------------------------------------
// Write and read: 16 lanes a vector, 8 channels (16 bytes of BF16/FP16, 8 of
// codes) a lane; a CTA takes 16 or 64 tokens of one head (blockIdx.y) of K or V
// (blockIdx.z), one or four tokens a lane, whose loads are all under way before the
// first is used.  Bound by memory: 256 + 129 bytes a vector (5.5 TB/s writing
// 73397 tokens x 8 heads, 6.1 TB/s reading 65536).
// ---------------------------------------------------------------------------
constexpr int kCacheThreads = 256;
// Tokens a lane: four where the calls are long enough to fill the GPU, else one,
// which spreads a short call over more SMs.  One against four, writing x 8 heads:
// 64 tokens 4.1 and 4.8 us, 8192 tokens 17.5 and 14.9 us, 73397 tokens 105 and
// 81 us; reading 65536 tokens 86 and 65 us.
constexpr int kCacheGroups = kCacheThreads / 16;

template <bool kHalf, int kEach>
__global__ void __launch_bounds__(kCacheThreads)
    kv_write_kernel(CacheView c, FastDiv by_page, RowsView k, RowsView v, const int32_t* __restrict__ slots, int32_t T,
                    unsigned int* status) {
  const int sub = threadIdx.x & 15, h = blockIdx.y;
  const int t0 = blockIdx.x * (kCacheGroups * kEach) + (threadIdx.x >> 4);
  const RowsView& x = blockIdx.z ? v : k;
  const uint16_t* src = static_cast<const uint16_t*>(x.ptr) + h * x.sh + 8 * sub;
  uint8_t* codes = blockIdx.z ? c.v : c.k;
  uint8_t* scales = blockIdx.z ? c.vs : c.ks;
  uint4 raw[kEach];
  int32_t slot[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int t = t0 + i * kCacheGroups;
    slot[i] = -1;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (t < T) {
      slot[i] = __ldg(slots + t);
      raw[i] = __ldg(reinterpret_cast<const uint4*>(src + t * x.st));
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    float f[8], amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = unpack2<kHalf>(w[j]);
      f[2 * j] = a.x;
      f[2 * j + 1] = a.y;
      // A NaN counts as an infinity: fmaxf would drop it.
      amax = fmaxf(amax, fmaxf(a.x == a.x ? fabsf(a.x) : INFINITY, a.y == a.y ? fabsf(a.y) : INFINITY));
    }
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
    if (slot[i] < 0) continue;
    const int32_t p = slot[i] / by_page;
    if (p >= c.pages) {
      if (sub == 0 && h == 0) atomicOr(status, kPagedBadIndex);
      continue;
    }
    const uint32_t e = scale_byte(amax);
    uint2 out = make_uint2(0u, 0u);
    if (e != 255u) {
      const float r = inverse_scale(e);
      out.x = cvt_e4m3x2(f[0] * r, f[1] * r) | (cvt_e4m3x2(f[2] * r, f[3] * r) << 16);
      out.y = cvt_e4m3x2(f[4] * r, f[5] * r) | (cvt_e4m3x2(f[6] * r, f[7] * r) << 16);
    }
    const int64_t row = (static_cast<int64_t>(p) * c.heads + h) * c.page + (slot[i] - p * c.page);
    reinterpret_cast<uint2*>(codes + row * 128)[sub] = out;
    if (sub == 0) scales[row] = static_cast<uint8_t>(e);
  }
}

template <bool kHalf, int kEach>
__global__ void __launch_bounds__(kCacheThreads)
    kv_read_kernel(CacheView c, FastDiv by_page, RowsView k, RowsView v, const int32_t* __restrict__ slots, int32_t T,
                   unsigned int* status) {
  const int sub = threadIdx.x & 15, h = blockIdx.y;
  const int t0 = blockIdx.x * (kCacheGroups * kEach) + (threadIdx.x >> 4);
  const RowsView& x = blockIdx.z ? v : k;
  uint16_t* dst = static_cast<uint16_t*>(x.ptr) + h * x.sh + 8 * sub;
  const uint8_t* codes = blockIdx.z ? c.v : c.k;
  const uint8_t* scales = blockIdx.z ? c.vs : c.ks;
  uint2 raw[kEach];
  uint32_t e[kEach];
  int32_t slot[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int t = t0 + i * kCacheGroups;
    slot[i] = t < T ? __ldg(slots + t) : -1;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    raw[i] = make_uint2(0u, 0u);                     // a slot that holds nothing reads as zeros
    e[i] = 127u;
    if (slot[i] >= 0) {
      const int32_t p = slot[i] / by_page;
      if (p < c.pages) {
        const int64_t row = (static_cast<int64_t>(p) * c.heads + h) * c.page + (slot[i] - p * c.page);
        raw[i] = reinterpret_cast<const uint2*>(codes + row * 128)[sub];
        e[i] = scales[row];
      } else if (sub == 0 && h == 0) {
        atomicOr(status, kPagedBadIndex);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int t = t0 + i * kCacheGroups;
    if (t >= T) break;
    const float s = scale_value(e[i]);
    uint32_t h2[4], o[4];
    cvt_e4m3x4_to_f16x2x2(raw[i].x, h2[0], h2[1]);
    cvt_e4m3x4_to_f16x2x2(raw[i].y, h2[2], h2[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = unpack2<true>(h2[j]);
      o[j] = pack2<kHalf>(a.x * s, a.y * s);
    }
    *reinterpret_cast<uint4*>(dst + t * x.st) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ---------------------------------------------------------------------------
// Attention: parameters and the sequences of a batch
// ---------------------------------------------------------------------------
struct PagedParams {
  CacheView c;
  RowsView q, o;
  float* lse;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* kv_lens;
  const int32_t* cu_q;
  int32_t B, T, Hq, group;
  FastDiv by_group, by_page;
  int32_t causal, window;
  int32_t most;             // tokens that a page table row holds
  int32_t unit;             // log2 of the key blocks between the places where work may be cut
  float c2;                 // softmax_scale * log2(e)
  int32_t k_most;           // the largest scale of K that a product takes within FP32's range (many rows)
  int32_t q32, o32;         // rows of q, of o lie at multiples of 32 bytes
  unsigned int* status;
};

// Sequence b: query rows [q0, q0 + ql), kv cached tokens.  Whatever the
// arrays hold, the rows lie within q and the tokens within the page table.
struct Seq {
  int q0, ql, kv;
  int bad;                  // 1: something was cut off; 2: cu_q descends here
};

__device__ __forceinline__ Seq load_seq(const PagedParams& P, int b) {
  Seq s;
  int a = b, e = b + 1;
  if (P.cu_q) {
    a = __ldg(P.cu_q + b);
    e = __ldg(P.cu_q + b + 1);
  }
  const int kv = __ldg(P.kv_lens + b);
  s.bad = e < a ? 2 : a < 0 || e > P.T || kv < 0 || kv > P.most;
  s.q0 = min(max(a, 0), P.T);
  s.ql = min(max(e, s.q0), P.T) - s.q0;
  s.kv = min(max(kv, 0), P.most);
  return s;
}

// Keys [lo, hi] that query row i of a sequence sees (hi < lo: none).
__device__ __forceinline__ void row_range(const PagedParams& P, const Seq& s, int i, int& lo, int& hi) {
  lo = 0;
  hi = s.kv - 1;
  if (P.causal) {
    hi = s.kv - s.ql + i;
    if (P.window > 0 && hi >= P.window) lo = hi - P.window + 1;
  }
}

}  // namespace ovc
