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

// A value that is the same in all lanes, by a shuffle: the compiler then keeps it,
// and what is computed from it alone, in uniform registers.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

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

// ---------------------------------------------------------------------------
// Write: 16 lanes per vector, 8 channels (16 bytes in, 8 out) a lane; blockIdx.y
// 0 takes K and 1 takes V.  Bound by memory: 256 + 129 bytes a vector.
// ---------------------------------------------------------------------------
constexpr int kCacheThreads = 256;
constexpr int kCacheVecs = kCacheThreads / 16;

template <bool kHalf>
__global__ void __launch_bounds__(kCacheThreads)
    kv_write_kernel(CacheView c, RowsView k, RowsView v, const int32_t* __restrict__ slots, int64_t nvec,
                    unsigned int* status) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kCacheVecs + (threadIdx.x >> 4);
  const int sub = threadIdx.x & 15;
  if (n >= nvec) return;                          // whole half-warps: the shuffles below stay within one
  const int64_t t = n / c.heads;
  const int h = static_cast<int>(n - t * c.heads);
  const int32_t slot = __ldg(slots + t);
  const int32_t p = slot / c.page;
  if (slot < 0) return;
  if (p >= c.pages) {
    if (sub == 0 && h == 0) atomicOr(status, kPagedBadIndex);
    return;
  }
  const RowsView& x = blockIdx.y ? v : k;
  const uint4 raw = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x.ptr) + t * x.st + h * x.sh) + sub);
  float f[8];
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack2<kHalf>(w[i]);
    f[2 * i] = a.x;
    f[2 * i + 1] = a.y;
    // A NaN counts as an infinity: fmaxf would drop it.
    amax = fmaxf(amax, fmaxf(a.x == a.x ? fabsf(a.x) : INFINITY, a.y == a.y ? fabsf(a.y) : INFINITY));
  }
  const unsigned mask = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, d));
  const uint32_t e = scale_byte(amax);
  uint2 out = make_uint2(0u, 0u);
  if (e != 255u) {
    const float r = inverse_scale(e);
    out.x = cvt_e4m3x2(f[0] * r, f[1] * r) | (cvt_e4m3x2(f[2] * r, f[3] * r) << 16);
    out.y = cvt_e4m3x2(f[4] * r, f[5] * r) | (cvt_e4m3x2(f[6] * r, f[7] * r) << 16);
  }
  const int64_t row = (static_cast<int64_t>(p) * c.heads + h) * c.page + (slot - p * c.page);
  reinterpret_cast<uint2*>((blockIdx.y ? c.v : c.k) + row * 128)[sub] = out;
  if (sub == 0) (blockIdx.y ? c.vs : c.ks)[row] = static_cast<uint8_t>(e);
}

// ---------------------------------------------------------------------------
// Read: the same split, the other way round.
// ---------------------------------------------------------------------------
template <bool kHalf>
__global__ void __launch_bounds__(kCacheThreads)
    kv_read_kernel(CacheView c, RowsView k, RowsView v, const int32_t* __restrict__ slots, int64_t nvec,
                   unsigned int* status) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kCacheVecs + (threadIdx.x >> 4);
  const int sub = threadIdx.x & 15;
  if (n >= nvec) return;
  const int64_t t = n / c.heads;
  const int h = static_cast<int>(n - t * c.heads);
  const int32_t slot = __ldg(slots + t);
  const int32_t p = slot / c.page;
  uint4 out = make_uint4(0u, 0u, 0u, 0u);
  if (slot >= 0 && p < c.pages) {
    const int64_t row = (static_cast<int64_t>(p) * c.heads + h) * c.page + (slot - p * c.page);
    const uint2 raw = reinterpret_cast<const uint2*>((blockIdx.y ? c.v : c.k) + row * 128)[sub];
    const float s = scale_value((blockIdx.y ? c.vs : c.ks)[row]);
    uint32_t h2[4];
    cvt_e4m3x4_to_f16x2x2(raw.x, h2[0], h2[1]);
    cvt_e4m3x4_to_f16x2x2(raw.y, h2[2], h2[3]);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = unpack2<true>(h2[i]);
      o[i] = pack2<kHalf>(a.x * s, a.y * s);
    }
    out = make_uint4(o[0], o[1], o[2], o[3]);
  } else if (slot >= 0 && sub == 0 && h == 0) {
    atomicOr(status, kPagedBadIndex);
  }
  const RowsView& x = blockIdx.y ? v : k;
  reinterpret_cast<uint4*>(static_cast<uint16_t*>(x.ptr) + t * x.st + h * x.sh)[sub] = out;
}

// ---------------------------------------------------------------------------
// Attention: parameters and the sequences of a batch
// ---------------------------------------------------------------------------
// Division of 0 <= n < 2^31 by a number known at the launch: with 2^(s-1) < d <=
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
  unsigned int* status;
};

// Sequence b: query rows [q0, q0 + ql), kv cached tokens.  Whatever the
// arrays hold, the rows lie within q and the tokens within the page table.
struct Seq {
  int q0, ql, kv;
  bool bad;
};

__device__ __forceinline__ Seq load_seq(const PagedParams& P, int b) {
  Seq s;
  int a = b, e = b + 1;
  if (P.cu_q) {
    a = __ldg(P.cu_q + b);
    e = __ldg(P.cu_q + b + 1);
  }
  const int kv = __ldg(P.kv_lens + b);
  s.bad = a < 0 || e < a || e > P.T || kv < 0 || kv > P.most;
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
    if (P.window > 0) lo = max(0, hi - P.window + 1);
  }
}

}  // namespace ovc
