// paged_simple.cuh -- attention over the paged cache in its simplest form: one
// warp per query row and head, four channels a lane, keys one by one with a
// running maximum and sum in FP32.
#pragma once

#include "paged.cuh"

namespace ovc {

template <bool kHalf>
__global__ void __launch_bounds__(256) paged_simple_kernel(const __grid_constant__ PagedParams P) {
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / P.Hq), hq = static_cast<int>(w - static_cast<int64_t>(t) * P.Hq);
  if (t >= P.T) return;
  const int h = hq / P.group;
  int b = -1;
  Seq s{};
  for (int i = 0; i < P.B; ++i) {
    const Seq x = load_seq(P, i);
    if (x.bad && lane == 0) atomicOr(P.status, kPagedBadIndex);
    if (t >= x.q0 && t < x.q0 + x.ql) b = i, s = x;
  }
  if (b < 0) return;
  const uint2 qr = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(P.q.ptr) + t * P.q.st + hq * P.q.sh) + lane);
  const float2 qa = unpack2<kHalf>(qr.x), qb = unpack2<kHalf>(qr.y);
  int lo, hi;
  row_range(P, s, t - s.q0, lo, hi);
  float m = kNegInf, l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = lo; j <= hi; ++j) {
    const int p = __ldg(P.table + b * P.table_stride + j / P.c.page);
    if (p < 0 || p >= P.c.pages) {
      if (lane == 0) atomicOr(P.status, kPagedBadIndex);
      continue;
    }
    const int64_t row = (static_cast<int64_t>(p) * P.c.heads + h) * P.c.page + j % P.c.page;
    uint32_t h0, h1;
    cvt_e4m3x4_to_f16x2x2(reinterpret_cast<const uint32_t*>(P.c.k + row * 128)[lane], h0, h1);
    const float2 ka = unpack2<true>(h0), kb = unpack2<true>(h1);
    float d = qa.x * ka.x + qa.y * ka.y + qb.x * kb.x + qb.y * kb.y;
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, x);
    const float z = d * scale_value(P.c.ks[row]) * P.c2;
    const float mn = fmaxf(m, z);
    const float f = mn == kNegInf ? 1.0f : exp2f(m - mn);
    const float pr = exp2f(z - (mn == kNegInf ? 0.0f : mn));
    m = mn;
    l = l * f + pr;
    cvt_e4m3x4_to_f16x2x2(reinterpret_cast<const uint32_t*>(P.c.v + row * 128)[lane], h0, h1);
    const float2 va = unpack2<true>(h0), vb = unpack2<true>(h1);
    const float g = pr * scale_value(P.c.vs[row]);
    acc[0] = acc[0] * f + g * va.x;
    acc[1] = acc[1] * f + g * va.y;
    acc[2] = acc[2] * f + g * vb.x;
    acc[3] = acc[3] * f + g * vb.y;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.o.ptr) + t * P.o.st + hq * P.o.sh)[lane] =
      make_uint2(pack2<false>(acc[0] * inv, acc[1] * inv), pack2<false>(acc[2] * inv, acc[3] * inv));
  if (P.lse && lane == 0)
    P.lse[static_cast<int64_t>(t) * P.Hq + hq] = l == 0.0f ? kNegInf : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace ovc
