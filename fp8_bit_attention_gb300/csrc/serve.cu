// serve.cu -- libovc's steps between two attention calls over a paged cache (see
// include/ovc.h): the pages of growing sequences, tokens moved inside the cache,
// drafted tokens verified.  A translation unit of its own; nothing here allocates.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "ovc.h"
#include "drafts.cuh"
#include "host.cuh"
#include "move.cuh"
#include "paged_args.cuh"
#include "pages.cuh"

namespace ovc {
namespace {

constexpr int64_t kMost = 0x7FFFFC00;

bool pages_ok(const ovc_kv_pages* p) {
  if (!p || p->rows < 1 || p->rows > kReserveRows || p->pages < 1 || p->pages > kMost || p->width < 1) return false;
  if (p->page < 16 || p->page > 1024 || p->page % 16) return false;
  return p->pages * p->page <= kMost && static_cast<int64_t>(p->width) * p->page <= kMost && at4(p->page_table) &&
         at4(p->kv_lens) && at16(p->refs);
}

PagesView view(const ovc_kv_pages* p, const DeviceState* dev) {
  return {p->page_table, p->kv_lens, p->refs, static_cast<int32_t>(p->rows), p->width, static_cast<int32_t>(p->pages),
          p->page, fast_div(p->page), dev->status};
}

template <typename... Params, typename... Args>
ovc_status launch_clusters(void (*fn)(Params...), dim3 grid, int threads, size_t smem, int ctas, cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fn, args...) != cudaSuccess) {
    cudaGetLastError();
    return OVC_ERR_CUDA;
  }
  return launched();
}

// The least power of two, at most `most`, with which `units` clusters have `want` CTAs.
int clusters_for(int64_t units, int64_t want, int most) {
  int c = 1;
  while (c < most && units * c < want) c *= 2;
  return c;
}

std::mutex g_serve_mu;
bool g_serve_init[64];

ovc_status serve_init(int device) {
  std::lock_guard<std::mutex> lock(g_serve_mu);
  if (g_serve_init[device]) return OVC_OK;
  if (cudaFuncSetAttribute(pages_reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(reserve_smem(kReserveRows))) != cudaSuccess ||
      cudaFuncSetAttribute(pages_reserve_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
      cudaFuncSetAttribute(kv_compact_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, CompactShape<128>::kSmem) != cudaSuccess ||
      cudaFuncSetAttribute(kv_compact_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, CompactShape<64>::kSmem) != cudaSuccess)
    return OVC_ERR_CUDA;
  g_serve_init[device] = true;
  return OVC_OK;
}

}  // namespace
}  // namespace ovc

using namespace ovc;

extern "C" {

ovc_status ovc_kv_pages_reserve(const ovc_kv_pages* p, const int32_t* lens, int32_t* src, int32_t* dst, int32_t* tokens,
                                void* stream) {
  if (!pages_ok(p) || !at4(lens) || !at4(src) || !at4(dst) || !at4(tokens)) return OVC_ERR_INVALID_ARG;
  DeviceState* dev = nullptr;
  ovc_status st = device_state(&dev);
  if (st != OVC_OK) return st;
  st = serve_init(dev->index);
  if (st != OVC_OK) return st;
  int shift = 0;
  while (p->pages > (int64_t{kReserveBlock} << shift) * kReserveChunks) ++shift;
  // 4, 8 and 16 CTAs: 600000 pages 41, 25 and 16 us; 131072 pages 12.3, 11.1 and 10.8
  // us (one CTA 18.2); 1, 2 and 4, 32768 pages: 8.1, 7.7 and 7.4 us; 8192 pages: one
  // CTA 6.4, two 7.3 us.
  const int ctas = clusters_for(1, (p->pages - 1) / (2 * kReserveBlock) + 1, kReserveClusters);
  return launch_clusters(pages_reserve_kernel, dim3(ctas), kReserveThreads, reserve_smem(static_cast<int>(p->rows)), ctas,
                         static_cast<cudaStream_t>(stream), view(p, dev), lens, ReserveOut{src, dst, tokens}, shift, reserve_hash(static_cast<int>(p->rows)));
}

ovc_status ovc_kv_pages_release(const ovc_kv_pages* p, const int32_t* lens, void* stream) {
  if (!pages_ok(p) || !at4(lens)) return OVC_ERR_INVALID_ARG;
  DeviceState* dev = nullptr;
  const ovc_status st = device_state(&dev);
  if (st != OVC_OK) return st;
  // A CTA a row.  Wide ones where all rows run at once and may drop many pages.  128,
  // 256, 512 and 1024 threads: 256 rows dropping up to 2048 pages 13.2, 8.1, 5.5 and
  // 4.8 us; 960 rows dropping 450 each 9.1, 7.4, 8.1 and 11.3 us; 64 rows dropping one
  // or none 3.3, 3.3, 3.2 and 3.5 us.
  const int threads = p->width <= 128 ? 128 : p->width <= 512 || p->rows > 2 * dev->sms ? 256 : 1024;
  pages_release_kernel<<<static_cast<unsigned>(p->rows), threads, 0, static_cast<cudaStream_t>(stream)>>>(view(p, dev), lens);
  return launched();
}

ovc_status ovc_kv_pages_fork(const ovc_kv_pages* p, const int32_t* parents, const int32_t* children, int64_t n, void* stream) {
  if (!pages_ok(p) || !at4(parents) || !at4(children) || n < 1 || n > p->rows) return OVC_ERR_INVALID_ARG;
  DeviceState* dev = nullptr;
  const ovc_status st = device_state(&dev);
  if (st != OVC_OK) return st;
  pages_fork_kernel<<<static_cast<unsigned>(n), kForkThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      view(p, dev), parents, children, static_cast<int32_t>(n));
  return launched();
}

ovc_status ovc_kv_copy(const ovc_kv_cache* to, const ovc_kv_cache* from, const int32_t* src, const int32_t* dst,
                       const int32_t* tokens, int64_t n, void* stream) {
  if (!from) from = to;
  if (!cache_ok(to) || !cache_ok(from) || to->heads != from->heads || to->page != from->page) return OVC_ERR_INVALID_ARG;
  if (!at4(src) || !at4(dst) || (tokens && !at4(tokens)) || n < 1 || n > 0x40000000) return OVC_ERR_INVALID_ARG;
  DeviceState* dev = nullptr;
  const ovc_status st = device_state(&dev);
  if (st != OVC_OK) return st;
  CopyParams P{};
  P.to = view(to);
  P.from = view(from);
  P.src = src;
  P.dst = dst;
  P.tokens = tokens;
  P.n = static_cast<int32_t>(n);
  P.groups = (P.to.page + 31) / 32;
  P.by_groups = fast_div(P.groups);
  P.by_heads = fast_div(P.to.heads);
  P.status = dev->status;
  const int64_t units = int64_t{2} * P.to.heads * P.groups, warps = kCopyThreads / 32;
  const dim3 grid(static_cast<unsigned>((units + warps - 1) / warps), static_cast<unsigned>(std::min<int64_t>(n, 65535)),
                  static_cast<unsigned>((n + 65534) / 65535));
  kv_copy_kernel<<<grid, kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(P);
  return launched();
}

ovc_status ovc_kv_compact(const ovc_kv_cache* c, const ovc_kv_pages* p, const int32_t* keep, int64_t keep_stride,
                          const int32_t* cu_keep, int64_t n, void* stream) {
  if (!cache_ok(c) || !pages_ok(p) || c->page != p->page || c->pages != p->pages || c->heads > 32767)
    return OVC_ERR_INVALID_ARG;
  if (!at4(keep) || !at4(cu_keep) || n < 1 || n > kMost || (keep_stride != 0 && keep_stride < n)) return OVC_ERR_INVALID_ARG;
  DeviceState* dev = nullptr;
  ovc_status st = device_state(&dev);
  if (st != OVC_OK) return st;
  CompactParams C{};
  C.c = view(c);
  C.P = view(p, dev);
  C.keep = keep;
  C.keep_stride = keep_stride;
  C.cu = cu_keep;
  C.n = static_cast<int32_t>(n);
  st = serve_init(dev->index);
  if (st != OVC_OK) return st;
  const int64_t units = p->rows * c->heads * 2;
  // Half the channels a CTA where clusters of the largest size would leave SMs
  // without two CTAs.  Whole and half: 49152 moved of one sequence of 65536, 8 heads,
  // 49 and 42 us; 8 sequences up to 32768, half kept, 38 and 40 us.
  const bool halves = units * kCompactClusters < kCompactCtas * dev->sms;
  const int parts = halves ? 2 : 1;
  // One CTA a unit where they fill the SMs; else more than run at once, as sequences
  // may differ in length.  2, 4 and 6 CTAs: 8 ragged sequences up to 32768 x 8 heads
  // 50, 38 and 44 us, 8 of 16384 50, 54 and 59 us.  1 and 2 CTAs: three quarters of 32
  // sequences of 4096 71 and 82 us, half of 32 ragged ones up to 16384 83 and 89 us, a
  // few tokens of 16 sequences 7.5 and 13 us.
  const int64_t fit = units >= dev->sms ? 1 : 18 * dev->sms / 5 / (units * parts);
  const int ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kCompactClusters, fit)));
  return launch_clusters(halves ? kv_compact_kernel<64> : kv_compact_kernel<128>,
                         dim3(ctas, static_cast<unsigned>(units / p->rows * parts), static_cast<unsigned>(p->rows)), kCompactThreads + 32,
                         halves ? CompactShape<64>::kSmem : CompactShape<128>::kSmem, ctas, static_cast<cudaStream_t>(stream), C);
}

ovc_status ovc_verify_drafts(const ovc_drafts* d, int32_t* tokens, int32_t* accepted, void* stream) {
  if (!d || d->B < 1 || d->B > 0xFFFFFF || d->N < 0 || d->V < 1 || d->V > kMost || d->N + d->B > kMost) return OVC_ERR_INVALID_ARG;
  if (d->dtype != OVC_BF16 && d->dtype != OVC_FP16 && d->dtype != OVC_FP32) return OVC_ERR_UNSUPPORTED;
  const uintptr_t mask = d->dtype == OVC_FP32 ? 3u : 1u;
  if (!d->target || (reinterpret_cast<uintptr_t>(d->target) & mask) || d->target_stride < 0) return OVC_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(d->draft) & mask) || (d->draft && d->draft_stride < 0)) return OVC_ERR_INVALID_ARG;
  if ((d->N && (!at4(d->drafts) || !at4(d->accept_u))) || !at4(d->sample_u) || !at4(tokens) || !at4(accepted)) return OVC_ERR_INVALID_ARG;
  if (d->cu_drafts ? !at4(d->cu_drafts) : d->N % d->B != 0) return OVC_ERR_INVALID_ARG;
  DeviceState* dev = nullptr;
  const ovc_status st = device_state(&dev);
  if (st != OVC_OK) return st;
  DraftParams P{};
  P.cu = d->cu_drafts;
  P.each = static_cast<int32_t>(d->N / d->B);
  P.N = static_cast<int32_t>(d->N);
  P.V = static_cast<int32_t>(d->V);
  P.drafts = d->drafts;
  P.target = d->target;
  P.draft = d->draft;
  P.target_stride = d->target_stride;
  P.draft_stride = d->draft_stride;
  P.accept_u = d->accept_u;
  P.sample_u = d->sample_u;
  P.tokens = tokens;
  P.accepted = accepted;
  P.status = dev->status;
  const int most = clusters_for(1, (d->V + 4095) / 4096, kDraftClusters);
  // As many CTAs as run at once (about 8/9 of the places, as clusters leave some
  // empty).  One, two and four times as many: 64 x 131072 FP32 17.2, 20.8 and 21.2
  // us, 256 x 100003 BF16 without draft 20.0, 25.3 and 31.6 us.
  const int ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, int64_t{kDraftCtas} * dev->sms * 8 / 9 / d->B)));
  const int64_t tile = d->dtype == OVC_FP32 ? kDraftTile<2> : kDraftTile<0>;
  while (d->V + 7 > (tile << P.tile_shift) * kDraftTiles * ctas) ++P.tile_shift;       // rows begin up to 7 tokens behind a tile
  const auto launch = [&](auto* with, auto* without) {
    return launch_clusters(d->draft ? with : without, dim3(static_cast<unsigned>(d->B * ctas)),
                           d->draft ? kDraftThreads<true> : kDraftThreads<false>, 0, ctas, static_cast<cudaStream_t>(stream), P);
  };
  if (d->dtype == OVC_FP32) return launch(verify_drafts_kernel<2, true>, verify_drafts_kernel<2, false>);
  if (d->dtype == OVC_FP16) return launch(verify_drafts_kernel<1, true>, verify_drafts_kernel<1, false>);
  return launch(verify_drafts_kernel<0, true>, verify_drafts_kernel<0, false>);
}

}  // extern "C"
