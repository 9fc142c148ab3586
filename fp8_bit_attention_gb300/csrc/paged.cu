// paged.cu -- libovc's paged FP8 KV cache (see include/ovc.h): the entry
// points that check arguments and launch on the caller's stream.  A
// translation unit of its own, compiled beside ovc.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "ovc.h"
#include "host.cuh"
#include "paged.cuh"
#include "paged_chunk.cuh"
#include "paged_decode.cuh"

namespace ovc {
namespace {

static_assert(kPagedBadIndex == kStatusBadIndex, "status bits");

bool at16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool at4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool cache_ok(const ovc_kv_cache* c) {
  if (!c || c->pages < 1 || c->heads < 1 || c->page < 16 || c->page > 1024 || c->page % 16) return false;
  if (!at16(c->k) || !at16(c->v) || !at16(c->k_scale) || !at16(c->v_scale)) return false;
  constexpr int64_t kMost = (int64_t{1} << 31) - 1024;
  return c->heads <= 65535 && c->pages <= kMost && c->pages * c->page <= kMost &&
         c->pages * c->page * c->heads <= kMost;
}

ovc_status rows_ok(const ovc_rows* r) {
  if (!r || r->T < 1 || r->H < 1 || r->T > 0x7FFFFC00 || r->H > 65535 * 256) return OVC_ERR_INVALID_ARG;
  if (!at16(r->ptr) || r->stride_t % 8 || r->stride_h % 8 || r->stride_t < 0 || r->stride_h < 0) return OVC_ERR_INVALID_ARG;
  return r->dtype == OVC_BF16 || r->dtype == OVC_FP16 ? OVC_OK : OVC_ERR_UNSUPPORTED;
}

// An output's rows: as above, and no two of them overlap.
ovc_status out_ok(const ovc_rows* r) {
  const ovc_status st = rows_ok(r);
  if (st != OVC_OK) return st;
  const bool t_inner = r->T == 1 || (r->H > 1 && r->stride_t < r->stride_h);
  const int64_t inner = t_inner ? r->stride_t : r->stride_h, outer = t_inner ? r->stride_h : r->stride_t;
  const int64_t n = t_inner ? r->T : r->H, m = t_inner ? r->H : r->T;
  if (n > 1 && inner < 128) return OVC_ERR_INVALID_ARG;
  return m > 1 && (outer < 128 || (n > 1 && (outer - 128) / (n - 1) < inner)) ? OVC_ERR_INVALID_ARG : OVC_OK;
}

bool at32(const ovc_rows* r) {
  return (reinterpret_cast<uintptr_t>(r->ptr) & 31u) == 0 && r->stride_t % 16 == 0 && r->stride_h % 16 == 0;
}

CacheView view(const ovc_kv_cache* c) {
  return {c->k, c->v, c->k_scale, c->v_scale, static_cast<int32_t>(c->pages), static_cast<int32_t>(c->heads),
          static_cast<int32_t>(c->page)};
}

RowsView view(const ovc_rows* r) { return {r->ptr, r->stride_t, r->stride_h}; }

ovc_status launched() { return cudaGetLastError() == cudaSuccess ? OVC_OK : OVC_ERR_CUDA; }

// Arguments that ovc_kv_write and ovc_kv_read (with its check of the rows) share.
ovc_status cache_call_ok(const ovc_kv_cache* c, const ovc_rows* k, const ovc_rows* v, const int32_t* slots,
                         ovc_status (*ok)(const ovc_rows*)) {
  if (!cache_ok(c) || !at4(slots)) return OVC_ERR_INVALID_ARG;
  ovc_status st = ok(k);
  if (st != OVC_OK) return st;
  st = ok(v);
  if (st != OVC_OK) return st;
  if (k->T != v->T || k->H != c->heads || v->H != c->heads || k->dtype != v->dtype) return OVC_ERR_INVALID_ARG;
  return OVC_OK;
}

// Whether four tokens a lane would leave less than two CTAs an SM.
bool few_tokens(const ovc_rows* r, const DeviceState* dev) {
  return (r->T + 4 * kCacheGroups - 1) / (4 * kCacheGroups) * r->H * 2 < 2 * dev->sms;
}

dim3 cache_grid(const ovc_rows* r, bool few) {
  const int64_t tokens = kCacheGroups * (few ? 1 : 4);
  return dim3(static_cast<unsigned>((r->T + tokens - 1) / tokens), static_cast<unsigned>(r->H), 2);
}

bool batch_ok(const ovc_paged_batch* b) {
  if (!b || b->B < 1 || b->B > 0x7FFFFFF || b->table_width < 1 || b->table_stride < b->table_width) return false;
  if (!at4(b->page_table) || !at4(b->kv_lens) || (b->cu_q && !at4(b->cu_q))) return false;
  return b->max_q >= 0 && (b->causal == 0 || b->causal == 1) && b->window >= 0 && (b->causal || b->window == 0);
}

ovc_status paged_ok(const ovc_rows* q, const ovc_kv_cache* c, const ovc_paged_batch* b) {
  if (!cache_ok(c) || !batch_ok(b)) return OVC_ERR_INVALID_ARG;
  const ovc_status st = rows_ok(q);
  if (st != OVC_OK) return st;
  if (q->H % c->heads || (!b->cu_q && q->T != b->B)) return OVC_ERR_INVALID_ARG;
  return q->T * q->H <= 0x7FFFFC00 ? OVC_OK : OVC_ERR_INVALID_ARG;
}

// Cache codes as rows of 128 bytes, boxes of `box` rows, 128-byte swizzle.
bool make_cache_map(CUtensorMap* m, const void* base, int64_t rows, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {128};
  cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int common_divisor(int a, int b) { return b ? common_divisor(b, a % b) : a; }

constexpr uint64_t kTimeoutNs = 4000000000ull;    // 4 s per wait
constexpr int kMaxSms = 160;                      // that a persistent grid uses
// The least share worth a CTA.  16, 8 and 4 blocks of 16 keys: 1 sequence of 1024
// keys, 8 KV heads and 16 rows 16.5, 14.5, 15.1 us; other calls alike.  2 to 8
// blocks of 128: alike.
constexpr int kDecodeMinShare = 8;                // blocks of 16 keys
constexpr int kChunkMinShare = 4;                 // blocks of 128 keys

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Query rows of a tile: the smallest of the kernels' that holds a sequence's
// rows of one KV head.  Tiles of 8, 16 and 256 (a call of at most 128 rows works
// on 128), 8 KV heads, times in us with queries in BF16 and FP16:
//                              rows       8            16           256
//   1 sequence of 1024 keys      8    12.6  12.4   13.4  12.4   16.6  16.5
//                               16    12.6  12.6   14.5  13.9   16.6  18.5
//                               32    14.6  14.5   16.6  14.5   18.6  18.6
//   256 sequences of 256         8      43    41     64    53    107   113
//                               16      66    64     71    60    111   115
//                               32     121   117    127   103    111   115
//   16 sequences of 8192         8      55    54     76    62     77   110
//                               16      92    92     80    68     76   111
//                               32     163   162    142   117     78   111
//   8 sequences of 65536         8     170   169    241   197    236   359
//                               16     322   321    249   202    237   359
//                               32     623   622    471   379    237   360
// For 9 to 16 rows the middle one is the best with FP16, and never far off with
// BF16, where the best depends on lengths that the host does not know.
int tile_rows(const ovc_rows* q, const ovc_kv_cache* c, const ovc_paged_batch* b) {
  const int64_t group = q->H / c->heads;
  const int64_t most = (b->cu_q ? (b->max_q > 0 ? b->max_q : q->T) : 1) * group;
  return most <= 8 ? 8 : most <= 16 ? 16 : kChRows;
}

// CTAs per SM of the kernel with tiles of R rows.
int ctas_per_sm(int R) { return R == 8 ? kDecodeCtas<1> : R == 16 ? kDecodeCtas<2> : 1; }

size_t work_bytes(int R, PagedWork* w, void* base) {
  uint8_t* p = static_cast<uint8_t*>(base);
  const size_t ctas = static_cast<size_t>(kMaxSms) * ctas_per_sm(R);
  const size_t o = up256(ctas * 2 * R * 512), l = up256(ctas * 2 * R * 8);
  if (w) {
    w->o = reinterpret_cast<float*>(p);
    w->ml = reinterpret_cast<float2*>(p + o);
    w->cut = reinterpret_cast<CutTile*>(p + o + l);
  }
  return o + l + up256(ctas * sizeof(CutTile));
}

// The unit of paged_plan.cuh's line: the least with which all tiles' places are
// sure to fit 31 bits, whatever the lengths.
int line_unit(const ovc_rows* q, const ovc_kv_cache* c, const ovc_paged_batch* b, int R, int BK) {
  const double tiles = (static_cast<double>(q->T) * (q->H / c->heads) / R + b->B) * c->heads;
  const double blocks = static_cast<double>(b->table_width) * c->page / BK + kTileCost<kDecKeys> + 1;
  int unit = 0;
  while (tiles * (std::ldexp(blocks, -unit) + 1) > 2.0e9 && unit < 27) ++unit;
  return unit;
}

using PagedFn = decltype(&paged_decode_kernel<false, 1>);

struct PagedKernel {
  PagedFn fn;
  int threads, smem;
};

PagedKernel kernel_for(bool half, int R) {
  if (R == 8) return {half ? paged_decode_kernel<true, 1> : paged_decode_kernel<false, 1>, kDecThreads, sizeof(DecodeSmem)};
  if (R == 16) return {half ? paged_decode_kernel<true, 2> : paged_decode_kernel<false, 2>, kDecThreads, sizeof(DecodeSmem)};
  if (half) return {paged_chunk_kernel<true>, kChThreads, sizeof(ChunkSmem<true>)};
  return {paged_chunk_kernel<false>, kChThreads, sizeof(ChunkSmem<false>)};
}

std::mutex g_paged_mu;
bool g_paged_init[64];

// Shared memory limits of the attention kernels, once per device.
ovc_status paged_init(int device) {
  std::lock_guard<std::mutex> lock(g_paged_mu);
  if (g_paged_init[device]) return OVC_OK;
  for (const int R : {8, 16, kChRows})
    for (int half = 0; half < 2; ++half) {
      const PagedKernel k = kernel_for(half, R);
      if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) != cudaSuccess) return OVC_ERR_CUDA;
    }
  g_paged_init[device] = true;
  return OVC_OK;
}

// The join, launched while the attention kernel before it still runs.
template <int R, int kWarps>
cudaError_t launch_join(const PagedParams& P, const PagedWork& w, int ctas, int groups, cudaStream_t s) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, groups);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<R, kWarps>, P, w);
}

}  // namespace
}  // namespace ovc

using namespace ovc;

extern "C" {

ovc_status ovc_kv_write(const ovc_kv_cache* c, const ovc_rows* k, const ovc_rows* v, const int32_t* slots,
                        void* stream) {
  ovc_status st = cache_call_ok(c, k, v, slots, rows_ok);
  if (st != OVC_OK) return st;
  DeviceState* dev = nullptr;
  st = device_state(&dev);
  if (st != OVC_OK) return st;
  const bool few = few_tokens(k, dev);
  auto* fn = k->dtype == OVC_FP16 ? (few ? kv_write_kernel<true, 1> : kv_write_kernel<true, 4>)
                                  : (few ? kv_write_kernel<false, 1> : kv_write_kernel<false, 4>);
  fn<<<cache_grid(k, few), kCacheThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      view(c), fast_div(static_cast<int32_t>(c->page)), view(k), view(v), slots, static_cast<int32_t>(k->T), dev->status);
  return launched();
}

ovc_status ovc_kv_read(const ovc_kv_cache* c, const int32_t* slots, const ovc_rows* k, const ovc_rows* v,
                       void* stream) {
  ovc_status st = cache_call_ok(c, k, v, slots, out_ok);
  if (st != OVC_OK) return st;
  DeviceState* dev = nullptr;
  st = device_state(&dev);
  if (st != OVC_OK) return st;
  const bool few = few_tokens(k, dev);
  auto* fn = k->dtype == OVC_FP16 ? (few ? kv_read_kernel<true, 1> : kv_read_kernel<true, 4>)
                                  : (few ? kv_read_kernel<false, 1> : kv_read_kernel<false, 4>);
  fn<<<cache_grid(k, few), kCacheThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      view(c), fast_div(static_cast<int32_t>(c->page)), view(k), view(v), slots, static_cast<int32_t>(k->T), dev->status);
  return launched();
}

size_t ovc_paged_attention_workspace_bytes(const ovc_rows* q, const ovc_kv_cache* c, const ovc_paged_batch* b) {
  return paged_ok(q, c, b) == OVC_OK ? work_bytes(tile_rows(q, c, b), nullptr, nullptr) : 0;
}

ovc_status ovc_paged_attention(const ovc_rows* q, const ovc_kv_cache* c, const ovc_paged_batch* b,
                               float softmax_scale, const ovc_rows* o, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream) {
  ovc_status st = paged_ok(q, c, b);
  if (st != OVC_OK) return st;
  st = out_ok(o);
  if (st != OVC_OK) return st;
  if (o->T != q->T || o->H != q->H || o->dtype != OVC_BF16 || (lse && !at4(lse))) return OVC_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return OVC_ERR_INVALID_ARG;
  const double sm = softmax_scale <= 0.0f ? 1.0 / std::sqrt(128.0) : static_cast<double>(softmax_scale);
  const float c2 = static_cast<float>(1.4426950408889634074 * sm);
  if (!std::isfinite(c2)) return OVC_ERR_INVALID_ARG;
  if (workspace_bytes < ovc_paged_attention_workspace_bytes(q, c, b)) return OVC_ERR_WORKSPACE_TOO_SMALL;
  DeviceState* dev = nullptr;
  st = device_state(&dev);
  if (st != OVC_OK) return st;
  PagedParams P{};
  P.c = view(c);
  P.q = view(q);
  P.o = view(o);
  P.q32 = at32(q);
  P.o32 = at32(o);
  P.lse = lse;
  P.table = b->page_table;
  P.table_stride = b->table_stride;
  P.most = static_cast<int32_t>(std::min<int64_t>(b->table_width * c->page, 0x7FFFFF00));
  P.kv_lens = b->kv_lens;
  P.cu_q = b->cu_q;
  P.B = static_cast<int32_t>(b->B);
  P.T = static_cast<int32_t>(q->T);
  P.Hq = static_cast<int32_t>(q->H);
  P.group = static_cast<int32_t>(q->H / c->heads);
  P.by_group = fast_div(P.group);
  P.by_page = fast_div(P.c.page);
  P.causal = b->causal;
  P.window = b->window < P.most ? b->window : 0;
  P.c2 = c2;
  // A product of codes is below 448 * 448 * 128 * (1 + 2^-4) < 2^25, and c2 below 2^x.
  int x = 0;
  std::frexp(P.c2, &x);
  P.k_most = 127 + 103 - std::max(x, 0);
  P.status = dev->status;
  PagedMaps M{};
  M.rows = static_cast<int32_t>(c->pages * c->heads * c->page);
  const int R = tile_rows(q, c, b), BK = R == kChRows ? kChKeys : kDecKeys;
  M.box = common_divisor(static_cast<int>(c->page), BK);
  M.min_share = R == kChRows ? kChunkMinShare : kDecodeMinShare;
  M.timeout_ns = kTimeoutNs;
  if (!make_cache_map(&M.k, c->k, M.rows, M.box) || !make_cache_map(&M.v, c->v, M.rows, M.box)) return OVC_ERR_CUDA;
  st = paged_init(dev->index);
  if (st != OVC_OK) return st;
  P.unit = line_unit(q, c, b, R, BK);
  PagedWork w;
  work_bytes(R, &w, workspace);
  const int ctas = (dev->sms < kMaxSms ? dev->sms : kMaxSms) * ctas_per_sm(R);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const PagedKernel k = kernel_for(q->dtype == OVC_FP16, R);
  k.fn<<<ctas, k.threads, k.smem, s>>>(P, M, w);
  st = launched();
  if (st != OVC_OK) return st;
  const cudaError_t err = R == 8    ? launch_join<8, 4>(P, w, ctas, 4, s)
                          : R == 16 ? launch_join<16, 4>(P, w, ctas, 8, s)
                                    : launch_join<kChRows, 1>(P, w, ctas, 8, s);
  if (err != cudaSuccess) return OVC_ERR_CUDA;
  return launched();
}

}  // extern "C"
