// paged_args.cuh -- checks of arguments that the translation units of the paged
// cache share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ovc.h"
#include "paged.cuh"

namespace ovc {

inline bool at16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool at4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline bool cache_ok(const ovc_kv_cache* c) {
  if (!c || c->pages < 1 || c->heads < 1 || c->page < 16 || c->page > 1024 || c->page % 16) return false;
  if (!at16(c->k) || !at16(c->v) || !at16(c->k_scale) || !at16(c->v_scale)) return false;
  constexpr int64_t kMost = (int64_t{1} << 31) - 1024;
  return c->heads <= 65535 && c->pages <= kMost && c->pages * c->page <= kMost &&
         c->pages * c->page * c->heads <= kMost;
}

inline CacheView view(const ovc_kv_cache* c) {
  return {c->k, c->v, c->k_scale, c->v_scale, static_cast<int32_t>(c->pages), static_cast<int32_t>(c->heads),
          static_cast<int32_t>(c->page)};
}

inline ovc_status launched() { return cudaGetLastError() == cudaSuccess ? OVC_OK : OVC_ERR_CUDA; }

}  // namespace ovc
