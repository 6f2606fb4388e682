// Host-side pieces that the translation units of the library share.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/spec_verify.h"

namespace sv {

// Limit (ns) of every bounded device wait in the calls that follow.
unsigned long long wait_limit_ns();

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// The code of a runtime call.  A failure is also kept by the runtime as this thread's
// last error: it is cleared, so that no later call takes it for its own launch's.
inline int code_of(cudaError_t e) {
  if (e == cudaSuccess) return SV_OK;
  (void)cudaGetLastError();
  return SV_ERR_CUDA;
}

// Launches that may begin while the kernel before them in the stream ends; the
// kernel waits for that one (griddepcontrol.wait) before it touches memory.
inline void overlap_launch(cudaLaunchAttribute& a) {
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
}

// The checks of a paged cache that the host can make: of 16 bits, or of e4m3 codes.
inline int check_pools(const sv_kv_cache& c, int step) {  // (step: what sizes and strides are multiples of)
  if (c.batch < 0 || c.num_pages < 1 || c.max_pages < 0 || c.kv_heads < 1 || c.kv_heads > 65535)
    return SV_ERR_SCALAR;
  if (c.head_dim < step || c.head_dim > SV_MAX_HEAD_DIM || c.head_dim % step) return SV_ERR_SCALAR;
  if (c.page_size < 16 || c.page_size > 4096 || (c.page_size & (c.page_size - 1)))
    return SV_ERR_SCALAR;
  for (int i = 0; i < 3; ++i)
    for (int64_t s : {c.k_strides[i], c.v_strides[i]})
      if (s <= 0 || s % step || s >= ((int64_t)1 << 38)) return SV_ERR_SCALAR;
  if (c.batch == 0) return SV_OK;
  if (!c.k_pages || !c.v_pages || !c.kv_len || (c.max_pages > 0 && !c.page_table))
    return SV_ERR_NULL;
  if (!aligned(c.k_pages, 16) || !aligned(c.v_pages, 16) || !aligned(c.kv_len, 4) ||
      !aligned(c.page_table, 4))
    return SV_ERR_ALIGN;
  return SV_OK;
}
inline int check_cache(const sv_kv_cache& c) {
  if (c.dtype != SV_BF16 && c.dtype != SV_F16) return SV_ERR_SCALAR;
  return check_pools(c, 8);
}
inline int check_cache_e4m3(const sv_kv_cache& c, const sv_kv_scales& s) {
  if (c.dtype != SV_E4M3 || s.block < 1 || s.block > SV_MAX_BLOCK || (s.block & (s.block - 1)) ||
      s.block > c.page_size)
    return SV_ERR_SCALAR;
  const int rc = check_pools(c, 16);
  if (rc || c.batch == 0) return rc;
  if (!s.k || !s.v) return SV_ERR_NULL;
  return aligned(s.k, 4) && aligned(s.v, 4) ? SV_OK : SV_ERR_ALIGN;
}

}  // namespace sv
