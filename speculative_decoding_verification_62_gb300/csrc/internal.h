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

// The checks of a paged cache that the host can make.
inline int check_cache(const sv_kv_cache& c) {
  if (c.dtype != SV_BF16 && c.dtype != SV_F16) return SV_ERR_SCALAR;
  if (c.batch < 0 || c.num_pages < 1 || c.max_pages < 0 || c.kv_heads < 1 || c.kv_heads > 65535)
    return SV_ERR_SCALAR;
  if (c.head_dim < 8 || c.head_dim > SV_MAX_HEAD_DIM || c.head_dim % 8) return SV_ERR_SCALAR;
  if (c.page_size < 16 || c.page_size > 4096 || (c.page_size & (c.page_size - 1)))
    return SV_ERR_SCALAR;
  for (int i = 0; i < 3; ++i)
    for (int64_t s : {c.k_strides[i], c.v_strides[i]})
      if (s <= 0 || s % 8 || s >= ((int64_t)1 << 38)) return SV_ERR_SCALAR;
  if (c.batch == 0) return SV_OK;
  if (!c.k_pages || !c.v_pages || !c.kv_len || (c.max_pages > 0 && !c.page_table))
    return SV_ERR_NULL;
  if (!aligned(c.k_pages, 16) || !aligned(c.v_pages, 16) || !aligned(c.kv_len, 4) ||
      !aligned(c.page_table, 4))
    return SV_ERR_ALIGN;
  return SV_OK;
}

}  // namespace sv
