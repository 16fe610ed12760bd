// Argument checks of the C entry points that live beside their kernels.
#pragma once

#include "../../include/bytecross.h"
#include "kernels.h"

#include <stdarg.h>
#include <stdio.h>

namespace bc {

inline bc_status entry_fail(bc_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline bc_status entry_fail(bc_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_error(buf);
  return s;
}

inline bc_status entry_cuda(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return BC_OK;
  cudaGetLastError();
  return entry_fail(BC_ECUDA, "%s: %s", where, cudaGetErrorString(e));
}

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Launch with programmatic stream serialisation (the kernel starts with
// pdl_wait()).
template <typename K, typename... A>
cudaError_t launch_op(K kern, dim3 grid, dim3 block, size_t smem, cudaStream_t st, const A&... a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a...);
}

}  // namespace bc
