// Host-side helpers of pad_api.cpp that the library's other host files use:
// descriptor checks, failure reports and the library-owned scratch.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <memory>
#include <mutex>

#include "pad.h"

namespace pad {

// Sets pad_last_error() (printf form) and returns `st`.
pad_status host_fail(pad_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
pad_status host_cuda_fail(cudaError_t e, const char *what);
// Non-null, of this dtype and rank, sizes and strides >= 0.
pad_status host_check_tensor(const pad_tensor *t, const char *name, pad_dtype dt, int ndim);
// Last dim contiguous, base and row strides 16-byte aligned.
pad_status host_check_rows16(const pad_tensor *t, const char *name, int64_t elem_bytes);
// Device (or managed) memory of `device`.
pad_status host_check_device_ptr(const void *p, int device, const char *name);
int host_sm_count(int device);
// The envelope of pad_decode (W: table width).
pad_status host_check_shape(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t bs, int64_t W);

// One scratch buffer per (device, stream), at least `bytes` long, contents
// arbitrary; freed by pad_release_workspace.  It grows outside stream capture
// only, and a buffer that a capture has seen is kept, not freed, when a larger
// one replaces it: the captured graph still uses it.
//
// The caller holds it until `hold` goes: a thread that wants the same stream's waits,
// so that one call's kernels stay together, and so does a release.  Other streams'
// are not waited for.
struct ScratchHold {
  void *ptr = nullptr;
  std::shared_ptr<void> owner;
  std::unique_lock<std::mutex> lock;  // (released before its owner)
};
pad_status host_scratch(int device, cudaStream_t stream, size_t bytes, ScratchHold *hold);

typedef CUresult (*TensorMapEncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                      const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                      CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                      CUtensorMapFloatOOBfill);
TensorMapEncodeFn host_tensor_map_encoder();  // null if the driver lacks it

}  // namespace pad
