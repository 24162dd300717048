// Host-side helpers shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_ffn.h"

namespace moe {

constexpr int kMaxExperts = 1024;  // planner keeps 32 x E histogram words in shared memory
constexpr int kMaxDevices = 64;

inline bool valid_block_m(int bm) { return bm == 16 || bm == 32 || bm == 64 || bm == 128; }

// Records a formatted message for moe_last_error() and returns `code`.
int fail(int code, const char* fmt, ...);
// Records "<what>: <cuda error string>" and returns MOE_ERR_CUDA.
int cuda_fail(const char* what, cudaError_t err = cudaGetLastError());

// The driver's cuTensorMapEncodeTiled, or null where it cannot be had.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder();

// Device address of the current device's status word, which kernels set when
// a bounded wait runs out and moe_device_status() reads.
int status_word(const char* nm, int** word);

// Number of SMs of the current device (cached per device).
int sm_count();

}  // namespace moe
