// Types and conversions shared by the kernels of the training operators.
#pragma once

#include <hip/hip_runtime.h>

#include "vb_train_internal.h"

namespace vb {

typedef __bf16 bf16;
typedef _Float16 f16;
typedef float f32x4 __attribute__((ext_vector_type(4)));

// of a grid made by grid_of
__device__ __forceinline__ unsigned workgroup_number() { return blockIdx.z * GRID_X + blockIdx.x; }

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  return (float)v;
}
// to nearest even
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  return (T)v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

}  // namespace vb
