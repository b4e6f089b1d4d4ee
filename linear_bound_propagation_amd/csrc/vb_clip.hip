// The global norm of many gradient tensors and clipping to it.
#include "vb_train_device.h"
#include "vb_train_internal.h"

namespace vb {

namespace {

// tensor of this workgroup: the last one whose first workgroup is not after it
__device__ __forceinline__ int clip_tensor(const ClipTable& t, unsigned b) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= b) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <typename T>
__device__ double chunk_squares(const T* g, long long beg, long long end) {
  double s = 0.0;
  for (long long i = beg + threadIdx.x; i < end; i += 256) {
    const double v = (double)to_f32(g[i]);
    s += v * v;
  }
  return s;
}

// Squares and their sum in float64: a float32 square would overflow from 2^64 on
// and lose values below 2^-75.
__global__ __launch_bounds__(256) void clip_partial_kernel(ClipTable t, double* partial) {
  __shared__ double red[256];
  const int i = clip_tensor(t, blockIdx.x);
  const long long beg = (long long)(blockIdx.x - t.first[i]) * CLIP_CHUNK;
  const long long end = min(t.n[i], beg + CLIP_CHUNK);
  double s;
  if (t.dtype[i] == VB_F32) s = chunk_squares((const float*)t.grad[i], beg, end);
  else if (t.dtype[i] == VB_BF16) s = chunk_squares((const bf16*)t.grad[i], beg, end);
  else s = chunk_squares((const f16*)t.grad[i], beg, end);
  red[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o >= 1; o >>= 1) {
    if ((int)threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) partial[blockIdx.x] = red[0];
}

__global__ __launch_bounds__(256) void clip_norm_kernel(const double* partial, long long n, float max_norm,
                                                        float* norm, float* scale) {
  __shared__ double red[256];
  double s = 0.0;
  for (long long i = threadIdx.x; i < n; i += 256) s += partial[i];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o >= 1; o >>= 1) {
    if ((int)threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const double v = sqrt(red[0]);
    *norm = (float)v;
    *scale = v > (double)max_norm && (float)v < INFINITY ? (float)((double)max_norm / v) : 1.f;
  }
}

template <typename T>
__device__ void chunk_scale(const T* g, T* out, long long beg, long long end, float s) {
  for (long long i = beg + threadIdx.x; i < end; i += 256) out[i] = from_f32<T>(to_f32(g[i]) * s);
}

__global__ __launch_bounds__(256) void clip_scale_kernel(ClipTable t, const float* scale) {
  const int i = clip_tensor(t, blockIdx.x);
  const float s = *scale;
  if (s == 1.f && t.out[i] == t.grad[i]) return;
  const long long beg = (long long)(blockIdx.x - t.first[i]) * CLIP_CHUNK;
  const long long end = min(t.n[i], beg + CLIP_CHUNK);
  if (t.dtype[i] == VB_F32) chunk_scale((const float*)t.grad[i], (float*)t.out[i], beg, end, s);
  else if (t.dtype[i] == VB_BF16) chunk_scale((const bf16*)t.grad[i], (bf16*)t.out[i], beg, end, s);
  else chunk_scale((const f16*)t.grad[i], (f16*)t.out[i], beg, end, s);
}

}  // namespace

hipError_t launch_clip_partial(const ClipTable& t, double* partial, hipStream_t st) {
  clip_partial_kernel<<<t.first[t.count], 256, 0, st>>>(t, partial);
  return hipGetLastError();
}

hipError_t launch_clip_norm(const double* partial, long long n, float max_norm, float* norm, float* scale,
                            hipStream_t st) {
  clip_norm_kernel<<<1, 256, 0, st>>>(partial, n, max_norm, norm, scale);
  return hipGetLastError();
}

hipError_t launch_clip_scale(const ClipTable& t, const float* scale, hipStream_t st) {
  clip_scale_kernel<<<t.first[t.count], 256, 0, st>>>(t, scale);
  return hipGetLastError();
}

}  // namespace vb
