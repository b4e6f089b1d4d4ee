// The global norm of many gradient tensors and clipping to it.
//
// Tensors travel in the kernels' argument block, cut into chunks.  One launch squares
// and sums each chunk, another scales; a second read of the gradients cannot be avoided,
// since the scale depends on all of them, but the scaling goes through the chunks from
// the last one back, so that what the squaring read last still lies in the 256 MB
// memory-side cache.  The chunks' sums are added in order by every workgroup of the
// scaling, or, when there are many, by a launch of their own.  Very few numbers are done
// by one workgroup in one launch.
// What bounds it: HBM.  302 million bf16 numbers (48 tensors) into another list: 333 us,
// 5.4 TB/s over two reads and a write; of 89 610 float32 numbers (six tensors) the
// launches.
// 16-byte accesses at any element alignment; they cost extra only where a line is
// crossed.
#include "vb_train_device.h"
#include "vb_train_internal.h"

namespace vb {

namespace {

// tensor of chunk b: the last one whose first chunk is not after it
template <int N>
__device__ __forceinline__ int clip_tensor(const ClipTable<N>& t, unsigned b) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= b) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <typename T>
struct Vec {
  static constexpr int EC = 16 / sizeof(T);
  typedef T type __attribute__((ext_vector_type(16 / sizeof(T))));
  typedef type loose __attribute__((aligned(sizeof(T))));
};

// Squares and their sum in float64: a float32 square would overflow from 2^64 on and
// lose values below 2^-75.  TH threads.
template <typename T, int TH>
__device__ __forceinline__ double squares(const void* p, long long beg, long long end, int tid) {
  constexpr int EC = Vec<T>::EC;
  const T* g = (const T*)p + beg;
  const int n = (int)(end - beg), full = n / EC;
  double s = 0.0;
#pragma unroll 4
  for (int c = tid; c < full; c += TH) {
    const typename Vec<T>::type v = *(const typename Vec<T>::loose*)(g + c * EC);
#pragma unroll
    for (int e = 0; e < EC; ++e) {
      const double x = (double)to_f32((T)v[e]);
      s = fma(x, x, s);
    }
  }
  if (tid < n - full * EC) {
    const double x = (double)to_f32(g[full * EC + tid]);
    s = fma(x, x, s);
  }
  return s;
}

template <typename T, int TH>
__device__ __forceinline__ void scaled(const void* p, void* q, long long beg, long long end, int tid, float s) {
  constexpr int EC = Vec<T>::EC;
  const T* g = (const T*)p + beg;
  T* o = (T*)q + beg;
  const int n = (int)(end - beg), full = n / EC;
  constexpr int U = 4;  // loads in flight: out may be the gradient itself, so they do not pass the stores
  for (int c = tid; c < full; c += U * TH) {
    typename Vec<T>::type v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + u * TH < full) v[u] = *(const typename Vec<T>::loose*)(g + (c + u * TH) * EC);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int e = 0; e < EC; ++e) v[u][e] = from_f32<T>(to_f32((T)v[u][e]) * s);
      if (c + u * TH < full) *(typename Vec<T>::loose*)(o + (c + u * TH) * EC) = v[u];
    }
  }
  if (tid < n - full * EC) o[full * EC + tid] = from_f32<T>(to_f32(g[full * EC + tid]) * s);
}

template <int TH, int N>
__device__ __forceinline__ double chunk_squares(const ClipTable<N>& t, unsigned b, int tid) {
  const int i = clip_tensor(t, b);
  const long long beg = (long long)(b - t.first[i]) * t.chunk, end = min(t.n[i], beg + t.chunk);
  if (t.dtype[i] == VB_F32) return squares<float, TH>(t.grad[i], beg, end, tid);
  if (t.dtype[i] == VB_BF16) return squares<bf16, TH>(t.grad[i], beg, end, tid);
  return squares<f16, TH>(t.grad[i], beg, end, tid);
}

template <int TH, int N>
__device__ __forceinline__ void chunk_scaled(const ClipTable<N>& t, unsigned b, int tid, float s) {
  const int i = clip_tensor(t, b);
  if (s == 1.f && t.out[i] == t.grad[i]) return;
  const long long beg = (long long)(b - t.first[i]) * t.chunk, end = min(t.n[i], beg + t.chunk);
  if (t.dtype[i] == VB_F32) scaled<float, TH>(t.grad[i], t.out[i], beg, end, tid, s);
  else if (t.dtype[i] == VB_BF16) scaled<bf16, TH>(t.grad[i], t.out[i], beg, end, tid, s);
  else scaled<f16, TH>(t.grad[i], t.out[i], beg, end, tid, s);
}

// Sum over a workgroup of TH threads, given to all of them.
template <int TH>
__device__ __forceinline__ double block_sum(double s) {
  __shared__ double red[TH / 64];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  s = red[0];
#pragma unroll
  for (int i = 1; i < TH / 64; ++i) s += red[i];
  return s;
}

// The scale of a norm; the norm is written by one thread.
__device__ __forceinline__ float clip_factor(double squares, float max_norm, float* norm, bool write) {
  const double v = sqrt(squares);
  if (write) *norm = (float)v;
  return v > (double)max_norm && (float)v < INFINITY ? (float)((double)max_norm / v) : 1.f;
}

template <int N>
__global__ __launch_bounds__(256) void clip_partial_kernel(ClipTable<N> t, double* partial) {
  const double s = block_sum<256>(chunk_squares<256>(t, blockIdx.x, threadIdx.x));
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(1024) void clip_norm_kernel(const double* partial, long long n, float max_norm,
                                                         float* norm, float* scale) {
  double s = 0.0;
#pragma unroll 4
  for (long long i = threadIdx.x; i < n; i += 1024) s += partial[i];
  s = block_sum<1024>(s);
  if (threadIdx.x == 0) *scale = clip_factor(s, max_norm, norm, true);
}

// n > 0: from the chunks' sums (the first launch's last workgroup writes the norm)
template <int N>
__global__ __launch_bounds__(256) void clip_scale_kernel(ClipTable<N> t, const float* scale, const double* partial, int n,
                                                         float max_norm, float* norm) {
  float f;
  if (n > 0) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += 256) s += partial[i];
    f = clip_factor(block_sum<256>(s), max_norm, norm, norm && blockIdx.x == 0 && threadIdx.x == 0);
  } else {
    f = *scale;
  }
  chunk_scaled<256>(t, gridDim.x - 1 - blockIdx.x, threadIdx.x, f);
}

// Everything at once: a chunk per wavefront at a time.
template <int N>
__global__ __launch_bounds__(1024) void clip_small_kernel(ClipTable<N> t, float max_norm, float* norm) {
  const unsigned chunks = t.first[t.count];
  double s = 0.0;
  for (unsigned b = threadIdx.x >> 6; b < chunks; b += 16) s += chunk_squares<64>(t, b, threadIdx.x & 63);
  // the barrier inside also separates the last read of a tensor from the first write
  const float f = clip_factor(block_sum<1024>(s), max_norm, norm, threadIdx.x == 0);
  for (unsigned b = threadIdx.x >> 6; b < chunks; b += 16) chunk_scaled<64>(t, b, threadIdx.x & 63, f);
}

}  // namespace

template <int N>
hipError_t launch_clip_partial(const ClipTable<N>& t, double* partial, hipStream_t st) {
  clip_partial_kernel<<<t.first[t.count], 256, 0, st>>>(t, partial);
  return hipGetLastError();
}

hipError_t launch_clip_norm(const double* partial, long long n, float max_norm, float* norm, float* scale,
                            hipStream_t st) {
  clip_norm_kernel<<<1, 1024, 0, st>>>(partial, n, max_norm, norm, scale);
  return hipGetLastError();
}

template <int N>
hipError_t launch_clip_scale(const ClipTable<N>& t, const float* scale, const double* partial, int n, float max_norm,
                             float* norm, hipStream_t st) {
  clip_scale_kernel<<<t.first[t.count], 256, 0, st>>>(t, scale, partial, n, max_norm, norm);
  return hipGetLastError();
}

template <int N>
hipError_t launch_clip_small(const ClipTable<N>& t, float max_norm, float* norm, hipStream_t st) {
  clip_small_kernel<<<1, 1024, 0, st>>>(t, max_norm, norm);
  return hipGetLastError();
}

template hipError_t launch_clip_partial(const ClipTable<CLIP_TENSORS>&, double*, hipStream_t);
template hipError_t launch_clip_partial(const ClipTable<CLIP_FEW_TENSORS>&, double*, hipStream_t);
template hipError_t launch_clip_scale(const ClipTable<CLIP_TENSORS>&, const float*, const double*, int, float, float*,
                                      hipStream_t);
template hipError_t launch_clip_scale(const ClipTable<CLIP_FEW_TENSORS>&, const float*, const double*, int, float,
                                      float*, hipStream_t);
template hipError_t launch_clip_small(const ClipTable<CLIP_TENSORS>&, float, float*, hipStream_t);
template hipError_t launch_clip_small(const ClipTable<CLIP_FEW_TENSORS>&, float, float*, hipStream_t);

}  // namespace vb
