// Softmax cross entropy of integer labels and its gradient.
#include "vb_train_device.h"
#include "vb_train_internal.h"

namespace vb {

namespace {

// sum over the workgroup's four wavefronts, given to every thread
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = (red[0] + red[1]) + (red[2] + red[3]);
  __syncthreads();
  return v;
}
__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  __syncthreads();
  return v;
}

// to float32 accuracy for float32 logits, else the hardware exponential (relative
// error 2^-20 at -16, where p is far below a 16-bit gradient's last place)
template <typename T>
__device__ __forceinline__ float exp_of(float v) {
  return sizeof(T) == 4 ? expf(v) : __expf(v);
}

// count of the rows that are not ignored
__global__ __launch_bounds__(256) void loss_count_kernel(const int64_t* labels, long long rows, int64_t ignore,
                                                         long long* count) {
  __shared__ long long red[256];
  long long c = 0;
  for (long long r = threadIdx.x; r < rows; r += 256) c += labels[r] != ignore;
  red[threadIdx.x] = c;
  __syncthreads();
  if (threadIdx.x == 0) {
    c = 0;
    for (int i = 0; i < 256; ++i) c += red[i];
    *count = c;
  }
}

// one workgroup per row
template <typename T>
__global__ __launch_bounds__(256) void loss_row_kernel(vb_cross_entropy_args p, const long long* count,
                                                       float* row_loss) {
  __shared__ float red[4];
  const long long r = blockIdx.x;
  const T* z = (const T*)p.logits + r * p.ld;
  T* d = p.dlogits ? (T*)p.dlogits + r * p.ld_d : nullptr;
  const int64_t t = p.labels[r];
  const int n = p.classes;
  if (t == p.ignore_index) {
    if (d)
      for (int i = threadIdx.x; i < n; i += 256) d[i] = (T)0.f;
    if (threadIdx.x == 0) row_loss[r] = 0.f;
    return;
  }
  // the mean is a sum of z / n: it stays finite for logits of the type's lowest value
  const float rn = 1.f / (float)n;
  float top = -INFINITY, mean = 0.f;
  for (int i = threadIdx.x; i < n; i += 256) {
    const float v = to_f32(z[i]);
    top = fmaxf(top, v);
    mean += v * rn;
  }
  top = block_max(top, red);
  mean = p.label_smoothing > 0.f ? block_sum(mean, red) : 0.f;
  float sum = 0.f;
  for (int i = threadIdx.x; i < n; i += 256) sum += exp_of<T>(to_f32(z[i]) - top);
  sum = block_sum(sum, red);
  const float eps = p.label_smoothing;
  const bool bad = t < 0 || t >= n;
  const float zt = bad ? NAN : to_f32(z[t]);
  const float lse = logf(sum);
  float loss = (1.f - eps) * (lse + (top - zt));
  if (eps > 0.f) loss += eps * (lse + (top - mean));
  __syncthreads();  // z[t] is read before a gradient over the same memory is written
  if (threadIdx.x == 0) row_loss[r] = loss;
  if (!d) return;
  const float s = bad ? NAN : p.grad_scale / (float)*count;
  const float inv = 1.f / sum, off = eps / (float)n;
  for (int i = threadIdx.x; i < n; i += 256) {
    float v = exp_of<T>(to_f32(z[i]) - top) * inv - off;
    if (i == t) v -= 1.f - eps;
    d[i] = from_f32<T>(v * s);
  }
}

__global__ __launch_bounds__(256) void loss_mean_kernel(const float* row_loss, long long rows, const long long* count,
                                                        float* loss) {
  __shared__ double red[256];
  double s = 0.0;
  for (long long r = threadIdx.x; r < rows; r += 256) s += row_loss[r];
  red[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int i = 0; i < 256; ++i) s += red[i];
    *loss = *count ? (float)(s / (double)*count) : 0.f;
  }
}

}  // namespace

hipError_t launch_cross_entropy(const vb_cross_entropy_args& p, void* ws, hipStream_t st) {
  long long* count = (long long*)ws;
  float* row_loss = p.row_loss ? p.row_loss : (float*)((char*)ws + 16);
  loss_count_kernel<<<1, 256, 0, st>>>(p.labels, p.rows, p.ignore_index, count);
  if (p.rows > 0) {
    const unsigned blocks = (unsigned)p.rows;
    if (p.dtype == VB_F32) loss_row_kernel<float><<<blocks, 256, 0, st>>>(p, count, row_loss);
    else if (p.dtype == VB_BF16) loss_row_kernel<bf16><<<blocks, 256, 0, st>>>(p, count, row_loss);
    else loss_row_kernel<f16><<<blocks, 256, 0, st>>>(p, count, row_loss);
  }
  if (p.loss) loss_mean_kernel<<<1, 256, 0, st>>>(row_loss, p.rows, count, p.loss);
  return hipGetLastError();
}

}  // namespace vb
