// Softmax cross entropy of integer labels and its gradient.
//
// A row is read once and stays in registers: its maximum, the sum of its exponentials
// and its gradient are taken from there, so that a pass moves the logits once in and
// the gradient once out.  TH threads have a row, CH chunks of 16 bytes each: a wavefront
// per row up to 4 KB, a workgroup of 256 or 1024 threads up to 256 KB (65536 float32 or
// 131072 16-bit classes).  Longer rows are read twice (one_row_twice).
// Chunks lie on 16-byte boundaries of memory whatever the row's start; the first and the
// last one are taken element by element.
//
// What bounds it: HBM.  4096 x 65536 in bf16, 1.07 GB in and out: 211 us, 5.1 TB/s, as
// fast as a large copy.  The count of the rows that the mean divides by is a launch of
// its own: counted by every row's workgroup it took the time twice over (408 us), the
// labels' loads delaying the row's.
#include "vb_train_device.h"
#include "vb_train_internal.h"

namespace vb {

namespace {

// To float32 accuracy for float32 logits, else the hardware exponential, whose argument is
// rounded (relative error 2^-20 at -16).  In a 16-bit gradient that is nothing.  In a loss the
// numbers far below the top count little, and the float32 sum's own rounding is as large: worst
// relative error of 64 losses of 65536 normal logits 2^-22.8 in bfloat16, 2^-22.5 in float32.
template <typename T>
__device__ __forceinline__ float exp_of(float v) {
  return sizeof(T) == 4 ? expf(v) : __expf(v);
}

template <typename T>
struct Vec {
  static constexpr int EC = 16 / sizeof(T);
  typedef T type __attribute__((ext_vector_type(16 / sizeof(T))));
  typedef type loose __attribute__((aligned(sizeof(T))));
};

struct Maximum {
  __device__ static float join(float a, float b) { return fmaxf(a, b); }
};
struct Sum {
  __device__ static float join(float a, float b) { return a + b; }
};

// Over the TH threads of a row, given to all of them; red: a word per wavefront.
template <typename Op, int TH>
__device__ __forceinline__ float over_row(float v, float* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = Op::join(v, __shfl_xor(v, o, 64));
  if (TH == 64) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < TH / 64; ++i) v = Op::join(v, red[i]);
  __syncthreads();
  return v;
}

// Keeps the compiler from carrying a row's converted or exponentiated values from one
// use to the next beside the row itself (three times the registers).
template <typename V, int CH>
__device__ __forceinline__ void forget(V (&v)[CH]) {
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    u32x4 w = __builtin_bit_cast(u32x4, v[k]);
    asm volatile("" : "+v"(w));
    v[k] = __builtin_bit_cast(V, w);
  }
}

// One row.  scale: grad_scale / n.  Returns the row's loss.
template <typename T, int TH, int CH>
__device__ __forceinline__ float one_row(const vb_cross_entropy_args& p, long long r, float scale, float* red) {
  typedef typename Vec<T>::type V;
  typedef typename Vec<T>::loose LV;
  constexpr int EC = Vec<T>::EC;
  const int tid = threadIdx.x % TH;
  const T* z = (const T*)p.logits + r * p.ld;
  T* d = p.dlogits ? (T*)p.dlogits + r * p.ld_d : nullptr;
  const int n = p.classes;
  const int lead = (int)((uintptr_t)z % 16 / sizeof(T));  // elements before the row in its first chunk
  const int chunks = (lead + n + EC - 1) / EC;
  const int64_t t = p.labels[r];
  if (t == p.ignore_index) {
    if (d)
      for (int c = tid; c < chunks; c += TH) {
        const int i0 = c * EC - lead;
        if (i0 >= 0 && i0 + EC <= n) {
          V v;
#pragma unroll
          for (int e = 0; e < EC; ++e) v[e] = (T)0.f;
          *(LV*)(d + i0) = v;
        } else {
          for (int i = max(i0, 0); i < min(i0 + EC, n); ++i) d[i] = (T)0.f;
        }
      }
    return 0.f;
  }
  const bool bad = t < 0 || t >= n;
  const float zt = bad ? NAN : to_f32(z[t]);
  const float eps = p.label_smoothing;
  V v[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = tid + k * TH, i0 = c * EC - lead;
    if (c < chunks && i0 >= 0 && i0 + EC <= n) {
      v[k] = *(const V*)(z + i0);
    } else {
#pragma unroll
      for (int e = 0; e < EC; ++e) v[k][e] = i0 + e >= 0 && i0 + e < n ? z[i0 + e] : (T)(-INFINITY);
    }
  }
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int e = 0; e < EC; ++e) top = fmaxf(top, to_f32((T)v[k][e]));
  top = over_row<Maximum, TH>(top, red);
  forget(v);
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    if (tid + k * TH >= chunks) break;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < EC; ++e) s += exp_of<T>(to_f32((T)v[k][e]) - top);
    sum += s;
  }
  sum = over_row<Sum, TH>(sum, red);
  forget(v);
  const float lse = logf(sum);
  float loss = (1.f - eps) * (lse + (top - zt));
  if (eps > 0.f) {
    // a sum of z / n: finite for logits of the type's lowest value
    const float rn = 1.f / (float)n;
    float mean = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int e = 0; e < EC; ++e) {
        const int i = (tid + k * TH) * EC - lead + e;
        mean += i >= 0 && i < n ? to_f32((T)v[k][e]) * rn : 0.f;
      }
    mean = over_row<Sum, TH>(mean, red);
    forget(v);
    loss += eps * (lse + (top - mean));
  }
  if (!d) return loss;
  // (p - eps / n) scale, and at the label (p - (1 - eps) - eps / n) scale
  const float s = bad ? NAN : scale, inv = 1.f / sum, off = eps / (float)n;
  const int tc = bad ? -1 : ((int)t + lead) / EC, te = bad ? 0 : ((int)t + lead) % EC;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = tid + k * TH, i0 = c * EC - lead;
    if (c >= chunks) break;
    float g[EC];
#pragma unroll
    for (int e = 0; e < EC; ++e) g[e] = exp_of<T>(to_f32((T)v[k][e]) - top) * inv - off;
    if (c == tc) {
#pragma unroll
      for (int e = 0; e < EC; ++e)
        if (e == te) g[e] -= 1.f - eps;
    }
    V o;
#pragma unroll
    for (int e = 0; e < EC; ++e) o[e] = from_f32<T>(g[e] * s);
    if (i0 >= 0 && i0 + EC <= n) {
      *(LV*)(d + i0) = o;
    } else {
#pragma unroll
      for (int e = 0; e < EC; ++e)
        if (i0 + e >= 0 && i0 + e < n) d[i0 + e] = o[e];
    }
  }
  return loss;
}

// Rows too long for registers: the maximum and the sum of exponentials in one pass (a
// thread rescales its sum when its maximum grows), the gradient in a second.
template <typename T>
__device__ __forceinline__ float one_row_twice(const vb_cross_entropy_args& p, long long r, float scale, float* red) {
  typedef typename Vec<T>::type V;
  typedef typename Vec<T>::loose LV;
  constexpr int TH = 1024, U = 4, EC = Vec<T>::EC;
  const T* z = (const T*)p.logits + r * p.ld;
  T* d = p.dlogits ? (T*)p.dlogits + r * p.ld_d : nullptr;
  const int n = p.classes, tid = threadIdx.x;
  const int lead = (int)((uintptr_t)z % 16 / sizeof(T)), chunks = (lead + n + EC - 1) / EC;
  const int64_t t = p.labels[r];
  const bool ignored = t == p.ignore_index, bad = t < 0 || t >= n;
  if (ignored && !d) return 0.f;
  const float zt = bad ? NAN : to_f32(z[t]);
  const float eps = p.label_smoothing, rn = 1.f / (float)n;
  auto chunk = [&](int c) {
    const int i0 = c * EC - lead;
    V v;
    if (c < chunks && i0 >= 0 && i0 + EC <= n) {
      v = *(const V*)(z + i0);
    } else {
#pragma unroll
      for (int e = 0; e < EC; ++e) v[e] = i0 + e >= 0 && i0 + e < n ? z[i0 + e] : (T)(-INFINITY);
    }
    return v;
  };
  // The running maximum starts at the lowest finite number: a thread without a finite
  // logit then holds a sum of zeros (or NaN from +inf or NaN), not -inf minus -inf.
  constexpr float LOW = -3.402823466e38f;
  float top = LOW, sum = 0.f, mean = 0.f;
  if (!ignored) {
    for (int c = tid; c < chunks; c += U * TH) {
      V v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = chunk(c + u * TH);
      float m = top;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < EC; ++e) m = fmaxf(m, to_f32((T)v[u][e]));
      sum *= exp_of<T>(top - m);
      top = m;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < EC; ++e) {
          const float x = to_f32((T)v[u][e]);
          const int i = (c + u * TH) * EC - lead + e;
          sum += exp_of<T>(x - m);
          if (eps > 0.f && i >= 0 && i < n) mean += x * rn;
        }
    }
    const float all = over_row<Maximum, TH>(top, red);
    sum = over_row<Sum, TH>(sum * exp_of<T>(top - all), red);
    if (sum == 0.f) sum = NAN;  // no finite logit at all: 0 / 0, as the formula
    top = all;
  }
  const float lse = logf(sum);
  float loss = (1.f - eps) * (lse + (top - zt));
  if (eps > 0.f) loss += eps * (lse + (top - over_row<Sum, TH>(mean, red)));
  if (ignored) loss = 0.f;
  if (!d) return loss;
  const float s = bad ? NAN : scale, inv = 1.f / sum, off = eps / (float)n;
  const int at = bad ? -1 - EC : (int)t;
  for (int c = tid; c < chunks; c += U * TH) {
    V v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = chunk(c + u * TH);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i0 = (c + u * TH) * EC - lead;
      if (i0 >= n) break;
      V o;
#pragma unroll
      for (int e = 0; e < EC; ++e) {
        float g = exp_of<T>(to_f32((T)v[u][e]) - top) * inv - off;
        if (i0 + e == at) g -= 1.f - eps;
        o[e] = ignored ? (T)0.f : from_f32<T>(g * s);
      }
      if (i0 >= 0 && i0 + EC <= n) {
        *(LV*)(d + i0) = o;
      } else {
#pragma unroll
        for (int e = 0; e < EC; ++e)
          if (i0 + e >= 0 && i0 + e < n) d[i0 + e] = o[e];
      }
    }
  }
  return loss;
}

// count of the rows that are not ignored, over a workgroup of 1024
__device__ __forceinline__ long long count_rows(const int64_t* labels, long long rows, int64_t ignore) {
  __shared__ int red[16];
  int c = 0;
  for (long long r = threadIdx.x; r < rows; r += 1024) c += labels[r] != ignore;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) c += __shfl_xor(c, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = c;
  __syncthreads();
  long long n = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) n += red[i];
  return n;
}

// mean of the rows' losses, in float64 and a fixed order, over a workgroup of 1024
__device__ __forceinline__ void mean_loss(const float* row_loss, long long rows, long long count, float* loss) {
  __shared__ double red[16];
  double s = 0.0;
  for (long long r = threadIdx.x; r < rows; r += 1024) s += row_loss[r];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int i = 0; i < 16; ++i) s += red[i];
    *loss = count ? (float)(s / (double)count) : 0.f;
  }
}

__global__ __launch_bounds__(1024) void loss_count_kernel(const int64_t* labels, long long rows, int64_t ignore,
                                                          long long* count) {
  const long long n = count_rows(labels, rows, ignore);
  if (threadIdx.x == 0) *count = n;
}

__global__ __launch_bounds__(1024) void loss_mean_kernel(const float* row_loss, long long rows, const long long* count,
                                                         float* loss) {
  mean_loss(row_loss, rows, *count, loss);
}

// Rows of up to 128 KB leave registers for two rows per CU at a time, so that one loads
// while the other computes (4096 x 65536 in bf16: 237 us, one row at a time 271).
template <typename T, int TH, int CH>
__global__ __launch_bounds__(TH < 256 ? 256 : TH, CH <= 8 ? 8 : 4) void loss_rows_kernel(vb_cross_entropy_args p,
                                                                        const long long* count, float* row_loss) {
  __shared__ float red[16];
  constexpr int PER = TH < 256 ? 256 / TH : 1;
  const long long r = (long long)workgroup_number() * PER + threadIdx.x / TH;
  if (r >= p.rows) return;  // whole wavefronts, and no barrier when PER > 1
  const float scale = p.grad_scale / (float)*count;
  float loss;
  if constexpr (CH > 0) loss = one_row<T, TH, CH>(p, r, scale, red);
  else loss = one_row_twice<T>(p, r, scale, red);
  if (threadIdx.x % TH == 0) row_loss[r] = loss;
}

// A few short rows: everything in one launch of one workgroup, a wavefront per row.
template <typename T>
__global__ __launch_bounds__(1024) void loss_small_kernel(vb_cross_entropy_args p, float* row_loss) {
  const long long count = count_rows(p.labels, p.rows, p.ignore_index);
  const float scale = p.grad_scale / (float)count;
  for (long long r = threadIdx.x >> 6; r < p.rows; r += 16) {
    const float loss = one_row<T, 64, 1>(p, r, scale, nullptr);
    if ((threadIdx.x & 63) == 0) row_loss[r] = loss;
  }
  __syncthreads();  // row_loss is written: the barrier waits for this workgroup's stores
  if (p.loss) mean_loss(row_loss, p.rows, count, p.loss);
}

template <typename T>
hipError_t launch_typed(const vb_cross_entropy_args& p, void* ws, hipStream_t st) {
  long long* count = (long long*)ws;
  float* row_loss = p.row_loss ? p.row_loss : (float*)((char*)ws + 16);
  // the most chunks a row touches: one more when rows start off 16-byte boundaries
  const bool aligned = (uintptr_t)p.logits % 16 == 0 && p.ld * sizeof(T) % 16 == 0;
  const long long chunks = ((long long)p.classes * sizeof(T) + 15) / 16 + !aligned;
  if (p.rows <= 64 && chunks <= 64) {
    loss_small_kernel<T><<<1, 1024, 0, st>>>(p, row_loss);
    return hipGetLastError();
  }
  loss_count_kernel<<<1, 1024, 0, st>>>(p.labels, p.rows, p.ignore_index, count);
  if (const hipError_t e = hipGetLastError()) return e;
  if (p.rows > 0) {
    const dim3 rows = grid_of(p.rows), quads = grid_of((p.rows + 3) / 4);
    if (chunks <= 64) loss_rows_kernel<T, 64, 1><<<quads, 256, 0, st>>>(p, count, row_loss);
    else if (chunks <= 256) loss_rows_kernel<T, 64, 4><<<quads, 256, 0, st>>>(p, count, row_loss);
    else if (chunks <= 1024) loss_rows_kernel<T, 256, 4><<<rows, 256, 0, st>>>(p, count, row_loss);
    else if (chunks <= 2048) loss_rows_kernel<T, 256, 8><<<rows, 256, 0, st>>>(p, count, row_loss);
    else if (chunks <= 4096) loss_rows_kernel<T, 1024, 4><<<rows, 1024, 0, st>>>(p, count, row_loss);
    else if (chunks <= 8192) loss_rows_kernel<T, 1024, 8><<<rows, 1024, 0, st>>>(p, count, row_loss);
    else if (chunks <= 10240) loss_rows_kernel<T, 1024, 10><<<rows, 1024, 0, st>>>(p, count, row_loss);
    else if (chunks <= 12288) loss_rows_kernel<T, 1024, 12><<<rows, 1024, 0, st>>>(p, count, row_loss);
    else if (chunks <= 16384) loss_rows_kernel<T, 1024, 16><<<rows, 1024, 0, st>>>(p, count, row_loss);
    else loss_rows_kernel<T, 1024, 0><<<rows, 1024, 0, st>>>(p, count, row_loss);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (p.loss) loss_mean_kernel<<<1, 1024, 0, st>>>(row_loss, p.rows, count, p.loss);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cross_entropy(const vb_cross_entropy_args& p, void* ws, hipStream_t st) {
  if (p.dtype == VB_F32) return launch_typed<float>(p, ws, st);
  if (p.dtype == VB_BF16) return launch_typed<bf16>(p, ws, st);
  return launch_typed<f16>(p, ws, st);
}

}  // namespace vb
