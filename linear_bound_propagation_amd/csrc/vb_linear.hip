// The fused linear layer y = act(x W^T + bias + residual) and the products of
// its backward pass.
#include "vb_train_device.h"
#include "vb_train_internal.h"

namespace vb {

namespace {

typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));

// exp and the normal CDF: to float32 accuracy for float32 data; for 16-bit data
// the hardware exponential (relative error 2^-21 over the range that matters) and
// 1 + erf (absolute error 2^-24, lost only where Phi < 2^-15).
template <typename T>
__device__ __forceinline__ float exp_of(float v) {
  return sizeof(T) == 4 ? expf(v) : __expf(v);
}
template <typename T>
__device__ __forceinline__ float normal_cdf(float v) {
  return sizeof(T) == 4 ? 0.5f * erfcf(v * -0.70710678118654752f) : 0.5f * (1.f + erff(v * 0.70710678118654752f));
}

template <typename T>
__device__ __forceinline__ float act_value(float v, int act) {
  if (act == VB_ACT_RELU) return v < 0.f ? 0.f : v;  // NaN stays NaN
  if (act == VB_ACT_GELU) return v * normal_cdf<T>(v);
  if (act == VB_ACT_SILU) return v / (1.f + exp_of<T>(-v));
  return v;
}

// dy * act'(pre) from what the forward pass saved
template <typename T>
__device__ __forceinline__ float act_grad(float dy, float s, int act) {
  if (act == VB_ACT_RELU) return s > 0.f ? dy : 0.f;
  if (act == VB_ACT_GELU)
    return dy * (normal_cdf<T>(s) + s * (0.3989422804014327f * exp_of<T>(-0.5f * s * s)));
  if (act == VB_ACT_SILU) {
    const float q = 1.f / (1.f + exp_of<T>(-s));
    return dy * (q * (1.f + s * (1.f - q)));
  }
  return dy;
}

constexpr int BM = 64, BN = 64, BK = 32;

template <typename T>
struct Tile;
template <>
struct Tile<float> {
  static constexpr int LD = BK + 4;
  __device__ static f32x4 mfma(const float* a, const float* b, int r, int g, f32x4 c) {
#pragma unroll
    for (int k = 0; k < BK; k += 4)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r * LD + k + g], b[r * LD + k + g], c, 0, 0, 0);
    return c;
  }
};
template <>
struct Tile<bf16> {
  static constexpr int LD = BK + 8;
  __device__ static f32x4 mfma(const bf16* a, const bf16* b, int r, int g, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(*(const bf16x8*)(a + r * LD + 8 * g),
                                                   *(const bf16x8*)(b + r * LD + 8 * g), c, 0, 0, 0);
  }
};
template <>
struct Tile<f16> {
  static constexpr int LD = BK + 8;
  __device__ static f32x4 mfma(const f16* a, const f16* b, int r, int g, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(*(const f16x8*)(a + r * LD + 8 * g),
                                                  *(const f16x8*)(b + r * LD + 8 * g), c, 0, 0, 0);
  }
};

// 64 x 64 outputs per workgroup of four wavefronts (32 x 32 each), operands of
// any strides through LDS in 32-deep steps.  MFMA rows run along n and columns
// along m, so a lane holds four consecutive n of one row of the output.
template <typename T>
__global__ __launch_bounds__(256) void product_kernel(Product p, int tiles_n) {
  constexpr int LD = Tile<T>::LD;
  __shared__ __align__(16) T as[BM * LD];
  __shared__ __align__(16) T bs[BN * LD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const long long m0 = (long long)(blockIdx.x / tiles_n) * BM;
  const int n0 = (int)(blockIdx.x % tiles_n) * BN;
  const T* a = (const T*)p.a;
  const T* b = (const T*)p.b;
  const int r16 = lane & 15, g = lane >> 4;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  f32x4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (long long k0 = 0; k0 < p.K; k0 += BK) {
    for (int e = tid; e < BM * BK; e += 256) {
      // consecutive threads along the operand's contiguous dimension
      const int r = p.sak == 1 ? e / BK : e % BM, k = p.sak == 1 ? e % BK : e / BM;
      const bool ok = m0 + r < p.M && k0 + k < p.K;
      as[r * LD + k] = ok ? a[(m0 + r) * p.sam + (k0 + k) * p.sak] : (T)0.f;
    }
    for (int e = tid; e < BN * BK; e += 256) {
      const int r = p.sbk == 1 ? e / BK : e % BN, k = p.sbk == 1 ? e % BK : e / BN;
      const bool ok = n0 + r < p.N && k0 + k < p.K;
      bs[r * LD + k] = ok ? b[(n0 + r) * p.sbn + (k0 + k) * p.sbk] : (T)0.f;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = Tile<T>::mfma(bs + (wn + 16 * i) * LD, as + (wm + 16 * j) * LD, r16, g, acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const long long m = m0 + wm + 16 * j + r16;
    if (m >= p.M) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + wn + 16 * i + 4 * g + q;
        if (n >= p.N) continue;
        float v = acc[i][j][q];
        if (p.bias) v += to_f32(((const T*)p.bias)[n]);
        if (p.res) v += to_f32(((const T*)p.res)[m * p.ld_res + n]);
        if (p.pre) ((T*)p.pre)[m * p.ld_pre + n] = from_f32<T>(v);
        ((T*)p.out)[m * p.ld_out + n] = from_f32<T>(act_value<T>(v, p.act));
      }
  }
}

// 64 columns per workgroup, four rows at a time
template <typename T>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGrad p) {
  __shared__ float red[4][64];
  const int c = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int n = blockIdx.x * 64 + c;
  float sum = 0.f;
  if (n < p.n)
    for (long long m = w; m < p.rows; m += 4) {
      const float s = p.saved ? to_f32(((const T*)p.saved)[m * p.ld_saved + n]) : 0.f;
      const float v = act_grad<T>(to_f32(((const T*)p.dy)[m * p.ld_dy + n]), s, p.act);
      if (p.g) ((T*)p.g)[m * p.ld_g + n] = from_f32<T>(v);
      if (p.dres) ((T*)p.dres)[m * p.ld_dres + n] = from_f32<T>(v);
      sum += v;
    }
  red[w][c] = sum;
  __syncthreads();
  if (w == 0 && n < p.n && p.dbias)
    ((T*)p.dbias)[n] = from_f32<T>((red[0][c] + red[1][c]) + (red[2][c] + red[3][c]));
}

__global__ __launch_bounds__(256) void fill_zero_kernel(unsigned short* p, long long rows, long long n, long long ld) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i < rows * n) p[i / n * ld + i % n] = 0;
}

}  // namespace

hipError_t launch_product(const Product& p, int dtype, hipStream_t st) {
  const int tn = (p.N + BN - 1) / BN;
  const long long blocks = (p.M + BM - 1) / BM * tn;
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  if (dtype == VB_F32) product_kernel<float><<<dim3((unsigned)blocks), 256, 0, st>>>(p, tn);
  else if (dtype == VB_BF16) product_kernel<bf16><<<dim3((unsigned)blocks), 256, 0, st>>>(p, tn);
  else product_kernel<f16><<<dim3((unsigned)blocks), 256, 0, st>>>(p, tn);
  return hipGetLastError();
}

hipError_t launch_act_grad(const ActGrad& p, int dtype, hipStream_t st) {
  const unsigned blocks = (unsigned)((p.n + 63) / 64);
  if (dtype == VB_F32) act_grad_kernel<float><<<blocks, 256, 0, st>>>(p);
  else if (dtype == VB_BF16) act_grad_kernel<bf16><<<blocks, 256, 0, st>>>(p);
  else act_grad_kernel<f16><<<blocks, 256, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_fill_zero(void* p, long long rows, long long row_bytes, long long ld_bytes, hipStream_t st) {
  const long long n = row_bytes / 2;
  const long long blocks = (rows * n + 255) / 256;
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  fill_zero_kernel<<<dim3((unsigned)blocks), 256, 0, st>>>((unsigned short*)p, rows, n, ld_bytes / 2);
  return hipGetLastError();
}

}  // namespace vb
