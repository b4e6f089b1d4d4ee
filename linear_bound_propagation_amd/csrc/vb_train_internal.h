// Internal interface between the host side (vb_train.cpp) and the kernels
// (vb_linear.hip, vb_loss.hip, vb_clip.hip) of the training operators.
#pragma once

#include <hip/hip_runtime_api.h>
#include <cstddef>
#include <cstdint>

#include "vb_train.h"

namespace vb {

// Sets the calling thread's error description (vb_api.cpp) and returns s.
vb_status set_error(vb_status s, const char* msg) noexcept;

inline size_t elem_size(int dtype) { return dtype == VB_F32 ? 4 : 2; }

// C[m][n] = sum_k A(m, k) B(n, k), with A(m, k) = a[m * sam + k * sak] and
// B(n, k) = b[n * sbn + k * sbk] (one stride of each operand is 1).
struct Product {
  const void* a;
  const void* b;
  long long sam, sak, sbn, sbk;
  long long M;
  int N;
  long long K;
  // epilogue: v = sum + bias[n] + res[m][n]; pre = v; out = act(v)
  const void* bias;
  const void* res;
  long long ld_res;
  void* out;
  long long ld_out;
  void* pre;
  long long ld_pre;
  int act;
};
hipError_t launch_product(const Product& p, int dtype, hipStream_t st);

// g = dy * act'(saved) -> g and dres (each optional), and the column sums of the
// unrounded g -> dbias (optional).
struct ActGrad {
  const void* dy;
  const void* saved;
  long long ld_dy, ld_saved;
  void* g;
  long long ld_g;
  void* dres;
  long long ld_dres;
  void* dbias;
  long long rows;
  int n;
  int act;
};
hipError_t launch_act_grad(const ActGrad& p, int dtype, hipStream_t st);
hipError_t launch_fill_zero(void* p, long long rows, long long row_bytes, long long ld_bytes, hipStream_t st);

// ws: one int64 (count of the rows that are not ignored)
hipError_t launch_cross_entropy(const vb_cross_entropy_args& p, void* ws, hipStream_t st);

// Gradient tensors in the kernels' argument block: CLIP_TENSORS of them at a time.
constexpr int CLIP_TENSORS = 112;
constexpr int CLIP_CHUNK = 16384;  // elements of one workgroup
struct ClipTable {
  const void* grad[CLIP_TENSORS];
  void* out[CLIP_TENSORS];
  long long n[CLIP_TENSORS];
  unsigned first[CLIP_TENSORS + 1];  // workgroups before tensor i of this launch
  unsigned char dtype[CLIP_TENSORS];
  int count;
};
hipError_t launch_clip_partial(const ClipTable& t, double* partial, hipStream_t st);
hipError_t launch_clip_norm(const double* partial, long long n, float max_norm, float* norm, float* scale,
                            hipStream_t st);
hipError_t launch_clip_scale(const ClipTable& t, const float* scale, hipStream_t st);

}  // namespace vb
