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

// The bytes of a matrix: rows of `bytes`, `ld` bytes apart (no less than `bytes`).
struct Span {
  uintptr_t at;
  int64_t rows, bytes, ld;
};
inline bool is_empty(const Span& s) { return !s.at || s.rows <= 0 || s.bytes <= 0; }

// Do two matrices share a byte?  Rows may lie between each other's.
inline bool overlap(Span a, Span b) {
  if (is_empty(a) || is_empty(b)) return false;
  const int64_t d = (int64_t)(a.at - b.at);  // a's start, seen from b's
  if (d >= (b.rows - 1) * b.ld + b.bytes || -d >= (a.rows - 1) * a.ld + a.bytes) return false;
  // the first row of b, counted on before and past its ends, that ends after byte s
  auto row_after = [&](int64_t s) {
    const int64_t q = s - b.bytes;
    return (q >= 0 ? q / b.ld : -((-q + b.ld - 1) / b.ld)) + 1;
  };
  if (a.ld == b.ld) {  // row r of a lies to row r + j of b as row 0 to row j, whatever r
    for (int64_t j = row_after(d), end = j + 2; j < end; ++j)
      if (j * b.ld < d + a.bytes && -j < a.rows && j < b.rows) return true;
    return false;
  }
  if (a.rows > b.rows) return overlap(b, a);
  for (int64_t r = 0; r < a.rows; ++r) {
    const int64_t s = d + r * a.ld, first = row_after(s), j = first < 0 ? 0 : first;
    if (j < b.rows && j * b.ld < s + a.bytes) return true;
  }
  return false;
}

// Grid of `blocks` workgroups, at most 2^31: a dimension of a launch holds less than 2^32
// work-items, so from GRID_X workgroups of up to 1024 threads on they go on in z (y is the
// kernel's).  Kernels number them by workgroup_number, and those past the last have no work.
constexpr unsigned GRID_X = 1u << 21;  // a multiple of the number of XCDs
inline dim3 grid_of(long long blocks, unsigned y = 1) {
  if (blocks <= GRID_X) return dim3((unsigned)blocks, y);
  return dim3(GRID_X, y, (unsigned)((blocks + GRID_X - 1) / GRID_X));
}

// C(m, n) = sum_k A(m, k) B(n, k) with A(m, k) = a[m * lda + k], or a[k * lda + m] when
// across_a (likewise b); across_a implies across_b.  Unless
// product_is_narrow, both operands are chunked (is_chunked over their rows as
// stored; a row along the reduction may also be one that launch_pack filled with zeros).
// With passes = 2 (16-bit types, across_b) A is 2 a + 2^(1 - p) a_low, p the type's
// significand bits, and a_low is stored like a.
struct Product {
  const void* a;
  const void* a_low;
  int passes;
  const void* b;
  long long lda, ldb;
  bool across_a, across_b;
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
  // workspace of product_bytes: float32 parts of a reduction split over workgroups
  float* partial;
  // set by launch_product
  int ld_partial, split_steps;
};
struct Tiling {
  int bm, bn, splits;
  double us;  // as estimated
};
bool product_is_narrow(const Product& p, int dtype);
size_t product_bytes(const Product& p, int dtype);
hipError_t launch_product(const Product& p, int dtype, hipStream_t st);

// Rows of n elements that start on 16-byte boundaries, end on one, and are near enough
// for 32-bit offsets within a tile.
constexpr long long MAX_CHUNKED_ROW = 1 << 22;
bool is_chunked(const void* p, long long ld, long long n, int dtype);
// Bytes of a row of n elements rounded up to 16.
inline size_t chunked_row(long long n, int dtype) { return (n * elem_size(dtype) + 15) / 16 * 16; }
// Copies rows of n elements to chunked rows, zeros to the end of the last chunk; two
// matrices at once (dst NULL: none).
struct PackJob {
  const void* src;
  long long ld, rows;
  int n;
  void* dst;
  // set by launch_pack
  int chunks;
  unsigned blocks;
};
struct PackJobs {
  PackJob job[2];
};
hipError_t launch_pack(PackJobs jobs, int dtype, hipStream_t st);

// v = dy * act'(saved), in float32: g = v (rows of ld_g elements that start on 16-byte
// boundaries, zeros to the end of the last chunk) or, with g_low, v = 2 g + 2^(1 - p) g_low
// as in Product; dres = v, dbias = column sums of v; each optional.  partial:
// act_grad_bytes of workspace for dbias.
struct ActGrad {
  const void* dy;
  const void* saved;
  long long ld_dy, ld_saved;
  void* g;
  void* g_low;
  long long ld_g;
  void* dres;
  long long ld_dres;
  void* dbias;
  float* partial;
  long long rows;
  int n;
  int act;
  // set by launch_act_grad: rows of a workgroup, workgroups
  int part_rows;
  unsigned blocks;
};
// dbias from sums over parts of the rows, parts x n
struct ColumnSums {
  const float* partial;
  int parts, n;
  void* out;  // NULL: nothing to sum
};
size_t act_grad_bytes(long long rows, int n, int dtype);
// sums: set if dbias is left for launch_column_sums or launch_pair
hipError_t launch_act_grad(const ActGrad& p, PackJobs jobs, int dtype, ColumnSums& sums, hipStream_t st);
hipError_t launch_column_sums(const ColumnSums& s, int dtype, hipStream_t st);
// Both products of a backward pass by one launch, with tiles of this side (0: use two)
int pair_tile(const Product& dx, const Product& dw, int dtype);
hipError_t launch_pair(const Product& dx, const Product& dw, int tile, const ColumnSums& s, int dtype, hipStream_t st);
hipError_t launch_fill_zero(void* p, long long rows, long long row_bytes, long long ld_bytes, hipStream_t st);

// ws: the count of the rows that are not ignored (int64, in 16 bytes), then the rows' losses
// (float32) if the caller does not want them
hipError_t launch_cross_entropy(const vb_cross_entropy_args& p, void* ws, hipStream_t st);

// Gradient tensors in the kernels' argument block, cut into chunks of `chunk` elements:
// up to CLIP_TENSORS of them at a time, or CLIP_FEW_TENSORS in a block an eighth as long
// (six tensors: 8.3 us a call against 8.9).
constexpr int CLIP_TENSORS = 112, CLIP_FEW_TENSORS = 16;
constexpr int CLIP_CHUNK = 16384;        // of a workgroup of 256
constexpr int CLIP_FEW_CHUNK = 2048;     // the same, while there are at most
constexpr int CLIP_FEW = 1024;           // this many chunks
constexpr long long CLIP_MAX_CHUNKS = (1 << 24) - 1;  // of a call: 2^38 elements
constexpr int CLIP_SMALL_CHUNK = 512;    // of a wavefront, when one workgroup does all:
constexpr long long CLIP_SMALL = 16384;  // up to this many elements
template <int N>
struct ClipTable {
  const void* grad[N];
  void* out[N];
  long long n[N];
  unsigned first[N + 1];  // chunks before tensor i of this launch
  unsigned char dtype[N];
  int count, chunk;
};
template <int N>
hipError_t launch_clip_partial(const ClipTable<N>& t, double* partial, hipStream_t st);
hipError_t launch_clip_norm(const double* partial, long long n, float max_norm, float* norm, float* scale,
                            hipStream_t st);
// n > 0: the scale from n chunks' sums (norm: written, unless NULL), else from *scale
template <int N>
hipError_t launch_clip_scale(const ClipTable<N>& t, const float* scale, const double* partial, int n, float max_norm,
                             float* norm, hipStream_t st);
template <int N>
hipError_t launch_clip_small(const ClipTable<N>& t, float max_norm, float* norm, hipStream_t st);

}  // namespace vb
