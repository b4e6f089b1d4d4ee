// Layer norm and its backward pass.
//
// A row is read once and stays in registers: TH threads have a row, CH chunks of 16 bytes
// each (a wavefront per row up to 4 KB, a workgroup up to 128 KB).  Longer rows are read
// again for each step (CH = 0).  Rows may start anywhere: 16-byte accesses at element
// alignment are ordinary ones here, which cost extra only where a line is crossed; the last
// chunk is taken element by element where the row ends inside it.
#include <algorithm>

#include "vb_train_device.h"
#include "vb_train_internal.h"

namespace vb {

namespace {

template <typename T>
struct Vec {
  static constexpr int EC = 16 / sizeof(T);
  typedef T type __attribute__((ext_vector_type(16 / sizeof(T))));
  typedef type loose __attribute__((aligned(sizeof(T))));
};

// Elements i0 .. of a row of n, zeros past its end.
template <typename T>
__device__ __forceinline__ typename Vec<T>::type load_chunk(const T* row, int i0, int n) {
  constexpr int EC = Vec<T>::EC;
  typename Vec<T>::type v;
  if (i0 + EC <= n) {
    v = *(const typename Vec<T>::loose*)(row + i0);
  } else {
#pragma unroll
    for (int e = 0; e < EC; ++e) v[e] = i0 + e < n ? row[i0 + e] : (T)0.f;
  }
  return v;
}
template <typename T>
__device__ __forceinline__ void store_chunk(T* row, int i0, int n, const float* x) {
  constexpr int EC = Vec<T>::EC;
  typename Vec<T>::type v;
#pragma unroll
  for (int e = 0; e < EC; ++e) v[e] = from_f32<T>(x[e]);
  if (i0 + EC <= n) {
    *(typename Vec<T>::loose*)(row + i0) = v;
  } else {
#pragma unroll
    for (int e = 0; e < EC; ++e)
      if (i0 + e < n) row[i0 + e] = v[e];
  }
}
// weight or bias in float32; `none` where there is none
template <typename T>
__device__ __forceinline__ void load_factors(const T* p, int i0, int n, float none, float* f) {
  constexpr int EC = Vec<T>::EC;
  if (p) {
    const typename Vec<T>::type v = load_chunk(p, i0, n);
#pragma unroll
    for (int e = 0; e < EC; ++e) f[e] = to_f32((T)v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < EC; ++e) f[e] = none;
  }
}

// Keeps the compiler from carrying a row's converted values from one use to the next beside
// the row itself (three times the registers).
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

// Sums of a and b over the TH threads of a row, given to all of them; red: two words per
// wavefront, free again after the next barrier but one.
template <int TH>
__device__ __forceinline__ void sum_row(float& a, float& b, float (*red)[2]) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    a += __shfl_xor(a, o, 64);
    b += __shfl_xor(b, o, 64);
  }
  if (TH == 64) return;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][0] = a, red[threadIdx.x >> 6][1] = b;
  __syncthreads();
  a = red[0][0], b = red[0][1];
#pragma unroll
  for (int i = 1; i < TH / 64; ++i) a += red[i][0], b += red[i][1];
  __syncthreads();
}

// rows of a workgroup at a time
constexpr int rows_at_once(int th) { return th < 256 ? 256 / th : 1; }

// Differences are taken from the row's first element, whose distance from the others is as small
// as the row's own spread (equal numbers: 0, exactly), then from their mean, and as that is
// rounded, the mean of what is left comes beside the squares and is taken off as well.
template <typename T, int TH, int CH>
__global__ __launch_bounds__(TH < 256 ? 256 : TH) void norm_kernel(vb_layer_norm_fwd p) {
  constexpr int EC = Vec<T>::EC, PER = rows_at_once(TH);
  __shared__ float red[TH / 64][2];
  const long long r = (long long)workgroup_number() * PER + threadIdx.x / TH;
  if (r >= p.rows) return;  // whole wavefronts, and no barrier when PER > 1
  const int tid = threadIdx.x % TH, n = p.n, chunks = (n + EC - 1) / EC;
  const T* x = (const T*)p.x + r * p.ld_x;
  T* y = (T*)p.y + r * p.ld_y;
  typename Vec<T>::type v[CH ? CH : 1];
  // f(chunk, its first element) for each chunk of this thread
  auto each = [&](auto&& f) {
    if constexpr (CH > 0) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int i0 = (tid + k * TH) * EC;
        if (i0 < n) f(v[k], i0);
      }
    } else {
      for (int c = tid; c < chunks; c += TH) f(load_chunk(x, c * EC, n), c * EC);
    }
  };
  if constexpr (CH > 0) {
#pragma unroll
    for (int k = 0; k < CH; ++k) v[k] = load_chunk(x, (tid + k * TH) * EC, n);
  }
  const float inv = 1.f / (float)n, x0 = to_f32(x[0]);
  float first = 0.f, unused = 0.f;
  each([&](auto c, int i0) {
#pragma unroll
    for (int e = 0; e < EC; ++e) first += i0 + e < n ? to_f32((T)c[e]) - x0 : 0.f;
  });
  sum_row<TH>(first, unused, red);
  if constexpr (CH > 0) forget(v);
  first *= inv;
  float rest = 0.f, squares = 0.f;
  each([&](auto c, int i0) {
#pragma unroll
    for (int e = 0; e < EC; ++e) {
      const float d = i0 + e < n ? to_f32((T)c[e]) - x0 - first : 0.f;
      rest += d;
      squares = fmaf(d, d, squares);
    }
  });
  sum_row<TH>(rest, squares, red);
  if constexpr (CH > 0) forget(v);
  rest *= inv;
  float var = squares * inv - rest * rest;
  if (var < 0.f) var = 0.f;  // NaN stays
  const float rstd = 1.f / sqrtf(var + p.eps);
  each([&](auto c, int i0) {
    float w[EC], b[EC], o[EC];
    load_factors((const T*)p.weight, i0, n, 1.f, w);
    load_factors((const T*)p.bias, i0, n, 0.f, b);
#pragma unroll
    for (int e = 0; e < EC; ++e) o[e] = fmaf((to_f32((T)c[e]) - x0 - first - rest) * rstd, w[e], b[e]);
    store_chunk(y, i0, n, o);
  });
  if (tid == 0) {
    if (p.mean) p.mean[r] = x0 + (first + rest);
    if (p.rstd) p.rstd[r] = rstd;
  }
}

// ---------------------------------------------------------------------------
// Backward.  With dweight or dbias (SUMS) a workgroup goes through rows `gridDim.x` rows (of
// rows_at_once) apart and keeps their sums over its rows in registers, two float32 per column:
// x and dy are then read once.  Its sums are one of the parts that norm_sum_kernel adds.
template <typename T, int TH, int CH, bool SUMS>
__global__ __launch_bounds__(TH < 256 ? 256 : TH) void norm_grad_kernel(vb_layer_norm_bwd p, float* partial) {
  typedef typename Vec<T>::type V;
  constexpr int EC = Vec<T>::EC, PER = rows_at_once(TH), C1 = CH ? CH : 1;
  __shared__ float red[TH / 64][2];
  const int tid = threadIdx.x % TH, n = p.n, chunks = (n + EC - 1) / EC;
  const float inv = 1.f / (float)n;
  float sum_w[C1][EC], sum_b[C1][EC];
#pragma unroll
  for (int k = 0; k < C1; ++k)
#pragma unroll
    for (int e = 0; e < EC; ++e) sum_w[k][e] = sum_b[k][e] = 0.f;
  const unsigned groups = SUMS ? gridDim.x : 0;
  const bool with_x = p.dx || p.dweight;
  for (long long r = (long long)workgroup_number() * PER + threadIdx.x / TH; r < p.rows; r += (long long)groups * PER) {
    const T* x = (const T*)p.x + r * p.ld_x;
    const T* dy = (const T*)p.dy + r * p.ld_dy;
    const float mean = with_x ? p.mean[r] : 0.f, rstd = with_x ? p.rstd[r] : 0.f;
    V xv[C1], dv[C1];
    if constexpr (CH > 0) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int i0 = (tid + k * TH) * EC;
        xv[k] = with_x ? load_chunk(x, i0, n) : V{};
        dv[k] = load_chunk(dy, i0, n);
      }
    }
    // f(number of the chunk, its first element, xh, dy) for each chunk of this thread
    auto each = [&](auto&& f) {
      auto one = [&](int k, int i0, V xc, V dc) {
        float xh[EC], d[EC];
#pragma unroll
        for (int e = 0; e < EC; ++e) {
          xh[e] = i0 + e < n ? (to_f32((T)xc[e]) - mean) * rstd : 0.f;
          d[e] = to_f32((T)dc[e]);
        }
        f(k, i0, xh, d);
      };
      if constexpr (CH > 0) {
#pragma unroll
        for (int k = 0; k < CH; ++k)
          if ((tid + k * TH) * EC < n) one(k, (tid + k * TH) * EC, xv[k], dv[k]);
      } else {
        for (int c = tid; c < chunks; c += TH) one(0, c * EC, load_chunk(x, c * EC, n), load_chunk(dy, c * EC, n));
      }
    };
    float along = 0.f, level = 0.f;
    each([&](int k, int i0, const float* xh, const float* d) {
      float w[EC];
      load_factors((const T*)p.weight, i0, n, 1.f, w);
#pragma unroll
      for (int e = 0; e < EC; ++e) {
        const float g = d[e] * w[e];
        level += g;
        along = fmaf(g, xh[e], along);
        if (SUMS) {
          sum_w[k][e] = fmaf(d[e], xh[e], sum_w[k][e]);
          sum_b[k][e] += d[e];
        }
      }
    });
    if (!p.dx) continue;
    sum_row<TH>(along, level, red);
    if constexpr (CH > 0) forget(xv), forget(dv);
    along *= inv, level *= inv;
    T* dx = (T*)p.dx + r * p.ld_dx;
    const T* res = p.dresidual ? (const T*)p.dresidual + r * p.ld_dres : nullptr;
    each([&](int, int i0, const float* xh, const float* d) {
      float w[EC], q[EC], o[EC];
      load_factors((const T*)p.weight, i0, n, 1.f, w);
      load_factors(res, i0, n, 0.f, q);
#pragma unroll
      for (int e = 0; e < EC; ++e) o[e] = fmaf(rstd, fmaf(-along, xh[e], fmaf(d[e], w[e], -level)), q[e]);
      store_chunk(dx, i0, n, o);
    });
    if (!SUMS) return;
  }
  if constexpr (SUMS) {
    // rows side by side in a workgroup: their sums meet in LDS, a chunk of each thread at a time
    __shared__ float both[PER > 1 ? PER : 1][PER > 1 ? 64 * EC * 2 : 1];
    float* out = partial + (long long)workgroup_number() * 2 * n;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int i0 = (tid + k * TH) * EC;
      if constexpr (PER > 1) {
        __syncthreads();
        float* mine = both[threadIdx.x / TH];
#pragma unroll
        for (int e = 0; e < EC; ++e) mine[e * 64 + tid] = sum_w[k][e], mine[(EC + e) * 64 + tid] = sum_b[k][e];
        __syncthreads();
        if (threadIdx.x < TH) {
#pragma unroll
          for (int e = 0; e < EC; ++e)
#pragma unroll
            for (int j = 1; j < PER; ++j) {
              sum_w[k][e] += both[j][e * 64 + tid];
              sum_b[k][e] += both[j][(EC + e) * 64 + tid];
            }
        }
      }
      if (threadIdx.x < TH) {
#pragma unroll
        for (int e = 0; e < EC; ++e)
          if (i0 + e < n) out[i0 + e] = sum_w[k][e], out[n + i0 + e] = sum_b[k][e];
      }
    }
  }
}

// dweight and dbias of rows too long for their sums to stay in registers: a thread has a
// chunk of columns and every eighth of the workgroup's rows, 32 chunks a workgroup.
constexpr int LONG_ROWS = 64;
template <typename T>
__global__ __launch_bounds__(256) void norm_columns_kernel(vb_layer_norm_bwd p, float* partial) {
  constexpr int EC = Vec<T>::EC;
  __shared__ float red[2][8][32 * EC + 1];
  const unsigned across = (p.n + 32 * EC - 1) / (32 * EC), block = workgroup_number();
  const unsigned bx = block % across;
  const long long by = block / across, m0 = by * LONG_ROWS;
  if (m0 >= p.rows) return;  // the whole workgroup
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5, i0 = (bx * 32 + c) * EC;
  float sw[EC], sb[EC];
#pragma unroll
  for (int e = 0; e < EC; ++e) sw[e] = sb[e] = 0.f;
  if (i0 < p.n)
    for (long long m = m0 + w; m < min(m0 + LONG_ROWS, (long long)p.rows); m += 8) {
      const typename Vec<T>::type d = load_chunk((const T*)p.dy + m * p.ld_dy, i0, p.n);
      typename Vec<T>::type x{};
      float mean = 0.f, rstd = 0.f;
      if (p.dweight) {
        x = load_chunk((const T*)p.x + m * p.ld_x, i0, p.n);
        mean = p.mean[m], rstd = p.rstd[m];
      }
#pragma unroll
      for (int e = 0; e < EC; ++e) {
        const float g = to_f32((T)d[e]);
        sw[e] = fmaf(g, (to_f32((T)x[e]) - mean) * rstd, sw[e]);
        sb[e] += g;
      }
    }
#pragma unroll
  for (int e = 0; e < EC; ++e) red[0][w][c * EC + e] = sw[e], red[1][w][c * EC + e] = sb[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * EC; i += 256) {
    const int k = i / (32 * EC), j = i % (32 * EC), col = bx * 32 * EC + j;
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += red[k][q][j];
    if (col < p.n) partial[(by * 2 + k) * p.n + col] = s;
  }
}

// dweight and dbias from the parts, in their order: 64 columns per workgroup, in 16 sums of
// every 16th part, eight loads at a time.
template <typename T>
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float* partial, int parts, int n, T* dweight, T* dbias) {
  __shared__ float red[16][64];
  const int c = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + c;  // of 2 n
  constexpr int U = 8;
  float v = 0.f;
  if (col < 2 * n) {
    const float* q = partial + col;
    const long long step = 2LL * n;
    int i = w;
    for (; i + 16 * (U - 1) < parts; i += 16 * U) {
      float x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) x[u] = q[(i + 16 * u) * step];
#pragma unroll
      for (int u = 0; u < U; ++u) v += x[u];
    }
    for (; i < parts; i += 16) v += q[i * step];
  }
  red[w][c] = v;
  __syncthreads();
  if (w || col >= 2 * n) return;
  float sum = red[0][c];
#pragma unroll
  for (int k = 1; k < 16; ++k) sum += red[k][c];
  T* out = col < n ? dweight : dbias;
  if (out) out[col < n ? col : col - n] = from_f32<T>(sum);
}

template <typename T>
int chunks_of(int n) {
  return (n + Vec<T>::EC - 1) / Vec<T>::EC;
}

template <typename T, int TH, int CH>
hipError_t norm_rows(const vb_layer_norm_fwd& p, hipStream_t st) {
  constexpr int PER = rows_at_once(TH);
  norm_kernel<T, TH, CH><<<grid_of((p.rows + PER - 1) / PER), TH < 256 ? 256 : TH, 0, st>>>(p);
  return hipGetLastError();
}

template <typename T>
hipError_t norm_typed(const vb_layer_norm_fwd& p, hipStream_t st) {
  const int chunks = chunks_of<T>(p.n);
  if (chunks <= 64) return norm_rows<T, 64, 1>(p, st);
  if (chunks <= 128) return norm_rows<T, 64, 2>(p, st);
  if (chunks <= 256) return norm_rows<T, 64, 4>(p, st);
  if (chunks <= 512) return norm_rows<T, 256, 2>(p, st);
  if (chunks <= 1024) return norm_rows<T, 256, 4>(p, st);
  if (chunks <= 2048) return norm_rows<T, 256, 8>(p, st);
  if (chunks <= 4096) return norm_rows<T, 1024, 4>(p, st);
  if (chunks <= 8192) return norm_rows<T, 1024, 8>(p, st);
  return norm_rows<T, 1024, 0>(p, st);
}

// Workgroups that keep the sums of their rows, or rows of a part where a row is too long.
constexpr int SUM_GROUPS = 512, SUM_CHUNKS = 2048;
long long parts_of(long long rows, int n, int chunks) {
  if (chunks > SUM_CHUNKS) return (rows + LONG_ROWS - 1) / LONG_ROWS;
  const int per = chunks <= 256 ? 4 : 1;
  return std::min<long long>((rows + per - 1) / per, SUM_GROUPS);
}

template <typename T, int TH, int CH, bool SUMS>
hipError_t norm_grad_rows(const vb_layer_norm_bwd& p, float* partial, unsigned parts, hipStream_t st) {
  constexpr int PER = rows_at_once(TH);
  const dim3 grid = SUMS ? dim3(parts) : grid_of((p.rows + PER - 1) / PER);
  norm_grad_kernel<T, TH, CH, SUMS><<<grid, TH < 256 ? 256 : TH, 0, st>>>(p, partial);
  return hipGetLastError();
}

template <typename T, bool SUMS>
hipError_t norm_grad_sized(const vb_layer_norm_bwd& p, float* partial, unsigned parts, hipStream_t st) {
  const int chunks = chunks_of<T>(p.n);
  if (chunks <= 64) return norm_grad_rows<T, 64, 1, SUMS>(p, partial, parts, st);
  if (chunks <= 128) return norm_grad_rows<T, 64, 2, SUMS>(p, partial, parts, st);
  if (chunks <= 256) return norm_grad_rows<T, 64, 4, SUMS>(p, partial, parts, st);
  if (chunks <= 512) return norm_grad_rows<T, 256, 2, SUMS>(p, partial, parts, st);
  if (chunks <= 1024) return norm_grad_rows<T, 256, 4, SUMS>(p, partial, parts, st);
  if (chunks <= 2048) return norm_grad_rows<T, 1024, 2, SUMS>(p, partial, parts, st);
  if constexpr (!SUMS) {
    if (chunks <= 4096) return norm_grad_rows<T, 1024, 4, false>(p, partial, parts, st);
    return norm_grad_rows<T, 1024, 0, false>(p, partial, parts, st);
  }
  return hipErrorInvalidValue;
}

template <typename T>
hipError_t norm_grad_typed(const vb_layer_norm_bwd& p, float* ws, hipStream_t st) {
  if (!p.dweight && !p.dbias) return norm_grad_sized<T, false>(p, nullptr, 0, st);
  const int chunks = chunks_of<T>(p.n);
  const long long parts = parts_of(p.rows, p.n, chunks);
  if (chunks <= SUM_CHUNKS) {
    if (const hipError_t e = norm_grad_sized<T, true>(p, ws, (unsigned)parts, st)) return e;
  } else {
    // before dx, which may lie over dy
    const long long blocks = parts * ((p.n + 32 * Vec<T>::EC - 1) / (32 * Vec<T>::EC));
    if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    norm_columns_kernel<T><<<grid_of(blocks), 256, 0, st>>>(p, ws);
    if (const hipError_t e = hipGetLastError()) return e;
    if (p.dx)
      if (const hipError_t e = norm_grad_sized<T, false>(p, nullptr, 0, st)) return e;
  }
  norm_sum_kernel<T><<<(2 * p.n + 63) / 64, 1024, 0, st>>>(ws, (int)parts, p.n, (T*)p.dweight, (T*)p.dbias);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm(const vb_layer_norm_fwd& p, hipStream_t st) {
  if (p.dtype == VB_F32) return norm_typed<float>(p, st);
  if (p.dtype == VB_BF16) return norm_typed<bf16>(p, st);
  return norm_typed<f16>(p, st);
}

size_t norm_grad_bytes(long long rows, int n, int dtype) {
  const int ec = 16 / (int)elem_size(dtype), chunks = (n + ec - 1) / ec;
  return (size_t)parts_of(rows, n, chunks) * 2 * n * 4;
}

hipError_t launch_layer_norm_grad(const vb_layer_norm_bwd& p, float* ws, hipStream_t st) {
  if (p.dtype == VB_F32) return norm_grad_typed<float>(p, ws, st);
  if (p.dtype == VB_BF16) return norm_grad_typed<bf16>(p, ws, st);
  return norm_grad_typed<f16>(p, ws, st);
}

}  // namespace vb
