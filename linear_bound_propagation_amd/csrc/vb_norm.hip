// Layer norm and its backward pass.
//
// A row is read once and stays in registers: TH threads have a row, CH chunks of 16 bytes
// each.  Forward: 16 lanes per row up to 256 bytes, a wavefront up to 4 KB, a workgroup up to 128
// KB.  Backward, where a row is two or three: 16 lanes up to 256 bytes, a wavefront up to 1 KB, a
// workgroup up to 64 KB for dx.  Longer rows are read again for each step (CH = 0).  With dweight or
// dbias a row's columns have two float32 sums each in registers as well, up to rows of 32 KB; of
// longer ones, and of some short matrices (by_columns), dy and x are read twice.  Rows may start
// anywhere: 16-byte accesses at element alignment are ordinary ones here, which cost extra only where
// a line is crossed.
//
// What bounds it: HBM.  8192 x 8192 in bf16, 268 MB: 50 us, 5.4 TB/s (a large copy: 5.0);
// backward at 8192 x 4096 with dresidual, dweight and dbias, 268 MB and 17 of parts: 56 us.  Of float32
// rows beyond 8192 numbers the second reading: 2048 x 16384 138 us, 671 MB at 4.9 TB/s of 403 that one
// pass would move; 2048 x 8192 in one pass 44 us.
#include <algorithm>
#include <type_traits>

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
__device__ __forceinline__ typename Vec<T>::type load_part(const T* row, int i0, int n) {
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
__device__ __forceinline__ typename Vec<T>::type all_of(float f) {
  typename Vec<T>::type v;
#pragma unroll
  for (int e = 0; e < Vec<T>::EC; ++e) v[e] = (T)f;
  return v;
}

// A thread's chunks of a row of at least one: number k is TH chunks after number k - 1.  The row's
// last chunk ends with the row, so that some of its elements (skip of them) are the chunk's
// before it too: they count nothing in sums and are stored twice, alike.  Chunks past the end are
// that one again, and count nothing at all.  All threads then load as many whole chunks: no
// branch stands between a load and those of the rows after it.
// With CH = 0 a thread goes through as many chunks as the row has, each loaded where it is used.
template <typename T, int TH, int CH>
struct Chunks {
  static constexpr int EC = Vec<T>::EC;
  typedef typename Vec<T>::type V;
  typedef typename Vec<T>::loose L;
  int tid, n;
  __device__ int count() const { return CH ? CH : ((n + EC - 1) / EC - tid + TH - 1) / TH; }
  __device__ int begin(int k) const { return CH ? min((tid + k * TH) * EC, n - EC) : (tid + k * TH) * EC; }
  // elements before `skip` or from `end` on are not this chunk's
  __device__ int skip(int k) const { return CH ? min((tid + k * TH) * EC - begin(k), EC) : 0; }
  __device__ int end(int k) const { return CH ? EC : min(n - begin(k), EC); }
  __device__ V load(const T* row, int k) const {
    if constexpr (CH > 0) return *(const L*)(row + begin(k));
    else return load_part(row, begin(k), n);
  }
  __device__ void store(T* row, int k, const float* x) const {
    V v;
#pragma unroll
    for (int e = 0; e < EC; ++e) v[e] = from_f32<T>(x[e]);
    if (CH == 0 && end(k) < EC) {
#pragma unroll
      for (int e = 0; e < EC; ++e)
        if (e < end(k)) row[begin(k) + e] = v[e];
    } else if (skip(k) < EC) {
      *(L*)(row + begin(k)) = v;
    }
  }
  // zeros where x is not this chunk's
  __device__ void mask(int k, float* x) const {
    if (skip(k) == 0 && end(k) == EC) return;
#pragma unroll
    for (int e = 0; e < EC; ++e)
      if (e < skip(k) || e >= end(k)) x[e] = 0.f;
  }
  // f(k) for each chunk
  template <typename F>
  __device__ void each(F&& f) const {
    if constexpr (CH > 0) {
#pragma unroll
      for (int k = 0; k < CH; ++k) f(k);
    } else {
      for (int k = 0; k < count(); ++k) f(k);
    }
  }
};

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

// Sum over 16 lanes, or a wavefront, given to all of them: four steps within 16 lanes on the
// vector units (quad permutes, half mirror, mirror), then the four rows' sums as scalars.  (Six
// shuffles through LDS are six of its latencies on a row's critical path.)
template <int LANES>
__device__ __forceinline__ float sum_lanes(float v) {
  auto step = [](float x, auto ctrl) {
    return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v = step(v, std::integral_constant<int, 0xB1>());   // lane ^ 1
  v = step(v, std::integral_constant<int, 0x4E>());   // lane ^ 2
  v = step(v, std::integral_constant<int, 0x141>());  // 7 - lane, of 8
  v = step(v, std::integral_constant<int, 0x140>());  // 15 - lane, of 16
  if (LANES == 16) return v;
  auto row = [&](int lane) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane)); };
  return (row(0) + row(16)) + (row(32) + row(48));
}

// Sums of a and b over the TH threads of a row, given to all of them in a[0] and b[0]; red: two
// words per wavefront, of two sets in turn, so that one barrier does (all of the workgroup's
// threads).  S numbers of a thread are added as those of S TH threads would be.
template <int TH, int S>
__device__ __forceinline__ void sum_row(float (&a)[S], float (&b)[S], float (*red)[2]) {
  constexpr int W = TH / 64;
  static_assert(S == 1 || W >= 1, "numbers of whole wavefronts");
#pragma unroll
  for (int s = 0; s < S; ++s) a[s] = sum_lanes<TH == 16 ? 16 : 64>(a[s]), b[s] = sum_lanes<TH == 16 ? 16 : 64>(b[s]);
  if constexpr (S * W > 1) {
    const int wave = threadIdx.x >> 6, row = wave / W;
    red += row * S * W;
#pragma unroll
    for (int s = 0; s < S; ++s)
      if ((threadIdx.x & 63) == 0) red[s * W + wave - row * W][0] = a[s], red[s * W + wave - row * W][1] = b[s];
    __syncthreads();
    a[0] = red[0][0], b[0] = red[0][1];
#pragma unroll
    for (int i = 1; i < S * W; ++i) a[0] += red[i][0], b[0] += red[i][1];
  }
}
template <int TH>
__device__ __forceinline__ void sum_row(float& a, float& b, float (*red)[2]) {
  float x[1] = {a}, y[1] = {b};
  sum_row<TH, 1>(x, y, red);
  a = x[0], b = y[0];
}

// The mean is the row's first element and the mean of the differences from it, so that it is
// exact for equal numbers, whatever their size, and off by the rounding of the row's spread else.
// What it is off by, the mean of the differences from it, comes beside their squares and is
// taken off as well.
// Workgroups of WG threads have WG / TH rows at a time.
template <typename T, int WG, int TH, int CH>
__global__ __launch_bounds__(WG) void norm_kernel(vb_layer_norm_fwd p) {
  typedef typename Vec<T>::type V;
  constexpr int EC = Vec<T>::EC, PER = WG / TH;
  static_assert(PER == 1 || TH <= 64, "rows that end before others pass no barrier");
  __shared__ float red[2][WG / 64][2];
  const long long r = (long long)workgroup_number() * PER + threadIdx.x / TH;
  if (r >= p.rows) return;
  const Chunks<T, TH, CH> c{(int)threadIdx.x % TH, p.n};
  const T* x = (const T*)p.x + r * p.ld_x;
  T* y = (T*)p.y + r * p.ld_y;
  V v[CH ? CH : 1];
  if constexpr (CH > 0) c.each([&](int k) { v[k] = c.load(x, k); });
  auto differences = [&](int k, float from, float* d) {
    V u;
    if constexpr (CH > 0) u = v[k];
    else u = c.load(x, k);
#pragma unroll
    for (int e = 0; e < EC; ++e) d[e] = to_f32((T)u[e]) - from;
  };
  const float inv = 1.f / (float)p.n, x0 = to_f32(x[0]);
  float first = 0.f, unused = 0.f;
  c.each([&](int k) {
    float d[EC];
    differences(k, x0, d);
    c.mask(k, d);
#pragma unroll
    for (int e = 0; e < EC; ++e) first += d[e];
  });
  sum_row<TH>(first, unused, red[0]);
  if constexpr (CH > 0) forget(v);
  first = x0 + first * inv;
  float rest = 0.f, squares = 0.f;
  c.each([&](int k) {
    float d[EC];
    differences(k, first, d);
    c.mask(k, d);
#pragma unroll
    for (int e = 0; e < EC; ++e) rest += d[e], squares = fmaf(d[e], d[e], squares);
  });
  sum_row<TH>(rest, squares, red[1]);
  if constexpr (CH > 0) forget(v);
  rest *= inv;
  float var = squares * inv - rest * rest;
  if (var < 0.f) var = 0.f;  // NaN stays
  const float rstd = 1.f / sqrtf(var + p.eps);
  c.each([&](int k) {
    float d[EC];
    differences(k, first, d);
    const V w = p.weight ? c.load((const T*)p.weight, k) : all_of<T>(1.f);
    const V b = p.bias ? c.load((const T*)p.bias, k) : all_of<T>(0.f);
#pragma unroll
    for (int e = 0; e < EC; ++e) d[e] = fmaf((d[e] - rest) * rstd, to_f32((T)w[e]), to_f32((T)b[e]));
    c.store(y, k, d);
  });
  if (c.tid == 0) {
    if (p.mean) p.mean[r] = first + rest;
    if (p.rstd) p.rstd[r] = rstd;
  }
}

// ---------------------------------------------------------------------------
// Backward.

// A row of the backward pass in registers.
template <typename T, int CH>
struct GradRow {
  typename Vec<T>::type x[CH ? CH : 1], dy[CH ? CH : 1], res[CH ? CH : 1];
  float mean, rstd;
};

template <typename T, int TH, int CH, bool RES>
struct Grad {
  static constexpr int EC = Vec<T>::EC;
  typedef typename Vec<T>::type V;
  const vb_layer_norm_bwd& p;
  Chunks<T, TH, CH> c;
  V w[CH ? CH : 1];

  __device__ V weight(int k) const { return p.weight ? c.load((const T*)p.weight, k) : all_of<T>(1.f); }
  __device__ void load_weight() {
    if constexpr (CH > 0) c.each([&](int k) { w[k] = weight(k); });
  }
  __device__ void load(long long r, GradRow<T, CH>& row) const {
    row.mean = p.mean[r], row.rstd = p.rstd[r];
    if constexpr (CH > 0)
      c.each([&](int k) {
        row.x[k] = c.load((const T*)p.x + r * p.ld_x, k);
        row.dy[k] = c.load((const T*)p.dy + r * p.ld_dy, k);
        if (RES) row.res[k] = c.load((const T*)p.dresidual + r * p.ld_dres, k);
      });
  }
  // chunk k's xh, dy and weight
  __device__ void values(long long r, const GradRow<T, CH>& row, int k, float* xh, float* d, float* wf) const {
    V xv, dv, wv;
    if constexpr (CH > 0) xv = row.x[k], dv = row.dy[k], wv = w[k];
    else xv = c.load((const T*)p.x + r * p.ld_x, k), dv = c.load((const T*)p.dy + r * p.ld_dy, k), wv = weight(k);
#pragma unroll
    for (int e = 0; e < EC; ++e) {
      xh[e] = (to_f32((T)xv[e]) - row.mean) * row.rstd;
      d[e] = to_f32((T)dv[e]);
      wf[e] = to_f32((T)wv[e]);
    }
  }
  // f(k, xh, dy) of each chunk beside the row's two sums (S > 1: of chunk k in number k)
  template <int S, typename F>
  __device__ void sums(long long r, const GradRow<T, CH>& row, float (&along)[S], float (&level)[S], F&& f) const {
#pragma unroll
    for (int s = 0; s < S; ++s) along[s] = level[s] = 0.f;
    c.each([&](int k) {
      const int s = S > 1 ? k : 0;
      float xh[EC], d[EC], g[EC];
      values(r, row, k, xh, d, g);
#pragma unroll
      for (int e = 0; e < EC; ++e) g[e] *= d[e];
      c.mask(k, xh), c.mask(k, d), c.mask(k, g);
#pragma unroll
      for (int e = 0; e < EC; ++e) level[s] += g[e], along[s] = fmaf(g[e], xh[e], along[s]);
      f(k, xh, d);
    });
  }
  // dx from the sums over n
  __device__ void store(long long r, const GradRow<T, CH>& row, float along, float level) const {
    c.each([&](int k) {
      float xh[EC], d[EC], wf[EC], o[EC];
      values(r, row, k, xh, d, wf);
      V q{};
      if constexpr (RES && CH > 0) q = row.res[k];
      else if constexpr (RES) q = c.load((const T*)p.dresidual + r * p.ld_dres, k);
#pragma unroll
      for (int e = 0; e < EC; ++e) o[e] = fmaf(row.rstd, fmaf(-along, xh[e], fmaf(d[e], wf[e], -level)), to_f32((T)q[e]));
      c.store((T*)p.dx + r * p.ld_dx, k, o);
    });
  }
};

// Floats of a part's row: its columns' sums start on 16-byte boundaries.
__host__ __device__ inline int part_row(int n) { return (n + 3) / 4 * 4; }

// dweight and dbias of few rows, or of rows too long for their sums to stay in registers or
// shorter than a chunk: a thread has a chunk of columns and every (WG / ACROSS)th of the
// workgroup's part_rows rows, ACROSS chunks a workgroup (one, of rows shorter than that).
constexpr int COLUMN_ROWS = 64;
template <typename T, int WG, int ACROSS>
constexpr int column_words = 2 * (WG / ACROSS) * (ACROSS * Vec<T>::EC + 1);
template <typename T, int WG, int ACROSS>
__device__ __forceinline__ void sum_columns(const vb_layer_norm_bwd& p, unsigned block, int part_rows, float* partial, float* words) {
  typedef typename Vec<T>::type V;
  constexpr int EC = Vec<T>::EC, U = 4, SIDE = WG / ACROSS, COLS = ACROSS * EC;
  float(*red)[SIDE][COLS + 1] = (float(*)[SIDE][COLS + 1])words;
  const unsigned across = (p.n + COLS - 1) / COLS;
  const unsigned bx = block % across;
  const long long by = block / across, m0 = by * part_rows, end = min(m0 + part_rows, (long long)p.rows);
  if (m0 >= p.rows) return;  // the whole workgroup
  const int c = threadIdx.x % ACROSS, w = threadIdx.x / ACROSS, i0 = (bx * ACROSS + c) * EC;
  float sw[EC], sb[EC];
#pragma unroll
  for (int e = 0; e < EC; ++e) sw[e] = sb[e] = 0.f;
  if (i0 < p.n)
    for (long long m = m0 + w; m < end; m += SIDE * U) {
      V d[U], x[U];
      float mean[U], rstd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long r = m + SIDE * u;
        d[u] = x[u] = V{};
        mean[u] = rstd[u] = 0.f;
        if (r >= end) continue;
        d[u] = load_part((const T*)p.dy + r * p.ld_dy, i0, p.n);
        if (p.dweight) {
          x[u] = load_part((const T*)p.x + r * p.ld_x, i0, p.n);
          mean[u] = p.mean[r], rstd[u] = p.rstd[r];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < EC; ++e) {
          const float g = to_f32((T)d[u][e]);
          sw[e] = fmaf(g, (to_f32((T)x[u][e]) - mean[u]) * rstd[u], sw[e]);
          sb[e] += g;
        }
    }
#pragma unroll
  for (int e = 0; e < EC; ++e) red[0][w][c * EC + e] = sw[e], red[1][w][c * EC + e] = sb[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * COLS; i += WG) {
    const int k = i / COLS, j = i % COLS, col = bx * COLS + j;
    float s = 0.f;
#pragma unroll 32
    for (int q = 0; q < SIDE; ++q) s += red[k][q][j];
    if (col >= p.n) continue;
    if (partial) {
      partial[(by * 2 + k) * part_row(p.n) + col] = s;
    } else {
      T* out = (T*)(k ? p.dbias : p.dweight);
      if (out) out[col] = from_f32<T>(s);
    }
  }
}

// norm_sums_kernel has 512 threads for the rows that 256 with two chunks each have here: their sums
// are added in its order, so that dx has the same bits without dweight and dbias.
template <int TH, int CH>
constexpr int sums_apart = TH == 256 && CH == 2 ? 2 : 1;
template <typename T, int WG, int TH, int CH, bool RES>
__device__ __forceinline__ void dx_rows(const vb_layer_norm_bwd& p, unsigned block, float (*red)[2]) {
  constexpr int PER = WG / TH, S = sums_apart<TH, CH>;
  static_assert(PER == 1 || TH <= 64, "rows that end before others pass no barrier");
  const long long r = (long long)block * PER + threadIdx.x / TH;
  if (r >= p.rows) return;
  Grad<T, TH, CH, RES> g{p, {(int)threadIdx.x % TH, p.n}};
  GradRow<T, CH> row;
  g.load(r, row);
  g.load_weight();
  float along[S], level[S];
  g.sums(r, row, along, level, [](int, const float*, const float*) {});
  sum_row<TH, S>(along, level, red);
  if constexpr (CH > 0) forget(row.x), forget(row.dy), forget(g.w);
  const float inv = 1.f / (float)p.n;
  g.store(r, row, along[0] * inv, level[0] * inv);
}

template <typename T, int WG, int TH, int CH, bool RES>
__global__ __launch_bounds__(WG) void norm_dx_kernel(vb_layer_norm_bwd p) {
  __shared__ float red[WG / 64 * sums_apart<TH, CH>][2];
  dx_rows<T, WG, TH, CH, RES>(p, workgroup_number(), red);
}

// Few rows: the workgroups of dx, then those of dweight and dbias, of one launch (16 x 100 in
// float32: 3.0 us, in two 5.5; 64 x 16384 in bf16 5.2 and 9.2).
template <typename T, int WG, int TH, int CH, bool RES>
__global__ __launch_bounds__(WG) void norm_few_kernel(vb_layer_norm_bwd p, unsigned row_blocks) {
  __shared__ float words[column_words<T, WG, 32>];
  if (blockIdx.x < row_blocks) dx_rows<T, WG, TH, CH, RES>(p, blockIdx.x, (float(*)[2])words);
  else sum_columns<T, WG, 32>(p, blockIdx.x - row_blocks, COLUMN_ROWS, nullptr, words);
}

// dx (DX) and the sums of dweight and dbias in one pass: a workgroup goes through the rows, WG / TH
// at a time, and keeps its rows' sums in registers, two float32 per column.  A row is on its way
// while another is worked on, by loads without conditions, as the compiler waits for all
// loads behind one (16384 x 2000 in float16 62 us with, 42 without): past the end they are of the
// last row.  Not where two chunks of 1024 threads would spill for it (4096 x 16384 in bf16: 209
// us, without 114).  The sums of rows side by side meet in LDS, and a workgroup's are one of the
// parts that norm_sum_kernel adds.
template <typename T, int WG, int TH, int CH, bool DX, bool RES>
__global__ __launch_bounds__(WG) void norm_sums_kernel(vb_layer_norm_bwd p, float* partial) {
  constexpr int EC = Vec<T>::EC, PER = WG / TH, AHEAD = CH == 1 || WG < 1024;
  __shared__ float red[2][WG / 64][2];
  Grad<T, TH, CH, RES> g{p, {(int)threadIdx.x % TH, p.n}};
  const int n = p.n, side = threadIdx.x / TH;
  const float inv = 1.f / (float)n;
  float sum_w[CH][EC], sum_b[CH][EC];
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int e = 0; e < EC; ++e) sum_w[k][e] = sum_b[k][e] = 0.f;
  const long long first = (long long)workgroup_number() * PER, step = (long long)gridDim.x * PER;
  GradRow<T, CH> row[AHEAD + 1];
  g.load_weight();
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) g.load(min(first + side + i * step, p.rows - 1), row[i]);
  int set = 0;
  for (long long r0 = first; r0 < p.rows; r0 += step) {
    const long long r = r0 + side;
    g.load(min(r + AHEAD * step, p.rows - 1), row[AHEAD]);
    float along[1], level[1];
    g.sums(r, row[0], along, level, [&](int k, const float* xh, const float* d) {
#pragma unroll
      for (int e = 0; e < EC; ++e) {
        if (PER == 1 || r < p.rows) {
          sum_w[k][e] = fmaf(d[e], xh[e], sum_w[k][e]);
          sum_b[k][e] += d[e];
        }
      }
    });
    if (DX) {
      sum_row<TH, 1>(along, level, red[set]);
      set ^= 1;
      forget(row[0].x), forget(row[0].dy), forget(g.w);
      if (r < p.rows) g.store(r, row[0], along[0] * inv, level[0] * inv);
    }
    forget(g.w);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) row[i] = row[i + 1];
  }
  __shared__ __align__(16) float both[PER > 1 ? PER : 1][2][PER > 1 ? TH * EC : 4];
  float* out = partial + (long long)workgroup_number() * 2 * part_row(n);
  g.c.each([&](int k) {
    const int at = PER > 1 ? g.c.begin(k) - k * TH * EC : g.c.begin(k), skip = g.c.skip(k);
    float *to_w = PER > 1 ? both[side][0] : out, *to_b = PER > 1 ? both[side][1] : out + part_row(n);
    if (PER > 1) __syncthreads();
    if (skip == 0) {
#pragma unroll
      for (int e = 0; e < EC; e += 4) {
        *(f32x4*)(to_w + at + e) = f32x4{sum_w[k][e], sum_w[k][e + 1], sum_w[k][e + 2], sum_w[k][e + 3]};
        *(f32x4*)(to_b + at + e) = f32x4{sum_b[k][e], sum_b[k][e + 1], sum_b[k][e + 2], sum_b[k][e + 3]};
      }
    } else {
#pragma unroll
      for (int e = 0; e < EC; ++e)
        if (e >= skip) to_w[at + e] = sum_w[k][e], to_b[at + e] = sum_b[k][e];
    }
    if constexpr (PER > 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * TH * EC; i += WG) {
        const int of = i / (TH * EC), j = i % (TH * EC), col = k * TH * EC + j;
        float sum = both[0][of][j];
#pragma unroll
        for (int q = 1; q < PER; ++q) sum += both[q][of][j];
        if (col < n) out[of * part_row(n) + col] = sum;
      }
    }
  });
}

template <typename T, int ACROSS>
__global__ __launch_bounds__(256) void norm_columns_kernel(vb_layer_norm_bwd p, int part_rows, float* partial) {
  __shared__ float red[column_words<T, 256, ACROSS>];
  sum_columns<T, 256, ACROSS>(p, workgroup_number(), part_rows, partial, red);
}

// dweight and dbias from the parts, in their order: 64 columns per workgroup, in 16 sums of
// every 16th part, eight loads at a time.
template <typename T>
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float* partial, int parts, int n, T* dweight, T* dbias) {
  __shared__ float red[16][64];
  const int c = threadIdx.x & 63, w = threadIdx.x >> 6, across = (n + 63) / 64;
  const int of = blockIdx.x / across, col = blockIdx.x % across * 64 + c;
  constexpr int U = 8;
  float v = 0.f;
  if (col < n) {
    const long long step = 2LL * part_row(n);
    const float* q = partial + (long long)of * part_row(n) + col;
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
  if (w || col >= n) return;
  float sum = red[0][c];
#pragma unroll
  for (int k = 1; k < 16; ++k) sum += red[k][c];
  T* out = of ? dbias : dweight;
  if (out) out[col] = from_f32<T>(sum);
}

template <typename T>
int chunks_of(int n) {
  return (n + Vec<T>::EC - 1) / Vec<T>::EC;
}

template <typename T, int WG, int TH, int CH>
hipError_t norm_rows(const vb_layer_norm_fwd& p, hipStream_t st) {
  constexpr int PER = WG / TH;
  norm_kernel<T, WG, TH, CH><<<grid_of((p.rows + PER - 1) / PER), WG, 0, st>>>(p);
  return hipGetLastError();
}

template <typename T>
hipError_t norm_typed(const vb_layer_norm_fwd& p, hipStream_t st) {
  const int chunks = chunks_of<T>(p.n);
  if (p.n < Vec<T>::EC) return norm_rows<T, 256, 16, 0>(p, st);
  if (chunks <= 16) return norm_rows<T, 256, 16, 1>(p, st);
  if (chunks <= 64) return norm_rows<T, 256, 64, 1>(p, st);
  if (chunks <= 128) return norm_rows<T, 256, 64, 2>(p, st);
  if (chunks <= 256) return norm_rows<T, 256, 64, 4>(p, st);
  if (chunks <= 512) return norm_rows<T, 256, 256, 2>(p, st);
  if (chunks <= 1024) return norm_rows<T, 256, 256, 4>(p, st);
  if (chunks <= 2048) return norm_rows<T, 512, 512, 4>(p, st);
  if (chunks <= 4096) return norm_rows<T, 1024, 1024, 4>(p, st);
  if (chunks <= 8192) return norm_rows<T, 1024, 1024, 8>(p, st);
  return norm_rows<T, 1024, 1024, 0>(p, st);
}

// Parts of the sums: workgroups that keep those of their rows, one a CU, as each part is
// written and read again (8192 x 4096 in bf16 with 512 parts of 512 threads: 68 against 63 us).
constexpr int SUM_GROUPS = 256, SUM_CHUNKS = 2048;
long long groups_of(long long rows, int chunks) {
  const int per = chunks <= 16 ? 64 : chunks <= 64 ? 16 : chunks <= 128 ? 8 : chunks <= 256 ? 4 : chunks <= 512 ? 2 : 1;
  return std::min<long long>((rows + per - 1) / per, SUM_GROUPS);
}
// By columns where sums do not stay in registers (or rows are less than a chunk), and where one
// workgroup has all rows of a column (64 x 16384 in bf16: 5.2 us, as parts 13.2; 33 x 2001 in float16 5.5
// and 7.3).  Between those, of long rows that end on a chunk's boundary (a row's odd end takes a
// workgroup loads of single elements: 200 x 6001 in bf16 15.9 us, as parts 14.0), where reading the rows
// twice costs less than a part for nearly every row: us as parts | by columns, 16 bits at 8192 70 rows
// 9.6 | 10.5, 100 11.0 | 10.5, 256 16.8 | 11.8, 512 17.4 | 15.7, 640 16.8 | 18.2; at 16384 128 17.7 | 12.4,
// 512 25.7 | 24.1, 768 30.0 | 31.9; float32 at 4096 128 7.6 | 9.4, 200 10.5 | 9.9, 300 11.3 | 10.9, 400 11.7 |
// 12.0; at 8192 70 9.3 | 9.9, 256 16.6 | 14.0, 384 17.9 | 18.0; rows of 8 KB and less the same or slower.
bool by_columns(long long rows, int n, int es) {
  const int chunks = (n * es + 15) / 16;
  if (n * es < 16 || chunks > SUM_CHUNKS || rows <= COLUMN_ROWS) return true;
  return chunks > 512 && n * es % 16 == 0 && rows * n > 700000 && rows * es <= 1100;
}
// Rows of a part by columns: COLUMN_ROWS, or four of each thread where a row is less than a chunk;
// more where there would be over COLUMN_PARTS parts, each of whose numbers is added to a float32
// sum (2^24 x 7 in float16, dx and all: with a part per 64 rows 6.6 ms, so 3.0).
constexpr int COLUMN_PARTS = 1024;
int column_rows(long long rows, int n, int es) {
  const int unit = n * es < 16 ? 1024 : COLUMN_ROWS;
  const long long parts = (rows + unit - 1) / unit;
  return unit * (int)((parts + COLUMN_PARTS - 1) / COLUMN_PARTS);
}
long long parts_of(long long rows, int n, int es) {
  if (!by_columns(rows, n, es)) return groups_of(rows, (n * es + 15) / 16);
  const int per = column_rows(rows, n, es);
  return (rows + per - 1) / per;
}

template <typename T, int WG, int TH, int CH>
hipError_t norm_sums_rows(const vb_layer_norm_bwd& p, float* partial, unsigned parts, hipStream_t st) {
  if (!p.dx) norm_sums_kernel<T, WG, TH, CH, false, false><<<parts, WG, 0, st>>>(p, partial);
  else if (!p.dresidual) norm_sums_kernel<T, WG, TH, CH, true, false><<<parts, WG, 0, st>>>(p, partial);
  else norm_sums_kernel<T, WG, TH, CH, true, true><<<parts, WG, 0, st>>>(p, partial);
  return hipGetLastError();
}

template <typename T>
hipError_t norm_sums(const vb_layer_norm_bwd& p, float* partial, unsigned parts, hipStream_t st) {
  const int chunks = chunks_of<T>(p.n);
  if (chunks <= 16) return norm_sums_rows<T, 1024, 16, 1>(p, partial, parts, st);
  if (chunks <= 64) return norm_sums_rows<T, 1024, 64, 1>(p, partial, parts, st);
  if (chunks <= 128) return norm_sums_rows<T, 1024, 128, 1>(p, partial, parts, st);
  if (chunks <= 256) return norm_sums_rows<T, 1024, 256, 1>(p, partial, parts, st);
  if (chunks <= 512) return norm_sums_rows<T, 1024, 512, 1>(p, partial, parts, st);
  if (chunks <= 1024) return norm_sums_rows<T, 512, 512, 2>(p, partial, parts, st);
  return norm_sums_rows<T, 1024, 1024, 2>(p, partial, parts, st);
}

// What norm_dx launches: dx, of few rows dweight and dbias, or both.
enum Wanted { DX, COLUMNS, BOTH };

template <typename T, int WG, int TH, int CH>
hipError_t norm_dx_rows(const vb_layer_norm_bwd& p, Wanted what, hipStream_t st) {
  constexpr int PER = WG / TH;
  const long long blocks = what == COLUMNS ? 0 : (p.rows + PER - 1) / PER;
  if (what == DX) {
    if (p.dresidual) norm_dx_kernel<T, WG, TH, CH, true><<<grid_of(blocks), WG, 0, st>>>(p);
    else norm_dx_kernel<T, WG, TH, CH, false><<<grid_of(blocks), WG, 0, st>>>(p);
  } else {
    const unsigned all = (unsigned)blocks + (p.n + 32 * Vec<T>::EC - 1) / (32 * Vec<T>::EC);
    if (p.dresidual) norm_few_kernel<T, WG, TH, CH, true><<<all, WG, 0, st>>>(p, (unsigned)blocks);
    else norm_few_kernel<T, WG, TH, CH, false><<<all, WG, 0, st>>>(p, (unsigned)blocks);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t norm_dx(const vb_layer_norm_bwd& p, Wanted what, hipStream_t st) {
  const int chunks = chunks_of<T>(p.n);
  if (p.n < Vec<T>::EC) return norm_dx_rows<T, 256, 16, 0>(p, what, st);
  if (chunks <= 16) return norm_dx_rows<T, 256, 16, 1>(p, what, st);
  if (chunks <= 64) return norm_dx_rows<T, 256, 64, 1>(p, what, st);
  if (chunks <= 128) return norm_dx_rows<T, 128, 128, 1>(p, what, st);
  if (chunks <= 256) return norm_dx_rows<T, 256, 256, 1>(p, what, st);
  if (chunks <= 512) return norm_dx_rows<T, 256, 256, 2>(p, what, st);
  if (chunks <= 1024) return norm_dx_rows<T, 512, 512, 2>(p, what, st);
  if (chunks <= 2048) return norm_dx_rows<T, 1024, 1024, 2>(p, what, st);
  if (chunks <= 4096) return norm_dx_rows<T, 1024, 1024, 4>(p, what, st);
  return norm_dx_rows<T, 1024, 1024, 0>(p, what, st);
}

template <typename T>
hipError_t norm_grad_typed(const vb_layer_norm_bwd& p, float* ws, hipStream_t st) {
  if (!p.dweight && !p.dbias) return norm_dx<T>(p, DX, st);
  const long long parts = parts_of(p.rows, p.n, sizeof(T));
  if (p.rows <= COLUMN_ROWS) {
    if (p.dx && p.dx != p.dy) return norm_dx<T>(p, BOTH, st);
    if (const hipError_t e = norm_dx<T>(p, COLUMNS, st)) return e;  // before dx, which may lie over dy
    return p.dx ? norm_dx<T>(p, DX, st) : hipSuccess;
  }
  if (!by_columns(p.rows, p.n, sizeof(T))) {
    if (const hipError_t e = norm_sums<T>(p, ws, (unsigned)parts, st)) return e;
  } else {
    // before dx here too
    const int per = column_rows(p.rows, p.n, sizeof(T));
    if (p.n < Vec<T>::EC) norm_columns_kernel<T, 1><<<(unsigned)parts, 256, 0, st>>>(p, per, ws);
    else norm_columns_kernel<T, 32><<<grid_of(parts * ((p.n + 32 * Vec<T>::EC - 1) / (32 * Vec<T>::EC))), 256, 0, st>>>(p, per, ws);
    if (const hipError_t e = hipGetLastError()) return e;
    if (p.dx)
      if (const hipError_t e = norm_dx<T>(p, DX, st)) return e;
  }
  norm_sum_kernel<T><<<(p.n + 63) / 64 * 2, 1024, 0, st>>>(ws, (int)parts, p.n, (T*)p.dweight, (T*)p.dbias);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm(const vb_layer_norm_fwd& p, hipStream_t st) {
  if (p.dtype == VB_F32) return norm_typed<float>(p, st);
  if (p.dtype == VB_BF16) return norm_typed<bf16>(p, st);
  return norm_typed<f16>(p, st);
}

size_t norm_grad_bytes(long long rows, int n, int dtype) {
  return (size_t)parts_of(rows, n, (int)elem_size(dtype)) * 2 * part_row(n) * 4;
}

hipError_t launch_layer_norm_grad(const vb_layer_norm_bwd& p, float* ws, hipStream_t st) {
  if (p.dtype == VB_F32) return norm_grad_typed<float>(p, ws, st);
  if (p.dtype == VB_BF16) return norm_grad_typed<bf16>(p, ws, st);
  return norm_grad_typed<f16>(p, ws, st);
}

}  // namespace vb
