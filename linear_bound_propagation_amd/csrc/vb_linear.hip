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

// ---------------------------------------------------------------------------
// The large product C = A B^T of operands whose rows are contiguous along the
// reduction and start on 16-byte boundaries.
//
// Workgroups of WM x WN wavefronts compute BM x BN tiles.  Both operands pass
// through a ring of NS stages in LDS, each 64 bytes of the reduction deep (32 16-bit
// or 16 float32 numbers), loaded straight from global memory.  NS - 1 stages are in
// flight at a time: all workgroups of an XCD reach new memory together, so a stage's
// first touch waits for HBM and needs about two microseconds of products to hide
// (with two stages of 128 bytes the matrix cores were busy 57 % of the clocks).
// A wavefront's tile is MT x NT blocks of 16 x 16 outputs (v_mfma 16x16x32: at this
// size the card is limited by power, and on the same random operands, from registers,
// the 16-wide instructions ran at 1.63 GHz against 1.52 GHz for 32x32x16).  A stage is
// two phases: the products of the upper half of the rows, under which the lower half
// is read from LDS; then the barrier; then the products of the lower half, under which
// the next stage's upper half and columns are read.  No wavefront waits on the barrier
// or on LDS with idle matrix cores.
// Chunk c of row r lies at position c ^ ((r >> 2) & 3) of the row: the 16 rows that
// a quarter of a wavefront reads together (256 bytes a clock) then fall on different
// LDS banks; measured 4.1 clocks a 1 KB read, against 16 for c ^ (r & 3).  A direct
// load writes 64 consecutive chunks (16 rows), so the permutation is done on the
// global side; a row's four lanes still cover its 64 bytes.
// Float32 uses the same bytes: MFMA step s of a chunk takes element s of it for
// both operands, which permutes the reduction alike on both sides.

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes of a row; mma: the products of a wavefront's 64 chunks (16 rows x 4) of each operand
template <typename T>
struct Chunk;
template <>
struct Chunk<float> {
  typedef f32x4 type;
  static constexpr int MFMAS = 4;
  __device__ static f32x4 mma(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
    for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
    return c;
  }
};
template <>
struct Chunk<bf16> {
  typedef bf16x8 type;
  static constexpr int MFMAS = 1;
  __device__ static f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Chunk<f16> {
  typedef f16x8 type;
  static constexpr int MFMAS = 1;
  __device__ static f32x4 mma(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

// what a lane loads past the end of the reduction
__device__ const u32x4 zero_chunk = {0, 0, 0, 0};

__device__ __forceinline__ void load_to_lds(const void* g, void* l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                   (__attribute__((address_space(3))) void*)l, 16, 0, 0);
}

// The activation of VEC values; one branch for all of them.
template <typename T, int VEC>
__device__ __forceinline__ void activate(float* x, int act) {
  if (act == VB_ACT_NONE) return;
  if (act == VB_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = act_value<T>(x[i], VB_ACT_RELU);
  } else if (act == VB_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = act_value<T>(x[i], VB_ACT_GELU);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = act_value<T>(x[i], VB_ACT_SILU);
  }
}

// Bias, residual and activation of VEC consecutive outputs of row m from n on, and
// their 2 VEC- or 4 VEC-byte accesses (VEC > 1: the caller has checked the alignment).
template <typename T, int VEC>
__device__ __forceinline__ void finish(const Product& p, long long m, int n, const float* v) {
  typedef T TV __attribute__((ext_vector_type(VEC)));
  float x[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) x[i] = v[i];
  auto add = [&](const T* q) {
    const TV t = *(const TV*)q;
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] += to_f32((T)t[i]);
  };
  auto put = [&](T* q) {
    TV t;
#pragma unroll
    for (int i = 0; i < VEC; ++i) t[i] = from_f32<T>(x[i]);
    *(TV*)q = t;
  };
  if (p.bias) add((const T*)p.bias + n);
  if (p.res) add((const T*)p.res + m * p.ld_res + n);
  if (p.pre) put((T*)p.pre + m * p.ld_pre + n);
  activate<T, VEC>(x, p.act);
  put((T*)p.out + m * p.ld_out + n);
}

// Tile of a workgroup: workgroups go round the eight XCDs in turn, so each XCD takes
// a contiguous run of tiles, walked in bands of eight tile rows; the 32 tiles that an
// XCD has at a time then share 8 row and 4 column panels through its L2.
__device__ __forceinline__ void tile_of(unsigned bid, int tm, int tn, int& i, int& j) {
  const unsigned total = (unsigned)tm * tn, q = total / 8, r = total % 8, x = bid % 8;
  const unsigned id = x * q + min(x, r) + bid / 8;
  const unsigned band = id / (8u * tn), in = id % (8u * tn);
  const unsigned rows = min(8u, (unsigned)tm - band * 8);
  i = band * 8 + in % rows;
  j = in / rows;
}

// Scheduling of one step: M MFMAs with D LDS reads and (nl of V) loads to LDS between
template <int M, int D, int V>
__device__ __forceinline__ void interleave(int nl) {
#pragma unroll
  for (int i = 0; i < M; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (i < D) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    if (nl && i < V) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
  }
}

template <typename T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, BM == 64 ? 4 : 2) void gemm_kernel(Product p, int tm, int tn) {
  typedef typename Chunk<T>::type C;
  constexpr int NW = WM * WN, LA = BM / 16 / NW, LB = BN / 16 / NW, NS = 4, STAGE = (BM + BN) * 64;
  constexpr int TM = BM / WM, TN = BN / WN, MT = TM / 16, NT = TN / 16, MH = MT / 2;
  __shared__ __align__(16) char lds[NS * STAGE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int ti, tj;
  tile_of(blockIdx.x, tm, tn, ti, tj);
  const long long m0 = (long long)ti * BM;
  const int n0 = tj * BN;
  const int chunks = (int)(p.K * sizeof(T) / 16), stages = (chunks + 3) / 4, full = chunks / 4;
  const char* a = (const char*)p.a + m0 * p.sam * sizeof(T);
  const char* b = (const char*)p.b + (long long)n0 * p.sbn * sizeof(T);
  const int lr = lane >> 2, lc = (lane & 3) ^ (lane >> 4);
  // byte offsets of this lane's chunks in the first stage; rows past the end repeat the last row
  unsigned oa[LA], ob[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i)
    oa[i] = (unsigned)min((long long)((i * NW + wave) * 16 + lr), p.M - 1 - m0) * (unsigned)(p.sam * sizeof(T)) + lc * 16;
#pragma unroll
  for (int i = 0; i < LB; ++i)
    ob[i] = (unsigned)min((i * NW + wave) * 16 + lr, p.N - 1 - n0) * (unsigned)(p.sbn * sizeof(T)) + lc * 16;
  auto issue = [&](int t, int base) {  // a stage that the reduction fills
    const char* at = a + (long long)t * 64;
    const char* bt = b + (long long)t * 64;
    char* l = lds + base + wave * 1024;
#pragma unroll
    for (int i = 0; i < LA; ++i) load_to_lds(at + oa[i], l + i * NW * 1024);
#pragma unroll
    for (int i = 0; i < LB; ++i) load_to_lds(bt + ob[i], l + BM * 64 + i * NW * 1024);
  };
  auto issue_part = [&](int t, int base) {  // any stage: zeros past the end
    const char* at = a + (long long)t * 64;
    const char* bt = b + (long long)t * 64;
    char* l = lds + base + wave * 1024;
    const bool in = t * 4 + lc < chunks;
#pragma unroll
    for (int i = 0; i < LA; ++i) load_to_lds(in ? (const void*)(at + oa[i]) : &zero_chunk, l + i * NW * 1024);
#pragma unroll
    for (int i = 0; i < LB; ++i)
      load_to_lds(in ? (const void*)(bt + ob[i]) : &zero_chunk, l + BM * 64 + i * NW * 1024);
  };
  // The next stage has landed (all but the loads of the NS - 2 stages after it), this
  // wavefront has its reads of the last stage, and so have the others.
  auto join = [] {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NS - 2) * (LA + LB)) : "memory");
  };
  auto join_all = [] { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

  const int wm = wave / WN, wn = wave % WN, r16 = lane & 15, quarter = lane >> 4;
  const int pos = (quarter ^ ((lane >> 2) & 3)) * 16;
  const int ra = (wm * TM + r16) * 64 + pos, rb = (BM + wn * TN + r16) * 64 + pos;
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  C fa[MT], fb[2][NT];
  auto fetch_a = [&](int base, int h) {
#pragma unroll
    for (int i = h * MH; i < h * MH + MH; ++i) fa[i] = *(const C*)(lds + base + ra + i * 1024);
  };
  auto fetch_b = [&](int base, int f) {
#pragma unroll
    for (int j = 0; j < NT; ++j) fb[f][j] = *(const C*)(lds + base + rb + j * 1024);
  };
  auto multiply = [&](int h, int f) {
#pragma unroll
    for (int i = h * MH; i < h * MH + MH; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = Chunk<T>::mma(fa[i], fb[f][j], acc[i][j]);
  };
  auto after = [](int base, int n) {  // the ring position n stages on
    const int x = base + n * STAGE;
    return x >= NS * STAGE ? x - NS * STAGE : x;
  };
  // A stage, its columns in fb[f]: loads() starts the loads of a later stage, wait() is
  // one of the joins.  The reads are spread between the MFMAs; left to itself the
  // compiler sinks them to their uses to save registers.
  auto stage = [&](int cur, int f, auto&& loads, int nl, auto&& wait) {
    __builtin_amdgcn_sched_barrier(0);
    loads();
    fetch_a(cur, 1);
    multiply(0, f);
    interleave<MH * NT * Chunk<T>::MFMAS, MH, LA + LB>(nl);
    __builtin_amdgcn_sched_barrier(0);
    wait();
    __builtin_amdgcn_sched_barrier(0);
    const int nxt = after(cur, 1);
    fetch_b(nxt, f ^ 1);  // after the last stage, of nothing that is used
    fetch_a(nxt, 0);
    multiply(1, f);
    interleave<MH * NT * Chunk<T>::MFMAS, MH + NT, 0>(0);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto none = [] {};
  for (int i = 0; i < NS - 1; ++i)
    if (i < full) issue(i, i * STAGE);
    else if (i < stages) issue_part(i, i * STAGE);
  if (full >= NS - 1) join(); else join_all();
  fetch_b(0, 0);
  fetch_a(0, 0);
  int t = 0, cur = 0;
  for (; t + NS < full; t += 2) {
    stage(cur, 0, [&] { issue(t + NS - 1, after(cur, NS - 1)); }, LA + LB, join);
    cur = after(cur, 1);
    stage(cur, 1, [&] { issue(t + NS, after(cur, NS - 1)); }, LA + LB, join);
    cur = after(cur, 1);
  }
  for (; t < stages; t += 2) {
    if (t + NS - 1 < stages) issue_part(t + NS - 1, after(cur, NS - 1));
    stage(cur, 0, none, 0, join_all);
    cur = after(cur, 1);
    if (t + 1 == stages) break;
    if (t + NS < stages) issue_part(t + NS, after(cur, NS - 1));
    stage(cur, 1, none, 0, join_all);
    cur = after(cur, 1);
  }
  join_all();
  // Outputs leave through LDS, 32 rows of the wavefront's tile at a time in its own
  // part of it, so that a row's outputs are written as whole 128-byte pieces.
  constexpr int LDE = TN + 4, VEC = 16 / sizeof(T), LPR = TN / VEC, RPI = 64 / LPR;
  static_assert(NW * 32 * LDE * 4 <= NS * STAGE, "the output staging fits the operand stages");
  float* e = (float*)lds + wave * 32 * LDE;
  const unsigned long long mis =
      (unsigned long long)p.out | (unsigned long long)p.res | (unsigned long long)p.pre | (unsigned long long)p.bias |
      (unsigned long long)((p.ld_out | p.ld_res | p.ld_pre) * (long long)sizeof(T));
  const bool aligned = (mis & 15) == 0;
#pragma unroll
  for (int i = 0; i < MT; i += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) e[(16 * h + 4 * quarter + q) * LDE + j * 16 + r16] = acc[i + h][j][q];
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const long long mb = m0 + wm * TM + i * 16;
    const int nb = n0 + wn * TN;
    if (aligned && nb + TN <= p.N) {
      const int row = lane / LPR, col = (lane % LPR) * VEC;
#pragma unroll
      for (int r = 0; r < 32; r += RPI)
        if (mb + r + row < p.M) finish<T, VEC>(p, mb + r + row, nb + col, e + (r + row) * LDE + col);
    } else {
      const int cols = min(TN, p.N - nb);
      for (int k = lane; k < 32 * TN; k += 64) {
        const int row = k / TN, col = k % TN;
        if (mb + row < p.M && col < cols) finish<T, 1>(p, mb + row, nb + col, e + row * LDE + col);
      }
    }
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
  }
}

template <typename T, int BM, int BN, int WM, int WN>
hipError_t launch_gemm(const Product& p, hipStream_t st) {
  const long long tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN;
  if (tm * tn > 0x7fffffffLL) return hipErrorInvalidValue;
  gemm_kernel<T, BM, BN, WM, WN><<<dim3((unsigned)(tm * tn)), 64 * WM * WN, 0, st>>>(p, (int)tm, (int)tn);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_gemm_sized(const Product& p, hipStream_t st) {
  auto tiles = [&](int b) { return (p.M + b - 1) / b * ((p.N + b - 1) / b); };
  if (tiles(256) >= 200) return launch_gemm<T, 256, 256, 2, 4>(p, st);
  if (tiles(128) >= 200) return launch_gemm<T, 128, 128, 2, 2>(p, st);
  return launch_gemm<T, 64, 64, 2, 2>(p, st);
}

// rows contiguous along the reduction, 16-byte chunks throughout, 32-bit offsets within a tile's rows
bool chunked(const void* p, long long row, long long el, long long K, int es) {
  return el == 1 && (uintptr_t)p % 16 == 0 && row * es % 16 == 0 && K * es % 16 == 0 && row * es <= (1 << 22);
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
  const int es = (int)elem_size(dtype);
  if (chunked(p.a, p.sam, p.sak, p.K, es) && chunked(p.b, p.sbn, p.sbk, p.K, es)) {
    if (dtype == VB_F32) return launch_gemm_sized<float>(p, st);
    if (dtype == VB_BF16) return launch_gemm_sized<bf16>(p, st);
    return launch_gemm_sized<f16>(p, st);
  }
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
