// The fused linear layer y = act(x W^T + bias + residual), the gated one y = act(gate) * up
// with (gate | up) = x W^T + bias, and the products of their backward passes.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "vb_train_device.h"
#include "vb_train_internal.h"

namespace vb {

namespace {

typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));

// exp and the normal CDF: to float32 accuracy for float32 data.  For 16-bit data the
// hardware exponential, whose argument v log2(e) is rounded (relative error |v| 2^-24, of
// results that are rounded to 2^-9 or 2^-12), and, on its exp(-v^2 / 2) = e, a polynomial in
// t = 1 / (1 + 0.35 |v|) for Phi(-|v|) / e, fitted here to the smallest relative error over
// |v| < 14.5 (2^-20.6; e is 0 beyond), so that the lower tail keeps its bits too.
template <typename T>
__device__ __forceinline__ float exp_of(float v) {
  return sizeof(T) == 4 ? expf(v) : __expf(v);
}
template <typename T>
__device__ __forceinline__ float normal_cdf(float v, float e) {
  if (sizeof(T) == 4) return 0.5f * erfcf(v * -0.70710678118654752f);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.35f, fabsf(v), 1.f));
  float r = 4.8901788890e-2f;
  r = fmaf(r, t, -2.0196606219e-1f);
  r = fmaf(r, t, 2.4040395021e-1f);
  r = fmaf(r, t, -1.6829561442e-2f);
  r = fmaf(r, t, 1.5587112308e-1f);
  r = fmaf(r, t, 1.3337899745e-1f);
  r = fmaf(r, t, 1.4026702940e-1f);
  r = fmaf(r, t, -2.7130148737e-5f);
  return v < 0.f ? e * r : 1.f - e * r;
}

template <typename T>
__device__ __forceinline__ float act_value(float v, int act) {
  if (act == VB_ACT_RELU) return v < 0.f ? 0.f : v;  // NaN stays NaN
  if (act == VB_ACT_GELU) return v * normal_cdf<T>(v, exp_of<T>(-0.5f * v * v));
  if (act == VB_ACT_SILU) return v / (1.f + exp_of<T>(-v));
  return v;
}

// dy * act'(pre) from what the forward pass saved
template <typename T>
__device__ __forceinline__ float act_grad(float dy, float s, int act) {
  if (act == VB_ACT_RELU) return s > 0.f ? dy : 0.f;
  if (act == VB_ACT_GELU) {
    const float e = exp_of<T>(-0.5f * s * s);
    return dy * (normal_cdf<T>(s, e) + s * (0.3989422804014327f * e));
  }
  if (act == VB_ACT_SILU) {
    const float q = 1.f / (1.f + exp_of<T>(-s));
    return dy * (q * (1.f + s * (1.f - q)));
  }
  return dy;
}

// ---------------------------------------------------------------------------
// The large product C(m, n) = sum_k A(m, k) B(n, k).  An operand is stored with the
// reduction along its rows (x and W in the forward pass) or across them (W for dx; g
// and x for dweight); rows start on 16-byte boundaries.
//
// Workgroups of WM x WN wavefronts compute BM x BN tiles.  Both operands pass through
// a ring of NS stages in LDS, each 128 or 64 bytes of the reduction deep, loaded straight
// from global memory.  NS - 1 stages are in flight at a time: all workgroups of an XCD
// reach new memory together, so a stage's first touch waits for HBM.
// A wavefront's tile is MT x NT blocks of 16 x 16 outputs (v_mfma 16x16x32: at this
// size the card is limited by power, and on the same random operands, from registers,
// the 16-wide instructions ran at 1.63 GHz against 1.52 GHz for 32x32x16).  A stage is
// worked off in steps of 64 bytes (32 16-bit or 16 float32 numbers), a step in two phases:
// the products of the upper half of the rows, under which the lower half is read from
// LDS; after a stage's last step the barrier; then the products of the lower half, under
// which the next step's upper half and columns are read.  No wavefront waits on the
// barrier or on LDS with idle matrix cores.
//
// What bounds it: in 16 bits the card's power (8192 x 8192 -> 8192 in bf16 0.97 ms, 1.13
// PFLOP/s at about 1.4 GHz; the library's product 0.84 ms), in float32 the matrix cores
// (8192 x 8192 -> 4096 3.78 ms, 145 TFLOP/s; the library's 3.60 ms).  Gated, 4096 x 4096 -> 2 x 8192
// in bf16: 432 us, 1.27 PFLOP/s, 462 with both projections written out (the library's product
// alone 388); gate and up as columns of one tile cost nothing that the same product as a
// linear layer does not, and its outputs are half as many.
//
// The MFMA wants, per lane, chunk q = lane / 16 (16 bytes along the reduction) of row
// lane % 16.
//  - Reduction along the rows: a stage holds its depth of each row, and a lane reads its
//    chunk.  Chunk c of row r lies at position c ^ ((r >> 1) & 7) (64 bytes deep: c ^ ((r >>
//    2) & 3)): the 16 rows that a quarter of a wavefront reads together (256 bytes a clock)
//    then fall on different LDS banks; measured 4.1 clocks a 1 KB read, against 16 for a
//    position c ^ (r & 3).
//  - Reduction across the rows: a stage holds depth / element size rows of BM (BN)
//    elements.  16-bit operands are turned by the transposing LDS read (a group of 16
//    lanes reads four rows of 16 elements, lane i receives column i); float32 ones are
//    read element by element.  The rows of such a read lie at one bank offset, so
//    blocks of 16 columns are permuted within a row by row_swizzle.
// A direct load writes 64 consecutive chunks of LDS, so either permutation is done on
// the global side, within pieces of the depth (along) or whole rows (across).
// Float32 uses the same bytes: MFMA step s of a chunk takes element s of it for both
// operands, which permutes the reduction alike on both sides.

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes of a row; mma: MFMA s of the MFMAS that multiply a wavefront's 64 chunks (16
// rows x 4) of each operand.  The MFMAs of one block of outputs wait for each other, so
// other blocks come between (float32, one after the other: 75 % of the rate).
template <typename T>
struct Chunk;
template <>
struct Chunk<float> {
  typedef f32x4 type;
  static constexpr int MFMAS = 4, BITS = 24;
  __device__ static f32x4 mma(f32x4 a, f32x4 b, f32x4 c, int s) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
  }
};
template <>
struct Chunk<bf16> {
  typedef bf16x8 type;
  static constexpr int BITS = 8;  // of a number's significand
  static constexpr int MFMAS = 1;
  __device__ static f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c, int) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Chunk<f16> {
  typedef f16x8 type;
  static constexpr int BITS = 11;
  static constexpr int MFMAS = 1;
  __device__ static f32x4 mma(f16x8 a, f16x8 b, f32x4 c, int) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

// what a lane loads past the end of the reduction
__device__ const u32x4 zero_chunk = {0, 0, 0, 0};

// 16 bytes per lane from global memory to LDS, lane after lane from l on (uniform).  In
// assembly, since the compiler, which cannot tell the stages of the ring apart, would
// wait for every such load before the next transposing read; nothing is returned in
// registers, and the kernels wait for the loads themselves (join).  The instruction
// takes the LDS address from M0, a wait state after it is written; M0 is a reserved
// register, which the compiler keeps nothing in for these kernels (they index no
// registers and use no other instruction that reads it).
__device__ __forceinline__ unsigned lds_address(const void* l) {
  return __builtin_amdgcn_readfirstlane((unsigned)(unsigned long long)(__attribute__((address_space(3))) const void*)l);
}
__device__ __forceinline__ void load_to_lds(const void* base, unsigned off, unsigned l) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(l), "v"(off), "s"(base));
}
__device__ __forceinline__ void load_to_lds(const void* g, unsigned l) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(l), "v"(g));
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

// Bias, residual and activation of VEC consecutive outputs of row m from n on, in one
// access each; 16-byte accesses at element alignment are ordinary ones here, which cost
// extra only where a line is crossed (output rows 3996 wide one element at a time: 147
// us for 4096 x 4096 -> 3996 in bf16, and 111 us for 4096 outputs).
template <typename T, int VEC>
__device__ __forceinline__ void finish(const Product& p, long long m, int n, const float* v) {
  typedef T TV __attribute__((ext_vector_type(VEC)));
  typedef TV LV __attribute__((aligned(sizeof(T))));
  float x[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) x[i] = v[i];
  auto add = [&](const T* q) {
    const TV t = *(const LV*)q;
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] += to_f32((T)t[i]);
  };
  auto put = [&](T* q) {
    TV t;
#pragma unroll
    for (int i = 0; i < VEC; ++i) t[i] = from_f32<T>(x[i]);
    *(LV*)q = t;
  };
  if (p.bias) add((const T*)p.bias + n);
  if (p.res) add((const T*)p.res + m * p.ld_res + n);
  if (p.pre) put((T*)p.pre + m * p.ld_pre + n);
  activate<T, VEC>(x, p.act);
  put((T*)p.out + m * p.ld_out + n);
}

// The same for the gated layer: VEC outputs of row m from n on, from their gates and ups.
template <typename T, int VEC>
__device__ __forceinline__ void finish_gated(const Product& p, long long m, int n, const float* gate, const float* up) {
  typedef T TV __attribute__((ext_vector_type(VEC)));
  typedef TV LV __attribute__((aligned(sizeof(T))));
  float g[VEC], u[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) g[i] = gate[i], u[i] = up[i];
  auto add = [&](const T* q, float* x) {
    const TV t = *(const LV*)q;
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] += to_f32((T)t[i]);
  };
  auto put = [&](T* q, const float* x) {
    TV t;
#pragma unroll
    for (int i = 0; i < VEC; ++i) t[i] = from_f32<T>(x[i]);
    *(LV*)q = t;
  };
  if (p.bias) add((const T*)p.bias + n, g), add((const T*)p.bias + p.N + n, u);
  if (p.pre) put((T*)p.pre + m * p.ld_pre + n, g), put((T*)p.pre + m * p.ld_pre + p.N + n, u);
  activate<T, VEC>(g, p.act);
#pragma unroll
  for (int i = 0; i < VEC; ++i) g[i] *= u[i];
  put((T*)p.out + m * p.ld_out + n, g);
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

// Scheduling of one phase: D LDS reads between M MFMAs
template <int M, int D>
__device__ __forceinline__ void interleave() {
  constexpr int PER = (D + M - 1) / M;
#pragma unroll
  for (int i = 0; i < M; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (i * PER < D) __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);
  }
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

// One operand of a workgroup's tile: ROWS of its rows (ACROSS: columns), its loads into
// a stage and its reads from one.
template <typename T, int ROWS, int NW, bool ACROSS, int DEPTH>
struct Operand {
  typedef typename Chunk<T>::type C;
  static constexpr int ES = sizeof(T), L = ROWS * DEPTH / 1024 / NW;
  static constexpr int STEP_ROWS = 64 / ES;       // rows of a 64-byte step when ACROSS
  static constexpr int RPL = 1024 / DEPTH;        // rows of a load otherwise
  static constexpr int RB = ROWS * ES;            // bytes of a stage's row when ACROSS
  static constexpr int PER_BLOCK = ES;            // chunks of a block of 16 elements
  static constexpr int READS = ACROSS ? (ES == 4 ? 4 : 2) : 1;  // LDS reads of a fetch
  const char* base;   // first stage
  long long step;     // bytes from stage to stage
  unsigned off[L];    // this lane's chunks in the first stage
  int lane, wave;

  // what a row k of a stage is permuted by (ACROSS), in blocks of 16 elements: the rows
  // read together (quarter 4 q .. in float32; 8 q + 0..3 for two q in 16 bits) differ,
  // over the 256 bytes that LDS serves at once
  __device__ static int row_swizzle(int k) {
    if (ES == 4) return (k >> 2) & 3;
    if (ROWS >= 128) return (k & 3) | ((k >> 3) & 1) << 2;
    return ((k >> 1) & 1) | ((k >> 3) & 1) << 1;
  }
  // row (of the stage) and chunk that lane's i-th load brings when ACROSS
  __device__ int row_of(int i) const { return ((i * NW + wave) * 1024 + lane * 16) / RB; }
  __device__ int chunk_of(int i) const {
    const int at = ((i * NW + wave) * 1024 + lane * 16) % RB / 16;
    return ((at / PER_BLOCK) ^ row_swizzle(row_of(i))) * PER_BLOCK + at % PER_BLOCK;
  }
  // position of chunk c of row r otherwise: rows of a quarter wavefront on different banks
  __device__ static int along_swizzle(int r) { return DEPTH == 64 ? (r >> 2) & 3 : (r >> 1) & 7; }
  __device__ int chunk_along() const {  // the rows of all of a wavefront's loads are alike to the swizzle
    return (lane % (DEPTH / 16)) ^ along_swizzle(wave * RPL + lane / (DEPTH / 16));
  }

  // rows (ACROSS: columns) from r0 on of `count`; past the end the last one is repeated
  __device__ void init(const void* p, long long ld, long long r0, long long count, int first_stage, int w, int l) {
    lane = l, wave = w;
    if (ACROSS) {
      step = ld * DEPTH;  // DEPTH / ES rows of ld * ES bytes
      base = (const char*)p + r0 * ES + first_stage * step;
      const int last = (int)min(((count - r0) * ES + 15) / 16 - 1, (long long)(RB / 16 - 1));
#pragma unroll
      for (int i = 0; i < L; ++i) off[i] = (unsigned)row_of(i) * (unsigned)(ld * ES) + min(chunk_of(i), last) * 16;
    } else {
      step = DEPTH;
      base = (const char*)p + r0 * ld * ES + first_stage * step;
#pragma unroll
      for (int i = 0; i < L; ++i)
        off[i] = (unsigned)min((long long)((i * NW + wave) * RPL + lane / (DEPTH / 16)), count - 1 - r0) *
                     (unsigned)(ld * ES) +
                 chunk_along() * 16;
    }
  }
  // a stage that the reduction fills
  __device__ void load(int t, unsigned lds) const {
    const char* at = base + t * step;
#pragma unroll
    for (int i = 0; i < L; ++i) load_to_lds(at, off[i], lds + (i * NW + wave) * 1024);
  }
  // any stage: zeros past the end of the reduction's K elements
  __device__ void load_part(int t, unsigned lds, int K) const {
    const char* at = base + t * step;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const bool in = ACROSS ? t * (DEPTH / ES) + row_of(i) < K : (t * (DEPTH / 16) + chunk_along()) * (16 / ES) < K;
      load_to_lds(in ? (const void*)(at + off[i]) : &zero_chunk, lds + (i * NW + wave) * 1024);
    }
  }
  // where a lane reads: block b of 16 rows (columns) in the first step of a stage
  __device__ int place(int b) const {
    const int r16 = lane & 15, quarter = lane >> 4;
    if (!ACROSS) return (b * 16 + r16) * DEPTH + (quarter ^ along_swizzle(r16)) * 16;
    if (ES == 4) return quarter * 4 * RB + (b ^ quarter) * 64 + r16 * 4;
    const int k = quarter * 8 + (r16 >> 2);
    return k * RB + (b ^ row_swizzle(k)) * 32 + (r16 & 3) * 8;
  }
  // from there, in step u (0 or, with a depth of 128, 1)
  __device__ static C fetch(const char* lds, int at, int u) {
    const char* p = lds + (ACROSS ? at + u * STEP_ROWS * RB : u ? at ^ 64 : at);
    if constexpr (!ACROSS) {
      return *(const C*)p;
    } else if constexpr (ES == 4) {
      return C{*(const float*)p, *(const float*)(p + RB), *(const float*)(p + 2 * RB), *(const float*)(p + 3 * RB)};
    } else {
      typedef __attribute__((address_space(3))) s16x4* lds4;
      union {
        s16x4 h[2];
        C c;
      } u;
      u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)p);
      u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 4 * RB));
      return u.c;
    }
  }
};

// Stages of 128 bytes (whole lines of an operand along: 192 us against 210 with 64 at
// 4096 x 8192 -> 4096, bf16), three of them, or two for the largest tiles; those have four
// of 64 bytes when both operands lie across, whose loads are whole lines anyway.
template <int BM, int BN, bool XA, bool XB>
struct Ring {
  static constexpr bool LARGE = BM == 256 && BN == 256;
  static constexpr int DEPTH = LARGE && XA && XB ? 64 : 128, NS = !LARGE ? 3 : DEPTH == 128 ? 2 : 4;
  static constexpr int BYTES = NS * (BM + BN) * DEPTH;
};

// Workgroup number `block` of those that the tiles take, part `split` of the reduction.  TWO: A
// in two parts (an instance of its own: its registers and branches would cost the others 4 %).
// GATED: B's stage holds BN / 2 of the gate's rows, then the same ones of up, and a wavefront's
// column blocks are gate and up in turn, so that its tile has both of TN / 2 outputs.
template <typename T, int BM, int BN, int WM, int WN, bool XA, bool XB, bool TWO, bool GATED = false>
__device__ __forceinline__ void gemm_tile(Product p, int tm, int tn, unsigned block, unsigned split, char* lds) {
  typedef typename Chunk<T>::type C;
  constexpr int DEPTH = Ring<BM, BN, XA, XB>::DEPTH, NS = Ring<BM, BN, XA, XB>::NS;
  constexpr int NW = WM * WN, STAGE = (BM + BN) * DEPTH, KS = DEPTH / sizeof(T);
  constexpr int TM = BM / WM, TN = BN / WN, MT = TM / 16, NT = TN / 16, MH = MT / 2;
  typedef Operand<T, BM, NW, XA, DEPTH> OA;
  constexpr int BO = GATED ? BN / 2 : BN, TO = GATED ? TN / 2 : TN;  // outputs of a tile's, a wavefront's row
  static_assert(!GATED || (!XA && !XB && !TWO && NT % 2 == 0), "gated: the forward product");
  typedef Operand<T, BO, NW, XB, DEPTH> OB;
  constexpr int LA = OA::L, LB = OB::L * (GATED ? 2 : 1), RA = OA::READS, RB = OB::READS;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int ti, tj;
  tile_of(block, tm, tn, ti, tj);
  const long long m0 = (long long)ti * BM;
  const int n0 = tj * BO;
  // this workgroup's part of the reduction
  const int first = split * (p.split_steps / (DEPTH / 64));
  const int K = (int)min(p.K - (long long)first * KS, (long long)p.split_steps * (64 / (int)sizeof(T)));
  const int stages = (K + KS - 1) / KS, full = K / KS;
  OA a;
  OB b;
  a.init(p.a, p.lda, m0, p.M, first, wave, lane);
  b.init(p.b, p.ldb, n0, p.N, first, wave, lane);
  // up's rows lie as the gate's do
  OB up = b;
  if constexpr (GATED) up.base += p.N * p.ldb * (long long)sizeof(T);
  const unsigned lds0 = lds_address(lds);
  auto issue = [&](int t, int base) {
    a.load(t, lds0 + base), b.load(t, lds0 + base + BM * DEPTH);
    if constexpr (GATED) up.load(t, lds0 + base + (BM + BO) * DEPTH);
  };
  auto issue_part = [&](int t, int base) {
    a.load_part(t, lds0 + base, K), b.load_part(t, lds0 + base + BM * DEPTH, K);
    if constexpr (GATED) up.load_part(t, lds0 + base + (BM + BO) * DEPTH, K);
  };
  // The next stage has landed (all but the loads of the NS - 2 stages after it), this
  // wavefront has its reads of the last stage, and so have the others.
  auto join = [] {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NS - 2) * (LA + LB)) : "memory");
  };
  auto join_all = [] { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

  const int wm = wave / WN, wn = wave % WN, r16 = lane & 15, quarter = lane >> 4;
  int pa[MT], pb[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) pa[i] = a.place(wm * MT + i);
#pragma unroll
  for (int j = 0; j < NT; ++j)
    pb[j] = GATED ? (BM + j % 2 * BO) * DEPTH + b.place((wn * NT + j) / 2) : BM * DEPTH + b.place(wn * NT + j);
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  C fa[MT], fb[2][NT];
  auto fetch_a = [&](int base, int u, int h) {
#pragma unroll
    for (int i = h * MH; i < h * MH + MH; ++i) fa[i] = OA::fetch(lds + base, pa[i], u);
  };
  auto fetch_b = [&](int base, int u, int f) {
#pragma unroll
    for (int j = 0; j < NT; ++j) fb[f][j] = OB::fetch(lds + base, pb[j], u);
  };
  auto multiply = [&](int h, int f) {
#pragma unroll
    for (int s = 0; s < Chunk<T>::MFMAS; ++s)
#pragma unroll
      for (int i = h * MH; i < h * MH + MH; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = Chunk<T>::mma(fa[i], fb[f][j], acc[i][j], s);
  };
  auto after = [](int base, int n) {  // the ring position n stages on
    const int x = base + n * STAGE;
    return x >= NS * STAGE ? x - NS * STAGE : x;
  };
  // A step of 64 bytes (u of its stage), its columns in fb[f]: loads() starts the loads of
  // a later stage, wait() is one of the joins after the last step of a stage.  The reads
  // are spread between the MFMAs; left to itself the compiler sinks them to their uses to
  // save registers.
  auto step = [&](int cur, int u, int f, auto&& loads, auto&& wait) {
    __builtin_amdgcn_sched_barrier(0);
    loads();
    fetch_a(cur, u, 1);
    multiply(0, f);
    interleave<MH * NT * Chunk<T>::MFMAS, MH * RA>();
    __builtin_amdgcn_sched_barrier(0);
    const bool last = u == DEPTH / 64 - 1;
    if (last) wait();
    __builtin_amdgcn_sched_barrier(0);
    const int nxt = last ? after(cur, 1) : cur;
    fetch_b(nxt, last ? 0 : u + 1, f ^ 1);  // after the last stage, of nothing that is used
    fetch_a(nxt, last ? 0 : u + 1, 0);
    multiply(1, f);
    interleave<MH * NT * Chunk<T>::MFMAS, MH * RA + NT * RB>();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto none = [] {};
  // A in two parts: the low parts' products first, scaled down, then the high ones' on top
  // of them (one after the other: accumulators for both would not fit the registers).  A low
  // sum that is not finite met an infinity or NaN of B; the high parts alone have the sign.
  const long long low = TWO ? (const char*)p.a_low - (const char*)p.a : 0;
  auto each = [&](auto&& f) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = f(acc[i][j][q]);
  };
  a.base += low;
  for (int pass = 0;; ++pass) {
    if constexpr (TWO) {
      // nothing computed from these is carried round the loop (it would be 40 registers)
#pragma unroll
      for (int i = 0; i < MT; ++i) asm volatile("" : "+v"(pa[i]));
#pragma unroll
      for (int j = 0; j < NT; ++j) asm volatile("" : "+v"(pb[j]));
#pragma unroll
      for (int i = 0; i < LA; ++i) asm volatile("" : "+v"(a.off[i]));
#pragma unroll
      for (int i = 0; i < LB; ++i) asm volatile("" : "+v"(b.off[i]));
      asm volatile("" : "+v"(a.lane), "+v"(b.lane));
    }
    for (int i = 0; i < NS - 1; ++i)
      if (i < full) issue(i, i * STAGE);
      else if (i < stages) issue_part(i, i * STAGE);
    if (full >= NS - 1) join(); else join_all();
    fetch_b(0, 0, 0);
    fetch_a(0, 0, 0);
    int t = 0, cur = 0;
    if constexpr (DEPTH == 128) {
      for (; t + NS - 1 < full; ++t) {
        step(cur, 0, 0, [&] { issue(t + NS - 1, after(cur, NS - 1)); }, none);
        step(cur, 1, 1, none, join);
        cur = after(cur, 1);
      }
      for (; t < stages; ++t) {
        if (t + NS - 1 < stages) issue_part(t + NS - 1, after(cur, NS - 1));
        step(cur, 0, 0, none, none);
        step(cur, 1, 1, none, join_all);
        cur = after(cur, 1);
      }
    } else {
      for (; t + NS < full; t += 2) {
        step(cur, 0, 0, [&] { issue(t + NS - 1, after(cur, NS - 1)); }, join);
        cur = after(cur, 1);
        step(cur, 0, 1, [&] { issue(t + NS, after(cur, NS - 1)); }, join);
        cur = after(cur, 1);
      }
      for (; t < stages; t += 2) {
        if (t + NS - 1 < stages) issue_part(t + NS - 1, after(cur, NS - 1));
        step(cur, 0, 0, none, join_all);
        cur = after(cur, 1);
        if (t + 1 == stages) break;
        if (t + NS < stages) issue_part(t + NS, after(cur, NS - 1));
        step(cur, 0, 1, none, join_all);
        cur = after(cur, 1);
      }
    }
    join_all();
    if (!TWO || pass == 1) break;
    a.base -= low;
    each([](float v) { return fabsf(v) < INFINITY ? v * (1.f / (1 << Chunk<T>::BITS)) : 0.f; });
  }
  if (TWO) each([](float v) { return 2.f * v; });
  // Outputs leave through LDS, 32 rows of the wavefront's tile at a time in its own
  // part of it, so that a row's outputs are written as whole 128-byte pieces.
  // GATED: the gates in the first half of a row, then the ups.
  constexpr int LDE = TN + 4, VEC = 16 / sizeof(T), LPR = TO / VEC, RPI = 64 / LPR;
  static_assert(NW * 32 * LDE * 4 <= NS * STAGE, "the output staging fits the operand stages");
  float* e = (float*)lds + wave * 32 * LDE;
#pragma unroll
  for (int i = 0; i < MT; i += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) e[(16 * h + 4 * quarter + q) * LDE + (GATED ? j % 2 * TO + j / 2 * 16 : j * 16) + r16] = acc[i + h][j][q];
    __builtin_amdgcn_wave_barrier();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const long long mb = m0 + wm * TM + i * 16;
    const int nb = n0 + wn * TO;
    if (p.partial) {
      // float32 sums of this part, rows of N rounded up to four (GATED: the gates', then the ups')
      float* part = p.partial + (split * p.M + mb) * (long long)p.ld_partial + nb;
      const int row = lane / (TN / 4), col = lane % (TN / 4) * 4, of = col % TO, to = col == of ? of : of + p.ld_partial / 2;
#pragma unroll
      for (int r = 0; r < 32; r += 256 / TN)
        if (mb + r + row < p.M && nb + of < p.N)
          *(f32x4*)(part + (r + row) * (long long)p.ld_partial + to) = *(const f32x4*)(e + (r + row) * LDE + col);
    } else {
      const int row = lane / LPR, col = (lane % LPR) * VEC;
#pragma unroll
      for (int r = 0; r < 32; r += RPI) {
        const float* v = e + (r + row) * LDE + col;
        if (mb + r + row < p.M && nb + col < p.N) {
          if constexpr (GATED) {
            if (nb + col + VEC <= p.N) {
              finish_gated<T, VEC>(p, mb + r + row, nb + col, v, v + TO);
            } else {
              for (int k = 0; nb + col + k < p.N; ++k) finish_gated<T, 1>(p, mb + r + row, nb + col + k, v + k, v + TO + k);
            }
          } else if (nb + col + VEC <= p.N) {
            finish<T, VEC>(p, mb + r + row, nb + col, v);
          } else {
            for (int k = 0; nb + col + k < p.N; ++k) finish<T, 1>(p, mb + r + row, nb + col + k, v + k);
          }
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
  }
}

template <typename T, int BM, int BN, int WM, int WN, bool XA, bool XB, bool TWO, bool GATED = false>
__global__ __launch_bounds__(64 * WM * WN, BN == 64 ? 3 : 2) void gemm_kernel(Product p, int tm, int tn) {
  __shared__ __align__(16) char lds[Ring<BM, BN, XA, XB>::BYTES];
  const unsigned block = workgroup_number();
  if (block >= (unsigned)tm * tn) return;  // the whole workgroup
  gemm_tile<T, BM, BN, WM, WN, XA, XB, TWO, GATED>(p, tm, tn, block, blockIdx.y, lds);
}

// dbias from the sums of act_grad_kernel's workgroups: 64 columns per workgroup, in 16 sums
// of every 16th part whatever the number of wavefronts, eight loads at a time (650 parts:
// 10.5 us one at a time)
template <typename T, int NW>
__device__ __forceinline__ void sum_columns(const ColumnSums& s, unsigned block, float* red) {
  constexpr int U = NW / 2;
  const int c = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int col = block * 64 + c;
  float v[16 / NW];
#pragma unroll
  for (int k = 0; k < 16 / NW; ++k) v[k] = 0.f;
  if (col < s.n) {
    int i = w;
    for (; i + 16 * U <= s.parts; i += 16 * U) {
      float x[U][16 / NW];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < 16 / NW; ++k) x[u][k] = s.partial[(long long)(i + 16 * u + k * NW) * s.n + col];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < 16 / NW; ++k) v[k] += x[u][k];
    }
    for (; i < s.parts; i += 16)
#pragma unroll
      for (int k = 0; k < 16 / NW; ++k)
        if (i + k * NW < s.parts) v[k] += s.partial[(long long)(i + k * NW) * s.n + col];
  }
#pragma unroll
  for (int k = 0; k < 16 / NW; ++k) red[(w + k * NW) * 64 + c] = v[k];
  __syncthreads();
  if (w == 0 && col < s.n) {
    float sum = red[c];
#pragma unroll
    for (int k = 1; k < 16; ++k) sum += red[k * 64 + c];
    ((T*)s.out)[col] = from_f32<T>(sum);
  }
}

template <typename T>
__global__ __launch_bounds__(1024) void column_sum_kernel(ColumnSums s) {
  __shared__ float red[1024];
  sum_columns<T, 16>(s, blockIdx.x, red);
}

// Both products of a backward pass, and dbias, by one launch: the sums' workgroups, then
// the tiles of the product that takes longer for one, then the other's; of a product whose
// reduction is split, the tiles of its first part, of its second, ...
template <typename T, int BM, int BN, int WM, int WN, bool TWO>
__global__ __launch_bounds__(64 * WM * WN, BN == 64 ? 3 : 2) void pair_kernel(Product dx, Product dw, ColumnSums s, int tn,
                                                                              int splits_x, int splits_w, bool dx_first) {
  __shared__ __align__(16) char lds[Ring<BM, BN, false, true>::BYTES];
  static_assert(Ring<BM, BN, false, true>::BYTES == Ring<BM, BN, true, true>::BYTES, "one ring for both");
  unsigned block = workgroup_number();
  const unsigned sums = s.out ? (s.n + 63) / 64 : 0;
  if (block < sums) {
    sum_columns<T, WM * WN>(s, block, (float*)lds);
    return;
  }
  block -= sums;
  const int tx = (int)((dx.M + BM - 1) / BM), tw = (int)((dw.M + BM - 1) / BM);
  const unsigned nx = (unsigned)tx * tn * splits_x, nw = (unsigned)tw * tn * splits_w;
  if (block >= nx + nw) return;  // the whole workgroup
  const unsigned first = dx_first ? nx : nw;
  const bool second = block >= first;
  if (second) block -= first;
  if (second != dx_first) {
    const unsigned tiles = (unsigned)tx * tn, split = splits_x > 1 ? block / tiles : 0;
    gemm_tile<T, BM, BN, WM, WN, false, true, TWO>(dx, tx, tn, block - split * tiles, split, lds);
  } else {
    const unsigned tiles = (unsigned)tw * tn, split = splits_w > 1 ? block / tiles : 0;
    gemm_tile<T, BM, BN, WM, WN, true, true, TWO>(dw, tw, tn, block - split * tiles, split, lds);
  }
}

// ---------------------------------------------------------------------------
// Few rows: the weights are read once and their reading is the time.  Rows may
// start anywhere; 16-byte loads at element alignment are ordinary loads here, which
// cost extra only where a line is crossed.

template <typename T>
struct Loose;  // 16 bytes of consecutive elements at element alignment
template <>
struct Loose<float> {
  typedef f32x4 type __attribute__((aligned(4)));
};
template <>
struct Loose<bf16> {
  typedef bf16x8 type __attribute__((aligned(2)));
};
template <>
struct Loose<f16> {
  typedef f16x8 type __attribute__((aligned(2)));
};

template <typename T>
__device__ __forceinline__ typename Chunk<T>::type load_loose(const T* p) {
  return *(const typename Loose<T>::type*)p;
}

// Up to four rows: R weight rows per workgroup, whose four wavefronts take the chunks
// of the reduction in turn (1 KB of a row per load, R loads and a chunk of each x row,
// which stay in the L1 cache, per step); float32 multiply-adds on the vector units.  1 x
// 4096 -> 16384 in bf16: 23.3 us, 134 MB at 5.8 TB/s, what reading them takes.
// GATED: half of the weight rows are the gate's, half the same ones of up.
template <typename T, int MR, int R, bool GATED>
__global__ __launch_bounds__(256) void rows_kernel(Product p) {
  typedef typename Chunk<T>::type C;
  constexpr int EC = 16 / sizeof(T);
  __shared__ float red[4][R * MR];
  constexpr int RO = GATED ? R / 2 : R;  // outputs
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * RO, chunks = (int)(p.K / EC), tail = (int)(p.K % EC);
  const T* w[R];
  const T* x[MR];
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = (const T*)p.b + (long long)(min(n0 + r % RO, p.N - 1) + r / RO * p.N) * p.ldb;
#pragma unroll
  for (int m = 0; m < MR; ++m) x[m] = (const T*)p.a + min((long long)m, p.M - 1) * p.lda;
  float acc[R][MR];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MR; ++m) acc[r][m] = 0.f;
#pragma unroll 2
  for (int c = threadIdx.x; c < chunks; c += 256) {
    C wv[R], xv[MR];
#pragma unroll
    for (int r = 0; r < R; ++r) wv[r] = load_loose(w[r] + (long long)c * EC);
#pragma unroll
    for (int m = 0; m < MR; ++m) xv[m] = load_loose(x[m] + (long long)c * EC);
#pragma unroll
    for (int e = 0; e < EC; ++e)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int m = 0; m < MR; ++m) acc[r][m] = fmaf(to_f32((T)wv[r][e]), to_f32((T)xv[m][e]), acc[r][m]);
  }
  if ((int)threadIdx.x < tail) {
    const long long k = (long long)chunks * EC + threadIdx.x;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int m = 0; m < MR; ++m) acc[r][m] = fmaf(to_f32(w[r][k]), to_f32(x[m][k]), acc[r][m]);
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MR; ++m) {
      const float s = wave_sum(acc[r][m]);
      if (lane == 0) red[wave][m * R + r] = s;
    }
  __syncthreads();
  const int t = threadIdx.x, m = t / RO, n = n0 + t % RO;
  if (t < RO * MR && m < p.M && n < p.N) {
    auto sum = [&](int i) { return (red[0][i] + red[1][i]) + (red[2][i] + red[3][i]); };
    if constexpr (GATED) {
      const float gate = sum(m * R + t % RO), up = sum(m * R + RO + t % RO);
      finish_gated<T, 1>(p, m, n, &gate, &up);
    } else {
      const float v = sum(t);
      finish<T, 1>(p, m, n, &v);
    }
  }
}

// Up to 16 MB rows: 16 NB weight rows per workgroup along the MFMA rows, the x rows along
// its columns; the NW wavefronts take runs of 128 bytes of the reduction in turn (two
// MFMA steps) and their sums meet in LDS.  Many wavefronts on 16 weight rows where those
// are needed to fill the card, else four on 64, which read x a quarter as often; a
// workgroup's first run is its number's, as workgroups that went through the reduction
// in step would read the same memory channels (32 weight rows: 38 against 28.5 us).
// Measured at 16 x 4096 -> 16384 | 16 x 4096 -> 4096, bf16: 35.5 | 12.8 us and 26.4 | 22.1
// us (float32 75 | 22.8 and 50 | 41); longer runs and other numbers lie between.
// Weight rows are read in chunks that lie on 16-byte boundaries of memory, wherever the
// rows start: rows `period` apart (1, 2, 4 or 8) start at one distance `lead` from a
// boundary, a workgroup takes rows of one distance, and its x chunks start as much
// earlier.  (7 x 5001 -> 3999 in float16: 20.6 us with weight chunks from the rows' starts,
// which cross a line every other time, 13.5 so.)
// GATED: half of the weight rows are the gate's, half the same ones of up, which may lie at
// another distance from a boundary.  Each half has blocks and x chunks of its own (the same
// chunks where the distances are), or, in a workgroup of one block, half the block and up's
// chunks off boundaries.  (7 x 5001 -> 3999 in float16: 33 us in blocks of both, 26 in blocks of
// their own; 16 x 1024 -> 1024 in float32, where workgroups are few: 6.4 and 8.7.)
template <typename T, int MB, int NB, int NW, bool GATED>
__global__ __launch_bounds__(64 * NW) void narrow_kernel(Product p, int period) {
  typedef typename Chunk<T>::type C;
  constexpr int EC = 16 / sizeof(T), H = GATED && NB > 1 ? 2 : 1, HB = NB / H, U = H == 2 ? 4 : 2, OUT = MB * NB * 256;
  __shared__ __align__(16) float red[NW][OUT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, quarter = lane >> 4;
  constexpr int RO = GATED ? 8 * NB : 16 * NB;  // outputs
  const int like = blockIdx.x % period, n0 = blockIdx.x / period * RO * period + like;
  if (like >= p.N) return;  // the whole workgroup
  const int last = p.N - 1 - (p.N - 1 - like) % period;
  const T* w[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int row = 16 * b + r16;
    w[b] = (const T*)p.b + (long long)(min(n0 + row % RO * period, last) + row / RO * p.N) * p.ldb;
  }
  const T* x[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) x[m] = (const T*)p.a + min((long long)(16 * m + r16), p.M - 1) * p.lda;
  f32x4 acc[NB][MB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[b][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const C* wv, const C (*xv)[MB]) {
#pragma unroll
    for (int q = 0; q < Chunk<T>::MFMAS; ++q)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[b][m] = Chunk<T>::mma(wv[b], xv[b / HB][m], acc[b][m], q);
  };
  // whole chunks first .. end - 1 (chunk c holds elements c EC - lead on), of which runs
  int lead[H], first[H], runs = 0x7fffffff;
  const int K = (int)p.K;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    lead[h] = __builtin_amdgcn_readfirstlane((int)((uintptr_t)w[h * HB] % 16 / sizeof(T)));
    first[h] = lead[h] > 0;
    runs = min(runs, max((lead[h] + K) / EC - first[h], 0) / (4 * U));
  }
  const bool alike = lead[0] == lead[H - 1];
  const int turn = runs ? (int)(blockIdx.x % (unsigned)runs) : 0;
  for (int s = wave; s < runs; s += NW) {
    const int run = s + turn < runs ? s + turn : s + turn - runs;
    C wv[U][NB], xv[U][H][MB];
    long long k0[H];
#pragma unroll
    for (int h = 0; h < H; ++h) k0[h] = (long long)(first[h] + run * (4 * U) + quarter) * EC - lead[h];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int u = 0; u < U; ++u)
        wv[u][b] = GATED && H == 1 ? load_loose(w[b] + k0[0] + u * 4 * EC) : *(const C*)(w[b] + k0[b / HB] + u * 4 * EC);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < MB; ++m) xv[u][0][m] = load_loose(x[m] + k0[0] + u * 4 * EC);
    if constexpr (H == 2) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int m = 0; m < MB; ++m) xv[u][1][m] = xv[u][0][m];
      if (!alike) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int m = 0; m < MB; ++m) xv[u][1][m] = load_loose(x[m] + k0[1] + u * 4 * EC);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(wv[u], xv[u]);
  }
  // the chunks left over and those that the row fills in part (the first one comes last),
  // zeros elsewhere, a step of four per wavefront
  int rest[H], total[H], most = 0;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    rest[h] = first[h] + runs * 4 * U, total[h] = (lead[h] + K + EC - 1) / EC - rest[h] + first[h];
    most = max(most, total[h]);
  }
  auto part = [&](const T* q, int i, int h) {
    const int c = i == total[h] - 1 && first[h] ? 0 : rest[h] + i, k0 = c * EC - lead[h];
    C v;
    if (GATED && K >= EC) {  // a whole chunk within the row, of which these elements stay
      const int from = max(min(k0, K - EC), 0), begin = i < total[h] ? max(k0, 0) : K, end = min(k0 + EC, K);
      v = load_loose(q + from);
#pragma unroll
      for (int e = 0; e < EC; ++e)
        if (from + e < begin || from + e >= end) v[e] = (T)0.f;
    } else if (i < total[h] && k0 >= 0 && k0 + EC <= K) {
      v = load_loose(q + k0);
    } else {
#pragma unroll
      for (int e = 0; e < EC; ++e) v[e] = i < total[h] && k0 + e >= 0 && k0 + e < K ? q[k0 + e] : (T)0.f;
    }
    return v;
  };
  for (int i0 = wave * 4; i0 < most; i0 += 4 * NW) {
    C wv[NB], xv[H][MB];
#pragma unroll
    for (int b = 0; b < NB; ++b) wv[b] = part(w[b], i0 + quarter, b / HB);
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int m = 0; m < MB; ++m) xv[h][m] = part(x[m], i0 + quarter, h);
    multiply(wv, xv);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int m = 0; m < MB; ++m) *(f32x4*)&red[wave][(b * MB + m) * 256 + lane * 4] = acc[b][m];
  __syncthreads();
  for (int o = threadIdx.x; o < 16 * MB * RO; o += 64 * NW) {
    const int n = o % RO, m = o / RO;
    auto sum = [&](int row) {  // of the workgroup's weight rows
      const int at = ((row >> 4) * MB + (m >> 4)) * 256 + (((row >> 2) & 3) * 16 + (m & 15)) * 4 + (row & 3);
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) v += red[k][at];
      return v;
    };
    const float v = sum(n), up = GATED ? sum(RO + n) : 0.f;
    if (m >= p.M || n0 + n * period >= p.N) continue;
    if constexpr (GATED) finish_gated<T, 1>(p, m, n0 + n * period, &v, &up);
    else finish<T, 1>(p, m, n0 + n * period, &v);
  }
}

int weight_rows_of(const Product& p) { return p.gated ? 2 * p.N : p.N; }

template <typename T, int MR, bool GATED>
hipError_t launch_rows(const Product& p, hipStream_t st) {
  // four workgroups a CU before a workgroup takes more weight rows
  if constexpr (GATED) {
    if (p.N >= 2048) rows_kernel<T, MR, 4, true><<<(p.N + 1) / 2, 256, 0, st>>>(p);
    else rows_kernel<T, MR, 2, true><<<p.N, 256, 0, st>>>(p);
  } else {
    if (p.N >= 4096) rows_kernel<T, MR, 4, false><<<(p.N + 3) / 4, 256, 0, st>>>(p);
    else if (p.N >= 2048) rows_kernel<T, MR, 2, false><<<(p.N + 1) / 2, 256, 0, st>>>(p);
    else rows_kernel<T, MR, 1, false><<<p.N, 256, 0, st>>>(p);
  }
  return hipGetLastError();
}

template <typename T, bool GATED>
hipError_t launch_narrow(const Product& p, hipStream_t st) {
  const int weight_rows = weight_rows_of(p);
  // One or two rows on the vector units where a row occupies the workgroup (two rows of
  // 1024 16-bit numbers -> 8192: 8.2 us against 6.1), up to four where there are few
  // workgroups of the other kind (4 x 8192 -> 1000 in bf16: 8.0 against 14.4 us, 4 x 4096 ->
  // 4096: 12.9 against 10.2).
  if (p.M <= 4 && (weight_rows <= 2048 || (p.M <= 2 && p.K * (long long)sizeof(T) >= 4096))) {
    if (p.M == 1) return launch_rows<T, 1, GATED>(p, st);
    if (p.M == 2) return launch_rows<T, 2, GATED>(p, st);
    return launch_rows<T, 4, GATED>(p, st);
  }
  int period = 1;
  while (period < 16 / (int)sizeof(T) && p.ldb * sizeof(T) * period % 16) period *= 2;
  auto blocks = [&](int rows) {
    if (GATED) rows /= 2;
    return (unsigned)((p.N + rows * period - 1LL) / (rows * period) * period);
  };
  // where the halves' distances from boundaries differ, blocks of their own are worth half the
  // workgroups (9 x 3001 -> 2501 in bf16: 15.9 against 21.3 us; alike, 16 x 4096 -> 2048: 13.9 and 10.6)
  const bool alike = p.N * p.ldb * (long long)sizeof(T) % 16 == 0;
  const bool many = blocks(64) >= 200, two = GATED && blocks(32) >= (alike ? 200 : 100);
  if (p.M <= 16) {
    if (many) narrow_kernel<T, 1, 4, 4, GATED><<<blocks(64), 256, 0, st>>>(p, period);
    else if (two) narrow_kernel<T, 1, GATED ? 2 : 1, 16, GATED><<<blocks(32), 1024, 0, st>>>(p, period);
    else narrow_kernel<T, 1, 1, 16, GATED><<<blocks(16), 1024, 0, st>>>(p, period);
  } else {
    if (many) narrow_kernel<T, 2, 4, 4, GATED><<<blocks(64), 256, 0, st>>>(p, period);
    else if (two) narrow_kernel<T, 2, GATED ? 2 : 1, 16, GATED><<<blocks(32), 1024, 0, st>>>(p, period);
    else narrow_kernel<T, 2, 1, 16, GATED><<<blocks(16), 1024, 0, st>>>(p, period);
  }
  return hipGetLastError();
}

// Adds the parts of a split reduction, in order, and finishes the outputs: four of a row
// per thread.
template <typename T, bool GATED>
__device__ __forceinline__ void join_quads(const Product& p, int splits, unsigned block) {
  const int quads = p.ld_partial / (GATED ? 8 : 4);
  const long long i = (long long)block * 256 + threadIdx.x;
  const long long m = i / quads;
  const int n = (int)(i % quads) * 4;
  if (m >= p.M) return;
  const long long step = p.M * p.ld_partial;
  auto join = [&](const float* q, float* x) {
    f32x4 v = *(const f32x4*)q;
    int s = 1;
    for (; s + 5 <= splits; s += 5) {  // five loads at a time
      f32x4 part[5];
#pragma unroll
      for (int k = 0; k < 5; ++k) part[k] = *(const f32x4*)(q + (s + k) * step);
#pragma unroll
      for (int k = 0; k < 5; ++k) v += part[k];
    }
    for (; s < splits; ++s) v += *(const f32x4*)(q + s * step);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = v[k];
  };
  const float* q = p.partial + m * p.ld_partial + n;
  float x[4], up[4];
  join(q, x);
  if constexpr (GATED) join(q + p.ld_partial / 2, up);
  auto put = [&](auto vec, int k) {
    if constexpr (GATED) finish_gated<T, vec.value>(p, m, n + k, x + k, up + k);
    else finish<T, vec.value>(p, m, n + k, x + k);
  };
  if (n + 4 <= p.N) {
    put(std::integral_constant<int, 4>(), 0);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n + k < p.N) put(std::integral_constant<int, 1>(), k);
  }
}

template <typename T, bool GATED>
__global__ __launch_bounds__(256) void join_kernel(Product p, int splits) {
  join_quads<T, GATED>(p, splits, workgroup_number());
}

// The same for those of two products that are split: the first's workgroups, then the other's.
template <typename T>
__global__ __launch_bounds__(256) void join_pair_kernel(Product a, int splits_a, Product b, int splits_b, unsigned first) {
  const unsigned block = workgroup_number();
  if (block < first) join_quads<T, false>(a, splits_a, block);
  else join_quads<T, false>(b, splits_b, block - first);
}

template <typename T, int BM, int BN, int WM, int WN>
hipError_t launch_gemm(const Product& p, int splits, hipStream_t st) {
  const int outputs = p.gated ? BN / 2 : BN;  // of a tile's row
  const long long tm = (p.M + BM - 1) / BM, tn = (p.N + outputs - 1) / outputs;
  if (tm * tn > 0x7fffffffLL) return hipErrorInvalidValue;
  const dim3 grid = grid_of(tm * tn, splits);
  constexpr int threads = 64 * WM * WN;
  constexpr bool TWO = sizeof(T) == 2;
  if (p.gated) {
    gemm_kernel<T, BM, BN, WM, WN, false, false, false, true><<<grid, threads, 0, st>>>(p, (int)tm, (int)tn);
  } else if (TWO && p.a_low) {
    if (p.across_a) gemm_kernel<T, BM, BN, WM, WN, true, true, TWO><<<grid, threads, 0, st>>>(p, (int)tm, (int)tn);
    else gemm_kernel<T, BM, BN, WM, WN, false, true, TWO><<<grid, threads, 0, st>>>(p, (int)tm, (int)tn);
  } else if (p.across_a) {
    gemm_kernel<T, BM, BN, WM, WN, true, true, false><<<grid, threads, 0, st>>>(p, (int)tm, (int)tn);
  } else if (p.across_b) {
    gemm_kernel<T, BM, BN, WM, WN, false, true, false><<<grid, threads, 0, st>>>(p, (int)tm, (int)tn);
  } else {
    gemm_kernel<T, BM, BN, WM, WN, false, false, false><<<grid, threads, 0, st>>>(p, (int)tm, (int)tn);
  }
  return hipGetLastError();
}

// float32 numbers of a row of parts
int partial_row(const Product& p) { return (p.N + 3) / 4 * (p.gated ? 8 : 4); }

// Splits p's reduction into about `splits` parts; returns how many.
template <typename T>
int set_splits(Product& p, int splits) {
  // in steps of 64 bytes, an even number of them to a part
  const int steps = (int)((p.K * (long long)sizeof(T) + 63) / 64);
  p.split_steps = ((steps + splits - 1) / splits + 1) / 2 * 2;
  splits = (steps + p.split_steps - 1) / p.split_steps;
  if (splits == 1) p.partial = nullptr;
  p.ld_partial = partial_row(p);
  return splits;
}
long long join_blocks(const Product& p, int splits) {
  return splits > 1 ? (p.M * (p.ld_partial / (p.gated ? 8 : 4)) + 255) / 256 : 0;
}

template <typename T>
hipError_t launch_tiled(Product p, const Tiling& t, hipStream_t st) {
  const int splits = set_splits<T>(p, t.splits);
  hipError_t e;
  if constexpr (sizeof(T) == 2) {
    if (t.bm == 256 && t.bn == 256) e = launch_gemm<T, 256, 256, 2, 4>(p, splits, st);
    else if (t.bm == 256) e = launch_gemm<T, 256, 128, 4, 2>(p, splits, st);
    else if (t.bm == 128) e = launch_gemm<T, 128, 128, 2, 4>(p, splits, st);
    else e = launch_gemm<T, 64, 64, 2, 2>(p, splits, st);
  } else {
    if (t.bm == 256) e = launch_gemm<T, 256, 128, 4, 2>(p, splits, st);
    else if (t.bm == 128) e = launch_gemm<T, 128, 128, 2, 4>(p, splits, st);
    else e = launch_gemm<T, 64, 64, 2, 2>(p, splits, st);
  }
  if (e != hipSuccess || splits == 1) return e;
  const long long blocks = join_blocks(p, splits);
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  if (p.gated) join_kernel<T, true><<<grid_of(blocks), 256, 0, st>>>(p, splits);
  else join_kernel<T, false><<<grid_of(blocks), 256, 0, st>>>(p, splits);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Rows that do not start on 16-byte boundaries or end in part of a chunk are copied to
// rows that do, zeros to the end of the chunk, before a large product; both operands of
// a call in one launch, a chunk per thread.
template <typename T>
__device__ __forceinline__ void pack_chunk(const PackJobs& jobs, unsigned block) {
  typedef typename Chunk<T>::type C;
  constexpr int EC = 16 / sizeof(T);
  const bool second = block >= jobs.job[0].blocks;
  const PackJob& j = jobs.job[second];
  const long long i = (long long)(block - (second ? jobs.job[0].blocks : 0)) * 256 + threadIdx.x;
  const long long r = i / j.chunks;
  const int c = (int)(i % j.chunks);
  if (r >= j.rows) return;
  const T* q = (const T*)j.src + r * j.ld + (long long)c * EC;
  C v;
  if ((c + 1) * EC <= j.n) {
    v = load_loose(q);
  } else {
#pragma unroll
    for (int e = 0; e < EC; ++e) v[e] = c * EC + e < j.n ? q[e] : (T)0.f;
  }
  *(C*)((T*)j.dst + i * EC) = v;
}

template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(PackJobs jobs) {
  pack_chunk<T>(jobs, workgroup_number());
}

// g = dy act'(saved), its copies and its column sums.  A thread has one chunk of columns
// and every eighth of the workgroup's rows (16-byte accesses at any alignment); the
// workgroup's 32 chunks of columns are summed over its rows in LDS, one float32 per
// column and workgroup.  HBM bounds it (4096 x 8192 in bf16, GELU: 51 us with both parts of
// g, 268 MB at 5.3 TB/s, 37 us with one, 201 MB at 5.5; its vector instructions alone are
// about 34 and 26 us).  Workgroups have 64 rows, or as few as 8 while there would be less than two
// workgroups a CU (1037 x 999 in float16: 13 us with 64 rows, 5.5 so).
int sum_rows(long long rows, int n, int chunk) {
  const long long across = (n + 32 * chunk - 1) / (32 * chunk);
  int r = 64;
  while (r > 8 && across * ((rows + r - 1) / r) < 512) r /= 2;
  return r;
}

// x = 2 h + 2^(1 - p) l with h and l of a type of p significand bits, to 2^(-2 p): h is half
// of x, as a factor act' of up to 1.13 takes float16's largest numbers out of its range, and
// l is scaled to about the size of h, as unscaled it would be one of float16's subnormal
// numbers from 2^-4 on down.
template <typename T>
__device__ __forceinline__ void split(float x, T& h, T& l) {
  const float half = 0.5f * x;
  h = from_f32<T>(half);
  l = fabsf(half) < INFINITY ? from_f32<T>((half - to_f32(h)) * (1 << Chunk<T>::BITS)) : (T)0.f;
}

template <typename T, int ACT>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGrad p, PackJobs jobs) {
  typedef typename Chunk<T>::type C;
  typedef typename Loose<T>::type LC;
  constexpr int EC = 16 / sizeof(T);
  __shared__ float red[8][32 * EC + 1];
  const unsigned block = workgroup_number();
  if (block >= p.blocks) {  // the copies that the products need, by the same launch
    pack_chunk<T>(jobs, block - p.blocks);
    return;
  }
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5;
  const unsigned across = (p.n + 32 * EC - 1) / (32 * EC), bx = block % across, by = block / across;
  const int n = (bx * 32 + c) * EC;
  const long long m0 = (long long)by * p.part_rows;
  const T* dy = (const T*)p.dy;
  const T* saved = (const T*)p.saved;
  float sum[EC];
#pragma unroll
  for (int e = 0; e < EC; ++e) sum[e] = 0.f;
  const int have = p.n - n;  // columns from this chunk on
  for (long long m = m0 + w; m < min(m0 + p.part_rows, p.rows) && have > 0; m += 8) {
    C d, s;
    if (have >= EC) {
      d = load_loose(dy + m * p.ld_dy + n);
      if (ACT != VB_ACT_NONE) s = load_loose(saved + m * p.ld_saved + n);
    } else {
#pragma unroll
      for (int e = 0; e < EC; ++e) {
        d[e] = e < have ? dy[m * p.ld_dy + n + e] : (T)0.f;
        if (ACT != VB_ACT_NONE) s[e] = e < have ? saved[m * p.ld_saved + n + e] : (T)0.f;
      }
    }
    C v, high, low;
#pragma unroll
    for (int e = 0; e < EC; ++e) {
      const float x = act_grad<T>(to_f32((T)d[e]), ACT == VB_ACT_NONE ? 0.f : to_f32((T)s[e]), ACT);
      sum[e] += x;
      v[e] = from_f32<T>(x);
      if (ACT == VB_ACT_GELU || ACT == VB_ACT_SILU) {
        T h, l;
        split<T>(x, h, l);
        high[e] = h, low[e] = l;
      }
    }
    if ((ACT == VB_ACT_GELU || ACT == VB_ACT_SILU) && p.g_low) {
      *(C*)((T*)p.g + m * p.ld_g + n) = high;
      *(C*)((T*)p.g_low + m * p.ld_g + n) = low;
    } else if (p.g) {
      *(C*)((T*)p.g + m * p.ld_g + n) = v;
    }
    if (p.dres) {
      T* o = (T*)p.dres + m * p.ld_dres + n;
      if (have >= EC) {
        *(LC*)o = v;
      } else {
#pragma unroll
        for (int e = 0; e < EC; ++e)
          if (e < have) o[e] = v[e];
      }
    }
  }
  if (!p.dbias) return;
#pragma unroll
  for (int e = 0; e < EC; ++e) red[w][c * EC + e] = sum[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * EC; i += 256) {
    const int col = bx * 32 * EC + i;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += red[k][i];
    if (col < p.n) {
      if (!p.partial) ((T*)p.dbias)[col] = from_f32<T>(s);
      else p.partial[(long long)by * p.n + col] = s;
    }
  }
}

// g of the gated layer, its copies and its column sums: as act_grad_kernel, each chunk of dy
// giving one of dgate and one of dup.  HBM bounds it (4096 x 8192 in bf16, SiLU, both parts of g:
// 86 us, 470 MB at 5.5 TB/s).
template <typename T, int ACT>
__global__ __launch_bounds__(256) void gate_grad_kernel(GateGrad p, PackJobs jobs) {
  typedef typename Chunk<T>::type C;
  typedef typename Loose<T>::type LC;
  constexpr int EC = 16 / sizeof(T);
  __shared__ float red[2][8][32 * EC + 1];
  const unsigned block = workgroup_number();
  if (block >= p.blocks) {  // the copies that the products need, by the same launch
    pack_chunk<T>(jobs, block - p.blocks);
    return;
  }
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5;
  const unsigned across = (p.n + 32 * EC - 1) / (32 * EC), bx = block % across, by = block / across;
  const int n = (bx * 32 + c) * EC;
  const long long m0 = (long long)by * p.part_rows;
  float sum[2][EC];
#pragma unroll
  for (int e = 0; e < EC; ++e) sum[0][e] = sum[1][e] = 0.f;
  const int have = p.n - n;  // columns from this chunk on
  const int pad = (int)(p.ld_g - 2LL * p.n);
  for (long long m = m0 + w; m < min(m0 + p.part_rows, p.rows) && have > 0; m += 8) {
    const T* dy = (const T*)p.dy + m * p.ld_dy + n;
    const T* pre = (const T*)p.pre + m * p.ld_pre + n;
    C d, gate, up;
    if (have >= EC) {
      d = load_loose(dy), gate = load_loose(pre), up = load_loose(pre + p.n);
    } else {
#pragma unroll
      for (int e = 0; e < EC; ++e) {
        d[e] = e < have ? dy[e] : (T)0.f;
        gate[e] = e < have ? pre[e] : (T)0.f;
        up[e] = e < have ? pre[p.n + e] : (T)0.f;
      }
    }
    C high[2], low[2];
#pragma unroll
    for (int e = 0; e < EC; ++e) {
      const float dv = to_f32((T)d[e]), gv = to_f32((T)gate[e]), uv = to_f32((T)up[e]);
      const float x[2] = {act_grad<T>(dv * uv, gv, ACT), dv * act_value<T>(gv, ACT)};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        sum[k][e] += x[k];
        T h = from_f32<T>(x[k]), l = (T)0.f;
        if (sizeof(T) == 2 && p.g_low) split<T>(x[k], h, l);
        high[k][e] = h, low[k][e] = l;
      }
    }
    auto put = [&](void* g, const C* v) {
      T* o = (T*)g + m * p.ld_g + n;
      if (have >= EC) {
        *(C*)o = v[0];
        *(LC*)(o + p.n) = v[1];
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < EC; ++e)
            if (e < have) o[k * p.n + e] = v[k][e];
      }
      if (have <= EC)
        for (int e = 0; e < pad; ++e) o[p.n + have + e] = (T)0.f;
    };
    if (p.g) put(p.g, high);
    if (sizeof(T) == 2 && p.g_low) put(p.g_low, low);
  }
  if (!p.dbias) return;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int e = 0; e < EC; ++e) red[k][w][c * EC + e] = sum[k][e];
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * EC; i += 256) {
    const int k = i / (32 * EC), j = i % (32 * EC), col = bx * 32 * EC + j;
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += red[k][q][j];
    if (col < p.n) {
      const long long at = (long long)k * p.n + col;
      if (!p.partial) ((T*)p.dbias)[at] = from_f32<T>(s);
      else p.partial[(long long)by * 2 * p.n + at] = s;
    }
  }
}

__global__ __launch_bounds__(256) void fill_zero_kernel(unsigned short* p, long long rows, long long n, long long ld) {
  const long long i = (long long)workgroup_number() * 256 + threadIdx.x;
  if (i < rows * n) p[i / n * ld + i % n] = 0;
}

unsigned pack_blocks(PackJobs& jobs, int dtype) {
  long long blocks = 0;
  for (PackJob& j : jobs.job) {
    if (!j.dst) j.rows = 0;
    j.chunks = (int)(chunked_row(j.n, dtype) / 16);
    const long long b = (j.rows * j.chunks + 255) / 256;
    blocks += b;
    if (blocks > 0x7fffffffLL) return ~0u;
    j.blocks = (unsigned)b;
  }
  return (unsigned)blocks;
}

template <typename T>
hipError_t launch_act_grad_typed(ActGrad p, const PackJobs& jobs, unsigned copies, ColumnSums& sums, hipStream_t st) {
  constexpr int EC = 16 / sizeof(T);
  p.part_rows = sum_rows(p.rows, p.n, EC);
  const long long parts = (p.rows + p.part_rows - 1) / p.part_rows;
  const long long blocks = parts * ((p.n + 32 * EC - 1) / (32 * EC));
  if (blocks + copies > 0x7fffffffLL) return hipErrorInvalidValue;
  p.blocks = (unsigned)blocks;
  if (parts == 1) p.partial = nullptr;
  else if (p.dbias) sums = {p.partial, (int)parts, p.n, p.dbias};
  const dim3 grid = grid_of(blocks + copies);
  if (p.act == VB_ACT_NONE) act_grad_kernel<T, VB_ACT_NONE><<<grid, 256, 0, st>>>(p, jobs);
  else if (p.act == VB_ACT_RELU) act_grad_kernel<T, VB_ACT_RELU><<<grid, 256, 0, st>>>(p, jobs);
  else if (p.act == VB_ACT_GELU) act_grad_kernel<T, VB_ACT_GELU><<<grid, 256, 0, st>>>(p, jobs);
  else act_grad_kernel<T, VB_ACT_SILU><<<grid, 256, 0, st>>>(p, jobs);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_gate_grad_typed(GateGrad p, const PackJobs& jobs, unsigned copies, ColumnSums& sums, hipStream_t st) {
  constexpr int EC = 16 / sizeof(T);
  p.part_rows = sum_rows(p.rows, p.n, EC);
  const long long parts = (p.rows + p.part_rows - 1) / p.part_rows;
  const long long blocks = parts * ((p.n + 32 * EC - 1) / (32 * EC));
  if (blocks + copies > 0x7fffffffLL) return hipErrorInvalidValue;
  p.blocks = (unsigned)blocks;
  if (parts == 1) p.partial = nullptr;
  else if (p.dbias) sums = {p.partial, (int)parts, 2 * p.n, p.dbias};
  const dim3 grid = grid_of(blocks + copies);
  if (p.act == VB_ACT_NONE) gate_grad_kernel<T, VB_ACT_NONE><<<grid, 256, 0, st>>>(p, jobs);
  else if (p.act == VB_ACT_RELU) gate_grad_kernel<T, VB_ACT_RELU><<<grid, 256, 0, st>>>(p, jobs);
  else if (p.act == VB_ACT_GELU) gate_grad_kernel<T, VB_ACT_GELU><<<grid, 256, 0, st>>>(p, jobs);
  else gate_grad_kernel<T, VB_ACT_SILU><<<grid, 256, 0, st>>>(p, jobs);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_pair_typed(Product dx, Product dw, const Pair& pair, const ColumnSums& s, hipStream_t st) {
  const int sx = set_splits<T>(dx, pair.splits_x), sw = set_splits<T>(dw, pair.splits_w);
  const int tile = pair.tile, tn = (dx.N + tile - 1) / tile;
  const long long tiles = ((dx.M + tile - 1) / tile * sx + (dw.M + tile - 1) / tile * sw) * tn;
  const long long blocks = tiles + (s.out ? (s.n + 63) / 64 : 0);
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  const bool first = dx.split_steps >= dw.split_steps;
  const dim3 grid = grid_of(blocks);
  constexpr bool TWO = sizeof(T) == 2;
  if (TWO && dx.a_low) {
    if (tile == 64) pair_kernel<T, 64, 64, 2, 2, TWO><<<grid, 256, 0, st>>>(dx, dw, s, tn, sx, sw, first);
    else pair_kernel<T, 128, 128, 2, 4, TWO><<<grid, 512, 0, st>>>(dx, dw, s, tn, sx, sw, first);
  } else {
    if (tile == 64) pair_kernel<T, 64, 64, 2, 2, false><<<grid, 256, 0, st>>>(dx, dw, s, tn, sx, sw, first);
    else pair_kernel<T, 128, 128, 2, 4, false><<<grid, 512, 0, st>>>(dx, dw, s, tn, sx, sw, first);
  }
  const hipError_t e = hipGetLastError();
  const long long jx = join_blocks(dx, sx), jw = join_blocks(dw, sw);
  if (e != hipSuccess || jx + jw == 0) return e;
  if (jx + jw > 0x7fffffffLL) return hipErrorInvalidValue;
  join_pair_kernel<T><<<grid_of(jx + jw), 256, 0, st>>>(dx, sx, dw, sw, (unsigned)jx);
  return hipGetLastError();
}

}  // namespace

// Tile and split of a large product by the time they would take on the CU with the most
// tiles: 64-byte steps, those of both passes, of `share` microseconds (64-wide tiles,
// three to a CU at a time, take `latency` where one has its CU to itself), the `fixed`
// part of each tile, mostly its outputs, what a second pass over the stages adds to it (29478 x
// 4544 of 36 float16 rows: tiles of 256 158 us, 256 x 128 133), and a launch.  Measured, in us at 1024 x 1024 x
// 1024 | 2048 x 4096 x 4096 | 4096 x 4096 x 4096 | 4096 x 4096 x 32: bf16 tiles of 64 6.9
// | 111 | 197 | 15.6, 128 10.0 | 85 | 140 | 15.6, 256 x 128 14 | 61 | 122 | 12.6, 256 24
// | 92 | 113 | 13.2; float32 tiles of 64 21 | 479 | 966 | 24, 128 62 | 475 | 948 | 25,
// 256 x 128 118 | 465 | 938 | 25.  A split costs the writing and reading of its float32
// parts, at 6 TB/s as they are in the caches, and another launch; it has to gain 8 %, as
// it also keeps a backward pass from one launch for both products.
namespace {

struct Kind {
  int bm, bn, per_cu;
  double fixed, latency, share, again;
  double ends(const Product& p) const { return fixed + (p.passes > 1 ? again : 0.0); }
};
const Kind k16[] = {{256, 256, 1, 8.0, 0.82, 0.82, 7.0}, {256, 128, 1, 4.5, 0.43, 0.43, 2.5}, {128, 128, 1, 3.0, 0.255, 0.255, 1.8},
                    {64, 64, 3, 0.8, 0.13, 0.115, 0.4}};
const Kind k32[] = {{256, 128, 1, 7.0, 1.80, 1.80, 0}, {128, 128, 1, 3.5, 0.915, 0.915, 0}, {64, 64, 3, 0.8, 0.275, 0.235, 0}};

long long steps_of(long long K, int dtype) { return (K * (long long)elem_size(dtype) + 63) / 64; }

}  // namespace

Tiling choose_tiling(int dtype, const Product& p) {
  const long long M = p.M, K = p.K;
  const int N = weight_rows_of(p);
  const Kind* kinds = dtype == VB_F32 ? k32 : k16;
  const int nk = dtype == VB_F32 ? 3 : 4;
  const long long stages = steps_of(K, dtype);
  auto time = [&](const Kind& c, int n, double ends) {
    const double tiles = (double)((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    const double on_cu = std::ceil(tiles * n / 256.0), run = (double)((stages + n - 1) / n) * p.passes;
    double us = std::fmax(c.latency, on_cu * c.share) * run + on_cu * ends + 3.0;
    if (n > 1) us += 2.0 + (2.0 * n * M * N * 4.0) / 6e6;
    return us;
  };
  Tiling best{64, 64, 1, 1e30};
  double unsplit = 0;
  for (int n = 1; n <= 32 && (n == 1 || n * 4 <= stages); n *= 2) {
    for (int k = 0; k < nk; ++k) {
      const double us = time(kinds[k], n, kinds[k].fixed);
      if (us < best.us && (n == 1 || us < 0.92 * unsplit)) best = Tiling{kinds[k].bm, kinds[k].bn, n, us};
    }
    if (n == 1) unsplit = best.us;
  }
  // the split stands, and with it the order of the sums
  if (p.passes > 1) best.us = 1e30;
  for (int k = 0; k < nk && p.passes > 1; ++k) {
    const double us = time(kinds[k], best.splits, kinds[k].ends(p));
    if (us < best.us) best = Tiling{kinds[k].bm, kinds[k].bn, best.splits, us};
  }
  return best;
}

namespace {

// When 256 CUs that take tiles one at a time, a of them for c us, then a2 for c2, are done.
double list_time(double a, double c, double a2, double c2) {
  const double q = std::floor(a / 256.0), rest = a - q * 256.0, early = q * c, late = early + c;
  auto done = [&](double t) {
    return (256.0 - rest) * std::floor((t - early) / c2 + 1e-6) + rest * std::fmax(std::floor((t - late) / c2 + 1e-6), 0.0);
  };
  double best = 1e30;
  for (const double base : {early, late}) {
    double t = base + std::fmax(std::floor(((a * c + a2 * c2) / 256.0 - base) / c2), 0.0) * c2;
    while (done(t) < a2) t += c2;
    best = std::fmin(best, t);
  }
  return std::fmax(best, rest > 0 ? late : early);
}

}  // namespace

size_t tiling_bytes(const Tiling& t, const Product& p) {
  return t.splits > 1 ? (size_t)t.splits * p.M * partial_row(p) * 4 : 0;
}

// Tiles with which both products of a backward pass take one launch, which fills the card while
// the first one ends, and their parts' sums another; or none where launches of their own are
// faster by the same model (each of those past the first: 2 us).  Together | apart, with g and
// dbias: 1024 x 1024 -> 1024 in bf16 19.4 | 23.7 us (64-wide tiles), float32 44 | 52; 1024 x 2048
// -> 2048 34 | 41 (128); 4096 x 2048 -> 2048 96 | 92; split (728 x 49 -> 780 in float16, two-part g)
// 16 | 28.  Each reduction is split as the product's own launch would split it, so that a gradient has
// the same bits alone as with the other.  In float32 a split pair takes 64-wide tiles or none: the
// model, which counts 128-wide ones at their full rate, finds those faster, and they are not (1121 x
// 2097 -> 14556: 128-wide 1193 us, 64-wide 1126, apart 1150; 622 x 1419 -> 2 x 4848 355, 315, 327; of 31
// drawn 29 are slower by up to 14 %, two faster by 1 and 4 %; in 16 bits 128-wide ones gain up to 18 %).
Pair choose_pair(const Product& dx, const Product& dw, int dtype) {
  const Tiling x = choose_tiling(dtype, dx), w = choose_tiling(dtype, dw);
  auto run_of = [&](const Product& p, int splits) { return (double)((steps_of(p.K, dtype) + splits - 1) / splits) * p.passes; };
  const bool dx_first = run_of(dx, x.splits) >= run_of(dw, w.splits);
  const Product &first = dx_first ? dx : dw, &second = dx_first ? dw : dx;
  const int splits = dx_first ? x.splits : w.splits, splits2 = dx_first ? w.splits : x.splits;
  const double run = run_of(first, splits), run2 = run_of(second, splits2);
  double join = 0.0;
  if (x.splits > 1 || w.splits > 1) join = 2.0 + 2.0 * (tiling_bytes(x, dx) + tiling_bytes(w, dw)) / 6e6;
  Pair best{0, x.splits, w.splits};
  double best_us = x.us + w.us + 2.0;
  const Kind* kinds = dtype == VB_F32 ? k32 + 1 : k16 + 2;
  for (int k = 0; k < 2; ++k) {
    const Kind& c = kinds[k];
    if (dtype == VB_F32 && join > 0.0 && c.bm > 64) continue;
    auto tiles = [&](const Product& p, int s) { return (double)((p.M + c.bm - 1) / c.bm) * ((p.N + c.bn - 1) / c.bn) * s; };
    const double n = tiles(first, splits), n2 = tiles(second, splits2);
    double us;
    if (c.per_cu == 1) {
      us = list_time(n, run * c.share + c.ends(dx), n2, run2 * c.share + c.ends(dw)) + 3.0;
    } else {  // a CU has its share of the steps and half a tile more; its tiles' ends overlap
      const double share = std::fmin(std::ceil(n / 256.0) * run + std::ceil(n2 / 256.0) * run2,
                                     (n * run + n2 * run2) / 256.0 + run / 2);
      us = std::fmax(c.latency * run, c.share * share) + c.ends(dx) * std::ceil((n + n2) / 256.0) + 3.0;
    }
    us += join;
    if (us < best_us) best_us = us, best.tile = c.bm;
  }
  return best;
}

size_t pair_bytes(const Pair& pair, const Product& p, int splits) {
  return pair.tile && splits > 1 ? (size_t)splits * p.M * partial_row(p) * 4 : 0;
}

// Long rows of few weights, gated: a split reduction has more wavefronts than the narrow kernel,
// whose time grows with the reduction and the rows, and with the weights only later.  Weights off
// 16-byte boundaries have to be copied for the split, about their reading and writing again; the
// narrow kernel reads those in place, 16-bit ones with more work for x.  In us, narrow | split: 16 x
// 8192 -> 300 in bf16 16.6 | 9.4, 7 x 8192 -> 2048 15.1 | 17.6; float32 7 x 4096 -> 300 13.9 | 11.6, -> 2048
// 15.6 | 23.5, 16 x 12000 -> 1000 50 | 33, 31 x 2048 -> 300 13.4 | 10.2; off boundaries float32 7 x 4097 -> 300
// 12.3 | 18.6, 7 x 8191 -> 150 21.5 | 19.7, -> 2048 35 | 85, 31 x 2049 -> 300 11.7 | 14.5, 31 x 5001 -> 150
// 23.4 | 17.9; bf16 16 x 8193 -> 600 28.8 | 19.5, -> 2048 30 | 40.  (Over 404 such products 0.6 % longer
// than the better of both on average, 30 % at worst; always split 15 %, never 42 %.)
namespace {

bool split_is_faster(const Product& p, int dtype) {
  const double k = p.K / 1000.0, rows = p.M > 16 ? p.M + 8.0 : p.M, mb = 2e-6 * p.N * p.K * elem_size(dtype);
  if (!is_chunked(p.b, p.ldb, p.K, dtype))
    return dtype == VB_F32 ? k * (2.2 + 0.05 * rows) > 14.5 + 0.5 * mb : k * (1.4 + 0.12 * rows) > 12.5 + 0.42 * mb;
  if (p.M > 16) return true;
  return dtype == VB_F32 ? k * (2.3 + 0.07 * rows) > 11.5 + 0.16 * mb : k * (1.0 + 0.04 * rows) > 9.5 + 0.1 * mb;
}

}  // namespace

// Up to 16 rows, and up to 32 where the weights are few (24 x 1024 -> 1024 in bf16: 5.2
// against 7.7 us; 24 x 4096 -> 4096: 14.7 against 13.2) or long and many (32 x 4096 ->
// 16384: 34 against 37, float32 63 against 72; 32 x 1024 -> 65536: 36 against 31).
bool product_is_narrow(const Product& p, int dtype) {
  if (p.across_a || p.across_b || p.tiled) return false;
  const long long row = p.K * (long long)elem_size(dtype);
  const int n = weight_rows_of(p);
  if (p.gated && p.M > 4 && p.N <= 2048 && row * (p.M > 16 ? 2 : 1) >= 16384 && split_is_faster(p, dtype)) return false;
  return p.M <= 16 || (p.M <= 32 && (n * row <= 8 << 20 || (n >= 12800 && row >= 8192)));
}

size_t product_bytes(const Product& p, int dtype) {
  if (product_is_narrow(p, dtype)) return 0;
  return tiling_bytes(choose_tiling(dtype, p), p);
}

hipError_t launch_product(const Product& p, int dtype, hipStream_t st) {
  if (product_is_narrow(p, dtype)) {
    if (dtype == VB_F32) return p.gated ? launch_narrow<float, true>(p, st) : launch_narrow<float, false>(p, st);
    if (dtype == VB_BF16) return p.gated ? launch_narrow<bf16, true>(p, st) : launch_narrow<bf16, false>(p, st);
    return p.gated ? launch_narrow<f16, true>(p, st) : launch_narrow<f16, false>(p, st);
  }
  const Tiling t = choose_tiling(dtype, p);
  if (dtype == VB_F32) return launch_tiled<float>(p, t, st);
  if (dtype == VB_BF16) return launch_tiled<bf16>(p, t, st);
  return launch_tiled<f16>(p, t, st);
}

bool is_chunked(const void* p, long long ld, long long n, int dtype) {
  const long long es = (long long)elem_size(dtype);
  return (uintptr_t)p % 16 == 0 && ld * es % 16 == 0 && n * es % 16 == 0 && ld * es <= MAX_CHUNKED_ROW;
}

hipError_t launch_pack(PackJobs jobs, int dtype, hipStream_t st) {
  const unsigned blocks = pack_blocks(jobs, dtype);
  if (blocks == ~0u) return hipErrorInvalidValue;
  if (!blocks) return hipSuccess;
  if (dtype == VB_F32) pack_kernel<float><<<grid_of(blocks), 256, 0, st>>>(jobs);
  else if (dtype == VB_BF16) pack_kernel<bf16><<<grid_of(blocks), 256, 0, st>>>(jobs);
  else pack_kernel<f16><<<grid_of(blocks), 256, 0, st>>>(jobs);
  return hipGetLastError();
}

size_t act_grad_bytes(long long rows, int n, int dtype) {
  const int per = sum_rows(rows, n, 16 / (int)elem_size(dtype));
  return rows > per ? (size_t)((rows + per - 1) / per) * n * 4 : 0;
}

hipError_t launch_act_grad(const ActGrad& p, PackJobs jobs, int dtype, ColumnSums& sums, hipStream_t st) {
  const unsigned copies = pack_blocks(jobs, dtype);
  if (copies == ~0u) return hipErrorInvalidValue;
  if (dtype == VB_F32) return launch_act_grad_typed<float>(p, jobs, copies, sums, st);
  if (dtype == VB_BF16) return launch_act_grad_typed<bf16>(p, jobs, copies, sums, st);
  return launch_act_grad_typed<f16>(p, jobs, copies, sums, st);
}

size_t gate_grad_bytes(long long rows, int n, int dtype) { return 2 * act_grad_bytes(rows, n, dtype); }

hipError_t launch_gate_grad(const GateGrad& p, PackJobs jobs, int dtype, ColumnSums& sums, hipStream_t st) {
  const unsigned copies = pack_blocks(jobs, dtype);
  if (copies == ~0u) return hipErrorInvalidValue;
  if (dtype == VB_F32) return launch_gate_grad_typed<float>(p, jobs, copies, sums, st);
  if (dtype == VB_BF16) return launch_gate_grad_typed<bf16>(p, jobs, copies, sums, st);
  return launch_gate_grad_typed<f16>(p, jobs, copies, sums, st);
}

hipError_t launch_column_sums(const ColumnSums& s, int dtype, hipStream_t st) {
  const unsigned blocks = (s.n + 63) / 64;
  if (dtype == VB_F32) column_sum_kernel<float><<<blocks, 1024, 0, st>>>(s);
  else if (dtype == VB_BF16) column_sum_kernel<bf16><<<blocks, 1024, 0, st>>>(s);
  else column_sum_kernel<f16><<<blocks, 1024, 0, st>>>(s);
  return hipGetLastError();
}

hipError_t launch_pair(const Product& dx, const Product& dw, const Pair& pair, const ColumnSums& s, int dtype, hipStream_t st) {
  if (dtype == VB_F32) return launch_pair_typed<float>(dx, dw, pair, s, st);
  if (dtype == VB_BF16) return launch_pair_typed<bf16>(dx, dw, pair, s, st);
  return launch_pair_typed<f16>(dx, dw, pair, s, st);
}

hipError_t launch_fill_zero(void* p, long long rows, long long row_bytes, long long ld_bytes, hipStream_t st) {
  const long long n = row_bytes / 2;
  const long long blocks = (rows * n + 255) / 256;
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  fill_zero_kernel<<<grid_of(blocks), 256, 0, st>>>((unsigned short*)p, rows, n, ld_bytes / 2);
  return hipGetLastError();
}

}  // namespace vb
