// The fused linear layer y = act(x W^T + bias + residual) and the products of
// its backward pass.
#include <algorithm>
#include <cmath>

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
// (8192 x 8192 -> 4096 3.78 ms, 145 TFLOP/s; the library's 3.60 ms).
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
template <typename T, int BM, int BN, int WM, int WN, bool XA, bool XB, bool TWO>
__device__ __forceinline__ void gemm_tile(Product p, int tm, int tn, unsigned block, unsigned split, char* lds) {
  typedef typename Chunk<T>::type C;
  constexpr int DEPTH = Ring<BM, BN, XA, XB>::DEPTH, NS = Ring<BM, BN, XA, XB>::NS;
  constexpr int NW = WM * WN, STAGE = (BM + BN) * DEPTH, KS = DEPTH / sizeof(T);
  constexpr int TM = BM / WM, TN = BN / WN, MT = TM / 16, NT = TN / 16, MH = MT / 2;
  typedef Operand<T, BM, NW, XA, DEPTH> OA;
  typedef Operand<T, BN, NW, XB, DEPTH> OB;
  constexpr int LA = OA::L, LB = OB::L, RA = OA::READS, RB = OB::READS;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int ti, tj;
  tile_of(block, tm, tn, ti, tj);
  const long long m0 = (long long)ti * BM;
  const int n0 = tj * BN;
  // this workgroup's part of the reduction
  const int first = split * (p.split_steps / (DEPTH / 64));
  const int K = (int)min(p.K - (long long)first * KS, (long long)p.split_steps * (64 / (int)sizeof(T)));
  const int stages = (K + KS - 1) / KS, full = K / KS;
  OA a;
  OB b;
  a.init(p.a, p.lda, m0, p.M, first, wave, lane);
  b.init(p.b, p.ldb, n0, p.N, first, wave, lane);
  const unsigned lds0 = lds_address(lds);
  auto issue = [&](int t, int base) { a.load(t, lds0 + base), b.load(t, lds0 + base + BM * DEPTH); };
  auto issue_part = [&](int t, int base) { a.load_part(t, lds0 + base, K), b.load_part(t, lds0 + base + BM * DEPTH, K); };
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
  for (int j = 0; j < NT; ++j) pb[j] = BM * DEPTH + b.place(wn * NT + j);
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
  constexpr int LDE = TN + 4, VEC = 16 / sizeof(T), LPR = TN / VEC, RPI = 64 / LPR;
  static_assert(NW * 32 * LDE * 4 <= NS * STAGE, "the output staging fits the operand stages");
  float* e = (float*)lds + wave * 32 * LDE;
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
    if (p.partial) {
      // float32 sums of this part, rows of N rounded up to four
      float* part = p.partial + (split * p.M + mb) * (long long)p.ld_partial + nb;
      const int row = lane / (TN / 4), col = lane % (TN / 4) * 4;
#pragma unroll
      for (int r = 0; r < 32; r += 256 / TN)
        if (mb + r + row < p.M && nb + col < p.N)
          *(f32x4*)(part + (r + row) * (long long)p.ld_partial + col) = *(const f32x4*)(e + (r + row) * LDE + col);
    } else {
      const int row = lane / LPR, col = (lane % LPR) * VEC;
#pragma unroll
      for (int r = 0; r < 32; r += RPI) {
        const float* v = e + (r + row) * LDE + col;
        if (mb + r + row < p.M && nb + col < p.N) {
          if (nb + col + VEC <= p.N) {
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

template <typename T, int BM, int BN, int WM, int WN, bool XA, bool XB, bool TWO>
__global__ __launch_bounds__(64 * WM * WN, BN == 64 ? 3 : 2) void gemm_kernel(Product p, int tm, int tn) {
  __shared__ __align__(16) char lds[Ring<BM, BN, XA, XB>::BYTES];
  const unsigned block = workgroup_number();
  if (block >= (unsigned)tm * tn) return;  // the whole workgroup
  gemm_tile<T, BM, BN, WM, WN, XA, XB, TWO>(p, tm, tn, block, blockIdx.y, lds);
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
// the tiles of the product with the longer reduction, then the other's.
template <typename T, int BM, int BN, int WM, int WN, bool TWO>
__global__ __launch_bounds__(64 * WM * WN, BN == 64 ? 3 : 2) void pair_kernel(Product dx, Product dw, ColumnSums s, int tn) {
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
  if (block >= ((unsigned)tx + tw) * tn) return;  // the whole workgroup
  const unsigned first = (dx.K >= dw.K ? tx : tw) * tn;
  if ((block < first) == (dx.K >= dw.K))
    gemm_tile<T, BM, BN, WM, WN, false, true, TWO>(dx, tx, tn, block < first ? block : block - first, 0, lds);
  else
    gemm_tile<T, BM, BN, WM, WN, true, true, TWO>(dw, tw, tn, block < first ? block : block - first, 0, lds);
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
template <typename T, int MR, int R>
__global__ __launch_bounds__(256) void rows_kernel(Product p) {
  typedef typename Chunk<T>::type C;
  constexpr int EC = 16 / sizeof(T);
  __shared__ float red[4][R * MR];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * R, chunks = (int)(p.K / EC), tail = (int)(p.K % EC);
  const T* w[R];
  const T* x[MR];
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = (const T*)p.b + (long long)min(n0 + r, p.N - 1) * p.ldb;
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
  const int t = threadIdx.x, m = t / R, n = n0 + t % R;
  if (t < R * MR && m < p.M && n < p.N) {
    const float v = (red[0][t] + red[1][t]) + (red[2][t] + red[3][t]);
    finish<T, 1>(p, m, n, &v);
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
template <typename T, int MB, int NB, int NW>
__global__ __launch_bounds__(64 * NW) void narrow_kernel(Product p, int period) {
  typedef typename Chunk<T>::type C;
  constexpr int EC = 16 / sizeof(T), U = 2, OUT = MB * NB * 256;
  __shared__ __align__(16) float red[NW][OUT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, quarter = lane >> 4;
  const int like = blockIdx.x % period, n0 = blockIdx.x / period * (16 * NB) * period + like;
  if (like >= p.N) return;  // the whole workgroup
  const int last = p.N - 1 - (p.N - 1 - like) % period;
  const T* w[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) w[b] = (const T*)p.b + (long long)min(n0 + (16 * b + r16) * period, last) * p.ldb;
  const int lead = __builtin_amdgcn_readfirstlane((int)((uintptr_t)w[0] % 16 / sizeof(T)));
  const T* x[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) x[m] = (const T*)p.a + min((long long)(16 * m + r16), p.M - 1) * p.lda;
  f32x4 acc[NB][MB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[b][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const C* wv, const C* xv) {
#pragma unroll
    for (int q = 0; q < Chunk<T>::MFMAS; ++q)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[b][m] = Chunk<T>::mma(wv[b], xv[m], acc[b][m], q);
  };
  // whole chunks first .. end - 1 (chunk c holds elements c EC - lead on), of which runs
  const int K = (int)p.K, first = lead > 0, end = (lead + K) / EC;
  const int runs = max(end - first, 0) / (4 * U);
  const int turn = runs ? (int)(blockIdx.x % (unsigned)runs) : 0;
  for (int s = wave; s < runs; s += NW) {
    const int run = s + turn < runs ? s + turn : s + turn - runs;
    C wv[U][NB], xv[U][MB];
    const long long k0 = (long long)(first + run * (4 * U) + quarter) * EC - lead;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int u = 0; u < U; ++u) wv[u][b] = *(const C*)(w[b] + k0 + u * 4 * EC);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < MB; ++m) xv[u][m] = load_loose(x[m] + k0 + u * 4 * EC);
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(wv[u], xv[u]);
  }
  // the chunks left over and those that the row fills in part (the first one comes last),
  // zeros elsewhere, a step of four per wavefront
  const int rest = first + runs * 4 * U, total = (lead + K + EC - 1) / EC - rest + first;
  auto part = [&](const T* q, int i) {
    const int c = i == total - 1 && first ? 0 : rest + i, k0 = c * EC - lead;
    C v;
    if (i < total && k0 >= 0 && k0 + EC <= K) {
      v = load_loose(q + k0);
    } else {
#pragma unroll
      for (int e = 0; e < EC; ++e) v[e] = i < total && k0 + e >= 0 && k0 + e < K ? q[k0 + e] : (T)0.f;
    }
    return v;
  };
  for (int i0 = wave * 4; i0 < total; i0 += 4 * NW) {
    C wv[NB], xv[MB];
#pragma unroll
    for (int b = 0; b < NB; ++b) wv[b] = part(w[b], i0 + quarter);
#pragma unroll
    for (int m = 0; m < MB; ++m) xv[m] = part(x[m], i0 + quarter);
    multiply(wv, xv);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int m = 0; m < MB; ++m) *(f32x4*)&red[wave][(b * MB + m) * 256 + lane * 4] = acc[b][m];
  __syncthreads();
  for (int o = threadIdx.x; o < OUT; o += 64 * NW) {
    const int n = o % (16 * NB), m = o / (16 * NB);
    const int at = ((n >> 4) * MB + (m >> 4)) * 256 + (((n >> 2) & 3) * 16 + (m & 15)) * 4 + (n & 3);
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) v += red[k][at];
    if (m < p.M && n0 + n * period < p.N) finish<T, 1>(p, m, n0 + n * period, &v);
  }
}

template <typename T, int MR>
hipError_t launch_rows(const Product& p, hipStream_t st) {
  // four workgroups a CU before a workgroup takes more weight rows
  if (p.N >= 4096) rows_kernel<T, MR, 4><<<(p.N + 3) / 4, 256, 0, st>>>(p);
  else if (p.N >= 2048) rows_kernel<T, MR, 2><<<(p.N + 1) / 2, 256, 0, st>>>(p);
  else rows_kernel<T, MR, 1><<<p.N, 256, 0, st>>>(p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_narrow(const Product& p, hipStream_t st) {
  // One or two rows on the vector units where a row occupies the workgroup (two rows of
  // 1024 16-bit numbers -> 8192: 8.2 us against 6.1), up to four where there are few
  // workgroups of the other kind (4 x 8192 -> 1000 in bf16: 8.0 against 14.4 us, 4 x 4096 ->
  // 4096: 12.9 against 10.2).
  if (p.M <= 4 && (p.N <= 2048 || (p.M <= 2 && p.K * (long long)sizeof(T) >= 4096))) {
    if (p.M == 1) return launch_rows<T, 1>(p, st);
    if (p.M == 2) return launch_rows<T, 2>(p, st);
    return launch_rows<T, 4>(p, st);
  }
  int period = 1;
  while (period < 16 / (int)sizeof(T) && p.ldb * sizeof(T) * period % 16) period *= 2;
  auto blocks = [&](int rows) { return (unsigned)((p.N + rows * period - 1LL) / (rows * period) * period); };
  const bool many = blocks(64) >= 200;
  if (p.M <= 16) {
    if (many) narrow_kernel<T, 1, 4, 4><<<blocks(64), 256, 0, st>>>(p, period);
    else narrow_kernel<T, 1, 1, 16><<<blocks(16), 1024, 0, st>>>(p, period);
  } else {
    if (many) narrow_kernel<T, 2, 4, 4><<<blocks(64), 256, 0, st>>>(p, period);
    else narrow_kernel<T, 2, 1, 16><<<blocks(16), 1024, 0, st>>>(p, period);
  }
  return hipGetLastError();
}

// Adds the parts of a split reduction, in order, and finishes the outputs: four of a row
// per thread.
template <typename T>
__global__ __launch_bounds__(256) void join_kernel(Product p, int splits) {
  const int quads = p.ld_partial / 4;
  const long long i = (long long)workgroup_number() * 256 + threadIdx.x;
  const long long m = i / quads;
  const int n = (int)(i % quads) * 4;
  if (m >= p.M) return;
  const float* q = p.partial + m * p.ld_partial + n;
  const long long step = p.M * p.ld_partial;
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
  const float x[4] = {v[0], v[1], v[2], v[3]};
  if (n + 4 <= p.N) {
    finish<T, 4>(p, m, n, x);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n + k < p.N) finish<T, 1>(p, m, n + k, x + k);
  }
}

template <typename T, int BM, int BN, int WM, int WN>
hipError_t launch_gemm(const Product& p, int splits, hipStream_t st) {
  const long long tm = (p.M + BM - 1) / BM, tn = (p.N + BN - 1) / BN;
  if (tm * tn > 0x7fffffffLL) return hipErrorInvalidValue;
  const dim3 grid = grid_of(tm * tn, splits);
  constexpr int threads = 64 * WM * WN;
  constexpr bool TWO = sizeof(T) == 2;
  if (TWO && p.a_low) {
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

template <typename T>
hipError_t launch_tiled(Product p, const Tiling& t, hipStream_t st) {
  // in steps of 64 bytes, an even number of them to a part
  const int steps = (int)((p.K * (long long)sizeof(T) + 63) / 64);
  p.split_steps = ((steps + t.splits - 1) / t.splits + 1) / 2 * 2;
  const int splits = (steps + p.split_steps - 1) / p.split_steps;
  if (splits == 1) p.partial = nullptr;
  p.ld_partial = (p.N + 3) / 4 * 4;
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
  const long long quads = p.M * (p.ld_partial / 4), blocks = (quads + 255) / 256;
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  join_kernel<T><<<grid_of(blocks), 256, 0, st>>>(p, splits);
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
hipError_t launch_pair_typed(Product dx, Product dw, int tile, const ColumnSums& s, hipStream_t st) {
  for (Product* p : {&dx, &dw})  // no split
    p->split_steps = (int)((p->K * (long long)sizeof(T) + 127) / 128 * 2), p->partial = nullptr;
  const int tn = (dx.N + tile - 1) / tile;
  const long long tiles = ((dx.M + tile - 1) / tile + (dw.M + tile - 1) / tile) * tn;
  const long long blocks = tiles + (s.out ? (s.n + 63) / 64 : 0);
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  constexpr bool TWO = sizeof(T) == 2;
  if (TWO && dx.a_low) {
    if (tile == 64) pair_kernel<T, 64, 64, 2, 2, TWO><<<grid_of(blocks), 256, 0, st>>>(dx, dw, s, tn);
    else pair_kernel<T, 128, 128, 2, 4, TWO><<<grid_of(blocks), 512, 0, st>>>(dx, dw, s, tn);
  } else {
    if (tile == 64) pair_kernel<T, 64, 64, 2, 2, false><<<grid_of(blocks), 256, 0, st>>>(dx, dw, s, tn);
    else pair_kernel<T, 128, 128, 2, 4, false><<<grid_of(blocks), 512, 0, st>>>(dx, dw, s, tn);
  }
  return hipGetLastError();
}

}  // namespace

// Tile and split of a large product by the time they would take on the CU with the most
// tiles: 64-byte steps, those of both passes, of `share` microseconds (64-wide tiles,
// three to a CU at a time, take `latency` where one has its CU to itself), the `fixed`
// part of each tile, mostly its outputs, and a launch.  Measured, in us at 1024 x 1024 x
// 1024 | 2048 x 4096 x 4096 | 4096 x 4096 x 4096 | 4096 x 4096 x 32: bf16 tiles of 64 6.9
// | 111 | 197 | 15.6, 128 10.0 | 85 | 140 | 15.6, 256 x 128 14 | 61 | 122 | 12.6, 256 24
// | 92 | 113 | 13.2; float32 tiles of 64 21 | 479 | 966 | 24, 128 62 | 475 | 948 | 25,
// 256 x 128 118 | 465 | 938 | 25.  A split costs the writing and reading of its float32
// parts, at 6 TB/s as they are in the caches, and another launch; it has to gain 8 %, as
// it also keeps a backward pass from one launch for both products.
namespace {

struct Kind {
  int bm, bn, per_cu;
  double fixed, latency, share;
};
const Kind k16[] = {{256, 256, 1, 8.0, 0.82, 0.82}, {256, 128, 1, 4.5, 0.43, 0.43}, {128, 128, 1, 3.0, 0.255, 0.255},
                    {64, 64, 3, 0.8, 0.13, 0.115}};
const Kind k32[] = {{256, 128, 1, 7.0, 1.80, 1.80}, {128, 128, 1, 3.5, 0.915, 0.915}, {64, 64, 3, 0.8, 0.275, 0.235}};

long long steps_of(long long K, int dtype) { return (K * (long long)elem_size(dtype) + 63) / 64; }

}  // namespace

Tiling choose_tiling(int dtype, const Product& p) {
  const long long M = p.M, K = p.K;
  const int N = p.N;
  const Kind* kinds = dtype == VB_F32 ? k32 : k16;
  const int nk = dtype == VB_F32 ? 3 : 4;
  const long long stages = steps_of(K, dtype);
  Tiling best{64, 64, 1, 1e30};
  double unsplit = 0;
  for (int n = 1; n <= 32 && (n == 1 || n * 4 <= stages); n *= 2) {
    for (int k = 0; k < nk; ++k) {
      const Kind& c = kinds[k];
      const double tiles = (double)((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
      const double on_cu = std::ceil(tiles * n / 256.0), run = (double)((stages + n - 1) / n) * p.passes;
      double us = std::fmax(c.latency, on_cu * c.share) * run + on_cu * c.fixed + 3.0;
      if (n > 1) us += 2.0 + (2.0 * n * M * N * 4.0) / 6e6;
      if (us < best.us && (n == 1 || us < 0.92 * unsplit)) best = Tiling{c.bm, c.bn, n, us};
    }
    if (n == 1) unsplit = best.us;
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

// Side of the tiles with which both products of a backward pass take one launch, which
// fills the card while the first one ends, or 0 where two launches are faster by the same
// model (the second one: 2 us).  Together | apart, with g and dbias: 1024 x 1024 -> 1024 in
// bf16 19.4 | 23.7 us (64-wide tiles), float32 44 | 52; 1024 x 2048 -> 2048 34 | 41 (128);
// 4096 x 2048 -> 2048 96 | 92.  A split reduction stays one, so that each gradient has the
// same bits alone as with the other.
int pair_tile(const Product& dx, const Product& dw, int dtype) {
  const Tiling x = choose_tiling(dtype, dx), w = choose_tiling(dtype, dw);
  if (x.splits > 1 || w.splits > 1) return 0;
  const Product &first = dx.K >= dw.K ? dx : dw, &second = dx.K >= dw.K ? dw : dx;
  const double run = (double)steps_of(first.K, dtype) * first.passes, run2 = (double)steps_of(second.K, dtype) * second.passes;
  int best = 0;
  double best_us = x.us + w.us + 2.0;
  const Kind* kinds = dtype == VB_F32 ? k32 + 1 : k16 + 2;
  for (int k = 0; k < 2; ++k) {
    const Kind& c = kinds[k];
    auto tiles = [&](const Product& p) { return (double)((p.M + c.bm - 1) / c.bm) * ((p.N + c.bn - 1) / c.bn); };
    const double n = tiles(first), n2 = tiles(second);
    double us;
    if (c.per_cu == 1) {
      us = list_time(n, run * c.share + c.fixed, n2, run2 * c.share + c.fixed) + 3.0;
    } else {  // a CU has its share of the steps and half a tile more; its tiles' ends overlap
      const double share = std::fmin(std::ceil(n / 256.0) * run + std::ceil(n2 / 256.0) * run2,
                                     (n * run + n2 * run2) / 256.0 + run / 2);
      us = std::fmax(c.latency * run, c.share * share) + c.fixed * std::ceil((n + n2) / 256.0) + 3.0;
    }
    if (us < best_us) best_us = us, best = c.bm;
  }
  return best;
}

size_t tiling_bytes(const Tiling& t, long long M, int N) {
  return t.splits > 1 ? (size_t)t.splits * M * ((N + 3) / 4 * 4) * 4 : 0;
}

// Up to 16 rows, and up to 32 where the weights are few (24 x 1024 -> 1024 in bf16: 5.2
// against 7.7 us; 24 x 4096 -> 4096: 14.7 against 13.2) or long and many (32 x 4096 ->
// 16384: 34 against 37, float32 63 against 72; 32 x 1024 -> 65536: 36 against 31).
bool product_is_narrow(const Product& p, int dtype) {
  if (p.across_a || p.across_b) return false;
  const long long row = p.K * (long long)elem_size(dtype);
  return p.M <= 16 || (p.M <= 32 && (p.N * row <= 8 << 20 || (p.N >= 12800 && row >= 8192)));
}

size_t product_bytes(const Product& p, int dtype) {
  if (product_is_narrow(p, dtype)) return 0;
  return tiling_bytes(choose_tiling(dtype, p), p.M, p.N);
}

hipError_t launch_product(const Product& p, int dtype, hipStream_t st) {
  if (product_is_narrow(p, dtype)) {
    if (dtype == VB_F32) return launch_narrow<float>(p, st);
    if (dtype == VB_BF16) return launch_narrow<bf16>(p, st);
    return launch_narrow<f16>(p, st);
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

hipError_t launch_column_sums(const ColumnSums& s, int dtype, hipStream_t st) {
  const unsigned blocks = (s.n + 63) / 64;
  if (dtype == VB_F32) column_sum_kernel<float><<<blocks, 1024, 0, st>>>(s);
  else if (dtype == VB_BF16) column_sum_kernel<bf16><<<blocks, 1024, 0, st>>>(s);
  else column_sum_kernel<f16><<<blocks, 1024, 0, st>>>(s);
  return hipGetLastError();
}

hipError_t launch_pair(const Product& dx, const Product& dw, int tile, const ColumnSums& s, int dtype, hipStream_t st) {
  if (dtype == VB_F32) return launch_pair_typed<float>(dx, dw, tile, s, st);
  if (dtype == VB_BF16) return launch_pair_typed<bf16>(dx, dw, tile, s, st);
  return launch_pair_typed<f16>(dx, dw, tile, s, st);
}

hipError_t launch_fill_zero(void* p, long long rows, long long row_bytes, long long ld_bytes, hipStream_t st) {
  const long long n = row_bytes / 2;
  const long long blocks = (rows * n + 255) / 256;
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  fill_zero_kernel<<<grid_of(blocks), 256, 0, st>>>((unsigned short*)p, rows, n, ld_bytes / 2);
  return hipGetLastError();
}

}  // namespace vb
