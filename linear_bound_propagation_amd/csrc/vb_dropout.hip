// Dropout with a mask from a counter-based generator.
//
// The mask is computed where it is used: seven rounds of Philox4x32 give four words, one per
// element, so that a pass moves x (and the residual) in and y out and nothing else.  A round is
// two 32 x 32 -> 64 bit products; a chunk of eight 16-bit elements takes 28 of them, which
// fits under its memory accesses (2^26 bf16 numbers, flat: 44.7 us, 6.0 TB/s, a plain copy 45.8;
// with ten rounds 63.7 us).  So HBM bounds it: 8192 x 4096 in bf16 27 us, 5.0 TB/s, as a large
// copy; 8192 x 8192 with a residual 71 us, 5.6 TB/s.  One chunk per thread: two or four gave 4.9
// and 5.3 TB/s of the flat case's 6.0.
#include <cmath>

#include "vb_train_device.h"
#include "vb_train_internal.h"

namespace vb {

namespace {

// Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3 (2011).
__device__ __forceinline__ void philox(uint64_t low, uint64_t high, uint64_t key, unsigned (&word)[4]) {
  unsigned c0 = (unsigned)low, c1 = (unsigned)(low >> 32), c2 = (unsigned)high, c3 = (unsigned)(high >> 32);
  unsigned k0 = (unsigned)key, k1 = (unsigned)(key >> 32);
#pragma unroll
  for (int round = 0; round < 7; ++round) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (unsigned)(b >> 32) ^ c1 ^ k0;
    c2 = (unsigned)(a >> 32) ^ c3 ^ k1;
    c1 = (unsigned)b, c3 = (unsigned)a;
    k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
  }
  word[0] = c0, word[1] = c1, word[2] = c2, word[3] = c3;
}

struct Dropout {
  vb_dropout_args p;
  unsigned threshold;  // kept if the word is no less,
  bool none;           // and not all are dropped
  float scale;
  int lanes;           // lanes of a row in a workgroup, a power of two
  unsigned across;     // workgroups of a row
  unsigned blocks;
};

// A thread has a chunk of 16 bytes: 256 / lanes rows of a workgroup side by side.
template <typename T>
__global__ __launch_bounds__(256) void dropout_kernel(Dropout d) {
  constexpr int EC = 16 / sizeof(T);
  typedef T V __attribute__((ext_vector_type(16 / sizeof(T))));
  typedef V LV __attribute__((aligned(sizeof(T))));
  const vb_dropout_args& p = d.p;
  const unsigned block = workgroup_number();
  if (block >= d.blocks) return;  // the whole workgroup
  const unsigned by = block / d.across, bx = block - by * d.across;
  const long long r = (long long)by * (256 / d.lanes) + threadIdx.x / d.lanes;
  const long long c0 = ((long long)bx * d.lanes + (threadIdx.x & (d.lanes - 1))) * EC;
  if (r >= p.rows || c0 >= p.n) return;
  const T* x = (const T*)p.x + r * p.ld_x + c0;
  const T* res = p.residual ? (const T*)p.residual + r * p.ld_res + c0 : nullptr;
  T* y = (T*)p.y + r * p.ld_y + c0;
  const uint64_t offset = p.offset + (p.step ? *p.step : 0);
  const int have = (int)min((long long)EC, p.n - c0);
  V xv, rv{};
  if (have == EC) {
    xv = *(const LV*)x;
    if (res) rv = *(const LV*)res;
  } else {
#pragma unroll
    for (int e = 0; e < EC; ++e) {
      xv[e] = e < have ? x[e] : (T)0.f;
      if (res) rv[e] = e < have ? res[e] : (T)0.f;
    }
  }
  V o;
  const uint64_t quad = (uint64_t)r * ((p.n + 3LL) / 4) + (uint64_t)c0 / 4;
#pragma unroll
  for (int q = 0; q < EC / 4; ++q) {
    unsigned word[4];
    philox(quad + q, offset, p.seed, word);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = to_f32((T)xv[q * 4 + e]) * d.scale;
      const bool keep = word[e] >= d.threshold && !d.none;
      o[q * 4 + e] = from_f32<T>(res ? to_f32((T)rv[q * 4 + e]) + (keep ? v : 0.f) : keep ? v : 0.f);
    }
  }
  if (have == EC) {
    *(LV*)y = o;
  } else {
#pragma unroll
    for (int e = 0; e < EC; ++e)
      if (e < have) y[e] = o[e];
  }
}

template <typename T>
hipError_t launch_typed(Dropout d, hipStream_t st) {
  constexpr int EC = 16 / sizeof(T);
  const long long chunks = (d.p.n + (long long)EC - 1) / EC;
  d.lanes = 1;
  while (d.lanes < 256 && d.lanes < chunks) d.lanes *= 2;
  const long long across = (chunks + d.lanes - 1) / d.lanes, per = 256 / d.lanes;
  const long long blocks = (d.p.rows + per - 1) / per * across;
  if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
  d.across = (unsigned)across, d.blocks = (unsigned)blocks;
  dropout_kernel<T><<<grid_of(blocks), 256, 0, st>>>(d);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const vb_dropout_args& p, hipStream_t st) {
  Dropout d{};
  d.p = p;
  const uint64_t drop = (uint64_t)std::nearbyint(p.p * 4294967296.), whole = UINT64_C(1) << 32;
  d.none = drop >= whole;
  d.threshold = (unsigned)drop;
  d.scale = d.none ? 0.f : (float)(4294967296. / (double)(whole - drop));
  if (p.dtype == VB_F32) return launch_typed<float>(d, st);
  if (p.dtype == VB_BF16) return launch_typed<bf16>(d, st);
  return launch_typed<f16>(d, st);
}

}  // namespace vb
