// rz_fixexp.cuh -- e^((z - zmax) / tau) as a 64-bit integer, for sums that
// must come out the same in every order.
//
// With c = log2(e) / tau (as c_hi + c_lo, both fp32) and y = (zmax - z) c >= 0:
//   d = zmax - z rounded, e its exact rounding error  (Knuth's two-term sum)
//   y = p + q,  p = d c_hi rounded,  q = its error + d c_lo + e c_hi
//   p = k / 1024 + r,  k = round(1024 p),  |r + q| <= 2^-11
//   2^-y = 2^-(k >> 10) * 2^-((k & 1023) / 1024) * 2^-(r + q)
// the second factor from a table of 30 fractional bits, the third as 1 + g
// with a cubic in r + q (truncated terms below 2^-50) and g rounded to 2^-32.
// So the weight's relative error is about 2^-32, random from element to
// element: it moves a running sum over K tokens by 2^-32 sqrt(K) of one of
// them.  The rounding to 2^-Q at the end is to nearest (a truncation would take
// 2^-Q / 2 from each of a row's many small weights).  Some 30 fp32 and integer
// instructions; the part's fp64 units (two FMAs a clock on an SM) would take
// fifty times as long.  A table of 64-bit entries with 2^-45 takes twice the
// shared-memory cycles, which bound the pass.
#pragma once

#include <cmath>
#include <cstdint>

namespace rz {

constexpr int kFixTableBits = 10;
constexpr int kFixTable = 1 << kFixTableBits;
constexpr int kFixQ = 44;

struct FixTable {
  uint32_t v[kFixTable];
};

// 2^(-j/1024) by the exponential series, rounded to 30 fractional bits.
constexpr FixTable make_fix_table() {
  FixTable t{};
  for (int j = 0; j < kFixTable; ++j) {
    const double x = -0.69314718055994530942 * j / kFixTable;
    double s = 1.0;
    for (int n = 19; n >= 1; --n) s = 1.0 + x / n * s;
    t.v[j] = static_cast<uint32_t>(s * 1073741824.0 + 0.5);  // 2^30
  }
  return t;
}

// The vocabulary's sum of weights stays below 2^63: fractional bits Q of a
// weight, at most 44.
__host__ __device__ inline int fix_bits(int V) {
  int lg = 0;
  while ((1 << lg) < V) ++lg;
  return 62 - lg < kFixQ ? 62 - lg : kFixQ;
}

struct FixScale {
  float zmax, c_hi, c_lo;
  float none;  // Q + 2: a larger y weighs nothing
  int drop;    // 61 - Q
  __host__ __device__ void bits(int q) {
    none = static_cast<float>(q + 2);
    drop = 61 - q;
  }
};

__host__ __device__ __forceinline__ uint32_t fix_bits_of(float x) {
#ifdef __CUDA_ARCH__
  return __float_as_uint(x);
#else
  union {
    float f;
    uint32_t u;
  } b;
  b.f = x;
  return b.u;
#endif
}

// Sums and products rounded one by one: a contraction would lose the errors
// that the two-term forms carry.
__host__ __device__ __forceinline__ float fx_add(float a, float b) {
#ifdef __CUDA_ARCH__
  return __fadd_rn(a, b);
#else
  return a + b;
#endif
}
__host__ __device__ __forceinline__ float fx_sub(float a, float b) { return fx_add(a, -b); }
__host__ __device__ __forceinline__ float fx_mul(float a, float b) {
#ifdef __CUDA_ARCH__
  return __fmul_rn(a, b);
#else
  return a * b;
#endif
}

// z <= zmax finite or -inf; tab: the table (shared memory on the device).
__host__ __device__ __forceinline__ uint64_t fix_weight(const FixScale& s, const uint32_t* tab,
                                                        float z) {
  const float d = fx_sub(s.zmax, z);
  const float zz = fx_sub(s.zmax, d);  // the part of z that d accounts for
  const float e = fx_add(fx_sub(s.zmax, fx_add(d, zz)), fx_sub(zz, z));
  const float p = fx_mul(d, s.c_hi);
  const float pc = fminf(p, s.none);   // (what is beyond, and z = -inf, weighs 0 below)
  float q = fmaf(d, s.c_hi, -p);
  q = fmaf(d, s.c_lo, q);
  q = fmaf(e, s.c_hi, q);
  const float big = 12288.f;           // spacing of floats there: 2^-10
  const float pk = fx_add(pc, big);
  const uint32_t k = fix_bits_of(pk) - fix_bits_of(big);
  const float r = fx_add(fx_sub(pc, fx_sub(pk, big)), q);
  float t = fmaf(r, -0.055504109f, 0.24022651f);  // -(ln 2)^3/6, (ln 2)^2/2
  t = fmaf(t, r, -0.69314718f);
  const float g = fx_mul(t, r);
  const float one = 2.9296875e-3f;     // 1.5 * 2^-9: spacing 2^-32
  const int32_t gi = static_cast<int32_t>(fix_bits_of(fx_add(g, one)) - fix_bits_of(one));
  const uint32_t w = tab[k & (kFixTable - 1)];
  const uint64_t v = (static_cast<uint64_t>(w) << 32) +
                     static_cast<uint64_t>(static_cast<int64_t>(static_cast<int32_t>(w)) * gi);
  const uint64_t w1 = ((v >> ((k >> kFixTableBits) + s.drop)) + 1) >> 1;  // v: 62 fractional bits
  return p < s.none ? w1 : 0;  // (no branch: a lane's weights are evaluated side by side)
}

}  // namespace rz
