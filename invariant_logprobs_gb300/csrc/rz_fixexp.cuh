// rz_fixexp.cuh -- e^((z - zmax) / tau) as a 64-bit integer, for sums that
// must come out the same in every order.
//
// With c = log2(e) / tau (as c_hi + c_lo, both fp32) and y = (zmax - z) c >= 0,
//   y = k / 1024 + r,  |r| <= 2^-10,
//   2^-y = 2^-(k >> 10) * 2^-((k & 1023) / 1024) * 2^-r:
// the second factor from a table of 30 fractional bits, the third as 1 + g with
// a cubic in r (truncated terms below 2^-46) and g rounded to 2^-32.
//
// k and r come from x c for x = z and x = zmax alike: h = x c_hi to the next
// 1/1024 (by adding 1.5 * 2^13, whose neighbours are 2^-10 apart), l = the rest
// of x c, one FMA for x c_hi - h and one for + x c_lo; then k = h_max - h as
// integers and r = l_max - l, with errors of 2^-34.  That holds while |x c| <
// 4096; z is taken no lower than zmax - (Q + 2.5) / c, below which it weighs
// nothing.  For a larger |zmax| c the difference d = zmax - z is formed first, with
// its exact rounding error e (Knuth's two-term sum), and y = d c + e c split.
//
// So the weight's relative error is about 2^-31, random from element to
// element: it moves a running sum over K tokens by 2^-31 sqrt(K) of one of
// them.  The rounding to 2^-Q at the end is to nearest (a truncation would take
// 2^-Q / 2 from each of a row's many small weights).  Some 30 fp32 and integer
// instructions; the part's fp64 units (two FMAs a clock on an SM) would take
// fifty times as long.  A table of 64-bit entries with 2^-45 takes twice the
// shared-memory cycles.
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

constexpr float kFixBig = 12288.f;  // 1.5 * 2^13

struct FixScale {
  float zmax, c_hi, c_lo;
  float floor;    // the least z that is told apart
  float l_max;    // the rest of zmax c
  uint32_t h_max; // zmax c to 1/1024, as the bits of that + kFixBig
  float none;     // Q + 2.5
  int drop;       // 61 - Q
  bool big;       // |zmax| c is too large for the direct split

  __host__ __device__ void init(float zmax_, float hi, float lo, int q) {
    zmax = zmax_;
    c_hi = hi;
    c_lo = lo;
    none = static_cast<float>(q) + 2.5f;
    drop = 61 - q;
    big = !(fx_mul(zmax < 0 ? -zmax : zmax, hi) < 4000.f);
    floor = fx_sub(zmax, none / hi);
    const float h = fmaf(zmax, c_hi, kFixBig);
    h_max = fix_bits_of(h);
    l_max = fmaf(zmax, c_lo, fmaf(zmax, c_hi, -fx_sub(h, kFixBig)));
  }
};

// The steps k and the rest r of y; z <= zmax finite or -inf.  kBig: for a scale
// that is big (a loop has it apart: a branch at each logit would keep a lane's
// evaluations from overlapping).
template <bool kBig>
__host__ __device__ __forceinline__ uint32_t fix_steps(const FixScale& s, float z, float& r) {
  if (!kBig) {
    const float x = fmaxf(z, s.floor);
    const float h = fmaf(x, s.c_hi, kFixBig);
    r = fx_sub(s.l_max, fmaf(x, s.c_lo, fmaf(x, s.c_hi, -fx_sub(h, kFixBig))));
    return s.h_max - fix_bits_of(h);
  }
  const float d = fx_sub(s.zmax, z);
  const float zz = fx_sub(s.zmax, d);  // the part of z that d accounts for
  const float e = fx_add(fx_sub(s.zmax, fx_add(d, zz)), fx_sub(zz, z));
  const float p = fx_mul(d, s.c_hi);
  if (!(p < s.none)) {                 // (and z = -inf)
    r = 0.f;
    return static_cast<uint32_t>(s.none * kFixTable);
  }
  const float q = fmaf(e, s.c_hi, fmaf(d, s.c_lo, fmaf(d, s.c_hi, -p)));
  const float h = fx_add(p, kFixBig);
  r = fx_add(fx_sub(p, fx_sub(h, kFixBig)), q);
  return fix_bits_of(h) - fix_bits_of(kFixBig);
}

// tab: the table (shared memory on the device).
__host__ __device__ __forceinline__ uint64_t fix_weight_at(const FixScale& s, const uint32_t* tab,
                                                           uint32_t k, float r) {
  float t = fmaf(r, -0.055504109f, 0.24022651f);  // -(ln 2)^3/6, (ln 2)^2/2
  t = fmaf(t, r, -0.69314718f);
  const float one = 2.9296875e-3f;     // 1.5 * 2^-9: spacing 2^-32
  const int32_t gi = static_cast<int32_t>(fix_bits_of(fmaf(t, r, one)) - fix_bits_of(one));
  const uint32_t w = tab[k & (kFixTable - 1)];
  const uint64_t v = (static_cast<uint64_t>(w) << 32) +
                     static_cast<uint64_t>(static_cast<int64_t>(static_cast<int32_t>(w)) * gi);
  return ((v >> ((k >> kFixTableBits) + s.drop)) + 1) >> 1;  // v: 62 fractional bits
}
__host__ __device__ __forceinline__ uint64_t fix_weight(const FixScale& s, const uint32_t* tab,
                                                        float z) {
  float r;
  const uint32_t k = s.big ? fix_steps<true>(s, z, r) : fix_steps<false>(s, z, r);
  return fix_weight_at(s, tab, k, r);
}

}  // namespace rz
