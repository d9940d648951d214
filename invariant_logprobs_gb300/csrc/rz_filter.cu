// rz_filter.cu -- sampling under temperature, top-k, top-p and min-p from a
// given uniform per row, with the kept set and log mu of the token.
//
// What is kept is a head of the row's order (logits descending, ties by the
// lowest index), so three cuts give three heads and the shortest is kept:
// every test is "key > t, or key = t and index <= i" with the logit's bits as
// an ordered 32-bit key.  Top-k's t is found by its count, top-p's by its
// mass, 8 bits of the key at a time; the masses are the 64-bit integers of
// rz_fixexp.cuh, whose sums come out the same in every order, so the atomics
// below change nothing from run to run and every decision is that of exact
// arithmetic.
#include <cuda_runtime.h>

#include <cstdint>

#include "rz.h"
#include "rz_fixexp.cuh"
#include "rz_internal.h"
#include "rz_keep.cuh"

namespace rz {
namespace {

constexpr int kFilterThreads = 1024;
constexpr int kFilterWarps = kFilterThreads / 32;

__device__ const FixTable g_fix_table = make_fix_table();

struct FilterArgs {
  const void* logits;
  long long ld;
  const float* temperature;
  const int32_t* top_k;
  const float *top_p, *min_p, *uniform;
  int32_t* tokens;
  float* logprob;
  int32_t* kept;
  uint32_t* keep;
  int* err;
  int V, words, chunks, fix_bits;
};

// Order of the logits as unsigned integers; -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t u = __float_as_uint(__fadd_rn(z, 0.f));
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // order_key(-inf)

// The kept head: key > t, or key = t and index <= last.
struct Cut {
  uint32_t t;
  int last;
  __device__ __forceinline__ bool has(float z, int v) const {
    const uint32_t k = order_key(z);
    return k > t || (k == t && v <= last);
  }
};
struct CutKept {
  Cut cut;
  int V;
  __device__ __forceinline__ uint32_t before(int) const { return 0xffu; }
  __device__ __forceinline__ uint32_t after(int col, const float (&v)[8], uint32_t) const {
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < V && cut.has(v[i], col + i)) bits |= 1u << i;
    return bits;
  }
};

// x * (f * 2^64) / 2^64, floor, for a float 0 <= f < 1; *exact = no remainder.
__device__ __forceinline__ uint64_t mul_frac(uint64_t x, float f, bool* exact) {
  const uint64_t m = static_cast<uint64_t>(static_cast<double>(f) * 18446744073709551616.0);
  *exact = x * m == 0;
  return __umul64hi(x, m);
}

struct FilterShared {
  uint64_t table[kFixTable];
  uint32_t count[256], lo[256], hi[256];
  uint64_t red[kFilterWarps];
  float redf[kFilterWarps];
  uint32_t digit;
  uint64_t above;  // count or mass above the digit
  uint64_t target;
  FixScale scale;
  int bad, last, n, warp;
  uint64_t rest;
};

__device__ __forceinline__ uint64_t block_sum(FilterShared& s, uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = x;
  __syncthreads();
  uint64_t t = 0;
  for (int w = 0; w < kFilterWarps; ++w) t += s.red[w];
  return t;
}

// The largest key t with (count or mass of the keys >= t) >= target, and what
// lies above t.  Only elements with key >= floor take part.
template <class E, bool kMass>
__device__ void select(FilterShared& s, const E* z, int V, uint32_t floor, uint64_t target,
                       uint32_t& t_out, uint64_t& above_out) {
  uint32_t prefix = 0;
  uint64_t above = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kFilterThreads) s.count[i] = s.lo[i] = s.hi[i] = 0;
    __syncthreads();
    for (int v = threadIdx.x; v < V; v += kFilterThreads) {
      const float x = to_f32(z[v]);
      const uint32_t k = order_key(x);
      if (k < floor || (shift < 24 && (k >> (shift + 8)) != prefix)) continue;
      const uint32_t b = (k >> shift) & 255u;
      if (kMass) {
        const uint64_t w = fix_weight(s.scale, s.table, x);
        const uint32_t wl = static_cast<uint32_t>(w);
        const uint32_t old = atomicAdd(&s.lo[b], wl);
        atomicAdd(&s.hi[b], static_cast<uint32_t>(w >> 32) + (old + wl < old ? 1u : 0u));
      } else {
        atomicAdd(&s.count[b], 1u);
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      uint64_t a = above;
      int b = 255;
      for (; b > 0; --b) {
        const uint64_t x = kMass ? (static_cast<uint64_t>(s.hi[b]) << 32) + s.lo[b]
                                 : static_cast<uint64_t>(s.count[b]);
        if (a + x >= target) break;
        a += x;
      }
      s.digit = b;
      s.above = a;
    }
    __syncthreads();
    prefix = prefix << 8 | s.digit;
    above = s.above;
    __syncthreads();
  }
  t_out = prefix;
  above_out = above;
}

template <class E>
__global__ void __launch_bounds__(kFilterThreads) filter_sample_kernel(const FilterArgs a) {
  extern __shared__ uint8_t smem[];
  FilterShared& s = *reinterpret_cast<FilterShared*>(smem);
  float2* states = reinterpret_cast<float2*>(smem + (sizeof(FilterShared) + 15) / 16 * 16);
  const long long row = blockIdx.x;
  const E* z = static_cast<const E*>(a.logits) + row * a.ld;
  const int V = a.V;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* keep = a.keep ? a.keep + row * a.words : nullptr;

  // ---- the row's maximum, NaN and +inf
  float m = -INFINITY;
  bool nan = false;
  int finite = 0;
  for (int v = threadIdx.x; v < V; v += kFilterThreads) {
    const float x = to_f32(z[v]);
    nan |= !(x == x);
    finite += x > -INFINITY;
    m = fmaxf(m, x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s.redf[warp] = m;
  for (int i = threadIdx.x; i < kFixTable; i += kFilterThreads) s.table[i] = g_fix_table.v[i];
  const bool any_nan = __syncthreads_or(nan);
  const int n_finite = static_cast<int>(block_sum(s, finite));
  m = s.redf[0];
  for (int w = 1; w < kFilterWarps; ++w) m = fmaxf(m, s.redf[w]);

  float temperature = a.temperature ? a.temperature[row] : 1.f;
  const bool greedy = temperature == 0.f;
  const float tau = row_tau(a.temperature, row);
  const float u = a.uniform[row];
  const float p = a.top_p ? a.top_p[row] : 1.f;
  const float mp = a.min_p ? a.min_p[row] : 0.f;
  int k = a.top_k ? a.top_k[row] : 0;
  if (k <= 0 || k > n_finite) k = n_finite;
  if (greedy) k = 1;
  const bool bad_param = !(tau == tau) || !(u >= 0.f && u < 1.f) || !(p == p) || !(mp <= 1.f);
  const bool bad_row = any_nan || !(m < INFINITY) || n_finite == 0;
  if (bad_param || bad_row) {
    if (keep)
      for (int i = threadIdx.x; i < a.words; i += kFilterThreads) keep[i] = 0u;
    if (threadIdx.x == 0) {
      a.tokens[row] = -1;
      a.logprob[row] = __int_as_float(0x7fc00000);
      if (a.kept) a.kept[row] = 0;
      if (a.err)
        atomicOr(a.err, (bad_param ? RZ_DEVERR_PARAM : 0) | (bad_row ? RZ_DEVERR_LOGITS : 0));
    }
    return;
  }
  if (threadIdx.x == 0) {
    const double c = 1.44269504088896340736 / static_cast<double>(tau);
    s.scale.zmax = m;
    s.scale.c_hi = static_cast<float>(c);
    s.scale.c_lo = static_cast<float>(c - static_cast<double>(s.scale.c_hi));
    s.scale.drop = kFixQ - a.fix_bits;
  }
  __syncthreads();
  const FixScale scale = s.scale;

  // ---- the cuts: key > t, or one of the first `ties` at key = t
  uint32_t t = kKeyNegInf;
  long long ties = 0;
  if (k < n_finite) {
    uint64_t above;
    select<E, false>(s, z, V, 0u, k, t, above);
    ties = k - static_cast<long long>(above);
  }
  if (p < 1.f) {
    uint64_t total = 0;
    for (int v = threadIdx.x; v < V; v += kFilterThreads) {
      const float x = to_f32(z[v]);
      if (order_key(x) > t) total += fix_weight(scale, s.table, x);
    }
    total = block_sum(s, total);
    if (ties > 0) total += ties * fix_weight(scale, s.table, key_value(t));
    bool exact = true;
    uint64_t target = p > 0.f ? mul_frac(total, p, &exact) : 0;
    if (!exact || target == 0) ++target;  // a token is in while what lies above it < p * total
    uint32_t tp;
    uint64_t above;
    select<E, true>(s, z, V, ties > 0 ? t : t + 1, target, tp, above);
    const uint64_t w = fix_weight(scale, s.table, key_value(tp));
    long long n = w > 0 ? static_cast<long long>((target - above + w - 1) / w) : 1;
    if (tp == t && n > ties) n = ties;
    t = tp;
    ties = n;
  }
  if (mp > 0.f) {
    const float zmin = __double2float_ru(static_cast<double>(m) +
                                         static_cast<double>(tau) * log(static_cast<double>(mp)));
    const uint32_t km = order_key(zmin);
    if (km > t) {
      t = km - 1;
      ties = 0;
    }
  }

  // ---- the index of the last tie that is in
  const int seg = (V + 32 * kFilterWarps - 1) / (32 * kFilterWarps) * 32;
  const int v0 = warp * seg, v1 = min(V, v0 + seg);
  int last = -1;
  if (ties > 0) {
    int n = 0;
    for (int v = v0 + lane; v < v1; v += 32) n += order_key(to_f32(z[v])) == t;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    __syncthreads();
    if (lane == 0) s.red[warp] = n;
    if (threadIdx.x == 0) s.last = V - 1;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp; ++w) before += static_cast<long long>(s.red[w]);
    if (before < ties && before + n >= ties) {
      long long left = ties - before;  // the left-th tie of this warp's columns
      for (int v = v0; v < v1; v += 32) {
        const bool tie = v + lane < v1 && order_key(to_f32(z[v + lane])) == t;
        const uint32_t b = __ballot_sync(0xffffffffu, tie);
        if (left <= __popc(b)) {
          if (lane == 0) s.last = v + static_cast<int>(__fns(b, 0, static_cast<int>(left)));
          break;
        }
        left -= __popc(b);
      }
    }
    __syncthreads();
    last = s.last;
  }
  const Cut cut{t, last};

  // ---- kept mass of each warp's columns, the kept set's bits
  uint64_t mass = 0;
  int n = 0;
  for (int v = v0; v < v1; v += 32) {
    bool in = false;
    if (v + lane < v1) {
      const float x = to_f32(z[v + lane]);
      in = cut.has(x, v + lane);
      if (in) mass += fix_weight(scale, s.table, x);
    }
    const uint32_t b = __ballot_sync(0xffffffffu, in);
    n += __popc(b);
    if (keep && lane == 0) keep[v >> 5] = b;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
  __syncthreads();
  if (threadIdx.x == 0) {
    s.n = 0;
    s.rest = 0;
    s.warp = kFilterWarps;
  }
  if (lane == 0) s.red[warp] = mass;
  __syncthreads();
  // u = 0 is the first kept token whatever its weight rounds to
  const bool first = u == 0.f;
  if (lane == 0 && n) {
    atomicAdd(&s.n, n);
    if (first) atomicMin(&s.warp, warp);
  }
  if (threadIdx.x == 0 && !first) {
    uint64_t total = 0;
    for (int w = 0; w < kFilterWarps; ++w) total += s.red[w];
    bool exact;
    uint64_t r = mul_frac(total, u, &exact);  // the token: running sum > u * total
    int w = 0;
    while (w < kFilterWarps - 1 && r >= s.red[w]) r -= s.red[w++];
    s.warp = w;
    s.rest = r;
  }
  // ---- log-sum-exp over the kept columns, as the learner takes it
  const float c = keep_scale(tau);
  const bool vec = row_aligned(z);
  const CutKept kept{cut, V};
  for (int ch = warp; ch < a.chunks; ch += kFilterWarps) {
    const float2 st = keep_fold(z, vec, V, ch, c, kept);
    if (lane == 0) states[ch] = st;
  }
  __syncthreads();
  if (warp != s.warp) return;
  const float2 st = keep_merge(states, a.chunks, c);
  uint64_t r = s.rest;
  for (int v = v0; v < v1; v += 32) {
    uint64_t w = 0;
    float x = 0.f;
    if (v + lane < v1) {
      x = to_f32(z[v + lane]);
      if (cut.has(x, v + lane)) w = first ? 1 : fix_weight(scale, s.table, x);
    }
    uint64_t inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const uint32_t b = __ballot_sync(0xffffffffu, inc > r);
    if (b) {
      if (lane == __ffs(b) - 1) {
        a.tokens[row] = v + lane;
        a.logprob[row] = keep_logprob_of(x, st, tau);
        if (a.kept) a.kept[row] = s.n;
      }
      break;
    }
    r -= __shfl_sync(0xffffffffu, inc, 31);
  }
}

template <class E>
cudaError_t launch(const FilterArgs& a, int64_t T, cudaStream_t st) {
  const size_t smem = (sizeof(FilterShared) + 15) / 16 * 16 +
                      static_cast<size_t>(a.chunks) * sizeof(float2);
  cudaError_t e = cudaFuncSetAttribute(filter_sample_kernel<E>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 131072);
  if (e != cudaSuccess) return e;
  filter_sample_kernel<E><<<static_cast<unsigned>(T), kFilterThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace rz

using namespace rz;

extern "C" int rz_filter_sample(const void* logits, int64_t ld, int32_t dtype, int64_t T,
                                int32_t V, const float* temperature, const int32_t* top_k,
                                const float* top_p, const float* min_p, const float* uniform,
                                int32_t* tokens_out, float* logprob_out, int32_t* kept_out,
                                uint32_t* keep_out, int32_t* err_flag, rz_stream_t stream) {
  if (T < 0 || T >= (int64_t(1) << 31) - 1 || V < 1 || V > (1 << 24)) return RZ_ERR_INVALID_ARG;
  if (dtype != RZ_DTYPE_F32 && dtype != RZ_DTYPE_BF16 && dtype != RZ_DTYPE_F16)
    return RZ_ERR_INVALID_ARG;
  if (ld < V || (T > 0 && (!logits || !uniform || !tokens_out || !logprob_out)))
    return RZ_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == RZ_DTYPE_F32 ? 4 : 2) != 0)
    return RZ_ERR_UNSUPPORTED;
  if (T == 0) return RZ_OK;
  if (!device_ok()) return RZ_ERR_UNSUPPORTED;
  FilterArgs a{logits,     ld,          temperature, top_k,    top_p, min_p,
               uniform,    tokens_out,  logprob_out, kept_out, keep_out, err_flag,
               V, (V + 31) / 32, (V + kKeepChunk - 1) / kKeepChunk, fix_bits(V)};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(RZ_PROF_LOGITS_ROWS, 1, st);
  const cudaError_t e = dtype == RZ_DTYPE_F32    ? launch<float>(a, T, st)
                        : dtype == RZ_DTYPE_BF16 ? launch<__nv_bfloat16>(a, T, st)
                                                 : launch<__half>(a, T, st);
  return e == cudaSuccess ? RZ_OK : RZ_ERR_CUDA;
}
