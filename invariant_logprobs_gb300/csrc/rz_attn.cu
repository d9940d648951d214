// rz_attn.cu -- decode attention of response groups over a paged cache: one
// query token per request, over its prompt's shared pages and its own.
//
//   s_j = scale q . k_j,  out = sum_j e^(s_j - lse) v_j,  lse = log sum_j e^(s_j).
//
// One pass over the tokens with a running maximum m, sum l and output o per
// query row:  m' = max(m, s_j),  l' = l e^(m - m') + e^(s_j - m'),  o likewise.
// One block per (request, query head); its warps take tokens in turn.
#include <cuda_runtime.h>

#include <cstdint>

#include "rz.h"
#include "rz_internal.h"
#include "rz_keep.cuh"

namespace rz {
namespace {

constexpr int kAttnThreads = 128;
constexpr int kAttnWarps = kAttnThreads / 32;
constexpr int kMaxD = 128;

struct AttnArgs {
  const void *q, *k, *v;
  long long qs[2], ks[3], vs[3];
  const int32_t *prefix_table, *prefix_lens, *cu_group, *table, *lens;
  void* out;
  float* lse;
  int* err;
  float scale;  // times log2 e
  int n_pages, page, prefix_width, P, width, B, Hq, Hkv, D;
};

template <class E>
__global__ void __launch_bounds__(kAttnThreads) attn_kernel(const AttnArgs a) {
  __shared__ float so[kAttnWarps][kMaxD], sm[kAttnWarps], sl[kAttnWarps];
  const int b = blockIdx.x, h = blockIdx.y;
  const int hk = h / (a.Hq / a.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int bad = 0;
  // the prompt of request b: the last g with cu[g] <= b < cu[g+1]
  // (offsets cut to 0 <= cu[0] <= ... <= B)
  int g = -1, lo = 0;
  for (int i = 0; i <= a.P && a.P > 0; ++i) {
    const int cu = a.cu_group[i];
    const int hi = min(max(cu, lo), a.B);
    if (hi != cu) bad |= RZ_DEVERR_CU_SEQLENS;
    if (i > 0 && lo <= b && b < hi) g = i - 1;
    lo = hi;
  }
  const E* q = static_cast<const E*>(a.q) + b * a.qs[0] + h * a.qs[1];
  float qv[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) qv[i] = lane + 32 * i < a.D ? to_f32(q[lane + 32 * i]) : 0.f;
  for (int part = 0; part < 2; ++part) {
    if (part == 0 && g < 0) continue;
    const int32_t* tab = part == 0 ? a.prefix_table + static_cast<long long>(g) * a.prefix_width
                                   : a.table + static_cast<long long>(b) * a.width;
    const long long room = static_cast<long long>(part == 0 ? a.prefix_width : a.width) * a.page;
    long long n = part == 0 ? a.prefix_lens[g] : a.lens[b];
    if (n < 0 || n > room) {
      bad |= RZ_DEVERR_PAGES;
      n = n < 0 ? 0 : room;
    }
    for (long long t = warp; t < n; t += kAttnWarps) {
      const long long j = t / a.page;
      const int pg = tab[j];
      if (pg < 0 || pg >= a.n_pages) {
        bad |= RZ_DEVERR_PAGES;
        continue;
      }
      const E* k = static_cast<const E*>(a.k) + pg * a.ks[0] + (t - j * a.page) * a.ks[1] + hk * a.ks[2];
      const E* v = static_cast<const E*>(a.v) + pg * a.vs[0] + (t - j * a.page) * a.vs[1] + hk * a.vs[2];
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < a.D) s = fmaf(qv[i], to_f32(k[lane + 32 * i]), s);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      s *= a.scale;
      const float mn = fmaxf(m, s);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m - ref), e = exp2f(s - ref);
      l = l * f + e;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i] *= f;
        if (lane + 32 * i < a.D) o[i] = fmaf(e, to_f32(v[lane + 32 * i]), o[i]);
      }
      m = mn;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) so[warp][lane + 32 * i] = o[i];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  if (bad && lane == 0 && a.err) atomicOr(a.err, bad);
  __syncthreads();
  float M = -INFINITY, L = 0.f, x = 0.f;
  for (int w = 0; w < kAttnWarps; ++w) M = fmaxf(M, sm[w]);
  const float ref = M == -INFINITY ? 0.f : M;
  const int d = threadIdx.x;
  for (int w = 0; w < kAttnWarps; ++w) {
    const float f = exp2f(sm[w] - ref);
    L += sl[w] * f;
    x += so[w][d] * f;
  }
  const long long r = static_cast<long long>(b) * a.Hq + h;
  if (d < a.D) {
    const float y = L > 0.f ? x / L : (L == 0.f ? 0.f : L);
    E* out = static_cast<E*>(a.out) + r * a.D + d;
    if (sizeof(E) == 2) *out = static_cast<E>(y);
  }
  if (d == 0 && a.lse) a.lse[r] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

}  // namespace
}  // namespace rz

using namespace rz;

extern "C" int rz_group_decode_attn(const void* q, const int64_t* q_stride, const void* k_cache,
                                    const void* v_cache, const int64_t* kv_stride,
                                    int32_t n_pages, int32_t page_size,
                                    const int32_t* prefix_table, int32_t prefix_width,
                                    const int32_t* prefix_lens, const int32_t* cu_group,
                                    int32_t P, const int32_t* table, int32_t width,
                                    const int32_t* lens, int32_t B, int32_t Hq, int32_t Hkv,
                                    int32_t D, int32_t dtype, float scale, void* out,
                                    float* lse_out, void* ws, size_t ws_bytes, int32_t* err_flag,
                                    rz_stream_t stream) {
  if (B < 0 || P < 0 || n_pages < 0 || page_size < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0)
    return RZ_ERR_INVALID_ARG;
  if (width < 0 || prefix_width < 0 || !(scale == scale)) return RZ_ERR_INVALID_ARG;
  if (dtype != RZ_DTYPE_BF16 && dtype != RZ_DTYPE_F16) return RZ_ERR_INVALID_ARG;
  if (P > 0 && (!prefix_table || !prefix_lens || !cu_group)) return RZ_ERR_INVALID_ARG;
  if (B > 0 && (!q || !q_stride || !kv_stride || !table || !lens || !out))
    return RZ_ERR_INVALID_ARG;
  if (B > 0 && n_pages > 0 && (!k_cache || !v_cache)) return RZ_ERR_INVALID_ARG;
  if (D < 8 || D > kMaxD || D % 8 != 0 || Hq / Hkv > 128) return RZ_ERR_UNSUPPORTED;
  if (B == 0) return RZ_OK;
  for (int i = 0; i < 6; ++i)
    if (kv_stride[i] % 8 != 0) return RZ_ERR_UNSUPPORTED;
  if (q_stride[0] % 8 != 0 || q_stride[1] % 8 != 0) return RZ_ERR_UNSUPPORTED;
  if (!a16(q) || !a16(k_cache) || !a16(v_cache) || !a16(out)) return RZ_ERR_UNSUPPORTED;
  const size_t need = rz_workspace_size(RZ_OP_GROUP_DECODE_ATTN, B, D, Hq, P);
  if (need > 0 && (!ws || ws_bytes < need || !a256(ws))) return RZ_ERR_WORKSPACE;
  if (!device_ok()) return RZ_ERR_UNSUPPORTED;
  AttnArgs a{};
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  for (int i = 0; i < 2; ++i) a.qs[i] = q_stride[i];
  for (int i = 0; i < 3; ++i) {
    a.ks[i] = kv_stride[i];
    a.vs[i] = kv_stride[3 + i];
  }
  a.prefix_table = prefix_table;
  a.prefix_lens = prefix_lens;
  a.cu_group = cu_group;
  a.table = table;
  a.lens = lens;
  a.out = out;
  a.lse = lse_out;
  a.err = err_flag;
  a.scale = scale * kLog2e;
  a.n_pages = n_pages;
  a.page = page_size;
  a.prefix_width = prefix_width;
  a.P = P;
  a.width = width;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(RZ_PROF_SMALL, 1, st);
  if (dtype == RZ_DTYPE_BF16)
    attn_kernel<__nv_bfloat16><<<dim3(B, Hq), kAttnThreads, 0, st>>>(a);
  else
    attn_kernel<__half><<<dim3(B, Hq), kAttnThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? RZ_OK : RZ_ERR_CUDA;
}
