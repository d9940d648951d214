// rz_pages.cu -- block tables and the slot map of a paged cache, built on the
// GPU from the requests' lengths.
//
// Request i holds lens_i tokens in ceil(lens_i / p) pages and adds new_i:
//   need_i = ceil((lens_i + new_i) / p) - ceil(lens_i / p),
//   o_i    = sum_{j < i} need_j,  cu_i = sum_{j < i} new_j,
//   table[i, ceil(lens_i / p) + j] = free[o_i + j],
//   slot(cu_i + t) = table[i, (lens_i + t) / p] p + (lens_i + t) % p.
// The two sums need every earlier request.  Each block adds up all requests
// before its own (8 bytes each, from L2) instead of waiting for other blocks,
// so nothing spins and the blocks are independent.  A step's few slots are
// then written by the same block; an admission's many by a second kernel over
// the slots, where each finds its request by bisection of cu.
#include <cuda_runtime.h>

#include <cstdint>

#include "rz.h"
#include "rz_internal.h"
#include "rz_ptx.cuh"

namespace rz {
namespace {

constexpr int kPageThreads = 256;
constexpr int kPageWarps = kPageThreads / 32;
constexpr int kMaxPer = 1024;           // requests of one block at most
constexpr int64_t kFusedSlots = 16384;  // slots one block writes itself
constexpr int kSlotsPerBlock = 2048;

struct PageArgs {
  const int32_t *lens, *news, *free_pages;
  int32_t* table;
  int64_t *slots, *cu;
  int32_t* used;
  int* err;
  int64_t n_free, n_slots;
  int B, page, width, per;
};

struct Need {
  int len, add, old_pages, need;  // clamped length, tokens, pages held, pages to take
};

__device__ __forceinline__ Need need_of(const PageArgs& a, int i, bool& bad) {
  Need n;
  n.len = a.lens[i];
  n.add = a.news[i];
  if (n.len < 0 || n.add < 0) {
    bad = true;
    n.len = max(n.len, 0);
    n.add = max(n.add, 0);
  }
  const long long full = (static_cast<long long>(n.len) + n.add + a.page - 1) / a.page;
  const long long old = (static_cast<long long>(n.len) + a.page - 1) / a.page;
  if (full > a.width) bad = true;
  n.old_pages = static_cast<int>(old < a.width ? old : a.width);
  n.need = static_cast<int>(full < a.width ? full : a.width) - n.old_pages;
  return n;
}

// The slot of new token t of a request with `len` cached tokens; -1 where the
// row has no page for it.
__device__ __forceinline__ long long slot_of(const PageArgs& a, int i, int len, long long t,
                                             bool& bad) {
  const long long pos = len + t;
  const long long j = pos / a.page;
  if (j >= a.width) return -1;  // flagged with the row's pages
  const int page = a.table[static_cast<long long>(i) * a.width + j];
  if (page < 0) {
    bad = true;
    return -1;
  }
  return static_cast<long long>(page) * a.page + (pos - j * a.page);
}

__device__ __forceinline__ longlong2 block_sum2(longlong2 v, longlong2* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  longlong2 s = make_longlong2(0, 0);
#pragma unroll
  for (int w = 0; w < kPageWarps; ++w) {
    s.x += scratch[w].x;
    s.y += scratch[w].y;
  }
  __syncthreads();
  return s;
}

__global__ void __launch_bounds__(kPageThreads) page_table_kernel(const PageArgs a, bool fused) {
  __shared__ longlong2 scratch[kPageWarps];
  __shared__ long long s_first[kMaxPer], s_cu[kMaxPer + 1];
  const int begin = blockIdx.x * a.per;
  const int count = min(a.per, a.B - begin);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool bad = false;

  longlong2 before = make_longlong2(0, 0);
  if (begin > 0) {
    for (int i = threadIdx.x; i < begin; i += kPageThreads) {
      const Need n = need_of(a, i, bad);
      before.x += n.need;
      before.y += n.add;
    }
    before = block_sum2(before, scratch);
  }
  // exclusive sums of the block's own requests, a round of threads at a time
  for (int r = 0; r < count; r += kPageThreads) {
    const int i = r + threadIdx.x;
    longlong2 v = make_longlong2(0, 0);
    if (i < count) {
      const Need n = need_of(a, begin + i, bad);
      v = make_longlong2(n.need, n.add);
    }
    longlong2 inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc.x, o);
      const long long y = __shfl_up_sync(0xffffffffu, inc.y, o);
      if (lane >= o) {
        inc.x += x;
        inc.y += y;
      }
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    longlong2 base = before;
    for (int w = 0; w < kPageWarps; ++w) {
      if (w < warp) {
        base.x += scratch[w].x;
        base.y += scratch[w].y;
      }
      before.x += scratch[w].x;
      before.y += scratch[w].y;
    }
    if (i < count) {
      s_first[i] = base.x + inc.x - v.x;
      s_cu[i] = base.y + inc.y - v.y;
      a.cu[begin + i] = s_cu[i];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    s_cu[count] = before.y;
    if (begin + count == a.B) {
      a.cu[a.B] = before.y;
      *a.used = static_cast<int32_t>(before.x < 0x7fffffffLL ? before.x : 0x7fffffffLL);
      if (before.y > a.n_slots) bad = true;
    }
  }
  __syncthreads();

  // new table entries, a warp per request
  for (int i = warp; i < count; i += kPageWarps) {
    const Need n = need_of(a, begin + i, bad);
    int32_t* row = a.table + static_cast<long long>(begin + i) * a.width + n.old_pages;
    for (int j = lane; j < n.need; j += 32) {
      const long long f = s_first[i] + j;
      if (f >= a.n_free) bad = true;
      row[j] = f < a.n_free ? a.free_pages[f] : -1;
    }
  }
  if (fused) {
    __syncthreads();  // the block wrote every entry that its slots read
    const long long total = s_cu[count];
    for (long long t = threadIdx.x; t < a.n_slots; t += kPageThreads) {
      long long slot = -1;
      if (t < total) {
        int lo = 0, hi = count;  // the last i with cu_i <= t: cu[lo] <= t < cu[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_cu[mid] <= t) lo = mid;
          else hi = mid;
        }
        slot = slot_of(a, begin + lo, max(a.lens[begin + lo], 0), t - s_cu[lo], bad);
      }
      a.slots[t] = slot;
    }
  }
  if (bad && a.err) atomicOr(a.err, RZ_DEVERR_PAGES);
}

__global__ void __launch_bounds__(kPageThreads) page_slot_kernel(const PageArgs a) {
  __shared__ int s_range[2];
  const long long t0 = static_cast<long long>(blockIdx.x) * kSlotsPerBlock;
  const long long t1 = min(t0 + kSlotsPerBlock, static_cast<long long>(a.n_slots));
  bool bad = false;
  // the requests of the block's first and last slot bound every bisection
  if (threadIdx.x < 2) {
    const long long t = threadIdx.x == 0 ? t0 : t1 - 1;
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    s_range[threadIdx.x] = lo;
  }
  __syncthreads();
  const long long total = a.cu[a.B];
  for (long long t = t0 + threadIdx.x; t < t1; t += kPageThreads) {
    long long slot = -1;
    if (t < total) {
      int lo = s_range[0], hi = s_range[1] + 1;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= t) lo = mid;
        else hi = mid;
      }
      slot = slot_of(a, lo, max(a.lens[lo], 0), t - a.cu[lo], bad);
    }
    a.slots[t] = slot;
  }
  if (bad && a.err) atomicOr(a.err, RZ_DEVERR_PAGES);
}

}  // namespace
}  // namespace rz

using namespace rz;

extern "C" int rz_page_tables(const int32_t* lens, const int32_t* new_lens, int32_t B,
                              const int32_t* free_pages, int64_t n_free, int32_t page_size,
                              int32_t* table, int32_t width, int64_t* slots_out, int64_t n_slots,
                              int64_t* cu_out, int32_t* used_out, int32_t* err_flag,
                              rz_stream_t stream) {
  if (B < 0 || n_free < 0 || n_slots < 0 || page_size < 1 || width < 1) return RZ_ERR_INVALID_ARG;
  if (static_cast<int64_t>(B) * width >= (int64_t(1) << 31) || n_slots >= (int64_t(1) << 40))
    return RZ_ERR_INVALID_ARG;
  if (!cu_out || !used_out || (n_slots > 0 && !slots_out)) return RZ_ERR_INVALID_ARG;
  if (B > 0 && (!lens || !new_lens || !table)) return RZ_ERR_INVALID_ARG;
  if (n_free > 0 && !free_pages) return RZ_ERR_INVALID_ARG;
  if (!device_ok()) return RZ_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  PageArgs a{lens, new_lens, free_pages, table, slots_out, cu_out, used_out, err_flag,
             n_free, n_slots, B, page_size, width, kMaxPer};
  const bool fused = B <= kMaxPer && n_slots <= kFusedSlots;
  if (!fused) {
    // about one block an SM; a block adds up what comes before it, so small
    // batches take few requests a block and large ones few blocks
    a.per = 64;
    while (a.per < kMaxPer && static_cast<int64_t>(a.per) * num_sms() < B) a.per *= 2;
  }
  const int blocks = B > 0 ? (B + a.per - 1) / a.per : 1;
  ProfScope ps(RZ_PROF_SMALL, fused ? 1 : 2, st);
  page_table_kernel<<<blocks, kPageThreads, 0, st>>>(a, fused);
  if (!fused && n_slots > 0) {
    const int64_t nb = (n_slots + kSlotsPerBlock - 1) / kSlotsPerBlock;
    page_slot_kernel<<<static_cast<unsigned>(nb), kPageThreads, 0, st>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? RZ_OK : RZ_ERR_CUDA;
}
