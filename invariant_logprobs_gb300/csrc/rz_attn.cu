// rz_attn.cu -- decode attention of response groups over a paged cache: one
// query token per request, over its prompt's shared pages and its own.
//
//   s_j = scale q . k_j,  out = sum_j e^(s_j - lse) v_j,  lse = log sum_j e^(s_j).
//
// Two kinds of items: a prompt's shared tokens with up to 128 query rows of
// one KV head (all the group's requests times the query heads of that KV
// head), and a request's own tokens with the query heads of one KV head.  An
// item's tokens come in tiles of 128; all items' tiles form one line that is
// cut into equal runs, one run per SM, so ragged groups balance without a
// host plan.  Where a run begins or ends inside an item, the item's result is
// in parts: each part is (m, l, O) with O = sum 2^(x_j - m) v_j,
// l = sum 2^(x_j - m), x = s log2 e, and the parts of a row are joined by
//   M = max m,  out = sum 2^(m - M) O / sum 2^(m - M) l.
//
// Three launches: plan_kernel (clean lengths, where each entry's tiles begin),
// attn_kernel (one persistent CTA per SM), join_kernel (a warp per query row).
//
// attn_kernel, per tile: S = Q K^T (128 rows x 128 tokens, tcgen05, fp32 in
// TMEM), the softmax terms P in 16 bits back into TMEM, O += P V with P as
// the TMEM operand.
//   warps 0-3  softmax: thread = query row = TMEM lane, so maximum, sum and
//              the rescaling of O need no exchange between threads.  The
//              reference m moves only when a row's maximum has grown by more
//              than 8 (a factor 2^8, far inside fp32's and fp16's range), so
//              O is rarely rescaled.  Warps without rows only keep step.
//   warps 4-7  loads: 16-byte asynchronous copies, swizzled by address, which
//              take any page size and stride and zero what lies past the
//              length; the reads of six to seven tiles a CTA are in flight.
//   warp 8     TMEM owner and MMA issuer: S of tile j+1 before P V of tile j.
// A tile's K and V are 64 KB at 128 columns; at its share of the memory an SM
// takes 2,800 clocks for that, while the two products take 1,100 and the
// softmax of a full warp about 1,000: the memory is what bounds it, whatever
// the number of rows.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "rz.h"
#include "rz_internal.h"
#include "rz_keep.cuh"

namespace rz {
namespace {

constexpr int kTile = 128;      // tokens per tile, query rows per item
constexpr int kMaxD = 128;
constexpr int kMaxCtas = 152;   // persistent CTAs at most (workspace size)
constexpr int kSoftWarps = 4, kLoadWarps = 4;
constexpr int kMmaWarp = kSoftWarps + kLoadWarps;
constexpr int kAttnThreads = 32 * (kMmaWarp + 1);
constexpr int kSlots = 5;       // ring of K and V tiles
constexpr int kLag = 3;         // fills issued but not yet announced
constexpr uint32_t kHalf = kTile * 128;       // 128 rows x 64 columns, 16 KB
constexpr uint32_t kSlotBytes = 2 * kHalf;    // 32 KB
constexpr int kMaskRing = 8;
constexpr uint32_t kSmemQ = 0;                             // two buffers
constexpr uint32_t kSmemKv = kSmemQ + 2 * kSlotBytes;
constexpr uint32_t kSmemCtl = kSmemKv + kSlots * kSlotBytes;
constexpr uint32_t kAttnSmem = kSmemCtl + 1024 + 1024;     // control block, alignment
// TMEM columns: O, two S, two P
constexpr uint32_t kColO = 0, kColS = 128, kColP = 384;
constexpr float kGrow = 8.f;

struct AttnArgs {
  const void *q, *k, *v;
  long long qs[2], ks[3], vs[3];
  const int32_t *prefix_table, *prefix_lens, *cu_group, *table, *lens;
  void* out;
  float* lse;
  int* err;
  float scale;  // times log2 e
  int n_pages, page, prefix_width, P, width, B, Hq, Hkv, D, rep, ctas;
  // workspace
  long long* starts;  // [P + B + 1] first tile of each entry
  int32_t* clen;      // [P + B] clean lengths
  int32_t* cu;        // [P + 1] clean offsets
  float *o_base, *o_extra;    // [2][B * Hq][D], [ctas][128][D]
  float2 *ml_base, *ml_extra;
};

struct AttnLayout {
  size_t starts, clen, cu, ml_base, ml_extra, o_base, o_extra, total;
};
AttnLayout attn_layout(int64_t B, int64_t P, int64_t Hq, int64_t D) {
  AttnLayout L{};
  const size_t rows = static_cast<size_t>(B) * static_cast<size_t>(Hq);
  const size_t e = static_cast<size_t>(B + P);
  L.starts = 0;
  L.clen = L.starts + al256((e + 1) * 8);
  L.cu = L.clen + al256(e * 4);
  L.ml_base = L.cu + al256((static_cast<size_t>(P) + 1) * 4);
  L.ml_extra = L.ml_base + al256(2 * rows * 8);
  L.o_base = L.ml_extra + al256(static_cast<size_t>(kMaxCtas) * kTile * 8);
  L.o_extra = L.o_base + al256(2 * rows * static_cast<size_t>(D) * 4);
  L.total = L.o_extra + al256(static_cast<size_t>(kMaxCtas) * kTile * static_cast<size_t>(D) * 4);
  return L;
}

// ------------------------------------------------------------------ plan
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int entry_len(const AttnArgs& a, int e, int& bad) {
  const int n = e < a.P ? a.prefix_lens[e] : a.lens[e - a.P];
  const long long room = static_cast<long long>(e < a.P ? a.prefix_width : a.width) * a.page;
  if (n < 0 || n > room) bad |= RZ_DEVERR_PAGES;
  return n < 0 ? 0 : (n > room ? static_cast<int>(room) : n);
}

// One block: each thread takes a run of entries.  Offsets of the groups are
// cut to 0 <= cu[0] <= ... <= B by a running maximum.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const AttnArgs a) {
  __shared__ long long warp_sum[32];
  __shared__ int warp_max[32];
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int bad = 0;
  const auto scan = [&](auto v, auto* s, auto op) {  // exclusive; 0 is neutral
    auto inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const auto y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc = op(inc, y);
    }
    if (lane == 31) s[warp] = inc;
    __syncthreads();
    auto base = decltype(v)(0);
    for (int w = 0; w < warp; ++w) base = op(base, s[w]);
    __syncthreads();
    const auto up = __shfl_up_sync(0xffffffffu, inc, 1);
    return lane > 0 ? op(base, up) : base;
  };
  if (a.P > 0) {
    const int per = (a.P + 1 + kPlanThreads - 1) / kPlanThreads;
    const int e0 = min(threadIdx.x * per, a.P + 1), e1 = min(e0 + per, a.P + 1);
    int mx = 0;
    for (int e = e0; e < e1; ++e) mx = max(mx, a.cu_group[e]);
    int run = scan(mx, warp_max, [](int x, int y) { return max(x, y); });
    for (int e = e0; e < e1; ++e) {
      const int c = a.cu_group[e];
      run = max(run, c);
      const int clean = min(run, a.B);
      if (clean != c) bad |= RZ_DEVERR_CU_SEQLENS;
      a.cu[e] = clean;
    }
    __syncthreads();
  }
  const int E = a.P + a.B;
  const int per = (E + kPlanThreads - 1) / kPlanThreads;
  const int e0 = min(threadIdx.x * per, E), e1 = min(e0 + per, E);
  const auto tiles = [&](int e, int len) -> long long {
    long long t = static_cast<long long>((len + kTile - 1) / kTile) * a.Hkv;
    if (e < a.P) {
      const long long rows = static_cast<long long>(a.cu[e + 1] - a.cu[e]) * a.rep;
      t *= (rows + kTile - 1) / kTile;
    }
    return t;
  };
  long long sum = 0;
  for (int e = e0; e < e1; ++e) {
    const int len = entry_len(a, e, bad);
    a.clen[e] = len;
    sum += tiles(e, len);
  }
  long long at = scan(sum, warp_sum, [](long long x, long long y) { return x + y; });
  for (int e = e0; e < e1; ++e) {
    a.starts[e] = at;
    at += tiles(e, a.clen[e]);
    if (e == E - 1) a.starts[E] = at;
  }
  if (bad && a.err) atomicOr(a.err, bad);
}

// The tiles of one CTA, item by item.
struct Walk {
  long long x, end;   // tiles of the whole line left to this CTA
  long long per;
  int e;              // entry: prompt e < P, request e - P
  // the part at x
  int head, row_tile, n_tiles, t0, t1, len, rows;
  bool first;         // begins at the item's first tile

  __device__ __forceinline__ void init(const AttnArgs& a, int cta) {
    const int E = a.P + a.B;
    const long long total = a.starts[E];
    per = (total + a.ctas - 1) / a.ctas;
    x = per * cta;
    end = min(x + per, total);
    e = 0;
    if (x >= end) return;
    int lo = 0, hi = E;  // starts[lo] <= x < starts[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.starts[mid] <= x) lo = mid;
      else hi = mid;
    }
    e = lo;
  }
  // Describe the part at x; false at the end.
  __device__ __forceinline__ bool part(const AttnArgs& a) {
    if (x >= end) return false;
    while (a.starts[e + 1] <= x) ++e;
    len = a.clen[e];
    n_tiles = (len + kTile - 1) / kTile;
    const long long at = x - a.starts[e];
    const long long item = at / n_tiles;
    t0 = static_cast<int>(at - item * n_tiles);
    const long long left = end - x;
    t1 = left < n_tiles - t0 ? t0 + static_cast<int>(left) : n_tiles;
    first = t0 == 0;
    if (e < a.P) {
      const int group_rows = (a.cu[e + 1] - a.cu[e]) * a.rep;
      const int row_tiles = (group_rows + kTile - 1) / kTile;
      head = static_cast<int>(item / row_tiles);
      row_tile = static_cast<int>(item) - head * row_tiles;
      rows = min(kTile, group_rows - row_tile * kTile);
    } else {
      head = static_cast<int>(item);
      row_tile = 0;
      rows = a.rep;
    }
    return true;
  }
  __device__ __forceinline__ void next() { x += t1 - t0; }
  // request and query head of row r of the part
  __device__ __forceinline__ void row(const AttnArgs& a, int r, int& b, int& h) const {
    if (e < a.P) {
      const int i = row_tile * kTile + r;
      b = a.cu[e] + i / a.rep;
      h = head * a.rep + i % a.rep;
    } else {
      b = e - a.P;
      h = head * a.rep + r;
    }
  }
};

struct AttnCtl {
  uint64_t kv_full[kSlots], kv_empty[kSlots];
  uint64_t q_empty[2], s_full[2], s_empty[2], p_full[2], pv_done[2], o_free, drain;
  uint32_t mask[kMaskRing][4];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(AttnCtl) <= 1024, "control block");

__device__ __forceinline__ void attn_abort(AttnCtl* c, int* err) {
  *const_cast<volatile int*>(&c->abort) = 1;
  if (err) atomicOr(err, RZ_DEVERR_TIMEOUT);
}
// One lane waits, the verdict is the warp's.
__device__ __forceinline__ bool warp_wait(AttnCtl* c, uint64_t* bar, uint32_t parity, int* err) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) {
    ok = mbar_wait(bar, parity, const_cast<volatile int*>(&c->abort), kWaitLimitNs) ? 1 : 0;
    if (!ok) attn_abort(c, err);
  }
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}

// A 128 x D tile of rows into its swizzled place: `row` is the start of this
// lane's row (row 32 w + lane of the tile), ok whether it is read or zeroed.
__device__ __forceinline__ void load_rows(uint32_t dst, const uint8_t* row, bool ok, int rows,
                                          int warp, int chunks) {
  const int lane = threadIdx.x & 31;
  const uint32_t valid = __ballot_sync(0xffffffffu, ok);
  const int per_row = chunks <= 8 ? 8 : 16;  // lanes of a row
  const int step = 32 / per_row;
  const int c = lane % per_row, sub = lane / per_row;
  const int limit = min(32, rows - 32 * warp);
  for (int r0 = 0; r0 < limit; r0 += step) {
    const int r = r0 + sub;
    const uint8_t* p = reinterpret_cast<const uint8_t*>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), r));
    if (c < chunks) {
      const int tr = 32 * warp + r;
      const uint32_t at = dst + (c >> 3) * kHalf + tr * 128 + (((c & 7) ^ (tr & 7)) << 4);
      cp_async16(at, p + 16 * c, (valid >> r) & 1u ? 16u : 0u);
    }
  }
}

template <class E>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  return pack_f16x2(lo, hi);
}

// Scores as the softmax takes them: sign (a negative scale), no scale at all,
// -inf at tokens that are not there.
__device__ __forceinline__ void adjust(uint32_t (&s)[32], uint32_t bits, bool all, bool flip,
                                       bool zero) {
  if (flip || zero) {
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = zero ? 0u : s[i] ^ 0x80000000u;
  }
  if (!all) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (!((bits >> i) & 1u)) s[i] = 0xff800000u;
  }
}

template <class E>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_kernel(const AttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem);
  AttnCtl* ctl = reinterpret_cast<AttnCtl*>(smem + kSmemCtl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&ctl->kv_full[s], kLoadWarps);
      mbar_init(&ctl->kv_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl->q_empty[b], 1);
      mbar_init(&ctl->s_full[b], 1);
      mbar_init(&ctl->s_empty[b], kSoftWarps);
      mbar_init(&ctl->p_full[b], kSoftWarps);
      mbar_init(&ctl->pv_done[b], 1);
    }
    mbar_init(&ctl->o_free, kSoftWarps);
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  if (a.D % 16 != 0) {
    // the products' depth is D rounded up to 16: those columns stay zero
    uint4* p = reinterpret_cast<uint4*>(smem);
    for (uint32_t i = threadIdx.x; i < kSmemCtl / 16; i += kAttnThreads)
      p[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  grid_dep_launch();
  grid_dep_wait();  // the plan

  Walk w;
  w.init(a, blockIdx.x);
  const int chunks = a.D / 8;

  if (warp >= kSoftWarps && warp < kMmaWarp) {
    // ---------------------------------------------------------------- loads
    const int lw = warp - kSoftWarps;
    int fill = 0;       // K and V tiles issued
    int told = 0;       // ... and announced
    bool ok = true;
    int bad = 0;
    int item = 0;       // parts begun
    uint32_t tile = 0;
    // Announce fills up to `upto`; their copies have been waited for.
    const auto announce = [&](int upto) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0)
        for (; told < upto; ++told) mbar_arrive(&ctl->kv_full[told % kSlots]);
      told = upto;
    };
    // Wait until the products have released a buffer.  If that takes waiting,
    // everything issued is announced first: it is what they wait for.
    const auto wait_free = [&](uint64_t* bar, uint32_t ph) {
      if (!__all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), ph))) {
        cp_async_wait<0>();
        announce(fill);
        ok = warp_wait(ctl, bar, ph, a.err);
      }
      return ok;
    };
    const auto claim = [&]() {  // the next slot of the ring
      return fill < kSlots || wait_free(&ctl->kv_empty[fill % kSlots],
                                        static_cast<uint32_t>((fill / kSlots + 1) & 1));
    };
    const auto issued = [&]() {
      cp_async_commit();
      ++fill;
      if (fill - told > kLag) {
        cp_async_wait<kLag>();
        announce(fill - kLag);
      }
    };
    while (ok && w.part(a)) {
      const int32_t* tab = w.e < a.P
                               ? a.prefix_table + static_cast<long long>(w.e) * a.prefix_width
                               : a.table + static_cast<long long>(w.e - a.P) * a.width;
      for (int t = w.t0; t < w.t1; ++t, ++tile) {
        // this lane's token of the tile
        const long long tok = static_cast<long long>(t) * kTile + 32 * lw + lane;
        bool valid = tok < w.len;
        long long ko = 0, vo = 0;
        if (valid) {
          const long long j = tok / a.page;
          const int pg = tab[j];
          if (pg >= 0 && pg < a.n_pages) {
            const long long off = tok - j * a.page;
            ko = pg * a.ks[0] + off * a.ks[1] + w.head * a.ks[2];
            vo = pg * a.vs[0] + off * a.vs[1] + w.head * a.vs[2];
          } else {
            valid = false;
            bad = RZ_DEVERR_PAGES;
          }
        }
        const uint32_t bits = __ballot_sync(0xffffffffu, valid);
        if (!claim()) break;
        if (t == w.t0) {
          // the part's query rows ride with its first K tile
          const int qb = item & 1;
          if (item >= 2) {
            const uint32_t ph = static_cast<uint32_t>((item / 2 + 1) & 1);
            if (!wait_free(&ctl->q_empty[qb], ph)) break;
          }
          const int r = 32 * lw + lane;
          const uint8_t* qrow = static_cast<const uint8_t*>(a.q);
          if (r < w.rows) {
            int b, h;
            w.row(a, r, b, h);
            qrow += 2 * (b * a.qs[0] + h * a.qs[1]);
          }
          load_rows(base + kSmemQ + qb * kSlotBytes, qrow, r < w.rows, w.rows, lw, chunks);
          ++item;
        }
        if (lane == 0) ctl->mask[tile % kMaskRing][lw] = bits;
        load_rows(base + kSmemKv + (fill % kSlots) * kSlotBytes,
                  static_cast<const uint8_t*>(a.k) + 2 * ko, valid, kTile, lw, chunks);
        issued();
        if (!claim()) break;
        load_rows(base + kSmemKv + (fill % kSlots) * kSlotBytes,
                  static_cast<const uint8_t*>(a.v) + 2 * vo, valid, kTile, lw, chunks);
        issued();
      }
      w.next();
    }
    cp_async_wait<0>();
    announce(fill);
    if (bad && a.err) atomicOr(a.err, bad);
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- products
    if (lane == 0) {
      const uint32_t fmt = sizeof(E) == 2 && std::is_same<E, __nv_bfloat16>::value
                               ? (1u << 7) | (1u << 10) : 0u;
      const uint32_t depth = (a.D + 15) / 16;
      const uint32_t idesc_s = (1u << 4) | fmt | ((kTile >> 3) << 17) | ((kTile >> 4) << 24);
      const uint32_t idesc_o = (1u << 4) | fmt | (1u << 16) | ((2 * depth) << 17) |
                               ((kTile >> 4) << 24);
      const volatile int* abort = const_cast<volatile int*>(&ctl->abort);
      bool ok = true;
      uint32_t tile = 0;   // S issued
      int item = 0, o_items = 0;
      bool pend = false, pend_first = false;  // the tile whose P V is due
      const auto pv = [&](uint32_t j, bool fresh) {
        const uint32_t b = j & 1u, use = (j >> 1) & 1u;
        const uint32_t f = 2 * j + 1;
        const uint32_t slot = f % kSlots;
        if (!mbar_wait(&ctl->kv_full[slot], (f / kSlots) & 1u, abort, kWaitLimitNs) ||
            !mbar_wait(&ctl->p_full[b], use, abort, kWaitLimitNs))
          return false;
        if (fresh) {
          if (o_items > 0 && !mbar_wait(&ctl->o_free, (o_items - 1) & 1u, abort, kWaitLimitNs))
            return false;
          ++o_items;
        }
        tc_fence_after();
        const uint32_t v = base + kSmemKv + slot * kSlotBytes;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          umma_f16_ts(tmem + kColO, tmem + kColP + 64 * b + 8 * k,
                      sdesc_sw128(v + 2048u * k, kHalf, 1024u), idesc_o,
                      (fresh && k == 0) ? 0u : 1u);
        umma_commit(&ctl->kv_empty[slot]);
        umma_commit(&ctl->pv_done[b]);
        return true;
      };
      while (ok && w.part(a)) {
        const uint32_t q = base + kSmemQ + (item & 1) * kSlotBytes;
        for (int t = w.t0; t < w.t1; ++t, ++tile) {
          const uint32_t b = tile & 1u, use = (tile >> 1) & 1u;
          const uint32_t f = 2 * tile;
          const uint32_t slot = f % kSlots;
          if (!mbar_wait(&ctl->kv_full[slot], (f / kSlots) & 1u, abort, kWaitLimitNs) ||
              !mbar_wait(&ctl->s_empty[b], use ^ 1u, abort, kWaitLimitNs)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t k0 = base + kSmemKv + slot * kSlotBytes;
          for (uint32_t k = 0; k < depth; ++k) {
            const uint32_t off = (k >> 2) * kHalf + (k & 3) * 32u;
            umma_bf16(tmem + kColS + 128 * b, sdesc_sw128(q + off, 16u, 1024u),
                      sdesc_sw128(k0 + off, 16u, 1024u), idesc_s, k > 0 ? 1u : 0u);
          }
          umma_commit(&ctl->kv_empty[slot]);
          umma_commit(&ctl->s_full[b]);
          if (t == w.t1 - 1) umma_commit(&ctl->q_empty[item & 1]);
          if (pend && !pv(tile - 1, pend_first)) {
            ok = false;
            break;
          }
          pend = true;
          pend_first = t == w.t0;
        }
        ++item;
        w.next();
      }
      if (ok && pend) ok = pv(tile - 1, pend_first);
      if (!ok) attn_abort(ctl, a.err);
      // no MMA is in flight when TMEM is freed
      umma_commit(&ctl->drain);
      if (!mbar_wait(&ctl->drain, 0, abort, kWaitLimitNs) && !*abort) attn_abort(ctl, a.err);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const int r = warp * 32 + lane;
    const bool flip = a.scale < 0.f, zero = a.scale == 0.f;
    const float sl = zero ? 1.f : fabsf(a.scale);
    uint32_t tile = 0;
    bool ok = true;
    while (ok && w.part(a)) {
      const bool live = warp * 32 < w.rows;
      float m = -INFINITY, l = 0.f;
      for (int t = w.t0; t < w.t1; ++t, ++tile) {
        const uint32_t b = tile & 1u, use = (tile >> 1) & 1u;
        if (!(ok = warp_wait(ctl, &ctl->s_full[b], use, a.err))) break;
        tc_fence_after();
        uint32_t bits[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) bits[i] = ctl->mask[tile % kMaskRing][i];
        if (live) {
          const uint32_t sc = lanes + kColS + 128 * b;
          const bool all = (bits[0] & bits[1] & bits[2] & bits[3]) == 0xffffffffu;
          // two passes over S, 64 columns in registers at a time: the
          // maximum, then the terms
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t s[2][32];
            tmem_ld32(sc + 64 * half, s[0]);
            tmem_ld32(sc + 64 * half + 32, s[1]);
            tmem_ld_wait();
            adjust(s[0], bits[2 * half], all, flip, zero);
            adjust(s[1], bits[2 * half + 1], all, flip, zero);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              mx[i & 1] = fmaxf(mx[i & 1], __uint_as_float(s[0][i]));
              mx[2 + (i & 1)] = fmaxf(mx[2 + (i & 1)], __uint_as_float(s[1][i]));
            }
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl;
          const bool grow = top > m + kGrow || (m == -INFINITY && top > m);
          if (t > w.t0 && __any_sync(0xffffffffu, grow)) {
            // O of the tiles before moves to the new reference
            const uint32_t pj = tile - 1;
            if (!(ok = warp_wait(ctl, &ctl->pv_done[pj & 1u], (pj >> 1) & 1u, a.err))) break;
            tc_fence_after();
            const float f = grow ? (m == -INFINITY ? 0.f : ex2_approx(m - top)) : 1.f;
            for (int i = 0; i < a.D; i += 32) {
              uint32_t o[32];
              tmem_ld32(lanes + kColO + i, o);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st32(lanes + kColO + i, o);
            }
            tmem_st_wait();
            l *= f;
          }
          if (grow) m = top;
          const float ref = m == -INFINITY ? 0.f : m;
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t s[2][32], pk[32];
            tmem_ld32(sc + 64 * half, s[0]);
            tmem_ld32(sc + 64 * half + 32, s[1]);
            tmem_ld_wait();
            if (half == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&ctl->s_empty[b]);
            }
            adjust(s[0], bits[2 * half], all, flip, zero);
            adjust(s[1], bits[2 * half + 1], all, flip, zero);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float p0 = ex2_approx(fmaf(__uint_as_float(s[i >> 4][2 * (i & 15)]), sl, -ref));
              const float p1 =
                  ex2_approx(fmaf(__uint_as_float(s[i >> 4][2 * (i & 15) + 1]), sl, -ref));
              acc[i & 3] += p0 + p1;
              pk[i] = pack2<E>(p0, p1);
            }
            tmem_st32(lanes + kColP + 64 * b + 32 * half, pk);
          }
          l += (acc[0] + acc[1]) + (acc[2] + acc[3]);
          tmem_st_wait();
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->s_empty[b]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_full[b]);
      }
      if (!ok) break;
      // the part's result
      const uint32_t pj = tile - 1;
      if (!(ok = warp_wait(ctl, &ctl->pv_done[pj & 1u], (pj >> 1) & 1u, a.err))) break;
      tc_fence_after();
      if (live) {
        long long at = static_cast<long long>(blockIdx.x) * kTile + r;
        if (w.first && r < w.rows) {
          int q, h;
          w.row(a, r, q, h);
          at = (static_cast<long long>(w.e < a.P ? 0 : a.B) + q) * a.Hq + h;
        }
        float* dst = (w.first ? a.o_base : a.o_extra) + at * a.D;
        for (int i = 0; i < a.D; i += 32) {
          uint32_t o[32];
          tmem_ld32(lanes + kColO + i, o);
          tmem_ld_wait();
          if (r < w.rows) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              if (i + k < a.D) st_global_v4(dst + i + k, o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
        if (r < w.rows) (w.first ? a.ml_base : a.ml_extra)[at] = make_float2(m, l);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->o_free);
      w.next();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ join
constexpr int kJoinThreads = 128;

__device__ __forceinline__ void put16(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put16(__half* p, float x) { *p = __float2half_rn(x); }

template <class E>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttnArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(a.B) * a.Hq) return;
  const int b = static_cast<int>(row / a.Hq), h = static_cast<int>(row - static_cast<long long>(b) * a.Hq);
  const int hk = h / a.rep;
  const int E_ = a.P + a.B;
  const long long total = a.starts[E_];
  const long long per = max((total + a.ctas - 1) / a.ctas, 1ll);
  // the prompt of request b
  int g = -1;
  if (a.P > 0 && b >= a.cu[0] && b < a.cu[a.P]) {
    int lo = 0, hi = a.P;  // cu[lo] <= b < cu[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= b) lo = mid;
      else hi = mid;
    }
    g = lo;
  }
  // the item's tiles [x0, x1) and the row in it, for prompt and own tokens
  const auto item = [&](int part, long long& x0, long long& x1, int& r) {
    const int e = part == 0 ? g : a.P + b;
    if (e < 0) return false;
    const int n = (a.clen[e] + kTile - 1) / kTile;
    if (n == 0) return false;
    long long idx = hk;
    r = h - hk * a.rep;
    if (part == 0) {
      const int i = (b - a.cu[g]) * a.rep + r;
      const int row_tiles = ((a.cu[g + 1] - a.cu[g]) * a.rep + kTile - 1) / kTile;
      idx = static_cast<long long>(hk) * row_tiles + i / kTile;
      r = i % kTile;
    }
    x0 = a.starts[e] + idx * n;
    x1 = x0 + n;
    return true;
  };
  float M = -INFINITY, L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int part = 0; part < 2; ++part) {
    long long x0, x1;
    int r;
    if (!item(part, x0, x1, r)) continue;
    const long long c0 = x0 / per, c1 = (x1 - 1) / per;
    for (long long c = c0; c <= c1; ++c) {
      const long long at = c == c0 ? (static_cast<long long>(part == 0 ? 0 : a.B) + b) * a.Hq + h
                                   : c * kTile + r;
      const float2 ml = (c == c0 ? a.ml_base : a.ml_extra)[at];
      const float* src = (c == c0 ? a.o_base : a.o_extra) + at * a.D;
      const float mn = fmaxf(M, ml.x);
      if (mn == -INFINITY) continue;  // no token yet
      const float f = exp2f(M - mn), fe = exp2f(ml.x - mn);
      L = L * f + ml.y * fe;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lane + 32 * i < a.D) o[i] = o[i] * f + src[lane + 32 * i] * fe;
      M = mn;
    }
  }
  E* out = static_cast<E*>(a.out) + row * a.D;
  const float inv = M == -INFINITY ? 0.f : 1.f / L;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane + 32 * i < a.D) put16(out + lane + 32 * i, o[i] * inv);
  if (lane == 0 && a.lse) a.lse[row] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <class K>
cudaError_t launch_after(K kern, int grid, int block, size_t smem, const AttnArgs& a,
                         cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <class E>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(attn_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kAttnSmem));
  if (e != cudaSuccess) return e;
  plan_kernel<<<1, kPlanThreads, 0, st>>>(a);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_after(attn_kernel<E>, a.ctas, kAttnThreads, kAttnSmem, a, st);
  const int per = kJoinThreads / 32;
  if (e == cudaSuccess)
    e = launch_after(join_kernel<E>, (a.B * a.Hq + per - 1) / per, kJoinThreads, 0, a, st);
  return e;
}

}  // namespace

size_t group_decode_attn_ws_bytes(int64_t B, int32_t P, int32_t Hq, int32_t D) {
  return attn_layout(B < 0 ? 0 : B, P < 0 ? 0 : P, Hq < 1 ? 1 : Hq, D < 1 ? 1 : D).total;
}

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
  if (static_cast<int64_t>(B) + P >= (1 << 30) || static_cast<int64_t>(B) * Hq >= (1 << 30))
    return RZ_ERR_INVALID_ARG;
  if (D < 8 || D > kMaxD || D % 8 != 0 || Hq / Hkv > kTile) return RZ_ERR_UNSUPPORTED;
  if (B == 0) return RZ_OK;
  for (int i = 0; i < 6; ++i)
    if (kv_stride[i] % 8 != 0) return RZ_ERR_UNSUPPORTED;
  if (q_stride[0] % 8 != 0 || q_stride[1] % 8 != 0) return RZ_ERR_UNSUPPORTED;
  if (!a16(q) || !a16(k_cache) || !a16(v_cache) || !a16(out)) return RZ_ERR_UNSUPPORTED;
  const AttnLayout L = attn_layout(B, P, Hq, D);
  if (!ws || ws_bytes < L.total || !a256(ws)) return RZ_ERR_WORKSPACE;
  if (!device_ok()) return RZ_ERR_UNSUPPORTED;
  AttnArgs a{};
  a.q = q;
  // a page past the pool is never read; with an empty pool nothing is
  a.k = n_pages > 0 ? k_cache : q;
  a.v = n_pages > 0 ? v_cache : q;
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
  a.rep = Hq / Hkv;
  a.ctas = num_sms() < kMaxCtas ? num_sms() : kMaxCtas;
  uint8_t* w8 = static_cast<uint8_t*>(ws);
  a.starts = reinterpret_cast<long long*>(w8 + L.starts);
  a.clen = reinterpret_cast<int32_t*>(w8 + L.clen);
  a.cu = reinterpret_cast<int32_t*>(w8 + L.cu);
  a.ml_base = reinterpret_cast<float2*>(w8 + L.ml_base);
  a.ml_extra = reinterpret_cast<float2*>(w8 + L.ml_extra);
  a.o_base = reinterpret_cast<float*>(w8 + L.o_base);
  a.o_extra = reinterpret_cast<float*>(w8 + L.o_extra);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ProfScope ps(RZ_PROF_SMALL, 3, st);
  const cudaError_t e =
      dtype == RZ_DTYPE_BF16 ? launch<__nv_bfloat16>(a, st) : launch<__half>(a, st);
  return e == cudaSuccess ? RZ_OK : RZ_ERR_CUDA;
}
