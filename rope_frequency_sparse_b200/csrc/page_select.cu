// page_select.cu -- the pages of a paged cache that one query per sequence
// attends to, chosen by a bound on their logits.
//
// For a page with elementwise minimum mn and maximum mx of its keys, no key of it
// has a larger q.k than sum_e max(q_e mn_e, q_e mx_e).  With the method's windows
// a pair counts where some key of the page is within reach:
//
//   score(p) = max over the query heads g of the kv head of
//              sum over pairs i with Dmin(p) <= W_i of
//              sum over the pair's two elements of max(q_e mn_e, q_e mx_e)
//
// Kept are the first n_first and last n_last pages and the highest scores, equal ones
// by lower index, as an ascending list, in the order of 64-bit sums.
//
// max(q mn, q mx) = min(q, 0) mn + max(q, 0) mx, so the scores of 16 pages are a
// product of their bounds as they are stored, 2 d elements a row, with the queries
// split by sign: 2 d / 16 warp-level MMAs for up to eight query heads.  These fp32
// sums are off by at most kEps of the sum S of the terms' magnitudes, which a second
// product over |bounds| and |queries| gives; a selection by them is the one by exact
// sums but for pages within 2 kEps max S of the last kept one, and those alone are
// scored again in fp64 and ranked.  (All pages in fp64 took 26 us of arithmetic for
// 16384 pages, 4 kv heads, 28 query heads; the bounds are read in 5.)  Where more than kAgain
// pages are that close, or a sum is not finite, every page is scored in fp64.
//
// First kernel: bound by the bounds' bytes, 4 d a page and kv head less the pairs
// that are out of reach.  Second kernel, one CTA per sequence and kv head, bound by
// its passes over the scores: the order-preserving bit patterns are binned linearly
// between the least and the greatest, and the bin of the last kept one again, until
// few are left; a bin's edges are exact, so any distribution ends (each round parts
// the least from the greatest).  The kept indices are emitted in order, a segment a warp.
#include <cuda_bf16.h>

#include <atomic>

#include "atf_internal.cuh"
#include "ptx.cuh"

namespace atf {

namespace {

using u64 = unsigned long long;

constexpr int kScoreThreads = 128;
constexpr int kBins = 2048, kBinBits = 11;
constexpr int kAgain = 256;       // pages that are scored again and ranked one against another
constexpr int kFewPages = 24;     // a bin of at most this many is not binned again: each goes to a warp
constexpr int kHeldKeys = 16384;  // scores that are kept in shared memory
// A step of 16 products is off by at most 18 * 2^-23 of the magnitudes summed so
// far; 16 steps stay below 2^-14.8, and the rest of 2^-14 covers the roundings of S
// and of the thresholds.
constexpr float kEps = 6.103515625e-05f;

__device__ __forceinline__ int select_len(const PageSelectParams& p, int b) {
  const int len = p.kv_len[b];
  const long long cap = static_cast<long long>(p.max_pages) << p.page_log2;
  if (len > cap) {
    atomicCAS(p.err, 0u, kErrBadLength);
    return static_cast<int>(cap);
  }
  return len < 0 ? 0 : len;
}

// Bit patterns whose unsigned order is the number's (-0 as +0).
__device__ __forceinline__ u64 sortable(double x) {
  const u64 u = static_cast<u64>(__double_as_longlong(x + 0.0));
  return (u >> 63) ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ unsigned sortable(float x) {
  const unsigned u = __float_as_uint(x + 0.0f);
  return (u >> 31) ? ~u : u | (1u << 31);
}
__device__ __forceinline__ float from_sortable(unsigned u) {
  return __uint_as_float((u >> 31) ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ int leading_zeros(u64 x) { return __clzll(x); }
__device__ __forceinline__ int leading_zeros(unsigned x) { return __clz(x); }

// Distance of a page's nearest key.
__device__ __forceinline__ int page_distance(const PageSelectParams& p, int len, int page) {
  return max(0, len - ((page + 1) << p.page_log2));
}

// Page in the pool, or -1 (recorded).
__device__ __forceinline__ int pool_page(const PageSelectParams& p, int entry) {
  if (entry >= 0 && entry < p.num_pages) return entry;
  atomicCAS(p.err, 0u, kErrBadPage);
  return -1;
}

}  // namespace

// Scores of 16 pages a warp.  Lane (row, kcol) holds, of pages `row` and `row` + 8,
// 16-byte pieces 4 j + kcol of the 2 d bounds, and of query head `row` the same
// pieces: the sum's order of elements is the MMA's to choose.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const __grid_constant__ PageSelectParams p) {
  constexpr int NJ = D / 32;  // pieces of the minima a lane holds, and of the maxima
  const int tid = threadIdx.x, lane = tid & 31, row = lane >> 2, kcol = lane & 3;
  const int hk = blockIdx.y % p.hkv, b = blockIdx.y / p.hkv, G = p.hq / p.hkv;
  __shared__ int sw[kMaxPairs];
  for (int i = tid; i < kMaxPairs; i += kScoreThreads) sw[i] = p.win.w[i];
  pdl_launch_dependents();
  pdl_wait();
  const int len = select_len(p, b), ps = 1 << p.page_log2;
  const int pages = (len + ps - 1) >> p.page_log2;
  if (static_cast<long long>(blockIdx.x) * (kScoreThreads / 2) >= pages) return;
  __syncthreads();
  const int pg0 = blockIdx.x * (kScoreThreads / 2) + (tid >> 5) * 16 + row;
  const int* table = p.page_table + static_cast<long long>(b) * p.max_pages;
  int page[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) page[r] = pg0 + 8 * r < pages ? table[pg0 + 8 * r] : -1;
  uint4 qv[NJ];  // loaded while the table's entries are on their way
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + b * p.q_stride + (static_cast<long long>(hk) * G + row) * D;
#pragma unroll
  for (int j = 0; j < NJ; ++j) qv[j] = row < G ? *reinterpret_cast<const uint4*>(q + 32 * j + 8 * kcol) : zero;
  uint4 v[2][2 * NJ];
  int near[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const bool live = pg0 + 8 * r < pages;
    if (live) page[r] = pool_page(p, page[r]);
    near[r] = live ? page_distance(p, len, pg0 + 8 * r) : 0;
    const uint4* bounds = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.bounds) +
                                                         (static_cast<long long>(max(page[r], 0)) * p.hkv + hk) * 2 * D);
#pragma unroll
    for (int j = 0; j < 2 * NJ; ++j) {  // windows grow with the pair: a piece out of reach as a whole is not read
      const bool reach = near[r] <= sw[16 * (j % NJ) + 4 * kcol + 3];
      v[r][j] = live && page[r] >= 0 && reach ? bounds[4 * j + kcol] : zero;
    }
  }
  float a[4] = {0.f, 0.f, 0.f, 0.f}, m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 2 * NJ; ++j) {
    uint32_t x[2][4], y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 qj = qv[j % NJ];
      const uint32_t w = k == 0 ? qj.x : k == 1 ? qj.y : k == 2 ? qj.z : qj.w;
      const uint32_t negative = ((w >> 15) & 0x00010001u) * 0xFFFFu;
      y[k] = j < NJ ? w & negative : w & ~negative;
      const int window = sw[16 * (j % NJ) + 4 * kcol + k];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4 z = v[r][j];
        x[r][k] = k == 0 ? z.x : k == 1 ? z.y : k == 2 ? z.z : z.w;
        if (near[r] > window) x[r][k] = 0u;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t f[4] = {x[0][2 * h], x[1][2 * h], x[0][2 * h + 1], x[1][2 * h + 1]};
      mma_bf16_16816(a, f, y[2 * h], y[2 * h + 1]);
      constexpr uint32_t kAbs = 0x7FFF7FFFu;
      const uint32_t fa[4] = {f[0] & kAbs, f[1] & kAbs, f[2] & kAbs, f[3] & kAbs};
      mma_bf16_16816(m, fa, y[2 * h] & kAbs, y[2 * h + 1] & kAbs);
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float best = -INFINITY, size = 0.f;  // of query heads 2 kcol, 2 kcol + 1
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (2 * kcol + e >= G) continue;
      best = fmaxf(best, a[2 * r + e]);
      size = m[2 * r + e] < INFINITY ? fmaxf(size, m[2 * r + e]) : INFINITY;  // NaN: infinite
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, off));
      size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, off));
    }
    if (kcol == 0 && pg0 + 8 * r < pages)
      p.keys[(static_cast<long long>(b) * p.hkv + hk) * p.max_pages + pg0 + 8 * r] =
          static_cast<u64>(sortable(best)) << 32 | __float_as_uint(size);
  }
}

namespace {

struct SelectShared {
  u64 cand[kAgain];
  int hist[kBins];
  u64 red[32];
  int warp_n[2][32];
  u64 lo, hi, cut;
  int need, count, n, above;
  int again[kAgain];
  unsigned least[32], greatest[32], size[32];
};

// Narrows [lo, hi], which holds the need-th highest of the keys get(i), i0 <= i < i1,
// until it is one key, or all of its `count` keys are needed, or they are at most
// `few`.  On return `need` counts within [lo, hi].
template <typename K, typename Get>
__device__ __forceinline__ void narrow(SelectShared* sh, Get get, int i0, int i1, K& lo, K& hi, int& need, int& count,
                                       int few) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x;
  while (lo < hi && count > few && count != need) {
    const int shift = max(0, static_cast<int>(sizeof(K)) * 8 - leading_zeros(hi - lo) - kBinBits);
    for (int i = tid; i < kBins; i += T) sh->hist[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = i0 + tid; i < i1; i += T) {
      const K k = get(i);
      if (k >= lo && k <= hi) atomicAdd(&sh->hist[static_cast<int>((k - lo) >> shift)], 1);
    }
    __syncthreads();
    // the bin of the need-th, counted from the top: eight bins a thread
    int sum = 0, incl = 0;
    const int top = kBins - 1 - 8 * tid;
    if (tid < kBins / 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += sh->hist[top - j];
      incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      if (lane == 31) sh->warp_n[0][warp] = incl;
    }
    __syncthreads();
    if (tid < kBins / 8) {
      int before = incl - sum;
      for (int w = 0; w < warp; ++w) before += sh->warp_n[0][w];
      if (before < need && need <= before + sum) {
        int bin = top;
        while (before + sh->hist[bin] < need) before += sh->hist[bin--];
        const K edge = lo + (static_cast<K>(bin) << shift);
        const K span = (static_cast<K>(1) << shift) - 1;
        sh->lo = edge;
        sh->hi = hi - edge < span ? hi : edge + span;
        sh->need = need - before;
        sh->count = sh->hist[bin];
      }
    }
    __syncthreads();
    lo = static_cast<K>(sh->lo);
    hi = static_cast<K>(sh->hi);
    need = sh->need;
    count = sh->count;
  }
}

// Least and greatest of the threads' values.
__device__ __forceinline__ void block_range(SelectShared* sh, u64& lo, u64& hi) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    u64 x = side ? hi : lo;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const u64 y = __shfl_xor_sync(0xffffffffu, x, off);
      x = side ? max(x, y) : min(x, y);
    }
    __syncthreads();
    if (lane == 0) sh->red[warp] = x;
    __syncthreads();
    for (int w = 0; w < warps; ++w) {
      const u64 y = sh->red[w];
      x = side ? max(x, y) : min(x, y);
    }
    (side ? hi : lo) = x;
  }
}

// Writes, in order, the pages i for which kept(i) is set, and the first `ties` for
// which tie(i) is; a segment of the pages a warp.
template <typename Kept, typename Tie>
__device__ __forceinline__ void emit(SelectShared* sh, int pages, int ties, int* out, Kept kept, Tie tie) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int seg = ((pages + warps - 1) / warps + 31) & ~31;
  const int b0 = min(pages, warp * seg), b1 = min(pages, b0 + seg);
  int a = 0, t = 0;
  for (int i = b0 + lane; i - lane < b1; i += 32) {
    a += __popc(__ballot_sync(0xffffffffu, i < b1 && kept(i)));
    t += __popc(__ballot_sync(0xffffffffu, i < b1 && tie(i)));
  }
  __syncthreads();  // the search still reads these
  if (lane == 0) sh->warp_n[0][warp] = a, sh->warp_n[1][warp] = t;
  __syncthreads();
  a = t = 0;
  for (int w = 0; w < warp; ++w) a += sh->warp_n[0][w], t += sh->warp_n[1][w];
  const unsigned below = (1u << lane) - 1;
  for (int i = b0 + lane; i - lane < b1; i += 32) {
    const bool k = i < b1 && kept(i), e = i < b1 && tie(i);
    const unsigned ma = __ballot_sync(0xffffffffu, k), mt = __ballot_sync(0xffffffffu, e);
    const int ai = a + __popc(ma & below), ti = t + __popc(mt & below);
    if (k || (e && ti < ties)) out[ai + min(ti, ties)] = i;
    a += __popc(ma);
    t += __popc(mt);
  }
}

// The 64-bit score of a page, by a warp; one order of sums for every page.
__device__ __forceinline__ u64 exact_score(const PageSelectParams& p, int b, int hk, int len, int page) {
  const int lane = threadIdx.x & 31, G = p.hq / p.hkv, d = p.d;
  const int entry = pool_page(p, p.page_table[static_cast<long long>(b) * p.max_pages + page]);
  const int near = page_distance(p, len, page);
  const uint32_t* bounds = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.bounds) +
                                                             (static_cast<long long>(max(entry, 0)) * p.hkv + hk) * 2 * d);
  uint32_t mn[2] = {0u, 0u}, mx[2] = {0u, 0u};
  for (int r = 0; r < d / 64; ++r) {
    const int pair = 32 * r + lane;
    if (entry >= 0 && near <= p.win.w[pair]) mn[r] = bounds[pair], mx[r] = bounds[d / 2 + pair];
  }
  const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.q) + b * p.q_stride +
                                                        static_cast<long long>(hk) * G * d);
  double best = -INFINITY;
  for (int g = 0; g < G; ++g) {
    double s = 0.0;
    for (int r = 0; r < d / 64; ++r) {
      const uint32_t w = q[g * (d / 2) + 32 * r + lane];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = e ? bf16hi_to_f32(w) : bf16lo_to_f32(w);
        const float l = e ? bf16hi_to_f32(mn[r]) : bf16lo_to_f32(mn[r]), h = e ? bf16hi_to_f32(mx[r]) : bf16lo_to_f32(mx[r]);
        s += fmax(static_cast<double>(x) * l, static_cast<double>(x) * h);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    best = fmax(best, s);
  }
  return sortable(best);
}

}  // namespace

// Threads: a multiple of 32, 256 to 1024.
__global__ void __launch_bounds__(1024) page_select_kernel(const __grid_constant__ PageSelectParams p, int held) {
  extern __shared__ unsigned s_keys[];  // `held` scores
  __shared__ SelectShared s;
  SelectShared* sh = &s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x, warps = T >> 5;
  const int hk = blockIdx.x % p.hkv, b = blockIdx.x / p.hkv;
  pdl_launch_dependents();
  pdl_wait();
  const int len = select_len(p, b);
  const int pages = (len + (1 << p.page_log2) - 1) >> p.page_log2;
  u64* keys = p.keys + (static_cast<long long>(b) * p.hkv + hk) * p.max_pages;
  int* out = p.selected + (static_cast<long long>(b) * p.hkv + hk) * p.n_sel;
  if (pages <= p.n_sel) {
    for (int i = tid; i < p.n_sel; i += T) out[i] = i < pages ? i : -1;
    return;
  }
  // pages [i0, i1) compete for `places`
  const int i0 = p.n_first, i1 = pages - p.n_last, places = p.n_sel - p.n_first - p.n_last;
  auto forced = [&](int i) { return i < i0 || i >= i1; };
  auto never = [](int) { return false; };
  if (places == 0) return emit(sh, pages, 0, out, forced, never);

  const bool hold = pages <= held;
  unsigned lo = ~0u, hi = 0u, size = 0u;
#pragma unroll 4
  for (int i = i0 + tid; i < i1; i += T) {
    const u64 x = keys[i];
    const unsigned k = static_cast<unsigned>(x >> 32);
    if (hold) s_keys[i] = k;
    lo = min(lo, k);
    hi = max(hi, k);
    size = max(size, static_cast<unsigned>(x));  // magnitudes: their bits are in their order
  }
  if (tid == 0) sh->n = sh->above = 0;
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  size = __reduce_max_sync(0xffffffffu, size);
  if (lane == 0) sh->least[warp] = lo, sh->greatest[warp] = hi, sh->size[warp] = size;
  __syncthreads();
  const int w = min(lane, warps - 1);
  lo = __reduce_min_sync(0xffffffffu, sh->least[w]);
  hi = __reduce_max_sync(0xffffffffu, sh->greatest[w]);
  size = __reduce_max_sync(0xffffffffu, sh->size[w]);
  // twice the largest error of a score; the constant covers products that vanish in fp32
  const float slack = 2.f * (kEps * __uint_as_float(size) + 1e-30f);
  auto approx = [&](int i) { return hold ? s_keys[i] : static_cast<unsigned>(keys[i] >> 32); };
  bool again = !(slack < INFINITY);
  if (!again) {
    int need = places, count = i1 - i0;
    narrow(sh, approx, i0, i1, lo, hi, need, count, kFewPages);
    const unsigned cut_lo = sortable(from_sortable(lo) - slack), cut_hi = sortable(from_sortable(hi) + slack);
    int above = 0;
#pragma unroll 4
    for (int i = i0 + tid; i < i1; i += T) {
      const unsigned k = approx(i);
      above += k > cut_hi;
      if (k >= cut_lo && k <= cut_hi) {
        const int at = atomicAdd(&sh->n, 1);
        if (at < kAgain) sh->again[at] = i;
      }
    }
    above = __reduce_add_sync(0xffffffffu, above);
    if (lane == 0) atomicAdd(&sh->above, above);
    __syncthreads();
    const int close = sh->n;
    need = places - sh->above;  // of the close ones
    again = close > kAgain;
    if (!again) {
      if (close > need) {
        for (int i = warp; i < close; i += warps) {
          const u64 x = exact_score(p, b, hk, len, sh->again[i]);
          if (lane == 0) sh->cand[i] = x;
        }
        __syncthreads();
      }
      if (tid < close) {
        const int mine = sh->again[tid];
        int before = 0;
        if (close > need)
          for (int j = 0; j < close; ++j)
            before += sh->cand[j] > sh->cand[tid] || (sh->cand[j] == sh->cand[tid] && sh->again[j] < mine);
        const unsigned mark = before < need ? ~0u : 0u;  // its score from here on
        if (hold)
          s_keys[mine] = mark;
        else
          keys[mine] = static_cast<u64>(mark) << 32;
      }
      __syncthreads();
      return emit(sh, pages, 0, out, [&](int i) { return forced(i) || approx(i) > cut_hi; }, never);
    }
  }

  // every score in 64 bits
  for (int i = i0 + warp; i < i1; i += warps) {
    const u64 x = exact_score(p, b, hk, len, i);
    if (lane == 0) keys[i] = x;
  }
  __syncthreads();
  if (tid == 0) sh->n = 0;
  u64 lo64 = ~0ull, hi64 = 0;
  for (int i = i0 + tid; i < i1; i += T) lo64 = min(lo64, keys[i]), hi64 = max(hi64, keys[i]);
  block_range(sh, lo64, hi64);
  int need = places, count = i1 - i0;
  narrow(sh, [&](int i) { return keys[i]; }, i0, i1, lo64, hi64, need, count, kAgain);
  // kept: every key above `cut`, and the first `ties` that equal it
  u64 cut = lo64;
  int ties = need;
  if (lo64 < hi64 && count == need) {  // all of the range
    cut = lo64 ? lo64 - 1 : 0;
    ties = lo64 ? 0 : count;
  } else if (lo64 < hi64) {
    for (int i = i0 + tid; i < i1; i += T) {
      const u64 k = keys[i];
      if (k >= lo64 && k <= hi64) sh->cand[atomicAdd(&sh->n, 1)] = k;
    }
    __syncthreads();
    if (tid < count) {
      const u64 mine = sh->cand[tid];
      int above = 0, equal = 0;
      for (int j = 0; j < count; ++j) {
        above += sh->cand[j] > mine;
        equal += sh->cand[j] == mine;
      }
      if (above < need && need <= above + equal) {  // so do its equals, with the same values
        sh->cut = mine;
        sh->need = need - above;
      }
    }
    __syncthreads();
    cut = sh->cut;
    ties = sh->need;
  }
  emit(sh, pages, ties, out, [&](int i) { return forced(i) || keys[i] > cut; },
       [&](int i) { return !forced(i) && keys[i] == cut; });
}

cudaError_t launch_page_select(const PageSelectParams& p, cudaStream_t s) {
  const int per = kScoreThreads / 2;
  const dim3 grid((p.max_pages + per - 1) / per, p.batch * p.hkv);
  cudaError_t e = launch_pdl(p.d == 64 ? page_score_kernel<64> : page_score_kernel<128>, grid, kScoreThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<u64> configured{0};  // one bit per device; setting it twice is harmless
  if (dev >= 64 || !(configured.load(std::memory_order_acquire) & (1ull << dev))) {
    e = cudaFuncSetAttribute(page_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldKeys * 4);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured.fetch_or(1ull << dev, std::memory_order_acq_rel);
  }
  const int held = p.max_pages < kHeldKeys ? p.max_pages : kHeldKeys;
  const int threads = p.max_pages <= 2048 ? 256 : 1024;
  return launch_pdl(page_select_kernel, p.batch * p.hkv, threads, held * 4, s, p, held);
}

}  // namespace atf
