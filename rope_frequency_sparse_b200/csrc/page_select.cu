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
// that are out of reach.  Second kernel (it scores short lists itself), one CTA per
// sequence and kv head, bound by its passes over the scores: the order-preserving bit patterns are binned linearly
// between the least and the greatest, and the bin of the last kept one again, until
// few are left; a bin's edges are exact, so any distribution ends (each round parts
// the least from the greatest).  Where the places are at most a quarter of the groups
// of 16 pages with one that competes, those are searched by their highest scores first, and
// pages only in those that can hold a kept one: one SM's passes over 16384 scores took 12 us.
//
// Measured, selection and decode of the selected pages: 64 of 16384 pages for 28 query
// and 4 kv heads of 128, 24.3 us (15 of them here); 48 of up to 1024 pages of 32
// sequences, 44.9 us (18 here).
#include <cuda_bf16.h>

#include "atf_internal.cuh"
#include "ptx.cuh"
#include "select_groups.cuh"

namespace atf {

namespace {

using u64 = unsigned long long;

constexpr int kScoreThreads = 128;
constexpr int kSelectThreads = 512;
// Pages of a list that one CTA scores and selects: eight lists of up to 250 pages take
// 15.3 us with their decode, 16.5 by two kernels; 32 x 4 of up to 1024 would take 53
// against 49.
constexpr int kShort = 512;
constexpr int kBins = 1024, kBinBits = 10;  // eight bins a thread of the smallest block
constexpr int kAgain = 256;       // pages that are scored again and ranked one against another
constexpr int kCandidates = 4096;  // pages that are looked at one by one, of groups with a high score
constexpr int kFewGroups = 24;    // a bin of at most this many groups is not binned again
constexpr int kHeld = 4;          // scores that a thread holds in registers at most
// A step of 16 products is off by at most 18 * 2^-23 of the magnitudes summed so
// far; the four steps of a sum stay below 2^-16.8, and the rest of 2^-16 covers the
// sums' own sum and the roundings of S and of the thresholds.
constexpr float kEps = 1.52587890625e-05f;

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

// What the first kernel leaves of a list of two pages or more in its max_pages 64-bit
// words of workspace: the pages' scores, sortable, and of each group of 16 pages the
// bits of the greatest S and the highest score that competes for a place (0: none).
struct Scores {
  unsigned *key, *size, *high;
  __device__ Scores(const PageSelectParams& p, int list)
      : key(reinterpret_cast<unsigned*>(p.keys + static_cast<long long>(list) * p.max_pages)),
        size(key + p.max_pages),
        high(size + (p.max_pages + kGroup - 1) / kGroup) {}
  __device__ Scores(unsigned* key_, unsigned* size_, unsigned* high_) : key(key_), size(size_), high(high_) {}
};

}  // namespace

// Scores of 16 pages a warp.  Lane (row, kcol) holds, of pages `row` and `row` + 8,
// 16-byte pieces 4 j + kcol of the 2 d bounds, and of query head `row` the same
// pieces: the sum's order of elements is the MMA's to choose.
template <int D>
__device__ __forceinline__ void score_group(const PageSelectParams& p, int b, int hk, int len, int pages, int group,
                                            const int* sw, const Scores& out) {
  constexpr int NJ = D / 32;  // pieces of the minima a lane holds, and of the maxima
  const int lane = threadIdx.x & 31, row = lane >> 2, kcol = lane & 3, G = p.hq / p.hkv;
  const int pg0 = group * kGroup + row;
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
  float a4[4][4], m[4] = {0.f, 0.f, 0.f, 0.f};  // four sums of scores: less error, shorter chains
#pragma unroll
  for (int i = 0; i < 4; ++i) a4[i][0] = a4[i][1] = a4[i][2] = a4[i][3] = 0.f;
#pragma unroll
  for (int jp = 0; jp < NJ; ++jp) {
    const int* w = sw + 16 * jp + 4 * kcol;
    // out of reach of all 16 pages: nothing was read
    if (!__any_sync(0xffffffffu, near[0] <= w[3] || near[1] <= w[3])) continue;
    if (__any_sync(0xffffffffu, near[0] > w[0] || near[1] > w[0])) {  // out of reach in part
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = jp; j < 2 * NJ; j += NJ) {
          if (near[r] > w[0]) v[r][j].x = 0u;
          if (near[r] > w[1]) v[r][j].y = 0u;
          if (near[r] > w[2]) v[r][j].z = 0u;
          if (near[r] > w[3]) v[r][j].w = 0u;
        }
    }
    const uint32_t q4[4] = {qv[jp].x, qv[jp].y, qv[jp].z, qv[jp].w};
#pragma unroll
    for (int j = jp; j < 2 * NJ; j += NJ) {
      const uint32_t x0[4] = {v[0][j].x, v[0][j].y, v[0][j].z, v[0][j].w};
      const uint32_t x1[4] = {v[1][j].x, v[1][j].y, v[1][j].z, v[1][j].w};
      uint32_t y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t negative = ((q4[k] >> 15) & 0x00010001u) * 0xFFFFu;
        y[k] = j < NJ ? q4[k] & negative : q4[k] & ~negative;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        constexpr uint32_t kAbs = 0x7FFF7FFFu;
        const uint32_t f[4] = {x0[2 * h], x1[2 * h], x0[2 * h + 1], x1[2 * h + 1]};
        const uint32_t fa[4] = {f[0] & kAbs, f[1] & kAbs, f[2] & kAbs, f[3] & kAbs};
        mma_bf16_16816(a4[(2 * jp + h) & 3], f, y[2 * h], y[2 * h + 1]);
        mma_bf16_16816(m, fa, y[2 * h] & kAbs, y[2 * h + 1] & kAbs);
      }
    }
  }
  float a[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) a[e] = (a4[0][e] + a4[1][e]) + (a4[2][e] + a4[3][e]);
  float size = 0.f;   // greatest S of the warp's pages
  unsigned high = 0;  // and greatest score of those that compete for a place
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float best = -INFINITY;  // of query heads 2 kcol, 2 kcol + 1
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (2 * kcol + e >= G) continue;
      best = fmaxf(best, a[2 * r + e]);
      size = m[2 * r + e] < INFINITY ? fmaxf(size, m[2 * r + e]) : INFINITY;  // NaN: infinite
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, off));
    const int pg = pg0 + 8 * r;
    if (kcol == 0 && pg < pages) out.key[pg] = sortable(best);
    if (pg >= p.n_first && pg < pages - p.n_last) high = max(high, sortable(best));
  }
  const unsigned bits = __reduce_max_sync(0xffffffffu, __float_as_uint(size));  // in the order of magnitudes
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0 && pg0 < pages) out.size[group] = bits, out.high[group] = high;
}

template <int D>
__global__ void __launch_bounds__(kScoreThreads, 4) page_score_kernel(const __grid_constant__ PageSelectParams p) {
  const int hk = blockIdx.y % p.hkv, b = blockIdx.y / p.hkv;
  __shared__ int sw[kMaxPairs];
  for (int i = threadIdx.x; i < kMaxPairs; i += kScoreThreads) sw[i] = p.win.w[i];
  pdl_launch_dependents();
  pdl_wait();
  const int len = select_len(p, b);
  const int pages = (len + (1 << p.page_log2) - 1) >> p.page_log2;
  if (pages <= p.n_sel || static_cast<long long>(blockIdx.x) * (kScoreThreads / 2) >= pages) return;
  __syncthreads();
  score_group<D>(p, b, hk, len, pages, blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5), sw,
                 Scores(p, b * p.hkv + hk));
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
  unsigned char mark[kAgain];
  unsigned least[32], greatest[32], size[32];
  unsigned key[kCandidates];
  int page[kCandidates];
  int groups[kCandidates / kGroup], n_groups, n_kept;
  int w[kMaxPairs];
};

// Narrows [lo, hi], which holds the need-th highest of the keys that each(f) calls
// f(i, key, j) for, until it is one key, or all of its `count` keys are needed, or they
// are at most `few`.  On return `need` counts within [lo, hi].  Each round takes kBinBits
// off the range; a rank that the keys do not hold ends the search where it stands.
template <typename K, typename Each>
__device__ __forceinline__ void narrow(SelectShared* sh, Each each, K& lo, K& hi, int& need, int& count, int few) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x;
  while (lo < hi && count > few && count != need) {
    const int shift = max(0, static_cast<int>(sizeof(K)) * 8 - leading_zeros(hi - lo) - kBinBits);
    for (int i = tid; i < kBins; i += T) sh->hist[i] = 0;
    __syncthreads();
    if (tid == 0) sh->lo = sh->hi = lo, sh->need = need, sh->count = count;  // what a bin with the rank replaces
    each([&](int, K k, int) {
      if (k >= lo && k <= hi) atomicAdd(&sh->hist[static_cast<int>((k - lo) >> shift)], 1);
    });
    __syncthreads();
    // the bin of the need-th, counted from the top: eight bins a thread
    int n[8], sum = 0, incl = 0;
    const int top = kBins - 1 - 8 * tid;
    if (tid < kBins / 8) {
      const int4 x = *reinterpret_cast<const int4*>(&sh->hist[top - 3]), y = *reinterpret_cast<const int4*>(&sh->hist[top - 7]);
      n[0] = x.w, n[1] = x.z, n[2] = x.y, n[3] = x.x, n[4] = y.w, n[5] = y.z, n[6] = y.y, n[7] = y.x;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += n[j];
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
        int bin = top, in = n[0];
#pragma unroll
        for (int j = 1; j < 8; ++j)
          if (before + in < need) before += in, bin = top - j, in = n[j];
        const K edge = lo + (static_cast<K>(bin) << shift);
        const K span = (static_cast<K>(1) << shift) - 1;
        sh->lo = edge;
        sh->hi = hi - edge < span ? hi : edge + span;
        sh->need = need - before;
        sh->count = in;
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

// This thread's pages: 32 j + lane of its warp's segment of the list.  The scores of
// up to kMine of them are held in registers.
struct Mine {
  int first, rounds;  // of the warp: every lane makes the same rounds
  __device__ Mine(int pages) {
    const int warps = blockDim.x >> 5;
    rounds = ((pages + warps - 1) / warps + 31) >> 5;
    first = static_cast<int>(threadIdx.x >> 5) * rounds * 32 + (threadIdx.x & 31);
  }
};

// Writes, in order, the pages for which kept(i) is set, and the first `ties` for which
// tie(i) is.
template <typename Kept, typename Tie>
__device__ __forceinline__ void emit(SelectShared* sh, const Mine& mine, int pages, int ties, int* out, Kept kept, Tie tie) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned below = (1u << lane) - 1;
  int a = 0, t = 0;
  for (int j = 0; j < mine.rounds; ++j) {
    const int i = mine.first + 32 * j;
    a += __popc(__ballot_sync(0xffffffffu, i < pages && kept(i)));
    t += __popc(__ballot_sync(0xffffffffu, i < pages && tie(i)));
  }
  __syncthreads();  // the search still reads these
  if (lane == 0) sh->warp_n[0][warp] = a, sh->warp_n[1][warp] = t;
  __syncthreads();
  a = __reduce_add_sync(0xffffffffu, lane < warp ? sh->warp_n[0][lane] : 0);
  t = __reduce_add_sync(0xffffffffu, lane < warp ? sh->warp_n[1][lane] : 0);
  for (int j = 0; j < mine.rounds; ++j) {
    const int i = mine.first + 32 * j;
    const bool k = i < pages && kept(i), e = i < pages && tie(i);
    const unsigned ma = __ballot_sync(0xffffffffu, k), mt = __ballot_sync(0xffffffffu, e);
    const int ai = a + __popc(ma & below), ti = t + __popc(mt & below);
    if (k || (e && ti < ties)) out[ai + min(ti, ties)] = i;
    a += __popc(ma);
    t += __popc(mt);
  }
}

// The 64-bit score of a page, by a warp: four lanes a query head, each d/4 elements.
// One order of sums for every page.
template <int D>
__device__ __forceinline__ u64 exact_score(const PageSelectParams& p, const int* windows, int b, int hk, int len, int page) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, G = p.hq / p.hkv;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + b * p.q_stride +
                                                  (static_cast<long long>(hk) * G + min(g, G - 1)) * D);
  // every load under way, then a rolled loop over the pieces: this runs for a few pages
  // a launch, and the fetch of straight-line code took longer than its execution
  uint4 xs[D / 32], mns[D / 32], mxs[D / 32];
#pragma unroll
  for (int j = 0; j < D / 32; ++j) xs[j] = q[4 * j + c];
  const int entry = pool_page(p, p.page_table[static_cast<long long>(b) * p.max_pages + page]);
  const int near = page_distance(p, len, page);
  const uint4* bounds = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.bounds) +
                                                       (static_cast<long long>(max(entry, 0)) * p.hkv + hk) * 2 * D);
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    mns[j] = entry >= 0 ? bounds[4 * j + c] : zero;
    mxs[j] = entry >= 0 ? bounds[D / 8 + 4 * j + c] : zero;
  }
  double part[8] = {0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};  // side by side: a chain of fp64 sums is slow
#pragma unroll 1
  for (int j = 0; j < D / 32; ++j) {
    const uint4 x = xs[j], mn = mns[j], mx = mxs[j];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w = k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w;
      const uint32_t l = k == 0 ? mn.x : k == 1 ? mn.y : k == 2 ? mn.z : mn.w;
      const uint32_t h = k == 0 ? mx.x : k == 1 ? mx.y : k == 2 ? mx.z : mx.w;
      const bool on = near <= windows[16 * j + 4 * c + k];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const double y = e ? bf16hi_to_f32(w) : bf16lo_to_f32(w);
        const double best = fmax(y * (e ? bf16hi_to_f32(l) : bf16lo_to_f32(l)), y * (e ? bf16hi_to_f32(h) : bf16lo_to_f32(h)));
        part[2 * k + e] += on ? best : 0.0;
      }
    }
  }
  double s = ((part[0] + part[1]) + (part[2] + part[3])) + ((part[4] + part[5]) + (part[6] + part[7]));
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) s = fmax(s, __shfl_xor_sync(0xffffffffu, s, off));
  return sortable(s);
}

// Of the `close` pages in sh->again marks the `need` best by 64-bit scores, equal ones
// by lower index.
template <int D>
__device__ __forceinline__ void mark_best(SelectShared* sh, const PageSelectParams& p, int b, int hk, int len, int close,
                                          int need) {
  const int tid = threadIdx.x;
  if (close > need) {
    for (int i = tid >> 5; i < close; i += blockDim.x >> 5) {
      const u64 x = exact_score<D>(p, sh->w, b, hk, len, sh->again[i]);
      if ((tid & 31) == 0) sh->cand[i] = x;
    }
    __syncthreads();
  }
  for (int i = tid; i < close; i += blockDim.x) {
    int before = 0;
    if (close > need)
      for (int j = 0; j < close; ++j)
        before += sh->cand[j] > sh->cand[i] || (sh->cand[j] == sh->cand[i] && sh->again[j] < sh->again[i]);
    sh->mark[i] = before < need;
  }
  __syncthreads();
}

}  // namespace

// kScore: short lists, whose pages this kernel scores itself, to shared memory.
// kMine: scores that a thread holds in registers; 0: more pages than that, the
// scores are read again from memory by each pass.  128 to
// kSelectThreads threads.
template <int D, int kMine, bool kScore>
__global__ void __launch_bounds__(kSelectThreads) page_select_kernel(const __grid_constant__ PageSelectParams p) {
  __shared__ __align__(16) SelectShared s;
  SelectShared* sh = &s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x, warps = T >> 5;
  const int hk = blockIdx.x % p.hkv, b = blockIdx.x / p.hkv;
  for (int i = tid; i < kMaxPairs; i += T) sh->w[i] = p.win.w[i];  // read after many barriers
  pdl_launch_dependents();
  pdl_wait();
  const int len = select_len(p, b);
  const int pages = (len + (1 << p.page_log2) - 1) >> p.page_log2;
  u64* keys = p.keys + static_cast<long long>(blockIdx.x) * p.max_pages;  // 64-bit scores, where they are needed
  __shared__ unsigned s_key[kScore ? kShort : 1], s_size[kScore ? kShort / kGroup : 1], s_high[kScore ? kShort / kGroup : 1];
  const Scores scores = kScore ? Scores(s_key, s_size, s_high) : Scores(p, blockIdx.x);
  int* out = p.selected + (static_cast<long long>(b) * p.hkv + hk) * p.n_sel;
  if (pages <= p.n_sel) {
    for (int i = tid; i < p.n_sel; i += T) out[i] = i < pages ? i : -1;
    return;
  }
  if constexpr (kScore) {
    __syncthreads();
    for (int i = warp; i * kGroup < pages; i += warps) score_group<D>(p, b, hk, len, pages, i, sh->w, scores);
    __syncthreads();
  }
  // pages [i0, i1) compete for `places`
  const int i0 = p.n_first, i1 = pages - p.n_last, places = p.n_sel - p.n_first - p.n_last;
  const Mine mine(pages);
  auto forced = [&](int i) { return i < i0 || i >= i1; };
  auto never = [](int) { return false; };
  if (places == 0) return emit(sh, mine, pages, 0, out, forced, never);

  unsigned lo = ~0u, hi = 0u, size = 0u;
  const int groups = (pages + kGroup - 1) / kGroup;
  auto range = [&]() {  // of the block, and the greatest S; sh->n and sh->above are cleared
    if (tid == 0) sh->n = sh->above = sh->n_groups = sh->n_kept = 0;
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    size = __reduce_max_sync(0xffffffffu, size);
    if (lane == 0) sh->least[warp] = lo, sh->greatest[warp] = hi, sh->size[warp] = size;
    __syncthreads();
    const int w = min(lane, warps - 1);
    lo = __reduce_min_sync(0xffffffffu, sh->least[w]);
    hi = __reduce_max_sync(0xffffffffu, sh->greatest[w]);
    size = __reduce_max_sync(0xffffffffu, sh->size[w]);
  };
  // twice the largest error of a score; the constant covers products that vanish in fp32
  auto slack_of = [](unsigned size) { return 2.f * (kEps * __uint_as_float(size) + 1e-30f); };
  auto below = [](unsigned k, float by) { return sortable(from_sortable(k) - by); };

  // ---- few places in a long list: only groups whose highest score is among the
  // `places` highest of the groups, or close below, hold a kept page
  const SelectGroups rivals = select_groups(pages, p.n_first, p.n_last, places);
  if (rivals.search) {
    auto each_group = [&](auto f) {
#pragma unroll 4
      for (int i = rivals.first + tid; i < rivals.first + rivals.count; i += T) f(i, scores.high[i], 0);
    };
    each_group([&](int i, unsigned k, int) {
      lo = min(lo, k);
      hi = max(hi, k);
      size = max(size, scores.size[i]);
    });
    range();
    const float slack = slack_of(size);
    if (slack < INFINITY) {
      const unsigned top = hi;
      int need = places, count = rivals.count;
      narrow(sh, each_group, lo, hi, need, count, kFewGroups);
      const unsigned least = below(lo, slack);
      each_group([&](int i, unsigned k, int) {
        if (k < least) return;
        const int at = atomicAdd(&sh->n_groups, 1);
        if (at < kCandidates / kGroup) sh->groups[at] = i;
      });
      __syncthreads();
      const int n = sh->n_groups;
      if (n <= kCandidates / kGroup) {
        for (int x0 = 0; x0 < n * kGroup; x0 += T) {
          const int x = x0 + tid, i = x < n * kGroup ? sh->groups[x / kGroup] * kGroup + x % kGroup : pages;
          const unsigned k = i < pages && !forced(i) ? scores.key[i] : 0;
          const unsigned in = __ballot_sync(0xffffffffu, k >= least);  // least is above 0: `places` pages or more
          int at = 0;
          if (lane == 0) at = atomicAdd(&sh->n, __popc(in));
          at = __shfl_sync(0xffffffffu, at, 0) + __popc(in & ((1u << lane) - 1));
          if (k >= least) sh->key[at] = k, sh->page[at] = i;
        }
        __syncthreads();
        const int m = sh->n;
        auto each_candidate = [&](auto f) {
          for (int x = tid; x < m; x += T) f(x, sh->key[x], 0);
        };
        lo = least, need = places, count = m;
        hi = top;
        narrow(sh, each_candidate, lo, hi, need, count, 1);
        const unsigned cut_lo = below(lo, slack), cut_hi = below(hi, -slack);
        __syncthreads();
        if (tid == 0) sh->n = 0;
        __syncthreads();
        for (int x = tid; x < m; x += T) {
          const unsigned k = sh->key[x];
          if (k > cut_hi) {
            atomicAdd(&sh->above, 1);
          } else if (k >= cut_lo) {
            const int at = atomicAdd(&sh->n, 1);
            if (at < kAgain) sh->again[at] = sh->page[x];
          }
        }
        __syncthreads();
        const int close = sh->n;
        if (close <= kAgain) {
          mark_best<D>(sh, p, b, hk, len, close, places - sh->above);
          // the kept candidates by index, between the forced pages
          for (int x = tid; x < m; x += T) {
            const unsigned k = sh->key[x];
            bool keep = k > cut_hi;
            if (!keep && k >= cut_lo) {
              int at = 0;
              while (sh->again[at] != sh->page[x]) ++at;
              keep = sh->mark[at];
            }
            if (keep) sh->hist[atomicAdd(&sh->n_kept, 1)] = sh->page[x];
          }
          __syncthreads();
          for (int x = tid; x < p.n_sel; x += T) {
            if (x < i0) {
              out[x] = x;
            } else if (x >= i0 + places) {
              out[x] = pages - p.n_sel + x;
            } else {
              const int i = sh->hist[x - i0];
              int before = 0;
              for (int y = 0; y < places; ++y) before += sh->hist[y] < i;
              out[i0 + before] = i;
            }
          }
          return;
        }
      }
    }
    __syncthreads();
    lo = ~0u, hi = 0u;
  }

  // ---- every page
  unsigned mk[kMine ? kMine : 1];
  for (int i = tid; i < groups; i += T) size = max(size, scores.size[i]);
  if constexpr (kMine > 0) {
#pragma unroll
    for (int j = 0; j < kMine; ++j) mk[j] = scores.key[min(mine.first + 32 * j, pages - 1)];  // all under way at once
  }
  auto each = [&](auto f) {
    if constexpr (kMine > 0) {
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const int i = mine.first + 32 * j;
        if (j < mine.rounds && !forced(i)) f(i, mk[j], j);
      }
    } else {
#pragma unroll 8
      for (int i = i0 + tid; i < i1; i += T) f(i, scores.key[i], 0);
    }
  };
  each([&](int, unsigned k, int) { lo = min(lo, k), hi = max(hi, k); });
  range();
  const float slack = slack_of(size);
  bool again = !(slack < INFINITY);
  if (!again) {
    int need = places, count = i1 - i0;
    narrow(sh, each, lo, hi, need, count, 1);
    const unsigned cut_lo = below(lo, slack), cut_hi = below(hi, -slack);
    int above = 0;
    unsigned bits = 0, unsure = 0;  // this thread's pages that are kept, and that are scored again
    each([&](int i, unsigned k, int j) {
      if (k > cut_hi) {
        ++above;
        bits |= 1u << j;
      } else if (k >= cut_lo) {
        unsure |= 1u << j;
        const int at = atomicAdd(&sh->n, 1);
        if (at < kAgain) sh->again[at] = i;
      }
    });
    above = __reduce_add_sync(0xffffffffu, above);
    if (lane == 0) atomicAdd(&sh->above, above);
    __syncthreads();
    const int close = sh->n;
    need = places - sh->above;  // of the close ones
    again = close > kAgain;
    if (!again) {
      mark_best<D>(sh, p, b, hk, len, close, need);
      auto chosen = [&](int i) {
        int at = 0;
        while (sh->again[at] != i) ++at;
        return sh->mark[at] != 0;
      };
      if constexpr (kMine > 0) {
        for (; unsure; unsure &= unsure - 1) {
          const int j = __ffs(unsure) - 1;
          if (chosen(mine.first + 32 * j)) bits |= 1u << j;
        }
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          const int i = mine.first + 32 * j;
          if (j < mine.rounds && i < pages && forced(i)) bits |= 1u << j;
        }
        const int n = __reduce_add_sync(0xffffffffu, __popc(bits));
        if (lane == 0) sh->warp_n[1][warp] = n;
        __syncthreads();
        int at = __reduce_add_sync(0xffffffffu, lane < warp ? sh->warp_n[1][lane] : 0);
        if (!n) return;
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          const unsigned m = __ballot_sync(0xffffffffu, bits >> j & 1);
          if (bits >> j & 1) out[at + __popc(m & ((1u << lane) - 1))] = mine.first + 32 * j;
          at += __popc(m);
        }
      } else {
        auto kept = [&](int i) {
          if (forced(i)) return true;
          const unsigned k = scores.key[i];
          return k > cut_hi || (k >= cut_lo && chosen(i));
        };
        emit(sh, mine, pages, 0, out, kept, never);
      }
      return;
    }
  }

  // every score in 64 bits
  for (int i = i0 + warp; i < i1; i += warps) {
    const u64 x = exact_score<D>(p, sh->w, b, hk, len, i);
    if (lane == 0) keys[i] = x;
  }
  __syncthreads();
  if (tid == 0) sh->n = 0;
  auto each64 = [&](auto f) {
    for (int i = i0 + tid; i < i1; i += T) f(i, keys[i], 0);
  };
  u64 lo64 = ~0ull, hi64 = 0;
  each64([&](int, u64 k, int) { lo64 = min(lo64, k), hi64 = max(hi64, k); });
  block_range(sh, lo64, hi64);
  int need = places, count = i1 - i0;
  narrow(sh, each64, lo64, hi64, need, count, kAgain);
  // kept: every key above `cut`, and the first `ties` that equal it
  u64 cut = lo64;
  int ties = need;
  if (lo64 < hi64 && count == need) {  // all of the range
    cut = lo64 ? lo64 - 1 : 0;
    ties = lo64 ? 0 : count;
  } else if (lo64 < hi64) {
    each64([&](int, u64 k, int) {
      if (k >= lo64 && k <= hi64) sh->cand[atomicAdd(&sh->n, 1)] = k;
    });
    __syncthreads();
    for (int i = tid; i < count; i += T) {
      const u64 own = sh->cand[i];
      int above = 0, equal = 0;
      for (int j = 0; j < count; ++j) {
        above += sh->cand[j] > own;
        equal += sh->cand[j] == own;
      }
      if (above < need && need <= above + equal) {  // so do its equals, with the same values
        sh->cut = own;
        sh->need = need - above;
      }
    }
    __syncthreads();
    cut = sh->cut;
    ties = sh->need;
  }
  emit(sh, mine, pages, ties, out, [&](int i) { return forced(i) || keys[i] > cut; },
       [&](int i) { return !forced(i) && keys[i] == cut; });
}

template <int D>
static cudaError_t launch_select(const PageSelectParams& p, cudaStream_t s) {
  const int lists = p.batch * p.hkv;
  // The lengths are on the device: the form goes by the table's width.  Short sequences in
  // wide tables pay for it (32 lists x 4 of up to 1024 pages in tables of 32768: 108 us with
  // their decode, 44 in tables of 1024).
  // short lists: a warp a group of pages, so that an SM holds several of many lists
  const int threads = p.max_pages <= 128 ? 128 : p.max_pages <= 256 ? 256 : kSelectThreads;
  if (p.max_pages <= kShort) return launch_pdl(page_select_kernel<D, kHeld, true>, lists, threads, 0, s, p);
  const int per = kScoreThreads / 2;
  const dim3 grid((p.max_pages + per - 1) / per, lists);
  cudaError_t e = launch_pdl(page_score_kernel<D>, grid, kScoreThreads, 0, s, p);
  if (e != cudaSuccess) return e;
  if (p.max_pages > kSelectThreads * kHeld) return launch_pdl(page_select_kernel<D, 0, false>, lists, kSelectThreads, 0, s, p);
  return launch_pdl(page_select_kernel<D, kHeld, false>, lists, p.max_pages <= 256 * kHeld ? 256 : kSelectThreads, 0, s, p);
}

cudaError_t launch_page_select(const PageSelectParams& p, cudaStream_t s) {
  return p.d == 64 ? launch_select<64>(p, s) : launch_select<128>(p, s);
}

}  // namespace atf
