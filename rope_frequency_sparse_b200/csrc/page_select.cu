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
// Products of two bf16 numbers are exact in fp32; their sums are fp64, so that the
// order of close pages does not hang on the summation order.  Kept are the first
// n_first and last n_last pages and the highest scores, equal ones by lower
// index, as an ascending list.
//
// Reads 4 d bytes per page and kv head, the bound of the first kernel: d/16 lanes
// per page read its two rows whole.  The second kernel finds each list's
// threshold by radix digits of the scores' order-preserving bit patterns and emits
// the kept indices in order.
#include <cuda_bf16.h>

#include "atf_internal.cuh"
#include "ptx.cuh"

namespace atf {

namespace {

constexpr int kScoreThreads = 128;
constexpr int kSelThreads = 512;

__device__ __forceinline__ int select_len(const PageSelectParams& p, int b) {
  const int len = p.kv_len[b];
  const long long cap = static_cast<long long>(p.max_pages) << p.page_log2;
  if (len > cap) {
    atomicCAS(p.err, 0u, kErrBadLength);
    return static_cast<int>(cap);
  }
  return len < 0 ? 0 : len;
}

// Bit pattern whose unsigned order is the number's (-0 as +0).
__device__ __forceinline__ unsigned long long sortable(double x) {
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));
  return (u >> 63) ? ~u : u | (1ull << 63);
}
constexpr unsigned long long kKeep = ~0ull;  // above every score

}  // namespace

template <int D>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const __grid_constant__ PageSelectParams p) {
  constexpr int NC = D / 16, kPages = kScoreThreads / NC;  // pages of a CTA
  __shared__ __align__(16) float sq[8 * D];
  __shared__ int sw[kMaxPairs];
  const int tid = threadIdx.x, c = tid % NC;
  const int hk = blockIdx.y % p.hkv, b = blockIdx.y / p.hkv;
  const int G = p.hq / p.hkv;
  const int len = select_len(p, b), ps = 1 << p.page_log2;
  const int pages = (len + ps - 1) >> p.page_log2;
  if (static_cast<long long>(blockIdx.x) * kPages >= pages) return;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + b * p.q_stride + static_cast<long long>(hk) * G * D;
  for (int i = tid; i < G * D; i += kScoreThreads) sq[i] = __bfloat162float(q[i]);
  for (int i = tid; i < D / 2; i += kScoreThreads) sw[i] = p.win.w[i];
  __syncthreads();
  const int pg = blockIdx.x * kPages + tid / NC;
  const bool live = pg < pages;
  int page = live ? p.page_table[static_cast<long long>(b) * p.max_pages + pg] : -1;
  if (live && (page < 0 || page >= p.num_pages)) {
    atomicCAS(p.err, 0u, kErrBadPage);
    page = -1;
  }
  const int near = len - 1 - min(pg * ps + ps - 1, len - 1);
  float mn[16], mx[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) mn[k] = mx[k] = 0.f;
  if (page >= 0) {
    const uint4* row = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.bounds) +
                                                      (static_cast<long long>(page) * p.hkv + hk) * 2 * D + 16 * c);
    const uint4 v[4] = {row[0], row[1], row[D / 8], row[D / 8 + 1]};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t l[4] = {v[j].x, v[j].y, v[j].z, v[j].w}, h[4] = {v[2 + j].x, v[2 + j].y, v[2 + j].z, v[2 + j].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (near <= sw[8 * c + 4 * j + k]) {
          mn[8 * j + 2 * k] = bf16lo_to_f32(l[k]);
          mn[8 * j + 2 * k + 1] = bf16hi_to_f32(l[k]);
          mx[8 * j + 2 * k] = bf16lo_to_f32(h[k]);
          mx[8 * j + 2 * k + 1] = bf16hi_to_f32(h[k]);
        }
    }
  }
  double best = -INFINITY;
  for (int g = 0; g < G; ++g) {
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float x = sq[g * D + 16 * c + k];
      s += static_cast<double>(fmaxf(x * mn[k], x * mx[k]));
    }
#pragma unroll
    for (int off = 1; off < NC; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    best = fmax(best, s);
  }
  if (live && c == 0) {
    const bool forced = pg < p.n_first || pg >= pages - p.n_last;
    p.keys[(static_cast<long long>(b) * p.hkv + hk) * p.max_pages + pg] = forced ? kKeep : sortable(best);
  }
}

__global__ void __launch_bounds__(kSelThreads) page_select_kernel(const __grid_constant__ PageSelectParams p) {
  __shared__ int hist[256];
  __shared__ int s_digit, s_need;
  __shared__ int s_warp[2][kSelThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.x % p.hkv, b = blockIdx.x / p.hkv;
  const int len = select_len(p, b);
  const int pages = (len + (1 << p.page_log2) - 1) >> p.page_log2;
  const unsigned long long* keys = p.keys + (static_cast<long long>(b) * p.hkv + hk) * p.max_pages;
  int* out = p.selected + (static_cast<long long>(b) * p.hkv + hk) * p.n_sel;
  if (pages <= p.n_sel) {
    for (int i = tid; i < p.n_sel; i += kSelThreads) out[i] = i < pages ? i : -1;
    return;
  }
  // the threshold: digits of the n_sel-th highest key from the top, until the keys
  // that share them are all kept
  unsigned long long prefix = 0, mask = 0;
  int need = p.n_sel;  // still to be kept among the keys that match prefix under mask
  for (int shift = 56; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < pages; i += kSelThreads) {
      const unsigned long long k = keys[i];
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int d = 255, n = need;
      while (d > 0 && hist[d] < n) n -= hist[d--];
      s_digit = d;
      s_need = n;
    }
    __syncthreads();
    need = s_need;
    const bool all = hist[s_digit] == need;
    prefix |= static_cast<unsigned long long>(s_digit) << shift;
    mask |= 255ull << shift;
    __syncthreads();
    if (all) break;
  }
  // keys above the prefix, and the first `need` that match it, in index order
  int done = 0, ties = 0;
  for (int i0 = 0; i0 < pages; i0 += kSelThreads) {
    const int i = i0 + tid;
    const unsigned long long k = i < pages ? keys[i] & mask : 0;
    const bool above = i < pages && k > prefix, tie = i < pages && k == prefix;
    const unsigned ba = __ballot_sync(0xffffffffu, above), bt = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) {
      s_warp[0][warp] = __popc(ba);
      s_warp[1][warp] = __popc(bt);
    }
    __syncthreads();
    int a0 = 0, t0 = ties, an = 0, tn = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w == warp) a0 = an, t0 = ties + tn;
      an += s_warp[0][w];
      tn += s_warp[1][w];
    }
    const unsigned below = (1u << lane) - 1;
    a0 += __popc(ba & below);
    t0 += __popc(bt & below);
    // kept so far: every key above, and ties up to `need`
    if (above || (tie && t0 < need)) out[done + a0 + min(t0, need) - min(ties, need)] = i;
    done += an + min(ties + tn, need) - min(ties, need);
    ties += tn;
    __syncthreads();
  }
}

cudaError_t launch_page_select(const PageSelectParams& p, cudaStream_t s) {
  const int per = kScoreThreads / (p.d / 16);
  const dim3 grid((p.max_pages + per - 1) / per, p.batch * p.hkv);
  p.d == 64 ? page_score_kernel<64><<<grid, kScoreThreads, 0, s>>>(p)
            : page_score_kernel<128><<<grid, kScoreThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  page_select_kernel<<<p.batch * p.hkv, kSelThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace atf
