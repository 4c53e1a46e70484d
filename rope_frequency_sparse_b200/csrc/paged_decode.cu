// paged_decode.cu -- one rotated query per sequence against a paged key-value
// cache, with the per-pair distance windows of the method; over all pages of a
// sequence or over a given list of them.
//
//   logit(n) = (1/sqrt d) sum_{i : L-1-n <= W_i} q_pair_i . k_pair_i,  softmax, P V
//
// HBM-bound: 2 (d + 2 * active pairs) bytes and 4 * (query heads per kv head) *
// d flops a key.  Keys are stored per page in 8-pair chunks, so a page whose keys
// lie beyond the windows of the low chunks is read from its first live chunk on:
// one TMA box of d/16 chunks starts at that chunk, and what reaches past the last
// chunk is filled with zeros without being read.
//
// Lengths and page tables stay on the device, so a captured call follows growing
// sequences.  The work of the batch is one list of 128-key tiles, ordered by
// (sequence, kv head, tile) and weighted by the bytes each tile reads; each of
// 148 CTAs (one per SM) takes an equal piece of it.  A CTA finds its piece from
// the lengths alone: closed-form tile weights, a block-wide prefix sum over the
// batch and a binary search.  A sequence and head that lies within one CTA is
// finished there; of the others a CTA can hold at most two pieces (the first and
// the last of its list), each written as a partial (sum, max, row sum), and a
// second kernel joins them.
//
// Inside a CTA a producer warp walks the list, looks pages up one tile ahead and
// fills a ring of tiles with TMA; four consumer warps take 32 keys of each tile.
// Keys are the M rows and query heads (up to 8) the N columns of the warp-level
// MMAs, S^T = K~ Q~^T and O^T += V^T P^T, so no row of them is padding; P^T
// goes from accumulators to operand by a register transpose (movmatrix).  P is
// rounded to bf16 for the product with V (relative 2^-9 a weight, as the prefill
// and decode do); its sums, the maxima and O stay fp32.
#include <cuda_bf16.h>

#include <atomic>

#include "atf_internal.cuh"
#include "ptx.cuh"

namespace atf {

namespace {

constexpr int kPdConsumers = 4;
constexpr int kPdThreads = (kPdConsumers + 1) * 32;
constexpr int kTileKeys = 128;
constexpr int kMaxTilePages = 8;  // pages of 16
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct PdCfg {
  static constexpr int NC = D / 16;
  static constexpr int HALF = kTileKeys * D * 2;  // bytes of a tile's keys, and of its values
  static constexpr int STAGE = 2 * HALF;
  static constexpr int NSTG = D == 128 ? 3 : 6;
  static constexpr int Q = 8 * D * 2;
  static constexpr int OROW = D + 4;              // padded so that a warp's stores spread over the banks
  static constexpr int MERGE = kPdConsumers * 8 * OROW * 4;
};

struct StageInfo {
  int key0[kMaxTilePages];   // first key of each page of the tile
  int keys[kMaxTilePages];   // its live keys (0: no such page)
  int clo;                   // first chunk loaded
  int len;                   // keys of the sequence
  int b, hk;
  int flags;                 // kFirst, kLast, kEnd
  int slot;                  // partial slot of the CTA, -1: the whole sequence, write the output
};
constexpr int kFirst = 1, kLast = 2, kEnd = 4;

template <int D>
struct PdShared {
  uint64_t full[PdCfg<D>::NSTG], empty[PdCfg<D>::NSTG];
  uint64_t join[2];  // the consumer warps meet before and after their states are joined
  StageInfo info[PdCfg<D>::NSTG];
  int w[kMaxPairs];
  int abort;
  long long scan[kPdThreads / 32];
  int start_b, start_ok;
  long long start_base, total;
  float mw[kPdConsumers][8], lw[kPdConsumers][8];
};

template <int D>
constexpr int pd_smem_bytes() {
  return PdCfg<D>::NSTG * (PdCfg<D>::STAGE + PdCfg<D>::Q) + PdCfg<D>::MERGE + static_cast<int>(sizeof(PdShared<D>)) + 1024;
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ int clamped_len(const PagedDecodeParams& p, int b) {
  const int len = p.kv_len[b];
  const long long cap = static_cast<long long>(p.max_pages) << p.page_log2;
  if (len > cap) {
    atomicCAS(p.err, 0u, kErrBadLength);
    return static_cast<int>(cap);
  }
  return len < 0 ? 0 : len;
}

// Tiles of a sequence (at least one, so that an empty sequence writes its zeros).
__device__ __forceinline__ int tiles_of(const PagedDecodeParams& p, int len) {
  int keys = len;
  if (p.selected) {
    const int pages = (len + (1 << p.page_log2) - 1) >> p.page_log2;
    keys = min(p.n_sel, pages) << p.page_log2;
  }
  return max(1, (keys + kTileKeys - 1) / kTileKeys);
}

// Weight of tiles [0, t) of a sequence in 32-byte reads a key: value row plus
// live key chunks.  Chunk c is out of reach of the whole tiles before (len - W -
// 1) / 128, W the window of its last pair.  A list of pages weighs full rows.
template <int NC>
__device__ __forceinline__ long long tile_weight(const PagedDecodeParams& p, const int* w, int len, int t) {
  long long x = 2LL * NC * t;
  if (!p.selected) {
#pragma unroll
    for (int c = 0; c < NC; ++c) x -= min(t, max(0, (len - w[8 * c + 7] - 1) / kTileKeys));
  }
  return x;
}

// Smallest t in [0, tiles] with tile_weight(t) >= x.
template <int NC>
__device__ __forceinline__ int tile_at(const PagedDecodeParams& p, const int* w, int len, int tiles, long long x) {
  int lo = 0, hi = tiles;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (tile_weight<NC>(p, w, len, mid) >= x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kPdThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ PagedDecodeParams p) {
  using C = PdCfg<D>;
  constexpr int NC = C::NC, NSTG = C::NSTG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sStage = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = sStage + NSTG * C::STAGE;
  float* sO = reinterpret_cast<float*>(sQ + NSTG * C::Q);
  PdShared<D>* sh = reinterpret_cast<PdShared<D>*>(reinterpret_cast<uint8_t*>(sO) + C::MERGE);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x, ncta = gridDim.x;
  const int G = p.hq / p.hkv;

  if (tid == 0) {
    for (int s = 0; s < NSTG; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], kPdConsumers);
    }
    mbar_init(&sh->join[0], kPdConsumers);
    mbar_init(&sh->join[1], kPdConsumers);
    sh->abort = 0;
    sh->start_ok = 0;
    fence_mbar_init();
  }
  if (tid == kPdConsumers * 32) prefetch_tmap(&tm_k), prefetch_tmap(&tm_v);
  for (int i = tid; i < kMaxPairs; i += kPdThreads) sh->w[i] = p.win.w[i];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();

  // ---- where this CTA's piece of the tile list begins
  const int per = (p.batch + kPdThreads - 1) / kPdThreads;  // sequences a thread sums
  const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = clamped_len(p, b);
    mine += tile_weight<NC>(p, sh->w, len, tiles_of(p, len)) * p.hkv;
  }
  long long incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) sh->scan[warp] = incl;
  __syncthreads();
  long long total = 0, before = incl - mine;
  for (int i = 0; i < kPdThreads / 32; ++i) {
    if (i < warp) before += sh->scan[i];
    total += sh->scan[i];
  }
  const long long from = total / ncta * cta + total % ncta * cta / ncta;
  const long long to = total / ncta * (cta + 1) + total % ncta * (cta + 1) / ncta;
  if (from < to && from >= before && from < before + mine) {
    long long base = before;
    for (int b = b0; b < b1; ++b) {
      const int len = clamped_len(p, b);
      const long long x = tile_weight<NC>(p, sh->w, len, tiles_of(p, len)) * p.hkv;
      if (from < base + x) {
        sh->start_b = b;
        sh->start_base = base;
        sh->start_ok = 1;
        break;
      }
      base += x;
    }
  }
  __syncthreads();

  if (warp == kPdConsumers) {
    // ================================================================ producer
    int it = 0;              // stages filled
    bool ok = true, has_partial0 = false;
    int meta_b = -1, meta_hk = 0, meta_last = 0;
    const int ps = 1 << p.page_log2, ppt = kTileKeys >> p.page_log2;
    int b = sh->start_b, hk = 0;
    long long base = sh->start_base;  // weight before (b, hk)
    bool more = sh->start_ok != 0;
    if (more) {
      const int len = clamped_len(p, b);
      const long long unit = tile_weight<NC>(p, sh->w, len, tiles_of(p, len));
      hk = static_cast<int>((from - base) / unit);
      base += unit * hk;
    }
    while (more && ok) {
      const int len = clamped_len(p, b);
      const int tiles = tiles_of(p, len);
      const long long unit = tile_weight<NC>(p, sh->w, len, tiles);
      const int t0 = from > base ? tile_at<NC>(p, sh->w, len, tiles, from - base) : 0;
      const int t1 = to >= base + unit ? tiles : tile_at<NC>(p, sh->w, len, tiles, to - base);
      if (t0 < t1) {
        int slot = -1;
        if (t0 > 0) {
          slot = 0;
          has_partial0 = true;
        } else if (t1 < tiles) {
          slot = 1;
          const long long x = base + tile_weight<NC>(p, sh->w, len, tiles - 1);  // where its last tile begins
          meta_b = b;
          meta_hk = hk;
          // the CTA whose piece holds x: the largest j with floor(j * total / ncta) <= x
          int lo = cta, hi = ncta - 1;
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (total / ncta * mid + total % ncta * mid / ncta <= x)
              lo = mid;
            else
              hi = mid - 1;
          }
          meta_last = lo;
          if (lane == 0) p.meta[cta] = make_int4(meta_b, meta_hk, meta_last, 0);
        }
        const int pages = (len + ps - 1) >> p.page_log2;
        const int* list = p.selected ? p.selected + (static_cast<long long>(b) * p.hkv + hk) * p.n_sel : nullptr;
        const int count = list ? min(p.n_sel, pages) : pages;
        const int* table = p.page_table + static_cast<long long>(b) * p.max_pages;
        // this lane's page of a tile: logical index (-1: none) and index in the pool
        auto look_up = [&](int t, int& logical, int& page) {
          const int i = t * ppt + lane;
          logical = page = -1;
          if (lane < ppt && i < count) {
            logical = list ? list[i] : i;
            if (logical >= pages) {
              atomicCAS(p.err, 0u, kErrBadSelect);
              logical = -1;
            }
            if (logical >= 0) {
              page = table[logical];
              if (page < 0 || page >= p.num_pages) {
                atomicCAS(p.err, 0u, kErrBadPage);
                logical = -1;
              }
            }
          }
        };
        int logical, page;
        look_up(t0, logical, page);
        for (int t = t0; t < t1; ++t) {
          int logical_next = -1, page_next = -1;
          if (t + 1 < t1) look_up(t + 1, logical_next, page_next);
          const int st = it % NSTG;
          if (it >= NSTG && !warp_wait(&sh->empty[st], ((it / NSTG) - 1) & 1, &sh->abort, p.err, 0x501)) {
            ok = false;
            break;
          }
          StageInfo* info = &sh->info[st];
          const int key0 = max(logical, 0) << p.page_log2;
          const int keys = logical >= 0 ? min(ps, len - key0) : 0;
          const int near = __reduce_max_sync(0xffffffffu, keys > 0 ? key0 + keys - 1 : -1);
          int clo = 0;
          if (near >= 0)
            while (clo < NC - 1 && sh->w[8 * clo + 7] < len - 1 - near) ++clo;
          if (lane < ppt) {
            info->key0[lane] = key0;
            info->keys[lane] = keys;
          }
          const unsigned live = __ballot_sync(0xffffffffu, keys > 0);
          const bool first = t == t0;
          if (lane == 0) {
            info->clo = clo;
            info->len = len;
            info->b = b;
            info->hk = hk;
            info->flags = (first ? kFirst : 0) | (t + 1 == t1 ? kLast : 0);
            info->slot = slot;
          }
          __syncwarp();
          uint8_t* stg = sStage + st * C::STAGE;
          if (lane == 0) {
            const uint32_t q_bytes = G * D * 2;
            mbar_arrive_expect_tx(&sh->full[st], __popc(live) * 2 * ps * D * 2 + (first ? q_bytes : 0));
            if (first)
              bulk_load(sQ + st * C::Q,
                        static_cast<const __nv_bfloat16*>(p.q) + b * p.q_stride + static_cast<long long>(hk) * G * D, q_bytes,
                        &sh->full[st]);
          }
          __syncwarp();
          if (keys > 0) {
            const int row = page * p.hkv + hk;
            tma_load_4d(stg + lane * ps * D * 2, &tm_k, &sh->full[st], 0, 0, clo, row);
            tma_load_4d(stg + C::HALF + lane * ps * D * 2, &tm_v, &sh->full[st], 0, 0, 0, row);
          }
          logical = logical_next;
          page = page_next;
          ++it;
        }
      }
      base += unit;
      if (++hk == p.hkv) hk = 0, ++b;
      more = b < p.batch && base < to;
    }
    if (ok) {  // the end mark
      const int st = it % NSTG;
      if (it >= NSTG) ok = warp_wait(&sh->empty[st], ((it / NSTG) - 1) & 1, &sh->abort, p.err, 0x502);
      if (ok && lane == 0) {
        sh->info[st].flags = kEnd;
        mbar_arrive(&sh->full[st]);
      }
    }
    if (lane == 0 && meta_b < 0) p.meta[cta] = make_int4(-1, 0, 0, 0);
    if (!has_partial0 && lane < G) {  // no piece of an earlier CTA's sequence here
      float* part = p.partials + (static_cast<long long>(cta) * 2 * 8 + lane) * (D + 2);
      part[D] = -INFINITY;
      part[D + 1] = 0.f;
    }
    if (!ok && lane == 0) {  // wait (bounded) for the copies in flight
      for (int s = 0; s < NSTG && s < it; ++s) {
        const int last = (it - 1 - s) / NSTG * NSTG + s;  // the last fill of stage s
        const long long c0 = clock64();
        while (!mbar_try_wait(&sh->full[s], (last / NSTG) & 1) && clock64() - c0 < kWaitLimitCycles) {
        }
      }
    }
    return;
  }

  // ================================================================ consumers
  const float scale = kLog2e * rsqrtf(static_cast<float>(D));
  const int kcol = lane & 3, krow = lane >> 2;  // this lane's pair in a half chunk / head pair, and key row / dim row
  const int psmask = (1 << p.page_log2) - 1, pbytes = D * 2 << p.page_log2, cbytes = 32 << p.page_log2;
  uint32_t qf[NC][2];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // of heads 2*kcol, 2*kcol + 1
  float o[D / 16][4];  // O^T: dims 16u + krow (+8), heads 2*kcol (+1)
  int joins = 0;
  // a bounded wait, so that a warp that gave up does not hold the others
  auto meet = [&](int which) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->join[which]);
    return warp_wait(&sh->join[which], joins & 1, &sh->abort, p.err, 0x504);
  };
  for (int it = 0;; ++it) {
    const int st = it % NSTG;
    if (!warp_wait(&sh->full[st], (it / NSTG) & 1, &sh->abort, p.err, 0x503)) return;
    const StageInfo* info = &sh->info[st];
    const int flags = info->flags;
    if (flags & kEnd) return;
    if (flags & kFirst) {
      const uint8_t* q = sQ + st * C::Q + krow * (D * 2) + kcol * 4;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) qf[c][e] = krow < G ? *reinterpret_cast<const uint32_t*>(q + c * 32 + e * 16) : 0u;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
#pragma unroll
      for (int u = 0; u < D / 16; ++u) o[u][0] = o[u][1] = o[u][2] = o[u][3] = 0.f;
    }
    const int clo = info->clo, qpos = info->len - 1;
    const uint32_t stg = smem_u32(sStage + st * C::STAGE);

    // ---- S^T of this warp's 32 keys, pairs beyond their window zeroed
    float s[2][4];
    int live[2];  // live keys from this 16-key block's first on
    uint32_t blk[2];  // page offset and slot of the block
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const int j = 32 * warp + 16 * mt, pg = j >> p.page_log2, off = j & psmask;
      live[mt] = info->keys[pg] - off;
      blk[mt] = static_cast<uint32_t>(pg * pbytes) | static_cast<uint32_t>(off) << 24;
      const int far = qpos - (info->key0[pg] + off);  // distance of the block's first key
      s[mt][0] = s[mt][1] = s[mt][2] = s[mt][3] = 0.f;
      const int row = off + (lane & 7) + (lane & 8);
      const uint32_t ka = stg + pg * pbytes + row * 32 + (((lane >> 4) ^ ((row >> 2) & 1)) << 4);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (c < clo) continue;
        uint32_t a[4];
        ldsm_x4(ka + (c - clo) * cbytes, a);
        if (far > sh->w[8 * c]) {  // some pair of the chunk is out of reach of some key
          const int wl = sh->w[8 * c + kcol], wh = sh->w[8 * c + 4 + kcol];
          if (far - krow > wl) a[0] = 0u;
          if (far - krow - 8 > wl) a[1] = 0u;
          if (far - krow > wh) a[2] = 0u;
          if (far - krow - 8 > wh) a[3] = 0u;
        }
        mma_bf16_16816(s[mt], a, qf[c][0], qf[c][1]);
      }
    }
    // ---- online softmax of heads 2*kcol, 2*kcol + 1
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[mt][e] = krow + (e & 2) * 4 < live[mt] ? s[mt][e] * scale : -INFINITY;
        mx[e & 1] = fmaxf(mx[e & 1], s[mt][e]);
      }
    float mu[2], corr[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], off));
      const float mn = fmaxf(m[e], mx[e]);
      mu[e] = mn == -INFINITY ? 0.f : mn;  // no live key yet
      corr[e] = ex2_approx(m[e] - mu[e]);
      m[e] = mn;
      l[e] *= corr[e];
    }
    if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
      for (int u = 0; u < D / 16; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[u][e] *= corr[e & 1];
    }
    uint32_t pb[2][2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        pr[e] = ex2_approx(s[mt][e] - mu[e & 1]);
        l[e & 1] += pr[e];
      }
      pb[mt][0] = movmatrix_t(pack_bf16x2(pr[0], pr[1]));
      pb[mt][1] = movmatrix_t(pack_bf16x2(pr[2], pr[3]));
    }
    // ---- O^T += V^T P^T
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const int key = static_cast<int>(blk[mt] >> 24) + (lane & 7) + ((lane >> 4) << 3);
      const uint32_t va = stg + C::HALF + (blk[mt] & 0xFFFFFFu);
      // rows behind the last key may hold anything: their values count as zero
      const int n = live[mt] - 2 * kcol;
      const uint32_t keep0 = n >= 2 ? 0xFFFFFFFFu : n == 1 ? 0xFFFFu : 0u;
      const uint32_t keep1 = n >= 10 ? 0xFFFFFFFFu : n == 9 ? 0xFFFFu : 0u;
#pragma unroll
      for (int u = 0; u < D / 16; ++u) {
        const int dim = 16 * u + (lane & 8);
        uint32_t a[4];
        ldsm_x4_t(va + (dim >> 6) * (128 << p.page_log2) + key * 128 + ((((dim & 63) >> 3) ^ (key & 7)) << 4), a);
        a[0] &= keep0;
        a[1] &= keep0;
        a[2] &= keep1;
        a[3] &= keep1;
        mma_bf16_16816(o[u], a, pb[mt][0], pb[mt][1]);
      }
    }
    const int b = info->b, hk = info->hk, slot = info->slot;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->empty[st]);
    if (!(flags & kLast)) continue;

    // ---- join the four warps
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], off);
      if (krow == 0) {
        sh->mw[warp][2 * kcol + e] = m[e];
        sh->lw[warp][2 * kcol + e] = l[e];
      }
    }
#pragma unroll
    for (int u = 0; u < D / 16; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) sO[(warp * 8 + 2 * kcol + (e & 1)) * C::OROW + 16 * u + krow + (e & 2) * 4] = o[u][e];
    asm volatile("bar.sync 1, 128;" ::: "memory");
    for (int i = tid; i < G * D; i += kPdConsumers * 32) {
      const int g = i / D, e = i % D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kPdConsumers; ++w) M = fmaxf(M, sh->mw[w][g]);
      float acc = 0.f, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kPdConsumers; ++w) {
        const float f = M == -INFINITY ? 0.f : ex2_approx(sh->mw[w][g] - M);
        acc += sO[(w * 8 + g) * C::OROW + e] * f;
        sum += sh->lw[w][g] * f;
      }
      const long long row = static_cast<long long>(b) * p.hq + hk * G + g;
      if (slot < 0) {
        static_cast<__nv_bfloat16*>(p.out)[row * D + e] = __float2bfloat16(M == -INFINITY ? 0.f : acc / sum);
        if (p.lse && e == 0) p.lse[row] = M == -INFINITY ? -INFINITY : (M + log2f(sum)) * kLn2;
      } else {
        float* part = p.partials + ((static_cast<long long>(cta) * 2 + slot) * 8 + g) * (D + 2);
        part[e] = acc;
        if (e == 0) {
          part[D] = M;
          part[D + 1] = sum;
        }
      }
    }
    if (!meet(1)) return;
    ++joins;
  }
}

// Joins the pieces of the sequence and head that CTA blockIdx.x began and did not
// end: its slot 1 and slot 0 of the CTAs up to meta.z.  blockIdx.y = query head.
template <int D>
__global__ void __launch_bounds__(D) paged_combine_kernel(const __grid_constant__ PagedDecodeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 meta = p.meta[blockIdx.x];
  const int G = p.hq / p.hkv, g = blockIdx.y, e = threadIdx.x;
  if (meta.x < 0) return;
  const int first = blockIdx.x, n = meta.z - first + 1;
  auto part = [&](int i) { return p.partials + ((static_cast<long long>(first + i) * 2 + (i == 0)) * 8 + g) * (D + 2); };
  float M = -INFINITY;
  for (int i = 0; i < n; ++i) M = fmaxf(M, part(i)[D]);
  float a = 0.f, l = 0.f;
  for (int i = 0; i < n; ++i) {
    const float mi = part(i)[D];
    if (mi == -INFINITY) continue;
    const float f = ex2_approx(mi - M);
    a += part(i)[e] * f;
    l += part(i)[D + 1] * f;
  }
  const long long row = static_cast<long long>(meta.x) * p.hq + meta.y * G + g;
  static_cast<__nv_bfloat16*>(p.out)[row * D + e] = __float2bfloat16(M == -INFINITY ? 0.f : a / l);
  if (p.lse && e == 0) p.lse[row] = M == -INFINITY ? -INFINITY : (M + log2f(l)) * kLn2;
}

template <int D>
static cudaError_t launch_pd(const PagedDecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  auto kern = paged_decode_kernel<D>;
  constexpr int bytes = pd_smem_bytes<D>();
  static_assert(bytes <= 227 * 1024, "shared memory budget");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<unsigned long long> configured{0};  // one bit per device; setting it twice is harmless
  if (dev >= 64 || !(configured.load(std::memory_order_acquire) & (1ull << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured.fetch_or(1ull << dev, std::memory_order_acq_rel);
  }
  kern<<<kPagedCtas, kPdThreads, bytes, s>>>(tk, tv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPagedCtas, p.hq / p.hkv);
  cfg.blockDim = dim3(D);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel<D>, p);
}

cudaError_t launch_paged_decode(const PagedDecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  return p.d == 64 ? launch_pd<64>(p, tk, tv, s) : launch_pd<128>(p, tk, tv, s);
}

}  // namespace atf
