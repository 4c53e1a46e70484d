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
// sequences.  The work of the batch is one list of tiles of 64 keys (128 for long
// caches of heads of 64), ordered by (sequence, kv head, tile) and weighed by the
// bytes each tile reads and a constant; each of 148 CTAs (one per SM) takes an equal
// piece of it.  A CTA finds its piece from the lengths alone: closed-form tile
// weights, a prefix sum over the batch and a search, 32 points at a time.  A sequence
// and head that lies within one CTA is finished there; of the others a CTA can hold
// at most two pieces (the first and the last of its list), each written as a partial
// (sum, max, row sum), and a second kernel joins them.
//
// Measured, 28 query and 4 kv heads of 128, theta 1e7, alpha 1, a few passes from a cool
// start: 887 us for four sequences of 1048576 keys (97 % of the copy rate on the bytes
// needed), 82.7 us for 64 of up to 8192 in pages of 16 (85 %), 39.6 us for one of 131072
// (74 %: about 4 us until the first tile and 3 from the last to the joined output).  Call
// after call the largest runs into the power limit: 1010 to 1045 us (82 to 85 %).
//
// Inside a CTA four producer warps walk the list and fill a ring of tiles with TMA,
// every fourth tile each; a lane looks up the page of one box of 32, a group of
// boxes ahead (one producer warp that looked pages up tile by tile held the ring
// empty: 1090 us against 941 for four sequences of 1048576 keys, 28 query and 4 kv
// heads).  Two groups of four consumer warps take the tiles in turn, 16 keys a warp (32
// of a tile of 128); at the end of a piece they leave their states to four warps that join them and write,
// and go on (joined by the consumers themselves a piece cost 1.7 us).
// Keys are the M rows and query heads (up to 8) the N columns of the warp-level
// MMAs, S^T = K~ Q~^T and O^T += V^T P^T, so no row of them is padding; P^T
// goes from accumulators to operand by a register transpose (movmatrix).  P goes into
// the product with V as two bf16 parts, a weight and what its rounding left, off by
// 2^-16 of the weight: the output is then off by its own rounding alone (rms against 64
// bits 0.0017; 0.0024 with P in one part, at 131072 keys).  The second product costs 14 us of
// 887 for four sequences of 1048576 keys (58 of 1043 at the power limit) and 0.4 of 82.7 for
// the batch of 64.  The weights' sums, the maxima and O stay fp32.
#include <cuda_bf16.h>

#include <atomic>

#include "atf_internal.cuh"
#include "ptx.cuh"

namespace atf {

namespace {

constexpr int kPdGroups = 2;  // of four warps, 16 keys of a tile apiece
constexpr int kPdConsumers = 4 * kPdGroups;
constexpr int kPdProducers = 4;  // warps that fill the ring, every fourth tile each
constexpr int kPdJoiners = 4;    // warps that join the consumers' states at the end of a piece
constexpr int kPdThreads = (kPdConsumers + kPdProducers + kPdJoiners) * 32;
constexpr int kPerLane = 4;  // sequences that a lane sums in a small batch
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;  // log2 of the largest weight
constexpr float kLn2 = 0.6931471805599453f;

template <int D, int KB_, int NSTG_>
struct PdCfg {
  static constexpr int NC = D / 16;
  static constexpr int KB = KB_;                   // blocks of 16 keys of a tile that a warp takes
  static constexpr int TILE = 64 * KB;             // keys of a tile of the work
  static constexpr int TILE_LOG2 = KB == 2 ? 7 : 6;
  static constexpr int BOXES = TILE / 16;          // of the smallest pages
  static constexpr int HALF = TILE * D * 2;        // bytes of a tile's keys, and of its values
  static constexpr int STAGE = 2 * HALF;
  static constexpr int NSTG = NSTG_;               // stages of the ring
  // A producer last saw the tile NSTG + kPdProducers before its next one consumed; a parity
  // wait needs the phase before the one it waits for completed, 2 NSTG tiles before.
  static_assert(NSTG >= kPdProducers, "stages");
  // What a tile and a sequence's head cost beside their bytes, in 32-byte reads a key.
  // Measured in two batches (28 query and 4 kv heads of 128): without them four
  // sequences of 1048576 keys take 945 us, their near tiles being larger, and 64 of
  // up to 8192 86 us, some CTAs holding ten of them; with them 893 and 83.
  static constexpr int TILE_COST = 16 / KB, PIECE_COST = 64 / KB;
  static constexpr int Q = 8 * D * 2;
  static constexpr int OROW = D + 4;              // padded so that a warp's stores spread over the banks
  static constexpr int MERGE = kPdConsumers * 8 * OROW * 4;
};

template <int D, int KB, int NSTG>
struct __align__(16) StageInfo {
  int4 tile;                // keys of the sequence; first chunk loaded | flags | slot + 1; sequence; kv head
  int2 box[PdCfg<D, KB, NSTG>::BOXES];  // first key of each box of the tile, and its live keys (0: no such page)
};
// In tile.y: bits 0-7 the first chunk loaded, 8-10 these flags, 16-17 one more than the
// CTA's partial slot (0: the whole sequence, write the output).
constexpr int kFirst = 0x100, kLast = 0x200, kEnd = 0x400;

template <int D, int KB, int NSTG>
struct PdShared {
  uint64_t full[PdCfg<D, KB, NSTG>::NSTG], empty[PdCfg<D, KB, NSTG>::NSTG];
  uint64_t left, joined;  // the consumers have left their states; the joiners are done with them
  StageInfo<D, KB, NSTG> info[PdCfg<D, KB, NSTG>::NSTG];
  int w[kMaxPairs];
  int abort;
  long long scan[kPdThreads / 32];
  int start_b, start_len;  // the sequence that this CTA's piece begins in (-1: no piece)
  long long start_base;
  float mw[kPdConsumers][8], lw[kPdConsumers][8];  // maxima and row sums that the consumers have left
  int left_b, left_hk, left_slot;                  // and of what (left_b -1: that was the last)
  int passed;                                      // stages that the first consumer has passed
};

template <int D, int KB, int NSTG>
constexpr int pd_smem_bytes() {
  return PdCfg<D, KB, NSTG>::NSTG * (PdCfg<D, KB, NSTG>::STAGE + PdCfg<D, KB, NSTG>::Q) + PdCfg<D, KB, NSTG>::MERGE + static_cast<int>(sizeof(PdShared<D, KB, NSTG>)) + 1024;
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
template <int TILE>
__device__ __forceinline__ int tiles_of(const PagedDecodeParams& p, int len) {
  int keys = len;
  if (p.selected) {
    const int pages = (len + (1 << p.page_log2) - 1) >> p.page_log2;
    keys = min(p.n_sel, pages) << p.page_log2;
  }
  return max(1, (keys - 1) / TILE + 1);
}

// Weight of tiles [0, t) of a sequence in 32-byte reads a key: value row plus
// live key chunks, and the costs above.  Chunk c is out of reach of the whole tiles
// before (len - W - 1) / TILE, W the window of its last pair.  A list of pages weighs
// full rows.
template <int D, int KB, int NSTG>
struct TileWeight {
  using C = PdCfg<D, KB, NSTG>;
  static constexpr int NC = C::NC;
  int dead[NC];
  __device__ __forceinline__ TileWeight(const PagedDecodeParams& p, const int* w, int len) {
#pragma unroll
    for (int c = 0; c < NC; ++c) dead[c] = p.selected ? 0 : max(0, len - w[8 * c + 7] - 1) >> C::TILE_LOG2;
  }
  __device__ __forceinline__ int operator()(int t) const {
    int x = (2 * NC + C::TILE_COST) * t;
#pragma unroll
    for (int c = 0; c < NC; ++c) x -= min(t, dead[c]);
    return t > 0 ? x + C::PIECE_COST : 0;
  }
};

// Smallest t in [0, tiles] with weight(t) >= x, by a warp: 32 points at a time.
template <int D, int KB, int NSTG>
__device__ __forceinline__ int tile_at(const TileWeight<D, KB, NSTG>& weight, int tiles, int x) {
  int lo = 0, hi = tiles;
  while (lo < hi) {
    const int step = (hi - lo + 32) >> 5;  // hi is a candidate too
    const int t = min(hi, lo + static_cast<int>(threadIdx.x & 31) * step + step - 1);
    const int first = __ffs(__ballot_sync(0xffffffffu, t >= hi || weight(t) >= x)) - 1;
    lo += first * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// begin(j) = floor(total * j / kPagedCtas): where the piece of CTA j begins.
struct Pieces {
  long long each;
  int rest;
  __device__ __forceinline__ explicit Pieces(long long total)
      : each(total / kPagedCtas), rest(static_cast<int>(total - each * kPagedCtas)) {}
  __device__ __forceinline__ long long begin(int j) const { return each * j + rest * j / kPagedCtas; }
};

// A stage of the ring and the parity of its next phase.
template <int N>
struct RingPos {
  int st = 0;
  uint32_t parity = 0;
  __device__ void next() {
    if (++st == N) st = 0, parity ^= 1;
  }
};

// A block of 16 keys that a warp takes of a tile.
struct Block {
  uint32_t k_at;  // this lane's first row of its keys
  int far;        // distance of its first key
  int dirty;      // chunks of which some pair is out of reach of some key: the first ones
};

// S^T of a warp's KB blocks over the chunks CLO..NC-1, the first `dirty` chunks
// masked by their pairs' windows.  Every load is issued before the first product.
template <int NC, int CLO, int KB>
__device__ __forceinline__ void qk_tile(float (*s)[4], const Block* blocks, uint32_t cbytes, uint32_t odd, const uint32_t (*qf)[2],
                                        const int* w, int krow, int kcol) {
  uint32_t a[KB][NC - CLO][4];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int j = 0; j < NC - CLO; ++j) ldsm_x4((blocks[kb].k_at + j * cbytes) ^ ((j & 1) ? odd : 0u), a[kb][j]);
  float t[KB][4];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) t[kb][0] = t[kb][1] = t[kb][2] = t[kb][3] = 0.f;
#pragma unroll
  for (int j = 0; j < NC - CLO; ++j) {
    constexpr int c0 = CLO;
    const int c = c0 + j;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      if (c < blocks[kb].dirty) {  // some pair of the chunk is out of reach of some key
        const int far = blocks[kb].far, wl = w[8 * c + kcol], wh = w[8 * c + 4 + kcol];
        if (far - krow > wl) a[kb][j][0] = 0u;
        if (far - krow - 8 > wl) a[kb][j][1] = 0u;
        if (far - krow > wh) a[kb][j][2] = 0u;
        if (far - krow - 8 > wh) a[kb][j][3] = 0u;
      }
      mma_bf16_16816((j & 1) ? t[kb] : s[kb], a[kb][j], qf[c][0], qf[c][1]);
    }
  }
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[kb][e] += t[kb][e];
}

template <int NC, int CLO, int KB>
__device__ __forceinline__ void qk_from(int clo, float (*s)[4], const Block* blocks, uint32_t cbytes, uint32_t odd,
                                        const uint32_t (*qf)[2], const int* w, int krow, int kcol) {
  if constexpr (CLO < NC - 1) {
    if (clo != CLO) return qk_from<NC, CLO + 1, KB>(clo, s, blocks, cbytes, odd, qf, w, krow, kcol);
  }
  qk_tile<NC, CLO, KB>(s, blocks, cbytes, odd, qf, w, krow, kcol);
}

}  // namespace

template <int D, int KB, int NSTG>
__global__ void __launch_bounds__(kPdThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ PagedDecodeParams p) {
  using C = PdCfg<D, KB, NSTG>;
  constexpr int NC = C::NC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sStage = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = sStage + NSTG * C::STAGE;
  float* sO = reinterpret_cast<float*>(sQ + NSTG * C::Q);
  PdShared<D, KB, NSTG>* sh = reinterpret_cast<PdShared<D, KB, NSTG>*>(reinterpret_cast<uint8_t*>(sO) + C::MERGE);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x;
  const int G = p.hq / p.hkv;
  const int box_log2 = min(p.page_log2, C::TILE_LOG2), box = 1 << box_log2;  // keys of a TMA box

  if (tid == 0) {
    for (int s = 0; s < NSTG; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], kPdConsumers);
    }
    mbar_init(&sh->left, kPdConsumers);
    mbar_init(&sh->joined, kPdJoiners);
    sh->abort = 0;
    sh->passed = 0;
    sh->start_b = -1;
    fence_mbar_init();
  }
  if (tid == kPdConsumers * 32) prefetch_tmap(&tm_k), prefetch_tmap(&tm_v);
  for (int i = tid; i < kMaxPairs; i += kPdThreads) sh->w[i] = p.win.w[i];
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();

  // ---- where this CTA's piece of the tile list begins: the sequences' weights, summed
  // up to each.  Small batches are summed by every producer warp for itself, which
  // needs no barrier (two barriers and the block's sums took 0.9 us of a call's 9)
  const bool alone = p.batch <= 32 * kPerLane;
  long long total = 0, base = 0;  // weight of all, and before the piece's first sequence
  int b = -1, len = 0;            // the piece's first sequence (-1: no piece)
  auto weight_of = [&](int n) { return static_cast<long long>(TileWeight<D, KB, NSTG>(p, sh->w, n)(tiles_of<C::TILE>(p, n))) * p.hkv; };
  auto scan = [&](long long x, int lanes) {  // inclusive, over the warp's first lanes
    for (int off = 1; off < lanes; off <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += o;
    }
    return x;
  };
  if (alone) {
    if (warp >= kPdConsumers && warp < kPdConsumers + kPdProducers) {
      int n[kPerLane];
      long long x[kPerLane], mine = 0;
      const int per = (p.batch + 31) >> 5;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) n[j] = j < per && lane * per + j < p.batch ? clamped_len(p, lane * per + j) : -1;
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) {
        x[j] = 0;
        if (j < per) mine += x[j] = n[j] >= 0 ? weight_of(n[j]) : 0;  // a branch for the warp
      }
      const long long incl = scan(mine, min(p.batch, 32));
      total = __shfl_sync(0xffffffffu, incl, min(p.batch, 32) - 1);
      const Pieces pieces(total);
      const long long from = pieces.begin(cta);
      long long at = incl - mine;
      const unsigned holds = __ballot_sync(0xffffffffu, from < pieces.begin(cta + 1) && from >= at && from < incl);
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) {
        if (b < 0 && n[j] >= 0 && from < at + x[j]) b = lane * per + j, len = n[j], base = at;
        at += x[j];
      }
      const int src = holds ? __ffs(holds) - 1 : 0;
      b = __shfl_sync(0xffffffffu, holds ? b : -1, src);
      len = __shfl_sync(0xffffffffu, len, src);
      base = __shfl_sync(0xffffffffu, base, src);
    }
  } else {
    const int per = (p.batch + kPdThreads - 1) / kPdThreads;  // sequences a thread sums
    const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
    long long mine = 0;
    for (int i = b0; i < b1; ++i) mine += weight_of(clamped_len(p, i));
    const long long incl = scan(mine, 32);
    if (lane == 31) sh->scan[warp] = incl;
    __syncthreads();
    long long at = incl - mine;
#pragma unroll
    for (int i = 0; i < kPdThreads / 32; ++i) {
      if (i < warp) at += sh->scan[i];
      total += sh->scan[i];
    }
    const Pieces pieces(total);
    const long long from = pieces.begin(cta);
    if (from < pieces.begin(cta + 1) && from >= at && from < at + mine) {
      for (int i = b0; i < b1; ++i) {
        const int n = clamped_len(p, i);
        const long long x = weight_of(n);
        if (from < at + x) {
          sh->start_b = i;
          sh->start_len = n;
          sh->start_base = at;
          break;
        }
        at += x;
      }
    }
    __syncthreads();
    b = sh->start_b;
    len = sh->start_len;
    base = sh->start_base;
  }

  if (warp >= kPdConsumers && warp < kPdConsumers + kPdProducers) {
    // ================================================================ producer
    RingPos<NSTG> ring;
    const int pw = warp - kPdConsumers;
    int it = 0;  // stages passed
    bool ok = true, has_partial0 = false, has_meta = false;
    const int ps = 1 << p.page_log2, sub_log2 = p.page_log2 - box_log2, boxes = C::TILE >> box_log2;
    const uint32_t box_bytes = static_cast<uint32_t>(D * 2) << box_log2;
    const Pieces pieces(total);
    const long long from = pieces.begin(cta), to = pieces.begin(cta + 1);
    int hk = 0;
    bool more = b >= 0;
    while (more && ok) {
      const int tiles = tiles_of<C::TILE>(p, len);
      const TileWeight<D, KB, NSTG> weight(p, sh->w, len);
      const int unit = weight(tiles);
      while (from >= base + unit) base += unit, ++hk;  // heads before the piece, at its beginning only
      const int t0 = from > base ? tile_at<D, KB, NSTG>(weight, tiles, static_cast<int>(from - base)) : 0;
      const int pages = (len + ps - 1) >> p.page_log2;
      const int* list = p.selected ? p.selected + (static_cast<long long>(b) * p.hkv + hk) * p.n_sel : nullptr;
      const int count = list ? min(p.n_sel, pages) : pages;
      const int* table = p.page_table + static_cast<long long>(b) * p.max_pages;
      // 32 boxes at a time, a lane each (under way before t1 is looked for): of the group in use the page in the
      // sequence (-1: none) and in the pool, and, on their way, the next group's
      // entries of the table and the list entries of the one after it
      auto listed = [&](int i) {  // page of box i in the sequence
        const int k = i >> sub_log2;
        return k < count ? (list ? list[k] : k) : -1;
      };
      auto in_pool = [&](int& logical) {  // its page in the pool, not yet looked at
        if (logical >= pages) {
          atomicCAS(p.err, 0u, kErrBadSelect);
          logical = -1;
        }
        return logical >= 0 ? table[logical] : 0;
      };
      int logical_next = listed(t0 * boxes + lane);
      int page_next = in_pool(logical_next);
      int logical_far = listed(t0 * boxes + 32 + lane);
      const int t1 = to >= base + unit ? tiles : tile_at<D, KB, NSTG>(weight, tiles, static_cast<int>(to - base));
      if (t0 < t1) {
        const int slot = t0 > 0 ? 0 : t1 < tiles ? 1 : -1;
        if (slot == 0) has_partial0 = true;
        for (int tg = t0; tg < t1 && ok; tg += 32 >> (C::TILE_LOG2 - box_log2)) {
          // this lane's box of the group
          const int i = tg * boxes + lane;
          int logical = logical_next, page = page_next;
          logical_next = logical_far;
          page_next = in_pool(logical_next);
          logical_far = listed(i + 64);
          if (logical >= 0 && (page < 0 || page >= p.num_pages)) {
            atomicCAS(p.err, 0u, kErrBadPage);
            logical = -1;
          }
          const int slot0 = (i & ((1 << sub_log2) - 1)) << box_log2;  // its first slot
          const int key0 = (max(logical, 0) << p.page_log2) + slot0;
          const int keys = logical >= 0 ? max(0, min(box, len - key0)) : 0;
          const int row = page * p.hkv + hk;
          int near = keys > 0 ? key0 + keys - 1 : -1;  // last key of the box, then of its tile
          int live = keys > 0;                         // boxes of its tile to be loaded
          for (int off = 1; off < boxes; off <<= 1) {
            near = max(near, __shfl_xor_sync(0xffffffffu, near, off));
            live += __shfl_xor_sync(0xffffffffu, live, off);
          }
          int clo = 0;  // windows grow with the chunk: the chunks out of reach are the first ones
          if (near >= 0) {
#pragma unroll
            for (int c = 0; c < NC - 1; ++c) clo += sh->w[8 * c + 7] < len - 1 - near;
          }
          const int tile = i >> (C::TILE_LOG2 - box_log2);  // the tile of this lane's box
          const bool lead = (lane & (boxes - 1)) == 0;
          const int tg1 = min(t1, tg + (32 >> (C::TILE_LOG2 - box_log2)));
          for (int t = tg; t < tg1; ++t, ++it, ring.next()) {
            if (it % kPdProducers != pw) continue;
            if (it >= NSTG && !warp_wait(&sh->empty[ring.st], ring.parity ^ 1, &sh->abort, p.err, 0x601)) {
              ok = false;
              break;
            }
            StageInfo<D, KB, NSTG>* info = &sh->info[ring.st];
            if (tile == t) {
              info->box[lane & (boxes - 1)] = make_int2(key0, keys);
              if (lead) {
                info->tile = make_int4(len, clo | (t == t0 ? kFirst : 0) | (t + 1 == t1 ? kLast : 0) | (slot + 1) << 16, b, hk);
              }
            }
            __syncwarp();
            uint8_t* stg = sStage + ring.st * C::STAGE;
            uint64_t* full = &sh->full[ring.st];
            if (tile == t) {
              if (lead) {
                const uint32_t q_bytes = t == t0 ? G * D * 2 : 0;
                mbar_arrive_expect_tx(full, live * 2 * box_bytes + q_bytes);
                if (q_bytes)
                  bulk_load(sQ + ring.st * C::Q,
                            static_cast<const __nv_bfloat16*>(p.q) + b * p.q_stride + static_cast<long long>(hk) * G * D,
                            q_bytes, full);
              }
              if (keys > 0) {
                uint8_t* dst = stg + (lane & (boxes - 1)) * box_bytes;
                tma_load_4d(dst, &tm_k, full, 0, slot0 >> 2, clo, row);
                tma_load_4d(dst + C::HALF, &tm_v, full, 0, slot0, 0, row);
              }
            }
          }
        }
        if (slot == 1) {
          has_meta = true;
          const long long x = base + weight(tiles - 1);  // where its last tile begins
          // the CTA whose piece holds x: the largest j with begin(j) <= x
          int lo = cta, hi = kPagedCtas - 1;
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pieces.begin(mid) <= x)
              lo = mid;
            else
              hi = mid - 1;
          }
          if (pw == 0 && lane == 0) p.meta[cta] = make_int4(b, hk, lo, 0);
        }
      }
      base += unit;
      if (++hk == p.hkv) {
        hk = 0;
        if (++b < p.batch && base < to) len = clamped_len(p, b);
      }
      more = b < p.batch && base < to;
    }
    if (ok && it % kPdProducers == pw) {  // the end mark
      if (it >= NSTG) ok = warp_wait(&sh->empty[ring.st], ring.parity ^ 1, &sh->abort, p.err, 0x602);
      if (ok && lane == 0) {
        sh->info[ring.st].tile.y = kEnd;
        mbar_arrive(&sh->full[ring.st]);
      }
    }
    if (pw == 0 && lane == 0 && !has_meta) p.meta[cta] = make_int4(-1, 0, 0, 0);
    if (pw == 0 && !has_partial0 && lane < G)  // no piece of an earlier CTA's sequence here
      p.sums[cta * 16 + lane] = make_float2(-INFINITY, 0.f);
    if (!ok && lane == 0) {  // wait (bounded) for this warp's copies in flight
      for (int j = it > NSTG ? it - NSTG : 0; j < it; ++j) {
        if (j % kPdProducers != pw) continue;
        const long long c0 = clock64();
        while (!mbar_try_wait(&sh->full[j % NSTG], (j / NSTG) & 1) && clock64() - c0 < kWaitLimitCycles) {
        }
      }
    }
    return;
  }

  if (warp >= kPdConsumers) {
    // ================================================================ joiners
    for (int k = 0;; ++k) {
      // a piece may be as long as the kernel: the limit starts anew with each stage passed
      bool ok = mbar_try_wait(&sh->left, k & 1);
      int seen = -1;
      for (long long t0 = 0; !ok && !*static_cast<volatile int*>(&sh->abort); ok = mbar_try_wait(&sh->left, k & 1)) {
        const int now = *static_cast<volatile int*>(&sh->passed);
        if (now != seen) {
          seen = now;
          t0 = clock64();
        } else if (clock64() - t0 > kWaitLimitCycles) {
          atomicCAS(p.err, 0u, 0x604u);
          sh->abort = 1;
        }
      }
      if (!__all_sync(0xffffffffu, ok)) return;
      const int b = sh->left_b, hk = sh->left_hk, slot = sh->left_slot;
      if (b < 0) return;
      for (int i = tid - (kPdConsumers + kPdProducers) * 32; i < G * (D / 4); i += kPdJoiners * 32) {
        const int g = i / (D / 4), e = i % (D / 4) * 4;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kPdConsumers; ++w) top = fmaxf(top, sh->mw[w][g]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kPdConsumers; ++w) {
          if (sh->mw[w][g] == -INFINITY) continue;  // no key of the piece
          const float4 x = *reinterpret_cast<const float4*>(&sO[(w * 8 + g) * C::OROW + e]);
          const float f = ex2_approx(sh->mw[w][g] - top);
          acc.x += x.x * f, acc.y += x.y * f, acc.z += x.z * f, acc.w += x.w * f;
          sum += sh->lw[w][g] * f;
        }
        if (slot < 0) {
          const long long row = static_cast<long long>(b) * p.hq + hk * G + g;
          const float r = top == -INFINITY ? 0.f : 1.f / sum;
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * D + e) =
              make_uint2(pack_bf16x2(acc.x * r, acc.y * r), pack_bf16x2(acc.z * r, acc.w * r));
          if (p.lse && e == 0) p.lse[row] = top == -INFINITY ? -INFINITY : (top + log2f(sum)) * kLn2;
        } else {
          const int at = (cta * 2 + slot) * 8 + g;
          *reinterpret_cast<float4*>(p.partials + static_cast<long long>(at) * D + e) = acc;
          if (e == 0) p.sums[at] = make_float2(top, sum);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->joined);
    }
  }

  // ================================================================ consumers
  const float scale = kLog2e * rsqrtf(static_cast<float>(D));
  const int kcol = lane & 3, krow = lane >> 2;  // this lane's pair in a half chunk / head pair, and key row / dim row
  const int group = warp >> 2;
  // this warp's blocks of a tile: box, slot in it, and this lane's rows
  const uint32_t cbytes = 32u << box_log2, vhalf = 128u << box_log2;
  const uint32_t k_odd = box == 16 ? 64u : 0u;
  int bx[KB], off[KB];
  uint32_t k_at[KB], v_at[KB];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    const int key = 16 * ((warp & 3) * KB + kb);
    bx[kb] = key >> box_log2, off[kb] = key & (box - 1);
    const uint32_t at = bx[kb] * (static_cast<uint32_t>(D * 2) << box_log2);
    // a chunk's rows of four keys, 128 bytes each, lie 16-byte units swizzled by the
    // row's number in its 1024 bytes; chunks of 16 keys are half as long, so every
    // other one starts at row 4
    const int krow_ld = off[kb] + (lane & 15), vrow_ld = off[kb] + (lane & 7) + ((lane >> 4) << 3);
    k_at[kb] = at + (krow_ld >> 2) * 128 + ((((krow_ld & 3) * 2 + (lane >> 4)) ^ ((krow_ld >> 2) & 7)) << 4);
    v_at[kb] = C::HALF + at + vrow_ld * 128;
  }
  const int vrow_unit = lane & 7;  // of every block's row, modulo 8
  uint32_t qf[NC][2];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // of heads 2*kcol, 2*kcol + 1
  float o[D / 16][4];  // O^T: dims 16u + krow (+8), heads 2*kcol (+1)
  const int w_first = lane < NC ? sh->w[8 * lane] : 0x7fffffff;  // smallest window of chunk `lane`
  int pieces = 0, passed = 0;
  RingPos<NSTG> ring;
  // the joiners are done with the last piece's states (a bounded wait)
  auto joined = [&] { return pieces == 0 || warp_wait(&sh->joined, (pieces - 1) & 1, &sh->abort, p.err, 0x605); };
  auto leave = [&](int b, int hk, int slot) {
    if (tid == 0) sh->left_b = b, sh->left_hk = hk, sh->left_slot = slot;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->left);
    ++pieces;
  };
  for (int turn = 0;; turn = turn + 1 == kPdGroups ? 0 : turn + 1) {
    const int st = ring.st;
    if (!warp_wait(&sh->full[st], ring.parity, &sh->abort, p.err, 0x603)) return;
    ring.next();
    const int4 tile = sh->info[st].tile;
    int2 my[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) my[kb] = sh->info[st].box[bx[kb]];
    const int flags = tile.y;
    if (tid == 0) *static_cast<volatile int*>(&sh->passed) = ++passed;
    if (flags & kEnd) {
      if (joined()) leave(-1, 0, 0);
      return;
    }
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
    if (turn == group) {
      const uint32_t stg = smem_u32(sStage + st * C::STAGE);
      int live[KB];  // live keys from the block's first on
      Block blocks[KB];
      float s[KB][4];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        live[kb] = my[kb].y - off[kb];
        blocks[kb].k_at = stg + k_at[kb];
        blocks[kb].far = tile.x - 1 - (my[kb].x + off[kb]);
        blocks[kb].dirty = __popc(__ballot_sync(0xffffffffu, blocks[kb].far > w_first));
        s[kb][0] = s[kb][1] = s[kb][2] = s[kb][3] = 0.f;
      }

      // ---- S^T, pairs beyond their window zeroed
      qk_from<NC, 0, KB>(flags & 0xff, s, blocks, cbytes, k_odd, qf, sh->w, krow, kcol);
      // the values go through registers in two halves, of the row or of the keys; the
      // first is fetched while the softmax runs
      constexpr int UPH = KB * D / 32;  // groups of 16 dims of a half
      uint32_t va[UPH][4];
      auto load_v = [&](int half) {
        const int kb = KB == 1 ? 0 : half, u0 = KB == 1 ? half * UPH : 0;
#pragma unroll
        for (int u = 0; u < UPH; ++u) {
          const int dim = 16 * (u0 + u) + (lane & 8);
          ldsm_x4_t(stg + v_at[kb] + ((u0 + u) >> 2) * vhalf + ((((dim & 63) >> 3) ^ vrow_unit) << 4), va[u]);
        }
      };
      load_v(0);
      // ---- online softmax of heads 2*kcol, 2*kcol + 1.  The maximum that weights are
      // taken against is raised only where a logit is more than kSlack above it: they
      // stay below 2^kSlack, and most tiles need no reduction over the warp
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[kb][e] = krow + (e & 2) * 4 < live[kb] ? s[kb][e] * scale : -INFINITY;
          top[e & 1] = fmaxf(top[e & 1], s[kb][e]);
        }
      if (__any_sync(0xffffffffu, top[0] > m[0] + kSlack || top[1] > m[1] + kSlack)) {
        float corr[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = top[e];
#pragma unroll
          for (int sh_ = 4; sh_ < 32; sh_ <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh_));
          mx = fmaxf(m[e], mx);
          corr[e] = m[e] == -INFINITY ? 0.f : ex2_approx(m[e] - mx);
          m[e] = mx;
          l[e] *= corr[e];
        }
#pragma unroll
        for (int u = 0; u < D / 16; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[u][e] *= corr[e & 1];
      }
      uint32_t pb[KB][2], pl[KB][2];  // P^T rounded to bf16, and the rest of it
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pr[e] = ex2_approx(s[kb][e] - (m[e & 1] == -INFINITY ? 0.f : m[e & 1]));  // no live key yet
          l[e & 1] += pr[e];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t hi = pack_bf16x2(pr[2 * h], pr[2 * h + 1]);
          pb[kb][h] = movmatrix_t(hi);
          pl[kb][h] = movmatrix_t(pack_bf16x2(pr[2 * h] - bf16lo_to_f32(hi), pr[2 * h + 1] - bf16hi_to_f32(hi)));
        }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int kb = KB == 1 ? 0 : half, u0 = KB == 1 ? half * UPH : 0;
        if (half) load_v(half);
        if (live[kb] < 16) {  // rows behind the last key may hold anything: their values count as zero
          const int n = live[kb] - 2 * kcol;
          const uint32_t keep0 = n >= 2 ? 0xFFFFFFFFu : n == 1 ? 0xFFFFu : 0u;
          const uint32_t keep1 = n >= 10 ? 0xFFFFFFFFu : n == 9 ? 0xFFFFu : 0u;
#pragma unroll
          for (int u = 0; u < UPH; ++u) {
            va[u][0] &= keep0;
            va[u][1] &= keep0;
            va[u][2] &= keep1;
            va[u][3] &= keep1;
          }
        }
#pragma unroll
        for (int u = 0; u < UPH; ++u) mma_bf16_16816(o[u0 + u], va[u], pb[kb][0], pb[kb][1]);
#pragma unroll
        for (int u = 0; u < UPH; ++u) mma_bf16_16816(o[u0 + u], va[u], pl[kb][0], pl[kb][1]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->empty[st]);
    if (!(flags & kLast)) continue;

    // ---- the warp's state to the joiners
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int sh_ = 4; sh_ < 32; sh_ <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], sh_);
    if (!joined()) return;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (krow == 0) {
        sh->mw[warp][2 * kcol + e] = m[e];
        sh->lw[warp][2 * kcol + e] = l[e];
      }
#pragma unroll
      for (int u = 0; u < D / 16; ++u)
#pragma unroll
        for (int k = 0; k < 4; k += 2) sO[(warp * 8 + 2 * kcol + e) * C::OROW + 16 * u + krow + k * 4] = o[u][k + e];
    }
    leave(tile.z, tile.w, (flags >> 16) - 1);
  }
}

// Joins the pieces of the sequence and head that CTA blockIdx.x began and did not
// end: its slot 1 and slot 0 of the CTAs up to meta.z.  blockIdx.y = query head.
// Two loads deep: maxima and sums of all pieces that there could be are fetched with
// meta, and the first kAhead rounds of partial sums before the maxima are joined.
constexpr int kCombineThreads = 256;

template <int D>
__global__ void __launch_bounds__(kCombineThreads) paged_combine_kernel(const __grid_constant__ PagedDecodeParams p) {
  constexpr int kRow = D / 4, kSide = kCombineThreads / kRow;  // threads of a piece, pieces side by side
  constexpr int kAhead = 5, kWarps = kCombineThreads / 32;
  static_assert(kPagedCtas <= kCombineThreads, "a piece a thread");
  __shared__ float s_f[kPagedCtas], s_max[kWarps], s_sum[kWarps];
  __shared__ float4 s_acc[kCombineThreads];
  const int tid = threadIdx.x, g = blockIdx.y, first = blockIdx.x, G = p.hq / p.hkv;
  pdl_launch_dependents();
  pdl_wait();
  const int4 meta = p.meta[first];
  auto row_of = [&](int i) { return ((first + i) * 2 + (i == 0)) * 8 + g; };
  float2 own = first + tid < kPagedCtas ? p.sums[row_of(tid)] : make_float2(-INFINITY, 0.f);
  if (meta.x < 0) return;
  const int n = meta.z - first + 1;
  if (tid >= n) own = make_float2(-INFINITY, 0.f);
  const int side = tid / kRow, e = tid % kRow * 4;
  auto part = [&](int i) { return *reinterpret_cast<const float4*>(p.partials + static_cast<long long>(row_of(i)) * D + e); };
  float4 x[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = side + k * kSide;
    x[k] = i < n ? part(i) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float top = own.x;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if ((tid & 31) == 0) s_max[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_max[w]);
  const float f = own.x == -INFINITY ? 0.f : ex2_approx(own.x - top);
  if (tid < n) s_f[tid] = f;
  float sum = own.y * f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if ((tid & 31) == 0) s_sum[tid >> 5] = sum;
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int i, const float4& v) {
    const float w = s_f[i];
    if (w > 0.f) acc.x += v.x * w, acc.y += v.y * w, acc.z += v.z * w, acc.w += v.w * w;  // an empty piece holds no sums
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = side + k * kSide;
    if (i < n) add(i, x[k]);
  }
#pragma unroll 4
  for (int i = side + kAhead * kSide; i < n; i += kSide) add(i, part(i));
  s_acc[tid] = acc;
  __syncthreads();
  if (tid >= kRow) return;
#pragma unroll
  for (int k = 1; k < kSide; ++k) {
    const float4 v = s_acc[tid + k * kRow];
    acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
  }
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += s_sum[w];
  const long long row = static_cast<long long>(meta.x) * p.hq + meta.y * G + g;
  const float r = top == -INFINITY ? 0.f : 1.f / sum;
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * D + e) =
      make_uint2(pack_bf16x2(acc.x * r, acc.y * r), pack_bf16x2(acc.z * r, acc.w * r));
  if (p.lse && e == 0) p.lse[row] = top == -INFINITY ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <int D, int KB, int NSTG>
static cudaError_t launch_pd(const PagedDecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  auto kern = paged_decode_kernel<D, KB, NSTG>;
  constexpr int bytes = pd_smem_bytes<D, KB, NSTG>();
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
  e = launch_pdl(kern, kPagedCtas, kPdThreads, bytes, s, tk, tv, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_combine_kernel<D>, dim3(kPagedCtas, p.hq / p.hkv), kCombineThreads, 0, s, p);
}

// Stages: what fits.  Over listed pages heads of 128 take one less: the memory left
// makes the selection before it faster (48 of up to 1024 pages of 32 sequences: 44.7 us
// together, 47.2 with five), and its pieces are short; a long cache wants five (864 us
// against 902 for four sequences of 1048576 keys).
cudaError_t launch_paged_decode(const PagedDecodeParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  if (p.d == 128) return p.selected ? launch_pd<128, 1, 4>(p, tk, tv, s) : launch_pd<128, 1, 5>(p, tk, tv, s);
  return p.tile_keys == 128 ? launch_pd<64, 2, 6>(p, tk, tv, s) : launch_pd<64, 1, 8>(p, tk, tv, s);
}

}  // namespace atf
