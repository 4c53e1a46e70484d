// qk_norm_rope.cu -- RMS norm of every query and key head and the position
// rotation in one pass, to contiguous rows (the operands of the prefill) or, for
// new tokens of a batch, to a paged key-value cache.
//
//   y = x * rsqrt(mean(x^2) + eps) * w           (per head; skipped without w)
//   (y_a, y_b) of pair i turned by pos[axis(i)] * theta^(-2i/d)
//
// all in fp32 and rounded once.  The angle is reduced to a fraction of a turn by a
// 64-bit integer product that wraps (at position 2^20 an fp32 angle is off by more
// than a bf16 step; the product's table entry by 2^-34 turns at 2^31, and it takes a third
// of the time of fp64's multiply, round and convert).  Its upper 32 bits become an fp32
// number, half a step of which is 2^-26 of a turn: all but 2^-31 of the angle's error, at any position.  The sine
// and cosine of that fraction are fp32's for fp32 rows; for bf16 rows the fast ones,
// off by at most 2^-21 on [-pi, pi], 2^-13 of a bf16 half step.
//
// Bound by the rows' bytes, read once and written once.  One thread owns a token's
// 8-pair chunk c: elements 16c..16c+15 of a head (interleaved pairs) or 8c..8c+7 and
// d/2+8c..d/2+8c+7 (rotate-half), which are the 16 outputs 16c..16c+15 either way and
// one 32-byte row of the key pages, written by one store.  It evaluates the chunk's
// eight angles once for up to kRows heads, whose loads are all under way before the
// first is used (8192 tokens of 28 + 4 heads of 128: 23.9 us, 32 with one load at a
// time, 20.5 at the copy rate); the d/16 lanes of a head add their squares by shuffles.  Few rows
// take one head a thread: there the latency of a thread's chain is what counts.
#include <cuda_bf16.h>

#include "atf_internal.cuh"
#include "ptx.cuh"

namespace atf {

namespace {

constexpr int kNrThreads = 128;
constexpr int kRows = 4;  // heads of a thread where there are many

// 32 bytes to dst: one store where `wide` (dst 32-byte aligned), else two.
__device__ __forceinline__ void store32(void* dst, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <typename T, bool kHalf>
struct Chunk;  // 16 elements as loaded: the first components a[8] and second b[8] of eight pairs

template <bool kHalf>
struct Chunk<__nv_bfloat16, kHalf> {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int c, int d) {
    lo = *reinterpret_cast<const uint4*>(row + (kHalf ? 8 * c : 16 * c));
    hi = *reinterpret_cast<const uint4*>(row + (kHalf ? d / 2 + 8 * c : 16 * c + 8));
  }
  __device__ __forceinline__ void pairs(float* a, float* b) const {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (kHalf) {
        a[k] = (k & 1) ? bf16hi_to_f32(w[k >> 1]) : bf16lo_to_f32(w[k >> 1]);
        b[k] = (k & 1) ? bf16hi_to_f32(w[4 + (k >> 1)]) : bf16lo_to_f32(w[4 + (k >> 1)]);
      } else {
        a[k] = bf16lo_to_f32(w[k]);
        b[k] = bf16hi_to_f32(w[k]);
      }
    }
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* dst, const float* a, const float* b, bool wide) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(a[k], b[k]);
    store32(dst, w, wide);
  }
};

template <bool kHalf>
struct Chunk<float, kHalf> {
  float4 v[4];
  __device__ __forceinline__ void load(const float* row, int c, int d) {
    const float4* lo = reinterpret_cast<const float4*>(row + (kHalf ? 8 * c : 16 * c));
    const float4* hi = reinterpret_cast<const float4*>(row + (kHalf ? d / 2 + 8 * c : 16 * c + 8));
    v[0] = lo[0], v[1] = lo[1], v[2] = hi[0], v[3] = hi[1];
  }
  __device__ __forceinline__ void pairs(float* a, float* b) const {
    const float w[16] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w,
                         v[2].x, v[2].y, v[2].z, v[2].w, v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      a[k] = kHalf ? w[k] : w[2 * k];
      b[k] = kHalf ? w[8 + k] : w[2 * k + 1];
    }
  }
  __device__ __forceinline__ static void store(float* dst, const float* a, const float* b, bool wide) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[2 * k] = __float_as_uint(a[4 * h + k]), w[2 * k + 1] = __float_as_uint(b[4 * h + k]);
      store32(dst + 8 * h, w, wide);
    }
  }
};

struct RotaryShared {
  unsigned long long turns[kMaxPairs];  // pair 8 c + k at k * (d/16) + c: a warp's chunks side by side
  signed char axis[kMaxPairs];
  signed char chunk_axis[kMaxPairs / 8];  // of all the chunk's pairs, or -1: several
};

template <int D>
__device__ __forceinline__ void load_rotary(RotaryShared* sh, const RotaryTable& rot) {
  constexpr int NC = D / 16;
  for (int i = threadIdx.x; i < D / 2; i += blockDim.x) {
    sh->turns[(i & 7) * NC + (i >> 3)] = rot.turns[i];
    sh->axis[(i & 7) * NC + (i >> 3)] = static_cast<signed char>(rot.axis[i]);
  }
  if (threadIdx.x < NC) {
    int a = rot.axis[8 * threadIdx.x];
    for (int k = 1; k < 8; ++k) a = rot.axis[8 * threadIdx.x + k] == a ? a : -1;
    sh->chunk_axis[threadIdx.x] = static_cast<signed char>(a);
  }
  __syncthreads();
}

// Positions of a token on up to kMaxAxes axes.
struct Position {
  int at[kMaxAxes];
  __device__ __forceinline__ void load(const long long* pos, int n_axes, long long tokens, long long t) {
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) at[a] = a < n_axes ? static_cast<int>(pos[a * tokens + t]) : 0;
  }
};

// Norm weights and rotation of a chunk's eight pairs as one map, two pairs a word:
// a' = a ac + b bs, b' = a as + b bc.
struct Turn {
  uint64_t ac[4], bs[4], as[4], bc[4];
};

// Cosine and sine of pair 8 c + k at position p of its axis.
template <int D, bool kFast>
__device__ __forceinline__ void pair_angle(const RotaryShared* sh, int c, int k, int p, float* sn, float* cs) {
  const unsigned long long t = static_cast<unsigned long long>(static_cast<long long>(p)) * sh->turns[k * (D / 16) + c];
  const float part = static_cast<float>(static_cast<int>(t >> 32));  // of 2^32 of a turn, in [-1/2, 1/2)
  if (kFast) {
    const float x = 1.4629180792671596e-9f * part;  // 2 pi / 2^32
    *sn = __sinf(x);
    *cs = __cosf(x);
  } else {
    sincospif(4.656612873077393e-10f * part, sn, cs);  // 2 / 2^32
  }
}

template <int D, bool kFast>
__device__ __forceinline__ void chunk_turn(Turn& turn, const RotaryShared* sh, int c, const Position& pos, int n_axes, bool norm,
                                           const float* wa, const float* wb) {
  constexpr int NC = D / 16;
  const int chunk = n_axes > 1 ? sh->chunk_axis[c] : 0;
  auto on_axis = [&](int a) { return a == 1 ? pos.at[1] : a == 2 ? pos.at[2] : a == 3 ? pos.at[3] : pos.at[0]; };
  const int common = on_axis(chunk);
  float m[4][8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    int p = common;
    if (chunk < 0) p = on_axis(sh->axis[k * NC + c]);
    float sn, cs;
    pair_angle<D, kFast>(sh, c, k, p, &sn, &cs);
    m[0][k] = norm ? wa[k] * cs : cs;
    m[1][k] = norm ? -wb[k] * sn : -sn;
    m[2][k] = norm ? wa[k] * sn : sn;
    m[3][k] = norm ? wb[k] * cs : cs;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    turn.ac[k] = pack2(m[0][2 * k], m[0][2 * k + 1]);
    turn.bs[k] = pack2(m[1][2 * k], m[1][2 * k + 1]);
    turn.as[k] = pack2(m[2][2 * k], m[2][2 * k + 1]);
    turn.bc[k] = pack2(m[3][2 * k], m[3][2 * k + 1]);
  }
}

// One over the root mean square of a head whose chunks the d/16 neighbouring lanes
// hold; every lane of the warp calls it.
template <int D>
__device__ __forceinline__ float norm_scale(const uint64_t* a, const uint64_t* b, float eps) {
  uint64_t s2 = fmul2(a[0], a[0]);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k) s2 = ffma2(a[k], a[k], s2);
    s2 = ffma2(b[k], b[k], s2);
  }
  float x, y;
  unpack2(s2, x, y);
  x += y;
#pragma unroll
  for (int off = 1; off < D / 16; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return rsqrtf(x * (1.0f / D) + eps);
}

// The chunk of one head, turned and scaled: the first components to ya, the second to yb.
__device__ __forceinline__ void apply(const Turn& t, const uint64_t* a, const uint64_t* b, float scale, float* ya, float* yb) {
  const uint64_t r = pack2(scale, scale);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    unpack2(fmul2(r, ffma2(a[k], t.ac[k], fmul2(b[k], t.bs[k]))), ya[2 * k], ya[2 * k + 1]);
    unpack2(fmul2(r, ffma2(a[k], t.as[k], fmul2(b[k], t.bc[k]))), yb[2 * k], yb[2 * k + 1]);
  }
}

// One bf16 head's chunk normed, turned and rounded, two pairs at a time: for a thread
// with a single head, which needs no map kept.  Every lane of the warp calls it; the
// sum of squares is taken whether the lane's row has a norm or not.
template <int D, bool kHalf>
__device__ __forceinline__ void turn_one(uint32_t* y, const Chunk<__nv_bfloat16, kHalf>& in,
                                         const Chunk<__nv_bfloat16, kHalf>& weight, bool norm, float eps,
                                         const RotaryShared* sh, int c, const Position& pos, int n_axes) {
  constexpr int NC = D / 16;
  float a[8], b[8];
  in.pairs(a, b);
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) ss += a[k] * a[k] + b[k] * b[k];
#pragma unroll
  for (int off = 1; off < NC; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  const float scale = norm ? rsqrtf(ss * (1.0f / D) + eps) : 1.f;
  const int chunk = n_axes > 1 ? sh->chunk_axis[c] : 0;
  auto on_axis = [&](int a) { return a == 1 ? pos.at[1] : a == 2 ? pos.at[2] : a == 3 ? pos.at[3] : pos.at[0]; };
  const int common = on_axis(chunk);
  float wa[8], wb[8];
  if (norm) weight.pairs(wa, wb);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    int p = common;
    if (chunk < 0) p = on_axis(sh->axis[k * NC + c]);
    float sn, cs;
    pair_angle<D, true>(sh, c, k, p, &sn, &cs);
    const float u = norm ? a[k] * wa[k] * scale : a[k], v = norm ? b[k] * wb[k] * scale : b[k];
    y[k] = pack_bf16x2(u * cs - v * sn, u * sn + v * cs);
  }
}

__device__ __forceinline__ void pack_pairs(const float* x, uint64_t* y) {
#pragma unroll
  for (int k = 0; k < 4; ++k) y[k] = pack2(x[2 * k], x[2 * k + 1]);
}

// A token's chunk of up to R neighbouring heads and their weights.
template <typename T, int D, int R, bool kHalf>
struct Rows {
  Chunk<T, kHalf> in[R], weight;
  __device__ __forceinline__ void load(const T* x, int n, int c, const T* w) {
#pragma unroll
    for (int r = 0; r < R; ++r) in[r].load(x + (R == 1 ? 0 : min(r, n - 1)) * D, c, D);
    if (w) weight.load(w, c, D);
  }
  template <bool kFast>
  __device__ __forceinline__ void turn(Turn& t, const RotaryShared* sh, int c, const Position& pos, int n_axes, bool norm) const {
    float wa[8], wb[8];
    if (norm) weight.pairs(wa, wb);
    chunk_turn<D, kFast>(t, sh, c, pos, n_axes, norm, wa, wb);
  }
  // Heads r < n to out + r * d, where `live`; every lane of the warp calls it.
  __device__ __forceinline__ void finish(T* out, int n, const Turn& t, bool norm, float eps, bool live, bool wide) const {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float x[8], y[8];
      uint64_t a[4], b[4];
      in[r].pairs(x, y);
      pack_pairs(x, a);
      pack_pairs(y, b);
      apply(t, a, b, norm ? norm_scale<D>(a, b, eps) : 1.f, x, y);
      if (live && r < n) Chunk<T, kHalf>::store(out + r * D, x, y, wide);
    }
  }
};

}  // namespace

// Dense form.  Thread = (token, chunk), blockIdx.y = R query heads or, behind them, R
// key heads.  Registers for six CTAs an SM (four in fp32), five in the append below: its
// 32768 tokens of five prompts take 144 us at the three that fit unbounded, 110 at five.
template <typename T, int D, int R, bool kHalf>
__global__ void __launch_bounds__(kNrThreads, sizeof(T) == 2 ? 6 : 4) qk_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int NC = D / 16;
  __shared__ RotaryShared sh;
  load_rotary<D>(&sh, p.rot);
  pdl_launch_dependents();
  pdl_wait();
  const long long idx = static_cast<long long>(blockIdx.x) * kNrThreads + threadIdx.x;
  const int c = static_cast<int>(idx % NC);
  const bool live = idx / NC < p.tokens;
  const long long t = live ? idx / NC : p.tokens - 1;
  const int q_groups = (p.hq + R - 1) / R;
  const bool key = static_cast<int>(blockIdx.y) >= q_groups;
  const int heads = key ? p.hkv : p.hq, h = (key ? blockIdx.y - q_groups : blockIdx.y) * R, n = min(R, heads - h);
  const T* w = static_cast<const T*>(key ? p.k_weight : p.q_weight);
  Rows<T, D, R, kHalf> rows;
  rows.load(static_cast<const T*>(key ? p.k : p.q) + t * (key ? p.k_stride : p.q_stride) + h * D, n, c, w);
  Position pos;
  pos.load(p.pos, p.rot.n_axes, p.tokens, t);
  Turn turn;
  rows.template turn<sizeof(T) == 2>(turn, &sh, c, pos, p.rot.n_axes, w != nullptr);
  rows.finish(static_cast<T*>(key ? p.k_out : p.q_out) + (t * heads + h) * D + 16 * c, n, turn, w != nullptr, p.eps, live, p.wide);
}

template <typename T, int D, bool kHalf>
static cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t s) {
  const long long chunks = static_cast<long long>(p.tokens) * (D / 16);
  const unsigned blocks = static_cast<unsigned>((chunks + kNrThreads - 1) / kNrThreads);
  // kRows heads a thread once that still leaves every SM 128 threads (1024 tokens of 28 + 4
  // heads of 128: 4.6 us, one head a thread 6.6; 64 tokens 2.5 and 2.0)
  const bool many = chunks * (p.hq + p.hkv) >= 148LL * 128 * kRows;
  if (!many) return launch_pdl(qk_norm_rope_kernel<T, D, 1, kHalf>, dim3(blocks, p.hq + p.hkv), kNrThreads, 0, s, p);
  const int groups = (p.hq + kRows - 1) / kRows + (p.hkv + kRows - 1) / kRows;
  return launch_pdl(qk_norm_rope_kernel<T, D, kRows, kHalf>, dim3(blocks, groups), kNrThreads, 0, s, p);
}

template <typename T, int D>
static cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t s) {
  return p.pairing ? launch_norm_rope<T, D, true>(p, s) : launch_norm_rope<T, D, false>(p, s);
}

cudaError_t launch_qk_norm_rope(const NormRopeParams& p, cudaStream_t s) {
  if (p.fp32) return p.d == 64 ? launch_norm_rope<float, 64>(p, s) : launch_norm_rope<float, 128>(p, s);
  return p.d == 64 ? launch_norm_rope<__nv_bfloat16, 64>(p, s) : launch_norm_rope<__nv_bfloat16, 128>(p, s);
}

// ------------------------------------------------------------------ paged append

namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Physical page of logical page lp of sequence b, or -1 (recorded) where the
// table holds none.
__device__ __forceinline__ int page_of(const PagedAppendParams& p, int b, long long lp) {
  if (lp >= p.max_pages) {
    atomicCAS(p.err, 0u, kErrBadLength);
    return -1;
  }
  const int page = p.page_table[static_cast<long long>(b) * p.max_pages + lp];
  if (page < 0 || page >= p.num_pages) {
    atomicCAS(p.err, 0u, kErrBadPage);
    return -1;
  }
  return page;
}

// A key's and a value's chunk to slot `at` of a page.
template <int D>
__device__ __forceinline__ void store_slot(const PagedAppendParams& p, int page, int kvh, int c, int at, const uint32_t* k,
                                           const uint32_t* v) {
  const long long ps = 1LL << p.page_log2, head = static_cast<long long>(page) * p.hkv + kvh;
  store32(static_cast<bf16*>(p.k_pages) + ((head * (D / 16) + c) * ps + at) * 16, k, p.wide);
  store32(static_cast<bf16*>(p.v_pages) + (head * ps + at) * D + 16 * c, v, p.wide);
}

// Bounds row of chunk c: 8 words of minima or maxima.
template <int D>
__device__ __forceinline__ uint4* bounds_row(const PagedAppendParams& p, int page, int kvh, int which, int c) {
  return reinterpret_cast<uint4*>(static_cast<bf16*>(p.bounds) + ((static_cast<long long>(page) * p.hkv + kvh) * 2 + which) * D +
                                  16 * c);
}

__device__ __forceinline__ void load32(uint32_t* w, const bf16* x) {
  const uint4 a = reinterpret_cast<const uint4*>(x)[0], b = reinterpret_cast<const uint4*>(x)[1];
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

}  // namespace

// One token per sequence: thread = (sequence, head, chunk), the key heads of a
// sequence first.
template <int D, bool kHalf>
__global__ void __launch_bounds__(kNrThreads) paged_append_step_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int NC = D / 16;
  __shared__ RotaryShared sh;
  load_rotary<D>(&sh, p.rot);
  pdl_launch_dependents();
  pdl_wait();
  const int hq = p.q ? p.hq : 0, heads = p.hkv + hq;
  const long long idx = static_cast<long long>(blockIdx.x) * kNrThreads + threadIdx.x;
  const int c = static_cast<int>(idx % NC);
  const long long last = static_cast<long long>(p.batch) * heads - 1, row = min(idx / NC, last);
  const int b = static_cast<int>(row / heads), r = static_cast<int>(row % heads);
  const bool key = r < p.hkv;
  const long long slot = p.start[b];
  const bool live = idx / NC <= last && slot >= 0;
  const bf16* w = static_cast<const bf16*>(key ? p.k_weight : p.q_weight);
  Chunk<bf16, kHalf> in, cw;
  in.load(key ? static_cast<const bf16*>(p.k) + b * p.k_stride + r * D
              : static_cast<const bf16*>(p.q) + b * p.q_stride + (r - p.hkv) * D, c, D);
  if (w) cw.load(w, c, D);
  uint32_t v[8];
  if (key) load32(v, static_cast<const bf16*>(p.v) + b * p.v_stride + r * D + 16 * c);
  Position pos;
  if (p.pos)
    pos.load(p.pos, p.rot.n_axes, p.tokens, b);
  else
    pos.at[0] = static_cast<int>(slot), pos.at[1] = pos.at[2] = pos.at[3] = 0;
  const int page = live && key ? page_of(p, b, slot >> p.page_log2) : -1;
  const int at = static_cast<int>(slot & ((1 << p.page_log2) - 1));
  uint32_t old[2][8];
  const bool bound = p.bounds && page >= 0;
  if (bound && at)  // the page holds earlier keys
#pragma unroll
    for (int which = 0; which < 2; ++which)
      load32(old[which], reinterpret_cast<const bf16*>(bounds_row<D>(p, page, r, which, c)));
  uint32_t y[8];
  turn_one<D, kHalf>(y, in, cw, w != nullptr, p.eps, &sh, c, pos, p.pos ? p.rot.n_axes : 1);
  if (!live) return;
  if (!key) return store32(static_cast<bf16*>(p.q_out) + (static_cast<long long>(b) * hq + r - p.hkv) * D + 16 * c, y, p.wide);
  if (page < 0) return;
  store_slot<D>(p, page, r, c, at, y, v);
  if (!bound) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    uint32_t m[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) m[k] = !at ? y[k] : which ? max_bf16x2(y[k], old[1][k]) : min_bf16x2(y[k], old[0][k]);
    uint4* dst = bounds_row<D>(p, page, r, which, c);
    dst[0] = make_uint4(m[0], m[1], m[2], m[3]);
    dst[1] = make_uint4(m[4], m[5], m[6], m[7]);
  }
}

// Ragged batch.  The first p.items * hkv CTAs own each the new tokens of one sequence
// that fall into one page, for one kv head, so that the page's bounds have one
// writer; the others kRows query heads each of kApThreads / (d/16) rows.
// The CTA's size goes by the number of (page, kv head) items: of many, small CTAs leave
// few threads without a token; of few, large ones take fewer passes over a page.  At
// 64 / 128 / 256 threads: 2236 tokens of 60 sequences, 4 kv heads of 128, pages of 16:
// 10.3 / 11.3 / 19 us; 1594 tokens of 16 sequences, 3 kv heads, pages of 128: 17.3 / 11.1 / 7.2.
template <int D, bool kHalf, int kApThreads>
__global__ void __launch_bounds__(kApThreads, kApThreads == 256 ? 2 : 640 / kApThreads) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int NC = D / 16, kTok = kApThreads / NC;  // tokens in flight
  constexpr int kWarps = kApThreads / 32;
  __shared__ RotaryShared sh;
  __shared__ int s_item[3];  // sequence, first row, tokens
  __shared__ long long s_slot, s_scan[kWarps];  // first slot
  __shared__ uint32_t s_red[2][kWarps][D / 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = tid % NC;
  const int axes = p.pos ? p.rot.n_axes : 1;
  load_rotary<D>(&sh, p.rot);
  pdl_launch_dependents();
  pdl_wait();

  const long long kv_blocks = p.items * p.hkv;
  if (blockIdx.x >= kv_blocks) {
    // ---- queries
    const int groups = (p.hq + kRows - 1) / kRows;
    const long long i = blockIdx.x - kv_blocks;
    const int h = static_cast<int>(i % groups) * kRows, n = min(kRows, p.hq - h);
    const long long row0 = i / groups * kTok, row = row0 + tid / NC;
    const long long t = min(row, static_cast<long long>(p.tokens) - 1);
    Rows<bf16, D, kRows, kHalf> rows;
    const bf16* w = static_cast<const bf16*>(p.q_weight);
    rows.load(static_cast<const bf16*>(p.q) + t * p.q_stride + h * D, n, c, w);
    // the row's sequence: as many as end at or before it, over all sequences, the
    // warp's rows side by side
    constexpr int kPer = 32 / NC;
    int ended[kPer];
#pragma unroll
    for (int g = 0; g < kPer; ++g) ended[g] = 0;
    const long long first = row0 + warp * kPer;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int end = b0 + lane < p.batch ? p.cu[b0 + lane + 1] : 0x7fffffff;
#pragma unroll
      for (int g = 0; g < kPer; ++g) ended[g] += __popc(__ballot_sync(0xffffffffu, end <= first + g));
    }
    int b = ended[0];
#pragma unroll
    for (int g = 1; g < kPer; ++g) b = lane / NC == g ? ended[g] : b;
    bool live = row < p.tokens && b < p.batch;
    long long slot = 0;
    if (live) {
      const int r0 = p.cu[b], s0 = p.start[b];
      live = r0 >= 0 && r0 <= t && s0 >= 0;
      slot = s0 + (t - r0);
    }
    Position pos;
    if (p.pos)
      pos.load(p.pos, axes, p.tokens, t);
    else
      pos.at[0] = static_cast<int>(slot), pos.at[1] = pos.at[2] = pos.at[3] = 0;
    Turn turn;
    rows.template turn<true>(turn, &sh, c, pos, axes, w != nullptr);
    rows.finish(static_cast<bf16*>(p.q_out) + (t * p.hq + h) * D + 16 * c, n, turn, w != nullptr, p.eps, live, p.wide);
    return;
  }

  // ---- keys and values: the item's sequence, by a running count of (sequence, page)
  const long long item = blockIdx.x / p.hkv;
  const int kvh = static_cast<int>(blockIdx.x % p.hkv);
  if (tid == 0) s_item[2] = 0;
  long long before = 0;
  for (int b0 = 0; b0 < p.batch && before <= item; b0 += kApThreads) {
    const int b = b0 + tid;
    long long items = 0, r0 = 0, n = 0, s0 = -1;
    if (b < p.batch) {
      r0 = p.cu[b];
      const long long r1 = p.cu[b + 1];
      s0 = p.start[b];
      if (r0 < 0 || r1 < r0 || r1 > p.tokens) {
        atomicCAS(p.err, 0u, kErrBadRows);
      } else if (s0 >= 0 && r1 > r0) {
        n = r1 - r0;
        items = ((s0 + n - 1) >> p.page_log2) - (s0 >> p.page_log2) + 1;
      }
    }
    long long incl = items;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    __syncthreads();  // the last round's sums are read
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    long long mine = item - before - (incl - items);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) mine -= s_scan[w];
      before += s_scan[w];
    }
    if (mine >= 0 && mine < items) {
      const long long first = mine == 0 ? s0 : ((s0 >> p.page_log2) + mine) << p.page_log2;
      const long long end = min(s0 + n, ((first >> p.page_log2) + 1) << p.page_log2);
      s_item[0] = b;
      s_item[1] = static_cast<int>(r0 + (first - s0));
      s_item[2] = static_cast<int>(end - first);
      s_slot = first;
    }
  }
  __syncthreads();
  const int b = s_item[0], row0 = s_item[1], n = s_item[2];
  if (n == 0) return;
  const long long slot0 = s_slot;
  const int at0 = static_cast<int>(slot0 & ((1 << p.page_log2) - 1));
  const bf16* w = static_cast<const bf16*>(p.k_weight);
  // a token ahead: its key, value and positions
  Chunk<bf16, kHalf> next, cw;
  uint32_t v_next[8];
  Position pos_next;
  auto fetch = [&](int t) {  // clamped: lanes behind the last repeat it
    const long long tt = min(t, n - 1), row = row0 + tt;
    next.load(static_cast<const bf16*>(p.k) + row * p.k_stride + kvh * D, c, D);
    load32(v_next, static_cast<const bf16*>(p.v) + row * p.v_stride + kvh * D + 16 * c);
    if (p.pos)
      pos_next.load(p.pos, axes, p.tokens, row);
    else
      pos_next.at[0] = static_cast<int>(slot0 + tt), pos_next.at[1] = pos_next.at[2] = pos_next.at[3] = 0;
  };
  fetch(tid / NC);
  const int page = page_of(p, b, slot0 >> p.page_log2);
  if (w) cw.load(w, c, D);
  constexpr uint32_t kInf = 0x7F807F80u, kNegInf = 0xFF80FF80u;
  uint32_t lo[8], hi[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) lo[k] = kInf, hi[k] = kNegInf;
  for (int t0 = 0; t0 < n; t0 += kTok) {
    const int t = t0 + tid / NC;
    const Chunk<bf16, kHalf> in = next;
    const Position pos = pos_next;
    uint32_t v[8], y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = v_next[k];
    if (t0 + kTok < n) fetch(t + kTok);
    turn_one<D, kHalf>(y, in, cw, w != nullptr, p.eps, &sh, c, pos, axes);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      lo[k] = min_bf16x2(lo[k], y[k]);
      hi[k] = max_bf16x2(hi[k], y[k]);
    }
    if (t < n && page >= 0) store_slot<D>(p, page, kvh, c, at0 + t, y, v);
  }
  if (!p.bounds || page < 0) return;
#pragma unroll
  for (int off = NC; off < 32; off <<= 1)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      lo[k] = min_bf16x2(lo[k], __shfl_xor_sync(0xffffffffu, lo[k], off));
      hi[k] = max_bf16x2(hi[k], __shfl_xor_sync(0xffffffffu, hi[k], off));
    }
  if (lane < NC) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      s_red[0][warp][8 * c + k] = lo[k];
      s_red[1][warp][8 * c + k] = hi[k];
    }
  }
  __syncthreads();
  for (int i = tid; i < D; i += kApThreads) {  // word i % (D/2) of the minima, then of the maxima
    const int which = i / (D / 2), x = i % (D / 2);
    uint32_t* dst = reinterpret_cast<uint32_t*>(bounds_row<D>(p, page, kvh, which, 0)) + x;
    uint32_t r = s_red[which][0][x];
    for (int k = 1; k < kWarps; ++k) r = which ? max_bf16x2(r, s_red[1][k][x]) : min_bf16x2(r, s_red[0][k][x]);
    if (at0) r = which ? max_bf16x2(r, *dst) : min_bf16x2(r, *dst);
    *dst = r;
  }
}

long long paged_append_blocks(const PagedAppendParams& p) {
  const int tok = p.threads / (p.d / 16), groups = p.q ? (p.hq + kRows - 1) / kRows : 0;
  return p.items * p.hkv + (p.tokens + tok - 1LL) / tok * groups;
}

template <int D, bool kHalf>
static cudaError_t launch_append(const PagedAppendParams& p, cudaStream_t s) {
  if (p.cu) {
    const unsigned blocks = static_cast<unsigned>(paged_append_blocks(p));
    return p.threads == 64    ? launch_pdl(paged_append_kernel<D, kHalf, 64>, blocks, 64, 0, s, p)
           : p.threads == 128 ? launch_pdl(paged_append_kernel<D, kHalf, 128>, blocks, 128, 0, s, p)
                              : launch_pdl(paged_append_kernel<D, kHalf, 256>, blocks, 256, 0, s, p);
  }
  const long long threads = static_cast<long long>(p.batch) * (p.hkv + (p.q ? p.hq : 0)) * (D / 16);
  return launch_pdl(paged_append_step_kernel<D, kHalf>, static_cast<unsigned>((threads + kNrThreads - 1) / kNrThreads), kNrThreads,
                    0, s, p);
}

cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t s) {
  if (p.d == 64) return p.pairing ? launch_append<64, true>(p, s) : launch_append<64, false>(p, s);
  return p.pairing ? launch_append<128, true>(p, s) : launch_append<128, false>(p, s);
}

}  // namespace atf
