// qk_norm_rope.cu -- RMS norm of every query and key head and the position
// rotation in one pass, to contiguous rows (the operands of the prefill) or, for
// new tokens of a batch, to a paged key-value cache.
//
//   y = x * rsqrt(mean(x^2) + eps) * w           (per head; skipped without w)
//   (y_a, y_b) of pair i turned by pos[axis(i)] * theta^(-2i/d)
//
// all in fp32 and rounded once.  The angle is reduced to a fraction of a turn in
// fp64 (at position 2^20 an fp32 angle is off by more than a bf16 step), and the
// sine and cosine of that fraction are fp32.
//
// One thread owns a token's 8-pair chunk c: elements 16c..16c+15 of a head
// (interleaved pairs) or 8c..8c+7 and d/2+8c..d/2+8c+7 (rotate-half), which are
// the 16 outputs 16c..16c+15 either way and one 32-byte row of the key pages.  It
// evaluates the chunk's eight angles once and loops over heads; the d/16 lanes of
// a head add their squares by shuffles.
#include <cuda_bf16.h>

#include "atf_internal.cuh"
#include "ptx.cuh"

namespace atf {

namespace {

constexpr int kNrThreads = 128;

template <typename T>
struct Chunk;  // 16 elements as loaded: the first components a[8] and second b[8] of eight pairs

template <>
struct Chunk<__nv_bfloat16> {
  uint4 lo, hi;
  __device__ void load(const __nv_bfloat16* row, int c, int d, bool half) {
    lo = *reinterpret_cast<const uint4*>(row + (half ? 8 * c : 16 * c));
    hi = *reinterpret_cast<const uint4*>(row + (half ? d / 2 + 8 * c : 16 * c + 8));
  }
  __device__ void pairs(bool half, float* a, float* b) const {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (half) {
        a[k] = (k & 1) ? bf16hi_to_f32(w[k >> 1]) : bf16lo_to_f32(w[k >> 1]);
        b[k] = (k & 1) ? bf16hi_to_f32(w[4 + (k >> 1)]) : bf16lo_to_f32(w[4 + (k >> 1)]);
      } else {
        a[k] = bf16lo_to_f32(w[k]);
        b[k] = bf16hi_to_f32(w[k]);
      }
    }
  }
  __device__ static void store(__nv_bfloat16* dst, const float* a, const float* b) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(a[k], b[k]);
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
};

template <>
struct Chunk<float> {
  float4 v[4];
  __device__ void load(const float* row, int c, int d, bool half) {
    const float4* lo = reinterpret_cast<const float4*>(row + (half ? 8 * c : 16 * c));
    const float4* hi = reinterpret_cast<const float4*>(row + (half ? d / 2 + 8 * c : 16 * c + 8));
    v[0] = lo[0], v[1] = lo[1], v[2] = hi[0], v[3] = hi[1];
  }
  __device__ void pairs(bool half, float* a, float* b) const {
    const float w[16] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w,
                         v[2].x, v[2].y, v[2].z, v[2].w, v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      a[k] = half ? w[k] : w[2 * k];
      b[k] = half ? w[8 + k] : w[2 * k + 1];
    }
  }
  __device__ static void store(float* dst, const float* a, const float* b) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      reinterpret_cast<float4*>(dst)[k] = make_float4(a[2 * k], b[2 * k], a[2 * k + 1], b[2 * k + 1]);
  }
};

struct RotaryShared {
  double turns[kMaxPairs];
  unsigned char axis[kMaxPairs];
};

__device__ void load_rotary(RotaryShared* sh, const RotaryTable& rot, int d) {
  for (int i = threadIdx.x; i < d / 2; i += blockDim.x) {
    sh->turns[i] = rot.turns[i];
    sh->axis[i] = rot.axis[i];
  }
  __syncthreads();
}

// Cosine and sine of the eight angles of chunk c.
__device__ __forceinline__ void chunk_angles(const RotaryShared* sh, int c, const long long* pos, int n_axes, float* cs,
                                             float* sn) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    long long p = pos[0];
    if (n_axes > 1) {
      const int a = sh->axis[8 * c + k];
      p = a == 1 ? pos[1] : a == 2 ? pos[2] : a == 3 ? pos[3] : p;
    }
    const double t = static_cast<double>(p) * sh->turns[8 * c + k];
    sincospif(2.0f * static_cast<float>(t - rint(t)), &sn[k], &cs[k]);
  }
}

// Norm (with weights wa, wb of the eight pairs) and rotation of one head's chunk
// over the d/16 neighbouring lanes of the head; every lane of the warp calls it.
template <int D>
__device__ __forceinline__ void norm_rotate(float* a, float* b, bool norm, const float* wa, const float* wb, float eps,
                                            const float* cs, const float* sn) {
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) ss += a[k] * a[k] + b[k] * b[k];
#pragma unroll
    for (int off = 1; off < D / 16; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      a[k] *= r * wa[k];
      b[k] *= r * wb[k];
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float x = a[k], y = b[k];
    a[k] = x * cs[k] - y * sn[k];
    b[k] = x * sn[k] + y * cs[k];
  }
}

}  // namespace

// Dense form.  Thread = (token, chunk), blockIdx.y = a group of kNrRows heads of
// the queries and keys taken as one list.
constexpr int kNrRows = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kNrThreads) qk_norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int NC = D / 16;
  __shared__ RotaryShared sh;
  load_rotary(&sh, p.rot, D);
  const long long idx = static_cast<long long>(blockIdx.x) * kNrThreads + threadIdx.x;
  const int c = static_cast<int>(idx % NC);
  const bool live = idx / NC < p.tokens;
  const long long t = live ? idx / NC : p.tokens - 1;
  const bool half = p.pairing != 0;
  long long pos[kMaxAxes];
  for (int a = 0; a < kMaxAxes; ++a) pos[a] = a < p.rot.n_axes ? p.pos[static_cast<long long>(a) * p.tokens + t] : 0;
  float cs[8], sn[8];
  chunk_angles(&sh, c, pos, p.rot.n_axes, cs, sn);
  const int r1 = min(p.hq + p.hkv, (static_cast<int>(blockIdx.y) + 1) * kNrRows);
  for (int r = blockIdx.y * kNrRows; r < r1; ++r) {
    const bool key = r >= p.hq;
    const int h = key ? r - p.hq : r;
    const T* x = static_cast<const T*>(key ? p.k : p.q);
    if (!x) continue;
    const T* w = static_cast<const T*>(key ? p.k_weight : p.q_weight);
    Chunk<T> ch;
    ch.load(x + t * (key ? p.k_stride : p.q_stride) + h * D, c, D, half);
    float a[8], b[8], wa[8], wb[8];
    ch.pairs(half, a, b);
    if (w) {
      Chunk<T> cw;
      cw.load(w, c, D, half);
      cw.pairs(half, wa, wb);
    }
    norm_rotate<D>(a, b, w != nullptr, wa, wb, p.eps, cs, sn);
    T* out = static_cast<T*>(key ? p.k_out : p.q_out);
    if (live) Chunk<T>::store(out + (t * (key ? p.hkv : p.hq) + h) * D + 16 * c, a, b);
  }
}

cudaError_t launch_qk_norm_rope(const NormRopeParams& p, cudaStream_t s) {
  const long long threads = static_cast<long long>(p.tokens) * (p.d / 16);
  const dim3 grid(static_cast<unsigned>((threads + kNrThreads - 1) / kNrThreads), (p.hq + p.hkv + kNrRows - 1) / kNrRows);
  if (p.fp32)
    p.d == 64 ? qk_norm_rope_kernel<float, 64><<<grid, kNrThreads, 0, s>>>(p)
              : qk_norm_rope_kernel<float, 128><<<grid, kNrThreads, 0, s>>>(p);
  else
    p.d == 64 ? qk_norm_rope_kernel<__nv_bfloat16, 64><<<grid, kNrThreads, 0, s>>>(p)
              : qk_norm_rope_kernel<__nv_bfloat16, 128><<<grid, kNrThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ paged append

namespace {

// One new token's chunk of kv head kvh: its queries to q_out, its key and value
// to slot `at` of page `page` (page < 0: nowhere).  Returns the rounded key in
// kw.  Every lane of the warp calls it; `live` lanes write.
template <int D>
__device__ __forceinline__ void append_token(const PagedAppendParams& p, const RotaryShared* sh, long long row, long long slot,
                                             int kvh, int c, int page, int at, bool live, uint32_t* kw) {
  using T = __nv_bfloat16;
  const bool half = p.pairing != 0;
  const int G = p.hq / p.hkv;
  Chunk<T> kc;
  kc.load(static_cast<const T*>(p.k) + row * p.k_stride + kvh * D, c, D, half);
  const uint4* vr = reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + row * p.v_stride + kvh * D + 16 * c);
  const uint4 v0 = vr[0], v1 = vr[1];
  long long pos[kMaxAxes] = {slot, 0, 0, 0};
  if (p.pos)
    for (int a = 0; a < p.rot.n_axes; ++a) pos[a] = p.pos[static_cast<long long>(a) * p.tokens + row];
  float cs[8], sn[8], a[8], b[8], wa[8], wb[8];
  chunk_angles(sh, c, pos, p.pos ? p.rot.n_axes : 1, cs, sn);
  if (p.k_weight) {
    Chunk<T> cw;
    cw.load(static_cast<const T*>(p.k_weight), c, D, half);
    cw.pairs(half, wa, wb);
  }
  kc.pairs(half, a, b);
  norm_rotate<D>(a, b, p.k_weight != nullptr, wa, wb, p.eps, cs, sn);
#pragma unroll
  for (int k = 0; k < 8; ++k) kw[k] = pack_bf16x2(a[k], b[k]);
  if (live && page >= 0) {
    const long long ps = 1LL << p.page_log2;
    const long long head = static_cast<long long>(page) * p.hkv + kvh;
    uint4* kd = reinterpret_cast<uint4*>(static_cast<T*>(p.k_pages) + ((head * (D / 16) + c) * ps + at) * 16);
    kd[0] = make_uint4(kw[0], kw[1], kw[2], kw[3]);
    kd[1] = make_uint4(kw[4], kw[5], kw[6], kw[7]);
    uint4* vd = reinterpret_cast<uint4*>(static_cast<T*>(p.v_pages) + (head * ps + at) * D + 16 * c);
    vd[0] = v0;
    vd[1] = v1;
  }
  if (!p.q) return;
  if (p.q_weight) {
    Chunk<T> cw;
    cw.load(static_cast<const T*>(p.q_weight), c, D, half);
    cw.pairs(half, wa, wb);
  }
  for (int g = 0; g < G; ++g) {
    const int h = kvh * G + g;
    Chunk<T> qc;
    qc.load(static_cast<const T*>(p.q) + row * p.q_stride + h * D, c, D, half);
    qc.pairs(half, a, b);
    norm_rotate<D>(a, b, p.q_weight != nullptr, wa, wb, p.eps, cs, sn);
    if (live) Chunk<T>::store(static_cast<T*>(p.q_out) + (row * p.hq + h) * D + 16 * c, a, b);
  }
}

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

// Bounds rows of chunk c: 8 words of minima and of maxima.
template <int D>
__device__ __forceinline__ uint4* bounds_row(const PagedAppendParams& p, int page, int kvh, int which, int c) {
  return reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.bounds) +
                                  ((static_cast<long long>(page) * p.hkv + kvh) * 2 + which) * D + 16 * c);
}

}  // namespace

// One token per sequence: thread = (sequence, kv head, chunk).
template <int D>
__global__ void __launch_bounds__(64) paged_append_step_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int NC = D / 16;
  __shared__ RotaryShared sh;
  load_rotary(&sh, p.rot, D);
  const long long idx = static_cast<long long>(blockIdx.x) * 64 + threadIdx.x;
  const int c = static_cast<int>(idx % NC);
  const int kvh = static_cast<int>((idx / NC) % p.hkv);
  const long long bl = idx / NC / p.hkv;
  const int b = bl < p.batch ? static_cast<int>(bl) : p.batch - 1;
  const long long slot = p.start[b];
  const bool live = bl < p.batch && slot >= 0;
  const int page = live ? page_of(p, b, slot >> p.page_log2) : -1;
  const int at = static_cast<int>(slot & ((1 << p.page_log2) - 1));
  uint32_t kw[8];
  append_token<D>(p, &sh, b, slot, kvh, c, page, at, live, kw);
  if (p.bounds && page >= 0) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      uint4* row = bounds_row<D>(p, page, kvh, which, c);
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = kw[k];
      if (at) {  // the page holds earlier keys
        const uint4 o0 = row[0], o1 = row[1];
        const uint32_t o[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = which ? max_bf16x2(w[k], o[k]) : min_bf16x2(w[k], o[k]);
      }
      row[0] = make_uint4(w[0], w[1], w[2], w[3]);
      row[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

// Ragged batch: a CTA owns the new tokens of one sequence that fall into one
// page, for one kv head, so that the page's bounds have one writer.
template <int D>
__global__ void __launch_bounds__(kNrThreads) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int NC = D / 16, kTok = kNrThreads / NC;  // tokens in flight
  __shared__ RotaryShared sh;
  __shared__ int s_item[3];  // sequence, first row, tokens
  __shared__ long long s_slot;  // first slot
  __shared__ uint32_t s_red[2][kNrThreads / 32][D / 2];
  const int tid = threadIdx.x;
  // the item's sequence: running count of (sequence, page) items, one warp
  if (tid < 32) {
    long long before = 0;
    bool found = false;
    for (int b0 = 0; b0 < p.batch && !found; b0 += 32) {
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
        if (tid >= off) incl += o;
      }
      const long long mine = static_cast<long long>(blockIdx.x) - before - (incl - items);
      const bool here = mine >= 0 && mine < items;
      if (here) {
        const long long first = mine == 0 ? s0 : ((s0 >> p.page_log2) + mine) << p.page_log2;
        const long long end = min(s0 + n, ((first >> p.page_log2) + 1) << p.page_log2);
        s_item[0] = b;
        s_item[1] = static_cast<int>(r0 + (first - s0));
        s_item[2] = static_cast<int>(end - first);
        s_slot = first;
      }
      found = __any_sync(0xffffffffu, here);
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (!found && tid == 0) s_item[2] = 0;
  }
  load_rotary(&sh, p.rot, D);  // synchronises
  const int b = s_item[0], row0 = s_item[1], n = s_item[2];
  const long long slot0 = s_slot;
  if (n == 0) return;
  const int kvh = blockIdx.y, c = tid % NC;
  const int page = page_of(p, b, slot0 >> p.page_log2);
  const int at0 = static_cast<int>(slot0 & ((1 << p.page_log2) - 1));
  constexpr uint32_t kInf = 0x7F807F80u, kNegInf = 0xFF80FF80u;
  uint32_t lo[8], hi[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) lo[k] = kInf, hi[k] = kNegInf;
  for (int t0 = 0; t0 < n; t0 += kTok) {
    const int t = t0 + tid / NC;
    const bool live = t < n;
    const int tt = live ? t : n - 1;
    uint32_t kw[8];
    append_token<D>(p, &sh, row0 + tt, slot0 + tt, kvh, c, page, at0 + tt, live, kw);
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // a clamped lane repeats the last token's key
      lo[k] = min_bf16x2(lo[k], kw[k]);
      hi[k] = max_bf16x2(hi[k], kw[k]);
    }
  }
  if (!p.bounds || page < 0) return;
#pragma unroll
  for (int off = NC; off < 32; off <<= 1)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      lo[k] = min_bf16x2(lo[k], __shfl_xor_sync(0xffffffffu, lo[k], off));
      hi[k] = max_bf16x2(hi[k], __shfl_xor_sync(0xffffffffu, hi[k], off));
    }
  if ((tid & 31) < NC) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      s_red[0][tid >> 5][8 * c + k] = lo[k];
      s_red[1][tid >> 5][8 * c + k] = hi[k];
    }
  }
  __syncthreads();
  for (int i = tid; i < D; i += kNrThreads) {  // word i % (D/2) of the minima, then of the maxima
    const int which = i / (D / 2), w = i % (D / 2);
    uint32_t* dst = reinterpret_cast<uint32_t*>(bounds_row<D>(p, page, kvh, which, 0)) + w;
    uint32_t r = s_red[which][0][w];
    for (int k = 1; k < kNrThreads / 32; ++k) r = which ? max_bf16x2(r, s_red[1][k][w]) : min_bf16x2(r, s_red[0][k][w]);
    if (at0) r = which ? max_bf16x2(r, *dst) : min_bf16x2(r, *dst);
    *dst = r;
  }
}

cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t s) {
  if (!p.cu) {
    const long long threads = static_cast<long long>(p.batch) * p.hkv * (p.d / 16);
    const unsigned blocks = static_cast<unsigned>((threads + 63) / 64);
    p.d == 64 ? paged_append_step_kernel<64><<<blocks, 64, 0, s>>>(p)
              : paged_append_step_kernel<128><<<blocks, 64, 0, s>>>(p);
  } else {
    // a sequence with n > 0 new tokens touches at most (n - 1) / page + 2 pages
    const long long items = (p.tokens >> p.page_log2) + 2LL * (p.batch < p.tokens ? p.batch : p.tokens);
    const dim3 grid(static_cast<unsigned>(items), p.hkv);
    p.d == 64 ? paged_append_kernel<64><<<grid, kNrThreads, 0, s>>>(p)
              : paged_append_kernel<128><<<grid, kNrThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace atf
