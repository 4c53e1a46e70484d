// atf_internal.cuh -- kernel parameter blocks and launchers shared by the
// library's translation units (not part of the public C ABI).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/atf.h"

namespace atf {

constexpr int kMaxPairs = 64;      // d <= 128
constexpr int kMaxDecodeBatch = 64;  // sequences per decode launch

// Window table in the kernels' integer domain: W_i clamped to INT32_MAX (every
// distance the kernels can see is below 2^31, so clamping changes nothing).
struct Windows {
  int w[kMaxPairs];
};

struct RopeParams {
  const void* x;
  void* x_rot;      // nullable
  void* x_chunked;  // nullable, bf16 only: [B][H][d/16][S][16]
  int batch, seq, heads, d;
  long long pos_offset;
  int rotate;  // 0: copy, 1: RoPE, 2: rotate-half RoPE, 3: rotate-half copy (2, 3 write pairs interleaved)
  int fp32;    // 1: fp32 elements, 0: bf16
  double omega[kMaxPairs];
};

struct PrefillParams {
  const void* q;    // rotated queries  [B][q_len][Hq][d]
  const void* k;    // rotated keys     [B][kv_len][Hkv][d]
  const void* v;    // values           [B][kv_len][Hkv][d]
  void* out;        // [B][q_len][Hq][d]
  int batch, q_len, kv_len, hq, hkv, d;
  long long q_offset;
  unsigned long long* skipped;  // nullable
  unsigned int* err;            // device error word
  Windows win;
};

struct DecodeParams {
  const void* q;         // raw queries [B][Hq][d]
  const void* kc;        // rotated key cache, chunk-major [B][Hkv][d/16][n_cache][16]
  const void* v;         // value cache [B][n_cache][Hkv][d]
  void* out;             // [B][Hq][d]
  float* partials;       // [B][Hq][n_split][d + 2]
  int batch, hq, hkv, d, n_split;
  int pairing;           // atf_pairing of the raw queries
  long long n_cache;
  long long kv_len[kMaxDecodeBatch];    // keys in this cache: slots 0 .. kv_len-1
  long long q_pos[kMaxDecodeBatch];     // query position (its RoPE angle)
  long long key_pos0[kMaxDecodeBatch];  // position of slot 0 (a key range of a longer sequence)
  float* partial_out;           // nullable: [B][Hq][d + 2] merged (sum, max, row sum) instead of out
  unsigned long long* skipped;  // nullable
  unsigned int* err;
  Windows win;
  double omega[kMaxPairs];
};

struct AppendParams {
  const void* k_new;  // [total_new][hkv][d] bf16, sequences one after the other
  const void* v_new;  // same layout
  void* kc;           // rotated key cache, chunk-major [B][Hkv][d/16][n_cache][16]
  void* vc;           // value cache [B][n_cache][Hkv][d]
  int batch, hkv, d, pairing;
  long long n_cache;
  long long cu[kMaxDecodeBatch + 1];  // first row of sequence b in k_new / v_new
  long long pos[kMaxDecodeBatch];     // position (cache slot) of sequence b's first new token
  double omega[kMaxPairs];
};

// Rotation angles of up to four position axes: pair i of a token turns by
// pos[axis of i] * theta^(-2i/d), held in turns of 2^64.
constexpr int kMaxAxes = 4;
struct RotaryTable {
  unsigned long long turns[kMaxPairs];  // round(2^64 theta^(-2i/d) / (2 pi))
  unsigned char axis[kMaxPairs];    // < kMaxAxes
  int n_axes;
};

struct NormRopeParams {
  const void *q, *k;                // token t, head h at element t * stride + h * d
  long long q_stride, k_stride;
  void *q_out, *k_out;              // contiguous [tokens][heads][d], pairs interleaved
  const void *q_weight, *k_weight;  // [d] in the element type, nullable: no norm
  const long long* pos;             // [n_axes][tokens]
  int tokens, hq, hkv, d, pairing, fp32;
  bool wide;                        // the outputs are 32-byte aligned
  float eps;
  RotaryTable rot;
};

struct PagedAppendParams {
  const void *q, *k, *v;            // q nullable; token t, head h at element t * stride + h * d, bf16
  long long q_stride, k_stride, v_stride;
  void* q_out;                      // [tokens][hq][d]
  void *k_pages, *v_pages, *bounds; // bounds nullable
  const void *q_weight, *k_weight;
  const int *page_table, *start, *cu;  // cu nullable: one token per sequence
  const long long* pos;             // nullable: the slot
  int tokens, batch, hq, hkv, d, pairing, page_log2, max_pages, num_pages;
  long long items;                  // at least the pages that the new tokens of all sequences fall into
  int threads;                      // of a CTA of a ragged append: 64, 128 or 256
  bool wide;                        // q_out and the pages are 32-byte aligned
  float eps;
  unsigned int* err;
  RotaryTable rot;
};

struct PagedDecodeParams {
  const void* q;          // rotated queries, sequence b at element b * q_stride
  long long q_stride;
  const int *page_table, *kv_len, *selected;  // selected nullable: [batch][hkv][n_sel] logical pages
  void* out;              // [batch][hq][d] bf16
  float* lse;             // nullable [batch][hq]
  float* partials;        // [kPagedCtas][2][8][d] weighted sums of the pieces
  float2* sums;           // [kPagedCtas][2][8] their maxima and row sums
  int4* meta;             // [kPagedCtas]: split sequence, kv head, last CTA of the sequences begun by each CTA
  int batch, hq, hkv, d, page_log2, max_pages, num_pages, n_sel;
  int tile_keys;          // keys of the TMA boxes and tiles: 64, or 128 with d = 64
  unsigned int* err;
  Windows win;
};

struct PageSelectParams {
  const void* q;
  long long q_stride;
  const void* bounds;     // [num_pages][hkv][2][d] bf16
  const int *page_table, *kv_len;
  unsigned long long* keys;  // [batch][hkv][max_pages] scores in sortable form
  int* selected;          // [batch][hkv][n_sel]
  int batch, hq, hkv, d, page_log2, max_pages, num_pages, n_sel, n_first, n_last;
  unsigned int* err;
  Windows win;
};

// CTAs of a paged decode: one per SM of a B200.
constexpr int kPagedCtas = 148;
// Keys of a tile of its work, of up to `keys` keys of all sequences and kv heads: 64, but
// 128 where heads of 64 fill every CTA with eight tiles of 64 or more.  450091 keys of 4
// kv heads of 64 take 76 us in tiles of 64, 52 in tiles of 128; 777 keys 6.9 and 7.9.
constexpr int paged_tile_keys(int d, double keys) { return d == 64 && keys >= 8.0 * 64 * kPagedCtas ? 128 : 64; }

// Codes of the device error word for bad data in device arrays (the entry is
// skipped); bounded waits that expired record smaller codes.
constexpr unsigned int kErrBadData = 0x10000u;
constexpr unsigned int kErrBadPage = kErrBadData | 1;    // page index outside the pool
constexpr unsigned int kErrBadLength = kErrBadData | 2;  // more keys than the page table holds
constexpr unsigned int kErrBadRows = kErrBadData | 3;    // row offsets outside the input
constexpr unsigned int kErrBadSelect = kErrBadData | 4;  // selected page behind the sequence

// A launch that may start while the stream's previous kernel drains; the kernel
// calls pdl_wait() in every thread before it reads or writes what others write.
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const Args&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Launchers (return cudaGetLastError() of the launch).
cudaError_t launch_qk_norm_rope(const NormRopeParams& p, cudaStream_t s);
cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t s);
long long paged_append_blocks(const PagedAppendParams& p);  // CTAs of a ragged append
cudaError_t launch_paged_decode(const PagedDecodeParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                cudaStream_t s);
cudaError_t launch_page_select(const PageSelectParams& p, cudaStream_t s);
cudaError_t launch_rope(const RopeParams& p, cudaStream_t s);
cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t s);
cudaError_t launch_prefill_simt(const PrefillParams& p, cudaStream_t s);
cudaError_t launch_prefill_tc(const PrefillParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                              const CUtensorMap& tm_v, bool dense, cudaStream_t s);
cudaError_t launch_decode_merge(const float* parts, int n_parts, long long rows, int d, void* out, cudaStream_t s);
cudaError_t launch_decode(const DecodeParams& p, const CUtensorMap& tm_v, const CUtensorMap& tm_k,
                          cudaStream_t s);

// Device address of the library's error word on the current device (bounded
// waits record their code there), or NULL without a usable device.
unsigned int* device_error_word();

// Records a printf-style message as this thread's atf_last_error() and returns st.
atf_status report_error(atf_status st, const char* fmt, ...);

// Checks d, theta and alpha; records a message and returns its status.
atf_status check_method(int d, double theta, double alpha);

// Windows of the pairs in the kernels' integer domain.
void method_windows(int d, double theta, double alpha, Windows* out);

// Tiled tensor map of a 4-D bf16 tensor (dims innermost first, strides of dims
// 1..3 in bytes); elements outside read as zero.
atf_status tensor_map_4d(CUtensorMap* map, const void* base, const unsigned long long dims[4],
                         const unsigned long long strides[3], const unsigned int box[4], CUtensorMapSwizzle swizzle);

// Number of key-range splits per (sequence, kv head) for a decode launch.
int decode_num_splits(long long max_kv_len, int batch, int hkv);

}  // namespace atf
