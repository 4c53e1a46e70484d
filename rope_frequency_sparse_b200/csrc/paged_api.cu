// paged_api.cu -- C ABI of the per-head norms with rotation, the paged cache, its
// decode and its page selection (include/atf.h): argument checks, the rotation
// table, TMA descriptors and kernel launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/atf.h"
#include "atf_internal.cuh"

using namespace atf;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Rows of a strided operand: a stride in elements that keeps every row 16-byte
// aligned and holds its heads.
bool bad_stride(long long stride, long long row, int esz) { return stride < row || (stride * esz) % 16 != 0; }

// Whether [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

// Bytes from the first element of a [tokens][row] operand to its last.
size_t span(long long tokens, long long stride, long long row, int esz) {
  return tokens ? (static_cast<size_t>(tokens - 1) * stride + row) * esz : 0;
}

// log2 of a supported page size, or -1.
int page_log2(int page_size) {
  switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    default: return -1;
  }
}

atf_status rotary_table(const char* who, int d, double theta, int n_axes, const unsigned char* pair_axis,
                        RotaryTable* rot) {
  if (n_axes < 1 || n_axes > kMaxAxes)
    return report_error(ATF_ERR_UNSUPPORTED, "%s: n_axes %d outside [1, %d]", who, n_axes, kMaxAxes);
  if (n_axes > 1 && !pair_axis)
    return report_error(ATF_ERR_INVALID_ARG, "%s: several position axes need pair_axis", who);
  const long double turn = 18446744073709551616.0L / 6.283185307179586476925286766559L;  // 2^64 / (2 pi)
  // a thread's calls mostly share d and theta; the powers take longer than the launch
  static thread_local struct {
    int d = 0;
    double theta = 0.0;
    unsigned long long turns[kMaxPairs] = {};
  } last;
  if (last.d != d || last.theta != theta) {
    for (int i = 0; i < kMaxPairs; ++i)
      last.turns[i] = i < d / 2 ? static_cast<unsigned long long>(
                                      std::round(std::pow(static_cast<long double>(theta), -2.0L * i / d) * turn))
                                : 0ull;
    last.d = d;
    last.theta = theta;
  }
  rot->n_axes = n_axes;
  for (int i = 0; i < kMaxPairs; ++i) rot->turns[i] = last.turns[i], rot->axis[i] = 0;
  for (int i = 0; i < d / 2; ++i) {
    if (pair_axis) {
      if (pair_axis[i] >= n_axes)
        return report_error(ATF_ERR_INVALID_ARG, "%s: pair_axis[%d] = %d, but there are %d axes", who, i,
                            static_cast<int>(pair_axis[i]), n_axes);
      rot->axis[i] = pair_axis[i];
    }
  }
  return ATF_OK;
}

atf_status check_heads(const char* who, int heads, int kv_heads) {
  if (heads < 1 || kv_heads < 1) return report_error(ATF_ERR_INVALID_ARG, "%s: bad head counts", who);
  if (heads % kv_heads) return report_error(ATF_ERR_INVALID_ARG, "%s: heads %% kv_heads != 0", who);
  return ATF_OK;
}

// Sizes of a page pool and its tables.
atf_status check_pool(const char* who, int page_size, long long num_pages, int max_pages, int kv_heads) {
  const int lg = page_log2(page_size);
  if (lg < 0) return report_error(ATF_ERR_UNSUPPORTED, "%s: page size %d (16, 32, 64 or 128)", who, page_size);
  if (num_pages < 1 || max_pages < 1) return report_error(ATF_ERR_INVALID_ARG, "%s: empty page pool or table", who);
  if (num_pages > 0x7fffffffLL / kv_heads)
    return report_error(ATF_ERR_UNSUPPORTED, "%s: num_pages * kv_heads must stay below 2^31", who);
  if ((static_cast<long long>(max_pages) << lg) > 0x7fffff80LL)
    return report_error(ATF_ERR_UNSUPPORTED, "%s: max_pages * page_size must stay below 2^31", who);
  return ATF_OK;
}

constexpr size_t kMetaBytes = (kPagedCtas * sizeof(int4) + 255) / 256 * 256;

}  // namespace

extern "C" {

atf_status atf_qk_norm_rope(const atf_qk_norm_rope_args* a, void* stream) {
  const char* who = "qk_norm_rope";
  if (!a) return report_error(ATF_ERR_INVALID_ARG, "args is NULL");
  if (atf_status st = check_method(a->d, a->theta, 1.0)) return st;
  if (a->dtype != ATF_BF16 && a->dtype != ATF_FP32) return report_error(ATF_ERR_INVALID_ARG, "bad dtype %d", a->dtype);
  if (a->pairing != ATF_PAIRS_INTERLEAVED && a->pairing != ATF_PAIRS_ROTATE_HALF)
    return report_error(ATF_ERR_INVALID_ARG, "%s: pairing %d", who, a->pairing);
  if (a->tokens < 0 || a->heads < 0 || a->kv_heads < 0 || a->heads + static_cast<long long>(a->kv_heads) < 1)
    return report_error(ATF_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (a->heads + static_cast<long long>(a->kv_heads) > 65535)
    return report_error(ATF_ERR_UNSUPPORTED, "%s: more than 65535 heads", who);
  if (!(a->eps >= 0.f) || std::isinf(a->eps)) return report_error(ATF_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
  NormRopeParams p{};
  if (atf_status st = rotary_table(who, a->d, a->theta, a->n_axes, a->pair_axis, &p.rot)) return st;
  if (a->tokens == 0) return ATF_OK;
  if ((a->heads && (!a->q || !a->q_out)) || (a->kv_heads && (!a->k || !a->k_out)) || !a->pos)
    return report_error(ATF_ERR_INVALID_ARG, "%s: null pointer", who);
  const int esz = a->dtype == ATF_FP32 ? 4 : 2;
  const long long qrow = static_cast<long long>(a->heads) * a->d, krow = static_cast<long long>(a->kv_heads) * a->d;
  if ((a->heads && bad_stride(a->q_stride, qrow, esz)) || (a->kv_heads && bad_stride(a->k_stride, krow, esz)))
    return report_error(ATF_ERR_INVALID_ARG, "%s: strides must hold the heads and keep 16-byte alignment", who);
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->q_out) || !aligned16(a->k_out) || !aligned16(a->q_weight) ||
      !aligned16(a->k_weight) || !aligned16(a->pos))
    return report_error(ATF_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  const void* in[2] = {a->heads ? a->q : nullptr, a->kv_heads ? a->k : nullptr};
  const size_t in_bytes[2] = {span(a->tokens, a->q_stride, qrow, esz), span(a->tokens, a->k_stride, krow, esz)};
  void* out[2] = {a->heads ? a->q_out : nullptr, a->kv_heads ? a->k_out : nullptr};
  const size_t out_bytes[2] = {span(a->tokens, qrow, qrow, esz), span(a->tokens, krow, krow, esz)};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (overlap(in[i], in_bytes[i], out[j], out_bytes[j]))
        return report_error(ATF_ERR_INVALID_ARG, "%s: an output overlaps an input", who);
  if (overlap(out[0], out_bytes[0], out[1], out_bytes[1]))
    return report_error(ATF_ERR_INVALID_ARG, "%s: the outputs overlap", who);
  p.q = in[0];
  p.k = in[1];
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.q_out = out[0];
  p.k_out = out[1];
  p.q_weight = a->q_weight;
  p.k_weight = a->k_weight;
  p.pos = a->pos;
  p.tokens = a->tokens;
  p.hq = a->heads;
  p.hkv = a->kv_heads;
  p.d = a->d;
  p.pairing = a->pairing;
  p.fp32 = a->dtype == ATF_FP32;
  p.wide = aligned32(p.q_out) && aligned32(p.k_out);
  p.eps = a->eps;
  cudaError_t e = launch_qk_norm_rope(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(ATF_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  return ATF_OK;
}

atf_status atf_paged_append(const atf_paged_append_args* a, void* stream) {
  const char* who = "paged_append";
  if (!a) return report_error(ATF_ERR_INVALID_ARG, "args is NULL");
  if (atf_status st = check_method(a->d, a->theta, 1.0)) return st;
  if (a->pairing != ATF_PAIRS_INTERLEAVED && a->pairing != ATF_PAIRS_ROTATE_HALF)
    return report_error(ATF_ERR_INVALID_ARG, "%s: pairing %d", who, a->pairing);
  if (a->tokens < 0 || a->batch < 0) return report_error(ATF_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (atf_status st = check_heads(who, a->q ? a->heads : a->kv_heads, a->kv_heads)) return st;
  if (atf_status st = check_pool(who, a->page_size, a->num_pages, a->max_pages, a->kv_heads)) return st;
  if (a->kv_heads > 65535) return report_error(ATF_ERR_UNSUPPORTED, "%s: more than 65535 kv heads", who);
  if (!(a->eps >= 0.f) || std::isinf(a->eps)) return report_error(ATF_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
  if (!a->cu && a->tokens != a->batch)
    return report_error(ATF_ERR_INVALID_ARG, "%s: without cu each of the %d sequences has one of the %d tokens", who,
                        a->batch, a->tokens);
  PagedAppendParams p{};
  if (atf_status st = rotary_table(who, a->d, a->theta, a->n_axes, a->pair_axis, &p.rot)) return st;
  if (a->n_axes > 1 && !a->pos) return report_error(ATF_ERR_INVALID_ARG, "%s: several position axes need pos", who);
  if (a->tokens == 0 || a->batch == 0) return ATF_OK;
  if (!a->k || !a->v || !a->k_pages || !a->v_pages || !a->page_table || !a->start || (a->q && !a->q_out))
    return report_error(ATF_ERR_INVALID_ARG, "%s: null pointer", who);
  const long long qrow = static_cast<long long>(a->heads) * a->d, krow = static_cast<long long>(a->kv_heads) * a->d;
  if ((a->q && bad_stride(a->q_stride, qrow, 2)) || bad_stride(a->k_stride, krow, 2) || bad_stride(a->v_stride, krow, 2))
    return report_error(ATF_ERR_INVALID_ARG, "%s: strides must hold the heads and keep 16-byte alignment", who);
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->q_out) || !aligned16(a->k_pages) ||
      !aligned16(a->v_pages) || !aligned16(a->bounds) || !aligned16(a->q_weight) || !aligned16(a->k_weight) ||
      !aligned16(a->pos))
    return report_error(ATF_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  if (!aligned4(a->page_table) || !aligned4(a->start) || !aligned4(a->cu))
    return report_error(ATF_ERR_INVALID_ARG, "%s: int arrays must be 4-byte aligned", who);
  if (a->q) {
    const size_t nout = span(a->tokens, qrow, qrow, 2);
    if (overlap(a->q, span(a->tokens, a->q_stride, qrow, 2), a->q_out, nout) ||
        overlap(a->k, span(a->tokens, a->k_stride, krow, 2), a->q_out, nout) ||
        overlap(a->v, span(a->tokens, a->v_stride, krow, 2), a->q_out, nout))
      return report_error(ATF_ERR_INVALID_ARG, "%s: q_out overlaps an input", who);
  }
  p.err = device_error_word();
  if (!p.err) return report_error(ATF_ERR_CUDA, "no CUDA device / device error word unavailable");
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.q_stride = a->q_stride;
  p.k_stride = a->k_stride;
  p.v_stride = a->v_stride;
  p.q_out = a->q_out;
  p.k_pages = a->k_pages;
  p.v_pages = a->v_pages;
  p.bounds = a->bounds;
  p.q_weight = a->q_weight;
  p.k_weight = a->k_weight;
  p.page_table = a->page_table;
  p.start = a->start;
  p.cu = a->cu;
  p.pos = a->pos;
  p.tokens = a->tokens;
  p.batch = a->batch;
  p.hq = a->q ? a->heads : a->kv_heads;
  p.hkv = a->kv_heads;
  p.d = a->d;
  p.pairing = a->pairing;
  p.page_log2 = page_log2(a->page_size);
  p.max_pages = a->max_pages;
  p.num_pages = static_cast<int>(a->num_pages);
  // a sequence with n > 0 new tokens touches at most (n - 1) / page + 2 pages
  p.items = (p.tokens >> p.page_log2) + 2LL * (p.batch < p.tokens ? p.batch : p.tokens);
  const long long likely = ((p.tokens >> p.page_log2) + static_cast<long long>(p.batch)) * p.hkv;  // (page, kv head) items
  p.threads = likely >= 600 ? 64 : likely >= 148 ? 128 : 256;
  p.wide = aligned32(p.q_out) && aligned32(p.k_pages) && aligned32(p.v_pages);
  if (p.cu && paged_append_blocks(p) > 0x7fffffffLL)
    return report_error(ATF_ERR_UNSUPPORTED, "%s: too many tokens, sequences and heads for one call", who);
  p.eps = a->eps;
  cudaError_t e = launch_paged_append(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(ATF_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  return ATF_OK;
}

size_t atf_paged_decode_workspace_bytes(int batch, int heads, int kv_heads, int d) {
  if (batch <= 0 || heads <= 0 || kv_heads <= 0 || d <= 0) return 0;
  return kMetaBytes + static_cast<size_t>(kPagedCtas) * 2 * 8 * (d + 2) * sizeof(float);
}

atf_status atf_paged_decode(const atf_paged_decode_args* a, void* stream) {
  const char* who = "paged_decode";
  if (!a) return report_error(ATF_ERR_INVALID_ARG, "args is NULL");
  if (atf_status st = check_method(a->d, a->theta, a->alpha)) return st;
  if (a->batch < 0) return report_error(ATF_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (atf_status st = check_heads(who, a->heads, a->kv_heads)) return st;
  if (a->heads / a->kv_heads > 8) return report_error(ATF_ERR_UNSUPPORTED, "%s: at most 8 query heads per kv head", who);
  if (atf_status st = check_pool(who, a->page_size, a->num_pages, a->max_pages, a->kv_heads)) return st;
  if (a->selected && a->n_select < 1) return report_error(ATF_ERR_INVALID_ARG, "%s: n_select %d", who, a->n_select);
  if (a->batch == 0) return ATF_OK;
  if (!a->q || !a->k_pages || !a->v_pages || !a->page_table || !a->kv_len || !a->out)
    return report_error(ATF_ERR_INVALID_ARG, "%s: null pointer", who);
  if (bad_stride(a->q_stride, static_cast<long long>(a->heads) * a->d, 2))
    return report_error(ATF_ERR_INVALID_ARG, "%s: q_stride must hold the heads and keep 16-byte alignment", who);
  if (!aligned16(a->q) || !aligned16(a->k_pages) || !aligned16(a->v_pages) || !aligned16(a->out) || !aligned16(a->workspace))
    return report_error(ATF_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  if (!aligned4(a->page_table) || !aligned4(a->kv_len) || !aligned4(a->selected) || !aligned4(a->lse))
    return report_error(ATF_ERR_INVALID_ARG, "%s: int arrays and lse must be 4-byte aligned", who);
  const size_t need = atf_paged_decode_workspace_bytes(a->batch, a->heads, a->kv_heads, a->d);
  if (!a->workspace || a->workspace_bytes < need)
    return report_error(ATF_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed", who, need);
  PagedDecodeParams p{};
  p.err = device_error_word();
  if (!p.err) return report_error(ATF_ERR_CUDA, "no CUDA device / device error word unavailable");
  p.q = a->q;
  p.q_stride = a->q_stride;
  p.page_table = a->page_table;
  p.kv_len = a->kv_len;
  p.selected = a->selected;
  p.out = a->out;
  p.lse = a->lse;
  p.meta = static_cast<int4*>(a->workspace);
  p.partials = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + kMetaBytes);
  p.sums = reinterpret_cast<float2*>(p.partials + kPagedCtas * 2 * 8 * a->d);
  p.batch = a->batch;
  p.hq = a->heads;
  p.hkv = a->kv_heads;
  p.d = a->d;
  p.page_log2 = page_log2(a->page_size);
  p.max_pages = a->max_pages;
  p.num_pages = static_cast<int>(a->num_pages);
  p.n_sel = a->selected ? a->n_select : 0;
  method_windows(a->d, a->theta, a->alpha, &p.win);
  // keys (64 elements: a chunk of four slots, group of four slots, chunk, page and
  // head): a box is the chunks of up to a tile's slots; values (64 elements, slot,
  // half of the row, page and head): a box is as many rows, half by half; both with
  // the 128-byte swizzle
  const unsigned long long d = a->d, ps = a->page_size;
  const unsigned long long rows = static_cast<unsigned long long>(a->num_pages) * a->kv_heads;
  const unsigned long long kd[4] = {64, ps / 4, d / 16, rows}, ks[3] = {128, ps * 32, ps * d * 2};
  const double most = static_cast<double>(a->selected && a->n_select < a->max_pages ? a->n_select : a->max_pages) * a->page_size;
  p.tile_keys = paged_tile_keys(a->d, most * a->batch * a->kv_heads);
  const unsigned box = a->page_size < p.tile_keys ? a->page_size : p.tile_keys;
  const unsigned int kb[4] = {64, box / 4, static_cast<unsigned>(d / 16), 1};
  const unsigned long long vd[4] = {64, ps, d / 64, rows}, vs[3] = {d * 2, 128, ps * d * 2};
  const unsigned int vb[4] = {64, box, static_cast<unsigned>(d / 64), 1};
  CUtensorMap tk, tv;
  if (atf_status st = tensor_map_4d(&tk, a->k_pages, kd, ks, kb, CU_TENSOR_MAP_SWIZZLE_128B)) return st;
  if (atf_status st = tensor_map_4d(&tv, a->v_pages, vd, vs, vb, CU_TENSOR_MAP_SWIZZLE_128B)) return st;
  cudaError_t e = launch_paged_decode(p, tk, tv, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(ATF_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  return ATF_OK;
}

size_t atf_page_select_workspace_bytes(int batch, int kv_heads, int max_pages) {
  if (batch <= 0 || kv_heads <= 0 || max_pages <= 0) return 0;
  return static_cast<size_t>(batch) * kv_heads * max_pages * sizeof(unsigned long long);
}

atf_status atf_page_select(const atf_page_select_args* a, void* stream) {
  const char* who = "page_select";
  if (!a) return report_error(ATF_ERR_INVALID_ARG, "args is NULL");
  if (atf_status st = check_method(a->d, a->theta, a->alpha)) return st;
  if (a->batch < 0) return report_error(ATF_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (atf_status st = check_heads(who, a->heads, a->kv_heads)) return st;
  if (a->heads / a->kv_heads > 8) return report_error(ATF_ERR_UNSUPPORTED, "%s: at most 8 query heads per kv head", who);
  if (atf_status st = check_pool(who, a->page_size, a->num_pages, a->max_pages, a->kv_heads)) return st;
  if (static_cast<long long>(a->batch) * a->kv_heads > 65535)
    return report_error(ATF_ERR_UNSUPPORTED, "%s: batch * kv_heads above 65535", who);
  if (a->n_select < 1 || a->n_first < 0 || a->n_last < 0 || static_cast<long long>(a->n_first) + a->n_last > a->n_select)
    return report_error(ATF_ERR_INVALID_ARG, "%s: n_select %d must be positive and hold the %d first and %d last pages", who,
                        a->n_select, a->n_first, a->n_last);
  if (a->batch == 0) return ATF_OK;
  if (!a->q || !a->bounds || !a->page_table || !a->kv_len || !a->selected)
    return report_error(ATF_ERR_INVALID_ARG, "%s: null pointer", who);
  if (bad_stride(a->q_stride, static_cast<long long>(a->heads) * a->d, 2))
    return report_error(ATF_ERR_INVALID_ARG, "%s: q_stride must hold the heads and keep 16-byte alignment", who);
  if (!aligned16(a->q) || !aligned16(a->bounds) || !aligned16(a->workspace))
    return report_error(ATF_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  if (!aligned4(a->page_table) || !aligned4(a->kv_len) || !aligned4(a->selected))
    return report_error(ATF_ERR_INVALID_ARG, "%s: int arrays must be 4-byte aligned", who);
  const size_t need = atf_page_select_workspace_bytes(a->batch, a->kv_heads, a->max_pages);
  if (!a->workspace || a->workspace_bytes < need)
    return report_error(ATF_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed", who, need);
  PageSelectParams p{};
  p.err = device_error_word();
  if (!p.err) return report_error(ATF_ERR_CUDA, "no CUDA device / device error word unavailable");
  p.q = a->q;
  p.q_stride = a->q_stride;
  p.bounds = a->bounds;
  p.page_table = a->page_table;
  p.kv_len = a->kv_len;
  p.keys = static_cast<unsigned long long*>(a->workspace);
  p.selected = a->selected;
  p.batch = a->batch;
  p.hq = a->heads;
  p.hkv = a->kv_heads;
  p.d = a->d;
  p.page_log2 = page_log2(a->page_size);
  p.max_pages = a->max_pages;
  p.num_pages = static_cast<int>(a->num_pages);
  p.n_sel = a->n_select;
  p.n_first = a->n_first;
  p.n_last = a->n_last;
  method_windows(a->d, a->theta, a->alpha, &p.win);
  cudaError_t e = launch_page_select(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(ATF_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  return ATF_OK;
}

}  // extern "C"
