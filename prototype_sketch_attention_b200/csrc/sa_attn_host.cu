// C ABI of the multi-head cross attention and of its paged cache: argument checks and
// workspace plans. See include/sa_sketch.h for the contract of every entry point.
#include <cmath>
#include <cstdint>

#include "sa_common.cuh"
#include "sa_internal.h"
#include "sa_sketch.h"

namespace sa {
namespace {

constexpr int kMaxHeads = 1024;

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool on8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
bool on4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int status_of(cudaError_t e) {
  if (e == cudaSuccess) return SA_OK;
  cudaGetLastError();
  return SA_ERR_CUDA;
}

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && bytes >= need;
}

// log2 of a page size, or -1 (powers of two from 8 to 256)
int page_log2(int page_size) {
  for (int l = 3; l <= 8; ++l)
    if (page_size == 1 << l) return l;
  return -1;
}

int check_heads(int H, int Hkv, int d) {
  if (H < 1 || Hkv < 1 || H > kMaxHeads || Hkv > H || H % Hkv != 0) return SA_ERR_INVALID_ARG;
  return d == 64 || d == 128 ? SA_OK : SA_ERR_UNSUPPORTED;
}

int check_cross_sizes(int R, int64_t n_q, int64_t n_kv, int H, int Hkv, int d) {
  if (R < 0 || R > SA_MAX_USERS || n_q < 0 || n_q > INT32_MAX || n_kv < 0 || n_kv > INT32_MAX)
    return SA_ERR_INVALID_ARG;
  const int st = check_heads(H, Hkv, d);
  if (st != SA_OK) return st;
  // the kernels' grids count 128-row tiles of every user and head in 31 bits
  if ((n_q / 128 + R + 1) * H > INT32_MAX || (n_kv / 128 + R + 1) * Hkv > INT32_MAX)
    return SA_ERR_UNSUPPORTED;
  return SA_OK;
}

int check_cross(const CrossArgs& a) {
  const int st = check_cross_sizes(a.R, a.n_q, a.n_kv, a.H, a.Hkv, a.d);
  if (st != SA_OK) return st;
  if (!(a.scale > 0.f) || !std::isfinite(a.scale)) return SA_ERR_INVALID_ARG;
  if (!a.qoff || !a.koff || (a.n_q > 0 && (!a.Q || !a.out || !a.lse)) || (a.n_kv > 0 && (!a.K || !a.V)))
    return SA_ERR_INVALID_ARG;
  if (!on16(a.Q) || !on16(a.K) || !on16(a.V) || !on16(a.out) || !on16(a.rest) || !on16(a.lse) || !on8(a.qoff) ||
      !on8(a.koff))
    return SA_ERR_INVALID_ARG;
  if (a.q_stride < (long long)a.H * a.d || a.k_stride < (long long)a.Hkv * a.d ||
      a.v_stride < (long long)a.Hkv * a.d || a.q_stride % 8 || a.k_stride % 8 || a.v_stride % 8 ||
      a.q_stride > (1LL << 36) || a.k_stride > (1LL << 36) || a.v_stride > (1LL << 36))
    return SA_ERR_INVALID_ARG;
  return SA_OK;
}

}  // namespace
}  // namespace sa

using namespace sa;

extern "C" {

size_t sa_cross_attn_workspace_size(int R, int64_t n_q, int64_t n_kv, int H, int Hkv, int d,
                                    int backward) {
  int sms = 0;
  if (check_cross_sizes(R, n_q, n_kv, H, Hkv, d) != SA_OK || device_sms(&sms) != SA_OK) return 0;
  return cross_plan(R, n_q, n_kv, H, Hkv, d, backward != 0, sms, nullptr);
}

int sa_cross_attn_forward(const void* Q, int64_t q_stride, const int64_t* q_offsets, int R,
                          int64_t n_q, int H, int d, const void* K, int64_t k_stride,
                          const void* V, int64_t v_stride, const int64_t* kv_offsets,
                          int64_t n_kv, int Hkv, const uint8_t* key_mask, float scale, void* out,
                          void* out_rest, float* lse, void* workspace, size_t ws_bytes,
                          void* stream) {
  CrossArgs a = {};
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.qoff = q_offsets;
  a.koff = kv_offsets;
  a.R = R;
  a.H = H;
  a.Hkv = Hkv;
  a.d = d;
  a.n_q = n_q;
  a.n_kv = n_kv;
  a.mask = key_mask;
  a.scale = scale;
  a.out = out;
  a.rest = out_rest;
  a.lse = lse;
  int st = check_cross(a);
  if (st != SA_OK || (st = device_sms(&a.sms)) != SA_OK) return st;
  if (!workspace_ok(workspace, ws_bytes, cross_plan(R, n_q, n_kv, H, Hkv, d, false, a.sms, &a.plan)))
    return SA_ERR_WORKSPACE;
  a.workspace = workspace;
  return status_of(launch_cross_forward(a, static_cast<cudaStream_t>(stream)));
}

int sa_cross_attn_backward(const void* Q, int64_t q_stride, const int64_t* q_offsets, int R,
                           int64_t n_q, int H, int d, const void* K, int64_t k_stride,
                           const void* V, int64_t v_stride, const int64_t* kv_offsets,
                           int64_t n_kv, int Hkv, const uint8_t* key_mask, float scale,
                           const void* out, const void* out_rest, const float* lse,
                           const void* dout, void* dQ, void* dK, void* dV, void* workspace,
                           size_t ws_bytes, void* stream) {
  CrossArgs a = {};
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.qoff = q_offsets;
  a.koff = kv_offsets;
  a.R = R;
  a.H = H;
  a.Hkv = Hkv;
  a.d = d;
  a.n_q = n_q;
  a.n_kv = n_kv;
  a.mask = key_mask;
  a.scale = scale;
  a.out = const_cast<void*>(out);
  a.rest = const_cast<void*>(out_rest);
  a.lse = const_cast<float*>(lse);
  a.dout = dout;
  a.dQ = dQ;
  a.dK = dK;
  a.dV = dV;
  int st = check_cross(a);
  if (st != SA_OK) return st;
  if ((n_q > 0 && (!dout || !dQ)) || (n_kv > 0 && (!dK || !dV)) || !on16(dout) || !on16(dQ) ||
      !on16(dK) || !on16(dV))
    return SA_ERR_INVALID_ARG;
  if ((st = device_sms(&a.sms)) != SA_OK) return st;
  if (!workspace_ok(workspace, ws_bytes, cross_plan(R, n_q, n_kv, H, Hkv, d, true, a.sms, &a.plan)))
    return SA_ERR_WORKSPACE;
  a.workspace = workspace;
  return status_of(launch_cross_backward(a, static_cast<cudaStream_t>(stream)));
}

int sa_page_tables(const int32_t* cached_lens, const int32_t* new_lens, int R, int page_size,
                   const int32_t* free_pages, int64_t n_free, const int64_t* free_used,
                   int32_t* block_table, int max_pages, int64_t n_slots, int64_t* slots,
                   int64_t* new_offsets, int32_t* seq_lens, int64_t* free_used_out,
                   void* workspace, size_t ws_bytes, void* stream) {
  if (R < 0 || R > SA_MAX_USERS || max_pages < 0 || n_free < 0 || n_free > INT32_MAX ||
      n_slots < 0 || n_slots > INT32_MAX)
    return SA_ERR_INVALID_ARG;
  PageTablesArgs a = {};
  if ((a.log2_page = page_log2(page_size)) < 0) return SA_ERR_UNSUPPORTED;
  if (!new_offsets || !free_used_out || (n_free > 0 && !free_pages) || (n_slots > 0 && !slots) ||
      (R > 0 && (!cached_lens || !new_lens || !seq_lens || (max_pages > 0 && !block_table))))
    return SA_ERR_INVALID_ARG;
  if (!on4(cached_lens) || !on4(new_lens) || !on4(free_pages) || !on4(block_table) ||
      !on4(seq_lens) || !on8(free_used) || !on8(slots) || !on8(new_offsets) || !on8(free_used_out))
    return SA_ERR_INVALID_ARG;
  int st = device_sms(&a.sms);
  if (st != SA_OK) return st;
  if (!workspace_ok(workspace, ws_bytes, sizeof(WsHeader))) return SA_ERR_WORKSPACE;
  a.cached = cached_lens;
  a.fresh = new_lens;
  a.R = R;
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.free_used = free_used;
  a.table = block_table;
  a.max_pages = max_pages;
  a.n_slots = n_slots;
  a.slots = slots;
  a.new_offsets = new_offsets;
  a.seq_lens = seq_lens;
  a.free_used_out = free_used_out;
  a.hdr = static_cast<WsHeader*>(workspace);
  a.wide = on16(slots);
  return status_of(launch_page_tables(a, static_cast<cudaStream_t>(stream)));
}

int sa_paged_append(const void* K, int64_t k_stride, const void* V, int64_t v_stride,
                    const int64_t* slots, int64_t n, int Hkv, int d, int format, void* k_cache,
                    void* v_cache, float* k_scales, float* v_scales, int64_t n_pages,
                    int page_size, void* stream) {
  if (n < 0 || n > INT32_MAX || n_pages < 0 || n_pages > INT32_MAX ||
      (format != SA_CODEC_BF16 && format != SA_CODEC_FP8))
    return SA_ERR_INVALID_ARG;
  PagedAppendArgs a = {};
  int st = check_heads(Hkv, Hkv, d);
  if (st != SA_OK) return st;
  if ((a.log2_page = page_log2(page_size)) < 0 || n_pages * Hkv * page_size > INT32_MAX)
    return SA_ERR_UNSUPPORTED;
  a.fp8 = format == SA_CODEC_FP8;
  if ((n > 0 && (!K || !V || !slots)) ||
      (n_pages > 0 && (!k_cache || !v_cache || (a.fp8 && (!k_scales || !v_scales)))))
    return SA_ERR_INVALID_ARG;
  if (!on16(K) || !on16(V) || !on8(slots) || !on16(k_cache) || !on16(v_cache) || !on16(k_scales) ||
      !on16(v_scales))
    return SA_ERR_INVALID_ARG;
  if (k_stride < (long long)Hkv * d || v_stride < (long long)Hkv * d || k_stride % 8 || v_stride % 8)
    return SA_ERR_INVALID_ARG;
  if ((st = device_sms(&a.sms)) != SA_OK) return st;
  a.K = K;
  a.V = V;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slots = slots;
  a.n = n;
  a.n_pages = n_pages;
  a.Hkv = Hkv;
  a.d = d;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  return status_of(launch_paged_append(a, static_cast<cudaStream_t>(stream)));
}

namespace {
int check_paged_sizes(int R, int H, int Hkv, int d) {
  if (R < 0 || R > SA_MAX_USERS) return SA_ERR_INVALID_ARG;
  const int st = check_heads(H, Hkv, d);
  if (st != SA_OK) return st;
  return H / Hkv > 64 || (int64_t)R * H > INT32_MAX ? SA_ERR_UNSUPPORTED : SA_OK;
}
}  // namespace

size_t sa_paged_attn_workspace_size(int R, int H, int Hkv, int d) {
  int sms = 0;
  if (check_paged_sizes(R, H, Hkv, d) != SA_OK || device_sms(&sms) != SA_OK) return 0;
  return paged_attn_plan(R, H, Hkv, d, sms, nullptr);
}

int sa_paged_attn(const void* Q, int64_t q_stride, int R, int H, int d, const void* k_cache,
                  const void* v_cache, const float* k_scales, const float* v_scales, int format,
                  int64_t n_pages, int page_size, int Hkv, const int32_t* block_table,
                  int max_pages, const int32_t* seq_lens, int64_t window, float scale, void* out,
                  float* lse, void* workspace, size_t ws_bytes, void* stream) {
  int st = check_paged_sizes(R, H, Hkv, d);
  if (st != SA_OK) return st;
  if (n_pages < 0 || n_pages > INT32_MAX || max_pages < 0 || window < 0 || !(scale > 0.f) ||
      !std::isfinite(scale) || (format != SA_CODEC_BF16 && format != SA_CODEC_FP8))
    return SA_ERR_INVALID_ARG;
  PagedAttnArgs a = {};
  a.fp8 = format == SA_CODEC_FP8;
  if ((a.log2_page = page_log2(page_size)) < 0 || n_pages * Hkv * page_size > INT32_MAX ||
      (int64_t)max_pages * page_size > INT32_MAX - 256)  // (positions round up to a tile in 31 bits)
    return SA_ERR_UNSUPPORTED;
  if ((R > 0 && (!Q || !out || !seq_lens || (max_pages > 0 && !block_table))) ||
      (n_pages > 0 && (!k_cache || !v_cache || (a.fp8 && (!k_scales || !v_scales)))))
    return SA_ERR_INVALID_ARG;
  if (!on16(Q) || !on16(out) || !on16(lse) || !on16(k_cache) || !on16(v_cache) || !on16(k_scales) ||
      !on16(v_scales) || !on4(block_table) || !on4(seq_lens))
    return SA_ERR_INVALID_ARG;
  if (q_stride < (long long)H * d || q_stride % 8) return SA_ERR_INVALID_ARG;
  if ((st = device_sms(&a.sms)) != SA_OK) return st;
  if (!workspace_ok(workspace, ws_bytes, paged_attn_plan(R, H, Hkv, d, a.sms, &a.plan)))
    return SA_ERR_WORKSPACE;
  a.Q = Q;
  a.q_stride = q_stride;
  a.R = R;
  a.H = H;
  a.Hkv = Hkv;
  a.d = d;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.n_pages = n_pages;
  a.table = block_table;
  a.max_pages = max_pages;
  a.seq_lens = seq_lens;
  a.window = window;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  return status_of(launch_paged_attn(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
