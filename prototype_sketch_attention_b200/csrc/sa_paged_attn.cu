// Attention of one new token per request over the paged cache: the plain kernel. One warp
// per (request, head), one pass over the positions with the softmax's running maximum and sum.
#include <cuda_fp8.h>

#include <cmath>

#include "sa_common.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__global__ void paged_clear_kernel(WsHeader* hdr) { hdr->status = 0; }

template <int N, bool FP8>
__device__ __forceinline__ void cache_row(const void* cache, const float* scales, long long row,
                                          int lane, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const long long at = row * (32 * N) + lane + 32 * i;
    if (FP8) v[i] = float(static_cast<const __nv_fp8_e4m3*>(cache)[at]) * scales[row];
    else v[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(cache)[at]);
  }
}

template <int N, bool FP8>
__global__ void __launch_bounds__(128) paged_attn_kernel(PagedAttnArgs a, WsHeader* hdr) {
  constexpr int D = 32 * N;
  const int lane = threadIdx.x & 31;
  const long long w = blockIdx.x * 4LL + (threadIdx.x >> 5);
  const int r = (int)(w / a.H), h = (int)(w % a.H), hk = h / (a.H / a.Hkv);
  if (r >= a.R) return;
  long long len = a.seq_lens[r];
  if (len < 0 || len > ((long long)a.max_pages << a.log2_page)) {
    latch_status(&hdr->status, SA_ERR_BAD_OFFSETS);
    len = 0;
  }
  float q[N], o[N], k[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = __bfloat162float(((const __nv_bfloat16*)a.Q)[r * a.q_stride + h * D + lane + 32 * i]);
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (long long p = a.window > 0 && len > a.window ? len - a.window : 0; p < len; ++p) {
    const long long pg = a.table[(long long)r * a.max_pages + (p >> a.log2_page)];
    if (pg < 0 || pg >= a.n_pages) {
      latch_status(&hdr->status, SA_ERR_BAD_PAGES);
      continue;
    }
    const long long row = ((pg * a.Hkv + hk) << a.log2_page) + (p & ((1 << a.log2_page) - 1));
    cache_row<N, FP8>(a.k_cache, a.k_scales, row, lane, k);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) z = fmaf(q[i], k[i], z);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
    z *= a.scale * kLog2e;
    const float mn = fmaxf(m, z), f = ex2_approx(m - mn), e = ex2_approx(z - mn);
    cache_row<N, FP8>(a.v_cache, a.v_scales, row, lane, k);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * f + e * k[i];
    l = l * f + e;
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    ((__nv_bfloat16*)a.out)[((long long)r * a.H + h) * D + lane + 32 * i] = __float2bfloat16(o[i] * inv);
  if (lane == 0 && a.lse)
    a.lse[(long long)r * a.H + h] = l > 0.f ? (m + lg2_approx(l)) * kLn2 : -INFINITY;
}

}  // namespace

size_t paged_attn_plan(int R, int H, int Hkv, int d, int sms, PagedAttnPlan* p) {
  PagedAttnPlan q;
  q.total = sizeof(WsHeader);
  if (p) *p = q;
  return q.total;
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t s) {
  WsHeader* hdr = static_cast<WsHeader*>(a.workspace);
  paged_clear_kernel<<<1, 1, 0, s>>>(hdr);
  const long long n = ((long long)a.R * a.H + 3) / 4;
  if (n > 0) {
    if (a.d == 64 && a.fp8) paged_attn_kernel<2, true><<<(unsigned)n, 128, 0, s>>>(a, hdr);
    else if (a.d == 64) paged_attn_kernel<2, false><<<(unsigned)n, 128, 0, s>>>(a, hdr);
    else if (a.fp8) paged_attn_kernel<4, true><<<(unsigned)n, 128, 0, s>>>(a, hdr);
    else paged_attn_kernel<4, false><<<(unsigned)n, 128, 0, s>>>(a, hdr);
  }
  return cudaGetLastError();
}

}  // namespace sa
