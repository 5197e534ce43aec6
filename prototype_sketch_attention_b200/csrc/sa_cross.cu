// Multi-head cross attention over ragged users, forward and backward: the plain kernels.
// One warp per output row, every sum in fp32, one pass over the keys (or queries) with the
// running maximum and sum of the softmax. Bound by the warps' shuffles.
#include <cmath>

#include "sa_common.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__global__ void cross_check_kernel(const int64_t* qoff, const int64_t* koff, int R, long long n_q,
                                   long long n_kv, WsHeader* hdr) {
  int bad = 0;
  for (int u = threadIdx.x; u < R; u += blockDim.x)
    if (qoff[u + 1] < qoff[u] || koff[u + 1] < koff[u]) bad = 1;
  if (threadIdx.x == 0 && (qoff[0] != 0 || koff[0] != 0 || qoff[R] > n_q || koff[R] > n_kv)) bad = 1;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) hdr->status = bad ? SA_ERR_BAD_OFFSETS : 0;
}

// the user whose rows [off[u], off[u + 1]) hold row t, or -1
__device__ __forceinline__ int user_of_row(const int64_t* off, int R, long long t) {
  if (t >= off[R]) return -1;
  int lo = 0, hi = R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

template <int N>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, int lane, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __bfloat162float(p[lane + 32 * i]);
}

template <int N>
__device__ __forceinline__ float dot_row(const float (&a)[N], const float (&b)[N]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <int N>
__global__ void __launch_bounds__(128) cross_fwd_kernel(CrossArgs a, const WsHeader* hdr) {
  if (read_status(&hdr->status) != 0) return;
  constexpr int D = 32 * N;
  const int lane = threadIdx.x & 31;
  const long long w = blockIdx.x * 4LL + (threadIdx.x >> 5);
  const long long t = w / a.H;
  const int h = (int)(w % a.H), hk = h / (a.H / a.Hkv);
  if (t >= a.n_q) return;
  const int u = user_of_row(a.qoff, a.R, t);
  if (u < 0) return;
  float q[N], o[N], k[N];
  load_row<N>((const __nv_bfloat16*)a.Q + t * a.q_stride + h * D, lane, q);
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (long long j = a.koff[u]; j < a.koff[u + 1]; ++j) {
    if (a.mask && !a.mask[j]) continue;
    load_row<N>((const __nv_bfloat16*)a.K + j * a.k_stride + hk * D, lane, k);
    const float z = dot_row<N>(q, k) * a.scale * kLog2e;
    const float mn = fmaxf(m, z), f = ex2_approx(m - mn), p = ex2_approx(z - mn);
    load_row<N>((const __nv_bfloat16*)a.V + j * a.v_stride + hk * D, lane, k);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * f + p * k[i];
    l = l * f + p;
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* out = (__nv_bfloat16*)a.out + (t * a.H + h) * D;
#pragma unroll
  for (int i = 0; i < N; ++i) out[lane + 32 * i] = __float2bfloat16(o[i] * inv);
  if (lane == 0) a.lse[t * a.H + h] = l > 0.f ? (m + lg2_approx(l)) * kLn2 : -INFINITY;
}

// dQ of one (row, head), and delta = dout . out
template <int N>
__global__ void __launch_bounds__(128) cross_dq_kernel(CrossArgs a, const WsHeader* hdr, float* delta) {
  if (read_status(&hdr->status) != 0) return;
  constexpr int D = 32 * N;
  const int lane = threadIdx.x & 31;
  const long long w = blockIdx.x * 4LL + (threadIdx.x >> 5);
  const long long t = w / a.H;
  const int h = (int)(w % a.H), hk = h / (a.H / a.Hkv);
  if (t >= a.n_q) return;
  const int u = user_of_row(a.qoff, a.R, t);
  if (u < 0) return;
  float q[N], g[N], dq[N], k[N], v[N];
  load_row<N>((const __nv_bfloat16*)a.Q + t * a.q_stride + h * D, lane, q);
  load_row<N>((const __nv_bfloat16*)a.dout + (t * a.H + h) * D, lane, g);
  load_row<N>((const __nv_bfloat16*)a.out + (t * a.H + h) * D, lane, k);
  const float dl = dot_row<N>(g, k), lse = a.lse[t * a.H + h];
  if (lane == 0) delta[t * a.H + h] = dl;
#pragma unroll
  for (int i = 0; i < N; ++i) dq[i] = 0.f;
  for (long long j = a.koff[u]; j < a.koff[u + 1]; ++j) {
    if (a.mask && !a.mask[j]) continue;
    load_row<N>((const __nv_bfloat16*)a.K + j * a.k_stride + hk * D, lane, k);
    load_row<N>((const __nv_bfloat16*)a.V + j * a.v_stride + hk * D, lane, v);
    const float p = ex2_approx((dot_row<N>(q, k) * a.scale - lse) * kLog2e);
    const float ds = p * (dot_row<N>(g, v) - dl) * a.scale;
#pragma unroll
    for (int i = 0; i < N; ++i) dq[i] = fmaf(ds, k[i], dq[i]);
  }
  __nv_bfloat16* out = (__nv_bfloat16*)a.dQ + (t * a.H + h) * D;
#pragma unroll
  for (int i = 0; i < N; ++i) out[lane + 32 * i] = __float2bfloat16(dq[i]);
}

// dK and dV of one (key row, key head): over the user's query rows and the heads that share it
template <int N>
__global__ void __launch_bounds__(128) cross_dkv_kernel(CrossArgs a, const WsHeader* hdr,
                                                        const float* delta) {
  if (read_status(&hdr->status) != 0) return;
  constexpr int D = 32 * N;
  const int lane = threadIdx.x & 31;
  const long long w = blockIdx.x * 4LL + (threadIdx.x >> 5);
  const long long j = w / a.Hkv;
  const int hk = (int)(w % a.Hkv), G = a.H / a.Hkv;
  if (j >= a.n_kv) return;
  const int u = user_of_row(a.koff, a.R, j);
  if (u < 0) return;
  float q[N], g[N], dk[N], dv[N], k[N], v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dk[i] = dv[i] = 0.f;
  if (!a.mask || a.mask[j]) {
    load_row<N>((const __nv_bfloat16*)a.K + j * a.k_stride + hk * D, lane, k);
    load_row<N>((const __nv_bfloat16*)a.V + j * a.v_stride + hk * D, lane, v);
    for (long long t = a.qoff[u]; t < a.qoff[u + 1]; ++t) {
      for (int h = hk * G; h < (hk + 1) * G; ++h) {
        load_row<N>((const __nv_bfloat16*)a.Q + t * a.q_stride + h * D, lane, q);
        load_row<N>((const __nv_bfloat16*)a.dout + (t * a.H + h) * D, lane, g);
        const float p = ex2_approx((dot_row<N>(q, k) * a.scale - a.lse[t * a.H + h]) * kLog2e);
        const float ds = p * (dot_row<N>(g, v) - delta[t * a.H + h]) * a.scale;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dk[i] = fmaf(ds, q[i], dk[i]);
          dv[i] = fmaf(p, g[i], dv[i]);
        }
      }
    }
  }
  const long long at = (j * a.Hkv + hk) * D;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    ((__nv_bfloat16*)a.dK)[at + lane + 32 * i] = __float2bfloat16(dk[i]);
    ((__nv_bfloat16*)a.dV)[at + lane + 32 * i] = __float2bfloat16(dv[i]);
  }
}

template <int N>
cudaError_t backward_t(const CrossArgs& a, WsHeader* hdr, float* delta, cudaStream_t s) {
  const long long nq = (a.n_q * a.H + 3) / 4, nk = (a.n_kv * a.Hkv + 3) / 4;
  if (nq > 0) cross_dq_kernel<N><<<(unsigned)nq, 128, 0, s>>>(a, hdr, delta);
  if (nk > 0) cross_dkv_kernel<N><<<(unsigned)nk, 128, 0, s>>>(a, hdr, delta);
  return cudaGetLastError();
}

}  // namespace

size_t cross_plan(int R, long long n_q, long long n_kv, int H, int Hkv, int d, bool backward,
                  int sms, CrossPlan* p) {
  CrossPlan q;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  q.hdr = take(sizeof(WsHeader));
  if (backward) q.delta = take((size_t)n_q * H * sizeof(float));
  q.total = o;
  if (p) *p = q;
  return q.total;
}

cudaError_t launch_cross_forward(const CrossArgs& a, cudaStream_t s) {
  WsHeader* hdr = reinterpret_cast<WsHeader*>(static_cast<uint8_t*>(a.workspace) + a.plan.hdr);
  cross_check_kernel<<<1, 256, 0, s>>>(a.qoff, a.koff, a.R, a.n_q, a.n_kv, hdr);
  const long long n = (a.n_q * a.H + 3) / 4;
  if (n > 0) {
    if (a.d == 64) cross_fwd_kernel<2><<<(unsigned)n, 128, 0, s>>>(a, hdr);
    else cross_fwd_kernel<4><<<(unsigned)n, 128, 0, s>>>(a, hdr);
  }
  return cudaGetLastError();
}

cudaError_t launch_cross_backward(const CrossArgs& a, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws + a.plan.hdr);
  float* delta = reinterpret_cast<float*>(ws + a.plan.delta);
  cross_check_kernel<<<1, 256, 0, s>>>(a.qoff, a.koff, a.R, a.n_q, a.n_kv, hdr);
  return a.d == 64 ? backward_t<2>(a, hdr, delta, s) : backward_t<4>(a, hdr, delta, s);
}

}  // namespace sa
