// Multi-head cross attention over ragged users, forward and backward: the plain kernels.
// One warp per output row, every sum in fp32, one pass over the keys (or queries) with the
// running maximum and sum of the softmax. Bound by the warps' shuffles.
#include <cmath>

#include "sa_common.cuh"
#include "sa_cross.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

using cross::kLog2e;

// Block 0 lists the query tiles (pairs of 128-row tiles: pair_tokens tokens), block 1 the key
// tiles (128 rows). Both check both offset arrays; bad offsets leave no tiles.
__global__ void __launch_bounds__(1024) cross_schedule_kernel(const int64_t* __restrict__ qoff,
                                                              const int64_t* __restrict__ koff,
                                                              int R, long long n_q, long long n_kv,
                                                              int pair_tokens, WsHeader* hdr,
                                                              cross::Tile* __restrict__ qtiles,
                                                              cross::Tile* __restrict__ ktiles) {
  griddep_launch_dependents();
  __shared__ int first[1025], part[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool keys = blockIdx.x == 1;
  const int64_t* off = keys ? koff : qoff;
  cross::Tile* tiles = keys ? ktiles : qtiles;
  const int per = keys ? 128 : pair_tokens;
  int bad = 0;
  for (int u = tid; u < R; u += 1024)
    if (qoff[u + 1] < qoff[u] || koff[u + 1] < koff[u]) bad = 1;
  if (tid == 0 && (qoff[0] != 0 || koff[0] != 0 || qoff[R] > n_q || koff[R] > n_kv)) bad = 1;
  bad = __syncthreads_or(bad);
  int base = 0;
  if (!bad) {
    for (int u0 = 0; u0 < R; u0 += 1024) {
      const int u = u0 + tid, nu = min(1024, R - u0);
      const int n = u < R ? (int)((off[u + 1] - off[u] + per - 1) / per) : 0;
      int x = n;  // inclusive prefix sum over the block
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) part[warp] = x;
      __syncthreads();
      if (warp == 0) {
        int y = part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int z = __shfl_up_sync(0xffffffffu, y, o);
          if (lane >= o) y += z;
        }
        part[lane] = y;
      }
      __syncthreads();
      x += warp ? part[warp - 1] : 0;
      first[tid + 1] = x;
      if (tid == 0) first[0] = 0;
      __syncthreads();
      const int total = first[nu];
      for (int i = tid; i < total; i += 1024) {
        int lo = 0, hi = nu;  // first[lo] <= i < first[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (first[mid] <= i) lo = mid; else hi = mid;
        }
        tiles[base + i] = cross::Tile{u0 + lo, i - first[lo]};
      }
      base += total;
      __syncthreads();
    }
  }
  if (tid == 0) {
    if (keys) {
      hdr->pad[0] = base;
    } else {
      hdr->total_tiles = base;
      hdr->status = bad ? SA_ERR_BAD_OFFSETS : SA_OK;
    }
  }
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

namespace {

cross::CrossGeo geometry(int R, long long n_q, long long n_kv, int H, int Hkv, int sms) {
  cross::CrossGeo g;
  const int G = H / Hkv;
  g.pg = G & -G;
  if (g.pg > 128) g.pg = 128;
  const long long pair = 256 / g.pg, some = R < n_q ? R : n_q;
  g.pair_tiles = n_q / pair + some;
  g.key_tiles = n_kv / 128 + (R < n_kv ? R : n_kv);
  // With fewer CTAs than SMs (about one per user and head group, or per full tile), the
  // keys are split so that the SMs fill up, down to four key tiles a split.
  const long long full = (n_q + pair - 1) / pair;
  const long long ctas = (full > some ? full : some) * (H / g.pg);
  long long s = ctas > 0 ? sms / ctas : 1;
  const long long most = R > 0 ? n_kv / R / 512 : 1;
  if (s > most) s = most;
  g.splits = s < 1 ? 1 : (int)s;
  return g;
}

}  // namespace

bool cross::tmap_heads(CUtensorMap* m, const void* base, long long n, int heads, int d,
                       long long stride, int box_heads, int box_rows) {
  auto fn = tmap_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)(n > 0 ? n : 1)};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t cross_plan(int R, long long n_q, long long n_kv, int H, int Hkv, int d, bool backward,
                  int sms, CrossPlan* p) {
  const cross::CrossGeo g = geometry(R, n_q, n_kv, H, Hkv, sms);
  CrossPlan q;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  q.hdr = take(sizeof(WsHeader));
  q.qtiles = take((size_t)g.pair_tiles * sizeof(cross::Tile));
  q.ktiles = take((size_t)g.key_tiles * sizeof(cross::Tile));
  if (backward) {
    q.delta = take((size_t)n_q * H * sizeof(float));
  } else if (g.splits > 1) {
    q.part_o = take((size_t)g.splits * n_q * H * d * sizeof(float));
    q.part_lse = take((size_t)g.splits * n_q * H * sizeof(float));
  }
  q.total = o;
  if (p) *p = q;
  return q.total;
}

namespace {
cudaError_t launch_schedule(const CrossArgs& a, const cross::CrossGeo& g, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  cross_schedule_kernel<<<2, 1024, 0, s>>>(
      a.qoff, a.koff, a.R, a.n_q, a.n_kv, 256 / g.pg, reinterpret_cast<WsHeader*>(ws + a.plan.hdr),
      reinterpret_cast<cross::Tile*>(ws + a.plan.qtiles),
      reinterpret_cast<cross::Tile*>(ws + a.plan.ktiles));
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_cross_forward(const CrossArgs& a, cudaStream_t s) {
  CrossArgs b = a;
  if (b.n_kv == 0) b.K = b.V = b.Q;  // nothing is read through their tensor maps
  const cross::CrossGeo g = geometry(a.R, a.n_q, a.n_kv, a.H, a.Hkv, a.sms);
  const cudaError_t e = launch_schedule(a, g, s);
  return e != cudaSuccess || g.pair_tiles == 0 ? e : cross::launch_fwd(b, g, s);
}

cudaError_t launch_cross_backward(const CrossArgs& a, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  WsHeader* hdr = reinterpret_cast<WsHeader*>(ws + a.plan.hdr);
  float* delta = reinterpret_cast<float*>(ws + a.plan.delta);
  const cross::CrossGeo g = geometry(a.R, a.n_q, a.n_kv, a.H, a.Hkv, a.sms);
  const cudaError_t e = launch_schedule(a, g, s);
  if (e != cudaSuccess) return e;
  return a.d == 64 ? backward_t<2>(a, hdr, delta, s) : backward_t<4>(a, hdr, delta, s);
}

}  // namespace sa
