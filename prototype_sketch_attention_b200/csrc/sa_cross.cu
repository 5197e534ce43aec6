// Multi-head cross attention over ragged users: the schedule of tiles, the backward's row
// statistics, workspace plans and launch sequences. The tensor-core kernels are in
// sa_cross_fwd.cu and sa_cross_bwd.cu.
#include <cmath>

#include "sa_common.cuh"
#include "sa_cross.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

using cross::kLog2e;

// Block 0 lists the query tiles (pairs of 128-row tiles: pair_tokens tokens), block 1 the key
// tiles (128 rows). Both check both offset arrays; bad offsets leave no tiles. 1024 threads.
__device__ __forceinline__ void schedule_block(const int64_t* __restrict__ qoff,
                                               const int64_t* __restrict__ koff, int R,
                                               long long n_q, long long n_kv, int pair_tokens,
                                               WsHeader* hdr, cross::Tile* __restrict__ qtiles,
                                               cross::Tile* __restrict__ ktiles) {
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
      hdr->pad[1] = 0;  // the backward's item counter
    }
  }
}

// (lse2, delta = dout . out) of every query row of a user, at [head group][row][head of the group], where
// the backward's tiles find them contiguous. A row without kept keys gets lse2 = +inf: weight 0.
// LANES = d / 8 lanes per row and head, 16 bytes each.
template <int LANES>
__device__ __forceinline__ void stats_rows(const CrossArgs& a, int pg, long long first, long long step,
                                           float2* __restrict__ stats) {
  const long long rows = min((long long)a.qoff[a.R], a.n_q) * a.H;
  const int lane = threadIdx.x & (LANES - 1);
  const long long bound = (rows + 31) / 32 * 32;  // whole warps take part in the shuffles
  for (long long i = first; i < bound; i += step) {
    float s = 0.f;
    if (i < rows) {
      const uint4 x = reinterpret_cast<const uint4*>(a.dout)[i * LANES + lane];
      const uint4 y = reinterpret_cast<const uint4*>(a.out)[i * LANES + lane];
      uint4 r = make_uint4(0, 0, 0, 0);
      if (a.rest) r = reinterpret_cast<const uint4*>(a.rest)[i * LANES + lane];
      const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w}, w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        s = fmaf(__uint_as_float(u[z] << 16), __uint_as_float(v[z] << 16) + __uint_as_float(w[z] << 16), s);
        s = fmaf(__uint_as_float(u[z] & 0xffff0000u),
                 __uint_as_float(v[z] & 0xffff0000u) + __uint_as_float(w[z] & 0xffff0000u), s);
      }
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (i < rows && lane == 0) {
      const long long t = i / a.H;
      const int h = (int)(i - t * a.H), hu = h / pg;
      const float lse = a.lse[i];
      stats[((long long)hu * a.n_q + t) * pg + (h - hu * pg)] =
          make_float2(lse == -INFINITY ? INFINITY : lse * kLog2e, s);
    }
  }
}

// The forward's schedule, one block. An item is a query tile of one head group; its cost in
// half steps is 2 per key tile (1 when the rows fit in one 128-row tile) and a constant for
// its start and end. CTA b starts where the items' costs, in order, reach b / CTAs of their sum,
// rounded to an even key tile. (Boundaries rounded to whole items, with nothing to join, took 6 % less time
// with 8 items a CTA, 1 % less with 16 to 32, and three times as long with one user of 50,000 keys among 160
// of 200: 305 against 105 us at d = 64.)
__global__ void __launch_bounds__(1024)
cross_schedule_kernel(const int64_t* __restrict__ qoff, const int64_t* __restrict__ koff, int R, long long n_q,
                      long long n_kv, int tokens, int groups, int ctas, WsHeader* hdr,
                      cross::Tile* __restrict__ tiles, long long* __restrict__ costs,
                      cross::Start* __restrict__ starts) {
  griddep_launch_dependents();
  __shared__ int first[1025], part[32], keys[1024];
  __shared__ long long before[1024], cpart[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int bad = 0;
  for (int u = tid; u < R; u += 1024)
    if (qoff[u + 1] < qoff[u] || koff[u + 1] < koff[u]) bad = 1;
  if (tid == 0 && (qoff[0] != 0 || koff[0] != 0 || qoff[R] > n_q || koff[R] > n_kv)) bad = 1;
  bad = __syncthreads_or(bad);
  auto cost_of = [](int nkt, bool two) { return two ? 2 * nkt + 4 : nkt + 3; };
  int base = 0;
  long long cost = 0;
  if (!bad) {
    for (int u0 = 0; u0 < R; u0 += 1024) {
      const int u = u0 + tid, nu = min(1024, R - u0);
      int n = 0, nkt = 0;
      long long c = 0;
      if (u < R) {
        const int lq = (int)(qoff[u + 1] - qoff[u]);
        n = (lq + 2 * tokens - 1) / (2 * tokens);
        nkt = (int)((koff[u + 1] - koff[u] + 127) / 128);
        if (n > 0) c = (long long)(n - 1) * cost_of(nkt, true) + cost_of(nkt, lq - (n - 1) * 2 * tokens > tokens);
      }
      int x = n;  // inclusive prefix sums over the block
      long long y = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, x, o);
        const long long w = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
          x += v;
          y += w;
        }
      }
      if (lane == 31) {
        part[warp] = x;
        cpart[warp] = y;
      }
      __syncthreads();
      if (warp == 0) {
        int v = part[lane];
        long long w = cpart[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v1 = __shfl_up_sync(0xffffffffu, v, o);
          const long long w1 = __shfl_up_sync(0xffffffffu, w, o);
          if (lane >= o) {
            v += v1;
            w += w1;
          }
        }
        part[lane] = v;
        cpart[lane] = w;
      }
      __syncthreads();
      first[tid + 1] = x + (warp ? part[warp - 1] : 0);
      before[tid] = cost + y - c + (warp ? cpart[warp - 1] : 0);
      keys[tid] = nkt;
      if (tid == 0) first[0] = 0;
      __syncthreads();
      const int total = first[nu];
      for (int i = tid; i < total; i += 1024) {
        int lo = 0, hi = nu;  // first[lo] <= i < first[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (first[mid] <= i) lo = mid; else hi = mid;
        }
        const int k = i - first[lo];
        tiles[base + i] = cross::Tile{u0 + lo, k};
        costs[base + i] = before[lo] + (long long)k * cost_of(keys[lo], true);
      }
      base += total;
      cost += cpart[31];
      __syncthreads();
    }
  }
  if (tid == 0) {
    hdr->total_tiles = base;
    hdr->status = bad ? SA_ERR_BAD_OFFSETS : SA_OK;
    costs[base] = cost;
    starts[0] = cross::Start{0, 0, 0, 0};
    starts[ctas] = cross::Start{base, 0, 0, 0};
  }
  __syncthreads();
  const long long all = cost * groups;
  for (int b = tid; b < ctas && base > 0; b += 1024) {
    if (b == 0) continue;
    const long long at = all * b / ctas;
    int lo = 0, hi = base;  // the tile whose items hold boundary b
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (costs[mid] * groups <= at) lo = mid; else hi = mid;
    }
    const int c = (int)(costs[lo + 1] - costs[lo]);
    const cross::Tile tl = tiles[lo];
    const int nkt = (int)((koff[tl.user + 1] - koff[tl.user] + 127) / 128);
    const bool two = qoff[tl.user + 1] - qoff[tl.user] - (long long)tl.index * 2 * tokens > tokens;
    const long long in = at - costs[lo] * groups;
    cross::Start s{lo, (int)(in / c), (int)(in % c), 0};
    s.key = max(0, two ? (s.key - 4) / 2 : s.key - 3);
    s.key = (s.key + 1) / 2 * 2;
    if (s.key > nkt - 2) {  // the next item
      s.key = 0;
      if (++s.group == groups) {
        s.group = 0;
        ++s.tile;
      }
    }
    starts[b] = s;
  }
}

// The backward's: blocks 0 and 1 the schedule, the others lse2 and delta.
__global__ void __launch_bounds__(1024) cross_prep_kernel(CrossArgs a, int pg, WsHeader* hdr,
                                                          cross::Tile* qtiles, cross::Tile* ktiles,
                                                          float2* stats) {
  griddep_launch_dependents();
  if (blockIdx.x < 2) {
    schedule_block(a.qoff, a.koff, a.R, a.n_q, a.n_kv, 256 / pg, hdr, qtiles, ktiles);
    return;
  }
  const int lanes = a.d / 8;
  const long long first = ((blockIdx.x - 2) * 1024LL + threadIdx.x) / lanes;
  const long long step = (gridDim.x - 2) * (1024LL / lanes);
  if (a.d == 64) stats_rows<8>(a, pg, first, step, stats);
  else stats_rows<16>(a, pg, first, step, stats);
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
  // With fewer CTAs than SMs (about one per user and head group, or per full tile), the keys of the
  // backward's dQ items are split so that the SMs fill up, down to four key tiles a split. Measured at
  // d = 128, by the rule and with one split: a user's 40 queries, 8 heads over 2, 10K keys: 31 and 100 us; 1
  // query, 30K keys: 47 and 283; 4 users x 40 queries, 5K keys: 43 and 66; 8 users, 4 heads over 4, 3K
  // keys: 53 and 65; 2 users x 300 queries, 8 over 8, 2K keys: 44 and 41.
  const long long full = (n_q + pair - 1) / pair;
  const long long ctas = (full > some ? full : some) * (H / g.pg);
  long long s = ctas > 0 ? sms / ctas : 1;
  const long long most = R > 0 ? n_kv / R / 512 : 1;
  if (s > most) s = most;
  g.splits = s < 1 ? 1 : (int)s;
  g.ctas = sms;
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
    q.stats = take((size_t)n_q * H * sizeof(float2));
    if (g.splits > 1) q.part_o = take((size_t)g.splits * n_q * H * d * sizeof(float));
  } else {
    q.costs = take((size_t)(g.pair_tiles + 1) * sizeof(long long));
    q.starts = take((size_t)(g.ctas + 1) * sizeof(cross::Start));
    q.joins = take((size_t)g.ctas * (sizeof(cross::JoinItem) + sizeof(int)));
    q.part_o = take((size_t)2 * g.ctas * 256 * d * sizeof(float));
    q.part_lse = take((size_t)2 * g.ctas * 256 * sizeof(float));
  }
  q.total = o;
  if (p) *p = q;
  return q.total;
}

cudaError_t launch_cross_forward(const CrossArgs& a, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const cross::CrossGeo g = geometry(a.R, a.n_q, a.n_kv, a.H, a.Hkv, a.sms);
  cross_schedule_kernel<<<1, 1024, 0, s>>>(
      a.qoff, a.koff, a.R, a.n_q, a.n_kv, 128 / g.pg, a.H / g.pg, g.ctas,
      reinterpret_cast<WsHeader*>(ws + a.plan.hdr), reinterpret_cast<cross::Tile*>(ws + a.plan.qtiles),
      reinterpret_cast<long long*>(ws + a.plan.costs), reinterpret_cast<cross::Start*>(ws + a.plan.starts));
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || g.pair_tiles == 0) return e;
  CrossArgs b = a;
  if (b.n_kv == 0) b.K = b.V = b.Q;  // nothing is read through their tensor maps
  return cross::launch_fwd(b, g, s);
}

cudaError_t launch_cross_backward(const CrossArgs& a, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const cross::CrossGeo g = geometry(a.R, a.n_q, a.n_kv, a.H, a.Hkv, a.sms);
  long long grid = 2 + (a.n_q * a.H * (a.d / 8) + 1023) / 1024;
  if (grid > 4LL * a.sms) grid = 4LL * a.sms;
  cross_prep_kernel<<<(unsigned)grid, 1024, 0, s>>>(
      a, g.pg, reinterpret_cast<WsHeader*>(ws + a.plan.hdr),
      reinterpret_cast<cross::Tile*>(ws + a.plan.qtiles),
      reinterpret_cast<cross::Tile*>(ws + a.plan.ktiles),
      reinterpret_cast<float2*>(ws + a.plan.stats));
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  CrossArgs b = a;
  if (b.n_kv == 0) b.K = b.V = b.Q;  // nothing is read through the empty side's tensor maps
  if (b.n_q == 0) b.Q = b.dout = b.K;
  if (a.n_kv == 0 && a.n_q == 0) return cudaSuccess;
  return cross::launch_bwd(b, g, s);
}

}  // namespace sa
