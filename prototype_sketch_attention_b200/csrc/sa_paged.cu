// The paged key-value cache: block tables and slot maps from request lengths, and the
// append of new rows (bf16, or FP8 E4M3 with one scale per row).
#include <cuda_fp8.h>

#include "sa_common.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

constexpr float kE4m3Max = 448.0f;

constexpr int kUsers = 512;  // requests per chunk, one a thread

// Exclusive prefix sums over the block of two counts at once, and their totals.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long (&part)[2][kUsers / 32],
                                            long long& total_a, long long& total_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long a0 = a, b0 = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  __syncthreads();  // the last use of `part`
  if (lane == 31) {
    part[0][warp] = a;
    part[1][warp] = b;
  }
  __syncthreads();
  long long x = part[0][lane & 15], y = part[1][lane & 15];  // every warp sums the warps' totals
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, o, 16), v = __shfl_up_sync(0xffffffffu, y, o, 16);
    if ((lane & 15) >= o) {
      x += u;
      y += v;
    }
  }
  total_a = __shfl_sync(0xffffffffu, x, 15);
  total_b = __shfl_sync(0xffffffffu, y, 15);
  const long long ba = __shfl_sync(0xffffffffu, x, (warp + 15) & 15), bb = __shfl_sync(0xffffffffu, y, (warp + 15) & 15);
  a += (warp ? ba : 0) - a0;
  b += (warp ? bb : 0) - b0;
}

// One request's counts; bad: bit 0 lengths, bit 1 pages.
struct Request {
  int cached, fresh, have, need;  // positions held and new; pages held and to be taken
  __device__ void load(const PageTablesArgs& a, int r, int* bad) {
    cached = fresh = have = need = 0;
    if (r >= a.R) return;
    const int c = a.cached[r], n = a.fresh[r];
    const long long end = (long long)c + n;
    if (c < 0 || n < 0 || end > 0x7fffffffLL) {
      *bad |= 1;
      return;
    }
    const int ps = 1 << a.log2_page;
    have = (int)(((long long)c + ps - 1) >> a.log2_page);
    const int want = (int)((end + ps - 1) >> a.log2_page);
    if (want > a.max_pages) *bad |= 2;
    cached = c;
    fresh = n;
    need = want - have;
  }
};

// One launch. A verdict over all requests is needed before anything is written, so every block
// adds all of them up (two 4-byte reads a request), then walks them 512 at a time with
// their prefix sums in shared memory and writes its own share [s0, s1) of the slots, V a thread:
// one search for the request, then a walk; the thread of a new page's first position writes its
// table entry. V = 8 when there are many slots (bound: 8 bytes written a slot): a warp whose 256
// slots are one request's loads their ids all at once and keeps the request for its next slots. Two
// blocks a multiprocessor, all resident at once: 300 requests with 6.5 M slots in 18.3 us (26.0 with one
// block resident and four waves of them, 24.3 with two and the walk alone; a plain fill of the same
// bytes takes 8.5, and the sums before the first write 3). V = 1 for few slots (bound: the chain of
// loads, 3.6 us for 300 requests of one token). Block 0 also writes offsets and lengths.
template <int V>
__global__ void __launch_bounds__(kUsers, 2) page_tables_kernel(PageTablesArgs a) {
  __shared__ long long part[2][kUsers / 32];
  __shared__ int off[kUsers + 1], pg[kUsers], held[kUsers];  // first slot, free entry; positions held
  const int tid = threadIdx.x, ps = 1 << a.log2_page;
  const long long used = a.free_used ? *a.free_used : 0;
  const bool lead = blockIdx.x == 0;
  int bad = 0;
  Request q;
  q.load(a, tid, &bad);
  long long it = q.fresh, ip = q.need, tt, tp;
  if (a.R > kUsers) {
    Request x;
    for (int r = tid + kUsers; r < a.R; r += kUsers) {
      x.load(a, r, &bad);
      it += x.fresh;
      ip += x.need;
    }
  }
  block_scan2(it, ip, part, tt, tp);
  if (tt > a.n_slots) bad |= 1;
  if (used < 0 || used + tp > a.n_free) bad |= 2;
  const int bad1 = __syncthreads_or(bad & 1), bad2 = __syncthreads_or(bad & 2);
  const bool stop = bad1 || bad2;
  // slots, entries of the free list and positions are below 2^31
  const long long per = ((a.n_slots + gridDim.x - 1) / gridDim.x + 32 * V - 1) / (32 * V) * (32 * V);
  const int s0 = (int)min(a.n_slots, blockIdx.x * per), s1 = (int)min(a.n_slots, s0 + per);
  if (lead && tid == 0) {
    a.hdr->status = bad1 ? SA_ERR_BAD_OFFSETS : bad2 ? SA_ERR_BAD_PAGES : SA_OK;
    *a.free_used_out = stop ? used : used + tp;
    a.new_offsets[a.R] = stop ? 0 : tt;
  }
  for (long long i = max((long long)s0, stop ? 0 : tt) + tid; i < s1; i += kUsers) a.slots[i] = -1;
  if (stop) {
    if (lead)
      for (int r = tid; r < a.R; r += kUsers) {
        a.new_offsets[r] = 0;
        a.seq_lens[r] = a.cached[r];
      }
    return;
  }
  long long base_t = 0, base_p = used;
  for (int r0 = 0; r0 < a.R; r0 += kUsers) {
    const int nu = min(kUsers, a.R - r0);
    long long ct = tt, cp = tp;
    if (r0 > 0) q.load(a, r0 + tid, &bad);
    if (a.R > kUsers) {  // else the verdict's sums are this chunk's
      it = q.fresh;
      ip = q.need;
      block_scan2(it, ip, part, ct, cp);
    }
    if (tid < nu) {
      off[tid] = (int)(base_t + it);
      pg[tid] = (int)(base_p + ip);
      held[tid] = q.cached;
      if (lead) {
        a.new_offsets[r0 + tid] = base_t + it;
        a.seq_lens[r0 + tid] = q.cached + q.fresh;
      }
    }
    if (tid == 0) off[nu] = (int)(base_t + ct);
    __syncthreads();
    // A warp has 32 V slots at a time: lane l the pairs (V > 1) at 2 l + 64 k, so that a store
    // instruction covers 512 contiguous bytes
    constexpr int P = V > 1 ? 2 : 1;
    const int b0 = (int)base_t, e1 = (int)min((long long)s1, base_t + ct), lane = tid & 31;
    int last = 0;  // the request of the warp's last slots
    for (long long x = max(s0, b0) / (32 * V) * (32 * V) + 32LL * V * (tid >> 5); x < e1; x += V * kUsers) {
      auto within = [&]() {  // the warp's slots are all the same request's
        return V > 1 && x >= s0 && x + 32 * V <= e1 && off[last] <= x && x + 32 * V <= off[last + 1];
      };
      bool one = within();
      int lo = 0, hi = nu;  // off[lo] <= the lane's first slot < off[hi]
      if (!one) {
        const int f = max((int)x + P * lane, b0);
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (off[mid] <= f) lo = mid; else hi = mid;
        }
        last = __shfl_sync(0xffffffffu, lo, 0);
        one = within();
      }
      if (one) {  // the ids are loaded first, all at once
        const int at = held[last] - off[last], hx = (int)((held[last] + (long long)ps - 1) >> a.log2_page);
        int32_t* row = a.table + (long long)(r0 + last) * a.max_pages;
        const int32_t* fresh = a.free_pages + pg[last] - hx;
        int id[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int i = (int)x + 32 * P * (k / P) + P * lane + k % P, p = (at + i) >> a.log2_page;
          id[k] = k % P && ((at + i) & (ps - 1)) ? id[k - k % P] : p < hx ? row[p] : fresh[p];
        }
#pragma unroll
        for (int k = 0; k < V; k += P) {
          const int i = (int)x + 32 * k + P * lane;
          long long v[P];
#pragma unroll
          for (int y = 0; y < P; ++y) {
            const int pos = at + i + y, p = pos >> a.log2_page, z = pos & (ps - 1);
            if (p >= hx && z == 0) row[p] = id[k + y];
            v[y] = id[k + y] < 0 ? -1 : ((long long)id[k + y] << a.log2_page) + z;
          }
          if (P == 2 && a.wide) {
            *reinterpret_cast<longlong2*>(a.slots + i) = make_longlong2(v[0], v[P - 1]);
          } else {
#pragma unroll
            for (int y = 0; y < P; ++y) a.slots[i + y] = v[y];
          }
        }
        continue;
      }
#pragma unroll
      for (int k = 0; k < V / P; ++k) {
        const int i0 = (int)x + 32 * P * k + P * lane;
        long long v[P];
        int pos = 0;
#pragma unroll
        for (int y = 0; y < P; ++y) {
          const int i = i0 + y;
          const bool mine = i >= b0 && i < e1 && i >= s0;
          v[y] = -1;
          if (!mine) continue;
          const bool go = y > 0 && mine && i - 1 >= b0 && i - 1 >= s0 && i < off[lo + 1];
          while (off[lo + 1] <= i) ++lo;
          pos = held[lo] + (i - off[lo]);
          if (go && (pos & (ps - 1)) != 0) {  // the same page as the pair's first slot
            v[y] = v[0] < 0 ? -1 : v[0] + 1;
            continue;
          }
          const int p = pos >> a.log2_page, hx = (int)((held[lo] + (long long)ps - 1) >> a.log2_page);
          int32_t* entry = a.table + (long long)(r0 + lo) * a.max_pages + p;
          const int id = p < hx ? *entry : a.free_pages[pg[lo] + p - hx];
          if (p >= hx && (pos & (ps - 1)) == 0) *entry = id;
          v[y] = id < 0 ? -1 : ((long long)id << a.log2_page) + (pos & (ps - 1));
        }
        if (P == 2 && a.wide && i0 >= b0 && i0 >= s0 && i0 + 1 < e1) {
          *reinterpret_cast<longlong2*>(a.slots + i0) = make_longlong2(v[0], v[P - 1]);
        } else {
#pragma unroll
          for (int y = 0; y < P; ++y)
            if (i0 + y >= b0 && i0 + y >= s0 && i0 + y < e1) a.slots[i0 + y] = v[y];
        }
      }
    }
    base_t += ct;
    base_p += cp;
    __syncthreads();
  }
}

__device__ __forceinline__ uint32_t e4m3_code(float y) {
  const uint32_t c = __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
  return (c & 0x7Fu) == 0 ? 0u : c;  // +0 for zero
}

// Eight bf16 values to E4M3 codes with the row's scale (LANES lanes hold the row).
template <int LANES>
__device__ __forceinline__ uint2 quantise(uint4 w, unsigned mask, float* scale) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  float f[8], m = 0.f;
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    f[2 * y] = __uint_as_float(u[y] << 16);
    f[2 * y + 1] = __uint_as_float(u[y] & 0xFFFF0000u);
    m = fmaxf(m, fmaxf(fabsf(f[2 * y]), fabsf(f[2 * y + 1])));
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o, LANES));
  const float sc = m > 0.f ? __fdiv_rn(m, kE4m3Max) : 1.0f;
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int y = 0; y < 8; ++y) c[y >> 2] |= e4m3_code(__fdiv_rn(f[y], sc)) << (8 * (y & 3));
  *scale = sc;
  return make_uint2(c[0], c[1]);
}

// One (new position, key head) per LANES = d / 8 lanes, 16 bytes of K and of V each. Bound by
// reading the rows and writing the cache once in bf16 (300,001 rows of 2 heads of 128: 100 us, 0.94 of a copy's
// rate); in FP8 (140 us, 0.51) a lane makes 16 divisions for its 48 bytes. IDX is 32 bits where the rows fit (a 64-bit
// division a row costs more than its bytes).
template <int LANES, bool FP8, typename IDX>
__global__ void __launch_bounds__(256) paged_append_kernel(PagedAppendArgs a) {
  const int lane = threadIdx.x & (LANES - 1), ps = 1 << a.log2_page;
  const IDX rows = (IDX)a.n * (IDX)a.Hkv, step = (IDX)gridDim.x * (256 / LANES);
  const long long cap = a.n_pages << a.log2_page;
  const unsigned mask = (LANES == 16 ? 0xffffu : 0xffu) << (threadIdx.x & 31 & ~(LANES - 1));
  for (IDX x = (IDX)blockIdx.x * (256 / LANES) + threadIdx.x / LANES; x < rows; x += step) {
    const IDX i = x / (IDX)a.Hkv;
    const int h = (int)(x - i * (IDX)a.Hkv);
    const long long slot = a.slots[i];
    const uint4 kw = reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.K + (long long)i * a.k_stride + h * (LANES * 8))[lane];
    const uint4 vw = reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.V + (long long)i * a.v_stride + h * (LANES * 8))[lane];
    if (slot < 0 || slot >= cap) continue;
    const long long row = (((slot >> a.log2_page) * a.Hkv + h) << a.log2_page) + (slot & (ps - 1));
    if (!FP8) {
      reinterpret_cast<uint4*>(a.k_cache)[row * LANES + lane] = kw;
      reinterpret_cast<uint4*>(a.v_cache)[row * LANES + lane] = vw;
    } else {
      float ks, vs;
      reinterpret_cast<uint2*>(a.k_cache)[row * LANES + lane] = quantise<LANES>(kw, mask, &ks);
      reinterpret_cast<uint2*>(a.v_cache)[row * LANES + lane] = quantise<LANES>(vw, mask, &vs);
      if (lane == 0) {
        a.k_scales[row] = ks;
        a.v_scales[row] = vs;
      }
    }
  }
}

template <int LANES, bool FP8>
void append_t(const PagedAppendArgs& a, cudaStream_t s) {
  const long long rows = a.n * a.Hkv;
  long long g = (rows * LANES + 255) / 256;
  if (g > a.sms * 32LL) g = a.sms * 32LL;
  if (rows + g * 256 < (1LL << 32)) paged_append_kernel<LANES, FP8, uint32_t><<<(unsigned)g, 256, 0, s>>>(a);
  else paged_append_kernel<LANES, FP8, long long><<<(unsigned)g, 256, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_page_tables(const PageTablesArgs& a, cudaStream_t s) {
  // eight slots a thread once one a thread fills all threads (1 and 8, us: 300 slots 4.3 and 12.4; 90,000 6.3
  // and 6.3; 300,000 8.3 and 6.3; 6 M 43 and 16.5)
  const int v = a.n_slots > 2LL * a.sms * kUsers ? 8 : 1;
  long long g = (a.n_slots + v * kUsers - 1) / (v * kUsers);  // at most one pass of the threads each
  if (g < 1) g = 1;
  if (g > 2LL * a.sms) g = 2LL * a.sms;  // (one wave: every block repeats the sums)
  if (v == 8) page_tables_kernel<8><<<(unsigned)g, kUsers, 0, s>>>(a);
  else page_tables_kernel<1><<<(unsigned)g, kUsers, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
  if (a.n == 0 || a.n_pages == 0) return cudaSuccess;
  if (a.d == 128) {
    if (a.fp8) append_t<16, true>(a, s);
    else append_t<16, false>(a, s);
  } else {
    if (a.fp8) append_t<8, true>(a, s);
    else append_t<8, false>(a, s);
  }
  return cudaGetLastError();
}

}  // namespace sa
