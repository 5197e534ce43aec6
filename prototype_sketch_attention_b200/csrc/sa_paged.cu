// The paged key-value cache: block tables and slot maps from request lengths, and the
// append of new rows (bf16, or FP8 E4M3 with one scale per row).
#include <cuda_fp8.h>

#include "sa_common.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

constexpr float kE4m3Max = 448.0f;

// Inclusive prefix sums over the block (up to 1024 threads) of two counts at once.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long (&part)[2][32],
                                            long long& total_a, long long& total_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  __syncthreads();
  if (lane == 31) {
    part[0][warp] = a;
    part[1][warp] = b;
  }
  __syncthreads();
  long long ba = 0, bb = 0;
  total_a = total_b = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) {
      ba += part[0][w];
      bb += part[1][w];
    }
    total_a += part[0][w];
    total_b += part[1][w];
  }
  a += ba;
  b += bb;
}

// Every block first adds up all requests (the verdict is needed before anything is
// written), then walks the requests again, kUsers at a time, keeping their prefix sums in
// shared memory, and writes the slots of its own share [s0, s1) of the new positions. Block 0
// also writes the tables, offsets and lengths.
constexpr int kUsers = 512;
constexpr int kTableThreads = 512;

__global__ void __launch_bounds__(kTableThreads) page_tables_kernel(PageTablesArgs a) {
  __shared__ long long part[2][32];
  __shared__ long long off[kUsers + 1], pg[kUsers];
  const int tid = threadIdx.x, ps = 1 << a.log2_page;
  const long long used = a.free_used ? *a.free_used : 0;
  // verdict
  long long toks = 0, pages = 0;
  int bad = 0;  // bit 0: lengths, bit 1: pages
  for (int r = tid; r < a.R; r += blockDim.x) {
    const long long c = a.cached[r], n = a.fresh[r];
    if (c < 0 || n < 0 || c + n > 0x7fffffffLL) { bad |= 1; continue; }
    const long long have = (c + ps - 1) >> a.log2_page, want = (c + n + ps - 1) >> a.log2_page;
    if (want > a.max_pages) bad |= 2;
    toks += n;
    pages += want - have;
  }
  long long tt, tp;
  block_scan2(toks, pages, part, tt, tp);
  if (tt > a.n_slots) bad |= 1;
  if (used < 0 || used + tp > a.n_free) bad |= 2;
  const int bad1 = __syncthreads_or(bad & 1), bad2 = __syncthreads_or(bad & 2);
  const bool stop = bad1 || bad2;
  const bool lead = blockIdx.x == 0;
  const long long per = (a.n_slots + gridDim.x - 1) / gridDim.x;
  const long long s0 = min((long long)a.n_slots, blockIdx.x * per), s1 = min((long long)a.n_slots, s0 + per);
  if (lead && tid == 0) {
    a.hdr->status = bad1 ? SA_ERR_BAD_OFFSETS : bad2 ? SA_ERR_BAD_PAGES : SA_OK;
    *a.free_used_out = stop ? used : used + tp;
    a.new_offsets[a.R] = stop ? 0 : tt;
  }
  for (long long i = max(s0, stop ? 0 : tt) + tid; i < s1; i += blockDim.x) a.slots[i] = -1;
  if (stop) {
    if (lead)
      for (int r = tid; r < a.R; r += blockDim.x) {
        a.new_offsets[r] = 0;
        a.seq_lens[r] = a.cached[r];
      }
    return;
  }
  long long base_t = 0, base_p = used;
  for (int r0 = 0; r0 < a.R; r0 += kUsers) {
    const int r = r0 + tid, nu = min(kUsers, a.R - r0);
    long long c = 0, n = 0, have = 0, need = 0;
    if (tid < nu) {
      c = a.cached[r];
      n = a.fresh[r];
      have = (c + ps - 1) >> a.log2_page;
      need = ((c + n + ps - 1) >> a.log2_page) - have;
    }
    long long it = n, ip = need, ct, cp;
    block_scan2(it, ip, part, ct, cp);
    if (tid < nu) {
      off[tid] = base_t + it - n;
      pg[tid] = base_p + ip - need;
      if (lead) {
        a.new_offsets[r] = base_t + it - n;
        a.seq_lens[r] = (int)(c + n);
      }
    }
    if (tid == 0) off[nu] = base_t + ct;
    __syncthreads();
    if (lead) {
      for (int x = tid >> 5; x < nu; x += blockDim.x >> 5) {
        const long long cx = a.cached[r0 + x], nx = a.fresh[r0 + x];
        const long long hx = (cx + ps - 1) >> a.log2_page;
        const int nd = (int)(((cx + nx + ps - 1) >> a.log2_page) - hx);
        int32_t* row = a.table + (long long)(r0 + x) * a.max_pages + hx;
        for (int i = tid & 31; i < nd; i += 32) row[i] = a.free_pages[pg[x] + i];
      }
    }
    const long long e1 = min(s1, base_t + ct);
    for (long long i = max(s0, base_t) + tid; i < e1; i += blockDim.x) {
      int lo = 0, hi = nu;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= i) lo = mid; else hi = mid;
      }
      const long long cx = a.cached[r0 + lo], pos = cx + i - off[lo];
      const long long hx = (cx + ps - 1) >> a.log2_page, p = pos >> a.log2_page;
      const long long id = p < hx ? a.table[(long long)(r0 + lo) * a.max_pages + p]
                                  : a.free_pages[pg[lo] + p - hx];
      a.slots[i] = id < 0 ? -1 : (id << a.log2_page) + (pos & (ps - 1));
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

// One row of K or V per LANES lanes (LANES = d / 8, 16 bytes a lane).
template <int LANES, bool FP8>
__global__ void __launch_bounds__(256) paged_append_kernel(PagedAppendArgs a) {
  const int lane = threadIdx.x & (LANES - 1);
  const long long g0 = (blockIdx.x * 256LL + threadIdx.x) / LANES, gs = gridDim.x * (256LL / LANES);
  const long long rows = a.n * a.Hkv * 2, cap = a.n_pages << a.log2_page;
  const unsigned mask = (LANES == 16 ? 0xffffu : 0xffu) << (threadIdx.x & 31 & ~(LANES - 1));
  for (long long g = g0; g < rows; g += gs) {
    const long long i = g / (2 * a.Hkv);
    const int x = (int)(g - i * (2 * a.Hkv)), v = x >= a.Hkv, h = v ? x - a.Hkv : x;
    const long long slot = a.slots[i];
    if (slot < 0 || slot >= cap) continue;
    const __nv_bfloat16* src = (v ? (const __nv_bfloat16*)a.V + i * a.v_stride
                                  : (const __nv_bfloat16*)a.K + i * a.k_stride) + h * (LANES * 8);
    const uint4 w = reinterpret_cast<const uint4*>(src)[lane];
    const long long row = ((((slot >> a.log2_page) * a.Hkv) + h) << a.log2_page) +
                          (slot & ((1 << a.log2_page) - 1));
    if (!FP8) {
      reinterpret_cast<uint4*>(v ? a.v_cache : a.k_cache)[row * LANES + lane] = w;
    } else {
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
      reinterpret_cast<uint2*>(v ? a.v_cache : a.k_cache)[row * LANES + lane] = make_uint2(c[0], c[1]);
      if (lane == 0) (v ? a.v_scales : a.k_scales)[row] = sc;
    }
  }
}

}  // namespace

cudaError_t launch_page_tables(const PageTablesArgs& a, cudaStream_t s) {
  long long g = (a.n_slots + 4095) / 4096;
  if (g < 1) g = 1;
  if (g > a.sms) g = a.sms;
  page_tables_kernel<<<(unsigned)g, kTableThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
  if (a.n == 0 || a.n_pages == 0) return cudaSuccess;
  const int lanes = a.d / 8;
  long long g = (a.n * a.Hkv * 2 * lanes + 255) / 256;
  if (g > 148LL * 32) g = 148LL * 32;
  if (a.d == 128) {
    if (a.fp8) paged_append_kernel<16, true><<<(unsigned)g, 256, 0, s>>>(a);
    else paged_append_kernel<16, false><<<(unsigned)g, 256, 0, s>>>(a);
  } else {
    if (a.fp8) paged_append_kernel<8, true><<<(unsigned)g, 256, 0, s>>>(a);
    else paged_append_kernel<8, false><<<(unsigned)g, 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace sa
