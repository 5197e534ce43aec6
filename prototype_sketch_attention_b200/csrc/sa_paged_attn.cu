// Attention of one new token per request over the paged key-value cache (sm_100a).
//
// Bound by reading the cache once: 4 H operations a cached value pair against 2 or 4 bytes, so
// the products stay on mma.sync, whose operands come straight from the copied pages (16 query heads
// at most share a key head's rows; tcgen05 would pad them to 128). Keys are the rows of the products:
//   S^T [keys x heads] = K Q^T,   P = 2^(c S^T - m),   O^T [d x heads] += V^T P^T,   c = scale log2 e,
// so that 8 heads fill one n-tile, the running maximum and sum of a head stay in one lane column
// of S^T and O^T alike, and P^T becomes the next operand by an 8 x 8 transpose in registers.
//
// Work. A (request, key head, up to 16 of its query heads) is an item; its positions from the
// window on are cut into tiles of T keys (K and V: 16 KB, or 8 in FP8). All items' tiles in order are split
// evenly over the CTAs (one per SM) and within a CTA over its warps, each of which runs on its
// own: it copies its pages by TMA into a ring of two tiles and keeps the softmax state of its
// current item in registers. An item that one warp sees whole is written at once. Else the warps'
// parts are put together in the CTA, in order, and what spans CTAs by paged_join_kernel, in
// order: the result does not depend on timing. The 12 to 16 tiles in flight on an SM, 144 to
// 224 KB, are more than the 45 KB that the memory's latency times its rate needs.
//
// FP8 codes go to fp16 exactly (one conversion instruction a pair), and the products run in fp16.
// A head's query is brought to [2^8, 2^9) by a power of two, which costs nothing that fp32 sums
// would keep (what falls below fp16's steps is 2^-33 of the largest value). The second product's weights are
// p v_scale in a unit of each head's own, from its largest p v_scale so far: a value row's scale alone says
// little (the append gives a row of zeros the scale 1 among any neighbours: in a unit from the scales,
// neighbours of 1e-4 would lose all digits). The largest is at 1/2 to 2^8, and weights are rounded by 2^-11
// of their value, or by 2^-25 where they are below 2^-14. The same steps through bf16 took
// 9 integer instructions a word in place of 2 or 3. A key's scale multiplies its scores in fp32.
// Measured (of the 6,568 GB/s of a copy): 40 requests x 10K positions, 12 heads over 4, bf16: 0.141 ms
// (0.88); 300 x 1K-100K, 8 heads over 1, FP8: 0.300 ms (0.93; through bf16 0.393); 16 heads over 1 on
// such requests: 0.32 ms (0.82), and 0.19 to 0.20 at d = 64 (0.66 to 0.72; 0.19 with one unit for all
// heads), where the products' issue is the bound; one request of 1,900 positions 10.6 us, one of
// 100,000 24 us. The unit of the weights is decided with the maximum, by one vote, from log2 of the scales: a
// vote of its own on the products, after the exponentials, cost 140 us in place of 132 at 16 heads and d = 64.
#include <cmath>

#include "sa_cross.cuh"

namespace sa {
namespace {

using cross::kLn2;
using cross::kLog2e;
constexpr float kRaise = 8.f;  // raise a running maximum only when passed by this (log2 units)
constexpr float kUnits = 126.f;  // FP8: 2^m and the unit of o are at most this far apart
constexpr int kMaxWarps = 12;

template <int D, bool FP8, int NT>
struct Geo {
  static constexpr int T = D == 64 ? 64 : 32;             // keys per tile
  static constexpr int kRow = FP8 ? D : 128;              // bytes of a shared-memory row
  static constexpr int kHalves = FP8 ? 1 : D / 64;        // a bf16 row of 128 is two 128-byte halves
  static constexpr int kMat = T * D * (FP8 ? 1 : 2);      // bytes of K or of V
  static constexpr int kSlot = 2 * kMat + (FP8 ? 1024 : 0);  // and the scales (1024-aligned slots)
  // As many warps as fit with two slots each: 7 of 32 KB, or 12 of 18 KB; with 16 heads a warp needs
  // more registers than 12 leave it (8 against 9 with spills: 0.61 and 0.48 of the copy rate).
  static constexpr int kWarps = !FP8 ? 7 : NT == 1 ? 12 : 8;
  static constexpr int oBars = kWarps * 2 * kSlot;
  static constexpr size_t kSmem = 1024 + oBars + kWarps * 2 * 8;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // an 8 x 8 block of 16-bit values
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma16816_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four E4M3 codes to two pairs of fp16, in order.
__device__ __forceinline__ void e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// What a CTA leaves for the join: errors seen, and the item (request, sub) that it saw the start
// of and that goes on in later CTAs, up to tile `end` of the `total` tiles.
struct CtaInfo {
  long long end, total;
  int error, open, r, sub;
};

struct PagedParams {
  const __nv_bfloat16* Q;
  long long q_stride;
  int R, H, Hkv, G;
  int subs, heads;        // items per request (key heads x chunks of heads), heads of a chunk
  int chunks;
  const float* k_scales;
  const float* v_scales;
  int n_pages, log2_page, max_pages;
  const int32_t* table;
  const int32_t* seq_lens;
  long long window;
  float c;
  __nv_bfloat16* out;
  float* lse;
  float* parts;           // partial results: [CTAs][kMaxWarps][2], then [CTAs][2]
  CtaInfo* info;          // [CTAs]
  int* status;
  int ctas;
  long long budget;
};

// Tiles of one item of request r (all items of a request have as many), and its first tile.
__device__ __forceinline__ int request_tiles(const PagedParams& a, int len, int T, int* first_tile,
                                             int* first) {
  const int f = a.window > 0 && len > a.window ? (int)(len - a.window) : 0;
  *first = f;
  *first_tile = f / T;
  return (len + T - 1) / T - f / T;
}
__device__ __forceinline__ int checked_len(const PagedParams& a, int r, int* bad) {
  const int len = a.seq_lens[r];
  if (len < 0 || len > ((long long)a.max_pages << a.log2_page)) {
    *bad = SA_ERR_BAD_OFFSETS;
    return 0;
  }
  return len;
}

// The tile lists of the requests, seen by one warp: lane l owns the requests [l C, (l + 1) C).
struct Ranges {
  long long before;  // tiles (per item) before this lane's requests
  long long total;   // tiles of all items
  int C;
  __device__ void init(const PagedParams& a, int T, int lane, int* bad) {
    C = (a.R + 31) / 32;
    long long n = 0;
    const int r1 = min(a.R, (lane + 1) * C);
    for (int r = lane * C; r < r1; ++r) {
      int ft, f;
      n += request_tiles(a, checked_len(a, r, bad), T, &ft, &f);
    }
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    before = incl - n;
    total = __shfl_sync(0xffffffffu, incl, 31) * a.subs;
  }
  // the request whose items hold tile x (x < total), and the tiles before it; whole warp
  __device__ int find(const PagedParams& a, int T, int lane, long long x, long long* base) const {
    const unsigned le = __ballot_sync(0xffffffffu, before * a.subs <= x);
    int src = 31 - __clz(le);  // the last lane that starts at or before x
    long long b = __shfl_sync(0xffffffffu, before, src);
    int bad = 0;
    for (int r0 = src * C;; r0 += 32) {
      int n = 0, ft, f;
      if (r0 + lane < a.R) n = request_tiles(a, checked_len(a, r0 + lane, &bad), T, &ft, &f);
      long long incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, (b + incl) * a.subs > x);
      if (hit) {
        const int l = __ffs(hit) - 1;
        *base = (b + __shfl_sync(0xffffffffu, incl - n, l)) * a.subs;
        return r0 + l;
      }
      b += __shfl_sync(0xffffffffu, incl, 31);
      if (r0 + 32 >= a.R) {  // not reached for x < total
        *base = b * a.subs;
        return a.R - 1;
      }
    }
  }
};

// A place in the list of tiles: item (r, sub), tile t of [t0, t1).
struct Cursor {
  int r, sub, t, t0, t1, len, first;
  __device__ void request(const PagedParams& a, int T) {
    int bad;
    len = checked_len(a, r, &bad);
    t1 = request_tiles(a, len, T, &t0, &first);
    t1 += t0;
  }
  __device__ void next(const PagedParams& a, int T) {
    if (++t < t1) return;
    if (++sub == a.subs) {
      sub = 0;
      do {
        if (++r >= a.R) return;
        request(a, T);
      } while (t1 == t0);
    }
    t = t0;
  }
};

// A part of an item: running maximum and sum of every head, and the raw O^T fragments.
template <int D, int NT>
struct Part {
  static constexpr int kO = NT * D / 16 * 128;  // floats of O^T
  static constexpr int kStride = kO + 2 * 8 * NT;
};

template <int D, int NT>
struct State {
  float o[D / 16][NT][4];
  float r[NT][2], u[NT][2];  // FP8: o is in units of 2^r; u = 2^(m - r)
  float m[NT][2], l[NT][2];  // heads 8 nt + 2 (lane mod 4) and the next; l summed over this lane's keys
  __device__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      r[n][0] = r[n][1] = -INFINITY;
      u[n][0] = u[n][1] = 1.f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    }
  }
  __device__ void scale_o(int n, float f0, float f1) {  // of the two heads
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      o[i][n][0] *= f0;
      o[i][n][1] *= f1;
      o[i][n][2] *= f0;
      o[i][n][3] *= f1;
    }
  }
  __device__ void plain_units() {  // 2^m, as l
#pragma unroll
    for (int n = 0; n < NT; ++n) scale_o(n, 1.f / u[n][0], 1.f / u[n][1]);
  }
  __device__ void sum_l() {  // over the lanes that hold other keys of the same head
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
  }
  __device__ void store(float* p, int lane) const {  // after sum_l
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        reinterpret_cast<float4*>(p)[(i * NT + n) * 32 + lane] =
            make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
    if (lane < 4) {
      float* q = p + Part<D, NT>::kO;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          q[n * 8 + 2 * lane + e] = m[n][e];
          q[8 * NT + n * 8 + 2 * lane + e] = l[n][e];
        }
    }
  }
  __device__ void merge(const float* p, int lane) {  // both summed over lanes
    const float* q = p + Part<D, NT>::kO;
    float f[NT][2], g[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float pm = q[n * 8 + 2 * (lane & 3) + e], pl = q[8 * NT + n * 8 + 2 * (lane & 3) + e];
        const float mm = fmaxf(m[n][e], pm);
        f[n][e] = l[n][e] > 0.f ? ex2_approx(m[n][e] - mm) : 0.f;
        g[n][e] = pl > 0.f ? ex2_approx(pm - mm) : 0.f;
        m[n][e] = mm;
        l[n][e] = l[n][e] * f[n][e] + pl * g[n][e];
      }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float4 v = reinterpret_cast<const float4*>(p)[(i * NT + n) * 32 + lane];
        o[i][n][0] = o[i][n][0] * f[n][0] + v.x * g[n][0];
        o[i][n][1] = o[i][n][1] * f[n][1] + v.y * g[n][1];
        o[i][n][2] = o[i][n][2] * f[n][0] + v.z * g[n][0];
        o[i][n][3] = o[i][n][3] * f[n][1] + v.w * g[n][1];
      }
  }
};

// out of 16 columns of d (fragment i) and 8 heads, from (d, heads) to (head g, pairs of d).
template <bool FP8>
__device__ __forceinline__ void write_fragment(const float (&o)[4], float inv0, float inv1, bool write,
                                               __nv_bfloat16* row, int q4) {
  const uint32_t lo = transpose8(cvt_bf16x2(o[0] * inv0, o[1] * inv1));
  const uint32_t hi = transpose8(cvt_bf16x2(o[2] * inv0, o[3] * inv1));
  if (write) {
    if (FP8) {  // fragment rows 0-7 are d = 0, 2, .., 14 and rows 8-15 are d = 1, 3, .., 15
      *reinterpret_cast<uint2*>(row + 4 * q4) =
          make_uint2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
    } else {
      *reinterpret_cast<uint32_t*>(row + 2 * q4) = lo;
      *reinterpret_cast<uint32_t*>(row + 8 + 2 * q4) = hi;
    }
  }
}

// out and lse of an item from its finished state (l summed over lanes).
template <int D, bool FP8, int NT>
__device__ __forceinline__ void write_item(const PagedParams& a, const State<D, NT>& st, int r, int sub,
                                           int lane) {
  const int hk = sub / a.chunks, h0 = hk * a.G + (sub % a.chunks) * a.heads;
  const int nh = min(a.heads, (hk + 1) * a.G - h0);
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float i0 = st.l[n][0] == 0.f ? 0.f : 1.f / st.l[n][0];  // (a NaN stays one)
    const float i1 = st.l[n][1] == 0.f ? 0.f : 1.f / st.l[n][1];
    __nv_bfloat16* row = a.out + ((long long)r * a.H + h0 + 8 * n + g) * D;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      write_fragment<FP8>(st.o[i][n], i0, i1, 8 * n + g < nh, row + 16 * i, t);
    if (a.lse && g == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (8 * n + 2 * t + e < nh)
          a.lse[(long long)r * a.H + h0 + 8 * n + 2 * t + e] =
              st.l[n][e] == 0.f ? -INFINITY : (st.m[n][e] + lg2_approx(st.l[n][e])) * kLn2;
    }
  }
}

// Where a warp's (or CTA's) parts go: at most one that starts inside an item (its first) and one
// that ends inside an item it saw the start of (its last).
enum : int { kNone = 0, kOpen = 1, kEnds = 2 };  // kEnds: reaches the item's end

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(Geo<D, FP8, NT>::kWarps * 32, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                  const __grid_constant__ PagedParams a) {
  using L = Geo<D, FP8, NT>;
  constexpr int T = L::T, MT = T / 16, KS = D / 16, kWarps = L::kWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ int head_kind[kWarps], tail_kind[kWarps], errors;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
  griddep_launch_dependents();  // the join reads its inputs only after this grid has ended
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::oBars) + 2 * warp;
  const uint32_t slot0 = smem_u32(smem) + warp * 2 * L::kSlot;
  if (threadIdx.x == 0) errors = 0;
  if (lane == 0) {
    mbar_init(smem_u32(&bars[0]), 1);
    mbar_init(smem_u32(&bars[1]), 1);
    fence_mbar_init();
    head_kind[warp] = tail_kind[warp] = kNone;
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
  }
  __syncthreads();
  int bad = 0;

  Ranges rg;
  rg.init(a, T, lane, &bad);
  const long long W = rg.total;
  const long long ca = W * blockIdx.x / a.ctas, cb = W * (blockIdx.x + 1) / a.ctas;
  const long long xa = ca + (cb - ca) * warp / kWarps, xb = ca + (cb - ca) * (warp + 1) / kWarps;
  float* parts = a.parts + ((long long)blockIdx.x * kMaxWarps + warp) * 2 * Part<D, NT>::kStride;
  int last_r = 0, last_sub = 0;
  long long last_end = 0;  // the tile behind the last item
  bool dead = false;
  if (xa < xb) {
    long long base;
    Cursor cur;
    cur.r = rg.find(a, T, lane, xa, &base);
    cur.request(a, T);
    const int nt = cur.t1 - cur.t0;
    cur.sub = (int)((xa - base) / nt);
    cur.t = cur.t0 + (int)((xa - base) % nt);
    Cursor ahead = cur;

    // copies of one tile: lane -> (page, K or V, half); scales by the first lanes
    const int ps = 1 << a.log2_page, box = min(ps, T), np = T / box;
    const int kinds = 2 * L::kHalves;
    auto copy = [&](int slot) {
      const int hk = ahead.sub / a.chunks;
      const int p0 = ahead.t * T, pos = p0 + (lane / kinds) * box;  // this lane's first position
      const bool mine = lane < np * kinds && pos < ahead.len && pos + box > ahead.first;
      int page = -1;
      if (mine) {
        page = a.table[(long long)ahead.r * a.max_pages + (pos >> a.log2_page)];
        if (page < 0 || page >= a.n_pages) {
          bad = SA_ERR_BAD_PAGES;
          page = -1;
        }
      }
      const int copies = __popc(__ballot_sync(0xffffffffu, page >= 0));
      const uint32_t bar = smem_u32(&bars[slot]);
      const uint32_t dst = slot0 + slot * L::kSlot;
      if (lane == 0)
        mbar_arrive_expect_tx(bar, copies * box * L::kRow + (FP8 ? copies * box * 4 : 0));
      __syncwarp();
      if (page >= 0) {
        const int kind = lane % kinds, v = kind / L::kHalves, half = kind % L::kHalves;
        const int row = ((page * a.Hkv + hk) << a.log2_page) + (pos & (ps - 1));
        const uint32_t to = dst + v * L::kMat + half * T * 128 + (pos - p0) * L::kRow;
        tma_load_2d(to, v ? &tmap_v : &tmap_k, half * 64, row, bar);
        if (FP8)
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
              ::"r"(dst + 2 * L::kMat + v * T * 4 + (pos - p0) * 4),
                "l"((v ? a.v_scales : a.k_scales) + row), "r"(box * 4), "r"(bar)
              : "memory");
      }
      ahead.next(a, T);
    };
    const int n_tiles = (int)(xb - xa);
    copy(0);
    if (n_tiles > 1) copy(1);

    State<D, NT> st;
    uint32_t qf[KS][NT][2];
    float qc[NT][2];  // FP8: c times what the query's power of two took away
    bool fresh = true, from_start = false;
    for (int i = 0; i < n_tiles; ++i) {
      const int slot = i & 1;
      if (fresh) {  // a new item: its queries as the products' right operand
        st.clear();
        from_start = cur.t == cur.t0;
        const int hk = cur.sub / a.chunks, h0 = hk * a.G + (cur.sub % a.chunks) * a.heads;
        const int nh = min(a.heads, (hk + 1) * a.G - h0);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const __nv_bfloat16* qr = a.Q + cur.r * a.q_stride + (h0 + 8 * n + g) * D;
          const bool w = 8 * n + g < nh;
          uint32_t top = 0;  // FP8: the row's largest magnitude (bits of a float)
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            if (FP8) {
              const uint2 v = w ? *reinterpret_cast<const uint2*>(qr + 16 * ks + 4 * q4) : make_uint2(0, 0);
              qf[ks][n][0] = v.x;
              qf[ks][n][1] = v.y;
              top = max(top, max((v.x << 16) & 0x7fffffffu, v.x & 0x7fff0000u));
              top = max(top, max((v.y << 16) & 0x7fffffffu, v.y & 0x7fff0000u));
            } else {
              qf[ks][n][0] = w ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 2 * q4) : 0u;
              qf[ks][n][1] = w ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 8 + 2 * q4) : 0u;
            }
          }
          if (FP8) {
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = max((int)(top >> 23), 10) - 135;  // row max in [2^(e + 8), 2^(e + 9))
            const float down = pow2i(-e);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t v = qf[ks][n][x];
                qf[ks][n][x] = cvt_f16x2(__uint_as_float(v << 16) * down,
                                         __uint_as_float(v & 0xffff0000u) * down);
              }
            const float up = pow2i(e) * a.c;  // row g's; this lane's score columns are heads 2 q4, + 1
            qc[n][0] = __shfl_sync(0xffffffffu, up, 8 * q4);
            qc[n][1] = __shfl_sync(0xffffffffu, up, 8 * q4 + 4);
          }
        }
        fresh = false;
      }
      if (!mbar_wait_warp(smem_u32(&bars[slot]), (uint32_t)((i >> 1) & 1), &errors, a.budget)) {
        dead = true;
        break;
      }
      const uint32_t kb = slot0 + slot * L::kSlot, vb = kb + L::kMat;
      float* ksc = reinterpret_cast<float*>(smem + (kb - smem_u32(smem)) + 2 * L::kMat);
      const int p0 = cur.t * T;
      const bool edge = p0 < cur.first || p0 + T > cur.len;
      if (edge) {  // weight 0 meets these rows of V: they must not hold NaN
        uint8_t* vs = smem + (vb - smem_u32(smem));
        for (int x = lane; x < T * (L::kRow / 16) * L::kHalves; x += 32) {
          const int y = x % (L::kRow / 16), z = x / (L::kRow / 16), half = z / T, p = p0 + z % T;
          if (p < cur.first || p >= cur.len)
            *reinterpret_cast<uint4*>(vs + half * T * 128 + (z % T) * L::kRow + y * 16) =
                make_uint4(0, 0, 0, 0);
        }
        if (FP8)
          for (int x = lane; x < T; x += 32)
            if (p0 + x < cur.first || p0 + x >= cur.len) ksc[T + x] = 0.f;
        __syncwarp();
      }
      // ---- S^T = K Q^T
      float s[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[mt][n][0] = s[mt][n][1] = s[mt][n][2] = s[mt][n][3] = 0.f;
        const int row = mt * 16 + (lane & 15);
        if (FP8) {
#pragma unroll
          for (int ks = 0; ks < KS; ks += 2) {  // a 16-byte piece is 16 values: two steps a load
            const int ch = ks + (lane >> 4);
            uint32_t w[4];
            ldsm4(kb + row * L::kRow + ((D == 128 ? ch ^ (row & 7) : ch ^ ((row >> 1) & 3)) << 4), w);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // bytes 4t .. 4t + 3 of a piece: k = 2t, 2t + 1 and k = 2t + 8, 2t + 9
              uint32_t a0, a1, a2, a3;
              e4m3x4(w[2 * h], a0, a2);
              e4m3x4(w[2 * h + 1], a1, a3);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma16816_f16(s[mt][n], a0, a1, a2, a3, qf[ks + h][n][0], qf[ks + h][n][1]);
            }
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const int ch = 2 * ks + (lane >> 4);
            uint32_t w[4];
            ldsm4(kb + (ch >> 3) * T * 128 + row * 128 + (((ch & 7) ^ (row & 7)) << 4), w);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(s[mt][n], w[0], w[1], w[2], w[3], qf[ks][n][0], qf[ks][n][1]);
          }
        }
      }
      // ---- softmax along the keys: lane column = heads 2 q4 and 2 q4 + 1, rows g and g + 8
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          const float f = FP8 ? ksc[mt * 16 + g + 8 * hi] : a.c;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[mt][n][2 * hi + e] *= FP8 ? f * qc[n][e] : f;
        }
      if (edge) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hi = 0; hi < 2; ++hi) {
            const int p = p0 + mt * 16 + g + 8 * hi;
            if (p < cur.first || p >= cur.len) {
#pragma unroll
              for (int n = 0; n < NT; ++n) s[mt][n][2 * hi] = s[mt][n][2 * hi + 1] = -INFINITY;
            }
          }
      }
      float mx[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[n][e] = fmaxf(s[0][n][e], s[0][n][2 + e]);
#pragma unroll
          for (int mt = 1; mt < MT; ++mt) mx[n][e] = fmax3(mx[n][e], s[mt][n][e], s[mt][n][2 + e]);
        }
      float mw[NT][2];  // FP8: the maximum of log2(p v_scale) + m
      if (FP8) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const float v0 = lg2_approx(fabsf(ksc[T + mt * 16 + g])), v1 = lg2_approx(fabsf(ksc[T + mt * 16 + g + 8]));
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float w0 = s[mt][n][e] + v0, w1 = s[mt][n][2 + e] + v1;
              mw[n][e] = mt == 0 ? fmaxf(w0, w1) : fmax3(mw[n][e], w0, w1);
            }
        }
      }
      bool raise = false;  // (the vote goes over the lanes: their maxima are only needed behind it)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          raise = raise || mx[n][e] - st.m[n][e] > kRaise || (FP8 && mw[n][e] - st.r[n][e] > kRaise);
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx[n][e] = fmaxf(mx[n][e], __shfl_xor_sync(0xffffffffu, mx[n][e], x));
            const float mm = fmaxf(st.m[n][e], mx[n][e]);
            f[e] = st.m[n][e] > -INFINITY ? ex2_approx(st.m[n][e] - mm) : 0.f;
            st.m[n][e] = mm;
            st.l[n][e] *= f[e];
            if (FP8) {
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) mw[n][e] = fmaxf(mw[n][e], __shfl_xor_sync(0xffffffffu, mw[n][e], x));
              float r = mw[n][e] - st.r[n][e] > kRaise ? ceilf(mw[n][e]) : st.r[n][e];
              r = fmaxf(fminf(r, mm + kUnits), mm - kUnits);  // (u and 1 / u are normal numbers)
              f[e] = st.r[n][e] > -INFINITY ? ex2_approx(st.r[n][e] - r) : 0.f;
              st.r[n][e] = r;
              st.u[n][e] = mm > -INFINITY ? ex2_approx(mm - r) : 1.f;
            }
          }
          st.scale_o(n, f[0], f[1]);
        }
      }
      uint32_t pf[MT][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float m0 = st.m[n][0] == -INFINITY ? 0.f : st.m[n][0];
        const float m1 = st.m[n][1] == -INFINITY ? 0.f : st.m[n][1];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hi = 0; hi < 2; ++hi) {
            float e0 = ex2_approx(s[mt][n][2 * hi] - m0), e1 = ex2_approx(s[mt][n][2 * hi + 1] - m1);
            st.l[n][0] += e0;
            st.l[n][1] += e1;
            if (FP8) {
              const float vs = ksc[T + mt * 16 + g + 8 * hi];
              e0 = e0 * vs * st.u[n][0];
              e1 = e1 * vs * st.u[n][1];
            }
            pf[mt][n][hi] = transpose8(FP8 ? cvt_f16x2(e0, e1) : cvt_bf16x2(e0, e1));
          }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int kk = 0; kk < MT; ++kk) {
        if (FP8) {
          const int row = kk * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
          for (int dm = 0; dm < KS; dm += 2) {
            const int ch = dm + (lane >> 4);
            uint32_t w[4];
            ldsm4_t(vb + row * L::kRow + ((D == 128 ? ch ^ (row & 7) : ch ^ ((row >> 1) & 3)) << 4), w);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // a word is (key 2t: d, d + 1), (key 2t + 1: d, d + 1): pairs of keys instead
              uint32_t a0, a1, a2, a3;
              e4m3x4(__byte_perm(w[2 * h], 0, 0x3120), a0, a1);
              e4m3x4(__byte_perm(w[2 * h + 1], 0, 0x3120), a2, a3);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma16816_f16(st.o[dm + h][n], a0, a1, a2, a3, pf[kk][n][0], pf[kk][n][1]);
            }
          }
        } else {
          const int row = kk * 16 + (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
          for (int dm = 0; dm < KS; ++dm) {
            const int ch = 2 * dm + ((lane >> 3) & 1);
            uint32_t w[4];
            ldsm4_t(vb + (ch >> 3) * T * 128 + row * 128 + (((ch & 7) ^ (row & 7)) << 4), w);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(st.o[dm][n], w[0], w[1], w[2], w[3], pf[kk][n][0], pf[kk][n][1]);
          }
        }
      }
      if (edge) fence_proxy_async_smem();  // the zeros, before the next copy into this slot
      __syncwarp();
      if (i + 2 < n_tiles) copy(slot);
      // ---- the end of the item, or of this warp's tiles
      const bool ends = cur.t + 1 == cur.t1;
      if (ends || i + 1 == n_tiles) {
        st.sum_l();
        if (FP8) st.plain_units();
        if (ends && from_start) {
          write_item<D, FP8, NT>(a, st, cur.r, cur.sub, lane);
        } else if (!from_start) {
          st.store(parts, lane);
          if (lane == 0) head_kind[warp] = ends ? kEnds : kOpen;
        } else {
          st.store(parts + Part<D, NT>::kStride, lane);
          if (lane == 0) tail_kind[warp] = kOpen;
          last_r = cur.r;
          last_sub = cur.sub;
          last_end = xb + (cur.t1 - cur.t - 1);
        }
        fresh = true;
      }
      cur.next(a, T);
    }
    if (dead) {  // let the copies in flight land before the block leaves
      for (int x = 0; x < 2; ++x)
        for (int ph = 0; ph < 2; ++ph) mbar_wait_drain(smem_u32(&bars[x]), (uint32_t)ph, 2000000LL);
    }
  }
  // requests without positions: CTA b's are b, b + CTAs, ..., 32 a warp
  for (int r0 = blockIdx.x + a.ctas * 32 * warp; r0 < a.R; r0 += a.ctas * 32 * kWarps) {
    const int r = r0 + a.ctas * lane;
    int dummy;
    unsigned none = __ballot_sync(0xffffffffu, r < a.R && checked_len(a, r, &dummy) == 0);
    while (none) {
      const long long row = (long long)(r0 + a.ctas * (__ffs(none) - 1)) * a.H;
      none &= none - 1;
      for (int x = lane; x < a.H * D / 8; x += 32)
        reinterpret_cast<uint4*>(a.out + row * D)[x] = make_uint4(0, 0, 0, 0);
      for (int x = lane; a.lse && x < a.H; x += 32) a.lse[row + x] = -INFINITY;
    }
  }
  const int any_bad = __reduce_max_sync(0xffffffffu, (unsigned)bad);
  if (lane == 0 && any_bad) atomicMax(&errors, any_bad);
  if (threadIdx.x == 0) a.info[blockIdx.x].open = 0;
  __syncthreads();  // the warps' parts are written
  if (threadIdx.x == 0) a.info[blockIdx.x].error = errors;

  // ---- parts that belong together, in order: a warp whose last item goes on in later warps
  // (or the first warp with tiles, when the CTA starts inside an item) adds them to its own
  int lead = -1;  // 0: this warp's first part leads (the CTA's first), 1: its last part does
  if (tail_kind[warp] != kNone) lead = 1;
  if (head_kind[warp] != kNone) {
    int w = 0;
    while (w < warp && ca + (cb - ca) * w / kWarps == ca + (cb - ca) * (w + 1) / kWarps) ++w;
    if (w == warp) {  // (a warp may lead twice: its first part may end, and its last start, an item)
      State<D, NT> st;
      st.clear();
      st.merge(parts, lane);
      bool end = head_kind[warp] == kEnds;
      for (int x = warp + 1; x < kWarps && !end; ++x)
        if (head_kind[x] != kNone) {
          st.merge(parts + (x - warp) * 2 * Part<D, NT>::kStride, lane);
          end = head_kind[x] == kEnds;
        }
      // the CTA started inside this item: its part 0
      st.store(a.parts + ((long long)a.ctas * kMaxWarps * 2 + blockIdx.x * 2) * Part<D, NT>::kStride, lane);
    }
  }
  if (lead == 1) {
    State<D, NT> st;
    st.clear();
    st.merge(parts + Part<D, NT>::kStride, lane);
    bool end = false;
    for (int x = warp + 1; x < kWarps && !end; ++x)
      if (head_kind[x] != kNone) {
        st.merge(parts + (x - warp) * 2 * Part<D, NT>::kStride, lane);
        end = head_kind[x] == kEnds;
      }
    if (end) write_item<D, FP8, NT>(a, st, last_r, last_sub, lane);
    else {  // goes on in the next CTA: this CTA's part 1
      st.store(a.parts + ((long long)a.ctas * kMaxWarps * 2 + blockIdx.x * 2 + 1) * Part<D, NT>::kStride, lane);
      if (lane == 0) {
        CtaInfo& in = a.info[blockIdx.x];
        in.end = last_end;
        in.total = W;
        in.r = last_r;
        in.sub = last_sub;
        in.open = 1;
      }
    }
  }
}

// An item that spans CTAs: block b joins the one that starts in CTA b and goes on, from the parts
// of CTAs b .. b1 in order (groups of threads take every kGroups-th part each and are then put
// together). SLICED: the blocks (b, i) join 16 columns i of d each, for few items of many parts
// (one block took 20 us for the 148 parts of a lone request of 100K, the slices 10; with many items,
// of few parts each, the slices' blocks cost 3 to 5 us). Block (0, 0) also writes the device status.
template <int D, bool FP8, int NT, bool SLICED>
__global__ void __launch_bounds__(512)
paged_join_kernel(const __grid_constant__ PagedParams a) {
  constexpr int kFrags = SLICED ? NT : NT * D / 16;  // fragments (16 columns x 8 heads) of a block
  constexpr int kV = kFrags * 32, kHeads = 8 * NT, kGroups = 512 / kV;
  extern __shared__ float ml[];  // [2][CTAs][kHeads]: maxima, then weights; sums (-1: no part)
  __shared__ float tot_m[kHeads], tot_l[kHeads];
  __shared__ float4 acc_s[kGroups][kV];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b0 = blockIdx.x, ci = blockIdx.y;
  griddep_wait();
  if (b0 == 0 && ci == 0) {
    int bad = 0;
    for (int x = tid; x < a.ctas; x += 512) bad = max(bad, a.info[x].error);
    bad = __syncthreads_or(bad == SA_ERR_TIMEOUT) ? SA_ERR_TIMEOUT
          : __syncthreads_or(bad == SA_ERR_BAD_PAGES) ? SA_ERR_BAD_PAGES
          : __syncthreads_or(bad == SA_ERR_BAD_OFFSETS) ? SA_ERR_BAD_OFFSETS : SA_OK;
    if (tid == 0) *a.status = bad;
  }
  const CtaInfo in = a.info[b0];
  if (!in.open) return;
  const long long W = in.total;
  int b1 = (int)((in.end - 1) * a.ctas / W);  // the CTA that holds the item's last tile
  while (b1 + 1 < a.ctas && W * (b1 + 1) / a.ctas <= in.end - 1) ++b1;
  while (W * b1 / a.ctas > in.end - 1) --b1;
  const int nb = b1 - b0 + 1;
  auto part_of = [&](int x) {  // the first CTA's last part, then the others' first parts
    return a.parts + ((long long)a.ctas * kMaxWarps * 2 + (b0 + x) * 2 + (x == 0 ? 1 : 0)) * Part<D, NT>::kStride;
  };
  // thread t of a group holds float4 t: n-tile (t / 32) mod NT, heads 2 (t mod 4) + e; a group's first
  // parts are loaded ahead of the weights
  const int grp = tid / kV, t = tid % kV, hh = (t >> 5) % NT * 8 + 2 * (t & 3);
  auto load = [&](int x) { return (reinterpret_cast<const float4*>(part_of(x)) + ci * kV)[t]; };
  constexpr int kAhead = 4;
  float4 ahead[kAhead];
#pragma unroll
  for (int y = 0; y < kAhead; ++y)
    if (grp + y * kGroups < nb) ahead[y] = load(grp + y * kGroups);
  float* ms = ml;
  float* ls = ml + a.ctas * kHeads;
  for (int i = tid; i < nb * kHeads; i += 512) {
    const int x = i / kHeads, h = i % kHeads;
    const bool some = W * (b0 + x) / a.ctas < W * (b0 + x + 1) / a.ctas;  // else a CTA without tiles
    const float* q = part_of(x) + Part<D, NT>::kO;
    ms[i] = some ? q[h] : -INFINITY;
    ls[i] = some ? q[kHeads + h] : -1.f;
  }
  __syncthreads();
  if (warp < kHeads) {  // 16 warps: one head each
    float m = -INFINITY, l = 0.f;
    for (int x = lane; x < nb; x += 32)
      if (!(ls[x * kHeads + warp] <= 0.f)) m = fmaxf(m, ms[x * kHeads + warp]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int x = lane; x < nb; x += 32) {
      const int i = x * kHeads + warp;
      const float w = ls[i] <= 0.f ? 0.f : ex2_approx(ms[i] - m);
      l += ls[i] <= 0.f ? 0.f : w * ls[i];
      ms[i] = w;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      tot_m[warp] = m;
      tot_l[warp] = l;
    }
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int x, const float4& v) {
    if (ls[x * kHeads] < 0.f) return;  // a CTA without tiles left nothing
    const float2 w = *reinterpret_cast<const float2*>(ms + x * kHeads + hh);
    acc.x = fmaf(v.x, w.x, acc.x);
    acc.y = fmaf(v.y, w.y, acc.y);
    acc.z = fmaf(v.z, w.x, acc.z);
    acc.w = fmaf(v.w, w.y, acc.w);
  };
#pragma unroll
  for (int y = 0; y < kAhead; ++y)
    if (grp + y * kGroups < nb) add(grp + y * kGroups, ahead[y]);
#pragma unroll 4
  for (int x = grp + kAhead * kGroups; x < nb; x += kGroups) add(x, load(x));
  acc_s[grp][t] = acc;
  __syncthreads();
  if (warp < kFrags) {  // a warp per fragment writes, as the main kernel's warps do
    const int g = lane >> 2, q4 = lane & 3, hk = in.sub / a.chunks, n = warp % NT, i = ci + warp / NT;
    const int h0 = hk * a.G + (in.sub % a.chunks) * a.heads, nh = min(a.heads, (hk + 1) * a.G - h0);
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < kGroups; ++x) {
      const float4 u = acc_s[x][warp * 32 + lane];
      o[0] += u.x;
      o[1] += u.y;
      o[2] += u.z;
      o[3] += u.w;
    }
    const float l0 = tot_l[n * 8 + 2 * q4], l1 = tot_l[n * 8 + 2 * q4 + 1];
    write_fragment<FP8>(o, l0 == 0.f ? 0.f : 1.f / l0, l1 == 0.f ? 0.f : 1.f / l1, 8 * n + g < nh,
                        a.out + ((long long)in.r * a.H + h0 + 8 * n + g) * D + 16 * i, q4);
    if (a.lse && i == 0 && lane < 8 && 8 * n + lane < nh) {
      const float l = tot_l[n * 8 + lane];
      a.lse[(long long)in.r * a.H + h0 + 8 * n + lane] =
          l == 0.f ? -INFINITY : (tot_m[n * 8 + lane] + lg2_approx(l)) * kLn2;
    }
  }
}

// 2-D tensor map over the cache's rows, boxes of one row width x box_rows.
bool tmap_cache(CUtensorMap* m, const void* base, uint64_t rows, int d, bool fp8, int box_rows) {
  auto fn = tmap_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)d * (fp8 ? 1 : 2)};
  const cuuint32_t box[2] = {(cuuint32_t)(fp8 ? d : 64), (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            fp8 && d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool FP8, int NT>
cudaError_t launch_t(const PagedAttnArgs& a, PagedParams& p, cudaStream_t s) {
  using L = Geo<D, FP8, NT>;
  const int ps = 1 << a.log2_page, box = ps < L::T ? ps : L::T;
  CUtensorMap tk, tv;
  const uint64_t rows = (uint64_t)a.n_pages * a.Hkv * ps;
  if (!tmap_cache(&tk, rows ? a.k_cache : a.Q, rows ? rows : 1, D, FP8, box) ||
      !tmap_cache(&tv, rows ? a.v_cache : a.Q, rows ? rows : 1, D, FP8, box))
    return cudaErrorInvalidValue;
  cudaError_t e = cross::prepare_kernel<paged_attn_kernel<D, FP8, NT>>(L::kSmem);
  if (e != cudaSuccess) return e;
  paged_attn_kernel<D, FP8, NT><<<p.ctas, L::kWarps * 32, L::kSmem, s>>>(tk, tv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const bool sliced = (long long)a.R * p.subs * 8 <= p.ctas;  // items of more than eight parts
  auto join = sliced ? paged_join_kernel<D, FP8, NT, true> : paged_join_kernel<D, FP8, NT, false>;
  const size_t join_smem = (size_t)p.ctas * 2 * 8 * NT * sizeof(float);
  if ((e = sliced ? cross::prepare_kernel<paged_join_kernel<D, FP8, NT, true>>(join_smem)
                  : cross::prepare_kernel<paged_join_kernel<D, FP8, NT, false>>(join_smem)) != cudaSuccess)
    return e;
  return cross::launch_dependent(join, dim3((unsigned)p.ctas, sliced ? D / 16 : 1), dim3(512), join_smem, s,
                                 p);
}

__global__ void paged_clear_kernel(WsHeader* hdr) { hdr->status = 0; }

}  // namespace

size_t paged_attn_plan(int R, int H, int Hkv, int d, int sms, PagedAttnPlan* p) {
  PagedAttnPlan q;
  const int nt = H / Hkv > 8 ? 2 : 1;
  q.info = sizeof(WsHeader);
  q.parts = (q.info + (size_t)sms * sizeof(CtaInfo) + 255) / 256 * 256;
  const size_t part = ((size_t)nt * d / 16 * 128 + 16 * nt) * sizeof(float);
  q.total = q.parts + (size_t)sms * (2 * kMaxWarps + 2) * part;
  if (p) *p = q;
  return q.total;
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  WsHeader* hdr = static_cast<WsHeader*>(a.workspace);
  if (a.R == 0) {
    paged_clear_kernel<<<1, 1, 0, s>>>(hdr);
    return cudaGetLastError();
  }
  const int G = a.H / a.Hkv, nt = G > 8 ? 2 : 1;
  PagedParams p = {};
  p.Q = static_cast<const __nv_bfloat16*>(a.Q);
  p.q_stride = a.q_stride;
  p.R = a.R;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.G = G;
  p.heads = 8 * nt;
  p.chunks = (G + p.heads - 1) / p.heads;
  p.subs = a.Hkv * p.chunks;
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.n_pages = (int)a.n_pages;
  p.log2_page = a.log2_page;
  p.max_pages = a.max_pages;
  p.table = a.table;
  p.seq_lens = a.seq_lens;
  p.window = a.window;
  p.c = a.scale * kLog2e;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.info = reinterpret_cast<CtaInfo*>(ws + a.plan.info);
  p.parts = reinterpret_cast<float*>(ws + a.plan.parts);
  p.status = &hdr->status;
  p.ctas = a.sms;
  p.budget = kDefaultWaitBudget;
  if (a.d == 64) {
    if (a.fp8) return nt == 1 ? launch_t<64, true, 1>(a, p, s) : launch_t<64, true, 2>(a, p, s);
    return nt == 1 ? launch_t<64, false, 1>(a, p, s) : launch_t<64, false, 2>(a, p, s);
  }
  if (a.fp8) return nt == 1 ? launch_t<128, true, 1>(a, p, s) : launch_t<128, true, 2>(a, p, s);
  return nt == 1 ? launch_t<128, false, 1>(a, p, s) : launch_t<128, false, 2>(a, p, s);
}

}  // namespace sa
