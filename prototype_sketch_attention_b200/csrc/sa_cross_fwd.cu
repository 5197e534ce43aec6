// Multi-head cross attention, forward, on tcgen05 (sm_100a).
//
// Per 128-row tile of packed query rows (sa_cross.cuh) and key tile j of 128 rows:
//   S = Q K_j^T (TMEM, fp32),  m = running row maximum,  P = 2^(c (S - m)) as bf16 (TMEM, over S),
//   O += P V_j (TMEM, fp32),   l += row sums of P in fp32,         c = scale log2 e,
// and at the end out = O / l, lse = (c m + log2 l) ln 2. The running maximum is raised only when
// a tile's maximum exceeds it by more than 8 in log2 units (O and l are then rescaled; the
// weights stay below 2^8 otherwise, and bf16 keeps their relative precision at any size).
//
// One CTA works on two tiles (256 rows) of one user and head group, so that each key tile read
// from L2 serves 256 rows (one tile would need 64 bytes a clock of L2 reads against the
// tensor pipe, more than an SM gets), and so that one warpgroup's softmax runs while the
// tensor cores work for the other. When the rows fit in one tile, both warpgroups take that
// tile, on alternate key tiles, with an O, m and l each, merged at the end. When there are fewer
// CTAs than SMs and many keys, `splits` CTAs share a user's key tiles and leave fp32 partials that
// cross_join_kernel puts together in a fixed order.
//
// Roles (384 threads): warp 0 TMA (Q once, then K_0, V_0, K_1, V_1, ... through one ring of
// stages), warp 1 TMEM allocation and every MMA, warp 2 hands V tiles on, zeroing rows that
// the mask or the end of the range drops (weight 0 times NaN must not count), warps 4-11 two
// softmax warpgroups, one thread per row. P stays in TMEM as the A operand of the second MMA.
// Bound: at d = 128 a tile costs 1,024 tensor clocks and 1,024 clocks of exponentials (16 a
// clock and SM); at d = 64 the exponentials bound it.
#include <cmath>

#include "sa_cross.cuh"

namespace sa {
namespace cross {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr float kRaise = 8.f;
// The softmax warpgroups keep a row's 128 scores in registers. setmaxnreg.inc draws on the
// launch's 384 x 168 registers, so the split stays within them, and the launch refuses a build
// compiled to fewer.
constexpr int kRegsLaunch = 168, kRegsControl = 72, kRegsSoftmax = 216;
static_assert(128 * kRegsControl + 256 * kRegsSoftmax <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
__host__ __device__ constexpr uint32_t col_s(int w) { return w ? 128u : 0u; }
__host__ __device__ constexpr uint32_t col_o(int w) { return w ? 384u : 256u; }

template <int D>
struct FSmem {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTile = kBoxes * kBox;
  static constexpr int kNS = D == 128 ? 5 : 8;  // stages: 2 + 5 tiles of 32 KB, or 2 + 8 of 16 KB
  static constexpr int oQ = 0;
  static constexpr int oKV = 2 * kTile;
  static constexpr int oML = oKV + kNS * kTile;  // warpgroup 1's m and l (merge)
  static constexpr int oBars = oML + 2 * 128 * 4;
};

struct FBars {
  uint64_t q_full, full[8], empty[8];
  uint64_t v_ready[8];  // by key tile mod 8: fewer V tiles than that fit in the ring
  uint64_t s_full[2], o_done[2];
  uint64_t p_full[2][2];  // [tile][half of the keys]: the second product starts on the first half
  uint64_t merge, drain;
  uint32_t tmem_base;
};

struct FwdParams {
  const int64_t* qoff;
  const int64_t* koff;
  const Tile* tiles;
  WsHeader* hdr;
  const uint8_t* mask;
  int H, G, PG;          // heads, heads per key head, heads per tile
  int splits;
  float c;               // scale log2 e
  __nv_bfloat16* out;    // [n_q, H, D]
  float* lse;            // [n_q, H]
  float* part_o;         // [splits][n_q, H, D] (splits > 1)
  float* part_lse;       // [splits][n_q, H]
  long long n_q;
  long long budget;
};

// The 128 scores of this thread's row.
__device__ __forceinline__ void load_scores(uint32_t taddr, uint32_t (&s)[4][32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) tmem_ld32_raw(taddr + 32 * i, s[i]);
  tmem_wait_tie(s[0]);
  tie32(s[1]);
  tie32(s[2]);
  tie32(s[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cross_fwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                 const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ FwdParams a) {
  using L = FSmem<D>;
  constexpr int NS = L::kNS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  FBars* bars = reinterpret_cast<FBars*>(smem + L::oBars);
  int* status = &a.hdr->status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars->q_full), 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1);
      mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    for (int s = 0; s < 8; ++s) mbar_init(smem_u32(&bars->v_ready[s]), 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_u32(&bars->s_full[w]), 1);
      mbar_init(smem_u32(&bars->p_full[w][0]), 4);
      mbar_init(smem_u32(&bars->p_full[w][1]), 4);
      mbar_init(smem_u32(&bars->o_done[w]), 1);
    }
    mbar_init(smem_u32(&bars->merge), 4);
    mbar_init(smem_u32(&bars->drain), 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmap_q);
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  griddep_wait();  // the schedule

  const int groups = a.H / a.PG, tokens = 128 / a.PG;  // tokens per tile
  const long long g = blockIdx.x / groups;
  const int hu = (int)(blockIdx.x - g * groups);
  const bool work = g < a.hdr->total_tiles;
  int nkt = 0, j0 = 0, hk = 0, t0 = 0, t1 = 0, k0 = 0, k1 = 0;
  bool two = false;
  if (work) {
    const Tile tl = a.tiles[g];
    t0 = (int)a.qoff[tl.user] + tl.index * 2 * tokens;
    t1 = (int)a.qoff[tl.user + 1];
    k0 = (int)a.koff[tl.user];
    k1 = (int)a.koff[tl.user + 1];
    const int all = (k1 - k0 + 127) / 128;
    j0 = (int)((long long)all * blockIdx.y / a.splits);
    nkt = (int)((long long)all * (blockIdx.y + 1) / a.splits) - j0;
    k0 += j0 * 128;
    two = t1 - t0 > tokens;
    hk = hu * a.PG / a.G;
  }

  // every warp changes its register count inside its role's branch, so that the compiler
  // budgets each role for its count
  if (warp == 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    // ================= TMA
    if (lane == 0 && nkt > 0) {
      const uint32_t qf = smem_u32(&bars->q_full);
      mbar_arrive_expect_tx(qf, (two ? 2 : 1) * L::kTile);
      for (int w = 0; w < (two ? 2 : 1); ++w)
        for (int b = 0; b < L::kBoxes; ++b)
          tma_load_3d(sbase + L::oQ + w * L::kTile + b * kBox, &tmap_q, b * 64, hu * a.PG,
                      t0 + w * tokens, qf);
      int i = 0;
      for (; i < 2 * nkt; ++i) {
        const int st = i % NS;
        if (!mbar_wait(smem_u32(&bars->empty[st]), (uint32_t)(((i / NS) & 1) ^ 1), status, a.budget)) break;
        const uint32_t fb = smem_u32(&bars->full[st]);
        mbar_arrive_expect_tx(fb, L::kTile);
        for (int b = 0; b < L::kBoxes; ++b)
          tma_load_3d(sbase + L::oKV + st * L::kTile + b * kBox, (i & 1) ? &tmap_v : &tmap_k, b * 64, hk,
                      k0 + 128 * (i >> 1), fb);
      }
      for (int x = (i > NS ? i - NS : 0); x < i; ++x)
        mbar_wait_drain(smem_u32(&bars->full[x % NS]), (uint32_t)((x / NS) & 1), a.budget);
      mbar_wait_drain(qf, 0, a.budget);
    }
  } else if (warp == 1) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    // ================= MMAs. Tile w's order is S_w(0), [O_w(j), S_w(j + 1)]...: P_w(j) lies over
    // S_w(j), and the pipe runs a thread's MMAs in order, so S_w(j + 1) overwrites it only
    // after O_w(j) has read it.
    if (lane == 0 && nkt > 0) {
      const uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0);
      const uint32_t id_o = idesc_bf16_f32(128, D, 0, 1);
      bool ok = mbar_wait(smem_u32(&bars->q_full), 0, status, a.budget);
      auto scores = [&](int w, int j) {  // S_w = Q_w K_j^T
        const int i = 2 * j, st = i % NS;
        ok = ok && mbar_wait(smem_u32(&bars->full[st]), (uint32_t)((i / NS) & 1), status, a.budget);
        if (!ok) return;
        tc_fence_after();
        const uint64_t dq = smem_desc(sbase + L::oQ + (two ? w : 0) * L::kTile, 16, 1024, kSwizzle128B);
        const uint64_t dk = smem_desc(sbase + L::oKV + st * L::kTile, 16, 1024, kSwizzle128B);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma_f16(tmem + col_s(w), dq + kstep(ks), dk + kstep(ks), id_s, ks > 0 ? 1u : 0u);
        tc_commit(smem_u32(&bars->s_full[w]));
        if (!two || w == 1) tc_commit(smem_u32(&bars->empty[st]));
      };
      auto output = [&](int w, int j, int n) {  // O_w += P_w V_j; n: this tile's n-th key tile
        const int i = 2 * j + 1, st = i % NS;
        ok = ok && mbar_wait(smem_u32(&bars->v_ready[j & 7]), (uint32_t)((j >> 3) & 1), status, a.budget);
        const uint64_t dv = smem_desc(sbase + L::oKV + st * L::kTile, kBox, 1024, kSwizzle128B);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ok = ok && mbar_wait(smem_u32(&bars->p_full[w][h]), (uint32_t)(n & 1), status, a.budget);
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
            tc_mma_f16_ts(tmem + col_o(w), tmem + col_s(w) + 8 * ks, dv + (uint64_t)((ks * 2048) >> 4),
                          id_o, (n > 0 || ks > 0) ? 1u : 0u);
        }
        tc_commit(smem_u32(&bars->o_done[w]));
        if (!two || w == 1) tc_commit(smem_u32(&bars->empty[st]));
      };
      if (two) {
        scores(0, 0);
        scores(1, 0);
        for (int j = 0; ok && j < nkt; ++j)
          for (int w = 0; w < 2; ++w) {
            output(w, j, j);
            if (j + 1 < nkt) scores(w, j + 1);
          }
      } else {
        scores(0, 0);
        if (nkt > 1) scores(1, 1);
        for (int j = 0; ok && j < nkt; ++j) {
          output(j & 1, j, j >> 1);
          if (j + 2 < nkt) scores(j & 1, j + 2);
        }
      }
      tc_commit(smem_u32(&bars->drain));
      mbar_wait_drain(smem_u32(&bars->drain), 0, a.budget);
    }
  } else if (warp == 2) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    // ================= V tiles: zero the dropped rows
    MaskBytes mb;
    if (nkt > 0) mb.load(a.mask, k0, k1, lane);
    for (int j = 0; j < nkt; ++j) {
      const int i = 2 * j + 1, st = i % NS;
      uint32_t keep[4];
      const bool drop = mb.vote(a.mask, k0 + 128 * j, k1, lane, keep);
      if (j + 1 < nkt) mb.load(a.mask, k0 + 128 * (j + 1), k1, lane);
      if (!mbar_wait_warp(smem_u32(&bars->full[st]), (uint32_t)((i / NS) & 1), status, a.budget)) break;
      if (drop) {
        zero_rows(smem + L::oKV + st * L::kTile, L::kBoxes, keep, lane);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->v_ready[j & 7]));
    }
  } else if (warp == 3) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ================= softmax warpgroup w: tile w, or alternate key tiles of the only tile
    const int w = (warp - 4) >> 2;
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t st = tmem + lane_off + col_s(w), ot = tmem + lane_off + col_o(w);
    const int step = two ? 1 : 2, first = two ? 0 : w;
    const float c = a.c;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    int n = 0;
    MaskBytes mb;
    if (first < nkt) mb.load(a.mask, k0 + 128 * first, k1, lane);
    for (int j = first; j < nkt; j += step, ++n) {
      uint32_t keep[4];
      const bool drop = mb.vote(a.mask, k0 + 128 * j, k1, lane, keep);
      if (j + step < nkt) mb.load(a.mask, k0 + 128 * (j + step), k1, lane);
      if (!mbar_wait_warp(smem_u32(&bars->s_full[w]), (uint32_t)(n & 1), status, a.budget)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t s[4][32];
      load_scores(st, s);
      if (drop) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (!((keep[i] >> x) & 1u)) s[i][x] = 0xff800000u;  // -inf
      }
      float mx[4];  // four chains: the maximum is on the way to everything else
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mx[i] = fmaxf(__uint_as_float(s[i][0]), __uint_as_float(s[i][1]));
#pragma unroll
        for (int x = 2; x < 32; x += 2)
          mx[i] = fmax3(mx[i], __uint_as_float(s[i][x]), __uint_as_float(s[i][x + 1]));
      }
      const float mt = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
      const bool raise = (mt - m) * c > kRaise;  // false for -inf - -inf
      if (__any_sync(0xffffffffu, raise)) {
        const float f = raise ? ex2_approx((m - mt) * c) : 1.f;  // 0 for the first maximum
        if (n > 0) {
          // O_w holds every tile before this one once its last MMA has completed
          if (!mbar_wait_warp(smem_u32(&bars->o_done[w]), (uint32_t)((n - 1) & 1), status, a.budget)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < D; x += 16) {
            uint32_t o[16];
            tmem_ld16(ot + x, o);
            tmem_wait16(o);
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
            tmem_st16(ot + x, o);
          }
        }
        l *= f;
        if (raise) m = mt;
      }
      const float mc = m == -INFINITY ? 0.f : m * c;
      float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const float p0 = ex2_approx(fmaf(__uint_as_float(s[2 * h + (x >> 4)][(2 * x) & 31]), c, -mc));
          const float p1 = ex2_approx(fmaf(__uint_as_float(s[2 * h + (x >> 4)][(2 * x + 1) & 31]), c, -mc));
          ls[x & 3] += p0 + p1;
          pk[x] = cvt_bf16x2(p0, p1);
        }
        tmem_st32(st + 32 * h, pk);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[w][h]));
      }
      l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
    }
    // ---- this tile's (or half's) accumulator is complete
    if (ok && n > 0)
      ok = mbar_wait_warp(smem_u32(&bars->o_done[w]), (uint32_t)((n - 1) & 1), status, a.budget);
    tc_fence_after();
    float* ml = reinterpret_cast<float*>(smem + L::oML);
    float g0 = 1.f, g1 = 0.f;  // factors of O_0 and O_1 (two tiles: of this tile's own)
    bool write = work;
    if (!two) {
      if (w == 1) {
        ml[r] = m;
        ml[128 + r] = ok ? l : 0.f;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->merge));
        write = false;
      } else {
        const bool merged = mbar_wait_warp(smem_u32(&bars->merge), 0, status, a.budget);
        tc_fence_after();
        const float m1 = ml[r], l1 = merged ? ml[128 + r] : 0.f;
        const float mm = fmaxf(m, m1);
        g0 = l > 0.f ? ex2_approx((m - mm) * c) : 0.f;
        g1 = l1 > 0.f ? ex2_approx((m1 - mm) * c) : 0.f;
        l = l * g0 + l1 * g1;
        m = mm;
      }
    }
    const int t = t0 + (two ? w * tokens : 0) + r / a.PG;
    write = write && t < t1;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    g0 *= inv;
    g1 *= inv;
    const long long row = (long long)t * a.H + hu * a.PG + r % a.PG;
    const float lse = l > 0.f ? (m * c + lg2_approx(l)) * kLn2 : -INFINITY;
    if (a.splits > 1) {
      float* po = a.part_o + ((long long)blockIdx.y * a.n_q * a.H + row) * D;
      if (write) a.part_lse[(long long)blockIdx.y * a.n_q * a.H + row] = lse;
      if (nkt > 0 && work && (two || w == 0)) {
#pragma unroll 1
        for (int x = 0; x < D; x += 16) {
          uint32_t o[16], o1[16];
          tmem_ld16(ot + x, o);
          if (!two && nkt > 1) tmem_ld16(tmem + lane_off + col_o(1) + x, o1);
          tmem_wait16(o);
          if (!two && nkt > 1) tmem_wait16(o1);
          if (write) {
#pragma unroll
            for (int y = 0; y < 16; y += 4) {
              float v[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                v[z] = __uint_as_float(o[y + z]) * g0;
                if (!two && nkt > 1) v[z] = fmaf(__uint_as_float(o1[y + z]), g1, v[z]);
              }
              *reinterpret_cast<float4*>(po + x + y) = make_float4(v[0], v[1], v[2], v[3]);
            }
          }
        }
      }
    } else if (work && (two || w == 0)) {
      if (write) a.lse[row] = lse;
      __nv_bfloat16* po = a.out + row * D;
#pragma unroll 1
      for (int x = 0; x < D; x += 16) {
        uint32_t o[16], o1[16];
        if (nkt > 0) {
          tmem_ld16(ot + x, o);
          if (!two && nkt > 1) tmem_ld16(tmem + lane_off + col_o(1) + x, o1);
          tmem_wait16(o);
          if (!two && nkt > 1) tmem_wait16(o1);
        }
        if (write) {
          uint32_t pk[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            float v0 = 0.f, v1 = 0.f;
            if (nkt > 0) {
              v0 = __uint_as_float(o[2 * y]) * g0;
              v1 = __uint_as_float(o[2 * y + 1]) * g0;
              if (!two && nkt > 1) {
                v0 = fmaf(__uint_as_float(o1[2 * y]), g1, v0);
                v1 = fmaf(__uint_as_float(o1[2 * y + 1]), g1, v1);
              }
            }
            pk[y] = cvt_bf16x2(v0, v1);
          }
          *reinterpret_cast<uint4*>(po + x) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          *reinterpret_cast<uint4*>(po + x + 8) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// out = sum_s w_s O_s, w_s = exp(lse_s - lse), over the splits' normalised partials, in order.
// One warp per row; a split that saw no key (lse = -inf) left no O.
template <int D>
__global__ void __launch_bounds__(256) cross_join_kernel(const float* __restrict__ part_o,
                                                         const float* __restrict__ part_lse,
                                                         int splits, const int64_t* qoff, int R,
                                                         long long n_q, int H,
                                                         const WsHeader* hdr,
                                                         __nv_bfloat16* __restrict__ out,
                                                         float* __restrict__ lse_out) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long row = blockIdx.x * 8LL + (threadIdx.x >> 5), rows = n_q * H;
  if (read_status(&hdr->status) != 0 || row >= qoff[R] * H) return;
  float m = -INFINITY;
  for (int s = 0; s < splits; ++s) m = fmaxf(m, part_lse[s * rows + row]);
  float l = 0.f, o[D / 32];
#pragma unroll
  for (int x = 0; x < D / 32; ++x) o[x] = 0.f;
  if (m > -INFINITY) {
    for (int s = 0; s < splits; ++s) {
      const float ls = part_lse[s * rows + row];
      if (ls == -INFINITY) continue;
      const float wgt = ex2_approx((ls - m) * kLog2e);
      l += wgt;
      const float* po = part_o + (s * rows + row) * D;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) o[x] = fmaf(wgt, po[lane + 32 * x], o[x]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int x = 0; x < D / 32; ++x) out[row * D + lane + 32 * x] = __float2bfloat16(o[x] * inv);
  if (lane == 0) lse_out[row] = l > 0.f ? m + lg2_approx(l) * kLn2 : -INFINITY;
}

template <int D>
cudaError_t launch_t(const CrossArgs& a, const CrossGeo& geo, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  CUtensorMap tq, tk, tv;
  if (!tmap_heads(&tq, a.Q, a.n_q, a.H, D, a.q_stride, geo.pg, 128 / geo.pg) ||
      !tmap_heads(&tk, a.K, a.n_kv, a.Hkv, D, a.k_stride, 1, 128) ||
      !tmap_heads(&tv, a.V, a.n_kv, a.Hkv, D, a.v_stride, 1, 128))
    return cudaErrorInvalidValue;
  FwdParams p = {};
  p.qoff = a.qoff;
  p.koff = a.koff;
  p.tiles = reinterpret_cast<const Tile*>(ws + a.plan.qtiles);
  p.hdr = reinterpret_cast<WsHeader*>(ws + a.plan.hdr);
  p.mask = a.mask;
  p.H = a.H;
  p.G = a.H / a.Hkv;
  p.PG = geo.pg;
  p.splits = geo.splits;
  p.c = a.scale * kLog2e;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.part_o = reinterpret_cast<float*>(ws + a.plan.part_o);
  p.part_lse = reinterpret_cast<float*>(ws + a.plan.part_lse);
  p.n_q = a.n_q;
  p.budget = kDefaultWaitBudget;
  constexpr size_t smem = 1024 + FSmem<D>::oBars + sizeof(FBars);
  static_assert(smem <= 227 * 1024, "shared memory");
  cudaError_t e = prepare_kernel<cross_fwd_kernel<D>>(smem, kRegsLaunch);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(geo.pair_tiles * (a.H / geo.pg)), (unsigned)geo.splits);
  if ((e = launch_dependent(cross_fwd_kernel<D>, grid, dim3(kThreads), smem, s, tq, tk, tv, p)) != cudaSuccess)
    return e;
  if (geo.splits == 1) return cudaSuccess;
  return launch_dependent(cross_join_kernel<D>, dim3((unsigned)((a.n_q * a.H + 7) / 8)), dim3(256), 0, s,
                          (const float*)p.part_o, (const float*)p.part_lse, geo.splits, a.qoff, a.R,
                          a.n_q, a.H, (const WsHeader*)p.hdr, p.out, p.lse);
}

}  // namespace

cudaError_t launch_fwd(const CrossArgs& a, const CrossGeo& geo, cudaStream_t s) {
  return a.d == 64 ? launch_t<64>(a, geo, s) : launch_t<128>(a, geo, s);
}

}  // namespace cross
}  // namespace sa
