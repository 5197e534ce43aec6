// Multi-head cross attention, backward, on tcgen05 (sm_100a).
//
// With P = 2^(c S - lse2), c = scale log2 e, and delta = dout . out (made before this kernel):
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q.
// dQ sums over keys, dK and dV over queries and over the heads that share the key head. One
// pass that makes all three would have to add a 64 KB fp32 block of dQ per pair of tiles in global
// memory (about 6,000 clocks of L2 reductions on this GPU against 2,560 of tensor work, and an
// order that changes from run to run). So the grid has two kinds of CTA, each of which owns its
// output and keeps it in TMEM, at 7 products a pair of tiles in place of 5 and no atomics:
//   dK/dV CTA: a tile of 128 keys of one key head walks the user's packed query tiles (of every
//     head group that shares it). S^T = K Q^T and dP^T = V dO^T put keys on the TMEM lanes,
//     so P^T and dS^T, written as bf16 over S^T and dP^T, are the A operands in place:
//     dV += P^T dO, dK += dS^T Q. The rows' lse2 and delta run along the columns and come from
//     shared memory as broadcasts.
//   dQ CTA: a tile of 128 packed query rows walks the user's key tiles: S = Q K^T (two
//     buffers), dP = dO V^T, dS over S, dQ += dS K. When there are fewer such CTAs than SMs and
//     many keys, `splits` of them share a tile and leave fp32 partials, summed in order.
// Roles (384 threads): warp 0 TMA, warp 1 TMEM allocation and every MMA, warp 2 hands tiles on:
// it zeroes the rows that an MMA would multiply by 0 but must not read (dropped keys, rows past
// the user's end), and loads lse2 and delta; warps 4-11 two warpgroups for the elementwise
// step, 64 columns each, one thread per row. Within a CTA the tensor pipe runs ahead of the
// elementwise step: dK/dV: S(0) dP(0) | dV(i) S(i+1) | dK(i) dP(i+1) | ..., so the exponentials of
// tile i + 1 run while dK(i) and dP(i + 1) do; dQ: S(j + 1) while tile j is in the elementwise
// step, then dP(j + 1), dQ(j), S(j + 2).
// Bound at d = 128: 2,048 tensor clocks a pair of tiles in a dK/dV CTA, 1,536 in a dQ CTA, 1,024
// clocks of exponentials in both.
#include <cmath>

#include "sa_cross.cuh"

namespace sa {
namespace cross {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr int kRegsLaunch = 168, kRegsControl = 72, kRegsElem = 216;  // setmaxnreg draws on the launch's
static_assert(128 * kRegsControl + 256 * kRegsElem <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");

template <int D>
struct BSmem {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTile = kBoxes * kBox;
  static constexpr int kNS = D == 128 ? 5 : 8;  // ring stages of a dQ CTA
  static constexpr int kNSKv = kNS - 1;         // and of a dK/dV CTA, which has (lse2, delta) in the last
  static constexpr int oA = 0;                  // the CTA's own tile: K, V (dK/dV) or Q, dO (dQ)
  static constexpr int oRing = 2 * kTile;       // Q_i, dO_i, ... or K_j, V_j, ...
  static constexpr int oStat = oRing + kNSKv * kTile;  // 4 x 128 (lse2, delta)
  static constexpr int oBars = oRing + kNS * kTile;
  static_assert(4 * 128 * 8 <= kTile, "the statistics fit in one stage");
};

struct BBars {
  uint64_t own, full[8], empty[8];
  uint64_t ready[8];    // by tile number mod 8: fewer tile pairs than that fit in the ring
  uint64_t s_full[2], dp_full, p_full, ds_full, done;
  uint32_t tmem_base;
};

struct BwdParams {
  const int64_t* qoff;
  const int64_t* koff;
  const Tile* qtiles;      // pairs of query tiles
  const Tile* ktiles;
  WsHeader* hdr;
  const uint8_t* mask;
  const float2* stats;     // [H / PG][n_q PG] (lse2, delta)
  int H, Hkv, G, PG;
  int splits;
  long long kv_ctas;       // CTAs [0, kv_ctas) are dK/dV CTAs
  float c, scale;
  __nv_bfloat16 *dQ, *dK, *dV;
  float* part;             // [splits][n_q, H, D] (splits > 1)
  long long n_q;
  long long budget;
};

__device__ __forceinline__ uint64_t mn_step(int ks) { return (uint64_t)((ks * 2048) >> 4); }

// A row of D fp32 TMEM columns, times f, to bf16 (zero: what the accumulator holds is not used).
template <int COLS>
__device__ __forceinline__ void write_row(uint32_t taddr, bool have, bool write, bool zero, float f,
                                          __nv_bfloat16* row) {
#pragma unroll 1
  for (int x = 0; x < COLS; x += 16) {
    uint32_t o[16];
    if (have) {
      tmem_ld16(taddr + x, o);
      tmem_wait16(o);
    }
    if (write) {
      uint32_t pk[8];
#pragma unroll
      for (int y = 0; y < 8; ++y)
        pk[y] = zero || !have ? 0u
                              : cvt_bf16x2(__uint_as_float(o[2 * y]) * f, __uint_as_float(o[2 * y + 1]) * f);
      *reinterpret_cast<uint4*>(row + x) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      *reinterpret_cast<uint4*>(row + x + 8) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
    }
  }
}

// ---------------------------------------------------------------- dK and dV of a key tile
template <int D>
__device__ __forceinline__ void dkv_cta(const CUtensorMap* tmap_q, const CUtensorMap* tmap_do,
                                        const CUtensorMap* tmap_k, const CUtensorMap* tmap_v,
                                        const BwdParams& a, uint8_t* smem, uint32_t tmem) {
  using L = BSmem<D>;
  constexpr int NS = L::kNSKv;
  constexpr uint32_t cS = 0, cP = 128, cDV = 256, cDK = 384;
  const uint32_t sbase = smem_u32(smem);
  BBars* bars = reinterpret_cast<BBars*>(smem + L::oBars);
  int* status = &a.hdr->status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const long long g = blockIdx.x / a.Hkv;
  const int hk = (int)(blockIdx.x - g * a.Hkv), tokens = 128 / a.PG;
  const bool work = g < a.hdr->pad[0];
  int k0 = 0, k1 = 0, q0 = 0, q1 = 0, nqt = 0, n = 0;
  if (work) {
    const Tile tl = a.ktiles[g];
    k0 = (int)a.koff[tl.user] + tl.index * 128;
    k1 = (int)a.koff[tl.user + 1];
    q0 = (int)a.qoff[tl.user];
    q1 = (int)a.qoff[tl.user + 1];
    nqt = (q1 - q0 + tokens - 1) / tokens;
    n = nqt * (a.G / a.PG);  // (head group, query tile) steps
  }
  const int hu0 = hk * (a.G / a.PG);

  if (warp == 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (lane == 0 && n > 0) {
      const uint32_t ob = smem_u32(&bars->own);
      mbar_arrive_expect_tx(ob, 2 * L::kTile);
      for (int b = 0; b < L::kBoxes; ++b) {
        tma_load_3d(sbase + L::oA + b * kBox, tmap_k, b * 64, hk, k0, ob);
        tma_load_3d(sbase + L::oA + L::kTile + b * kBox, tmap_v, b * 64, hk, k0, ob);
      }
      int x = 0, grp = 0, qt = 0;
      for (; x < 2 * n; ++x) {
        const int st = x % NS;
        if (!mbar_wait(smem_u32(&bars->empty[st]), (uint32_t)(((x / NS) & 1) ^ 1), status, a.budget)) break;
        const uint32_t fb = smem_u32(&bars->full[st]);
        mbar_arrive_expect_tx(fb, L::kTile);
        for (int b = 0; b < L::kBoxes; ++b)
          tma_load_3d(sbase + L::oRing + st * L::kTile + b * kBox, (x & 1) ? tmap_do : tmap_q, b * 64,
                      (hu0 + grp) * a.PG, q0 + qt * tokens, fb);
        if ((x & 1) && ++qt == nqt) {
          qt = 0;
          ++grp;
        }
      }
      for (int y = (x > NS ? x - NS : 0); y < x; ++y)
        mbar_wait_drain(smem_u32(&bars->full[y % NS]), (uint32_t)((y / NS) & 1), a.budget);
      mbar_wait_drain(ob, 0, a.budget);
    }
  } else if (warp == 1) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (lane == 0 && n > 0) {
      const uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0), id_o = idesc_bf16_f32(128, D, 0, 1);
      const uint64_t dk = smem_desc(sbase + L::oA, 16, 1024, kSwizzle128B);
      const uint64_t dv = smem_desc(sbase + L::oA + L::kTile, 16, 1024, kSwizzle128B);
      bool ok = mbar_wait(smem_u32(&bars->own), 0, status, a.budget);
      auto ring = [&](int x) { return sbase + L::oRing + (x % NS) * L::kTile; };
      auto scores = [&](int i) {  // S^T = K Q_i^T
        ok = ok && mbar_wait(smem_u32(&bars->ready[i & 7]), (uint32_t)((i >> 3) & 1), status, a.budget);
        if (!ok) return;
        tc_fence_after();
        const uint64_t dq = smem_desc(ring(2 * i), 16, 1024, kSwizzle128B);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma_f16(tmem + cS, dk + kstep(ks), dq + kstep(ks), id_s, ks > 0 ? 1u : 0u);
        tc_commit(smem_u32(&bars->s_full[0]));
      };
      auto dprob = [&](int i) {  // dP^T = V dO_i^T
        const uint64_t ddo = smem_desc(ring(2 * i + 1), 16, 1024, kSwizzle128B);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma_f16(tmem + cP, dv + kstep(ks), ddo + kstep(ks), id_s, ks > 0 ? 1u : 0u);
        tc_commit(smem_u32(&bars->dp_full));
      };
      scores(0);
      if (ok) dprob(0);
      for (int i = 0; ok && i < n; ++i) {
        ok = mbar_wait(smem_u32(&bars->p_full), (uint32_t)(i & 1), status, a.budget);
        if (!ok) break;
        tc_fence_after();
        // dV += P^T dO_i; the packed P^T of warpgroup w's queries starts at column 64 w
        const uint64_t ddo = smem_desc(ring(2 * i + 1), kBox, 1024, kSwizzle128B);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc_mma_f16_ts(tmem + cDV, tmem + cS + 64 * (ks >> 2) + 8 * (ks & 3), ddo + mn_step(ks), id_o,
                        (i > 0 || ks > 0) ? 1u : 0u);
        tc_commit(smem_u32(&bars->empty[(2 * i + 1) % NS]));
        if (i + 1 < n) scores(i + 1);  // overwrites P^T after the MMAs above, in order
        ok = ok && mbar_wait(smem_u32(&bars->ds_full), (uint32_t)(i & 1), status, a.budget);
        if (!ok) break;
        tc_fence_after();
        const uint64_t dq = smem_desc(ring(2 * i), kBox, 1024, kSwizzle128B);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc_mma_f16_ts(tmem + cDK, tmem + cP + 64 * (ks >> 2) + 8 * (ks & 3), dq + mn_step(ks), id_o,
                        (i > 0 || ks > 0) ? 1u : 0u);
        tc_commit(smem_u32(&bars->empty[(2 * i) % NS]));
        if (i + 1 < n) dprob(i + 1);
      }
      tc_commit(smem_u32(&bars->done));
      mbar_wait_drain(smem_u32(&bars->done), 0, a.budget);
    }
  } else if (warp == 2) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    // ================= lse2 and delta of the tile's rows; rows past the user's end: weight 0,
    // and zeros in the Q and dO tiles
    float2* stat = reinterpret_cast<float2*>(smem + L::oStat);
    int grp = 0, qt = 0;
    for (int i = 0; i < n; ++i) {
      const int t = q0 + qt * tokens, rows = min(128, (q1 - t) * a.PG);
      const float2* src = a.stats + ((long long)(hu0 + grp) * a.n_q + t) * a.PG;
      float2 v[4];
#pragma unroll
      for (int y = 0; y < 4; ++y)
        v[y] = lane + 32 * y < rows ? src[lane + 32 * y] : make_float2(INFINITY, 0.f);
      bool ok = true;
      for (int x = 2 * i; x < 2 * i + 2; ++x)
        ok = ok && mbar_wait_warp(smem_u32(&bars->full[x % NS]), (uint32_t)((x / NS) & 1), status, a.budget);
      if (!ok) break;
      if (rows < 128) {
        uint32_t keep[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          keep[y] = rows >= 32 * y + 32 ? ~0u : rows > 32 * y ? (1u << (rows - 32 * y)) - 1u : 0u;
        zero_rows(smem + L::oRing + ((2 * i) % NS) * L::kTile, L::kBoxes, keep, lane);
        zero_rows(smem + L::oRing + ((2 * i + 1) % NS) * L::kTile, L::kBoxes, keep, lane);
        fence_proxy_async_smem();
      }
      // slot i mod 4 was last read for step i - 4, whose tiles left the ring long ago
#pragma unroll
      for (int y = 0; y < 4; ++y) stat[(i & 3) * 128 + lane + 32 * y] = v[y];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->ready[i & 7]));
      if (++qt == nqt) {
        qt = 0;
        ++grp;
      }
    }
  } else if (warp == 3) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsElem));
    // ================= elementwise: thread = key row, warpgroup w = queries [64 w, 64 w + 64)
    const int w = (warp - 4) >> 2, q4 = warp & 3, r = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t ts = tmem + lane_off + cS + 64 * w, tp = tmem + lane_off + cP + 64 * w;
    const float4* stat = reinterpret_cast<const float4*>(smem + L::oStat);  // two rows each
    const float c = a.c;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      if (!mbar_wait_warp(smem_u32(&bars->ready[i & 7]), (uint32_t)((i >> 3) & 1), status, a.budget) ||
          !mbar_wait_warp(smem_u32(&bars->s_full[0]), (uint32_t)(i & 1), status, a.budget)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float4* st = stat + (i & 3) * 64 + 32 * w;
      uint32_t s[2][32];
      tmem_ld32_raw(ts, s[0]);
      tmem_ld32_raw(ts + 32, s[1]);
      tmem_wait_tie(s[0]);
      tie32(s[1]);
      uint32_t pk[32];
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        const float4 f = st[x];
        uint32_t& a0 = s[x >> 4][(2 * x) & 31];
        uint32_t& a1 = s[x >> 4][(2 * x + 1) & 31];
        const float p0 = ex2_approx(fmaf(__uint_as_float(a0), c, -f.x));
        const float p1 = ex2_approx(fmaf(__uint_as_float(a1), c, -f.z));
        a0 = __float_as_uint(p0);
        a1 = __float_as_uint(p1);
        pk[x] = cvt_bf16x2(p0, p1);
      }
      tmem_st32(ts, pk);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->p_full));
      if (!mbar_wait_warp(smem_u32(&bars->dp_full), (uint32_t)(i & 1), status, a.budget)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t dp[32];
        tmem_ld32_raw(tp + 32 * h, dp);
        tmem_wait_tie(dp);
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float4 f = st[16 * h + x];
          pk[16 * h + x] = cvt_bf16x2(__uint_as_float(s[h][2 * x]) * (__uint_as_float(dp[2 * x]) - f.y),
                                      __uint_as_float(s[h][2 * x + 1]) * (__uint_as_float(dp[2 * x + 1]) - f.w));
        }
      }
      tmem_st32(tp, pk);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->ds_full));
    }
    // ---- warpgroup 0 writes dV, warpgroup 1 dK; a dropped key row gets 0
    const bool have = ok && n > 0 && mbar_wait_warp(smem_u32(&bars->done), 0, status, a.budget);
    tc_fence_after();
    const int j = k0 + r;
    const bool write = work && j < k1;
    const bool zero = write && a.mask && a.mask[j] == 0;
    write_row<D>(tmem + lane_off + (w ? cDK : cDV), have, write, zero, w ? a.scale : 1.f,
                 (w ? a.dK : a.dV) + ((long long)j * a.Hkv + hk) * D);
  }
}

// ---------------------------------------------------------------- dQ of a query tile
template <int D>
__device__ __forceinline__ void dq_cta(const CUtensorMap* tmap_q, const CUtensorMap* tmap_do,
                                       const CUtensorMap* tmap_k, const CUtensorMap* tmap_v,
                                       const BwdParams& a, uint8_t* smem, uint32_t tmem) {
  using L = BSmem<D>;
  constexpr int NS = L::kNS;
  constexpr uint32_t cP = 256, cDQ = 384;  // S buffers at 0 and 128
  const uint32_t sbase = smem_u32(smem);
  BBars* bars = reinterpret_cast<BBars*>(smem + L::oBars);
  int* status = &a.hdr->status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // CTA -> (tile of a pair, head group, split), the group fastest: neighbours share keys in L2
  const int groups = a.H / a.PG, tokens = 128 / a.PG;
  long long b = blockIdx.x - a.kv_ctas;
  const int hu = (int)(b % groups);
  b /= groups;
  const int half = (int)(b & 1);
  b >>= 1;
  const int split = (int)(b % a.splits);
  const long long g = b / a.splits;
  bool work = g < a.hdr->total_tiles;
  int t0 = 0, t1 = 0, k0 = 0, k1 = 0, n = 0;
  if (work) {
    const Tile tl = a.qtiles[g];
    t0 = (int)a.qoff[tl.user] + (tl.index * 2 + half) * tokens;
    t1 = (int)a.qoff[tl.user + 1];
    work = t0 < t1;
    k0 = (int)a.koff[tl.user];
    k1 = (int)a.koff[tl.user + 1];
    const int all = (k1 - k0 + 127) / 128;
    const int j0 = (int)((long long)all * split / a.splits);
    n = work ? (int)((long long)all * (split + 1) / a.splits) - j0 : 0;
    k0 += j0 * 128;
  }
  const int hk = hu * a.PG / a.G;

  if (warp == 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (lane == 0 && n > 0) {
      const uint32_t ob = smem_u32(&bars->own);
      mbar_arrive_expect_tx(ob, 2 * L::kTile);
      for (int bx = 0; bx < L::kBoxes; ++bx) {
        tma_load_3d(sbase + L::oA + bx * kBox, tmap_q, bx * 64, hu * a.PG, t0, ob);
        tma_load_3d(sbase + L::oA + L::kTile + bx * kBox, tmap_do, bx * 64, hu * a.PG, t0, ob);
      }
      int x = 0;
      for (; x < 2 * n; ++x) {
        const int st = x % NS;
        if (!mbar_wait(smem_u32(&bars->empty[st]), (uint32_t)(((x / NS) & 1) ^ 1), status, a.budget)) break;
        const uint32_t fb = smem_u32(&bars->full[st]);
        mbar_arrive_expect_tx(fb, L::kTile);
        for (int bx = 0; bx < L::kBoxes; ++bx)
          tma_load_3d(sbase + L::oRing + st * L::kTile + bx * kBox, (x & 1) ? tmap_v : tmap_k, bx * 64, hk,
                      k0 + 128 * (x >> 1), fb);
      }
      for (int y = (x > NS ? x - NS : 0); y < x; ++y)
        mbar_wait_drain(smem_u32(&bars->full[y % NS]), (uint32_t)((y / NS) & 1), a.budget);
      mbar_wait_drain(ob, 0, a.budget);
    }
  } else if (warp == 1) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (lane == 0 && n > 0) {
      const uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0), id_o = idesc_bf16_f32(128, D, 0, 1);
      const uint64_t dq = smem_desc(sbase + L::oA, 16, 1024, kSwizzle128B);
      const uint64_t ddo = smem_desc(sbase + L::oA + L::kTile, 16, 1024, kSwizzle128B);
      bool ok = mbar_wait(smem_u32(&bars->own), 0, status, a.budget);
      auto ring = [&](int x) { return sbase + L::oRing + (x % NS) * L::kTile; };
      auto scores = [&](int j) {  // S = Q K_j^T into buffer j mod 2
        ok = ok && mbar_wait(smem_u32(&bars->ready[j & 7]), (uint32_t)((j >> 3) & 1), status, a.budget);
        if (!ok) return;
        tc_fence_after();
        const uint64_t dk = smem_desc(ring(2 * j), 16, 1024, kSwizzle128B);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma_f16(tmem + 128 * (j & 1), dq + kstep(ks), dk + kstep(ks), id_s, ks > 0 ? 1u : 0u);
        tc_commit(smem_u32(&bars->s_full[j & 1]));
      };
      auto dprob = [&](int j) {  // dP = dO V_j^T
        const int x = 2 * j + 1;
        ok = ok && mbar_wait(smem_u32(&bars->full[x % NS]), (uint32_t)((x / NS) & 1), status, a.budget);
        if (!ok) return;
        tc_fence_after();
        const uint64_t dv = smem_desc(ring(x), 16, 1024, kSwizzle128B);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma_f16(tmem + cP, ddo + kstep(ks), dv + kstep(ks), id_s, ks > 0 ? 1u : 0u);
        tc_commit(smem_u32(&bars->dp_full));
        tc_commit(smem_u32(&bars->empty[x % NS]));
      };
      scores(0);
      dprob(0);
      if (n > 1) scores(1);
      for (int j = 0; ok && j < n; ++j) {
        ok = mbar_wait(smem_u32(&bars->ds_full), (uint32_t)(j & 1), status, a.budget);
        if (!ok) break;
        tc_fence_after();
        if (j + 1 < n) dprob(j + 1);  // dP(j) has been read
        if (!ok) break;
        const uint64_t dk = smem_desc(ring(2 * j), kBox, 1024, kSwizzle128B);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc_mma_f16_ts(tmem + cDQ, tmem + 128 * (j & 1) + 64 * (ks >> 2) + 8 * (ks & 3), dk + mn_step(ks),
                        id_o, (j > 0 || ks > 0) ? 1u : 0u);
        tc_commit(smem_u32(&bars->empty[(2 * j) % NS]));
        if (j + 2 < n) scores(j + 2);  // overwrites dS(j) after the MMAs above, in order
      }
      tc_commit(smem_u32(&bars->done));
      mbar_wait_drain(smem_u32(&bars->done), 0, a.budget);
    }
  } else if (warp == 2) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    // ================= K tiles: zero the dropped rows (dS = 0 meets them in dQ)
    MaskBytes mb;
    if (n > 0) mb.load(a.mask, k0, k1, lane);
    for (int j = 0; j < n; ++j) {
      uint32_t keep[4];
      const bool drop = mb.vote(a.mask, k0 + 128 * j, k1, lane, keep);
      if (j + 1 < n) mb.load(a.mask, k0 + 128 * (j + 1), k1, lane);
      const int x = 2 * j;
      if (!mbar_wait_warp(smem_u32(&bars->full[x % NS]), (uint32_t)((x / NS) & 1), status, a.budget)) break;
      if (drop) {
        zero_rows(smem + L::oRing + (x % NS) * L::kTile, L::kBoxes, keep, lane);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->ready[j & 7]));
    }
  } else if (warp == 3) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsElem));
    // ================= elementwise: thread = query row, warpgroup w = keys [64 w, 64 w + 64)
    const int w = (warp - 4) >> 2, q4 = warp & 3, r = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t tp = tmem + lane_off + cP + 64 * w;
    const int t = t0 + r / a.PG;
    const bool row_ok = work && t < t1;
    float lse2 = INFINITY, delta = 0.f;
    if (row_ok) {
      const float2 f = a.stats[((long long)hu * a.n_q + t) * a.PG + r % a.PG];
      lse2 = f.x;
      delta = f.y;
    }
    const float c = a.c;
    bool ok = true;
    MaskBytes mb;
    if (n > 0) mb.load(a.mask, k0, k1, lane);
    for (int j = 0; j < n; ++j) {
      uint32_t keep[4];
      const bool drop = mb.vote(a.mask, k0 + 128 * j, k1, lane, keep);
      if (j + 1 < n) mb.load(a.mask, k0 + 128 * (j + 1), k1, lane);
      const uint32_t kw[2] = {w ? keep[2] : keep[0], w ? keep[3] : keep[1]};
      const uint32_t ts = tmem + lane_off + 128 * (j & 1) + 64 * w;
      if (!mbar_wait_warp(smem_u32(&bars->s_full[j & 1]), (uint32_t)((j >> 1) & 1), status, a.budget)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t s[2][32];
      tmem_ld32_raw(ts, s[0]);
      tmem_ld32_raw(ts + 32, s[1]);
      tmem_wait_tie(s[0]);
      tie32(s[1]);
#pragma unroll
      for (int x = 0; x < 64; ++x)
        s[x >> 5][x & 31] = __float_as_uint(ex2_approx(fmaf(__uint_as_float(s[x >> 5][x & 31]), c, -lse2)));
      if (!mbar_wait_warp(smem_u32(&bars->dp_full), (uint32_t)(j & 1), status, a.budget)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t pk[32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t dp[32];
        tmem_ld32_raw(tp + 32 * h, dp);
        tmem_wait_tie(dp);
#pragma unroll
        for (int x = 0; x < 32; ++x)
          dp[x] = __float_as_uint(__uint_as_float(s[h][x]) * (__uint_as_float(dp[x]) - delta));
        if (drop) {
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (!((kw[h] >> x) & 1u)) dp[x] = 0u;
        }
#pragma unroll
        for (int x = 0; x < 16; ++x)
          pk[16 * h + x] = cvt_bf16x2(__uint_as_float(dp[2 * x]), __uint_as_float(dp[2 * x + 1]));
      }
      tmem_st32(ts, pk);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->ds_full));
    }
    // ---- each warpgroup writes half of the columns
    const bool have = ok && n > 0 && mbar_wait_warp(smem_u32(&bars->done), 0, status, a.budget);
    tc_fence_after();
    const long long row = ((long long)t * a.H + hu * a.PG + r % a.PG) * D + w * (D / 2);
    const uint32_t tq = tmem + lane_off + cDQ + w * (D / 2);
    if (a.splits == 1) {
      write_row<D / 2>(tq, have, row_ok, false, a.scale, a.dQ + row);
    } else {
      float* po = a.part + (long long)split * a.n_q * a.H * D + row;
#pragma unroll 1
      for (int x = 0; x < D / 2; x += 16) {
        uint32_t o[16];
        if (have) {
          tmem_ld16(tq + x, o);
          tmem_wait16(o);
        }
        if (row_ok) {
#pragma unroll
          for (int y = 0; y < 16; y += 4)
            *reinterpret_cast<float4*>(po + x + y) =
                have ? make_float4(__uint_as_float(o[y]), __uint_as_float(o[y + 1]),
                                   __uint_as_float(o[y + 2]), __uint_as_float(o[y + 3]))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cross_bwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_do,
                 const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                 const __grid_constant__ BwdParams a) {
  using L = BSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  BBars* bars = reinterpret_cast<BBars*>(smem + L::oBars);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars->own), 1);
    for (int s = 0; s < 8; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1);
      mbar_init(smem_u32(&bars->empty[s]), 1);
      mbar_init(smem_u32(&bars->ready[s]), 1);
    }
    mbar_init(smem_u32(&bars->s_full[0]), 1);
    mbar_init(smem_u32(&bars->s_full[1]), 1);
    mbar_init(smem_u32(&bars->dp_full), 1);
    mbar_init(smem_u32(&bars->p_full), 8);
    mbar_init(smem_u32(&bars->ds_full), 8);
    mbar_init(smem_u32(&bars->done), 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmap_q);
    tma_prefetch_desc(&tmap_do);
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
  griddep_wait();  // the schedule, lse2 and delta
  if (blockIdx.x < a.kv_ctas) dkv_cta<D>(&tmap_q, &tmap_do, &tmap_k, &tmap_v, a, smem, tmem);
  else dq_cta<D>(&tmap_q, &tmap_do, &tmap_k, &tmap_v, a, smem, tmem);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// dQ = scale times the sum of the splits' partials, in order.
__global__ void __launch_bounds__(256) cross_dq_join_kernel(const float4* __restrict__ part, int splits,
                                                            const int64_t* qoff, int R, long long n4,
                                                            int row4, float scale, const WsHeader* hdr,
                                                            uint2* __restrict__ dQ) {
  griddep_wait();
  if (read_status(&hdr->status) != 0) return;
  const long long end = qoff[R] * row4;  // float4 pieces of the users' rows
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < end; i += gridDim.x * 256LL) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = 0; x < splits; ++x) {
      const float4 v = part[x * n4 + i];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    dQ[i] = make_uint2(cvt_bf16x2(s.x * scale, s.y * scale), cvt_bf16x2(s.z * scale, s.w * scale));
  }
}

template <int D>
cudaError_t launch_t(const CrossArgs& a, const CrossGeo& geo, cudaStream_t s) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  CUtensorMap tq, tdo, tk, tv;
  if (!tmap_heads(&tq, a.Q, a.n_q, a.H, D, a.q_stride, geo.pg, 128 / geo.pg) ||
      !tmap_heads(&tdo, a.dout, a.n_q, a.H, D, (long long)a.H * D, geo.pg, 128 / geo.pg) ||
      !tmap_heads(&tk, a.K, a.n_kv, a.Hkv, D, a.k_stride, 1, 128) ||
      !tmap_heads(&tv, a.V, a.n_kv, a.Hkv, D, a.v_stride, 1, 128))
    return cudaErrorInvalidValue;
  BwdParams p = {};
  p.qoff = a.qoff;
  p.koff = a.koff;
  p.qtiles = reinterpret_cast<const Tile*>(ws + a.plan.qtiles);
  p.ktiles = reinterpret_cast<const Tile*>(ws + a.plan.ktiles);
  p.hdr = reinterpret_cast<WsHeader*>(ws + a.plan.hdr);
  p.mask = a.mask;
  p.stats = reinterpret_cast<const float2*>(ws + a.plan.stats);
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.G = a.H / a.Hkv;
  p.PG = geo.pg;
  p.splits = geo.splits;
  p.kv_ctas = geo.key_tiles * a.Hkv;
  p.c = a.scale * kLog2e;
  p.scale = a.scale;
  p.dQ = static_cast<__nv_bfloat16*>(a.dQ);
  p.dK = static_cast<__nv_bfloat16*>(a.dK);
  p.dV = static_cast<__nv_bfloat16*>(a.dV);
  p.part = reinterpret_cast<float*>(ws + a.plan.part_o);
  p.n_q = a.n_q;
  p.budget = kDefaultWaitBudget;
  constexpr size_t smem = 1024 + BSmem<D>::oBars + sizeof(BBars);
  static_assert(smem <= 227 * 1024, "shared memory");
  cudaError_t e = prepare_kernel<cross_bwd_kernel<D>>(smem, kRegsLaunch);
  if (e != cudaSuccess) return e;
  const long long ctas = p.kv_ctas + geo.pair_tiles * 2 * (a.H / geo.pg) * geo.splits;
  if (ctas == 0) return cudaSuccess;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  if ((e = launch_dependent(cross_bwd_kernel<D>, dim3((unsigned)ctas), dim3(kThreads), smem, s, tq, tdo, tk,
                            tv, p)) != cudaSuccess)
    return e;
  if (geo.splits == 1 || a.n_q == 0) return cudaSuccess;
  const long long n4 = a.n_q * a.H * D / 4;
  long long grid = (n4 + 255) / 256;
  if (grid > a.sms * 8LL) grid = a.sms * 8LL;
  return launch_dependent(cross_dq_join_kernel, dim3((unsigned)grid), dim3(256), 0, s,
                          reinterpret_cast<const float4*>(p.part), geo.splits, a.qoff, a.R, n4,
                          a.H * D / 4, a.scale, (const WsHeader*)p.hdr, static_cast<uint2*>(a.dQ));
}

}  // namespace

cudaError_t launch_bwd(const CrossArgs& a, const CrossGeo& geo, cudaStream_t s) {
  return a.d == 64 ? launch_t<64>(a, geo, s) : launch_t<128>(a, geo, s);
}

}  // namespace cross
}  // namespace sa
