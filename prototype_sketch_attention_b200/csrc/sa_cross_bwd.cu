// Multi-head cross attention, backward, on tcgen05 (sm_100a).
//
// With P = 2^(c S - lse2), c = scale log2 e, and delta = dout . out (made before this kernel):
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q.
// dQ sums over keys, dK and dV over queries and over the heads that share the key head. One
// pass that makes all three would have to add a 64 KB fp32 block of dQ per pair of tiles in global
// memory (about 6,000 clocks of L2 reductions on this GPU against 2,560 of tensor work, and an
// order that changes from run to run). So there are two kinds of item, each of which owns its
// output and keeps it in TMEM, at 7 products a pair of tiles in place of 5 and no atomics on data:
//   dK/dV: a tile of 128 keys of one key head against the user's packed query tiles (of every
//     head group that shares it). S^T = K Q^T and dP^T = V dO^T put keys on the TMEM lanes,
//     so P^T and dS^T, written as bf16 over S^T and dP^T, are the A operands in place:
//     dV += P^T dO, dK += dS^T Q. The rows' lse2 and delta run along the columns and come from
//     shared memory as broadcasts. At d = 64 there is room for a second S^T.
//   dQ: a tile of 128 packed query rows against the user's key tiles: S = Q K^T (two
//     buffers), dP = dO V^T, dS over S, dQ += dS K. When there are fewer such items than SMs and
//     many keys, `splits` of them share a tile and leave fp32 partials, summed in order.
// One CTA per SM takes items from a counter (which CTA computes an item does not change it) and
// runs through them without a stop: an item's own tiles, first loads and first products overlap
// the writing of the one before.
// Roles (384 threads): warp 0 TMA, warp 1 TMEM allocation and every MMA, warp 2 hands tiles on:
// it zeroes the rows that an MMA would multiply by 0 but must not read (dropped keys, rows past
// the user's end), and loads lse2 and delta; warp 3 takes the items; warps 4-11 two warpgroups for
// the elementwise step, 64 columns each, one thread per row. The tensor pipe runs ahead of the
// elementwise step: dK/dV: dV(i) and the next free S when P(i) is stored, dK(i) and dP(i+1) when
// dS(i) is, so the exponentials of tile i + 1 run while dK(i) and dP(i + 1) do; dQ: S(j+1) while
// tile j is in the elementwise step, then dP(j+1), dQ(j), S(j+2).
// K_j (and Q_i) is held from its first product to its last, V_j (dO_i) for half as long, so three
// slots of the one and two of the other; one ring of two pairs made every S wait for a load
// (3,700 clocks a step), and P^T through shared memory, which lets S^T go at once but
// leaves two slots of each, no less (3,700).
// Bound at d = 128: 2,048 tensor clocks a pair of tiles for dK/dV, 1,536 for dQ, 1,024
// clocks of exponentials in both. Measured (10 d a pair and head): 4 x 4096 queries and keys, 8 heads
// of 128: 725 us, 945 TFLOP/s; 40 x 300 over 10K keys, 8 heads over 2: 1.6 ms, 770 TFLOP/s; 40 x
// 100-300 over 1K-10K masked keys, 8 heads over 4: 540 us, 585 TFLOP/s: a dK/dV item has 2 to 5 steps there
// and its epilogue, which the tensor cores wait for, costs about one.
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
// Shared memory: the item's own tiles (K, V of dK/dV; Q, dO of dQ), then slots of a tile each: NK of
// Q_i or K_j, NV of dO_i or V_j. TMEM columns: dQ items: S 0 and 128, dP 256, dQ 384; dK/dV
// items: S^T, dP^T, dV, dK as below (what an epilogue reads starts at 256 or later).
template <int D>
struct BSmem {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTile = kBoxes * kBox;
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int NK = D == 128 ? 3 : 5, NV = kSlots - NK;
  static constexpr int oA = 0;
  static constexpr int oRing = 2 * kTile;
  static constexpr int oStat = oRing + kSlots * kTile;
  static constexpr int oItems = oStat + 2 * 256 * 4;  // a step: 128 of -lse2, 128 of -delta
  static constexpr int oBars = oItems + 2 * 32;
  static constexpr int kSBufs = D == 128 ? 1 : 2;
  static constexpr uint32_t cP = 128 * kSBufs, cDV = cP + 128, cDK = cDV + D;
};
constexpr uint32_t kColDp = 256, kColDq = 384;

struct BBars {
  uint64_t own, own_empty, full[8], empty[8];
  uint64_t ready[8];    // by step mod 8: fewer steps' tiles than that are in the slots
  uint64_t s_full[2], dp_full, p_full[2], ds_full[2], done, acc_free;
  uint64_t item_full[2], item_empty[2];
  uint32_t tmem_base;
};

enum : int { kEnd = -1, kDkv = 0, kDq = 1 };
struct Item {
  int kind, n;   // n: steps (query tiles of every sharing head group, or key tiles)
  int t0, t1;    // dK/dV: the user's query rows; dQ: the tile's first token, the user's end
  int k0, k1;    // the first key row, the user's end
  int h;         // key head (dK/dV) or head group (dQ)
  int aux;       // dK/dV: query tiles per head group; dQ: the split
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
  bool dq_first;           // the longer kind of item first
  float c, scale;
  __nv_bfloat16 *dQ, *dK, *dV;
  float* part;             // [splits][n_q, H, D] (splits > 1)
  long long n_q;
  long long budget;
};

constexpr int kConsumers = 11;  // warps that read an item: all but warp 3

// A warp's 32 rows x COLS fp32 TMEM columns, times f, to bf16: row i (of the warp's) goes to
// row_at(i), or nowhere when that is null. `zero` (of this lane's row): 0 whatever the accumulator
// holds. `read` is called once the accumulator has been read.
template <int COLS, typename RowAt, typename Read>
__device__ __forceinline__ void write_rows(uint32_t taddr, bool have, bool zero, float f, RowAt row_at,
                                           Read read, int lane) {
  constexpr int kStep = COLS < 64 ? COLS : 64;
#pragma unroll 1
  for (int x = 0; x < COLS; x += kStep) {
    uint32_t v[32];
#pragma unroll
    for (int h = 0; h < kStep / 32; ++h) {
      uint32_t o[32];
      if (have) {
        tmem_ld32_raw(taddr + x + 32 * h, o);
        tmem_wait_tie(o);
      }
#pragma unroll
      for (int y = 0; y < 16; ++y)
        v[16 * h + y] = zero || !have ? 0u
                                      : cvt_bf16x2(__uint_as_float(o[2 * y]) * f, __uint_as_float(o[2 * y + 1]) * f);
    }
    if (x + kStep == COLS) read();
    if (kStep < 64) {  // 64 bytes a row
      __nv_bfloat16* p = row_at(lane);
      if (p) {
#pragma unroll
        for (int y = 0; y < 4; ++y)
          reinterpret_cast<uint4*>(p + x)[y] = make_uint4(v[4 * y], v[4 * y + 1], v[4 * y + 2], v[4 * y + 3]);
      }
    } else {
      regroup(v, lane);
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        __nv_bfloat16* p = row_at(4 * y + (lane & 3));
        if (p)
          *reinterpret_cast<uint4*>(p + x + 8 * (lane >> 2)) =
              make_uint4(v[4 * y], v[4 * y + 1], v[4 * y + 2], v[4 * y + 3]);
      }
    }
  }
}

__device__ __forceinline__ bool get_item(BBars* bars, const Item* ring, int s, int lane, int* status,
                                         long long budget, Item* it) {
  const bool ok = mbar_wait_warp(smem_u32(&bars->item_full[s & 1]), (uint32_t)((s >> 1) & 1), status, budget);
  *it = ring[s & 1];
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[s & 1]));
  return ok && it->kind != kEnd;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cross_bwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_do,
                 const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                 const __grid_constant__ BwdParams a) {
  using L = BSmem<D>;
  constexpr int NK = L::NK, NV = L::NV;
  // d = 128 leaves no room to align by hand; the swizzle needs 1024 bytes, which dynamic shared
  // memory has when a kernel has no other (checked below)
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  BBars* bars = reinterpret_cast<BBars*>(smem + L::oBars);
  int* status = &a.hdr->status;
  if (sbase & 1023u) {
    griddep_wait();
    latch_status(status, SA_ERR_CUDA);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars->own), 1);
    mbar_init(smem_u32(&bars->own_empty), 1);
    for (int s = 0; s < 8; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1);
      mbar_init(smem_u32(&bars->empty[s]), s < NK ? 1 : 2);  // the last MMA that reads it; NK..: and warp 2
      mbar_init(smem_u32(&bars->ready[s]), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_u32(&bars->s_full[w]), 1);
      mbar_init(smem_u32(&bars->item_full[w]), 1);
      mbar_init(smem_u32(&bars->item_empty[w]), kConsumers);
    }
    mbar_init(smem_u32(&bars->dp_full), 1);
    mbar_init(smem_u32(&bars->p_full[0]), 8);
    mbar_init(smem_u32(&bars->p_full[1]), 8);
    mbar_init(smem_u32(&bars->ds_full[0]), 8);
    mbar_init(smem_u32(&bars->ds_full[1]), 8);
    mbar_init(smem_u32(&bars->done), 1);
    mbar_init(smem_u32(&bars->acc_free), 8);
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

  Item* items = reinterpret_cast<Item*>(smem + L::oItems);
  Item it;
  const int tokens = 128 / a.PG, sharing = a.G / a.PG;  // tokens per tile; head groups of a key head

  if (warp == 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    // ================= TMA
    uint32_t used = 0, loaded = 0;  // bit: parity of a slot's uses, and of its loads, so far
    uint32_t any = 0;               // slots ever loaded
    int own = 0;
    bool ok = true;
    for (int s = 0; ok && get_item(bars, items, s, lane, status, a.budget, &it); ++s) {
      if (lane == 0 && it.n > 0) {
        const bool dkv = it.kind == kDkv;
        const CUtensorMap *ma = dkv ? &tmap_k : &tmap_q, *mb = dkv ? &tmap_v : &tmap_do;
        const CUtensorMap *rx = dkv ? &tmap_q : &tmap_k, *ry = dkv ? &tmap_do : &tmap_v;
        ok = mbar_wait(smem_u32(&bars->own_empty), (uint32_t)((own & 1) ^ 1), status, a.budget);
        if (ok) {
          ++own;
          const uint32_t ob = smem_u32(&bars->own);
          const int y = dkv ? it.h : it.h * a.PG, z = dkv ? it.k0 : it.t0;
          mbar_arrive_expect_tx(ob, 2 * L::kTile);
          for (int b = 0; b < L::kBoxes; ++b) {
            tma_load_3d(sbase + L::oA + b * kBox, ma, b * 64, y, z, ob);
            tma_load_3d(sbase + L::oA + L::kTile + b * kBox, mb, b * 64, y, z, ob);
          }
        }
        int grp = 0, qt = 0;
        for (int x = 0; ok && x < it.n; ++x) {
          const int y = dkv ? (it.h * sharing + grp) * a.PG : it.h * a.PG / a.G;
          const int z = dkv ? it.t0 + qt * tokens : it.k0 + 128 * x;
          for (int v = 0; v < 2; ++v) {
            const int st = v ? NK + x % NV : x % NK;
            ok = ok && mbar_wait(smem_u32(&bars->empty[st]), ((used >> st) & 1u) ^ 1u, status, a.budget);
            if (!ok) break;
            const uint32_t fb = smem_u32(&bars->full[st]);
            mbar_arrive_expect_tx(fb, L::kTile);
            for (int b = 0; b < L::kBoxes; ++b)
              tma_load_3d(sbase + L::oRing + st * L::kTile + b * kBox, v ? ry : rx, b * 64, y, z, fb);
            used ^= 1u << st;
            loaded ^= 1u << st;
            any |= 1u << st;
          }
          if (++qt == it.aux) {  // (dQ items do not use them)
            qt = 0;
            ++grp;
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (lane == 0) {
      for (int x = 0; x < L::kSlots; ++x)
        if ((any >> x) & 1u) mbar_wait_drain(smem_u32(&bars->full[x]), ((loaded >> x) & 1u) ^ 1u, a.budget);
      if (own > 0) mbar_wait_drain(smem_u32(&bars->own), (uint32_t)((own - 1) & 1), a.budget);
    }
  } else if (warp == 1) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    // ================= MMAs
    const uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0), id_o = idesc_bf16_f32(128, D, 0, 1);
    constexpr uint32_t kStage = L::kTile >> 4;
    const uint32_t tm = broadcast(tmem), sb0 = broadcast(sbase), br = broadcast(smem_u32(bars));
    auto bar = [&](const uint64_t& b) {  // the address of a barrier, from the broadcast base
      return br + (uint32_t)(reinterpret_cast<const uint8_t*>(&b) - reinterpret_cast<const uint8_t*>(bars));
    };
    const uint32_t own_k = desc_k(sb0 + L::oA), ring_k = desc_k(sb0 + L::oRing), ring_mn = desc_mn(sb0 + L::oRing);
    uint32_t loaded = 0;                // bit: parity of a slot's loads before
    uint32_t pph = 0;                   // bit: parity of the uses of an S^T buffer before
    int own = 0, steps = 0;             // items with steps, steps before
    bool ok = true;
    auto wait = [&](uint32_t b, uint32_t parity) {
      ok = ok && mbar_wait_warp(b, parity, status, a.budget);
      return ok;
    };
    // acc += A B: A packed in TMEM, warpgroup w's 64 columns from column 64 w on
    auto accumulate = [&](uint32_t acc, uint32_t pk, uint32_t b, bool first) {
      if (first) mma_ts<0>(tm + acc, tm + pk, b, kDescHi, id_o);
      else mma_ts<1>(tm + acc, tm + pk, b, kDescHi, id_o);
#pragma unroll
      for (int ks = 1; ks < 8; ++ks)
        mma_ts<1>(tm + acc, tm + pk + 64 * (ks >> 2) + 8 * (ks & 3), b + mn_step(ks), kDescHi, id_o);
    };
    for (int s = 0; ok && get_item(bars, items, s, lane, status, a.budget, &it); ++s) {
      const int n = broadcast(it.n);
      const bool dkv = broadcast(it.kind) == kDkv;
      if (n == 0) continue;
      wait(bar(bars->own), (uint32_t)(own & 1));
      ++own;
      auto wait_ready = [&](int i) {
        const int x = steps + i;
        wait(bar(bars->ready[0]) + 8 * (x & 7), (uint32_t)((x >> 3) & 1));
        tc_fence_after();
      };
      auto wait_acc = [&]() {  // the accumulators of the item with steps before have been read
        if (own > 1) wait(bar(bars->acc_free), (uint32_t)(own & 1));
        tc_fence_after();
      };
      if (dkv) {
        // own: K, V; slots: Q_i in i mod NK, dO_i in NK + i mod NV
        constexpr int NB = L::kSBufs;
        auto scores = [&](int i) {  // S^T = K Q_i^T
          wait_ready(i);
          const uint32_t sb = NB == 1 ? 0 : i & 1;
          if (ok && elect_one()) {
            product_ss<D>(tm + 128 * sb, own_k, ring_k + (i % NK) * kStage, id_s);
            tc_commit(bar(bars->s_full[0]) + 8 * sb);
          }
          __syncwarp();
        };
        auto dprob = [&](int i) {  // dP^T = V dO_i^T
          if (ok && elect_one()) {
            product_ss<D>(tm + L::cP, own_k + kStage, ring_k + (NK + i % NV) * kStage, id_s);
            tc_commit(bar(bars->dp_full));
            if (i == n - 1) tc_commit(bar(bars->own_empty));  // (every S of the item precedes its last dP)
          }
          __syncwarp();
        };
        scores(0);
        dprob(0);
        if (NB == 2 && n > 1) scores(1);
        wait_acc();
        for (int i = 0; ok && i < n; ++i) {
          const int q = i % NK, g = NK + i % NV;
          const int pb = NB == 1 ? 0 : i & 1;
          if (!wait(bar(bars->p_full[0]) + 8 * pb, (pph >> pb) & 1u)) break;
          pph ^= 1u << pb;
          tc_fence_after();
          if (elect_one()) {
            accumulate(L::cDV, NB == 1 ? 0 : 128 * (i & 1), ring_mn + g * kStage, i == 0);  // dV += P^T dO_i
            tc_commit(bar(bars->empty[0]) + 8 * g);
          }
          __syncwarp();
          if (i + NB < n) scores(i + NB);  // overwrites P^T after the MMAs above, in order
          if (!wait(bar(bars->ds_full[0]) + 8 * ((steps + i) & 1), (uint32_t)(((steps + i) >> 1) & 1))) break;
          tc_fence_after();
          if (elect_one()) {
            accumulate(L::cDK, L::cP, ring_mn + q * kStage, i == 0);  // dK += dS^T Q_i
            tc_commit(bar(bars->empty[0]) + 8 * q);
          }
          __syncwarp();
          if (i + 1 < n) dprob(i + 1);  // overwrites dS^T after the MMAs above, in order
          loaded ^= (1u << q) | (1u << g);
        }
      } else {
        // own: Q, dO; slots: K_j in j mod NK, V_j in NK + j mod NV
        auto scores = [&](int j) {  // S = Q K_j^T into buffer j mod 2
          wait_ready(j);
          if (ok && elect_one()) {
            product_ss<D>(tm + 128 * (j & 1), own_k, ring_k + (j % NK) * kStage, id_s);
            tc_commit(bar(bars->s_full[0]) + 8 * (j & 1));
          }
          __syncwarp();
          loaded ^= 1u << (j % NK);
        };
        auto dprob = [&](int j) {  // dP = dO V_j^T
          const int v = NK + j % NV;
          if (!wait(bar(bars->full[0]) + 8 * v, (loaded >> v) & 1u)) return;
          loaded ^= 1u << v;
          tc_fence_after();
          if (elect_one()) {
            product_ss<D>(tm + kColDp, own_k + kStage, ring_k + v * kStage, id_s);
            tc_commit(bar(bars->dp_full));
            tc_commit(bar(bars->empty[0]) + 8 * v);
            if (j == n - 1) tc_commit(bar(bars->own_empty));  // (every S of the item precedes its last dP)
          }
          __syncwarp();
        };
        scores(0);
        wait_acc();
        dprob(0);
        if (n > 1) scores(1);
        for (int j = 0; ok && j < n; ++j) {
          if (!wait(bar(bars->ds_full[0]) + 8 * ((steps + j) & 1), (uint32_t)(((steps + j) >> 1) & 1))) break;
          tc_fence_after();
          if (j + 1 < n) dprob(j + 1);  // dP(j) has been read
          if (!ok) break;
          if (elect_one()) {
            accumulate(kColDq, 128 * (j & 1), ring_mn + (j % NK) * kStage, j == 0);  // dQ += dS K_j
            tc_commit(bar(bars->empty[0]) + 8 * (j % NK));
          }
          __syncwarp();
          if (j + 2 < n) scores(j + 2);  // overwrites dS(j) after the MMAs above, in order
        }
      }
      steps += n;
      if (elect_one()) tc_commit(bar(bars->done));
      __syncwarp();
    }
    // every commit of the issuing lane (the same lane is elected each time) has completed once its
    // last one has
    if (own > 0) mbar_wait_drain(smem_u32(&bars->done), (uint32_t)((own - 1) & 1), a.budget);
    __syncwarp();
  } else if (warp == 2) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    // ================= hands tiles on. dK/dV: lse2 and delta of the tile's rows; rows past the user's
    // end: weight 0, and zeros in the Q and dO tiles. dQ: zeros in the dropped rows of K.
    float* stat = reinterpret_cast<float*>(smem + L::oStat);
    uint32_t loaded = 0;
    int steps = 0;
    bool ok = true;
    for (int s = 0; ok && get_item(bars, items, s, lane, status, a.budget, &it); ++s) {
      const bool dkv = it.kind == kDkv;
      int grp = 0, qt = 0;
      MaskBytes mb;
      if (!dkv && it.n > 0) mb.load(a.mask, it.k0, it.k1, lane);
      for (int i = 0; ok && i < it.n; ++i, ++steps) {
        const int x = i % NK, y = NK + i % NV;
        const uint32_t xp = (loaded >> x) & 1u, yp = (loaded >> y) & 1u;
        loaded ^= (1u << x) | (1u << y);
        if (dkv) {
          const int t = it.t0 + qt * tokens, rows = min(128, (it.t1 - t) * a.PG);
          const float2* src = a.stats + ((long long)(it.h * sharing + grp) * a.n_q + t) * a.PG;
          float2 v[4];
#pragma unroll
          for (int z = 0; z < 4; ++z)
            v[z] = lane + 32 * z < rows ? src[lane + 32 * z] : make_float2(INFINITY, 0.f);
          ok = mbar_wait_warp(smem_u32(&bars->full[x]), xp, status, a.budget) &&
               mbar_wait_warp(smem_u32(&bars->full[y]), yp, status, a.budget);
          if (!ok) break;
          if (rows < 128) {
            uint32_t keep[4];
#pragma unroll
            for (int z = 0; z < 4; ++z)
              keep[z] = rows >= 32 * z + 32 ? ~0u : rows > 32 * z ? (1u << (rows - 32 * z)) - 1u : 0u;
            zero_rows(smem + L::oRing + x * L::kTile, L::kBoxes, keep, lane);
            zero_rows(smem + L::oRing + y * L::kTile, L::kBoxes, keep, lane);
            fence_proxy_async_smem();
          }
          // the place of two steps ago has been read for its dS (an item's tiles are loaded after the last
          // dP of the item before, so the phase before this one is over at an item's first steps too)
          ok = steps < 2 || mbar_wait_warp(smem_u32(&bars->ds_full[steps & 1]), (uint32_t)(((steps >> 1) & 1) ^ 1),
                                           status, a.budget);
          if (!ok) break;
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            stat[(steps & 1) * 256 + lane + 32 * z] = -v[z].x;
            stat[(steps & 1) * 256 + 128 + lane + 32 * z] = -v[z].y;
          }
          if (++qt == it.aux) {
            qt = 0;
            ++grp;
          }
        } else {
          uint32_t keep[4];
          const bool drop = mb.vote(a.mask, it.k0 + 128 * i, it.k1, lane, keep);
          if (i + 1 < it.n) mb.load(a.mask, it.k0 + 128 * (i + 1), it.k1, lane);
          ok = mbar_wait_warp(smem_u32(&bars->full[x]), xp, status, a.budget);
          if (!ok) break;
          if (drop) {
            zero_rows(smem + L::oRing + x * L::kTile, L::kBoxes, keep, lane);
            fence_proxy_async_smem();
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->ready[steps & 7]));
        // V too, after the fact: a wait by parity can tell a phase from the ones next to it only, so no
        // phase of a slot may go unseen, and the slot is free once this warp has seen it
        if (!dkv) ok = mbar_wait_warp(smem_u32(&bars->full[y]), yp, status, a.budget);
        if (ok && lane == 0) mbar_arrive(smem_u32(&bars->empty[y]));
      }
    }
  } else if (warp == 3) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    // ================= takes items, up to two ahead
    if (lane == 0) {
      const int groups = a.H / a.PG;
      const long long n_dkv = a.hdr->pad[0] * a.Hkv, n_dq = a.hdr->total_tiles * 2 * a.splits * groups;
      bool ok = true;
      for (int s = 0; ok;) {
        long long id = (long long)atomicAdd(reinterpret_cast<unsigned long long*>(&a.hdr->pad[1]), 1ull);
        Item x = {};
        x.kind = kEnd;
        if (id < n_dkv + n_dq) {
          const long long n1 = a.dq_first ? n_dq : n_dkv;
          const bool dq = (id < n1) == a.dq_first;
          if (id >= n1) id -= n1;
          if (!dq) {
            const Tile tl = a.ktiles[id / a.Hkv];
            x.kind = kDkv;
            x.h = (int)(id % a.Hkv);
            x.k0 = (int)a.koff[tl.user] + tl.index * 128;
            x.k1 = (int)a.koff[tl.user + 1];
            x.t0 = (int)a.qoff[tl.user];
            x.t1 = (int)a.qoff[tl.user + 1];
            x.aux = (x.t1 - x.t0 + tokens - 1) / tokens;
            x.n = x.aux * sharing;
          } else {
            // the group fastest: items of the same keys run at the same time
            x.kind = kDq;
            x.h = (int)(id % groups);
            id /= groups;
            const int half = (int)(id & 1);
            id >>= 1;
            x.aux = (int)(id % a.splits);
            const Tile tl = a.qtiles[id / a.splits];
            x.t0 = (int)a.qoff[tl.user] + (tl.index * 2 + half) * tokens;
            x.t1 = (int)a.qoff[tl.user + 1];
            if (x.t0 >= x.t1) continue;  // the pair's second tile has no rows
            const int k = (int)a.koff[tl.user];
            x.k1 = (int)a.koff[tl.user + 1];
            const int all = (x.k1 - k + 127) / 128;
            const int j0 = (int)((long long)all * x.aux / a.splits);
            x.n = (int)((long long)all * (x.aux + 1) / a.splits) - j0;
            x.k0 = k + j0 * 128;
          }
        }
        ok = mbar_wait(smem_u32(&bars->item_empty[s & 1]), (uint32_t)(((s >> 1) & 1) ^ 1), status, a.budget);
        if (!ok) break;
        items[s & 1] = x;
        mbar_arrive(smem_u32(&bars->item_full[s & 1]));
        ++s;
        if (x.kind == kEnd) break;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsElem));
    // ================= elementwise: thread = row (key of dK/dV, query of dQ), warpgroup w = columns
    // [64 w, 64 w + 64)
    const int w = (warp - 4) >> 2, q4 = warp & 3, r = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const float c = a.c;
    const uint64_t c2 = f2_pack(c, c);
    int steps = 0, own = 0;
    uint32_t sph = 0;  // bit b: parity of the uses of S buffer b so far
    bool ok = true;
    for (int s = 0; ok && get_item(bars, items, s, lane, status, a.budget, &it); ++s) {
      const int n = it.n;
      const bool dkv = it.kind == kDkv;
      if (dkv) {
        const uint32_t tp = tmem + lane_off + 64 * w + L::cP;
        for (int i = 0; i < n; ++i, ++steps) {
          if (!mbar_wait_warp(smem_u32(&bars->ready[steps & 7]), (uint32_t)((steps >> 3) & 1), status, a.budget) ||
              !mbar_wait_warp(smem_u32(&bars->s_full[L::kSBufs == 1 ? 0 : i & 1]),
                              (sph >> (L::kSBufs == 1 ? 0 : i & 1)) & 1u, status, a.budget)) {
            ok = false;
            break;
          }
          sph ^= 1u << (L::kSBufs == 1 ? 0 : i & 1);
          const uint32_t ts = tmem + lane_off + 64 * w + (L::kSBufs == 1 ? 0 : 128 * (i & 1));
          tc_fence_after();
          const ulonglong2* st =
              reinterpret_cast<const ulonglong2*>(smem + L::oStat + (steps & 1) * 1024 + 256 * w);
          uint32_t v[2][32];
          tmem_ld32_raw(ts, v[0]);
          tmem_ld32_raw(ts + 32, v[1]);
          tmem_wait_tie(v[0]);
          tie32(v[1]);
          uint32_t pk[32];
#pragma unroll
          for (int x = 0; x < 16; ++x) {  // four columns: -lse2 of them in one load
            const ulonglong2 f = st[x];
            uint32_t* e = &v[x >> 3][(4 * x) & 31];
            float p0, p1, p2, p3;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(e[0]), __uint_as_float(e[1])), c2, f.x), p0, p1);
            f2_unpack(f2_fma(f2_pack(__uint_as_float(e[2]), __uint_as_float(e[3])), c2, f.y), p2, p3);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            p2 = ex2_approx(p2);
            p3 = ex2_approx(p3);
            pk[2 * x] = cvt_bf16x2(p0, p1);
            pk[2 * x + 1] = cvt_bf16x2(p2, p3);
            e[0] = __float_as_uint(p0);
            e[1] = __float_as_uint(p1);
            e[2] = __float_as_uint(p2);
            e[3] = __float_as_uint(p3);
          }
          tmem_st32(ts, pk);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[L::kSBufs == 1 ? 0 : i & 1]));
          if (!mbar_wait_warp(smem_u32(&bars->dp_full), (uint32_t)(steps & 1), status, a.budget)) {
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
            for (int x = 0; x < 8; ++x) {
              const ulonglong2 f = st[32 + 8 * h + x];  // -delta
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int z = 4 * x + 2 * y;
                float d0, d1;
                f2_unpack(f2_mul(f2_pack(__uint_as_float(v[h][z]), __uint_as_float(v[h][z + 1])),
                                 f2_add(f2_pack(__uint_as_float(dp[z]), __uint_as_float(dp[z + 1])), y ? f.y : f.x)),
                          d0, d1);
                pk[16 * h + 2 * x + y] = cvt_bf16x2(d0, d1);
              }
            }
          }
          tmem_st32(tp, pk);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->ds_full[steps & 1]));
        }
      } else {
        const uint32_t tp = tmem + lane_off + kColDp + 64 * w;
        const int t = it.t0 + r / a.PG;
        float lse2 = INFINITY, delta = 0.f;
        if (t < it.t1) {
          const float2 f = a.stats[((long long)it.h * a.n_q + t) * a.PG + r % a.PG];
          lse2 = f.x;
          delta = f.y;
        }
        const uint64_t nl2 = f2_pack(-lse2, -lse2), nd2 = f2_pack(-delta, -delta);
        MaskBytes mb;
        if (n > 0) mb.load(a.mask, it.k0, it.k1, lane);
        for (int j = 0; j < n; ++j, ++steps) {
          uint32_t keep[4];
          const bool drop = mb.vote(a.mask, it.k0 + 128 * j, it.k1, lane, keep);
          if (j + 1 < n) mb.load(a.mask, it.k0 + 128 * (j + 1), it.k1, lane);
          const uint32_t ts = tmem + lane_off + 128 * (j & 1) + 64 * w;
          if (!mbar_wait_warp(smem_u32(&bars->s_full[j & 1]), (sph >> (j & 1)) & 1u, status, a.budget)) {
            ok = false;
            break;
          }
          sph ^= 1u << (j & 1);
          tc_fence_after();
          uint32_t v[2][32];
          tmem_ld32_raw(ts, v[0]);
          tmem_ld32_raw(ts + 32, v[1]);
          tmem_wait_tie(v[0]);
          tie32(v[1]);
#pragma unroll
          for (int x = 0; x < 64; x += 2) {
            float p0, p1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(v[x >> 5][x & 31]), __uint_as_float(v[x >> 5][(x & 31) + 1])), c2,
                             nl2), p0, p1);
            v[x >> 5][x & 31] = __float_as_uint(ex2_approx(p0));
            v[x >> 5][(x & 31) + 1] = __float_as_uint(ex2_approx(p1));
          }
          if (!mbar_wait_warp(smem_u32(&bars->dp_full), (uint32_t)(steps & 1), status, a.budget)) {
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
            for (int x = 0; x < 16; ++x) {
              float d0, d1;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(v[h][2 * x]), __uint_as_float(v[h][2 * x + 1])),
                               f2_add(f2_pack(__uint_as_float(dp[2 * x]), __uint_as_float(dp[2 * x + 1])), nd2)), d0, d1);
              pk[16 * h + x] = cvt_bf16x2(d0, d1);
            }
          }
          if (drop) {  // a pair's halves by the keep bits of its columns
            const uint32_t k0w = w ? keep[2] : keep[0], k1w = w ? keep[3] : keep[1];
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const uint32_t b = (x < 16 ? k0w : k1w) >> (2 * (x & 15));
              pk[x] &= ((b & 1u) ? 0xffffu : 0u) | ((b & 2u) ? 0xffff0000u : 0u);
            }
          }
          tmem_st32(ts, pk);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->ds_full[steps & 1]));
        }
      }
      // ---- the accumulators are complete
      bool have = false;
      if (n > 0) {
        have = ok && mbar_wait_warp(smem_u32(&bars->done), (uint32_t)(own & 1), status, a.budget);
        ok = have;
        ++own;
      }
      tc_fence_after();
      auto freed = [&]() {
        tc_fence_before();
        __syncwarp();
        // (an item without steps has no phase: it could pass before the MMA warp has seen the last)
        if (n > 0 && lane == 0) mbar_arrive(smem_u32(&bars->acc_free));
      };
      if (dkv) {  // warpgroup 0 writes dV, warpgroup 1 dK; a dropped key row gets 0
        const int j = it.k0 + r;
        const bool zero = a.mask && j < it.k1 && a.mask[j] == 0;
        __nv_bfloat16* out = w ? a.dK : a.dV;
        write_rows<D>(tmem + lane_off + (w ? L::cDK : L::cDV), have, zero, w ? a.scale : 1.f,
                      [&](int i) -> __nv_bfloat16* {
                        const int row = it.k0 + q4 * 32 + i;
                        return row < it.k1 ? out + ((long long)row * a.Hkv + it.h) * D : nullptr;
                      }, freed, lane);
      } else if (a.splits == 1) {  // each warpgroup writes half of the columns
        write_rows<D / 2>(tmem + lane_off + kColDq + w * (D / 2), have, false, a.scale,
                          [&](int i) -> __nv_bfloat16* {
                            const int x = q4 * 32 + i, t = it.t0 + x / a.PG;
                            return t < it.t1 ? a.dQ + ((long long)t * a.H + it.h * a.PG + x % a.PG) * D + w * (D / 2)
                                             : nullptr;
                          }, freed, lane);
      } else {
        const int t = it.t0 + r / a.PG;
        float* po = a.part + (((long long)it.aux * a.n_q + t) * a.H + it.h * a.PG + r % a.PG) * D + w * (D / 2);
#pragma unroll 1
        for (int x = 0; x < D / 2; x += 16) {
          uint32_t o[16];
          if (have) {
            tmem_ld16(tmem + lane_off + kColDq + w * (D / 2) + x, o);
            tmem_wait16(o);
          }
          if (x + 16 == D / 2) freed();
          if (t < it.t1) {
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
  // a dK/dV item walks a user's packed rows, a dQ item its keys; the longer kind first, so that short
  // items fill the end (d = 64, the other way round: 40 users x 200 queries, 3K keys, 8 heads over 4: 321 -> 337 us;
  // 40 x 100 queries, 5K keys: 459 -> 478; 10 x 600 queries, 300 keys, 16 heads over 2: 86 -> 94)
  p.dq_first = a.n_kv >= a.n_q * (a.H / a.Hkv);
  p.c = a.scale * kLog2e;
  p.scale = a.scale;
  p.dQ = static_cast<__nv_bfloat16*>(a.dQ);
  p.dK = static_cast<__nv_bfloat16*>(a.dK);
  p.dV = static_cast<__nv_bfloat16*>(a.dV);
  p.part = reinterpret_cast<float*>(ws + a.plan.part_o);
  p.n_q = a.n_q;
  p.budget = kDefaultWaitBudget;
  static_assert(sizeof(Item) == 32, "the item ring");
  constexpr size_t smem = BSmem<D>::oBars + sizeof(BBars);
  static_assert(smem <= 227 * 1024, "shared memory");
  cudaError_t e = prepare_kernel<cross_bwd_kernel<D>>(smem, kRegsLaunch);
  if (e != cudaSuccess) return e;
  if ((e = launch_dependent(cross_bwd_kernel<D>, dim3((unsigned)geo.ctas), dim3(kThreads), smem, s, tq, tdo, tk,
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
