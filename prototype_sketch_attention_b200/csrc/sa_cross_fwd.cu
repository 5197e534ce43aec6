// Multi-head cross attention, forward, on tcgen05 (sm_100a).
//
// Per 128-row tile of packed query rows (sa_cross.cuh) and key tile j of 128 rows:
//   S = Q K_j^T (TMEM, fp32),  m = running row maximum,  P = 2^(c (S - m)) as bf16 (TMEM, over S),
//   O += P V_j (TMEM, fp32),   l += row sums of P in fp32,         c = scale log2 e,
// and at the end out = O / l, lse = (c m + log2 l) ln 2. The running maximum is raised only when
// a tile's maximum exceeds it by more than 8 in log2 units (O and l are then rescaled; the
// weights stay below 2^8 otherwise, and bf16 keeps their relative precision at any size).
//
// An item is two tiles (256 rows) of one user and head group, so that each key tile read from L2
// serves 256 rows (one tile would need 64 bytes a clock of L2 reads against the tensor pipe,
// more than an SM gets), and so that one warpgroup's softmax runs while the tensor cores work
// for the other. When the rows fit in one tile, both warpgroups take that tile, on alternate
// key tiles, with an O, m and l each, merged at the end. The items' key tiles, in order, are split
// evenly over one CTA per SM (the schedule's Start records): an item that a boundary cuts is
// left by its CTAs as fp32 parts, which cross_join_kernel puts together in order. A CTA runs its
// items through without a stop: while the warpgroups write an item's rows the next item's
// queries and keys are loaded and its first scores computed (one CTA per item, with its
// set-up, first loads and epilogue exposed, lost 12,000 clocks an item: 4 x 4096 x 8 heads).
//
// Roles (384 threads): warp 0 TMA (Q once an item, then K_0, V_0, K_1, V_1, ... through one ring of
// stages), warp 1 TMEM allocation and every MMA, warp 2 hands V tiles on, zeroing rows that
// the mask or the end of the range drops (weight 0 times NaN must not count), warp 3 reads the
// schedule ahead, warps 4-11 two softmax warpgroups, one thread per row. P stays in TMEM as the A
// operand of the second MMA.
// Every wait is by parity, which tells a phase from its neighbours only: no role may skip a phase that
// it later waits behind, nor may one come and go unseen (see the waits below).
// Bound: at d = 128 a tile costs 1,024 tensor clocks and 1,024 clocks of exponentials (16 a
// clock and SM); at d = 64 the exponentials bound it. Measured (4 d H a pair): 4 x 4096 queries and
// keys, 8 heads of 128: 255 us, 1,077 TFLOP/s (265 with the rest); 40 x 300 over 10K keys, 8 heads over
// 2: 510 us, 960 TFLOP/s; 8 heads of 64 over 1,024 keys of their own: 92 us, where the last 44
// rows of each user's 300 fill a third of a tile and an item has 8 steps a tile.
#include <cmath>

#include "sa_cross.cuh"

namespace sa {
namespace cross {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr float kRaise = 8.f;
constexpr uint32_t kRest = 32;  // one-tile items: a half of P's rest lies this many columns behind it
// The softmax warpgroups keep a row's 128 scores in registers. setmaxnreg.inc draws on the
// launch's 384 x 168 registers, so the split stays within them, and the launch refuses a build
// compiled to fewer.
constexpr int kRegsLaunch = 168, kRegsControl = 72, kRegsSoftmax = 216;
static_assert(128 * kRegsControl + 256 * kRegsSoftmax <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");

template <int D>
struct FSmem {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTile = kBoxes * kBox;
  // TMEM columns: the score buffers, then the accumulators of the two tiles. At d = 64 a third
  // score buffer fits, and a warpgroup's next scores are there before it asks for them.
  static constexpr int kNB = D == 128 ? 2 : 3;
  static constexpr uint32_t kColO = kNB * 128;
  static constexpr int kNS = D == 128 ? 5 : 8;  // stages: 2 + 5 tiles of 32 KB, or 2 + 8 of 16 KB
  static constexpr int oQ = 0;
  static constexpr int oKV = 2 * kTile;
  static constexpr int oML = oKV + kNS * kTile;  // warpgroup 1's m and l (merge)
  static constexpr int oItems = oML + 2 * 128 * 4;
  static constexpr int oBars = oItems + 2 * 32;
};

struct FBars {
  uint64_t q_full, q_empty, full[8], empty[8];
  uint64_t v_ready[8];  // by V tile mod 8: fewer V tiles than that fit in the ring
  uint64_t s_full[3], o_done[2];
  // an item's last output of each accumulator: o_done may be two phases behind there (a third score
  // buffer lets a warpgroup run ahead), and a wait by parity tells adjacent phases apart only
  uint64_t o_last[2];
  uint64_t p_full[3][2];  // [buffer][half of the keys]: the second product starts on the first half
  uint64_t o_free, merge, drain;
  uint64_t item_full[2], item_empty[2];
  uint32_t tmem_base;
};

// One CTA's piece of an item, as warp 3 hands it to the others.
struct Item {
  int n;            // key tiles of this piece (-1: no more items)
  int t0, t1;       // first token of the tiles, one past the user's last
  int k0, k1;       // first key row of the piece, one past the user's last
  int hu, two;      // head group; rows in both tiles
  int part;         // -1: the whole item; else the part to leave
};

struct FwdParams {
  const int64_t* qoff;
  const int64_t* koff;
  const Tile* tiles;
  const Start* starts;   // [CTAs + 1]
  WsHeader* hdr;
  const uint8_t* mask;
  int H, G, PG;          // heads, heads per key head, heads per tile
  float c;               // scale log2 e
  __nv_bfloat16* out;    // [n_q, H, D]
  __nv_bfloat16* rest;   // [n_q, H, D], nullable: out's rounding
  float* lse;            // [n_q, H]
  JoinItem* joins;       // [CTAs]
  int* join_ctas;        // [CTAs]: from b on, the CTAs behind CTA b that work on joins[b]
  int ctas;
  float* part_o;         // [2 CTAs][256, D]
  float* part_lse;       // [2 CTAs][256], log2 units
  long long budget;
};

constexpr int kConsumers = 11;  // warps that read an item: all but warp 3

// The s-th item; false: none, or the wait gave up. Whole warp.
__device__ __forceinline__ bool get_item(FBars* bars, const Item* ring, int s, int lane, int* status,
                                         long long budget, Item* it) {
  const bool ok = mbar_wait_warp(smem_u32(&bars->item_full[s & 1]), (uint32_t)((s >> 1) & 1), status, budget);
  *it = ring[s & 1];
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[s & 1]));
  return ok && it->n >= 0;
}

// Two values as bf16, and what rounding took from them, as bf16 too.
__device__ __forceinline__ uint32_t round_pair(float x, float y, uint32_t& rest) {
  const uint32_t v = cvt_bf16x2(x, y);
  rest = cvt_bf16x2(x - __uint_as_float(v << 16), y - __uint_as_float(v & 0xffff0000u));
  return v;
}

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
  constexpr int NS = L::kNS, kNB = L::kNB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  FBars* bars = reinterpret_cast<FBars*>(smem + L::oBars);
  int* status = &a.hdr->status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars->q_full), 1);
    mbar_init(smem_u32(&bars->q_empty), 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1);
      mbar_init(smem_u32(&bars->empty[s]), 2);  // the last MMA that reads the stage, and warp 2
    }
    for (int s = 0; s < 8; ++s) mbar_init(smem_u32(&bars->v_ready[s]), 1);
    for (int b = 0; b < L::kNB; ++b) {
      mbar_init(smem_u32(&bars->s_full[b]), 1);
      mbar_init(smem_u32(&bars->p_full[b][0]), 4);
      mbar_init(smem_u32(&bars->p_full[b][1]), 4);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_u32(&bars->o_done[w]), 1);
      mbar_init(smem_u32(&bars->o_last[w]), 1);
      mbar_init(smem_u32(&bars->item_full[w]), 1);
      mbar_init(smem_u32(&bars->item_empty[w]), kConsumers);
    }
    mbar_init(smem_u32(&bars->o_free), 8);
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
  griddep_launch_dependents();  // the join reads its inputs only after this grid has ended
  griddep_wait();  // the schedule

  const int groups = a.H / a.PG, tokens = 128 / a.PG;  // tokens per tile
  Item* items = reinterpret_cast<Item*>(smem + L::oItems);
  Item it;

  // every warp changes its register count inside its role's branch, so that the compiler
  // budgets each role for its count
  if (warp == 0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    // ================= TMA
    int i = 0, nq = 0;  // ring entries and items loaded so far
    bool ok = true;
    for (int s = 0; ok && get_item(bars, items, s, lane, status, a.budget, &it); ++s) {
      if (lane == 0 && it.n > 0) {
        const uint32_t qf = smem_u32(&bars->q_full);
        ok = mbar_wait(smem_u32(&bars->q_empty), (uint32_t)((nq & 1) ^ 1), status, a.budget);
        if (ok) {
          ++nq;
          mbar_arrive_expect_tx(qf, (it.two ? 2 : 1) * L::kTile);
          for (int w = 0; w < (it.two ? 2 : 1); ++w)
            for (int b = 0; b < L::kBoxes; ++b)
              tma_load_3d(sbase + L::oQ + w * L::kTile + b * kBox, &tmap_q, b * 64, it.hu * a.PG,
                          it.t0 + w * tokens, qf);
        }
        const int hk = it.hu * a.PG / a.G;
        for (int x = 0; ok && x < 2 * it.n; ++x) {
          const int st = i % NS;
          ok = mbar_wait(smem_u32(&bars->empty[st]), (uint32_t)(((i / NS) & 1) ^ 1), status, a.budget);
          if (!ok) break;
          const uint32_t fb = smem_u32(&bars->full[st]);
          mbar_arrive_expect_tx(fb, L::kTile);
          for (int b = 0; b < L::kBoxes; ++b)
            tma_load_3d(sbase + L::oKV + st * L::kTile + b * kBox, (x & 1) ? &tmap_v : &tmap_k, b * 64, hk,
                        it.k0 + 128 * (x >> 1), fb);
          ++i;
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (lane == 0) {
      for (int x = (i > NS ? i - NS : 0); x < i; ++x)
        mbar_wait_drain(smem_u32(&bars->full[x % NS]), (uint32_t)((x / NS) & 1), a.budget);
      if (nq > 0) mbar_wait_drain(smem_u32(&bars->q_full), (uint32_t)((nq - 1) & 1), a.budget);
    }
  } else if (warp == 1) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    // ================= MMAs. Step q is tile (and accumulator) q mod 2 with key tile q / 2, or key
    // tile q of the only tile; its scores go to buffer (steps so far) mod kNB. P(q) lies over
    // S(q), and the pipe runs a thread's MMAs in order, so S(q + kNB) overwrites it only after
    // O(q) has read it. The next item's first scores follow the last O.
    const uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0);
    const uint32_t id_o = idesc_bf16_f32(128, D, 0, 1);
    const uint32_t tm = broadcast(tmem), sb0 = broadcast(sbase), br = broadcast(smem_u32(bars));
    auto bar = [&](const uint64_t& b) {  // the address of a barrier, from the broadcast base
      return br + (uint32_t)(reinterpret_cast<const uint8_t*>(&b) - reinterpret_cast<const uint8_t*>(bars));
    };
    const uint32_t q_lo = desc_k(sb0 + L::oQ), k_lo = desc_k(sb0 + L::oKV), v_lo = desc_mn(sb0 + L::oKV);
    constexpr uint32_t kStage = L::kTile >> 4;
    RingPos<NS> kpos, vpos;  // the next scores' K and the next output's V
    vpos.next();
    RingPos<kNB> sb, pb;     // their buffers
    int vi = 0, nq = 0;      // V tiles and items with keys so far
    bool ok = true;
    auto wait = [&](uint32_t b, uint32_t parity) {
      ok = ok && mbar_wait_warp(b, parity, status, a.budget);
      return ok;
    };
    for (int s = 0; ok && get_item(bars, items, s, lane, status, a.budget, &it); ++s) {
      const bool two = broadcast(it.two);
      const int n = broadcast(it.n), steps = two ? 2 * n : n;
      const bool wide = n == 1;  // P's rest, too (an item that is cut leaves pieces of two tiles at least)
      if (n == 0) continue;
      wait(bar(bars->q_full), (uint32_t)(nq & 1));
      ++nq;
      auto scores = [&](int q) {
        const bool last_use = !two || (q & 1);
        if (!wait(bar(bars->full[0]) + 8 * kpos.st, kpos.ph)) return;
        tc_fence_after();
        if (elect_one()) {
          product_ss<D>(tm + 128 * sb.st, q_lo + (two ? q & 1 : 0) * kStage, k_lo + kpos.st * kStage, id_s);
          tc_commit(bar(bars->s_full[0]) + 8 * sb.st);
          if (last_use) tc_commit(bar(bars->empty[0]) + 8 * kpos.st);
          if (q == steps - 1) tc_commit(bar(bars->q_empty));
        }
        __syncwarp();
        sb.next();
        if (last_use) {
          kpos.next();
          kpos.next();
        }
      };
      for (int q = 0; q < kNB && q < steps; ++q) scores(q);
      // the accumulators of the item with keys before have been read
      if (nq > 1) wait(bar(bars->o_free), (uint32_t)(nq & 1));
      tc_fence_after();
      for (int q = 0; ok && q < steps; ++q) {
        const int w = q & 1;
        const bool last_use = !two || w == 1;
        const uint32_t o = tm + L::kColO + D * w, p = tm + 128 * pb.st, b = v_lo + vpos.st * kStage;
        const uint32_t pf = bar(bars->p_full[0][0]) + 16 * pb.st;
        if (!wait(bar(bars->v_ready[0]) + 8 * (vi & 7), (uint32_t)((vi >> 3) & 1)) || !wait(pf, pb.ph)) break;
        tc_fence_after();
        if (elect_one()) {
          if (q < 2) mma_ts<0>(o, p, b, kDescHi, id_o);
          else mma_ts<1>(o, p, b, kDescHi, id_o);
#pragma unroll
          for (int ks = 1; ks < 4; ++ks) mma_ts<1>(o, p + 8 * ks, b + mn_step(ks), kDescHi, id_o);
          if (wide) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) mma_ts<1>(o, p + kRest + 8 * ks, b + mn_step(ks), kDescHi, id_o);
          }
        }
        __syncwarp();
        if (!wait(pf + 8, pb.ph)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t p1 = p + 32 + (wide ? kRest : 0);
#pragma unroll
          for (int ks = 4; ks < 8; ++ks) mma_ts<1>(o, p1 + 8 * (ks - 4), b + mn_step(ks), kDescHi, id_o);
          if (wide) {
#pragma unroll
            for (int ks = 4; ks < 8; ++ks) mma_ts<1>(o, p1 + kRest + 8 * (ks - 4), b + mn_step(ks), kDescHi, id_o);
          }
          tc_commit(bar(bars->o_done[0]) + 8 * w);
          if (q + 2 >= steps) tc_commit(bar(bars->o_last[0]) + 8 * w);
          if (last_use) tc_commit(bar(bars->empty[0]) + 8 * vpos.st);
        }
        __syncwarp();
        pb.next();
        if (last_use) {
          vpos.next();
          vpos.next();
          ++vi;
        }
        if (q + kNB < steps) scores(q + kNB);
      }
    }
    __syncwarp();
    // commits follow the MMAs of the thread that issued them: the same lane is elected each time
    if (elect_one()) {
      tc_commit(smem_u32(&bars->drain));
      mbar_wait_drain(smem_u32(&bars->drain), 0, a.budget);
    }
  } else if (warp == 2) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    // ================= V tiles: zero the dropped rows
    int base = 0, vbase = 0;
    bool ok = true;
    for (int s = 0; ok && get_item(bars, items, s, lane, status, a.budget, &it); ++s) {
      MaskBytes mb;
      if (it.n > 0) mb.load(a.mask, it.k0, it.k1, lane);
      for (int j = 0; ok && j < it.n; ++j) {
        const int i = base + 2 * j + 1, st = i % NS, v = vbase + j;
        uint32_t keep[4];
        const bool drop = mb.vote(a.mask, it.k0 + 128 * j, it.k1, lane, keep);
        if (j + 1 < it.n) mb.load(a.mask, it.k0 + 128 * (j + 1), it.k1, lane);
        // K first: a stage holds K and V in turn, and a wait by parity can tell a phase from the ones
        // next to it only. So no phase may go unseen: a stage is free once this warp has seen it too.
        ok = mbar_wait_warp(smem_u32(&bars->full[(i - 1) % NS]), (uint32_t)(((i - 1) / NS) & 1), status, a.budget);
        if (!ok) break;
        if (lane == 0) mbar_arrive(smem_u32(&bars->empty[(i - 1) % NS]));
        ok = mbar_wait_warp(smem_u32(&bars->full[st]), (uint32_t)((i / NS) & 1), status, a.budget);
        if (!ok) break;
        if (drop) {
          zero_rows(smem + L::oKV + st * L::kTile, L::kBoxes, keep, lane);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars->v_ready[v & 7]));
          mbar_arrive(smem_u32(&bars->empty[st]));
        }
      }
      base += 2 * it.n;
      vbase += it.n;
    }
  } else if (warp == 3) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    // ================= the schedule: this CTA's items, up to two ahead
    if (lane == 0) {
      Start at = a.starts[blockIdx.x];
      const Start end = a.starts[blockIdx.x + 1];
      const bool any = a.hdr->total_tiles > 0;
      bool ok = true;
      for (int s = 0; ok; ++s) {
        const bool more = any && (at.tile < end.tile || (at.tile == end.tile && (at.group < end.group ||
                                                         (at.group == end.group && at.key < end.key))));
        Item x;
        x.n = -1;
        if (more) {
          const Tile tl = a.tiles[at.tile];
          const int t = (int)a.qoff[tl.user] + tl.index * 2 * tokens, k = (int)a.koff[tl.user];
          x.t0 = t;
          x.t1 = (int)a.qoff[tl.user + 1];
          x.k1 = (int)a.koff[tl.user + 1];
          const int all = (x.k1 - k + 127) / 128;
          const bool cut = at.tile == end.tile && at.group == end.group;
          const int to = cut ? end.key : all;
          x.k0 = k + 128 * at.key;
          x.n = to - at.key;
          x.hu = at.group;
          x.two = x.t1 - t > tokens;
          x.part = at.key > 0 ? 2 * (int)blockIdx.x : cut ? 2 * (int)blockIdx.x + 1 : -1;
          at.key = 0;
          if (++at.group == groups) {
            at.group = 0;
            ++at.tile;
          }
        }
        ok = mbar_wait(smem_u32(&bars->item_empty[s & 1]), (uint32_t)(((s >> 1) & 1) ^ 1), status, a.budget);
        if (!ok) break;
        items[s & 1] = x;
        mbar_arrive(smem_u32(&bars->item_full[s & 1]));
        if (!more) break;
      }
    }
    __syncwarp();
    {  // what the join has to know, while the others work
      const int b = blockIdx.x;
      const Start at = a.starts[b], end = a.starts[b + 1];
      const bool any = a.hdr->total_tiles > 0, same = at.tile == end.tile && at.group == end.group;
      JoinItem it = {};
      if (any && end.key > 0 && !(same && at.key > 0)) {
        const Tile tl = a.tiles[end.tile];
        it.t0 = (int)a.qoff[tl.user] + tl.index * 2 * tokens;
        it.t1 = (int)a.qoff[tl.user + 1];
        it.group = end.group;
        it.parts = 1;
        for (int x0 = b + 1;; x0 += 32) {  // until a boundary lies in another item
          const int x = x0 + lane;
          bool in = false, works = false;  // (rounded boundaries leave some CTAs with nothing)
          if (x < a.ctas) {
            const Start z = a.starts[x], y = a.starts[x + 1];
            in = z.tile == end.tile && z.group == end.group;
            works = in && !(z.tile == y.tile && z.group == y.group && z.key == y.key);
          }
          const unsigned w = __ballot_sync(0xffffffffu, works);
          if (works) a.join_ctas[b + it.parts - 1 + __popc(w & ((1u << lane) - 1))] = x;
          it.parts += __popc(w);
          if (!__all_sync(0xffffffffu, in)) break;
        }
      }
      if (lane == 0) a.joins[b] = it;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ================= softmax warpgroup w: tile w, or alternate key tiles of the only tile
    const int w = (warp - 4) >> 2;
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t ot = tmem + lane_off + L::kColO + D * w;
    const float c = a.c;
    bool ok = true;
    // parities, a bit each: this warpgroup's steps; items where it had steps; items with keys, of one
    // tile and all (registers are short here)
    constexpr uint32_t kCnt = 1, kLasts = 2, kSingles = 4, kFilled = 8;
    uint32_t par = 0;
    auto parity = [&](uint32_t bit) { return (par & bit) ? 1u : 0u; };
    RingPos<kNB> base;         // the score buffer of the item's step 0
    for (int s = 0; ok; ++s) {
    // the item stays in the ring while it is worked on: registers are short here
    if (!mbar_wait_warp(smem_u32(&bars->item_full[s & 1]), (uint32_t)((s >> 1) & 1), status, a.budget)) break;
    const Item& it = items[s & 1];
    if (it.n < 0) break;
    const bool two = it.two;
    const int k0 = it.k0, k1 = it.k1;
    const int step = two ? 1 : 2, first = two ? 0 : w, nkt = it.n;
    float m = -INFINITY, l = 0.f;
    int n = 0;
    RingPos<kNB> sb = base;
    if (w) sb.next();
    for (int q = (two ? 2 * nkt : nkt) % (2 * kNB); q > 0; --q) base.next();
    MaskBytes mb;
    if (first < nkt) mb.load(a.mask, k0 + 128 * first, k1, lane);
    if (nkt == 1 && first == 0) {
      // At most 128 keys: P enters the product as two bf16, its value and what that rounding took. Of few keys
      // P's rounding does not average out, and the gradients' delta = dout . out inherits it: dQ and dK were off
      // by up to 1.52 times what fp32 sums and one rounding give (3 keys), and are by 1.43, of which dS's
      // rounding makes 1.41. Half of the scores at a time, to 32 columns of P and 32 of its rest in their
      // place. In this block of its own, with short loops: in the loop below the values that the rest needs
      // cost long items 4 to 7 %; so 40 x 300 over 1,024 keys take 2 % more, 100 x 300 over 128 keys 5 %.
      uint32_t keep[4];
      const bool drop = mb.vote(a.mask, k0, k1, lane, keep);
      ok = mbar_wait_warp(smem_u32(&bars->s_full[sb.st]), sb.ph, status, a.budget);
      const uint32_t st = tmem + lane_off + 128 * sb.st;
      tc_fence_after();
      auto scores = [&](int i, uint32_t (&x)[32]) {
        tmem_ld32_raw(st + 32 * i, x);
        tmem_wait_tie(x);
        if (drop) {
          const uint32_t kw = i == 0 ? keep[0] : i == 1 ? keep[1] : i == 2 ? keep[2] : keep[3];
#pragma unroll
          for (int y = 0; y < 32; ++y)
            if (!((kw >> y) & 1u)) x[y] = 0xff800000u;  // -inf
        }
      };
      if (ok) {
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          uint32_t x[32];
          scores(i, x);
#pragma unroll
          for (int y = 0; y < 32; y += 2) m = fmax3(m, __uint_as_float(x[y]), __uint_as_float(x[y + 1]));
        }
        const float mc = m == -INFINITY ? 0.f : m * c;
        float sum[2] = {0.f, 0.f};
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t hi[32], lo[32];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t x[32];
            scores(2 * h + i, x);
#pragma unroll
            for (int y = 0; y < 32; y += 2) {
              const float z0 = ex2_approx(fmaf(__uint_as_float(x[y]), c, -mc));
              const float z1 = ex2_approx(fmaf(__uint_as_float(x[y + 1]), c, -mc));
              sum[0] += z0;
              sum[1] += z1;
              hi[16 * i + y / 2] = round_pair(z0, z1, lo[16 * i + y / 2]);
            }
          }
          tmem_st32(st + 2 * kRest * h, hi);
          tmem_st32(st + 2 * kRest * h + kRest, lo);
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[sb.st][h]));
        }
        l = sum[0] + sum[1];
        n = 1;
        par ^= kCnt;
      }
    } else for (int j = first; j < nkt; j += step, ++n, par ^= kCnt) {
      uint32_t keep[4];
      const bool drop = mb.vote(a.mask, k0 + 128 * j, k1, lane, keep);
      if (j + step < nkt) mb.load(a.mask, k0 + 128 * (j + step), k1, lane);
      if (!mbar_wait_warp(smem_u32(&bars->s_full[sb.st]), sb.ph, status, a.budget)) {
        ok = false;
        break;
      }
      const uint32_t st = tmem + lane_off + 128 * sb.st;
      tc_fence_after();
      uint32_t sc[4][32];
      load_scores(st, sc);
      if (drop) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (!((keep[i] >> x) & 1u)) sc[i][x] = 0xff800000u;  // -inf
      }
      float mx[4];  // four chains: the maximum is on the way to everything else
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mx[i] = fmaxf(__uint_as_float(sc[i][0]), __uint_as_float(sc[i][1]));
#pragma unroll
        for (int x = 2; x < 32; x += 2)
          mx[i] = fmax3(mx[i], __uint_as_float(sc[i][x]), __uint_as_float(sc[i][x + 1]));
      }
      const float mt = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
      const bool raise = (mt - m) * c > kRaise;  // false for -inf - -inf
      if (__any_sync(0xffffffffu, raise)) {
        const float f = raise ? ex2_approx((m - mt) * c) : 1.f;  // 0 for the first maximum
        if (n > 0) {
          // O_w holds every tile before this one once its last MMA has completed
          if (!mbar_wait_warp(smem_u32(&bars->o_done[w]), parity(kCnt) ^ 1, status, a.budget)) {
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
      const uint64_t c2 = f2_pack(c, c), mc2 = f2_pack(-mc, -mc);
      uint64_t ls[2] = {0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          float z0, z1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sc[2 * h + (x >> 4)][(2 * x) & 31]),
                                   __uint_as_float(sc[2 * h + (x >> 4)][(2 * x + 1) & 31])), c2, mc2), z0, z1);
          z0 = ex2_approx(z0);
          z1 = ex2_approx(z1);
          ls[x & 1] = f2_add(ls[x & 1], f2_pack(z0, z1));
          pk[x] = cvt_bf16x2(z0, z1);
        }
        tmem_st32(st + 32 * h, pk);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[sb.st][h]));
      }
      sb.next();
      sb.next();
      float l0, l1;
      f2_unpack(f2_add(ls[0], ls[1]), l0, l1);
      l += l0 + l1;
    }
    // ---- this tile's (or half's) accumulator is complete
    if (ok && n > 0) {
      ok = mbar_wait_warp(smem_u32(&bars->o_last[w]), parity(kLasts), status, a.budget);
      par ^= kLasts;
    }
    tc_fence_after();
    float* ml = reinterpret_cast<float*>(smem + L::oML);
    float g0 = 1.f, g1 = 0.f;  // factors of O_0 and O_1 (two tiles: of this tile's own)
    // the item with keys before has been written, so warpgroup 0 has read its m and l (waited for at
    // every such item: phase by phase)
    if (w == 1 && nkt > 0)  // (passes at once for the first)
      ok = ok && mbar_wait_warp(smem_u32(&bars->o_free), parity(kFilled) ^ 1, status, a.budget);
    if (!two && nkt > 0) {
      if (w == 1) {
        ml[r] = m;
        ml[128 + r] = ok ? l : 0.f;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->merge));
      } else {
        ok = mbar_wait_warp(smem_u32(&bars->merge), parity(kSingles), status, a.budget) && ok;
        tc_fence_after();
        const float m1 = ml[r], l1 = ml[128 + r];
        const float mm = fmaxf(m, m1);
        g0 = l > 0.f ? ex2_approx((m - mm) * c) : 0.f;
        g1 = l1 > 0.f ? ex2_approx((m1 - mm) * c) : 0.f;
        l = l * g0 + l1 * g1;
        m = mm;
      }
      par ^= kSingles;
    }
    // an item of one key tile has no step of warpgroup 1, whose next wait for scores would then be two
    // phases ahead of the last it saw: tile 0's last output follows every score of the item
    if (w == 1 && nkt > 0)
      ok = ok && mbar_wait_warp(smem_u32(&bars->o_last[0]), parity(kFilled), status, a.budget);
    if (nkt > 0) par ^= kFilled;
    const int t = it.t0 + (two ? w * tokens : 0) + r / a.PG;
    const int part = it.part;
    const bool mine = two || w == 0, write = mine && t < it.t1;
    const int hu = it.hu;
    const float inv = l == 0.f ? 0.f : 1.f / l;  // (a NaN stays one)
    g0 *= inv;
    g1 *= inv;
    const float lse2 = l == 0.f ? -INFINITY : m * c + lg2_approx(l);
    if (write) {
      if (part < 0) a.lse[(long long)t * a.H + hu * a.PG + r % a.PG] = lse2 * kLn2;
      else a.part_lse[(long long)part * 256 + w * 128 + r] = lse2;
    }
    const int tw = it.t0 + (two ? w * tokens : 0), t1 = it.t1;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[s & 1]));
    // the accumulators have been read (an item without keys has no phase: it could pass before the
    // MMA warp has seen the last)
    auto freed = [&]() {
      tc_fence_before();
      __syncwarp();
      if (nkt > 0 && lane == 0) mbar_arrive(smem_u32(&bars->o_free));
    };
    if (mine && (nkt > 0 || part < 0)) {
      // 32 words of a row at a time: 32 columns of a part, or 64 of out as bf16 pairs
      auto columns = [&](int x, uint32_t (&o)[32]) {
        if (nkt > 0) {
          tmem_ld32_raw(ot + x, o);
          tmem_wait_tie(o);
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * g0);
          if (!two && nkt > 1) {
            uint32_t o1[32];
            tmem_ld32_raw(tmem + lane_off + L::kColO + D + x, o1);
            tmem_wait_tie(o1);
#pragma unroll
            for (int y = 0; y < 32; ++y)
              o[y] = __float_as_uint(fmaf(__uint_as_float(o1[y]), g1, __uint_as_float(o[y])));
          }
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = 0u;
        }
        if (x == D - 32) freed();
      };
      if (part < 0 && a.rest) {  // 32 columns: 16 words of out, 16 of rest
        __nv_bfloat16* to = (lane >> 4) ? a.rest : a.out;
#pragma unroll 1
        for (int x = 0; x < D; x += 32) {
          uint32_t v[32], o[32];
          columns(x, o);
#pragma unroll
          for (int y = 0; y < 16; ++y)
            v[y] = round_pair(__uint_as_float(o[2 * y]), __uint_as_float(o[2 * y + 1]), v[16 + y]);
          regroup(v, lane);
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int rr = q4 * 32 + 4 * y + (lane & 3), tt = tw + rr / a.PG;
            if (tt < t1)
              *reinterpret_cast<uint4*>(to + ((long long)tt * a.H + hu * a.PG + rr % a.PG) * D + x +
                                        8 * ((lane >> 2) & 3)) =
                  make_uint4(v[4 * y], v[4 * y + 1], v[4 * y + 2], v[4 * y + 3]);
          }
        }
      } else if (part < 0) {
#pragma unroll 1
        for (int x = 0; x < D; x += 64) {
          uint32_t v[32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[32];
            columns(x + 32 * h, o);
#pragma unroll
            for (int y = 0; y < 16; ++y)
              v[16 * h + y] = cvt_bf16x2(__uint_as_float(o[2 * y]), __uint_as_float(o[2 * y + 1]));
          }
          regroup(v, lane);
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int rr = q4 * 32 + 4 * y + (lane & 3), tt = tw + rr / a.PG;
            if (tt < t1)
              *reinterpret_cast<uint4*>(a.out + ((long long)tt * a.H + hu * a.PG + rr % a.PG) * D + x +
                                        8 * (lane >> 2)) =
                  make_uint4(v[4 * y], v[4 * y + 1], v[4 * y + 2], v[4 * y + 3]);
          }
        }
      } else {
#pragma unroll 1
        for (int x = 0; x < D; x += 32) {
          uint32_t v[32];
          columns(x, v);
          regroup(v, lane);
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int rr = q4 * 32 + 4 * y + (lane & 3);
            if (tw + rr / a.PG < t1)
              *reinterpret_cast<uint4*>(a.part_o + ((long long)part * 256 + w * 128 + rr) * D + x + 4 * (lane >> 2)) =
                  make_uint4(v[4 * y], v[4 * y + 1], v[4 * y + 2], v[4 * y + 3]);
          }
        }
      }
    } else {
      freed();
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

// Items that boundaries cut: a warp of block (b, y) joins four rows of the item that starts in CTA b and
// goes on, from the parts of the CTAs that worked on it, in order: out = sum w O, w = 2^(lse2 - total).
// Bound by the chain of loads: the item and its CTAs; the parts' lse2 and the first two parts' O;
// more O. (Looking the item up here and walking every CTA of it made one user's forward 18.6 us in
// place of 15.3; 64 or 128 rows a block instead of 32 cost the odd batch 4 us.) A part that saw no
// kept key (lse2 = -inf) left no O.
template <int D>
__global__ void __launch_bounds__(256) cross_join_kernel(const __grid_constant__ FwdParams a) {
  constexpr int C = D / 32;  // columns a lane
  griddep_wait();
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const JoinItem it = a.joins[b];
  // lane: the CTA of part lane (and of parts lane + 32, ... where there are more)
  const int cta0 = lane == 0 ? b : a.join_ctas[min(b + lane - 1, a.ctas - 1)];
  const int r0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * 4;
  if (it.parts < 2 || it.t0 + r0 / a.PG >= it.t1) return;
  int cta = cta0;
  auto load = [&](int x, float (&v)[4][C]) {  // part x of the lanes' 32
    const int c = __shfl_sync(0xffffffffu, cta, x & 31);
    const float* po = a.part_o + ((long long)(x == 0 ? 2 * b + 1 : 2 * c) * 256 + r0) * D + lane * C;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (D == 128) {
        const float4 f = *reinterpret_cast<const float4*>(po + i * D);
        v[i][0] = f.x;
        v[i][1] = f.y;
        v[i][2 % C] = f.z;
        v[i][3 % C] = f.w;
      } else {
        const float2 f = *reinterpret_cast<const float2*>(po + i * D);
        v[i][0] = f.x;
        v[i][1] = f.y;
      }
    }
  };
  auto turn = [&](int x) {  // the lanes' CTAs for parts x .. x + 31
    if (it.parts > 32) cta = x == 0 ? cta0 : a.join_ctas[min(b + x + lane - 1, a.ctas - 1)];
  };
  // lane: row lane mod 4 of part x + lane / 4
  auto lse2 = [&](int x) {
    const int k = x + (lane >> 2), c = __shfl_sync(0xffffffffu, cta, k & 31);
    return k < it.parts ? a.part_lse[(long long)(k == 0 ? 2 * b + 1 : 2 * c) * 256 + r0 + (lane & 3)] : -INFINITY;
  };
  float v[2][4][C], o[4][C] = {};
  load(0, v[0]);
  load(1, v[1]);
  float m = -INFINITY, l = 0.f;
  for (int x = 0; x < it.parts; x += 8) {
    if ((x & 31) == 0) turn(x);
    m = fmaxf(m, lse2(x));
  }
#pragma unroll
  for (int y = 4; y < 32; y <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, y));
  for (int x0 = 0; x0 < it.parts; x0 += 8) {
    if ((x0 & 31) == 0) turn(x0);
    const float ls = lse2(x0), w = ls == -INFINITY ? 0.f : ex2_approx(ls - m);
    l += w;
#pragma unroll
    for (int x = 0; x < 8; x += 2) {
      if (x0 + x >= it.parts) break;
      if (x0 + x > 0) {
        load(x0 + x, v[0]);
        if (x0 + x + 1 < it.parts) load(x0 + x + 1, v[1]);
      }
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = __shfl_sync(0xffffffffu, w, 4 * (x + z) + i);
          if (f != 0.f) {
#pragma unroll
            for (int y = 0; y < C; ++y) o[i][y] = fmaf(f, v[z][i][y], o[i][y]);
          }
        }
    }
  }
#pragma unroll
  for (int y = 4; y < 32; y <<= 1) l += __shfl_xor_sync(0xffffffffu, l, y);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int mine = r0 + (lane & 3), tm = it.t0 + mine / a.PG;
  if (lane < 4 && tm < it.t1)
    a.lse[(long long)tm * a.H + it.group * a.PG + mine % a.PG] = l == 0.f ? -INFINITY : (m + lg2_approx(l)) * kLn2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + i, t = it.t0 + r / a.PG;
    const float f = __shfl_sync(0xffffffffu, inv, i);
    if (t >= it.t1) continue;
    const long long at = (((long long)t * a.H + it.group * a.PG + r % a.PG) * D + lane * C) / 2;
#pragma unroll
    for (int y = 0; y < C / 2; ++y) {
      uint32_t rest;
      reinterpret_cast<uint32_t*>(a.out)[at + y] = round_pair(o[i][2 * y] * f, o[i][2 * y + 1] * f, rest);
      if (a.rest) reinterpret_cast<uint32_t*>(a.rest)[at + y] = rest;
    }
  }
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
  p.starts = reinterpret_cast<const Start*>(ws + a.plan.starts);
  p.hdr = reinterpret_cast<WsHeader*>(ws + a.plan.hdr);
  p.mask = a.mask;
  p.H = a.H;
  p.G = a.H / a.Hkv;
  p.PG = geo.pg;
  p.c = a.scale * kLog2e;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.rest = static_cast<__nv_bfloat16*>(a.rest);
  p.lse = a.lse;
  p.joins = reinterpret_cast<JoinItem*>(ws + a.plan.joins);
  p.join_ctas = reinterpret_cast<int*>(p.joins + geo.ctas);
  p.ctas = geo.ctas;
  p.part_o = reinterpret_cast<float*>(ws + a.plan.part_o);
  p.part_lse = reinterpret_cast<float*>(ws + a.plan.part_lse);
  p.budget = kDefaultWaitBudget;
  static_assert(sizeof(Item) == 32, "the item ring");
  constexpr size_t smem = 1024 + FSmem<D>::oBars + sizeof(FBars);
  static_assert(smem <= 227 * 1024, "shared memory");
  cudaError_t e = prepare_kernel<cross_fwd_kernel<D>>(smem, kRegsLaunch);
  if (e != cudaSuccess) return e;
  if ((e = launch_dependent(cross_fwd_kernel<D>, dim3((unsigned)geo.ctas), dim3(kThreads), smem, s, tq, tk, tv,
                            p)) != cudaSuccess)
    return e;
  return launch_dependent(cross_join_kernel<D>, dim3((unsigned)geo.ctas, 8), dim3(256), 0, s, p);
}

}  // namespace

cudaError_t launch_fwd(const CrossArgs& a, const CrossGeo& geo, cudaStream_t s) {
  return a.d == 64 ? launch_t<64>(a, geo, s) : launch_t<128>(a, geo, s);
}

}  // namespace cross
}  // namespace sa
