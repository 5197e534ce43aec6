// Device helpers shared by the multi-head cross attention's kernels (sm_100a).
//
// Rows. The G = H / Hkv query heads that share a key head are packed into the rows of a tile:
// with PG the largest power of two that divides G (at most 128), row r of a tile is token
// t0 + r / PG and head hu PG + r mod PG of head group hu < H / PG, so a key tile is read once
// for PG heads. A tile has 128 rows, 128 / PG tokens.
#pragma once

#include <cuda.h>

#include <atomic>

#include "sa_common.cuh"
#include "sa_internal.h"

namespace sa {
namespace cross {

constexpr int kBox = 16384;  // 128 rows x 128 bytes (64 bf16), 128B swizzle
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 3-D tiled load of one box.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// The MMA warps run their loops as a whole, on values that the compiler can see to be the same
// in every lane (broadcast()), and elect one lane only to issue: the MMA takes its operands
// from uniform registers, and in a branch of one lane each of them is moved there first (80
// clocks an MMA and 200 a wait, where the tensor cores take 32 to 64). Descriptors are a low word,
// to which offsets are added (the address field does not carry), and a constant high word.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0u;
}
template <typename T>
__device__ __forceinline__ T broadcast(T x) {
  return (T)__shfl_sync(0xffffffffu, (int)x, 0);
}

// kAcc: 1 accumulate, 0 overwrite.
template <int kAcc>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                       uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.eq.u32 p, %5, 1;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}"
      ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "n"(kAcc)
      : "memory");
}
// A in TMEM: [128 lanes] x bf16 pairs along the columns
template <int kAcc>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi,
                                       uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.eq.u32 p, %5, 1;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "n"(kAcc)
      : "memory");
}
// Low and high words of the descriptors of 128B-swizzled operands of 128-row boxes: K-major
// (leading offset unused), and MN-major (64-column boxes kBox apart).
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return (addr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr) { return (addr >> 4) | ((uint32_t)(kBox >> 4) << 16); }
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (kSwizzle128B << 29);

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16,"
      " %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Byte offset >> 4 of K step ks (16 of 128 or 64 columns) within a K-major operand made of
// 64-column boxes, and of 16 rows within an MN-major one.
__host__ __device__ constexpr uint32_t kstep(int ks) {
  return (uint32_t)((((ks >> 2) * kBox) + (ks & 3) * 32) >> 4);
}
__host__ __device__ constexpr uint32_t mn_step(int ks) { return (uint32_t)((ks * 2048) >> 4); }

// D = A B^T over D_ columns, both K-major in shared memory.
template <int D_>
__device__ __forceinline__ void product_ss(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc) {
  mma_ss<0>(d_tmem, a, b, kDescHi, idesc);
#pragma unroll
  for (int ks = 1; ks < D_ / 16; ++ks) mma_ss<1>(d_tmem, a + kstep(ks), b + kstep(ks), kDescHi, idesc);
}

// A place in a ring of N stages and the parity of its use.
template <int N>
struct RingPos {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == N) {
      st = 0;
      ph ^= 1u;
    }
  }
};

__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.ftz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Regroups a warp's 32 x 32 words (lane = row, register = column) so that register group s of
// lane l holds row 4 s + (l mod 4), columns 4 (l / 4) .. + 3: a store of a group by the warp covers
// four rows x 128 contiguous bytes (a row a lane would cost eight times the lines).
template <int LB, int GB>
__device__ __forceinline__ void regroup_step(uint32_t (&v)[32], int lane) {
  const bool hi = (lane >> LB) & 1;
#pragma unroll
  for (int gi = 0; gi < 8; ++gi) {
    if ((gi >> GB) & 1) continue;
    const int gj = gi | (1 << GB);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t send = hi ? v[4 * gi + c] : v[4 * gj + c];
      const uint32_t recv = __shfl_xor_sync(0xffffffffu, send, 1 << LB);
      if (hi) v[4 * gi + c] = recv; else v[4 * gj + c] = recv;
    }
  }
}
__device__ __forceinline__ void regroup(uint32_t (&v)[32], int lane) {
  regroup_step<4, 2>(v, lane);
  regroup_step<3, 1>(v, lane);
  regroup_step<2, 0>(v, lane);
}

// The keep bits of 128 rows from row0 on: rows at or past `end` and rows whose mask byte is 0
// are dropped. The load can run ahead of the vote; both are called by whole warps. Without
// a mask only a range's last tile needs a vote.
struct MaskBytes {
  uint32_t b[4];
  __device__ __forceinline__ void load(const uint8_t* mask, int row0, int end, int lane) {
    if (mask) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        b[i] = 32 * i + lane < end - row0 ? mask[(long long)row0 + 32 * i + lane] : 0u;
    }
  }
  // false: every row is kept (w unset)
  __device__ __forceinline__ bool vote(const uint8_t* mask, int row0, int end, int lane,
                                       uint32_t (&w)[4]) const {
    if (mask) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __ballot_sync(0xffffffffu, b[i] != 0u);
      return (w[0] & w[1] & w[2] & w[3]) != 0xffffffffu;
    }
    const int n = end - row0;
    if (n >= 128) return false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = n >= 32 * i + 32 ? ~0u : n > 32 * i ? (1u << (n - 32 * i)) - 1u : 0u;
    return true;
  }
};

// A whole warp zeroes the rows whose bit is 0 in a tile of `boxes` 128-row boxes: a dropped
// row meets weight 0 in a product, and 0 times what it holds must not be NaN. A lane per row,
// its 16-byte pieces in an order that keeps the lanes on different banks (a loop over the dropped
// rows, two at a time, held the V tiles back: 0.60 against 0.34 ms at one row in ten dropped).
__device__ __forceinline__ void zero_rows(uint8_t* tile, int boxes, const uint32_t (&w)[4], int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!((w[i] >> lane) & 1u)) {
      uint8_t* row = tile + (32 * i + lane) * 128;
      for (int b = 0; b < boxes; ++b)
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(row + b * kBox + ((c ^ (lane & 7)) << 4)) = make_uint4(0, 0, 0, 0);
    }
}

// A tile of the schedule: its user, and its place among the user's tiles.
struct Tile {
  int user, index;
};

// Where a CTA of the forward starts: query tile, head group, key tile.
struct Start {
  int tile, group, key, pad;
};

// The item that starts in a CTA of the forward and goes on in later ones: how many CTAs work on
// it (0: there is none), its rows, its head group.
struct JoinItem {
  int parts, t0, t1, group;
};

// Launch geometry, from the sizes that the host knows (lengths live on the device).
struct CrossGeo {
  int pg;                // heads packed into a tile
  long long pair_tiles;  // bound on the 256-row query tiles of all users
  long long key_tiles;   // bound on the 128-row key tiles of all users
  int splits;            // backward: CTAs that share a query tile's keys
  int ctas;              // forward: CTAs
};

// 3-D tensor map over bf16 rows of heads [n, heads, d], rows `stride` elements apart: boxes of
// 64 columns x box_heads x box_rows, 128B swizzle. n = 0 (nothing will be read): one row.
bool tmap_heads(CUtensorMap* m, const void* base, long long n, int heads, int d, long long stride,
                int box_heads, int box_rows);

// Dynamic shared memory of a kernel, set on its first launch on a device; regs > 0: the build must
// have given the kernel at least as many registers (setmaxnreg.inc waits for what the launch
// does not hold).
template <auto kern>
cudaError_t prepare_kernel(size_t smem, int regs = 0) {
  static std::atomic<uint64_t> done{0};  // one bit a device
  int id = 0;
  cudaError_t e = cudaGetDevice(&id);
  if (e != cudaSuccess) return e;
  if (id < 64 && ((done.load(std::memory_order_acquire) >> id) & 1u)) return cudaSuccess;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
    return e;
  if (regs > 0) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    if (fa.numRegs < regs) return cudaErrorInvalidConfiguration;
  }
  if (id < 64) done.fetch_or(1ull << id, std::memory_order_release);
  return cudaSuccess;
}

// A launch that may start while the grid before it in the stream drains: the kernel calls
// griddep_wait() before it touches memory.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                             const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_fwd(const CrossArgs& a, const CrossGeo& geo, cudaStream_t s);
cudaError_t launch_bwd(const CrossArgs& a, const CrossGeo& geo, cudaStream_t s);

}  // namespace cross
}  // namespace sa
