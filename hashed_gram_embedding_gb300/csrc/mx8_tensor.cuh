// The 5th-generation tensor cores with block scales (kind::mxf8f6f4): e4m3
// operands, K-major in shared memory with 128-byte swizzle (a row of a tile
// is 128 codes), float32 sums and the operands' scales in tensor memory.
#pragma once

#include "mx8.cuh"
#include "tensor_core.cuh"
#include "tma.cuh"

namespace ple {

// Instruction descriptor: both operands e4m3 and K-major, scales powers of
// two (bit 23); the low bits of the two block numbers choose the scale's byte
// in its column (operand B's at 4, A's at 29).
__host__ __device__ constexpr uint32_t mx_idesc(int m, int n) { return (uint32_t(n >> 3) << 17) | (1u << 23) | (uint32_t(m >> 4) << 24); }
__host__ __device__ constexpr uint32_t mx_block(int k) { return (uint32_t(k) << 4) | (uint32_t(k) << 29); }

// Descriptor of a piece of scales in shared memory: 32 rows of 16 bytes, no
// swizzle, groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t scales_operand(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) |
         (static_cast<uint64_t>(1) << 46);
}
__device__ __forceinline__ uint64_t codes_operand(uint32_t saddr) {
  return static_cast<uint64_t>(kOperandHigh) << 32 | operand(saddr);
}

// A piece of scales into four columns of tensor memory, in all four quarters
// of its lanes. Products issued after it by the same thread see it.
template <int kCtas>
__device__ __forceinline__ void scales_to_tmem(uint32_t at, uint32_t saddr) {
  if constexpr (kCtas == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(at), "l"(scales_operand(saddr)) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(at), "l"(scales_operand(saddr)) : "memory");
}

// d (+)= a b^T over 32 columns.
template <int kCtas>
__device__ __forceinline__ void mma_mx8(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t a_scales,
                                        uint32_t b_scales, bool add) {
  if constexpr (kCtas == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"(a_scales), "r"(b_scales), "r"(static_cast<uint32_t>(add))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"(a_scales), "r"(b_scales), "r"(static_cast<uint32_t>(add))
        : "memory");
}

// ---- a pair of CTAs ----

__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t at_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// Copies into this CTA's shared memory, counted on a barrier of either CTA:
// codes of some rows, from an atom (128 columns) on, each atom [row][128];
// pieces of scales.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int atom, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(atom), "r"(bar)
      : "memory");
}
// The same codes for a CTA by itself, and only as far as L2.
__device__ __forceinline__ void tma_load_atoms(uint32_t dst, const CUtensorMap* map, uint32_t bar, int atom, int row) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(atom), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_atoms(const CUtensorMap* map, int atom, int row) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(0), "r"(row), "r"(atom)
               : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Arrive at this barrier of both CTAs when the pair's products so far are done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ float4 read_cluster4(uint32_t at, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at_rank(at, rank)) : "memory");
  return v;
}

// Limit of a wait for sums, a step of the products that they come from: the
// waits of the warps that bring and issue these have it step by step.
#ifndef PLE_SUMS_WAIT_NS
#define PLE_SUMS_WAIT_NS kWaitLimitNs
#endif
// mbar_wait for the end of `steps` steps of products.
__device__ __noinline__ inline bool sums_wait(uint32_t bar, uint32_t parity, const volatile int* abort_flag, int steps) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns(), limit = uint64_t(PLE_SUMS_WAIT_NS) * steps;
  while (!*abort_flag && global_ns() - t0 < limit)
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
  return false;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// 32 columns of this thread's row, there once tmem_wait returns: the wait
// names the registers, so that nothing reads them before it.
__device__ __forceinline__ void tmem_ask(uint32_t at, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(at)
      : "memory");
}
template <int kLoads>
__device__ __forceinline__ void tmem_wait(float (&v)[kLoads][32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int c = 0; c < kLoads; ++c)
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(v[c][i]));
}

// Maps of an 8-bit tensor: its codes as [atom][row][128], its scales as rows
// of 512 bytes, one a piece.
ple_status mx_codes_map(CUtensorMap* map, const void* codes, int64_t rows, int columns, int box_rows, int box_atoms,
                        const char* name);
ple_status mx_scales_map(CUtensorMap* map, const void* scales, int64_t rows, int columns, int box_pieces,
                         const char* name);

}  // namespace ple
