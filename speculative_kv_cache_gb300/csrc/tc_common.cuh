// Helpers shared by the tcgen05 / TMA kernels: shared-memory matrix descriptors, 2-D tensor
// loads, tcgen05 fences, and the tensor-map builder.
#pragma once

#include <cuda.h>

#include "ig_common.cuh"

namespace ig {

// 2-D fp16 tensor [rows][cols] (cols contiguous) for TMA: boxes of 64 columns (one 128-byte
// swizzle atom) x box_rows rows, 128B swizzle, zero fill out of bounds.
ig_status make_map(CUtensorMap* m, const void* base, int rows, int cols, int box_rows);

// The same tensor (of 16-bit elements, cols 64 or 128) with its 64-column halves as a third dimension:
// a box is all columns of box_rows rows, one half after the other, each 128B-swizzled.
ig_status make_map_halves(CUtensorMap* m, const void* base, int rows, int cols, int box_rows);

// Heads of tokens, [tokens][heads][cols] (of 16-bit elements, cols 64 or 128), by columns, heads and tokens: a box is 64 columns
// of box_heads heads of box_tokens tokens, a head a row, 128B-swizzled; tokens past the last are zero.
ig_status make_map_heads(CUtensorMap* m, const void* base, int tokens, int heads, int cols, int box_tokens, int box_heads);

// Shared-memory matrix descriptor of a K-major, 128B-swizzled tile whose 8-row groups are
// 1024 bytes apart: start address >> 4 (bits 0-13), leading offset 16 B (unused for swizzled
// K-major tiles), stride offset 1024 B (bits 32-45), descriptor version 1 (bit 46), layout
// SWIZZLE_128B (bits 61-63 = 2).  Advancing the start address by 32 B selects the next 16-wide
// K step inside the swizzle atom.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

// tma_load_2d with an L2 policy
__device__ __forceinline__ void tma_load_2d_hint(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar,
                                                 uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
      "%3}], [%4], %5;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar)), "l"(pol)
      : "memory");
}

__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// Waits for a thread's loads from tensor memory, and ties the registers that they fill to the wait (nothing else keeps
// arithmetic on them behind it).
__device__ __forceinline__ void tm_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
               :
               : "memory");
  asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
// The same for two loads.
__device__ __forceinline__ void tm_wait_ld32(uint32_t (&r)[32], uint32_t (&r2)[32]) {
  tm_wait_ld32(r);
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile(""
                 : "+r"(r2[i]), "+r"(r2[i + 1]), "+r"(r2[i + 2]), "+r"(r2[i + 3]), "+r"(r2[i + 4]), "+r"(r2[i + 5]), "+r"(r2[i + 6]),
                   "+r"(r2[i + 7]));
}

}  // namespace ig
