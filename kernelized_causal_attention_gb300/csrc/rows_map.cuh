// TMA views of token-major bf16 rows and of stacks of [D][M] bf16 states, with
// their 4-D copies.
#pragma once

#include "tc.cuh"

namespace la {

// [B][N][heads][W] with rows ld elements apart (batch entries N ld apart) as
// (W, heads, N, B), boxes of 64 x 1 x 128 x 1 and the 128-byte swizzle: a
// narrower head and rows past N arrive as zeros and are not written by a store.
// base, W and ld multiples of 16 bytes.
bool make_rows_map(CUtensorMap* m, const void* base, int W, int heads, long ld, int N, int B);

// [n][D][M] states, boxes of 64 x 64 x 1 (zeros past D and M).
bool make_state_map(CUtensorMap* m, const void* base, int M, int D, long n);

namespace tc {

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(src))
      : "memory");
}

}  // namespace tc
}  // namespace la
