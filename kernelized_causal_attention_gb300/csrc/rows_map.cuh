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

// 32 lanes x 32 bit, 8 consecutive columns, TMEM -> registers; 4 raw columns back.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st4u(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

}  // namespace tc
}  // namespace la
