// Two fp32 values in one 64-bit register pair, and the instructions that take both; a
// division by a number known at the launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace la {

using u64 = unsigned long long;

__device__ __forceinline__ u64 pk(float x, float y) {
  u64 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ float2 un(u64 v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ u64 two(float x) { return pk(x, x); }
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}

// Whole numbers below 2^31 divided by d: one product.
struct Divide {
  uint32_t d, m;
  int s;
  explicit Divide(uint32_t d_ = 1) : d(d_), s(0) {
    while ((1ull << s) < d) ++s;
    m = static_cast<uint32_t>((((1ull << s) - d) << 32) / d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(m, n) + n) >> s; }
};

}  // namespace la
