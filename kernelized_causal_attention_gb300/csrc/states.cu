// States in 8 bits: [rows][M] fp32 rows (a state's D rows, head after head) become
// codes and one fp32 scale a row, and a token reads the codes directly.
//   scale = max |row| / top,  code = round(row / scale),  top = 127 (int8) or 448 (e4m3),
//   y = sum_d (phi(q_d) scale_d) code_d / sum_d phi(q_d) Z_d.
// The quotients are IEEE divisions, so a code is what the formula says, ties to even.
//
// All three kernels are bound by HBM: packing reads 4 and writes 1 byte a value, the
// token's read takes D (M + 8) bytes a head instead of D (4 M + 4).  2048 streams of 8
// heads, 64 x 64, int8: 14.5 us from HBM (79.7 MB, 0.81 of the copy rate), 12.4 again from
// what L2 holds of them (42.9 from fp32 states);
// 600 heads of 32 x 64 in e4m3, from L2: 2.4 us to pack, 2.0 to unpack.
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"
#include "scan.cuh"

namespace la {
namespace {

using bf16 = __nv_bfloat16;

// Four values of a row as four codes, low byte first, and back.
template <bool E4M3>
__device__ __forceinline__ uint32_t encode4(const float4& v, float scale) {
  const float f[4] = {v.x / scale, v.y / scale, v.z / scale, v.w / scale};
  uint32_t u = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t c;
    if (E4M3)
      c = __nv_cvt_float_to_fp8(f[i], __NV_SATFINITE, __NV_E4M3);
    else
      c = static_cast<uint32_t>(min(max(__float2int_rn(f[i]), -127), 127)) & 0xffu;
    u |= c << (8 * i);
  }
  return u;
}

__device__ __forceinline__ float2 half2_of_e4m3(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return __half22float2(__half2(h));
}

// Bytes of codes as fp32.  int8: the byte, its sign bit turned, in the last place of
// 2^23 is 2^23 + 128 + code.
template <bool E4M3>
__device__ __forceinline__ void decode4(uint32_t u, float* f) {
  if (E4M3) {
    const float2 a = half2_of_e4m3(u & 0xffffu), b = half2_of_e4m3(u >> 16);
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  } else {
    u ^= 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7650 | i)) - 8388736.f;
  }
}

// One thread a float4, M / 4 neighbouring lanes a row.  The magnitudes' bits are
// ordered as unsigned numbers with NaN above infinity, so their maximum also says
// whether the row is finite: if not, its scale is NaN.
template <int M, bool E4M3>
__global__ void __launch_bounds__(256) k_pack(const float4* S, uint32_t* code, float* scale, long n) {
  grid_dep_enter();
  constexpr int L = M / 4;
  const long e = (long)blockIdx.x * 256 + threadIdx.x;
  const float4 v = e < n ? S[e] : make_float4(0.f, 0.f, 0.f, 0.f);
  uint32_t m = max(max(__float_as_uint(fabsf(v.x)), __float_as_uint(fabsf(v.y))), max(__float_as_uint(fabsf(v.z)), __float_as_uint(fabsf(v.w))));
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (e >= n) return;
  const bool finite = m < 0x7f800000u;
  const float s = __uint_as_float(m) / (E4M3 ? 448.f : 127.f);
  code[e] = finite && s > 0.f ? encode4<E4M3>(v, s) : 0u;
  if (e % L == 0) scale[e / L] = finite ? s : __uint_as_float(0x7fffffffu);
}

template <int M, bool E4M3>
__global__ void __launch_bounds__(256) k_unpack(const uint32_t* code, const float* scale, float4* S, long n) {
  grid_dep_enter();
  const long e = (long)blockIdx.x * 256 + threadIdx.x;
  if (e >= n) return;
  float f[4];
  decode4<E4M3>(code[e], f);
  const float s = scale[e / (M / 4)];
  S[e] = make_float4(f[0] * s, f[1] * s, f[2] * s, f[3] * s);
}

// One warp a key head: a lane holds 16 columns of every RS-th row.  The weights
// phi(q_d) scale_d live two to a lane and are passed by shuffles; the lanes' sums are
// joined by halving: each exchange adds the half of the columns that the partner keeps.
// Seven blocks an SM, whose loads fill more of the time in which others compute, and codes
// marked as read once: 14.5 us for the 2048 x 8 heads above where they come from HBM, 16.1
// without the mark, 15.8 with the six blocks that 79 registers allow, 16.9 with neither;
// eight blocks spill (19.8).
template <int D, int M, bool E4M3, typename T>
__global__ void __launch_bounds__(128, 7)
    k_step_packed(const T* q, const uint4* code, const float* scale, const float* Z, T* y, int per, long heads) {
  grid_dep_enter();
  constexpr int L = M / 16, RS = 32 / L, K = (D + RS - 1) / RS, W = (D + 31) / 32;
  const int lane = threadIdx.x & 31, c = lane % L, r0 = lane / L;
  const long bhk = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (bhk >= heads) return;
  const uint4* p = code + bhk * (D * L);
  uint4 u[K];
#pragma unroll
  for (int k = 0; k < K; ++k) u[k] = r0 + k * RS < D ? __ldcs(p + k * 32 + lane) : make_uint4(0, 0, 0, 0);
  float z[W], sc[W];
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const int d = lane + 32 * w;
    z[w] = d < D ? Z[bhk * D + d] : 0.f;
    sc[w] = d < D ? scale[bhk * D + d] : 0.f;
  }
  for (int i = 0; i < per; ++i) {
    const long bh = bhk * per + i;
    float den = 0.f, wt[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int d = lane + 32 * w;
      const float f = d < D ? phi(to_f(q[bh * D + d])) : 0.f;
      den += z[w] != 0.f ? f * z[w] : 0.f;  // Z = 0: den = 0, whatever q holds
      wt[w] = f * sc[w];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    float a[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) a[j] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float f = __shfl_sync(0xffffffffu, wt[k * RS / 32], (r0 + k * RS) & 31);
      uint32_t x[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
      float g[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) asm volatile("" : "+r"(x[j]));  // decoded here, not ahead of the loop into four times the registers
#pragma unroll
      for (int j = 0; j < 4; ++j) decode4<E4M3>(x[j], g + 4 * j);
      if (D % RS == 0 || r0 + k * RS < D) {  // a lane without a row adds nothing
#pragma unroll
        for (int j = 0; j < 16; ++j) a[j] = fmaf(f, g[j], a[j]);
      }
    }
    int col = c * 16, n = 16;
#pragma unroll
    for (int o = 16; o >= L; o >>= 1) {
      if (n > 1) {
        n >>= 1;
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) {
            const float give = up ? a[j] : a[j + n], keep = up ? a[j + n] : a[j];
            a[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        col += up ? n : 0;
      } else {
        a[0] += __shfl_xor_sync(0xffffffffu, a[0], o);
      }
    }
    if (M == 64) {
#pragma unroll
      for (int j = 0; j < 2; ++j) y[bh * M + col + j] = from_f<T>(den != 0.f ? a[j] / den : 0.f);
    } else if (M == 32 || (lane & 1) == 0) {
      y[bh * M + col] = from_f<T>(den != 0.f ? a[0] / den : 0.f);
    }
  }
}

template <int M>
cudaError_t pack(const float* S, void* code, float* scale, long n, int fmt, cudaStream_t st) {
  return launch_pdl(fmt == 0 ? k_pack<M, false> : k_pack<M, true>, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, st,
                    (const float4*)S, (uint32_t*)code, scale, n);
}

template <int M>
cudaError_t unpack(const void* code, const float* scale, float* S, long n, int fmt, cudaStream_t st) {
  return launch_pdl(fmt == 0 ? k_unpack<M, false> : k_unpack<M, true>, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, st,
                    (const uint32_t*)code, scale, (float4*)S, n);
}

template <bool E4M3, typename T>
cudaError_t step(const void* q, const void* code, const float* scale, const float* Z, void* y, const CrossShape& s, cudaStream_t st) {
  const long heads = (long)s.B * s.Hk;
  cudaError_t e = cudaErrorInvalidValue;
  LA_DISPATCH_DM(s.D, s.M, (e = launch_pdl(k_step_packed<D_, M_, E4M3, T>, dim3(static_cast<unsigned>((heads + 3) / 4)), dim3(128), 0, st,
                                           (const T*)q, (const uint4*)code, scale, Z, (T*)y, s.H / s.Hk, heads)));
  return e;
}

}  // namespace

cudaError_t state_pack(const float* S, void* code, float* scale, long rows, int M, int fmt, cudaStream_t st) {
  const long n = rows * (M / 4);
  return M == 16 ? pack<16>(S, code, scale, n, fmt, st) : M == 32 ? pack<32>(S, code, scale, n, fmt, st) : pack<64>(S, code, scale, n, fmt, st);
}

cudaError_t state_unpack(const void* code, const float* scale, float* S, long rows, int M, int fmt, cudaStream_t st) {
  const long n = rows * (M / 4);
  return M == 16 ? unpack<16>(code, scale, S, n, fmt, st) : M == 32 ? unpack<32>(code, scale, S, n, fmt, st) : unpack<64>(code, scale, S, n, fmt, st);
}

cudaError_t cross_step_packed(const void* q, const void* code, const float* scale, const float* Z, void* y, int fmt, const CrossShape& s,
                              cudaStream_t st) {
  if (fmt == 0) return s.dtype == 0 ? step<false, float>(q, code, scale, Z, y, s, st) : step<false, bf16>(q, code, scale, Z, y, s, st);
  return s.dtype == 0 ? step<true, float>(q, code, scale, Z, y, s, st) : step<true, bf16>(q, code, scale, Z, y, s, st);
}

}  // namespace la
