// Register-tiled fp32 products over shared-memory tiles for the CUDA-core
// kernels of the scan and the cross attention: 256 threads as a 16 x 16 grid,
// each holding RR x CC neighbouring outputs, both operands read as vectors.
#pragma once

#include "common.cuh"

namespace la {

constexpr int FT = 64;   // rows of a tile (tokens)
constexpr int FLD = 68;  // leading dimension of a tile with 64 columns (16-byte rows, shifted banks)

template <int W>
__device__ __forceinline__ void lds_vec(const float* p, float (&f)[W]) {
  if constexpr (W == 4) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
  } else if constexpr (W == 2) {
    const float2 u = *reinterpret_cast<const float2*>(p);
    f[0] = u.x, f[1] = u.y;
  } else {
    f[0] = *p;
  }
}

// acc[r][c] += sum_k X[k][ty RR + r] Y[k][tx CC + c]; both leading dimensions
// multiples of four.
template <int RR, int CC>
__device__ __forceinline__ void ffma_mm(float (&acc)[RR][CC], const float* X, int ldx, const float* Y, int ldy, int K) {
  const float* xp = X + (threadIdx.x >> 4) * RR;
  const float* yp = Y + (threadIdx.x & 15) * CC;
#pragma unroll 4
  for (int k = 0; k < K; ++k) {
    float a[RR], b[CC];
    lds_vec<RR>(xp + k * ldx, a);
    lds_vec<CC>(yp + k * ldy, b);
#pragma unroll
    for (int r = 0; r < RR; ++r)
#pragma unroll
      for (int c = 0; c < CC; ++c) acc[r][c] = fmaf(a[r], b[c], acc[r][c]);
  }
}

// Rows [0, rows) of a token-major matrix (row r at g + r * stride, W values)
// into an fp32 tile, natural (nat[r * ldn + c]) and / or transposed
// (tr[c * FLD + r]); rows at or past `rows` are zero and not read.  Every row
// starts on a 16-byte boundary.  Neighbouring lanes take neighbouring rows, so
// that both forms are written without bank conflicts (along the columns the
// transposed one takes eight ways); a line of a row serves several turns from L1.
template <typename T, int W>
__device__ __forceinline__ void stage(const T* g, long stride, int rows, float* nat, int ldn, float* tr) {
  constexpr int VN = Vec16<T>::n, VPR = W / VN;
  const int r = threadIdx.x & 63;
#pragma unroll
  for (int v = threadIdx.x >> 6; v < VPR; v += 4) {
    const int c = v * VN;
    float f[VN];
    if (r < rows) {
      Vec16<T>::unpack(*reinterpret_cast<const uint4*>(g + r * stride + c), f);
    } else {
#pragma unroll
      for (int i = 0; i < VN; ++i) f[i] = 0.f;
    }
    if (nat != nullptr) {
#pragma unroll
      for (int i = 0; i < VN; i += 4) *reinterpret_cast<float4*>(nat + r * ldn + c + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    }
    if (tr != nullptr) {
#pragma unroll
      for (int i = 0; i < VN; ++i) tr[(c + i) * FLD + r] = f[i];
    }
  }
}

// A [D][M] fp32 matrix into a tile, natural (ld M + 4) and / or transposed (ld D + 4);
// lanes along its rows where only the natural form is wanted, else down its columns
// (the transposed form's banks).
template <int D, int M>
__device__ __forceinline__ void stage_state(const float* g, float* nat, float* tr) {
  for (int e = threadIdx.x; e < D * M / 4; e += 256) {
    const int d = tr == nullptr ? e / (M / 4) : e % D, m = tr == nullptr ? e % (M / 4) * 4 : e / D * 4;
    const float4 v = *reinterpret_cast<const float4*>(g + d * M + m);
    if (nat != nullptr) *reinterpret_cast<float4*>(nat + d * (M + 4) + m) = v;
    if (tr != nullptr) {
      tr[m * (D + 4) + d] = v.x;
      tr[(m + 1) * (D + 4) + d] = v.y;
      tr[(m + 2) * (D + 4) + d] = v.z;
      tr[(m + 3) * (D + 4) + d] = v.w;
    }
  }
}

// Sum over the 16 threads that hold one row (tx = 0 .. 15), to all of them.
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the block's 256 threads, to all of them; `red` holds 8 floats.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += red[i];
  return s;
}

// RR x CC outputs of this thread times a factor of their row, as T.
template <typename T, int CC>
__device__ __forceinline__ void store_cols(T* p, const float (&f)[CC]) {
#pragma unroll
  for (int c = 0; c < CC; ++c) p[c] = from_f<T>(f[c]);
}

}  // namespace la
