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
// for an fp32 tile, natural (nat[r * ldn + c]) and / or transposed
// (tr[c * FLD + r]); rows at or past `rows` are zero and not read.  Every row
// starts on a 16-byte boundary.  Neighbouring lanes take neighbouring rows, so
// that both forms are written without bank conflicts (along the columns the
// transposed one takes eight ways); a line of a row serves several turns from L1.
// Where registers allow, a tile's operands are all fetched before the first is put
// down, one trip to memory instead of one each (scan of 4 x 2048 x 32 x 64 x 64:
// forward 400 -> 380 us, gradients 1205 -> 1018; k_cross_read 12.7 -> 10.6; no gain
// where a tile has two operands and the block several tiles).
template <typename T, int W>
struct Rows {
  static constexpr int VN = Vec16<T>::n, VPR = W / VN, NV = (VPR + 3) / 4;
  uint4 u[NV];
  __device__ __forceinline__ void fetch(const T* g, long stride, int rows) {
    const int r = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = (threadIdx.x >> 6) + 4 * k;
      u[k] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows && v < VPR) u[k] = *reinterpret_cast<const uint4*>(g + r * stride + v * VN);
    }
  }
  __device__ __forceinline__ void clear() {  // this thread's row, threadIdx.x mod 64
#pragma unroll
    for (int k = 0; k < NV; ++k) u[k] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void put(float* nat, int ldn, float* tr) const {
    const int r = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = (threadIdx.x >> 6) + 4 * k, c = v * VN;
      if (v >= VPR) break;
      float f[VN];
      Vec16<T>::unpack(u[k], f);
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
};

// The same for a [D][M] fp32 matrix, natural (ld M + 4) and / or transposed (ld D + 4);
// lanes along its rows where only the natural form is wanted, else down its columns
// (the transposed form's banks).
template <int D, int M, bool TR>
struct State {
  static constexpr int NV = (D * M / 4 + 255) / 256;
  float4 u[NV];
  __device__ __forceinline__ static int row(int e) { return TR ? e % D : e / (M / 4); }
  __device__ __forceinline__ static int col(int e) { return TR ? e / D * 4 : e % (M / 4) * 4; }
  __device__ __forceinline__ void fetch(const float* g) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = threadIdx.x + 256 * k;
      if (e < D * M / 4) u[k] = *reinterpret_cast<const float4*>(g + row(e) * M + col(e));
    }
  }
  __device__ __forceinline__ void put(float* nat, float* tr) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = threadIdx.x + 256 * k, d = row(e), m = col(e);
      if (e >= D * M / 4) break;
      if (nat != nullptr) *reinterpret_cast<float4*>(nat + d * (M + 4) + m) = u[k];
      if (TR) {
        tr[m * (D + 4) + d] = u[k].x;
        tr[(m + 1) * (D + 4) + d] = u[k].y;
        tr[(m + 2) * (D + 4) + d] = u[k].z;
        tr[(m + 3) * (D + 4) + d] = u[k].w;
      }
    }
  }
};

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

// CC neighbouring outputs of one row, as T.
template <typename T, int CC>
__device__ __forceinline__ void store_cols(T* p, const float (&f)[CC]) {
#pragma unroll
  for (int c = 0; c < CC; ++c) p[c] = from_f<T>(f[c]);
}

}  // namespace la
