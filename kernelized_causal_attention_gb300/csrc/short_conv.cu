// Short causal depthwise convolution over token-major rows, the layer in front
// of the selective scan:
//   pre[t][c] = bias[c] + sum_j w[c][j] x[t - K + 1 + j][c],   y = silu(pre) or pre,
// with K = 2, 3 or 4 taps and rows before the first one taken from a history
// (the last K - 1 inputs, oldest first) or zero.  Gradients, with g = dy silu'(pre):
//   dx[t] = sum_j w[j] g[t + K - 1 - j],  dw[j] = sum_t g[t] x[t - K + 1 + j],  db = sum_t g[t].
//
// All three directions are bound by HBM traffic (about 2 K flops an element).
// A thread owns V neighbouring channels and walks a run of rows with the last K
// inputs (and, backward, the last K values of g) in registers, so every row is
// read once plus the K - 1 rows (backward 2 (K - 1)) before a run; rows are
// loaded four at a time, four rows ahead of their use.  Sums and SiLU are fp32; y,
// dx and the parameters' gradients are rounded once.  4 x 2048 x 2304 bf16, K = 4,
// L2 flushed: forward 22.5 us (75 MB, 0.49 of the copy rate), gradients 38.9
// (113 MB, 0.43): what is left is the start and the end of one wave of short walks
// (issue 52 to 56 %).  A ring of eight rows in flight spilled: 80 us for both
// against 61.
#include <algorithm>

#include "common.cuh"
#include "scan.cuh"

namespace la {
namespace {

using bf16 = __nv_bfloat16;

// V neighbouring channels as one vector (V > 1: the caller has checked the
// alignment), raw or as fp32.
template <typename T, int V>
struct Pack;
template <typename T>
struct Pack<T, 1> {
  using Raw = T;
  __device__ __forceinline__ static void open(const Raw& u, float (&f)[1]) { f[0] = to_f(u); }
  __device__ __forceinline__ static void st(T* p, const float (&f)[1]) { *p = from_f<T>(f[0]); }
};
template <>
struct Pack<float, 4> {
  using Raw = float4;
  __device__ __forceinline__ static void open(const Raw& u, float (&f)[4]) { f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w; }
  __device__ __forceinline__ static void st(float* p, const float (&f)[4]) { *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Pack<float, 2> {
  using Raw = float2;
  __device__ __forceinline__ static void open(const Raw& u, float (&f)[2]) { f[0] = u.x, f[1] = u.y; }
  __device__ __forceinline__ static void st(float* p, const float (&f)[2]) { *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]); }
};
template <>
struct Pack<bf16, 4> {
  using Raw = uint2;
  __device__ __forceinline__ static void open(const Raw& u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x << 16), f[1] = __uint_as_float(u.x & 0xffff0000u);
    f[2] = __uint_as_float(u.y << 16), f[3] = __uint_as_float(u.y & 0xffff0000u);
  }
  __device__ __forceinline__ static void st(bf16* p, const float (&f)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};
template <typename T, int V>
__device__ __forceinline__ void ld(const T* p, float (&f)[V]) {
  Pack<T, V>::open(*reinterpret_cast<const typename Pack<T, V>::Raw*>(p), f);
}

// The taps [j][channel] and the bias of V channels from c on.
template <typename T, int V, int K>
__device__ __forceinline__ void taps(const T* w, const T* bias, int c, float (&wk)[K][V], float (&bs)[V]) {
  float f[K][V];  // V K neighbouring values, channel after channel
#pragma unroll
  for (int q = 0; q < K; ++q) ld<T, V>(w + (long)c * K + q * V, f[q]);
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < K; ++j) wk[j][i] = f[(i * K + j) / V][(i * K + j) % V];
  if (bias != nullptr) {
    ld<T, V>(bias + c, bs);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) bs[i] = 0.f;
  }
}

// c += a b over V channels, two to an instruction where V > 1.
template <int V>
__device__ __forceinline__ void fma_v(float (&c)[V], const float (&a)[V], const float (&b)[V]) {
  if constexpr (V > 1) {
#pragma unroll
    for (int i = 0; i < V; i += 2)
      asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%0, %1};\n\t"
          "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
          : "+f"(c[i]), "+f"(c[i + 1])
          : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));
  } else {
    c[0] = fmaf(a[0], b[0], c[0]);
  }
}

template <int V>
__device__ __forceinline__ void zero(float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = 0.f;
}

template <typename T>
__device__ __forceinline__ float sigmoid(float x) {
  return sizeof(T) == 4 ? 1.f / (1.f + expf(-x)) : rcp_fast(1.f + ex2_fast(-1.4426950408889634f * x));
}

__device__ __forceinline__ int rows_of(const int* lengths, int b, int N) {
  return lengths == nullptr ? N : min(max(lengths[b], 0), N);
}

constexpr int U = 4;          // rows loaded at a time
constexpr int CG = 32;        // channel groups a block spans
constexpr int RG = 8;         // row runs a block spans

// y, and the history in place.  Rows at or past the sequence's length are
// written as zeros and not read.  The block of the first row group alone reads
// the history and, after a barrier, writes the new one.
template <typename T, int V, int K>
__global__ void __launch_bounds__(CG * RG, 3)
    k_conv_fwd(const T* __restrict__ x, const T* __restrict__ w, const T* __restrict__ bias, const int* __restrict__ lengths,
               T* state, T* __restrict__ y, int N, int C, long ldx, int silu, int run) {
  const int c = (blockIdx.x * CG + threadIdx.x) * V;
  const int b = blockIdx.z;
  const bool live = c < C;
  const int L = rows_of(lengths, b, N);
  const T* xb = x + (long)b * N * ldx + c;
  T* sb = state == nullptr ? nullptr : state + (long)b * (K - 1) * C + c;
  // grid.y is capped: a block walks row groups at the grid's stride
  for (int rg = blockIdx.y; (long)rg * RG * run < N; rg += gridDim.y) {
    const int t0 = (rg * RG + threadIdx.y) * run;
    if (live && t0 < N) {
      float wk[K][V], bs[V], h[K][V];
      taps<T, V, K>(w, bias, c, wk, bs);
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {  // the K - 1 rows before the run
        const int t = t0 - (K - 1) + j;
        if (t >= 0 && t < L)
          ld<T, V>(xb + t * ldx, h[j + 1]);
        else if (t < 0 && sb != nullptr)
          ld<T, V>(sb + (long)(t + K - 1) * C, h[j + 1]);
        else
          zero(h[j + 1]);
      }
      T* yb = y + ((long)b * N + t0) * C + c;
      using Raw = typename Pack<T, V>::Raw;
      Raw next[U];
      auto fetch = [&](int r0) {
        const T* p = xb + (t0 + r0) * ldx;
        if (r0 < run && t0 + r0 + U <= L) {
#pragma unroll
          for (int r = 0; r < U; ++r) next[r] = *reinterpret_cast<const Raw*>(p + r * ldx);
        } else {
#pragma unroll
          for (int r = 0; r < U; ++r) {
            next[r] = Raw{};
            if (r0 < run && t0 + r0 + r < L) next[r] = *reinterpret_cast<const Raw*>(p + r * ldx);
          }
        }
      };
      fetch(0);
#pragma unroll 1
      for (int r0 = 0; r0 < run && t0 + r0 < N; r0 += U) {
        Raw in[U];
        float o[U][V];
#pragma unroll
        for (int r = 0; r < U; ++r) in[r] = next[r];
        fetch(r0 + U);
#pragma unroll
        for (int r = 0; r < U; ++r) {  // rows past the length: zeros in, not used
#pragma unroll
          for (int j = 0; j < K - 1; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) h[j][i] = h[j + 1][i];
          Pack<T, V>::open(in[r], h[K - 1]);
#pragma unroll
          for (int i = 0; i < V; ++i) o[r][i] = bs[i];
#pragma unroll
          for (int j = 0; j < K; ++j) fma_v(o[r], wk[j], h[j]);
          if (silu) {
#pragma unroll
            for (int i = 0; i < V; ++i) o[r][i] *= sigmoid<T>(o[r][i]);
          }
        }
        T* q = yb + (long)r0 * C;
        if (t0 + r0 + U <= L) {
#pragma unroll
          for (int r = 0; r < U; ++r) Pack<T, V>::st(q + (long)r * C, o[r]);
        } else {
#pragma unroll
          for (int r = 0; r < U; ++r) {
            if (t0 + r0 + r >= L) zero(o[r]);
            if (t0 + r0 + r < N) Pack<T, V>::st(q + (long)r * C, o[r]);
          }
        }
      }
    }
    if (rg == 0 && state != nullptr) {
      __syncthreads();  // the history's readers are this block's first rows
      if (live && threadIdx.y == 0) {
        float n[K - 1][V];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
          const int t = L - (K - 1) + j;
          if (t >= 0)
            ld<T, V>(xb + t * ldx, n[j]);
          else
            ld<T, V>(sb + (long)(t + K - 1) * C, n[j]);
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) Pack<T, V>::st(sb + (long)j * C, n[j]);
      }
    }
  }
}

// dx, and each block's sums of g x and g over its rows into
// part[group][K + 1][C] (fp32; the last plane is the bias's).  History zero.  (At
// one channel a bound on the blocks makes the compiler take more than 64
// registers: 76 us fp32 against 64.)
template <typename T, int V, int K>
__global__ void __launch_bounds__(CG * RG, V == 1 ? 0 : 2)
    k_conv_bwd(const T* __restrict__ x, const T* __restrict__ w, const T* __restrict__ bias, const int* __restrict__ lengths,
               const T* __restrict__ dy, T* __restrict__ dx, float* __restrict__ part, int N, int C, long ldx, int silu,
               int groups, int walk) {
  const int run = walk - (K - 1);  // the last K - 1 rows of a walk only complete those before them
  __shared__ float red[K + 1][RG][CG * V];
  const int c = (blockIdx.x * CG + threadIdx.x) * V;
  const bool live = c < C;
  const int b = blockIdx.z;
  const int L = rows_of(lengths, b, N);
  const T* xb = x + (long)b * N * ldx + c;
  const T* gb = dy + (long)b * N * C + c;
  T* ob = dx + (long)b * N * C + c;
  float wk[K][V], bs[V];
  if (live) taps<T, V, K>(w, bias, c, wk, bs);
  for (int rg = blockIdx.y; rg < groups; rg += gridDim.y) {
    float sums[K + 1][V];
#pragma unroll
    for (int j = 0; j <= K; ++j) zero(sums[j]);
    const int t0 = (rg * RG + threadIdx.y) * run;
    if (live && t0 < N) {
      // h: x rows t - K + 1 .. t;  g: rows t - K + 1 .. t of dy silu'(pre).
      // Row t's g completes dx of row t - K + 1, so the run looks K - 1 rows ahead.
      float h[K][V], g[K][V];
#pragma unroll
      for (int j = 0; j < K; ++j) zero(g[j]);
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const int t = t0 - (K - 1) + j;
        if (t >= 0 && t < L)
          ld<T, V>(xb + t * ldx, h[j + 1]);
        else
          zero(h[j + 1]);
      }
      using Raw = typename Pack<T, V>::Raw;
      Raw xn[U], gn[U];
      auto fetch = [&](int r0) {
        const T *p = xb + (t0 + r0) * ldx, *q = gb + (long)(t0 + r0) * C;
        if (r0 < walk && t0 + r0 + U <= L) {
#pragma unroll
          for (int r = 0; r < U; ++r) {
            xn[r] = *reinterpret_cast<const Raw*>(p + r * ldx);
            gn[r] = *reinterpret_cast<const Raw*>(q + (long)r * C);
          }
        } else {
#pragma unroll
          for (int r = 0; r < U; ++r) {
            xn[r] = gn[r] = Raw{};
            if (r0 < walk && t0 + r0 + r < L) {
              xn[r] = *reinterpret_cast<const Raw*>(p + r * ldx);
              gn[r] = *reinterpret_cast<const Raw*>(q + (long)r * C);
            }
          }
        }
      };
      fetch(0);
#pragma unroll 1
      for (int r0 = 0; r0 < walk && t0 + r0 < N + K - 1; r0 += U) {
        Raw xi[U], gi[U];
#pragma unroll
        for (int r = 0; r < U; ++r) xi[r] = xn[r], gi[r] = gn[r];
        fetch(r0 + U);
        const bool whole = r0 > 0 && t0 + r0 + U <= L;  // every row complete and stored
        T* q = ob + (long)(t0 + r0 - (K - 1)) * C;
#pragma unroll
        for (int r = 0; r < U; ++r) {
#pragma unroll
          for (int j = 0; j < K - 1; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) h[j][i] = h[j + 1][i], g[j][i] = g[j + 1][i];
          Pack<T, V>::open(xi[r], h[K - 1]);
          Pack<T, V>::open(gi[r], g[K - 1]);  // zero past the length
          if (silu) {
            float p[V];
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = bs[i];
#pragma unroll
            for (int j = 0; j < K; ++j) fma_v(p, wk[j], h[j]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float s = sigmoid<T>(p[i]);
              g[K - 1][i] *= s * fmaf(p[i], 1.f - s, 1.f);
            }
          }
          if (r0 + r < run) {
#pragma unroll
            for (int i = 0; i < V; ++i) sums[K][i] += g[K - 1][i];
#pragma unroll
            for (int j = 0; j < K; ++j) fma_v(sums[j], g[K - 1], h[j]);
          }
          float o[V];  // of row t - (K - 1), which is complete
          zero(o);
#pragma unroll
          for (int j = 0; j < K; ++j) fma_v(o, wk[K - 1 - j], g[j]);
          if (whole) {
            Pack<T, V>::st(q + (long)r * C, o);
          } else if (r0 + r >= K - 1) {
            const int to = t0 + r0 + r - (K - 1);
            if (to >= L) zero(o);
            if (to < N) Pack<T, V>::st(q + (long)r * C, o);
          }
        }
      }
    }
    float* pb = part + ((long)b * groups + rg) * (K + 1) * C;
    __syncthreads();  // the last group's sums have been read
#pragma unroll
    for (int j = 0; j <= K; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) red[j][threadIdx.y][threadIdx.x * V + i] = sums[j][i];
    __syncthreads();
    for (int e = threadIdx.y * CG + threadIdx.x; e < (K + 1) * CG * V; e += CG * RG) {
      const int j = e / (CG * V), x_ = e % (CG * V), ch = blockIdx.x * CG * V + x_;
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < RG; ++q) s += red[j][q][x_];
      if (ch < C) pb[(long)j * C + ch] = s;
    }
  }
}

// dw[c][j] and db[c] from the P blocks' sums, in a fixed order: RS threads a
// value, each a strided share, joined in shared memory.
constexpr int RS = 8;
template <typename T>
__global__ void __launch_bounds__(32 * RS)
    k_conv_sum(const float* __restrict__ part, T* __restrict__ dw, T* __restrict__ db, int P, int C, int K) {
  grid_dep_enter();
  __shared__ float red[RS][32];
  const int c = blockIdx.x * 32 + threadIdx.x, j = blockIdx.y;
  float s = 0.f;
  if (c < C) {
    const float* p = part + (long)j * C + c;
    const long stride = (long)(K + 1) * C;
#pragma unroll 4
    for (int i = threadIdx.y; i < P; i += RS) s += p[i * stride];
  }
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < C) {
    for (int q = 1; q < RS; ++q) s += red[q][threadIdx.x];
    if (j < K)
      dw[(long)c * K + j] = from_f<T>(s);
    else if (db != nullptr)
      db[c] = from_f<T>(s);
  }
}

// One row for each of B streams: y, and the history shifted in place.
template <typename T, int V, int K>
__global__ void __launch_bounds__(128)
    k_conv_step(const T* __restrict__ x, const T* __restrict__ w, const T* __restrict__ bias, T* __restrict__ state,
                T* __restrict__ y, int B, int C, long ldx, int silu) {
  const int per = C / V;
  const long e = (long)blockIdx.x * 128 + threadIdx.x;
  if (e >= (long)B * per) return;
  const int b = (int)(e / per), c = (int)(e % per) * V;
  float h[K][V], o[V];
  T* sb = state + (long)b * (K - 1) * C + c;
#pragma unroll
  for (int j = 0; j < K - 1; ++j) ld<T, V>(sb + (long)j * C, h[j]);
  ld<T, V>(x + b * ldx + c, h[K - 1]);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float p = bias == nullptr ? 0.f : to_f(bias[c + i]);
#pragma unroll
    for (int j = 0; j < K; ++j) p = fmaf(to_f(w[(long)(c + i) * K + j]), h[j][i], p);
    o[i] = silu ? p * sigmoid<T>(p) : p;
  }
  Pack<T, V>::st(y + (long)b * C + c, o);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) Pack<T, V>::st(sb + (long)j * C, h[j + 1]);
}

// Rows a thread walks (a multiple of U): the walk that minimises whole waves of
// blocks times its length and start-up, `lost` of its rows being repeated.
struct Walk {
  int rows, groups;
  Walk(int N, long columns, int lost, int per_sm) {
    const long slots = (long)per_sm * sm_count();
    double best = 0;
    rows = U, groups = 1;
    for (int r = 2 * U; r <= 16 * U; r += U) {
      const int g = (N + (r - lost) * RG - 1) / ((r - lost) * RG);
      const long waves = (columns * g + slots - 1) / slots;
      const double cost = (double)waves * (r + 6);
      if (r == 2 * U || cost < best) best = cost, rows = r, groups = g;
    }
  }
};

Walk bwd_walk(const ConvShape& s, int v) {
  return Walk(s.N, (long)s.B * ((s.C + CG * v - 1) / (CG * v)), s.K - 1, 2);
}

// Channels a thread owns: four, or two for the gradients in fp32, whose rows in
// flight would not fit the registers otherwise; one where a row may start off
// such a vector (C, the row stride or x's base not its multiple; all other bases
// are 16-byte aligned by the interface).  Measured at 4 x 2048 x 2304, K = 4:
//   bf16 forward 22.5 us (one channel 45.1), gradients 38.9 (51.2);
//   fp32 forward 34.8 (two channels 36.9, one 47.1), gradients 59.4 (four 66.2, one 63.5).
constexpr int wide(bool bf, bool grad) { return grad && !bf ? 2 : 4; }
int channels(const void* x, const ConvShape& s, bool grad) {
  const int v = wide(s.dtype != 0, grad), elem = s.dtype == 0 ? 4 : 2;
  return s.C % v == 0 && s.ldx % v == 0 && reinterpret_cast<uintptr_t>(x) % (v * elem) == 0 ? v : 1;
}

#define LA_CONV_CASE(T, V, Kv, BODY) \
  { using T_ = T; constexpr int V_ = V, K_ = Kv; BODY; }
#define LA_CONV_K(T, V, K, BODY)             \
  do {                                       \
    if ((K) == 2) LA_CONV_CASE(T, V, 2, BODY) \
    else if ((K) == 3) LA_CONV_CASE(T, V, 3, BODY) \
    else LA_CONV_CASE(T, V, 4, BODY)          \
  } while (0)
#define LA_CONV_DISPATCH(dtype, v, WF, K, BODY)       \
  do {                                                \
    if ((dtype) == 0) {                               \
      if ((v) > 1) LA_CONV_K(float, WF, K, BODY);     \
      else LA_CONV_K(float, 1, K, BODY);              \
    } else {                                          \
      if ((v) > 1) LA_CONV_K(bf16, 4, K, BODY);       \
      else LA_CONV_K(bf16, 1, K, BODY);               \
    }                                                 \
  } while (0)

}  // namespace

size_t short_conv_bwd_ws_bytes(const ConvShape& s) {  // whichever form x's alignment leaves
  const int g = std::max(bwd_walk(s, 1).groups, bwd_walk(s, wide(s.dtype != 0, true)).groups);
  return sizeof(float) * s.B * (size_t)g * (s.K + 1) * s.C;
}

cudaError_t short_conv_fwd(const void* x, const void* w, const void* bias, const int* lengths, void* state, void* y,
                           const ConvShape& s, cudaStream_t st) {
  const int v = channels(x, s, false), per = CG * v;
  const Walk plan(s.N, (long)s.B * ((s.C + per - 1) / per), 0, 3);
  const dim3 grid((s.C + per - 1) / per, plan.groups < 65535 ? plan.groups : 65535, s.B), block(CG, RG);
  LA_CONV_DISPATCH(s.dtype, v, 4, s.K,
                   (k_conv_fwd<T_, V_, K_><<<grid, block, 0, st>>>((const T_*)x, (const T_*)w, (const T_*)bias, lengths,
                                                                   (T_*)state, (T_*)y, s.N, s.C, s.ldx, s.silu, plan.rows)));
  return cudaGetLastError();
}

cudaError_t short_conv_bwd(const void* x, const void* w, const void* bias, const int* lengths, const void* dy, void* dx,
                           void* dw, void* db, float* ws, const ConvShape& s, cudaStream_t st) {
  const int v = channels(x, s, true), per = CG * v;
  const Walk plan = bwd_walk(s, v);
  const int groups = plan.groups;
  const dim3 grid((s.C + per - 1) / per, groups < 65535 ? groups : 65535, s.B), block(CG, RG);
  LA_CONV_DISPATCH(s.dtype, v, 2, s.K,
                   (k_conv_bwd<T_, V_, K_><<<grid, block, 0, st>>>((const T_*)x, (const T_*)w, (const T_*)bias, lengths,
                                                                   (const T_*)dy, (T_*)dx, ws, s.N, s.C, s.ldx, s.silu,
                                                                   groups, plan.rows)));
  const dim3 sgrid((s.C + 31) / 32, s.K + 1), sblock(32, RS);
  const int P = s.B * groups;
  if (s.dtype == 0)
    return launch_pdl(k_conv_sum<float>, sgrid, sblock, 0, st, (const float*)ws, (float*)dw, (float*)db, P, s.C, s.K);
  return launch_pdl(k_conv_sum<bf16>, sgrid, sblock, 0, st, (const float*)ws, (bf16*)dw, (bf16*)db, P, s.C, s.K);
}

cudaError_t short_conv_step(const void* x, const void* w, const void* bias, void* state, void* y, const ConvShape& s,
                            cudaStream_t st) {
  const int v = channels(x, s, false);
  const long n = (long)s.B * (s.C / v);
  const unsigned grid = (unsigned)((n + 127) / 128);
  LA_CONV_DISPATCH(s.dtype, v, 4, s.K,
                   (k_conv_step<T_, V_, K_><<<grid, 128, 0, st>>>((const T_*)x, (const T_*)w, (const T_*)bias, (T_*)state,
                                                                  (T_*)y, s.B, s.C, s.ldx, s.silu)));
  return cudaGetLastError();
}

}  // namespace la
