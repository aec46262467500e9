// Layer norm over the groups of a row (one group: the whole row; H groups: every head
// of a scan's output by itself), behind an optional residual sum:
//   s = x + residual (kept in the rows' type), xh = (s - mean) rstd, y = xh w + b,
//   rstd = 1 / sqrt(mean((s - mean)^2) + eps),
// and its gradients, with dxh = w dy and ds the gradient that reaches s directly:
//   dx = (dxh - mean(dxh) - xh mean(dxh xh)) rstd + ds,  dw = sum dy xh,  db = sum dy.
//
// Bound by HBM: TPR threads hold a group's M values in registers, so each is read
// once; the variance is the mean of squared differences, in a second step over the
// registers.  Means, variances and all sums are fp32.  Backward, blocks walk rows at
// a stride that keeps a thread on the same columns, whose sums dw and db it holds in
// registers; a second kernel adds the blocks' sums up in a fixed order.
#include <algorithm>
#include <numeric>

#include "scan.cuh"

namespace la {
namespace {

using bf16 = __nv_bfloat16;

// V neighbouring values as one vector of up to 16 bytes (V > 1: the caller has
// checked the alignment).
template <typename T, int V>
struct Vec;
template <typename T>
struct Vec<T, 1> {
  __device__ __forceinline__ static void ld(const T* p, float* f) { f[0] = to_f(*p); }
  __device__ __forceinline__ static void st(T* p, const float* f) { *p = from_f<T>(f[0]); }
};
template <>
struct Vec<float, 4> {
  __device__ __forceinline__ static void ld(const float* p, float* f) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
  }
  __device__ __forceinline__ static void st(float* p, const float* f) { *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Vec<bf16, 8> {
  __device__ __forceinline__ static void ld(const bf16* p, float* f) { Vec16<bf16>::unpack(*reinterpret_cast<const uint4*>(p), f); }
  __device__ __forceinline__ static void st(bf16* p, const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Sums a and b over the TPR threads of a group; every thread gets them.  More than a
// warp: through red, which the barriers around it keep from being overwritten early.
template <int TPR>
__device__ __forceinline__ void group_sum(float& a, float& b, float2* red) {
  constexpr int in_warp = TPR < 32 ? TPR : 32;
#pragma unroll
  for (int o = in_warp / 2; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (TPR > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) a += red[i].x, b += red[i].y;
  }
}

struct NormArgs {
  const void *x, *res, *w, *b;
  void *y, *s;
  float *mean, *rstd;
  const int* lengths;
  long items, ldx, ldr;  // items: rows times groups; ldx, ldr: elements between rows
  int N, G, M;
  float eps;
};

// Columns of a thread: k-th vector at (k TPR + lane) V.
template <typename T, int V, int K, int TPR>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) k_norm_fwd(const NormArgs a) {
  constexpr int NT = TPR > 256 ? TPR : 256, PER = NT / TPR;
  __shared__ float2 red[TPR > 32 ? TPR / 32 : 1];
  static_assert(TPR <= 32 || PER == 1, "more than a warp: the whole block");
  const int lane = threadIdx.x % TPR;
  const long item = (long)blockIdx.x * PER + threadIdx.x / TPR;
  const bool in = item < a.items;  // every thread stays for the sums
  const long row = in ? item / a.G : 0;
  const int g = in ? static_cast<int>(item - row * a.G) : 0;
  const bool live = in && (a.lengths == nullptr || static_cast<int>(row % a.N) < a.lengths[row / a.N]);
  const T* x = static_cast<const T*>(a.x) + row * a.ldx + (long)g * a.M;
  const T* res = a.res == nullptr ? nullptr : static_cast<const T*>(a.res) + row * a.ldr + (long)g * a.M;
  T* y = static_cast<T*>(a.y) + item * a.M;
  T* s = a.res == nullptr ? nullptr : static_cast<T*>(a.s) + item * a.M;
  float f[K][V];
  float sum = 0.f, none = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * TPR + lane) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) f[k][i] = 0.f;
    if (live && c < a.M) {
      Vec<T, V>::ld(x + c, f[k]);
      if (res != nullptr) {
        float r[V];
        Vec<T, V>::ld(res + c, r);
#pragma unroll
        for (int i = 0; i < V; ++i) f[k][i] = to_f(from_f<T>(f[k][i] + r[i]));
      }
    }
    if (s != nullptr && in && c < a.M) Vec<T, V>::st(s + c, f[k]);
#pragma unroll
    for (int i = 0; i < V; ++i) sum += f[k][i];
  }
  group_sum<TPR>(sum, none, red);
  const float mean = sum / a.M;
  float sq = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if ((k * TPR + lane) * V < a.M) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f[k][i] -= mean;
        sq = fmaf(f[k][i], f[k][i], sq);
      }
    }
  }
  group_sum<TPR>(sq, none, red);
  const float rstd = rsqrtf(sq / a.M + a.eps);
  if (!in) return;
  const T *w = static_cast<const T*>(a.w) + (long)g * a.M, *b = a.b == nullptr ? nullptr : static_cast<const T*>(a.b) + (long)g * a.M;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * TPR + lane) * V;
    if (c < a.M) {
      float o[V], wv[V], bv[V];
      Vec<T, V>::ld(w + c, wv);
#pragma unroll
      for (int i = 0; i < V; ++i) bv[i] = 0.f;
      if (b != nullptr) Vec<T, V>::ld(b + c, bv);
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = live ? fmaf(f[k][i] * rstd, wv[i], bv[i]) : 0.f;
      Vec<T, V>::st(y + c, o);
    }
  }
  if (lane == 0 && a.mean != nullptr) {
    a.mean[item] = live ? mean : 0.f;
    a.rstd[item] = live ? rstd : 0.f;
  }
}

struct GradArgs {
  const void *s, *w, *dy, *ds;
  const float *mean, *rstd;
  const int* lengths;
  void* dx;
  float* part;  // [2][slots][M]: dw, db
  long items, lds, slots;
  int N, G, M;
};

// Slot (block, group of threads) takes items slot, slot + slots, ...; slots is a
// multiple of G, so a thread's columns, and their sums, stay the same.
template <typename T, int V, int K, int TPR>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) k_norm_bwd(const GradArgs a) {
  constexpr int NT = TPR > 256 ? TPR : 256, PER = NT / TPR;
  __shared__ float2 red[TPR > 32 ? TPR / 32 : 1];
  const int lane = threadIdx.x % TPR;
  const long slot = (long)blockIdx.x * PER + threadIdx.x / TPR;
  const int g = static_cast<int>(slot % a.G);
  const T* w = static_cast<const T*>(a.w) + (long)g * a.M;
  float dw[K][V], db[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[k][i] = db[k][i] = 0.f;
  for (long base = 0; base < a.items; base += a.slots) {  // the same steps for all threads: they meet in the sums
    const long item = base + slot;
    const bool in = item < a.items;
    const long row = in ? item / a.G : 0;
    const bool live = in && (a.lengths == nullptr || static_cast<int>(row % a.N) < a.lengths[row / a.N]);
    const T* s = static_cast<const T*>(a.s) + row * a.lds + (long)g * a.M;
    const long at = item * a.M;
    const float mean = live ? a.mean[item] : 0.f, rstd = live ? a.rstd[item] : 0.f;
    float f[K][V], d[K][V];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * TPR + lane) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) f[k][i] = d[k][i] = 0.f;
      if (live && c < a.M) {
        float wv[V];
        Vec<T, V>::ld(s + c, f[k]);
        Vec<T, V>::ld(static_cast<const T*>(a.dy) + at + c, d[k]);
        Vec<T, V>::ld(w + c, wv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          f[k][i] = (f[k][i] - mean) * rstd;
          dw[k][i] = fmaf(d[k][i], f[k][i], dw[k][i]);
          db[k][i] += d[k][i];
          d[k][i] *= wv[i];
          s1 += d[k][i];
          s2 = fmaf(d[k][i], f[k][i], s2);
        }
      }
    }
    group_sum<TPR>(s1, s2, red);
    s1 /= a.M, s2 /= a.M;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * TPR + lane) * V;
      if (in && c < a.M) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = (d[k][i] - s1 - f[k][i] * s2) * rstd;
        if (live && a.ds != nullptr) {
          float e[V];
          Vec<T, V>::ld(static_cast<const T*>(a.ds) + at + c, e);
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] += e[i];
        }
        Vec<T, V>::st(static_cast<T*>(a.dx) + at + c, o);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * TPR + lane) * V;
    if (c < a.M) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        a.part[slot * a.M + c + i] = dw[k][i];
        a.part[(a.slots + slot) * a.M + c + i] = db[k][i];
      }
    }
  }
}

// dw and db: column c of the [slots / G][C] partial sums, 32 columns a block, eight
// rows at a time.
template <typename T>
__global__ void __launch_bounds__(256) k_norm_join(const float* __restrict__ part, T* __restrict__ dw, T* __restrict__ db, long P, int C) {
  __shared__ float red[8][33];
  grid_dep_enter();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
  const float* p = part + (blockIdx.y ? P * C : 0);
  float v = 0.f;
  if (c < C)
    for (long i = ty; i < P; i += 8) v += p[i * C + c];
  red[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += red[i][tx];
    T* o = blockIdx.y ? db : dw;
    if (o != nullptr) o[c] = from_f<T>(v);
  }
}

// How a group is held: f<V, K, TPR>() of the smallest shape that covers M.
template <typename T, typename F>
cudaError_t shaped(int M, bool vec, F&& f) {
  constexpr int V = 16 / sizeof(T);
#define LA_NORM_SHAPE(VV, KK, TT) \
  if (M <= (VV) * (KK) * (TT)) return f.template run<VV, KK, TT>();
  if (vec) {
    LA_NORM_SHAPE(V, 1, 4)
    LA_NORM_SHAPE(V, 1, 8)
    LA_NORM_SHAPE(V, 1, 16)
    LA_NORM_SHAPE(V, 1, 32)
    LA_NORM_SHAPE(V, 2, 32)
    LA_NORM_SHAPE(V, 4, 32)
    LA_NORM_SHAPE(V, 1, 256)
    LA_NORM_SHAPE(V, 2, 256)
    LA_NORM_SHAPE(V, 4, 256)
    LA_NORM_SHAPE(V, 4, 512)
  } else {
    LA_NORM_SHAPE(1, 1, 8)
    LA_NORM_SHAPE(1, 1, 32)
    LA_NORM_SHAPE(1, 4, 32)
    LA_NORM_SHAPE(1, 4, 256)
    LA_NORM_SHAPE(1, 8, 256)
    LA_NORM_SHAPE(1, 8, 1024)
  }
#undef LA_NORM_SHAPE
  return cudaErrorInvalidValue;
}

template <typename T>
struct Forward {
  const NormArgs& a;
  cudaStream_t st;
  template <int V, int K, int TPR>
  cudaError_t run() {
    constexpr int NT = TPR > 256 ? TPR : 256, PER = NT / TPR;
    k_norm_fwd<T, V, K, TPR><<<static_cast<unsigned>((a.items + PER - 1) / PER), NT, 0, st>>>(a);
    return cudaGetLastError();
  }
};

struct SlotPlan {
  long blocks, slots;
};

// As many blocks as run at once, and a multiple of what keeps slots a multiple of G.
SlotPlan plan(long items, int G, int per, int threads) {
  const long unit = G / std::gcd(G, per);
  const long most = (items + per - 1) / per, want = std::min<long>(most, (long)sm_count() * (1024 / threads));
  const long blocks = (want + unit - 1) / unit * unit;
  return {blocks, blocks * per};
}

template <typename T>
struct Backward {
  GradArgs& a;
  void *dw, *db;
  cudaStream_t st;
  template <int V, int K, int TPR>
  cudaError_t run() {
    constexpr int NT = TPR > 256 ? TPR : 256, PER = NT / TPR;
    const SlotPlan p = plan(a.items, a.G, PER, NT);
    a.slots = p.slots;
    k_norm_bwd<T, V, K, TPR><<<static_cast<unsigned>(p.blocks), NT, 0, st>>>(a);
    const int C = a.G * a.M;
    return launch_pdl(k_norm_join<T>, dim3((C + 31) / 32, 2), dim3(256), 0, st, (const float*)a.part, (T*)dw, (T*)db, p.slots / a.G, C);
  }
};

struct Floats {
  long items;
  int G, M;
  size_t& n;
  template <int V, int K, int TPR>
  cudaError_t run() {
    constexpr int NT = TPR > 256 ? TPR : 256;
    n = 2 * static_cast<size_t>(plan(items, G, NT / TPR, NT).slots) * M;
    return cudaSuccess;
  }
};

bool vectors(const NormShape& s, long ld, std::initializer_list<const void*> ps) {
  const int V = s.dtype == 0 ? 4 : 8;
  const int M = s.C / s.G;
  if (M % V || ld % V) return false;
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  return true;
}

}  // namespace

// Either way of holding a group: the strides decide at the call.
size_t norm_bwd_ws_bytes(const NormShape& s) {
  size_t a = 0, b = 0;
  const int M = s.C / s.G;
  Floats fa{(long)s.B * s.N, s.G, M, a}, fb{(long)s.B * s.N, s.G, M, b};
  fa.items *= s.G, fb.items *= s.G;
  if (s.dtype == 0) {
    shaped<float>(M, true, fa), shaped<float>(M, false, fb);
  } else {
    shaped<bf16>(M, true, fa), shaped<bf16>(M, false, fb);
  }
  return 4 * std::max(a, b);
}

cudaError_t norm_fwd(const void* x, const void* res, const void* w, const void* b, const int* lengths, void* y, void* s, float* mean,
                     float* rstd, float eps, const NormShape& sh, cudaStream_t st) {
  const NormArgs a{x, res, w, b, y, s, mean, rstd, lengths, (long)sh.B * sh.N * sh.G, sh.ldx, sh.ldr, sh.N, sh.G, sh.C / sh.G, eps};
  const bool vec = vectors(sh, sh.ldx, {x, res}) && (res == nullptr || sh.ldr % (sh.dtype == 0 ? 4 : 8) == 0);
  if (sh.dtype == 0) return shaped<float>(a.M, vec, Forward<float>{a, st});
  return shaped<bf16>(a.M, vec, Forward<bf16>{a, st});
}

cudaError_t norm_bwd(const void* s, const void* w, const float* mean, const float* rstd, const int* lengths, const void* dy, const void* ds,
                     void* dx, void* dw, void* db, float* ws, const NormShape& sh, cudaStream_t st) {
  GradArgs a{s, w, dy, ds, mean, rstd, lengths, dx, ws, (long)sh.B * sh.N * sh.G, sh.ldx, 0, sh.N, sh.G, sh.C / sh.G};
  const bool vec = vectors(sh, sh.ldx, {s});
  if (sh.dtype == 0) return shaped<float>(a.M, vec, Backward<float>{a, dw, db, st});
  return shaped<bf16>(a.M, vec, Backward<bf16>{a, dw, db, st});
}

}  // namespace la
