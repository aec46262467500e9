// Layer norm over the groups of a row (one group: the whole row; H groups: every head
// of a scan's output by itself), behind an optional residual sum:
//   s = x + residual (kept in the rows' type), xh = (s - mean) rstd, y = xh w + b,
//   rstd = 1 / sqrt(mean((s - mean)^2) + eps),
// and its gradients, with dxh = w dy and ds the gradient that reaches s directly:
//   dx = (dxh - mean(dxh) - xh mean(dxh xh)) rstd + ds,  dw = sum dy xh,  db = sum dy.
//
// Bound by HBM: TPR threads hold a group's M values in registers, so each is read
// once, R groups at a time so that enough loads are on their way; the variance is the
// mean of squared differences, in a second step over the registers.  Means, variances
// and all sums are fp32.  Backward, blocks walk rows at a stride that keeps a thread on
// the same columns, whose sums dw and db it holds in registers; a second kernel adds the
// blocks' sums up in a fixed order.
#include <algorithm>
#include <numeric>

#include "scan.cuh"

namespace la {
namespace {

using bf16 = __nv_bfloat16;

// V neighbouring values as one vector of up to 16 bytes (V > 1: the caller has
// checked the alignment), as it lies in memory and as fp32.
template <typename T, int V>
struct Vec;
template <typename T>
struct Vec<T, 1> {
  using Raw = T;
  __device__ __forceinline__ static void open(const Raw& u, float* f) { f[0] = to_f(u); }
  __device__ __forceinline__ static Raw close(const float* f) { return from_f<T>(f[0]); }
};
template <>
struct Vec<float, 4> {
  using Raw = float4;
  __device__ __forceinline__ static void open(const Raw& u, float* f) { f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w; }
  __device__ __forceinline__ static Raw close(const float* f) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Vec<bf16, 8> {
  using Raw = uint4;
  __device__ __forceinline__ static void open(const Raw& u, float* f) { Vec16<bf16>::unpack(u, f); }
  __device__ __forceinline__ static Raw close(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <typename T, int V>
__device__ __forceinline__ typename Vec<T, V>::Raw get(const T* p) {
  return *reinterpret_cast<const typename Vec<T, V>::Raw*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void set(T* p, const typename Vec<T, V>::Raw& v) {
  *reinterpret_cast<typename Vec<T, V>::Raw*>(p) = v;
}

// A group of more than a warp is a block of its own.
template <int TPR>
constexpr int THREADS = TPR > 32 ? TPR : 256;

// Sums of n values each over the TPR threads of a group; every thread gets them.  More
// than a warp: through red, of which successive calls use alternate halves.
template <int TPR, int n>
struct Sums {
  float (*red)[n][TPR > 32 ? TPR / 32 : 1];
  int half = 0;
  __device__ __forceinline__ void operator()(float (&v)[n]) {
    constexpr int in_warp = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = in_warp / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < n; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (TPR > 32) {
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < n; ++i) red[half][i][threadIdx.x >> 5] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < n; ++i) {
        v[i] = 0.f;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) v[i] += red[half][i][w];
      }
      half ^= 1;
    }
  }
};

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

// Where an item (a group of a row) is.
struct Place {
  Divide groups, rows;  // by the groups of a row, by the rows of a sequence
  const int* lengths;
  long items;
  __device__ __forceinline__ void of(long item, bool& in, bool& live, uint32_t& row, uint32_t& g) const {
    in = item < items;
    const uint32_t i = in ? static_cast<uint32_t>(item) : 0u;
    row = groups(i);
    g = i - row * groups.d;
    live = in;
    if (lengths != nullptr) {
      const uint32_t b = rows(row);
      live = in && static_cast<int>(row - b * rows.d) < lengths[b];
    }
  }
};

struct NormArgs {
  const void *x, *res, *w, *b;
  void *y, *s;
  float *mean, *rstd;
  Place at;
  long ldx, ldr;  // elements between rows
  int M;
  float eps;
};

// Columns of a thread: k-th vector at (k TPR + lane) V.
template <typename T, int V, int K, int TPR, int R>
__global__ void __launch_bounds__(THREADS<TPR>) k_norm_fwd(const NormArgs a) {
  using Raw = typename Vec<T, V>::Raw;
  constexpr int PER = THREADS<TPR> / TPR;
  __shared__ float red[2][R][TPR > 32 ? TPR / 32 : 1];
  Sums<TPR, R> sum{red};
  const int lane = threadIdx.x % TPR;
  const long first = (long)blockIdx.x * (R * PER) + threadIdx.x / TPR;
  bool in[R], live[R];  // every thread stays for the sums
  uint32_t row[R], g[R];
  Raw x[R][K], res[R][K];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    a.at.of(first + r * PER, in[r], live[r], row[r], g[r]);
    const T* p = static_cast<const T*>(a.x) + row[r] * a.ldx + (long)g[r] * a.M;
    const T* q = static_cast<const T*>(a.res) + row[r] * a.ldr + (long)g[r] * a.M;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * TPR + lane) * V;
      x[r][k] = res[r][k] = Raw{};
      if (live[r] && c < a.M) {
        x[r][k] = get<T, V>(p + c);
        if (a.res != nullptr) res[r][k] = get<T, V>(q + c);
      }
    }
  }
  float f[R][K][V], v[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    v[r] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * TPR + lane) * V;
      Vec<T, V>::open(x[r][k], f[r][k]);
      if (a.res != nullptr) {
        float e[V];
        Vec<T, V>::open(res[r][k], e);
#pragma unroll
        for (int i = 0; i < V; ++i) f[r][k][i] += e[i];
        const Raw total = Vec<T, V>::close(f[r][k]);
        Vec<T, V>::open(total, f[r][k]);
        if (in[r] && c < a.M) set<T, V>(static_cast<T*>(a.s) + (first + r * PER) * a.M + c, total);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) v[r] += f[r][k][i];
    }
  }
  sum(v);
  float mean[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    mean[r] = v[r] / a.M;
    v[r] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if ((k * TPR + lane) * V < a.M) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          f[r][k][i] -= mean[r];
          v[r] = fmaf(f[r][k][i], f[r][k][i], v[r]);
        }
      }
  }
  sum(v);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (!in[r]) continue;
    const long item = first + r * PER;
    const float rstd = rsqrtf(v[r] / a.M + a.eps);
    const T *w = static_cast<const T*>(a.w) + (long)g[r] * a.M, *b = static_cast<const T*>(a.b) + (long)g[r] * a.M;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * TPR + lane) * V;
      if (c < a.M) {
        float o[V], wv[V], bv[V];
        Vec<T, V>::open(get<T, V>(w + c), wv);
#pragma unroll
        for (int i = 0; i < V; ++i) bv[i] = 0.f;
        if (a.b != nullptr) Vec<T, V>::open(get<T, V>(b + c), bv);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = live[r] ? fmaf(f[r][k][i] * rstd, wv[i], bv[i]) : 0.f;
        set<T, V>(static_cast<T*>(a.y) + item * a.M + c, Vec<T, V>::close(o));
      }
    }
    if (lane == 0 && a.mean != nullptr) {
      a.mean[item] = live[r] ? mean[r] : 0.f;
      a.rstd[item] = live[r] ? rstd : 0.f;
    }
  }
}

struct GradArgs {
  const void *s, *w, *dy, *ds;
  const float *mean, *rstd;
  void* dx;
  float* part;  // [2][rows][C]: dw, db
  Place at;
  long lds, slots;
  int M;
};

// How many groups' sums of its own a block leaves: those of its slots, or, where G
// divides them, of the G groups, added up over the slots that share one.
inline __host__ __device__ int distinct(int per, int G) { return per % G == 0 ? G : per; }

// Slot (block, group of threads) takes items slot, slot + slots, ...; slots is a
// multiple of G, so a thread's columns, and their sums, stay the same.
template <typename T, int V, int K, int TPR, int R>
__global__ void __launch_bounds__(THREADS<TPR>, (THREADS<TPR> < 512 ? 512 / THREADS<TPR> : 1)) k_norm_bwd(const GradArgs a) {
  using Raw = typename Vec<T, V>::Raw;
  constexpr int PER = THREADS<TPR> / TPR;
  __shared__ float red[2][2 * R][TPR > 32 ? TPR / 32 : 1];
  Sums<TPR, 2 * R> sum{red};
  const int lane = threadIdx.x % TPR;
  const long slot = (long)blockIdx.x * PER + threadIdx.x / TPR;
  const uint32_t own = static_cast<uint32_t>(slot % a.at.groups.d);
  const T* w = static_cast<const T*>(a.w) + (long)own * a.M;
  float dw[K][V], db[K][V];
  Raw wr[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * TPR + lane) * V;
    wr[k] = Raw{};
    if (c < a.M) wr[k] = get<T, V>(w + c);
#pragma unroll
    for (int i = 0; i < V; ++i) dw[k][i] = db[k][i] = 0.f;
  }
  for (long base = slot; base - slot < a.at.items; base += R * a.slots) {  // the same steps for all threads: they meet in the sums
    bool in[R], live[R];
    float mean[R], rstd[R];
    Raw sr[R][K], dr[R][K], er[R][K];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long item = base + r * a.slots, at = item * a.M;
      uint32_t row, g;
      a.at.of(item, in[r], live[r], row, g);
      const T* s = static_cast<const T*>(a.s) + row * a.lds + (long)g * a.M;
      mean[r] = live[r] ? a.mean[item] : 0.f, rstd[r] = live[r] ? a.rstd[item] : 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * TPR + lane) * V;
        sr[r][k] = dr[r][k] = er[r][k] = Raw{};
        if (live[r] && c < a.M) {
          sr[r][k] = get<T, V>(s + c);
          dr[r][k] = get<T, V>(static_cast<const T*>(a.dy) + at + c);
          if (a.ds != nullptr) er[r][k] = get<T, V>(static_cast<const T*>(a.ds) + at + c);
        }
      }
    }
    float v[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v[2 * r] = v[2 * r + 1] = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!live[r] || (k * TPR + lane) * V >= a.M) continue;
        float f[V], d[V], wv[V];
        Vec<T, V>::open(sr[r][k], f);
        Vec<T, V>::open(dr[r][k], d);
        Vec<T, V>::open(wr[k], wv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          f[i] = (f[i] - mean[r]) * rstd[r];
          dw[k][i] = fmaf(d[i], f[i], dw[k][i]);
          db[k][i] += d[i];
          d[i] *= wv[i];
          v[2 * r] += d[i];
          v[2 * r + 1] = fmaf(d[i], f[i], v[2 * r + 1]);
        }
      }
    }
    sum(v);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float s1 = v[2 * r] / a.M, s2 = v[2 * r + 1] / a.M;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * TPR + lane) * V;
        if (!in[r] || c >= a.M) continue;
        float f[V], d[V], wv[V], o[V];
        Vec<T, V>::open(sr[r][k], f);
        Vec<T, V>::open(dr[r][k], d);
        Vec<T, V>::open(wr[k], wv);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = (fmaf(d[i], wv[i], -s1) - (f[i] - mean[r]) * rstd[r] * s2) * rstd[r];
        if (a.ds != nullptr) {
          float e[V];
          Vec<T, V>::open(er[r][k], e);
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] += e[i];
        }
        if (!live[r])
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] = 0.f;
        set<T, V>(static_cast<T*>(a.dx) + (base + r * a.slots) * a.M + c, Vec<T, V>::close(o));
      }
    }
  }
  // the sums: [block][distinct groups][M], which is [..][C]
  const int G = a.at.groups.d, keep = distinct(PER, G);
  float* part = a.part + (long)blockIdx.x * keep * a.M;
  const long plane = (long)gridDim.x * keep * a.M;
  if constexpr (PER == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * TPR + lane) * V;
      if (c < a.M)
#pragma unroll
        for (int i = 0; i < V; ++i) part[c + i] = dw[k][i], part[plane + c + i] = db[k][i];
    }
  } else {
    __shared__ float all[PER * TPR * V * K];
    const int mine = threadIdx.x / TPR;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * TPR + lane) * V;
        if (c < a.M)
#pragma unroll
          for (int i = 0; i < V; ++i) all[mine * a.M + c + i] = which ? db[k][i] : dw[k][i];
      }
      __syncthreads();
      for (int e = threadIdx.x; e < keep * a.M; e += THREADS<TPR>) {
        float t = 0.f;
        for (int i = e; i < PER * a.M; i += keep * a.M) t += all[i];
        part[which * plane + e] = t;
      }
    }
  }
}

// dw and db: column c of the [P][C] partial sums, 32 columns a block, 32 rows at a time.
template <typename T>
__global__ void __launch_bounds__(1024) k_norm_join(const float* __restrict__ part, T* __restrict__ dw, T* __restrict__ db, long P, int C) {
  __shared__ float red[32][33];
  grid_dep_enter();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
  T* o = blockIdx.y ? db : dw;
  if (o == nullptr) return;
  const float* p = part + (blockIdx.y ? P * C : 0);
  float v = 0.f;
  if (c < C)
#pragma unroll 8
    for (long i = ty; i < P; i += 32) v += p[i * C + c];
  red[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 32; ++i) v += red[i][tx];
    o[c] = from_f<T>(v);
  }
}

// How a group is held: f.run<V, K, TPR, R>() of the first shape that covers M.
#define LA_NORM_SHAPE(VV, KK, TT, RR) \
  if (M <= (VV) * (KK) * (TT)) return f.template run<VV, KK, TT, RR>();
template <typename T, typename F>
cudaError_t fwd_shape(int M, bool vec, F&& f) {
  constexpr int V = 16 / sizeof(T);
  if (vec) {
    LA_NORM_SHAPE(V, 1, 4, 4)
    LA_NORM_SHAPE(V, 1, 8, 4)
    LA_NORM_SHAPE(V, 1, 16, 4)
    LA_NORM_SHAPE(V, 1, 32, 4)
    LA_NORM_SHAPE(V, 2, 32, 2)
    LA_NORM_SHAPE(V, 4, 32, 1)
    LA_NORM_SHAPE(V, 8, 32, 1)
    LA_NORM_SHAPE(V, 2, 256, 2)
    LA_NORM_SHAPE(V, 4, 256, 1)
    LA_NORM_SHAPE(V, 4, 512, 1)
  } else {
    LA_NORM_SHAPE(1, 1, 8, 4)
    LA_NORM_SHAPE(1, 1, 32, 4)
    LA_NORM_SHAPE(1, 4, 32, 2)
    LA_NORM_SHAPE(1, 4, 256, 2)
    LA_NORM_SHAPE(1, 8, 256, 1)
    LA_NORM_SHAPE(1, 8, 1024, 1)
  }
  return cudaErrorInvalidValue;
}
template <typename T, typename F>
cudaError_t bwd_shape(int M, bool vec, F&& f) {
  constexpr int V = 16 / sizeof(T);
  if (vec) {
    LA_NORM_SHAPE(V, 1, 4, 4)
    LA_NORM_SHAPE(V, 1, 8, 4)
    LA_NORM_SHAPE(V, 1, 16, 4)
    LA_NORM_SHAPE(V, 1, 32, 4)
    LA_NORM_SHAPE(V, 2, 32, 2)
    LA_NORM_SHAPE(V, 1, 128, 4)
    LA_NORM_SHAPE(V, 1, 256, 4)
    LA_NORM_SHAPE(V, 2, 256, 2)
    LA_NORM_SHAPE(V, 2, 512, 1)
    LA_NORM_SHAPE(V, 4, 512, 1)
  } else {
    LA_NORM_SHAPE(1, 1, 8, 4)
    LA_NORM_SHAPE(1, 1, 32, 4)
    LA_NORM_SHAPE(1, 4, 32, 2)
    LA_NORM_SHAPE(1, 4, 256, 2)
    LA_NORM_SHAPE(1, 8, 256, 1)
    LA_NORM_SHAPE(1, 8, 1024, 1)
  }
  return cudaErrorInvalidValue;
}
#undef LA_NORM_SHAPE

template <typename T>
struct Forward {
  const NormArgs& a;
  cudaStream_t st;
  template <int V, int K, int TPR, int R>
  cudaError_t run() {
    constexpr int ITEMS = THREADS<TPR> / TPR * R;
    k_norm_fwd<T, V, K, TPR, R><<<static_cast<unsigned>((a.at.items + ITEMS - 1) / ITEMS), THREADS<TPR>, 0, st>>>(a);
    return cudaGetLastError();
  }
};

// As many blocks as run at once (512 threads on an SM), and a multiple of what keeps
// slots a multiple of G.
long blocks_of(long items, int G, int per, int threads) {
  const long unit = G / std::gcd(G, per);
  const long most = (items + per - 1) / per, want = std::min<long>(most, (long)sm_count() * std::max(1, 512 / threads));
  return (want + unit - 1) / unit * unit;
}

template <typename T>
struct Backward {
  GradArgs& a;
  void *dw, *db;
  cudaStream_t st;
  template <int V, int K, int TPR, int R>
  cudaError_t run() {
    constexpr int NT = THREADS<TPR>, PER = NT / TPR;
    const int G = a.at.groups.d, C = G * a.M;
    const long blocks = blocks_of(a.at.items, G, PER, NT);
    a.slots = blocks * PER;
    k_norm_bwd<T, V, K, TPR, R><<<static_cast<unsigned>(blocks), NT, 0, st>>>(a);
    return launch_pdl(k_norm_join<T>, dim3((C + 31) / 32, 2), dim3(1024), 0, st, (const float*)a.part, (T*)dw, (T*)db,
                      blocks * distinct(PER, G) / G, C);
  }
};

struct Floats {
  long items;
  int G, M;
  size_t n;
  template <int V, int K, int TPR, int R>
  cudaError_t run() {
    constexpr int PER = THREADS<TPR> / TPR;
    n = 2 * static_cast<size_t>(blocks_of(items, G, PER, THREADS<TPR>)) * distinct(PER, G) * M;
    return cudaSuccess;
  }
};

Place place(const int* lengths, const NormShape& s) {
  return Place{Divide(static_cast<uint32_t>(s.G)), Divide(static_cast<uint32_t>(s.N)), lengths, (long)s.B * s.N * s.G};
}

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
  const int M = s.C / s.G;
  Floats a{(long)s.B * s.N * s.G, s.G, M, 0}, b = a;
  if (s.dtype == 0) {
    bwd_shape<float>(M, true, a), bwd_shape<float>(M, false, b);
  } else {
    bwd_shape<bf16>(M, true, a), bwd_shape<bf16>(M, false, b);
  }
  return 4 * std::max(a.n, b.n);
}

cudaError_t norm_fwd(const void* x, const void* res, const void* w, const void* b, const int* lengths, void* y, void* s, float* mean,
                     float* rstd, float eps, const NormShape& sh, cudaStream_t st) {
  const NormArgs a{x, res, w, b, y, s, mean, rstd, place(lengths, sh), sh.ldx, sh.ldr, sh.C / sh.G, eps};
  const bool vec = vectors(sh, sh.ldx, {x, res}) && (res == nullptr || sh.ldr % (sh.dtype == 0 ? 4 : 8) == 0);
  if (sh.dtype == 0) return fwd_shape<float>(a.M, vec, Forward<float>{a, st});
  return fwd_shape<bf16>(a.M, vec, Forward<bf16>{a, st});
}

cudaError_t norm_bwd(const void* s, const void* w, const float* mean, const float* rstd, const int* lengths, const void* dy, const void* ds,
                     void* dx, void* dw, void* db, float* ws, const NormShape& sh, cudaStream_t st) {
  GradArgs a{s, w, dy, ds, mean, rstd, dx, ws, place(lengths, sh), sh.ldx, 0, sh.C / sh.G};
  const bool vec = vectors(sh, sh.ldx, {s});
  if (sh.dtype == 0) return bwd_shape<float>(a.M, vec, Backward<float>{a, dw, db, st});
  return bwd_shape<bf16>(a.M, vec, Backward<bf16>{a, dw, db, st});
}

}  // namespace la
