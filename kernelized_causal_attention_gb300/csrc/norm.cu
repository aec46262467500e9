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
// blocks' sums up in a fixed order.  4 x 2048 x 2048 bf16 behind a residual sum: forward
// 20 us (134 MB, the copy rate), gradients 28 with cold caches (134 MB, 0.71) and 3 for the
// join; 32 groups of 64: 13.8 (67 MB, 0.72) and 20 (101 MB, 0.74): issue at 69 and 57 %,
// with 22 to 44 % of the warps for the registers that hold the groups.
#include <algorithm>
#include <numeric>

#include "pair.cuh"
#include "scan.cuh"

namespace la {
namespace {

using bf16 = __nv_bfloat16;

// V neighbouring values as one vector of up to 16 bytes (V > 1: the caller has
// checked the alignment), as it lies in memory and as pairs of fp32 (V = 1: with zero).
template <typename T, int V>
struct Vec;
template <typename T>
struct Vec<T, 1> {
  using Raw = T;
  __device__ __forceinline__ static void open(const Raw& u, u64* f) { f[0] = pk(to_f(u), 0.f); }
  __device__ __forceinline__ static Raw close(const u64* f) { return from_f<T>(un(f[0]).x); }
};
template <>
struct Vec<float, 4> {
  using Raw = float4;
  __device__ __forceinline__ static void open(const Raw& u, u64* f) { f[0] = pk(u.x, u.y), f[1] = pk(u.z, u.w); }
  __device__ __forceinline__ static Raw close(const u64* f) {
    const float2 a = un(f[0]), b = un(f[1]);
    return make_float4(a.x, a.y, b.x, b.y);
  }
};
template <>
struct Vec<bf16, 8> {
  using Raw = uint4;
  __device__ __forceinline__ static void open(const Raw& u, u64* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ static Raw close(const u64* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = un(f[i]);
      const __nv_bfloat162 h = __floats2bfloat162_rn(a.x, a.y);
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

// A vector (V = 1: a value) into a thread's own place in shared memory, zero without `some`:
// an asynchronous copy of 16 or 4 bytes, or a load and a store.
template <typename Raw, typename T>
__device__ __forceinline__ void fetch(Raw& to, const T* from, bool some) {
  if constexpr (sizeof(Raw) == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(&to)), "l"(from), "r"(some ? 16 : 0) : "memory");
  else if constexpr (sizeof(Raw) == 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(&to)), "l"(from), "r"(some ? 4 : 0) : "memory");
  else
    to = some ? *from : Raw{};
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
  long ldx, ldr, slots;  // ldx, ldr: elements between rows
  int M;
  float inv, eps;  // inv: 1 / M
};

// Slot (block, group of threads) takes R items slot, slot + slots, ...; slots is a
// multiple of G, so a thread's columns and their weights stay the same.  Its k-th vector
// of columns is at (k TPR + lane) V.
template <typename T, int V, int K, int TPR, int R>
__global__ void __launch_bounds__(THREADS<TPR>) k_norm_fwd(const NormArgs a) {
  grid_dep_enter();
  using Raw = typename Vec<T, V>::Raw;
  constexpr int PER = THREADS<TPR> / TPR, P = (V + 1) / 2;
  __shared__ float red[2][R][TPR > 32 ? TPR / 32 : 1];
  Sums<TPR, R> sum{red};
  const int lane = threadIdx.x % TPR;
  const long slot = (long)blockIdx.x * PER + threadIdx.x / TPR;
  bool in[R], live[R];  // every thread stays for the sums
  uint32_t g = 0;
  Raw x[R][K], res[R][K];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    uint32_t row, gr;
    a.at.of(slot + r * a.slots, in[r], live[r], row, gr);
    if (r == 0) g = gr;
    const T* p = static_cast<const T*>(a.x) + row * a.ldx + gr * a.M;
    const T* q = static_cast<const T*>(a.res) + row * a.ldr + gr * a.M;
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
  u64 f[R][K][P];
  float v[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    u64 t = 0ull;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * TPR + lane) * V;
      Vec<T, V>::open(x[r][k], f[r][k]);
      if (a.res != nullptr) {
        u64 e[P];
        Vec<T, V>::open(res[r][k], e);
#pragma unroll
        for (int i = 0; i < P; ++i) f[r][k][i] = add2(f[r][k][i], e[i]);
        const Raw total = Vec<T, V>::close(f[r][k]);
        Vec<T, V>::open(total, f[r][k]);
        if (in[r] && c < a.M) set<T, V>(static_cast<T*>(a.s) + (slot + r * a.slots) * a.M + c, total);
      }
#pragma unroll
      for (int i = 0; i < P; ++i) t = add2(t, f[r][k][i]);
    }
    const float2 tf = un(t);
    v[r] = tf.x + tf.y;
  }
  sum(v);
  float mean[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    mean[r] = v[r] * a.inv;
    const u64 off = pk(-mean[r], V == 1 ? 0.f : -mean[r]);
    u64 t = 0ull;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if ((k * TPR + lane) * V < a.M) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          f[r][k][i] = add2(f[r][k][i], off);
          t = fma2(f[r][k][i], f[r][k][i], t);
        }
      }
    const float2 tf = un(t);
    v[r] = tf.x + tf.y;
  }
  sum(v);
#pragma unroll
  for (int r = 0; r < R; ++r) v[r] = rsqrtf(fmaf(v[r], a.inv, a.eps));
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * TPR + lane) * V;
    if (c >= a.M) continue;
    u64 w[P], b[P];
    Vec<T, V>::open(get<T, V>(static_cast<const T*>(a.w) + g * a.M + c), w);
#pragma unroll
    for (int i = 0; i < P; ++i) b[i] = 0ull;
    if (a.b != nullptr) Vec<T, V>::open(get<T, V>(static_cast<const T*>(a.b) + g * a.M + c), b);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!in[r]) continue;
      u64 o[P];
      const u64 scale = two(v[r]);
#pragma unroll
      for (int i = 0; i < P; ++i) o[i] = live[r] ? fma2(mul2(f[r][k][i], scale), w[i], b[i]) : 0ull;
      set<T, V>(static_cast<T*>(a.y) + (slot + r * a.slots) * a.M + c, Vec<T, V>::close(o));
    }
  }
  if (lane == 0 && a.mean != nullptr) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (in[r]) {
        a.mean[slot + r * a.slots] = live[r] ? mean[r] : 0.f;
        a.rstd[slot + r * a.slots] = live[r] ? v[r] : 0.f;
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
  float inv;  // 1 / M
};

// How many groups' sums of its own a block leaves: those of its slots, or, where G
// divides them, of the G groups, added up over the slots that share one.
inline __host__ __device__ int distinct(int per, int G) { return per % G == 0 ? G : per; }

// Items as forward, R at a time until there are no more.  The next ones are on their way
// into shared memory (a thread's own places, so it waits for its own copies only) while R
// are worked on, and are read from there twice: 48.3 us both ways for 4 x 2048 x 2048 bf16
// with a residual, 54.5 with registers for them and loads that wait, 34.9 and 38.3 for 32
// groups of 64.  Two items at once 50.1 and 37.1; four spill (of three, the form of 128 threads
// does: 4 bytes).
template <typename T, int V, int K, int TPR, int R>
__global__ void __launch_bounds__(THREADS<TPR>, (THREADS<TPR> < 512 ? 512 / THREADS<TPR> : 1)) k_norm_bwd(const GradArgs a) {
  grid_dep_enter();
  using Raw = typename Vec<T, V>::Raw;
  constexpr int PER = THREADS<TPR> / TPR, P = (V + 1) / 2;
  __shared__ float red[2][2 * R][TPR > 32 ? TPR / 32 : 1];
  Sums<TPR, 2 * R> sum{red};
  const int lane = threadIdx.x % TPR;
  const long slot = (long)blockIdx.x * PER + threadIdx.x / TPR;
  const uint32_t own = static_cast<uint32_t>(slot) % a.at.groups.d;
  const T* w = static_cast<const T*>(a.w) + own * a.M;
  u64 dw[K][P], db[K][P], wv[K][P];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * TPR + lane) * V;
    Raw wr = Raw{};
    if (c < a.M) wr = get<T, V>(w + c);
    Vec<T, V>::open(wr, wv[k]);
#pragma unroll
    for (int i = 0; i < P; ++i) dw[k][i] = db[k][i] = 0ull;
  }
  extern __shared__ __align__(16) unsigned char room[];
  auto own_slot = [&](int stage, int t, int r, int k) -> Raw& {
    return reinterpret_cast<Raw*>(room)[(((stage * 3 + t) * R + r) * K + k) * THREADS<TPR> + threadIdx.x];
  };
  bool in[R];
  float mean[R], rstd[R];
  auto request = [&](long base, int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      bool live;
      uint32_t row, g;
      a.at.of(base + r * a.slots, in[r], live, row, g);
      const long item = in[r] ? base + r * a.slots : 0;
      const T *p[3] = {static_cast<const T*>(a.s) + row * a.lds + own * a.M, static_cast<const T*>(a.dy) + item * a.M,
                       static_cast<const T*>(a.ds) + item * a.M};
      mean[r] = live ? a.mean[item] : 0.f, rstd[r] = live ? a.rstd[item] : 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * TPR + lane) * V;
        const bool some = live && c < a.M;
#pragma unroll
        for (int t = 0; t < 3; ++t)
          if (t < 2 || a.ds != nullptr) fetch(own_slot(stage, t, r, k), some ? p[t] + c : p[t], some);
      }
    }
  };
  request(slot, 0);
  asm volatile("cp.async.commit_group;" ::: "memory");
  int stage = 0;
  for (long base = slot; base - slot < a.at.items; base += R * a.slots, stage ^= 1) {  // the same steps for all threads: they meet in the sums
    bool now[R];
    float off_[R], scale_[R];
#pragma unroll
    for (int r = 0; r < R; ++r) now[r] = in[r], off_[r] = -mean[r], scale_[r] = rstd[r];
    if (base + R * a.slots - slot < a.at.items) request(base + R * a.slots, stage ^ 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // all but the group just made
    // rows that are not live hold zeros, and rstd zero: they add nothing, and dx is zero
    float v[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      u64 t1 = 0ull, t2 = 0ull;
      const u64 off = two(off_[r]), scale = two(scale_[r]);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        u64 f[P], d[P];
        Vec<T, V>::open(own_slot(stage, 0, r, k), f);
        Vec<T, V>::open(own_slot(stage, 1, r, k), d);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          f[i] = mul2(add2(f[i], off), scale);
          dw[k][i] = fma2(d[i], f[i], dw[k][i]);
          db[k][i] = add2(db[k][i], d[i]);
          d[i] = mul2(d[i], wv[k][i]);
          t1 = add2(t1, d[i]);
          t2 = fma2(d[i], f[i], t2);
        }
      }
      const float2 a1 = un(t1), a2 = un(t2);
      v[2 * r] = a1.x + a1.y, v[2 * r + 1] = a2.x + a2.y;
    }
    sum(v);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!now[r]) continue;
      const u64 s1 = two(-v[2 * r] * a.inv), s2 = two(-v[2 * r + 1] * a.inv), off = two(off_[r]), scale = two(scale_[r]);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * TPR + lane) * V;
        if (c >= a.M) continue;
        u64 f[P], d[P], e[P];
        Vec<T, V>::open(own_slot(stage, 0, r, k), f);
        Vec<T, V>::open(own_slot(stage, 1, r, k), d);
        if (a.ds != nullptr) {
          Vec<T, V>::open(own_slot(stage, 2, r, k), e);
        } else {
#pragma unroll
          for (int i = 0; i < P; ++i) e[i] = 0ull;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
          f[i] = mul2(add2(f[i], off), scale);
          d[i] = fma2(f[i], s2, fma2(d[i], wv[k][i], s1));
          d[i] = fma2(d[i], scale, e[i]);
        }
        set<T, V>(static_cast<T*>(a.dx) + (base + r * a.slots) * a.M + c, Vec<T, V>::close(d));
      }
    }
  }
  // the sums: [block][distinct groups][M], which is [..][C]
  const int G = a.at.groups.d, keep = distinct(PER, G);
  float* part = a.part + (long)blockIdx.x * keep * a.M;
  const long plane = (long)gridDim.x * keep * a.M;
  auto spread = [&](float* to, const u64* from) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 t = un(from[i]);
      to[2 * i] = t.x;
      if (V > 1) to[2 * i + 1] = t.y;
    }
  };
  if constexpr (PER == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * TPR + lane) * V;
      if (c < a.M) spread(part + c, dw[k]), spread(part + plane + c, db[k]);
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
        if (c < a.M) spread(all + mine * a.M + c, which ? db[k] : dw[k]);
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
__global__ void __launch_bounds__(1024) k_norm_join(const float* part, T* dw, T* db, long P, int C) {
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

// How a group is held: f.run<V, K, TPR, R>() of the first shape that covers M.  Forward,
// both directions of 4 x 2048 x 2048 bf16 with a residual took 3 us more with one vector a
// thread than with two; 32 groups of 64 took 3 to 5 us more with two or four at once than
// with three.
#define LA_NORM_SHAPE(VV, KK, TT, RR) \
  if (M <= (VV) * (KK) * (TT)) return f.template run<VV, KK, TT, RR>();
template <typename T, typename F>
cudaError_t fwd_shape(int M, bool vec, F&& f) {
  constexpr int V = 16 / sizeof(T);
  if (vec) {
    LA_NORM_SHAPE(V, 1, 4, 3)
    LA_NORM_SHAPE(V, 1, 8, 3)
    LA_NORM_SHAPE(V, 1, 16, 3)
    LA_NORM_SHAPE(V, 1, 32, 3)
    LA_NORM_SHAPE(V, 2, 32, 2)
    LA_NORM_SHAPE(V, 4, 32, 1)
    LA_NORM_SHAPE(V, 2, 128, 2)
    LA_NORM_SHAPE(V, 2, 256, 2)
    LA_NORM_SHAPE(V, 4, 256, 1)
    if constexpr (V == 4) LA_NORM_SHAPE(V, 4, 512, 1)
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
    LA_NORM_SHAPE(V, 1, 4, 3)
    LA_NORM_SHAPE(V, 1, 8, 3)
    LA_NORM_SHAPE(V, 1, 16, 3)
    LA_NORM_SHAPE(V, 1, 32, 3)
    LA_NORM_SHAPE(V, 1, 64, 3)
    LA_NORM_SHAPE(V, 1, 128, 3)
    LA_NORM_SHAPE(V, 1, 256, 3)
    LA_NORM_SHAPE(V, 2, 256, 2)
    LA_NORM_SHAPE(V, 2, 512, 1)
    if constexpr (V == 4) LA_NORM_SHAPE(V, 4, 512, 1)
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

// At least `want` blocks, and a multiple of what keeps slots a multiple of G.
long in_units(long want, int G, int per) {
  const long unit = G / std::gcd(G, per);
  return (want + unit - 1) / unit * unit;
}

template <typename T>
struct Forward {
  NormArgs& a;
  cudaStream_t st;
  template <int V, int K, int TPR, int R>
  cudaError_t run() {
    constexpr int PER = THREADS<TPR> / TPR;
    const long blocks = in_units((a.at.items + R * PER - 1) / (R * PER), a.at.groups.d, PER);
    a.slots = blocks * PER;
    return launch_pdl(k_norm_fwd<T, V, K, TPR, R>, dim3(static_cast<unsigned>(blocks)), dim3(THREADS<TPR>), 0, st, a);
  }
};

// As many blocks as run at once: 512 threads on an SM.
long blocks_of(long items, int G, int per, int threads) {
  return in_units(std::min<long>((items + per - 1) / per, (long)sm_count() * std::max(1, 512 / threads)), G, per);
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
    constexpr int room = 2 * 3 * R * K * NT * V * static_cast<int>(sizeof(T));
    cudaError_t e = cudaFuncSetAttribute(k_norm_bwd<T, V, K, TPR, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, room);
    if (e != cudaSuccess) return e;
    if ((e = launch_pdl(k_norm_bwd<T, V, K, TPR, R>, dim3(static_cast<unsigned>(blocks)), dim3(NT), room, st, a)) != cudaSuccess) return e;
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
  const int M = sh.C / sh.G;
  NormArgs a{x, res, w, b, y, s, mean, rstd, place(lengths, sh), sh.ldx, sh.ldr, 0, M, 1.f / M, eps};
  const bool vec = vectors(sh, sh.ldx, {x, res}) && (res == nullptr || sh.ldr % (sh.dtype == 0 ? 4 : 8) == 0);
  if (sh.dtype == 0) return fwd_shape<float>(a.M, vec, Forward<float>{a, st});
  return fwd_shape<bf16>(a.M, vec, Forward<bf16>{a, st});
}

cudaError_t norm_bwd(const void* s, const void* w, const float* mean, const float* rstd, const int* lengths, const void* dy, const void* ds,
                     void* dx, void* dw, void* db, float* ws, const NormShape& sh, cudaStream_t st) {
  const int M = sh.C / sh.G;
  GradArgs a{s, w, dy, ds, mean, rstd, dx, ws, place(lengths, sh), sh.ldx, 0, M, 1.f / M};
  const bool vec = vectors(sh, sh.ldx, {s});
  if (sh.dtype == 0) return bwd_shape<float>(a.M, vec, Backward<float>{a, dw, db, st});
  return bwd_shape<bf16>(a.M, vec, Backward<bf16>{a, dw, db, st});
}

}  // namespace la
