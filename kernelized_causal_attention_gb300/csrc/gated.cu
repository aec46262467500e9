// Gated recurrence over token-major rows, one decay and one state a channel:
//   s = sigmoid(r), g = sigmoid(i), u = k s with k = scale softplus(lam), a = exp(-u),
//   h_n = a h_{n-1} + beta g x, beta = sqrt(1 - a^2),  y_n = h_n,
// and its gradients, with G_n = dy_n + a_{n+1} G_{n+1}:
//   dx = G beta g,  di = G beta x g (1 - g),  Q = a G (a g x u / beta - u h_{n-1}),
//   dr = (1 - s) Q,  dlam = sigmoid(lam) / softplus(lam) sum Q.
// (u / beta goes to zero with u, so a closed gate has no infinite term.)
//
// The recurrence is associative: a tile of TILE rows turns its first state h into
// A h + H, so a first pass forms every tile's (A, H), a second carries the states over
// the tiles, and a third replays each tile from its state.  A thread owns two channels
// and a strip of rows, whose a and b it keeps in registers between its own pass and the
// replay; a tile's strips are joined through shared memory.
#include <algorithm>

#include "scan.cuh"

namespace la {
namespace {

using bf16 = __nv_bfloat16;

constexpr int STRIP = 8;            // rows of a thread
constexpr int WARPS = 8;            // strips of a tile
constexpr int TILE = STRIP * WARPS;
constexpr int CH = 64;              // channels of a tile, two a lane

// 1 - exp(-u) for u >= 0 to about an ulp, also where u is tiny (a decay close to one is
// one minus it): the series below 1/2 (next term 6e-9), the exponential above.
template <typename T>
__device__ __forceinline__ float one_minus_exp(float u) {
  float p = fmaf(u, -1.f / 40320, 1.f / 5040);
  p = fmaf(u, p, -1.f / 720);
  p = fmaf(u, p, 1.f / 120);
  p = fmaf(u, p, -1.f / 24);
  p = fmaf(u, p, 1.f / 6);
  p = fmaf(u, p, -0.5f);
  p = fmaf(u, p, 1.f);
  float w = u * p;
  if (!(u < 0.5f)) w = 1.f - (sizeof(T) == 4 ? expf(-u) : ex2_fast(-1.4426950408889634f * u));
  return w;
}

// bf16: the hardware's exponential and reciprocal, 2^-22 beside the 2^-9 of the rows.
template <typename T>
__device__ __forceinline__ float sigmoid(float x) {
  return sizeof(T) == 4 ? 1.f / (1.f + expf(-x)) : rcp_fast(1.f + ex2_fast(-1.4426950408889634f * x));
}

__device__ __forceinline__ float rsqrt_fast(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Gate {
  float u, a, beta, ub;  // ub = u / beta
};
template <typename T>
__device__ __forceinline__ Gate gate(float k, float s) {
  Gate q;
  q.u = k * s;
  const float w = one_minus_exp<T>(q.u), om = w * (2.f - w);
  q.a = 1.f - w;
  const float ri = om > 1e-36f ? rsqrt_fast(om) : om == om ? 0.f : om;  // a NaN stays
  q.beta = om * ri;
  q.ub = q.u * ri;
  return q;
}

// Two neighbouring channels of a row, as one vector (PAIR: aligned, both there) or one by one.
template <typename T>
struct Two;
template <>
struct Two<float> {
  float2 v;
};
template <>
struct Two<bf16> {
  uint32_t v;
};
template <bool PAIR>
__device__ __forceinline__ Two<float> load2(const float* p, bool second) {
  if (PAIR) return {*reinterpret_cast<const float2*>(p)};
  return {make_float2(p[0], second ? p[1] : 0.f)};
}
template <bool PAIR>
__device__ __forceinline__ Two<bf16> load2(const bf16* p, bool second) {
  if (PAIR) return {*reinterpret_cast<const uint32_t*>(p)};
  const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
  return {static_cast<uint32_t>(q[0]) | (second ? static_cast<uint32_t>(q[1]) << 16 : 0u)};
}
__device__ __forceinline__ float2 open(const Two<float>& t) { return t.v; }
__device__ __forceinline__ float2 open(const Two<bf16>& t) { return make_float2(__uint_as_float(t.v << 16), __uint_as_float(t.v & 0xffff0000u)); }
template <bool PAIR>
__device__ __forceinline__ void store2(float* p, float2 v, bool second) {
  if (PAIR) {
    *reinterpret_cast<float2*>(p) = v;
  } else {
    p[0] = v.x;
    if (second) p[1] = v.y;
  }
}
template <bool PAIR>
__device__ __forceinline__ void store2(bf16* p, float2 v, bool second) {
  if (PAIR) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
  } else {
    p[0] = __float2bfloat16_rn(v.x);
    if (second) p[1] = __float2bfloat16_rn(v.y);
  }
}

struct Rows {
  const void *x, *r, *i, *lam;
  const int* lengths;
  long ldx, ldr, ldi;
  int N, C, groups, tiles;  // groups of CH channels, tiles of TILE rows
  float scale;
};

// Where a thread works.
struct Place {
  int tile, c, b, t0, L;  // its strip's first row, the sequence's valid rows
  bool first, second;     // which of its channels exist
  __device__ __forceinline__ explicit Place(const Rows& a) {
    tile = blockIdx.x / a.groups;
    c = (blockIdx.x % a.groups) * CH + 2 * (threadIdx.x & 31);
    b = blockIdx.y;
    t0 = tile * TILE + (threadIdx.x >> 5) * STRIP;
    L = valid_rows(a.lengths, b, a.N);
    first = c < a.C;
    second = c + 1 < a.C;
  }
};

template <typename T, bool PAIR>
__device__ __forceinline__ float2 rates(const Rows& a, const Place& p) {
  if (!p.first) return make_float2(0.f, 0.f);
  const float2 l = open(load2<PAIR>(static_cast<const T*>(a.lam) + p.c, p.second));
  return make_float2(a.scale * softplus(l.x), p.second ? a.scale * softplus(l.y) : 0.f);
}

template <typename T, bool PAIR>
__device__ __forceinline__ void fetch(Two<T> (&v)[STRIP], const void* base, long ld, const Rows& a, const Place& p) {
  const T* q = static_cast<const T*>(base) + ((long)p.b * a.N + p.t0) * ld + p.c;
#pragma unroll
  for (int j = 0; j < STRIP; ++j) {
    v[j] = Two<T>{};
    if (p.first && p.t0 + j < p.L) v[j] = load2<PAIR>(q + j * ld, p.second);
  }
}

// (A, H) of the strips of a tile, by strip and lane.
struct Strips {
  float2 A[WARPS][32], H[WARPS][32];
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }

// a and b = beta g x of a strip; rows past the length keep the state.
template <typename T>
__device__ __forceinline__ void decays(float2 (&av)[STRIP], float2 (&bv)[STRIP], const Two<T> (&x)[STRIP], const Two<T> (&r)[STRIP],
                                       const Two<T> (&g)[STRIP], float2 k, const Place& p) {
#pragma unroll
  for (int j = 0; j < STRIP; ++j) {
    av[j] = make_float2(1.f, 1.f), bv[j] = make_float2(0.f, 0.f);
    if (p.t0 + j < p.L) {
      const float2 xf = open(x[j]), rf = open(r[j]), gf = open(g[j]);
      const Gate g0 = gate<T>(k.x, sigmoid<T>(rf.x)), g1 = gate<T>(k.y, sigmoid<T>(rf.y));
      av[j] = make_float2(g0.a, g1.a);
      bv[j] = make_float2(g0.beta * (sigmoid<T>(gf.x) * xf.x), g1.beta * (sigmoid<T>(gf.y) * xf.y));
    }
  }
}

__device__ __forceinline__ long record(const Rows& a, const Place& p) { return ((long)p.b * a.tiles + p.tile) * a.C + p.c; }

// A tile's (A, H) from its rows.
template <typename T, bool PAIR>
__global__ void __launch_bounds__(32 * WARPS) k_gated_sums(const Rows a, float* __restrict__ recA, float* __restrict__ recH) {
  __shared__ Strips st;
  const Place p(a);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  Two<T> x[STRIP], r[STRIP], g[STRIP];
  fetch<T, PAIR>(r, a.r, a.ldr, a, p);
  fetch<T, PAIR>(g, a.i, a.ldi, a, p);
  fetch<T, PAIR>(x, a.x, a.ldx, a, p);
  float2 av[STRIP], bv[STRIP];
  decays<T>(av, bv, x, r, g, rates<T, PAIR>(a, p), p);
  float2 A = make_float2(1.f, 1.f), H = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < STRIP; ++j) {
    H = fma2(av[j], H, bv[j]);
    A = make_float2(A.x * av[j].x, A.y * av[j].y);
  }
  st.A[w][lane] = A, st.H[w][lane] = H;
  __syncthreads();
  if (w == 0 && p.first) {
#pragma unroll
    for (int i = 1; i < WARPS; ++i) {
      const float2 Ai = st.A[i][lane];
      H = fma2(Ai, H, st.H[i][lane]);
      A = make_float2(A.x * Ai.x, A.y * Ai.y);
    }
    const long at = record(a, p);
    recA[at] = A.x, recH[at] = H.x;
    if (p.second) recA[at + 1] = A.y, recH[at + 1] = H.y;
  }
}

// The states before each tile, into keep; h, if given, starts the recurrence and
// becomes the last state.
__global__ void __launch_bounds__(128) k_gated_carry(const float* __restrict__ recA, const float* __restrict__ recH, float* __restrict__ keep,
                                                     float* __restrict__ h, int C, int tiles, int reverse) {
  grid_dep_enter();
  const int c = blockIdx.x * 128 + threadIdx.x;
  if (c >= C) return;
  const long at = (long)blockIdx.y * tiles * C + c;
  float s = h == nullptr ? 0.f : h[(long)blockIdx.y * C + c];
#pragma unroll 8
  for (int t = 0; t < tiles; ++t) {
    const long e = at + (long)(reverse ? tiles - 1 - t : t) * C;
    keep[e] = s;
    s = fmaf(recA[e], s, recH[e]);
  }
  if (h != nullptr) h[(long)blockIdx.y * C + c] = s;
}

// y from the state before the tile: keep's, or, where the sequence is one tile, the
// caller's h (zero if null), which then becomes the last state; kept takes it.
template <typename T, bool PAIR>
__global__ void __launch_bounds__(32 * WARPS) k_gated_out(const Rows a, const float* __restrict__ keep, float* h, float* __restrict__ kept, T* __restrict__ y) {
  __shared__ Strips st;
  const Place p(a);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  Two<T> x[STRIP], r[STRIP], g[STRIP];
  if (keep != nullptr) grid_dep_enter();
  fetch<T, PAIR>(r, a.r, a.ldr, a, p);
  fetch<T, PAIR>(g, a.i, a.ldi, a, p);
  fetch<T, PAIR>(x, a.x, a.ldx, a, p);
  float2 av[STRIP], bv[STRIP];
  decays<T>(av, bv, x, r, g, rates<T, PAIR>(a, p), p);
  float2 A = make_float2(1.f, 1.f), H = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < STRIP; ++j) {
    H = fma2(av[j], H, bv[j]);
    A = make_float2(A.x * av[j].x, A.y * av[j].y);
  }
  st.A[w][lane] = A, st.H[w][lane] = H;
  float2 s = make_float2(0.f, 0.f);
  if (p.first && (keep != nullptr || h != nullptr)) {
    const float* from = keep != nullptr ? keep + record(a, p) : h + (long)p.b * a.C + p.c;
    s.x = from[0];
    if (p.second) s.y = from[1];
  }
  if (kept != nullptr && w == 0 && p.first) {
    float* to = kept + record(a, p);
    to[0] = s.x;
    if (p.second) to[1] = s.y;
  }
  __syncthreads();
  for (int i = 0; i < w; ++i) s = fma2(st.A[i][lane], s, st.H[i][lane]);
  T* o = y + ((long)p.b * a.N + p.t0) * a.C + p.c;
#pragma unroll
  for (int j = 0; j < STRIP; ++j) {
    s = fma2(av[j], s, bv[j]);
    if (p.first && p.t0 + j < a.N) store2<PAIR>(o + (long)j * a.C, p.t0 + j < p.L ? s : make_float2(0.f, 0.f), p.second);
  }
  if (keep == nullptr && h != nullptr && w == WARPS - 1 && p.first) {  // h's readers are this block, before its barrier
    float* to = h + (long)p.b * a.C + p.c;
    to[0] = s.x;
    if (p.second) to[1] = s.y;
  }
}

// The gradient's tile: from X, what arrives at its last row, to P X + Y, what leaves its
// first one (X_n = a_n (dy_n + X_{n+1})).
template <typename T, bool PAIR>
__global__ void __launch_bounds__(32 * WARPS) k_gated_back(const Rows a, const T* __restrict__ dy, float* __restrict__ recP, float* __restrict__ recY) {
  __shared__ Strips st;
  const Place p(a);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  Two<T> r[STRIP], d[STRIP];
  fetch<T, PAIR>(r, a.r, a.ldr, a, p);
  fetch<T, PAIR>(d, dy, a.C, a, p);
  const float2 k = rates<T, PAIR>(a, p);
  float2 P = make_float2(1.f, 1.f), Y = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = STRIP - 1; j >= 0; --j)
    if (p.t0 + j < p.L) {
      const float2 rf = open(r[j]), df = open(d[j]);
      const float2 av = make_float2(gate<T>(k.x, sigmoid<T>(rf.x)).a, gate<T>(k.y, sigmoid<T>(rf.y)).a);
      Y = make_float2(av.x * (df.x + Y.x), av.y * (df.y + Y.y));
      P = make_float2(P.x * av.x, P.y * av.y);
    }
  st.A[w][lane] = P, st.H[w][lane] = Y;
  __syncthreads();
  if (w == WARPS - 1 && p.first) {
#pragma unroll
    for (int i = WARPS - 2; i >= 0; --i) {
      const float2 Pi = st.A[i][lane];
      Y = fma2(Pi, Y, st.H[i][lane]);
      P = make_float2(P.x * Pi.x, P.y * Pi.y);
    }
    const long at = record(a, p);
    recP[at] = P.x, recY[at] = Y.x;
    if (p.second) recP[at + 1] = P.y, recY[at + 1] = Y.y;
  }
}

// All gradients of a tile, from the state before it (keep) and the gradient that
// arrives at its last row (arrive; null: zero), and its sums of Q.
template <typename T, bool PAIR>
__global__ void __launch_bounds__(32 * WARPS) k_gated_grad(const Rows a, const T* __restrict__ dy, const float* __restrict__ keep,
                                                           const float* __restrict__ arrive, T* __restrict__ dx, T* __restrict__ dr,
                                                           T* __restrict__ di, float* __restrict__ sums) {
  __shared__ Strips f, v;
  const Place p(a);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (arrive != nullptr) grid_dep_enter();
  Two<T> x[STRIP], r[STRIP], g[STRIP], d[STRIP];
  fetch<T, PAIR>(r, a.r, a.ldr, a, p);
  fetch<T, PAIR>(g, a.i, a.ldi, a, p);
  fetch<T, PAIR>(x, a.x, a.ldx, a, p);
  fetch<T, PAIR>(d, dy, a.C, a, p);
  const float2 k = rates<T, PAIR>(a, p);
  float2 av[STRIP], bv[STRIP];
  decays<T>(av, bv, x, r, g, k, p);
  float2 A = make_float2(1.f, 1.f), H = make_float2(0.f, 0.f), Y = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < STRIP; ++j) {
    H = fma2(av[j], H, bv[j]);
    A = make_float2(A.x * av[j].x, A.y * av[j].y);
  }
#pragma unroll
  for (int j = STRIP - 1; j >= 0; --j) {
    const float2 df = open(d[j]);
    Y = make_float2(av[j].x * (df.x + Y.x), av[j].y * (df.y + Y.y));
  }
  f.A[w][lane] = A, f.H[w][lane] = H;
  v.H[w][lane] = Y;
  const long at = record(a, p);
  float2 s = make_float2(0.f, 0.f), X = s;
  if (p.first) {
    s.x = keep[at];
    if (arrive != nullptr) X.x = arrive[at];
    if (p.second) {
      s.y = keep[at + 1];
      if (arrive != nullptr) X.y = arrive[at + 1];
    }
  }
  __syncthreads();
  for (int i = 0; i < w; ++i) s = fma2(f.A[i][lane], s, f.H[i][lane]);
  for (int i = WARPS - 1; i > w; --i) X = fma2(f.A[i][lane], X, v.H[i][lane]);
  float2 before[STRIP];
#pragma unroll
  for (int j = 0; j < STRIP; ++j) {
    before[j] = s;
    s = fma2(av[j], s, bv[j]);
  }
  float2 sum = make_float2(0.f, 0.f);
  const long row = ((long)p.b * a.N + p.t0) * a.C + p.c;
#pragma unroll
  for (int j = STRIP - 1; j >= 0; --j) {
    float2 ox = make_float2(0.f, 0.f), orr = ox, oi = ox;
    if (p.t0 + j < p.L) {
      const float2 xf = open(x[j]), rf = open(r[j]), gf = open(g[j]), df = open(d[j]);
      auto one = [](float xv, float rv, float gv, float dv, float kk, float hb, float& X1, float& acc, float& o0, float& o1, float& o2) {
        const float s1 = sigmoid<T>(rv), g1 = sigmoid<T>(gv);
        const Gate q = gate<T>(kk, s1);
        const float G = dv + X1, gx = g1 * xv, aG = q.a * G;
        const float Q = aG * (q.a * gx * q.ub - q.u * hb);
        X1 = aG;
        acc += Q;
        o0 = G * q.beta * g1;
        o1 = Q * (1.f - s1);
        o2 = G * q.beta * gx * (1.f - g1);
      };
      one(xf.x, rf.x, gf.x, df.x, k.x, before[j].x, X.x, sum.x, ox.x, orr.x, oi.x);
      one(xf.y, rf.y, gf.y, df.y, k.y, before[j].y, X.y, sum.y, ox.y, orr.y, oi.y);
    }
    if (p.first && p.t0 + j < a.N) {
      store2<PAIR>(dx + row + (long)j * a.C, ox, p.second);
      store2<PAIR>(dr + row + (long)j * a.C, orr, p.second);
      store2<PAIR>(di + row + (long)j * a.C, oi, p.second);
    }
  }
  __syncthreads();  // v is read
  v.A[w][lane] = sum;
  __syncthreads();
  if (w == 0 && p.first) {
#pragma unroll
    for (int i = 1; i < WARPS; ++i) {
      const float2 o = v.A[i][lane];
      sum.x += o.x, sum.y += o.y;
    }
    sums[at] = sum.x;
    if (p.second) sums[at + 1] = sum.y;
  }
}

// dlam from the [n][C] sums of Q, 32 channels a block, eight rows at a time.
template <typename T>
__global__ void __launch_bounds__(256) k_gated_lam(const float* __restrict__ sums, const T* __restrict__ lam, T* __restrict__ dlam, long n, int C) {
  __shared__ float red[8][33];
  grid_dep_enter();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
  float v = 0.f;
  if (c < C)
    for (long i = ty; i < n; i += 8) v += sums[i * C + c];
  red[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += red[i][tx];
    // sigmoid / softplus, which goes to one on the left: below -20 both are exp(lam) to fp32
    const float l = to_f(lam[c]), ratio = l < -20.f ? 1.f : 1.f / ((1.f + expf(-l)) * softplus(l));
    dlam[c] = from_f<T>(v * ratio);
  }
}

// One row a stream: h <- a h + beta g x, y = h.
template <typename T, bool PAIR>
__global__ void __launch_bounds__(256) k_gated_step(const Rows a, float* __restrict__ h, T* __restrict__ y) {
  const long b = blockIdx.x / a.groups;  // groups of 512 channels here
  const int c = 2 * ((blockIdx.x % a.groups) * 256 + threadIdx.x);
  if (c >= a.C) return;
  const bool second = c + 1 < a.C;
  const float2 x = open(load2<PAIR>(static_cast<const T*>(a.x) + b * a.ldx + c, second));
  const float2 r = open(load2<PAIR>(static_cast<const T*>(a.r) + b * a.ldr + c, second));
  const float2 g = open(load2<PAIR>(static_cast<const T*>(a.i) + b * a.ldi + c, second));
  const float2 l = open(load2<PAIR>(static_cast<const T*>(a.lam) + c, second));
  float2 s = open(load2<PAIR>(h + b * a.C + c, second));
  const Gate g0 = gate<T>(a.scale * softplus(l.x), sigmoid<T>(r.x)), g1 = gate<T>(a.scale * softplus(l.y), sigmoid<T>(r.y));
  s = make_float2(fmaf(g0.a, s.x, g0.beta * (sigmoid<T>(g.x) * x.x)), fmaf(g1.a, s.y, g1.beta * (sigmoid<T>(g.y) * x.y)));
  store2<PAIR>(h + b * a.C + c, s, second);
  store2<PAIR>(y + b * a.C + c, s, second);
}

Rows rows(const void* x, const void* r, const void* i, const void* lam, const int* lengths, const GatedShape& s) {
  return Rows{x, r, i, lam, lengths, s.ldx, s.ldr, s.ldi, s.N, s.C, (s.C + CH - 1) / CH, (s.N + TILE - 1) / TILE, s.scale};
}

// Pairs of channels as vectors: even widths and strides, aligned rows.
bool pairs(const Rows& a, int dtype) {
  const uintptr_t low = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.r) | reinterpret_cast<uintptr_t>(a.i);
  return ((a.ldx | a.ldr | a.ldi | a.C) & 1) == 0 && low % (dtype == 0 ? 8 : 4) == 0;
}

size_t records(const GatedShape& s) { return (size_t)s.B * ((s.N + TILE - 1) / TILE) * s.C; }

template <typename T, bool PAIR>
cudaError_t fwd(const Rows& a, float* h, float* keep, void* y, float* ws, const GatedShape& s, cudaStream_t st) {
  const dim3 grid(a.tiles * a.groups, s.B), block(32 * WARPS);
  if (a.tiles == 1) {
    k_gated_out<T, PAIR><<<grid, block, 0, st>>>(a, nullptr, h, keep, (T*)y);
    return cudaGetLastError();
  }
  float *recA = ws, *recH = ws + records(s), *to = keep != nullptr ? keep : ws + 2 * records(s);
  k_gated_sums<T, PAIR><<<grid, block, 0, st>>>(a, recA, recH);
  cudaError_t e = launch_pdl(k_gated_carry, dim3((s.C + 127) / 128, s.B), dim3(128), 0, st, (const float*)recA, (const float*)recH, to, h,
                                  s.C, a.tiles, 0);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_gated_out<T, PAIR>, grid, block, 0, st, a, (const float*)to, h, (float*)nullptr, (T*)y);
}

template <typename T, bool PAIR>
cudaError_t bwd(const Rows& a, const float* keep, const void* dy, void* dx, void* dr, void* di, void* dlam, float* ws, const GatedShape& s,
                cudaStream_t st) {
  const dim3 grid(a.tiles * a.groups, s.B), block(32 * WARPS);
  float *sums = ws, *recP = ws + records(s), *recY = recP + records(s), *arrive = recY + records(s);
  if (a.tiles == 1) {
    k_gated_grad<T, PAIR><<<grid, block, 0, st>>>(a, (const T*)dy, keep, nullptr, (T*)dx, (T*)dr, (T*)di, sums);
  } else {
    k_gated_back<T, PAIR><<<grid, block, 0, st>>>(a, (const T*)dy, recP, recY);
    cudaError_t e = launch_pdl(k_gated_carry, dim3((s.C + 127) / 128, s.B), dim3(128), 0, st, (const float*)recP, (const float*)recY, arrive,
                                    (float*)nullptr, s.C, a.tiles, 1);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_gated_grad<T, PAIR>, grid, block, 0, st, a, (const T*)dy, keep, (const float*)arrive, (T*)dx, (T*)dr, (T*)di, sums);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k_gated_lam<T>, dim3((s.C + 31) / 32), dim3(256), 0, st, (const float*)sums, (const T*)a.lam, (T*)dlam,
                         (long)s.B * a.tiles, s.C);
}

template <typename T, bool PAIR>
cudaError_t step(const Rows& a, float* h, void* y, const GatedShape& s, cudaStream_t st) {
  Rows wide = a;
  wide.groups = (s.C + 511) / 512;
  k_gated_step<T, PAIR><<<wide.groups * s.B, 256, 0, st>>>(wide, h, (T*)y);
  return cudaGetLastError();
}

}  // namespace

size_t gated_kept_bytes(const GatedShape& s) { return 4 * records(s); }
size_t gated_ws_bytes(const GatedShape& s, bool bwd) {
  if (bwd) return 4 * records(s) * (s.N > TILE ? 4 : 1);
  return s.N > TILE ? 12 * records(s) : 0;
}

#define LA_GATED(f, ...)                                                        \
  (s.dtype == 0 ? pairs(a, 0) ? f<float, true>(__VA_ARGS__) : f<float, false>(__VA_ARGS__) \
                : pairs(a, 1) ? f<bf16, true>(__VA_ARGS__) : f<bf16, false>(__VA_ARGS__))

cudaError_t gated_fwd(const void* x, const void* r, const void* i, const void* lam, const int* lengths, float* h, float* kept, void* y,
                      float* ws, const GatedShape& s, cudaStream_t st) {
  const Rows a = rows(x, r, i, lam, lengths, s);
  return LA_GATED(fwd, a, h, kept, y, ws, s, st);
}
cudaError_t gated_bwd(const void* x, const void* r, const void* i, const void* lam, const int* lengths, const float* kept, const void* dy,
                      void* dx, void* dr, void* di, void* dlam, float* ws, const GatedShape& s, cudaStream_t st) {
  const Rows a = rows(x, r, i, lam, lengths, s);
  return LA_GATED(bwd, a, kept, dy, dx, dr, di, dlam, ws, s, st);
}
cudaError_t gated_step(const void* x, const void* r, const void* i, const void* lam, float* h, void* y, const GatedShape& s, cudaStream_t st) {
  const Rows a = rows(x, r, i, lam, nullptr, s);
  return LA_GATED(step, a, h, y, s, st);
}
#undef LA_GATED

}  // namespace la
