// Rotary positions: pair j of a row at position p is turned by the angle p f_j,
//   (a, b) -> gain (a cos - b sin, b cos + a sin),
// where the pairs are (x[j], x[j + R/2]) or, interleaved, (x[2j], x[2j + 1]), and the
// columns from R on pass unchanged.  The gradient is the turn by the negative angle.
//
// Frequencies are whole numbers of 2^-64 turns a position, so that the product with
// the position, modulo 2^64, is the angle without its whole turns, exactly, at any
// position; its upper 32 bits go into the sine (2^-32 turns are 1.5e-9 radians).
//
// Bound by HBM: every value is read and written once.  Sine and cosine cost about 25
// instructions a row and pair; a thread forms those of its four pairs once and takes
// its row's heads, of queries and keys alike, in turn.
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace la {
namespace {

using bf16 = __nv_bfloat16;

// Sine and cosine of ph 2^-32 turns.  The nearest quarter turn is taken off in whole
// numbers; what is left, at most pi / 4, goes into the Taylor series (terms to t^9 and
// t^10: the next ones are below 2e-9).
__device__ __forceinline__ void sincos_turn(uint32_t ph, float& sn, float& cs) {
  const uint32_t quarter = (ph + (1u << 29)) >> 30;
  const float t = static_cast<float>(static_cast<int>(ph - (quarter << 30))) * 1.46291807927e-9f;  // 2 pi / 2^32
  const float z = t * t;
  float s = fmaf(z, 1.f / 362880, -1.f / 5040);
  s = fmaf(z, s, 1.f / 120);
  s = fmaf(z, s, -1.f / 6);
  s = fmaf(z * s, t, t);
  float c = fmaf(z, -1.f / 3628800, 1.f / 40320);
  c = fmaf(z, c, -1.f / 720);
  c = fmaf(z, c, 1.f / 24);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  const bool odd = quarter & 1;
  sn = odd ? c : s;
  cs = odd ? s : c;
  if (quarter & 2) sn = -sn;
  if ((quarter + 1) & 2) cs = -cs;
}

struct Side {  // one of the two tensors: element strides of batch entries, rows and heads
  const void* in;
  void* out;
  long ib, in_row, ih, ob, o_row, oh;
  int heads;
};

struct Turn {
  Side t[2];
  const unsigned long long* turns;
  const int *positions, *lengths;
  long rows;
  int N, D, R, per, per_row;  // per: heads a thread takes; per_row: a position for every row
  float gain;
  int inverse, in_place;
};

template <typename T>
struct Quad;
template <>
struct Quad<float> {
  using Raw = float4;
  __device__ __forceinline__ static void open(const Raw& u, float* f) { f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w; }
  __device__ __forceinline__ static Raw close(const float* f) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Quad<bf16> {
  using Raw = uint2;
  __device__ __forceinline__ static void open(const Raw& u, float* f) {
    f[0] = __uint_as_float(u.x << 16), f[1] = __uint_as_float(u.x & 0xffff0000u);
    f[2] = __uint_as_float(u.y << 16), f[3] = __uint_as_float(u.y & 0xffff0000u);
  }
  __device__ __forceinline__ static Raw close(const float* f) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};

// (a[i], b[i]) turned by the angle i.
template <int V>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const float (&c)[V], const float (&s)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float p = fmaf(a[i], c[i], -b[i] * s[i]);
    b[i] = fmaf(b[i], c[i], a[i] * s[i]);
    a[i] = p;
  }
}

constexpr int BATCH = 4;  // heads whose loads are on their way together

// A thread's unit of a head's row is two runs of V neighbouring values, V pairs in
// all (V = 4, aligned vectors) or, past R, values to copy; V = 1 takes any sizes and
// strides, its units past R being one value.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(V == 1 ? 1024 : 256) k_rotary(const Turn a, int units, int rb) {
  const int u = threadIdx.x % units, rl = threadIdx.x / units;
  const long row = (long)blockIdx.x * rb + rl;
  if (rl >= rb || row >= a.rows) return;
  const int turning = a.R / (2 * V);
  const bool copy = u >= turning;
  if (copy && a.in_place) return;
  const long b = row / a.N;
  const int n = static_cast<int>(row - b * a.N);
  const bool live = a.lengths == nullptr || n < a.lengths[b];
  if (!live && a.in_place) return;
  int o0, o1;
  if (copy) {
    o0 = V == 1 ? a.R + (u - turning) : a.R + (u - turning) * 2 * V;
    o1 = V == 1 ? o0 : o0 + V;
  } else if (INTER) {
    o0 = u * 2 * V, o1 = o0 + V;
  } else {
    o0 = u * V, o1 = a.R / 2 + o0;
  }
  const int all = a.t[0].heads + a.t[1].heads, first = blockIdx.y * a.per, last = min(first + a.per, all);
  auto input = [&](int h) {
    const bool second = h >= a.t[0].heads;
    const Side& t = a.t[second];
    return static_cast<const T*>(t.in) + b * t.ib + n * t.in_row + (second ? h - a.t[0].heads : h) * t.ih;
  };
  auto output = [&](int h) {
    const bool second = h >= a.t[0].heads;
    const Side& t = a.t[second];
    return static_cast<T*>(t.out) + b * t.ob + n * t.o_row + (second ? h - a.t[0].heads : h) * t.oh;
  };
  using Raw = std::conditional_t<V == 4, typename Quad<T>::Raw, T>;
  Raw r0[BATCH], r1[BATCH];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      r0[i] = r1[i] = Raw{};
      if (live && h0 + i < last) {
        const T* x = input(h0 + i);
        r0[i] = *reinterpret_cast<const Raw*>(x + o0);
        r1[i] = *reinterpret_cast<const Raw*>(x + o1);
      }
    }
  };
  fetch(first);
  float c[V], s[V];
  if (!copy && live) {
    const long long p = a.positions == nullptr ? n : a.per_row ? a.positions[row] : (long long)a.positions[b] + n;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const unsigned long long phase = static_cast<unsigned long long>(p) * a.turns[u * V + i];
      sincos_turn(static_cast<uint32_t>(phase >> 32), s[i], c[i]);
      c[i] *= a.gain;
      s[i] *= a.inverse ? -a.gain : a.gain;
    }
  }
#pragma unroll 1
  for (int h0 = first;;) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (h0 + i >= last) break;
      T* y = output(h0 + i);
      if constexpr (V == 4) {
        if (!copy && live) {
          float f[4], g[4];
          Quad<T>::open(r0[i], f);
          Quad<T>::open(r1[i], g);
          if (INTER) {
            float p[4] = {f[0], f[2], g[0], g[2]}, q[4] = {f[1], f[3], g[1], g[3]};
            turn<4>(p, q, c, s);
            f[0] = p[0], f[1] = q[0], f[2] = p[1], f[3] = q[1];
            g[0] = p[2], g[1] = q[2], g[2] = p[3], g[3] = q[3];
          } else {
            turn<4>(f, g, c, s);
          }
          r0[i] = Quad<T>::close(f);
          r1[i] = Quad<T>::close(g);
        }
      } else if (!copy && live) {
        float f[1] = {to_f(r0[i])}, g[1] = {to_f(r1[i])};
        turn<1>(f, g, c, s);
        r0[i] = from_f<T>(f[0]), r1[i] = from_f<T>(g[0]);
      }
      *reinterpret_cast<Raw*>(y + o0) = r0[i];
      if (V == 4 || !copy) *reinterpret_cast<Raw*>(y + o1) = r1[i];
    }
    h0 += BATCH;
    if (h0 >= last) break;
    fetch(h0);
  }
}

template <typename T>
cudaError_t launch(const Turn& a, bool vec, bool inter, cudaStream_t st) {
  const int units = vec ? a.D / 8 : a.R / 2 + (a.D - a.R);
  const int rb = units >= 256 ? 1 : 256 / units;
  const int threads = (rb * units + 31) / 32 * 32;
  const long blocks = (a.rows + rb - 1) / rb;
  const int all = a.t[0].heads + a.t[1].heads;
  const dim3 grid(static_cast<unsigned>(blocks), (all + a.per - 1) / a.per);
  if (vec)
    inter ? k_rotary<T, 4, true><<<grid, threads, 0, st>>>(a, units, rb) : k_rotary<T, 4, false><<<grid, threads, 0, st>>>(a, units, rb);
  else
    inter ? k_rotary<T, 1, true><<<grid, threads, 0, st>>>(a, units, rb) : k_rotary<T, 1, false><<<grid, threads, 0, st>>>(a, units, rb);
  return cudaGetLastError();
}

bool vectors(const Side& t, size_t elem) {
  const uintptr_t low = reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out);
  return low % (4 * elem) == 0 && (t.ib | t.in_row | t.ih) % 4 == 0;  // outputs are dense, or the inputs themselves
}

}  // namespace

cudaError_t rotary(const void* q, const void* k, void* oq, void* ok, const unsigned long long* turns, const int* positions,
                   const int* lengths, const RotaryShape& s, float gain, cudaStream_t st) {
  Turn a;
  a.turns = turns, a.positions = positions, a.lengths = lengths;
  a.rows = (long)s.B * s.N;
  a.N = s.N, a.D = s.D, a.R = s.R, a.per_row = s.per_row;
  a.gain = gain, a.inverse = s.inverse, a.in_place = q == oq;
  const void* in[2] = {q, k};
  void* out[2] = {oq, ok};
  const int heads[2] = {s.H, s.Hk};
  const long ld[2] = {s.ldq, s.ldk};
  bool vec = s.R % 8 == 0 && s.D % 8 == 0;
  for (int i = 0; i < 2; ++i) {
    Side& t = a.t[i];
    t.in = in[i], t.out = out[i], t.heads = heads[i];
    if (s.head_major) {
      t.ib = t.ob = (long)heads[i] * s.N * s.D, t.in_row = t.o_row = s.D, t.ih = t.oh = (long)s.N * s.D;
    } else {
      const long dense = (long)heads[i] * s.D;
      t.in_row = ld[i], t.ib = ld[i] * s.N, t.ih = t.oh = s.D;
      t.o_row = a.in_place ? ld[i] : dense, t.ob = t.o_row * s.N;
    }
    if (heads[i] > 0) vec = vec && vectors(t, s.dtype == 0 ? 4 : 2);
  }
  // heads a thread takes in turn: as many as leave every SM its threads
  const long items = a.rows * (s.D / 8 + 1);
  const int all = s.H + s.Hk;
  a.per = 1;
  while (a.per < all && a.per < 16 && items * ((all + 2 * a.per - 1) / (2 * a.per)) >= 2048l * sm_count()) a.per *= 2;
  return s.dtype == 0 ? launch<float>(a, vec, s.interleaved, st) : launch<bf16>(a, vec, s.interleaved, st);
}

}  // namespace la
