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
// instructions a row and pair; a thread forms those of its pairs once and takes its row's
// heads, of queries and keys alike, in turn.  4 x 2048 rows of 16 + 4 bf16 heads of 64 out
// of wider rows: 7.7 us (42 MB, 0.80 of the copy rate); 65536 fp32 rows of 8 + 8 heads of
// 64, half of each turned: 78 us (537 MB, the copy rate).
#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "pair.cuh"
#include "scan.cuh"

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
  Divide sequence;  // by N
  int D, R, per, per_row;  // per: heads a thread takes; per_row: a position for every row
  float gain;
  int inverse, in_place;
};

// V neighbouring values as one vector of 8 or 16 bytes, as it lies in memory and as
// pairs of fp32; V = 1: one value.
template <typename T, int V>
struct Run;
template <typename T>
struct Run<T, 1> {
  using Raw = T;
};
template <>
struct Run<float, 4> {
  using Raw = float4;
  __device__ __forceinline__ static void open(const Raw& u, u64* f) { f[0] = pk(u.x, u.y), f[1] = pk(u.z, u.w); }
  __device__ __forceinline__ static Raw close(const u64* f) {
    const float2 a = un(f[0]), b = un(f[1]);
    return make_float4(a.x, a.y, b.x, b.y);
  }
};
__device__ __forceinline__ u64 open2(uint32_t u) { return pk(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }
__device__ __forceinline__ uint32_t close2(u64 v) {
  const float2 f = un(v);
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
struct Run<bf16, 4> {
  using Raw = uint2;
  __device__ __forceinline__ static void open(const Raw& u, u64* f) { f[0] = open2(u.x), f[1] = open2(u.y); }
  __device__ __forceinline__ static Raw close(const u64* f) { return make_uint2(close2(f[0]), close2(f[1])); }
};
template <>
struct Run<bf16, 8> {
  using Raw = uint4;
  __device__ __forceinline__ static void open(const Raw& u, u64* f) { f[0] = open2(u.x), f[1] = open2(u.y), f[2] = open2(u.z), f[3] = open2(u.w); }
  __device__ __forceinline__ static Raw close(const u64* f) { return make_uint4(close2(f[0]), close2(f[1]), close2(f[2]), close2(f[3])); }
};

constexpr int BATCH = 4;  // heads whose loads are on their way together

// A thread's unit of a head's row is two runs of V neighbouring values, V pairs in
// all (V = 4 or, in bf16, 8: aligned vectors) or, past R, values to copy; V = 1 takes any
// sizes and strides, its units past R being one value.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(V == 1 ? 1024 : 256) k_rotary(const Turn a, int units, int rb) {
  grid_dep_enter();
  const int u = threadIdx.x % units, rl = threadIdx.x / units;
  const long row = (long)blockIdx.x * rb + rl;
  if (rl >= rb || row >= a.rows) return;
  const int turning = a.R / (2 * V);
  const bool copy = u >= turning;
  if (copy && a.in_place) return;
  const uint32_t seq = a.sequence(static_cast<uint32_t>(row));
  const long b = seq;
  const int n = static_cast<int>(static_cast<uint32_t>(row) - seq * a.sequence.d);
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
  using Raw = typename Run<T, V>::Raw;
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
  // cos and sin by pairs of angles; interleaved, the angle of each value's own pair
  constexpr int P = V > 1 ? V / 2 : 1;
  u64 cp[P], sp[P], np[P];
  if constexpr (V > 1) {
#pragma unroll
    for (int i = 0; i < P; ++i) cp[i] = pk(c[2 * i], c[2 * i + 1]), sp[i] = pk(s[2 * i], s[2 * i + 1]), np[i] = pk(-s[2 * i], -s[2 * i + 1]);
  }
#pragma unroll 1
  for (int h0 = first;;) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (h0 + i >= last) break;
      T* y = output(h0 + i);
      if constexpr (V > 1) {
        if (!copy && live) {
          u64 f[P], g[P];
          Run<T, V>::open(r0[i], f);
          Run<T, V>::open(r1[i], g);
          if constexpr (INTER) {  // a run holds (a, b) of V / 2 pairs
#pragma unroll
            for (int j = 0; j < P / 2; ++j) {
              auto pair = [&](u64& lo, u64& hi, int k) {  // two of the pairs
                const float2 p = un(lo), q = un(hi);
                const u64 av = pk(p.x, q.x), bv = pk(p.y, q.y);
                const float2 x = un(fma2(av, cp[k], mul2(bv, np[k]))), z = un(fma2(bv, cp[k], mul2(av, sp[k])));
                lo = pk(x.x, z.x), hi = pk(x.y, z.y);
              };
              pair(f[2 * j], f[2 * j + 1], j);
              pair(g[2 * j], g[2 * j + 1], P / 2 + j);
            }
          } else {
#pragma unroll
            for (int j = 0; j < P; ++j) {
              const u64 x = fma2(f[j], cp[j], mul2(g[j], np[j]));
              g[j] = fma2(g[j], cp[j], mul2(f[j], sp[j]));
              f[j] = x;
            }
          }
          r0[i] = Run<T, V>::close(f);
          r1[i] = Run<T, V>::close(g);
        }
      } else if (!copy && live) {
        const float f = to_f(r0[i]), g = to_f(r1[i]);
        r0[i] = from_f<T>(fmaf(f, c[0], -g * s[0])), r1[i] = from_f<T>(fmaf(g, c[0], f * s[0]));
      }
      *reinterpret_cast<Raw*>(y + o0) = r0[i];
      if (V > 1 || !copy) *reinterpret_cast<Raw*>(y + o1) = r1[i];
    }
    h0 += BATCH;
    if (h0 >= last) break;
    fetch(h0);
  }
}

template <typename T, int V>
cudaError_t launch(Turn& a, bool inter, cudaStream_t st) {
  const int units = V > 1 ? a.D / (2 * V) : a.R / 2 + (a.D - a.R);
  const int rb = units >= 256 ? 1 : 256 / units;
  const int threads = (rb * units + 31) / 32 * 32;
  const long blocks = (a.rows + rb - 1) / rb;
  // heads a thread takes in turn: as many as let the blocks run at once, three on an SM, and at most
  // eight (4 x 2048 rows, 20 heads: 7.7 us a pass with seven, 8.6 with four, 10 with all; 65536 fp32
  // rows of 16 heads: 78 us with three to seven, 84 with all)
  const int all = a.t[0].heads + a.t[1].heads;
  const long groups = std::max(1l, std::min<long>(all, 3l * sm_count() / blocks));
  a.per = std::min(8, static_cast<int>((all + groups - 1) / groups));
  const dim3 grid(static_cast<unsigned>(blocks), (all + a.per - 1) / a.per);
  return launch_pdl(inter ? k_rotary<T, V, true> : k_rotary<T, V, false>, grid, dim3(threads), 0, st, a, units, rb);
}

// Rows, heads and strides in whole runs of V values, aligned.
bool runs(const Turn& a, int V, size_t elem) {
  if (a.R % (2 * V) || a.D % (2 * V)) return false;
  for (const Side& t : a.t) {  // outputs are dense, or the inputs themselves
    const uintptr_t low = reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out);
    if (t.heads > 0 && (low % (V * elem) || (t.ib | t.in_row | t.ih) % V)) return false;
  }
  return true;
}

}  // namespace

cudaError_t rotary(const void* q, const void* k, void* oq, void* ok, const unsigned long long* turns, const int* positions,
                   const int* lengths, const RotaryShape& s, float gain, cudaStream_t st) {
  Turn a;
  a.turns = turns, a.positions = positions, a.lengths = lengths;
  a.rows = (long)s.B * s.N;
  a.sequence = Divide(static_cast<uint32_t>(s.N)), a.D = s.D, a.R = s.R, a.per_row = s.per_row;
  a.gain = gain, a.inverse = s.inverse, a.in_place = q == oq;
  const void* in[2] = {q, k};
  void* out[2] = {oq, ok};
  const int heads[2] = {s.H, s.Hk};
  const long ld[2] = {s.ldq, s.ldk};
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
  }
  if (s.dtype == 0) return runs(a, 4, 4) ? launch<float, 4>(a, s.interleaved, st) : launch<float, 1>(a, s.interleaved, st);
  return runs(a, 8, 2)   ? launch<bf16, 8>(a, s.interleaved, st)
         : runs(a, 4, 2) ? launch<bf16, 4>(a, s.interleaved, st)
                         : launch<bf16, 1>(a, s.interleaved, st);
}

}  // namespace la
