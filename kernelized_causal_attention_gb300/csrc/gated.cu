// Gated recurrence over token-major rows, one decay and one state a channel:
//   s = sigmoid(r), g = sigmoid(i), u = k s with k = scale softplus(lam), a = exp(-u),
//   h_n = a h_{n-1} + beta g x, beta = sqrt(1 - a^2),  y_n = h_n,
// and its gradients, with G_n = dy_n + a_{n+1} G_{n+1}:
//   dx = G beta g,  di = G beta x g (1 - g),  Q = a G (a g x u / beta - u h_{n-1}),
//   dr = (1 - s) Q,  dlam = sigmoid(lam) / softplus(lam) sum Q.
// (u / beta goes to zero with u, so a closed gate has no infinite term.)
//
// The recurrence is associative: a tile of rows turns its first state h into A h + H.
// One pass a direction reads every row once: resident blocks take tiles of rows of CH
// channels in turn, the next tile's rows on their way into shared memory (a warp's own
// rows, 16 bytes a copy) while one is worked on.  A thread has two channels of a strip of
// rows, whose a and b it keeps in registers; the strips are joined through shared memory,
// the tile's (A, H) goes to device memory, the tiles before it are looked up, and the
// strips are replayed from the state that these give.  Blocks run all at once (a
// cooperative launch) and take tiles in order, every grid's width one, so the first tile
// that is not done waits for none.
// The state passed on is the same sequence of fused multiply-adds whichever tiles had
// theirs already, so results repeat bit for bit.
//
// 4 x 2048 x 2048 bf16: forward 34 us (134 MB, 0.57 of the copy rate), gradients 64 (235
// MB, 0.54), clearing the words and joining dlam 2 each; 65536 x 512 bf16: forward
// 76 (268 MB, 0.52).  About 79 and 167 instructions for a warp's row (64 channels), issued
// at 55 % of the rate: a tile's phases (rows in, gates, the states before it, replay, rows
// out: 1300, 3700, 1800, 900, 300 cycles forward) follow one another on two blocks an SM;
// with the gates' arithmetic taken out a training pass took 89 us where it took 103 (102 now).
// One block a column that walks the rows would leave most SMs idle at these widths; three
// passes that read the rows twice took 216; three blocks an SM without rows ahead 113.
//
// These are decays of u < 1.  A warp whose strip has one u above that computes the strip's
// gates a second time, in the full form: with lam spread over -9 to 2 (scale 8) training takes
// 152 us for 102 and the prompt 120 for 77; over 0 to 2 149 and 117.
//
// 128 registers a thread; the bf16 gradients spill 4 bytes, the bf16 forward of rows off
// sixteen bytes 36 (multiples of four) and 68.
#include <algorithm>
#include <atomic>

#include "pair.cuh"
#include "scan.cuh"

namespace la {
namespace {

using bf16 = __nv_bfloat16;

constexpr int CH = 64;      // channels of a tile, two a lane
constexpr int WARPS = 8;    // strips of a tile
constexpr int KEEP = 64;    // rows of a gradient tile, and between the states kept for it
constexpr int FWD_WINDOW = 16, BACK_WINDOW = 32;  // tiles looked up before one must have its state
constexpr int BLOCKS = 2;   // on an SM; three of half the strips were slower: 107 us against 79 for 65536 x 512
template <typename T>
constexpr int FWD = sizeof(T) == 4 ? 8 : 16;  // rows of a strip, forward: 48 KB of rows a tile
template <typename T>
constexpr int BACK_STAGES = sizeof(T) == 4 ? 1 : 2;  // 64 and 32 KB of rows a gradient tile

// ---------------------------------------------------------- two channels at once

__device__ __forceinline__ float rsqrt_fast(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ u64 ex2_2(u64 v) {
  const float2 f = un(v);
  return pk(ex2_fast(f.x), ex2_fast(f.y));
}
__device__ __forceinline__ u64 rcp_2(u64 v) {
  const float2 f = un(v);
  return pk(rcp_fast(f.x), rcp_fast(f.y));
}

// w = 1 - exp(-u) on [0, 1], relative error 2^-22.6 at most (the fit alone 2^-25), so that a
// decay close to one is one minus it: a polynomial fitted to w / u.  Above, the exponential
// is the decay, which keeps its bits there, and w one minus that.
__device__ __forceinline__ u64 near_one(u64 u) {
  u64 p = fma2(u, two(0.00012918687f), two(-0.0013011073f));
  p = fma2(u, p, two(0.00827588f));
  p = fma2(u, p, two(-0.041647043f));
  p = fma2(u, p, two(0.16666345f));
  p = fma2(u, p, two(-0.4999998f));
  p = fma2(u, p, two(1.f));
  return mul2(u, p);
}
__device__ __forceinline__ u64 minus_one(u64 w) { return fma2(w, two(-1.f), two(1.f)); }
// beta = sqrt(w (1 + a)), with the smallest normal number under the root of its inverse: zero
// where w is, and half a step off from w = 5e-32 on.
__device__ __forceinline__ u64 root(u64 w, u64 a) {
  const u64 om = fma2(w, a, w);
  const float2 f = un(add2(om, two(1.2e-38f)));
  return mul2(om, pk(rsqrt_fast(f.x), rsqrt_fast(f.y)));
}
// The larger of three, NaN if one is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float v;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(v) : "f"(a), "f"(b), "f"(c));
  return v;
}

// A row's gates: s, g, a and beta.  Both sigmoids, 1 / (1 + e) each, come from one
// reciprocal of the product, unless that is near overflow or NaN (arguments below -69 in
// sum).  The short forms hold while the largest product stays below 1e30 and the largest
// u below one; the full form gives a channel for which they do the same bits.
struct Reach {
  float p = 0.f, u = 0.f;
  __device__ __forceinline__ bool quick() const { return (p < 1e30f) & (u < 1.f); }
};
__device__ __forceinline__ void gates_quick(u64 r, u64 i, u64 k, u64& s, u64& g, u64& a, u64& beta, Reach& reach) {
  const u64 scale = two(-1.4426950408889634f), one = two(1.f);
  const u64 d1 = add2(ex2_2(mul2(r, scale)), one), d2 = add2(ex2_2(mul2(i, scale)), one), p = mul2(d1, d2), q = rcp_2(p);
  s = mul2(q, d2), g = mul2(q, d1);
  const u64 u = mul2(k, s), w = near_one(u);
  const float2 pf = un(p), uf = un(u);
  reach.p = max3(reach.p, pf.x, pf.y), reach.u = max3(reach.u, uf.x, uf.y);
  a = minus_one(w);
  beta = root(w, a);
}
__device__ __forceinline__ u64 pick(bool x, bool y, u64 a, u64 b) {
  const float2 af = un(a), bf = un(b);
  return pk(x ? af.x : bf.x, y ? af.y : bf.y);
}
__device__ __forceinline__ void gates(u64 r, u64 i, u64 k, u64& s, u64& g, u64& a, u64& beta) {
  const u64 scale = two(-1.4426950408889634f), one = two(1.f);
  const u64 d1 = add2(ex2_2(mul2(r, scale)), one), d2 = add2(ex2_2(mul2(i, scale)), one), p = mul2(d1, d2), q = rcp_2(p);
  const float2 pf = un(p);
  s = pick(pf.x < 1e30f, pf.y < 1e30f, mul2(q, d2), rcp_2(d1)), g = pick(pf.x < 1e30f, pf.y < 1e30f, mul2(q, d1), rcp_2(d2));
  const u64 u = mul2(k, s);
  const float2 uf = un(u);
  const u64 e = ex2_2(mul2(u, scale));
  const u64 w = pick(uf.x < 1.f, uf.y < 1.f, near_one(u), minus_one(e));
  a = pick(uf.x < 1.f, uf.y < 1.f, minus_one(w), e);
  beta = root(w, a);
}

// ------------------------------------------------------------------------- rows

// Two neighbouring channels, as they lie in memory.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  using type = u64;
};
template <>
struct Raw<bf16> {
  using type = uint32_t;
};
__device__ __forceinline__ u64 open(u64 t) { return t; }
__device__ __forceinline__ u64 open(uint32_t t) { return pk(__uint_as_float(t << 16), __uint_as_float(t & 0xffff0000u)); }
template <typename T>
__device__ __forceinline__ typename Raw<T>::type close(u64 v) {
  if constexpr (sizeof(T) == 4) {
    return v;
  } else {
    const float2 f = un(v);
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
}
// The same from and to any address, channel by channel.
__device__ __forceinline__ u64 gather(const float* p, int n) { return pk(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f); }
__device__ __forceinline__ uint32_t gather(const bf16* p, int n) {
  const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
  return (n > 0 ? static_cast<uint32_t>(q[0]) : 0u) | (n > 1 ? static_cast<uint32_t>(q[1]) << 16 : 0u);
}
__device__ __forceinline__ void scatter(float* p, int n, u64 v) {
  const float2 f = un(v);
  if (n > 0) p[0] = f.x;
  if (n > 1) p[1] = f.y;
}
__device__ __forceinline__ void scatter(bf16* p, int n, uint32_t v) {
  unsigned short* q = reinterpret_cast<unsigned short*>(p);
  if (n > 0) q[0] = static_cast<unsigned short>(v);
  if (n > 1) q[1] = static_cast<unsigned short>(v >> 16);
}

struct Rows {
  const void *x, *r, *i, *lam;
  const int* lengths;
  const float* rate;  // scale softplus(lam), with zeros up to a multiple of CH (null: from lam)
  long ldx, ldr, ldi;
  int B, N, C, groups, tiles;  // groups of CH channels; tiles of a direction's rows
  float scale;
};

// Tiles that pass states on: by tile and column (batch entry and group) A, H and then the
// state behind the tile, 32 words each.
struct Chain {
  u64* word;
  int* err;
};

struct Job {
  int tile, col, b, c0, L;  // c0: first channel; L: the sequence's valid rows; tile < 0: none
};

__device__ __forceinline__ Job job_of(const Rows& a, int number, int total, bool reverse) {
  Job j{-1, 0, 0, 0, 0};
  if (number < total) {
    const int cols = a.groups * a.B, t = number / cols;
    j.col = number - t * cols;
    j.tile = reverse ? a.tiles - 1 - t : t;
    j.b = j.col / a.groups;
    j.c0 = (j.col - j.b * a.groups) * CH;
    j.L = valid_rows(a.lengths, j.b, a.N);
  }
  return j;
}

template <typename T>
__device__ __forceinline__ u64 rates(const Rows& a, int c) {
  if (a.rate != nullptr) return *reinterpret_cast<const u64*>(a.rate + c);
  const float2 l = un(open(gather(static_cast<const T*>(a.lam) + c, a.C - c)));
  return pk(c < a.C ? a.scale * softplus(l.x) : 0.f, c + 1 < a.C ? a.scale * softplus(l.y) : 0.f);
}

template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from, int bytes) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(to)), "l"(from), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(to)), "l"(from), "r"(bytes) : "memory");
}

// A warp's RW rows from t0 on of CH channels from c0 on into its own rows of shared
// memory; zeros past the length and the width.  UNIT: the bytes that rows, widths and
// strides are whole multiples of: 16 or 4, asynchronous copies of that many, or 2.
template <typename T, int UNIT, int RW>
__device__ __forceinline__ void bring(T* to, const void* base, long ld, const Rows& a, const Job& j, int t0) {
  const int lane = threadIdx.x & 31;
  const T* from = static_cast<const T*>(base) + ((long)j.b * a.N + t0) * ld + j.c0;
  if constexpr (UNIT == 16) {
    constexpr int E = 16 / sizeof(T), LR = CH / E, PER = 32 / LR;  // lanes a row, rows an instruction
    const int c = (lane % LR) * E, r0 = lane / LR;
    const bool wide = j.c0 + c < a.C;
    const T* q = from + r0 * ld + c;
    T* o = to + r0 * CH + c;
    if (t0 + RW <= j.L && j.c0 + CH <= a.C) {
#pragma unroll
      for (int r = 0; r < RW; r += PER) {
        copy_async<16>(o + r * CH, q, 16);
        q += PER * ld;
      }
    } else {
#pragma unroll
      for (int r = 0; r < RW; r += PER) {
        const bool in = wide && t0 + r0 + r < j.L;
        copy_async<16>(o + r * CH, in ? q : base, in ? 16 : 0);
        q += PER * ld;
      }
    }
  } else if constexpr (UNIT == 4) {
    constexpr int E = 4 / sizeof(T);
    for (int c = lane * E; c < CH; c += 32 * E) {
      const bool wide = j.c0 + c < a.C;
      const T* q = from + c;
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        const bool in = wide && t0 + r < j.L;
        copy_async<4>(to + r * CH + c, in ? q : base, in ? 4 : 0);
        q += ld;
      }
    }
  } else {
    const int n = a.C - j.c0 - 2 * lane;
#pragma unroll
    for (int r = 0; r < RW; ++r)
      reinterpret_cast<typename Raw<T>::type*>(to)[r * (CH / 2) + lane] = gather(from + r * ld + 2 * lane, t0 + r < j.L ? n : 0);
  }
}

// The way back: a warp's RW rows, as far as there are N.
template <typename T, int UNIT, int RW>
__device__ __forceinline__ void leave(T* out, const T* from, const Rows& a, const Job& j, int t0) {
  const int lane = threadIdx.x & 31;
  T* to = out + ((long)j.b * a.N + t0) * a.C + j.c0;
  if constexpr (UNIT == 16) {
    constexpr int E = 16 / sizeof(T), LR = CH / E, PER = 32 / LR;
    const int c = (lane % LR) * E, r0 = lane / LR;
    T* q = to + (long)r0 * a.C + c;
    const T* o = from + r0 * CH + c;
    const bool wide = j.c0 + c < a.C, all = t0 + RW <= a.N && j.c0 + CH <= a.C;
    if (all) {
#pragma unroll
      for (int r = 0; r < RW; r += PER) {
        *reinterpret_cast<uint4*>(q) = *reinterpret_cast<const uint4*>(o + r * CH);
        q += (long)PER * a.C;
      }
    } else {
#pragma unroll
      for (int r = 0; r < RW; r += PER) {
        if (wide && t0 + r0 + r < a.N) *reinterpret_cast<uint4*>(q) = *reinterpret_cast<const uint4*>(o + r * CH);
        q += (long)PER * a.C;
      }
    }
  } else {
    const int n = a.C - j.c0 - 2 * lane;
#pragma unroll 4
    for (int r = 0; r < RW; ++r)
      if (t0 + r < a.N) scatter(to + (long)r * a.C + 2 * lane, n, reinterpret_cast<const typename Raw<T>::type*>(from)[r * (CH / 2) + lane]);
  }
}

// -------------------------------------------------------------------- the chain

// Words of a tile start as EMPTY, a pair of NaNs that no sum gives (those are the
// canonical one), and say by themselves that they have come: a tile's words need no
// order among them, and one round trip brings them.
constexpr u64 EMPTY = ~0ull;
__device__ __forceinline__ void put(u64* p, u64 v) { asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory"); }
__device__ __forceinline__ u64 look(const u64* p) {
  u64 v;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}

template <int WINDOW>
struct Shared {
  u64 A[2][WARPS][32], H[2][WARPS][32];  // (A, H) of the strips, by lane; alternate tiles use alternate halves
  u64 wA[WINDOW][32], wH[WINDOW][32];    // of the tiles looked up; wH: the state where kind is 2
  u64 start[2][32];                      // the caller's state
  int kind[WINDOW];
};

// What the n tiles before this one (the j-th is at entry + j step of the chain) pass on:
// the nearest state, moved on by the tiles since.  All threads call it; warp w looks
// up the tiles w, w + WARPS, ...  The tile that is WINDOW back must have its state.
// A wait of two seconds gives up: zero, and the code in the status word.
template <int WINDOW>
__device__ __forceinline__ u64 look_up(Shared<WINDOW>& sh, const Chain& ch, long entry, long step, int n, int code) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int found = -1;
#pragma unroll 1
  for (int base = 0; base < WINDOW && found < 0; base += WARPS) {
    const int j = base + w;
    if (j < n) {
      const u64* p = ch.word + (entry + j * step) * 96 + lane;
      u64 A, H, t0 = 0;
      int kind = 0;
      for (int tries = 0; kind == 0; ++tries) {
        const u64 S = look(p + 64);
        A = look(p), H = look(p + 32);
        if (__all_sync(0xffffffffu, S != EMPTY)) {
          H = S, kind = 2;
        } else if (j != WINDOW - 1 && __all_sync(0xffffffffu, (A != EMPTY) & (H != EMPTY))) {
          kind = 1;
        } else if ((tries & 255) == 255) {
          const u64 now = tc::globaltimer_ns();
          if (t0 == 0) t0 = now;
          if (__any_sync(0xffffffffu, now - t0 > 2000000000ull)) {
            if (lane == 0) tcc::fail(ch.err, code);
            H = 0ull, kind = 2;
          }
        }
      }
      if (kind == 1) sh.wA[j][lane] = A;
      sh.wH[j][lane] = H;
      if (lane == 0) sh.kind[j] = kind;
    }
    __syncthreads();
    const int i = base + lane % WARPS;  // one load for all of them: 76 us for 79 where 38 tiles of a column are under way
    const unsigned states = __ballot_sync(0xffffffffu, sh.kind[i] == 2 && i < n);
    if (states != 0) found = base + __ffs(states) - 1;
  }
  u64 s = sh.wH[found][lane];
  for (int i = found - 1; i >= 0; --i) s = fma2(sh.wA[i][lane], s, sh.wH[i][lane]);
  return s;
}

// A call's words to EMPTY, and the channels' rates.
template <typename T>
__global__ void __launch_bounds__(256) k_gated_start(const Chain ch, long n, float* rate, const T* lam, float scale, int C, int padded) {
  tcc::grid_dep_wait();  // before letting the next kernel start: that one asks for its rows before it waits for this
  tcc::grid_dep_launch();
  const long e = (long)blockIdx.x * 256 + threadIdx.x, step = (long)gridDim.x * 256;
  for (long i = e; i < n * 48; i += step) reinterpret_cast<ulonglong2*>(ch.word)[i] = make_ulonglong2(EMPTY, EMPTY);
  for (long i = e; i < padded; i += step) rate[i] = i < C ? scale * softplus(to_f(lam[i])) : 0.f;
}

// ---------------------------------------------------------------------- forward

template <typename T, int UNIT, bool CHAIN>
__global__ void __launch_bounds__(32 * WARPS, BLOCKS)
    k_gated_fwd(const Rows a, const Chain ch, float* h, float* __restrict__ kept, T* __restrict__ y, int total) {
  constexpr int RW = FWD<T>, ROWS = WARPS * RW;
  using R = typename Raw<T>::type;
  extern __shared__ __align__(16) unsigned char room[];
  __shared__ Shared<FWD_WINDOW> sh;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, cols = a.groups * a.B;
  auto own = [&](int stage, int t) { return reinterpret_cast<T*>(room) + ((stage * 3 + t) * ROWS + w * RW) * CH; };
  auto request = [&](int stage, const Job& j) {
    const int t0 = j.tile * ROWS + w * RW;
    if (j.tile >= 0 && t0 < j.L) {
      bring<T, UNIT, RW>(own(stage, 1), a.r, a.ldr, a, j, t0);
      bring<T, UNIT, RW>(own(stage, 2), a.i, a.ldi, a, j, t0);
      bring<T, UNIT, RW>(own(stage, 0), a.x, a.ldx, a, j, t0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  Job job = job_of(a, blockIdx.x, total, false);
  request(0, job);
  if (CHAIN) tcc::grid_dep_wait();  // the chain's words and the rates
  for (int stage = 0, t = blockIdx.x; job.tile >= 0; stage ^= 1) {
    t += gridDim.x;
    const Job next = job_of(a, t, total, false);
    const int t0 = job.tile * ROWS + w * RW, c = job.c0 + 2 * lane, n = a.C - c;
    const bool live = job.tile == 0 || job.tile * ROWS < job.L;  // nothing behind the length passes anything on
    const u64 k = live ? rates<T>(a, c) : 0ull;
    if (CHAIN) {
      request(stage ^ 1, next);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(CHAIN ? 1 : 0) : "memory");
    __syncwarp();
    R* px = reinterpret_cast<R*>(own(stage, 0)) + lane;
    const R *pr = reinterpret_cast<const R*>(own(stage, 1)) + lane, *pi = reinterpret_cast<const R*>(own(stage, 2)) + lane;
    float* hp = h == nullptr ? nullptr : h + (long)job.b * a.C + c;
    u64 av[RW], bv[RW], A = two(1.f), H = 0ull;
    const bool full = t0 + RW <= job.L;  // the same for a warp
    if (live) {
      Reach reach;
      if (full) {
#pragma unroll
        for (int j = 0; j < RW; ++j) {
          u64 s, g, beta;
          gates_quick(open(pr[j * (CH / 2)]), open(pi[j * (CH / 2)]), k, s, g, av[j], beta, reach);
          bv[j] = mul2(beta, mul2(g, open(px[j * (CH / 2)])));
        }
      }
      if (!full || !reach.quick()) {
#pragma unroll
        for (int j = 0; j < RW; ++j) {
          av[j] = two(1.f), bv[j] = 0ull;  // rows past the length keep the state
          if (t0 + j < job.L) {
            u64 s, g, beta;
            gates(open(pr[j * (CH / 2)]), open(pi[j * (CH / 2)]), k, s, g, av[j], beta);
            bv[j] = mul2(beta, mul2(g, open(px[j * (CH / 2)])));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < RW; ++j) {
        H = fma2(av[j], H, bv[j]);
        A = mul2(A, av[j]);
      }
      sh.A[stage][w][lane] = A, sh.H[stage][w][lane] = H;
      if (job.tile == 0 && w == 0) sh.start[stage][lane] = hp == nullptr ? 0ull : gather(hp, n);
    }
    __syncthreads();
    if (live) {
      u64 s = job.tile == 0 ? sh.start[stage][lane] : 0ull;
      const bool last = (job.tile + 1) * ROWS >= job.L;  // of the tiles with valid rows
      if (CHAIN) {
        const long entry = (long)job.tile * cols + job.col;
        u64* word = ch.word + entry * 96 + lane;
        if (w == 0 && !last) {
#pragma unroll
          for (int i = 1; i < WARPS; ++i) {
            const u64 Ai = sh.A[stage][i][lane];
            H = fma2(Ai, H, sh.H[stage][i][lane]);
            A = mul2(A, Ai);
          }
          if (job.tile > 0) put(word, A), put(word + 32, H);
        }
        if (job.tile > 0) s = look_up(sh, ch, entry - cols, -cols, job.tile, 91);
        if (w == 0 && !last) {
          if (job.tile == 0) __threadfence();  // h is read before another tile replaces it
          put(word + 64, fma2(A, s, H));
        }
      }
#pragma unroll  // as many loads at once for every warp: 1 % of both directions
      for (int i = 0; i < WARPS - 1; ++i)
        if (i < w) s = fma2(sh.A[stage][i][lane], s, sh.H[stage][i][lane]);
      float* to = kept == nullptr ? nullptr : kept + ((long)job.b * ((a.N + KEEP - 1) / KEEP) + t0 / KEEP) * a.C + c;
      if (to != nullptr && t0 % KEEP == 0 && t0 < a.N) scatter(to, n, s);
      if (full) {
#pragma unroll
        for (int j = 0; j < RW; ++j) {
          s = fma2(av[j], s, bv[j]);
          px[j * (CH / 2)] = close<T>(s);
        }
      } else {
#pragma unroll
        for (int j = 0; j < RW; ++j) {
          s = fma2(av[j], s, bv[j]);
          px[j * (CH / 2)] = t0 + j < job.L ? close<T>(s) : R{};
        }
      }
      if (hp != nullptr && w == WARPS - 1 && last) {
        __threadfence();
        scatter(hp, n, s);
      }
    } else {
#pragma unroll
      for (int j = 0; j < RW; ++j) px[j * (CH / 2)] = R{};
    }
    __syncwarp();
    leave<T, UNIT, RW>(y, own(stage, 0), a, job, t0);
    __syncwarp();  // the rows are out before the next ones come in
    job = next;
  }
}

// -------------------------------------------------------------------- gradients

// All gradients of a tile, from the state before it (kept), and its sums of Q.  What
// arrives at a tile's last row is X = a G of the row behind it, passed on from the back:
// X_n = a_n (dy_n + X_{n+1}).  s, g, a and the states before the rows stay in registers,
// beta goes where the row's r and i were.
template <typename T, int UNIT, bool CHAIN>
__global__ void __launch_bounds__(32 * WARPS, BLOCKS)
    k_gated_bwd(const Rows a, const Chain ch, const T* __restrict__ dy, const float* __restrict__ kept, T* __restrict__ dx, T* __restrict__ dr,
                T* __restrict__ di, float* __restrict__ sums, int total) {
  constexpr int RW = KEEP / WARPS, STAGES = CHAIN ? BACK_STAGES<T> : 1;
  using R = typename Raw<T>::type;
  extern __shared__ __align__(16) unsigned char room[];
  __shared__ Shared<BACK_WINDOW> sh;
  __shared__ u64 sY[2][WARPS][32], total_of[WARPS][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, cols = a.groups * a.B;
  auto own = [&](int stage, int t) { return reinterpret_cast<T*>(room) + ((stage * 4 + t) * KEEP + w * RW) * CH; };
  auto request = [&](int stage, const Job& j) {
    const int t0 = j.tile * KEEP + w * RW;
    if (j.tile >= 0 && t0 < j.L) {
      bring<T, UNIT, RW>(own(stage, 1), a.r, a.ldr, a, j, t0);
      bring<T, UNIT, RW>(own(stage, 2), a.i, a.ldi, a, j, t0);
      bring<T, UNIT, RW>(own(stage, 0), a.x, a.ldx, a, j, t0);
      bring<T, UNIT, RW>(own(stage, 3), dy, a.C, a, j, t0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  tcc::grid_dep_launch();
  Job job = job_of(a, blockIdx.x, total, true);
  request(0, job);
  if (CHAIN) tcc::grid_dep_wait();  // the chain's words and the rates
  for (int half = 0, t = blockIdx.x; job.tile >= 0; half ^= 1) {
    const int stage = STAGES > 1 ? half : 0;
    t += gridDim.x;
    const Job next = job_of(a, t, total, true);
    const int t0 = job.tile * KEEP + w * RW, c = job.c0 + 2 * lane, n = a.C - c;
    const bool live = job.tile * KEEP < job.L;
    const long rec = ((long)job.b * a.tiles + job.tile) * a.C + c;
    const u64 k = live ? rates<T>(a, c) : 0ull;
    u64 s = live ? gather(kept + rec, n) : 0ull, X = 0ull, sum = 0ull;
    if (CHAIN) {
      if (STAGES > 1) request(stage ^ 1, next);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES > 1 ? 1 : 0) : "memory");
    __syncwarp();
    R *px = reinterpret_cast<R*>(own(stage, 0)) + lane, *pr = reinterpret_cast<R*>(own(stage, 1)) + lane,
      *pi = reinterpret_cast<R*>(own(stage, 2)) + lane;
    const R* pd = reinterpret_cast<const R*>(own(stage, 3)) + lane;
    u64 sv[RW], gv[RW], av[RW], bv[RW], A = two(1.f), H = 0ull, Y = 0ull;
    const bool full = t0 + RW <= job.L;  // the same for a warp
    if (live) {
      Reach reach;
      float2 beta_of[RW];
      if (full) {
#pragma unroll
        for (int j = 0; j < RW; ++j) {
          u64 beta;
          gates_quick(open(pr[j * (CH / 2)]), open(pi[j * (CH / 2)]), k, sv[j], gv[j], av[j], beta, reach);
          bv[j] = mul2(beta, mul2(gv[j], open(px[j * (CH / 2)])));
          beta_of[j] = un(beta);
        }
      }
      if (!full || !reach.quick()) {
#pragma unroll
        for (int j = 0; j < RW; ++j) {
          av[j] = two(1.f), sv[j] = gv[j] = bv[j] = 0ull, beta_of[j] = make_float2(0.f, 0.f);
          if (t0 + j < job.L) {
            u64 beta;
            gates(open(pr[j * (CH / 2)]), open(pi[j * (CH / 2)]), k, sv[j], gv[j], av[j], beta);
            bv[j] = mul2(beta, mul2(gv[j], open(px[j * (CH / 2)])));
            beta_of[j] = un(beta);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < RW; ++j) {
        if constexpr (sizeof(T) == 4) {
          pr[j * (CH / 2)] = pk(beta_of[j].x, beta_of[j].y);
        } else {
          pr[j * (CH / 2)] = __float_as_uint(beta_of[j].x), pi[j * (CH / 2)] = __float_as_uint(beta_of[j].y);
        }
        H = fma2(av[j], H, bv[j]);
        A = mul2(A, av[j]);
      }
      if (full) {
#pragma unroll
        for (int j = RW - 1; j >= 0; --j) Y = mul2(av[j], add2(open(pd[j * (CH / 2)]), Y));
      } else {
#pragma unroll
        for (int j = RW - 1; j >= 0; --j) Y = mul2(av[j], add2(t0 + j < job.L ? open(pd[j * (CH / 2)]) : 0ull, Y));
      }
      sh.A[half][w][lane] = A, sh.H[half][w][lane] = H, sY[half][w][lane] = Y;
    }
    __syncthreads();
    if (live) {
      if (CHAIN) {
        const int last = (job.L - 1) / KEEP;
        const long entry = (long)job.tile * cols + job.col;
        u64* word = ch.word + entry * 96 + lane;
        if (w == WARPS - 1 && job.tile > 0) {
#pragma unroll
          for (int i = WARPS - 2; i >= 0; --i) {
            const u64 Ai = sh.A[half][i][lane];
            Y = fma2(Ai, Y, sY[half][i][lane]);
            A = mul2(A, Ai);
          }
          if (job.tile < last) put(word, A), put(word + 32, Y);
        }
        if (job.tile < last) X = look_up(sh, ch, entry + cols, cols, last - job.tile, 92);
        if (w == WARPS - 1 && job.tile > 0) put(word + 64, fma2(A, X, Y));
      }
#pragma unroll
      for (int i = 0; i < WARPS; ++i) {
        if (i < w) s = fma2(sh.A[half][i][lane], s, sh.H[half][i][lane]);
        if (WARPS - 1 - i > w) X = fma2(sh.A[half][WARPS - 1 - i][lane], X, sY[half][WARPS - 1 - i][lane]);
      }
#pragma unroll
      for (int j = 0; j < RW; ++j) {  // bv becomes the state before the row
        const u64 after = fma2(av[j], s, bv[j]);
        bv[j] = s;
        s = after;
      }
      auto gradients = [&](int j, u64& ox, u64& orr, u64& oi) {
        const u64 one = two(1.f), neg = two(-1.f);
        u64 beta;
        if constexpr (sizeof(T) == 4)
          beta = pr[j * (CH / 2)];
        else
          beta = pk(__uint_as_float(pr[j * (CH / 2)]), __uint_as_float(pi[j * (CH / 2)]));
        const u64 inverse = rcp_2(add2(beta, two(1e-27f)));  // u is zero where beta is; any other beta is 1e-26 at least
        const u64 G = add2(open(pd[j * (CH / 2)]), X), gx = mul2(gv[j], open(px[j * (CH / 2)]));
        X = mul2(av[j], G);
        // Q = a G (a g x u / beta - u h)
        const u64 u = mul2(k, sv[j]);
        const u64 Q = mul2(X, fma2(mul2(u, neg), bv[j], mul2(mul2(av[j], gx), mul2(u, inverse))));
        sum = add2(sum, Q);
        const u64 Gb = mul2(G, beta);
        ox = mul2(Gb, gv[j]);
        orr = mul2(Q, fma2(sv[j], neg, one));
        oi = mul2(mul2(Gb, gx), fma2(gv[j], neg, one));
      };
      if (full) {
#pragma unroll
        for (int j = RW - 1; j >= 0; --j) {
          u64 ox, orr, oi;
          gradients(j, ox, orr, oi);
          px[j * (CH / 2)] = close<T>(ox), pr[j * (CH / 2)] = close<T>(orr), pi[j * (CH / 2)] = close<T>(oi);
        }
      } else {
#pragma unroll
        for (int j = RW - 1; j >= 0; --j) {
          u64 ox = 0ull, orr = 0ull, oi = 0ull;
          if (t0 + j < job.L) gradients(j, ox, orr, oi);
          px[j * (CH / 2)] = close<T>(ox), pr[j * (CH / 2)] = close<T>(orr), pi[j * (CH / 2)] = close<T>(oi);
        }
      }
      total_of[w][lane] = sum;
    } else {
#pragma unroll
      for (int j = 0; j < RW; ++j) px[j * (CH / 2)] = pr[j * (CH / 2)] = pi[j * (CH / 2)] = R{};
    }
    __syncthreads();
    if (w == 0) {
      if (live) {
#pragma unroll
        for (int i = 1; i < WARPS; ++i) sum = add2(sum, total_of[i][lane]);
      }
      scatter(sums + rec, n, sum);
    }
    leave<T, UNIT, RW>(dx, own(stage, 0), a, job, t0);
    leave<T, UNIT, RW>(dr, own(stage, 1), a, job, t0);
    leave<T, UNIT, RW>(di, own(stage, 2), a, job, t0);
    __syncwarp();  // the rows are out before the next ones come in
    if (CHAIN && STAGES == 1) request(0, next);
    job = next;
  }
}

// dlam from the [n][C] sums of Q: 32 channels a block, 32 rows at a time, in a fixed order.
template <typename T>
__global__ void __launch_bounds__(1024) k_gated_lam(const float* sums, const T* lam, T* dlam, long n, int C) {
  __shared__ float red[32][33];
  grid_dep_enter();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
  float v = 0.f;
  if (c < C)
#pragma unroll 4
    for (long i = ty; i < n; i += 32) v += sums[i * C + c];
  red[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 32; ++i) v += red[i][tx];
    // sigmoid / softplus, which goes to one on the left: below -20 both are exp(lam) to fp32
    const float l = to_f(lam[c]), ratio = l < -20.f ? 1.f : 1.f / ((1.f + expf(-l)) * softplus(l));
    dlam[c] = from_f<T>(v * ratio);
  }
}

// One row a stream: h <- a h + beta g x, y = h.
template <typename T, bool PAIR>
__global__ void __launch_bounds__(256) k_gated_step(const Rows a, float* h, T* y) {
  grid_dep_enter();
  using R = typename Raw<T>::type;
  const long b = blockIdx.x / a.groups;  // groups of 512 channels here
  const int c = 2 * ((blockIdx.x % a.groups) * 256 + threadIdx.x), n = a.C - c;
  if (n <= 0) return;
  auto get = [&](const void* base, long ld) {
    const T* p = static_cast<const T*>(base) + b * ld + c;
    return open(PAIR ? *reinterpret_cast<const R*>(p) : gather(p, n));
  };
  float* hp = h + b * a.C + c;
  const u64 x = get(a.x, a.ldx), r = get(a.r, a.ldr), i = get(a.i, a.ldi);
  const float2 l = un(get(a.lam, 0));
  u64 st = PAIR ? *reinterpret_cast<const u64*>(hp) : gather(hp, n), s, g, av, beta;
  gates(r, i, pk(a.scale * softplus(l.x), a.scale * softplus(l.y)), s, g, av, beta);
  st = fma2(av, st, mul2(beta, mul2(g, x)));
  if (PAIR) {
    *reinterpret_cast<u64*>(hp) = st;
    *reinterpret_cast<R*>(y + b * a.C + c) = close<T>(st);
  } else {
    scatter(hp, n, st);
    scatter(y + b * a.C + c, n, close<T>(st));
  }
}

Rows rows(const void* x, const void* r, const void* i, const void* lam, const int* lengths, const GatedShape& s) {
  return Rows{x, r, i, lam, lengths, nullptr, s.ldx, s.ldr, s.ldi, s.B, s.N, s.C, (s.C + CH - 1) / CH, 0, s.scale};
}

// Rows, widths and strides in whole vectors of `bytes`.
bool whole(const Rows& a, int dtype, int bytes) {
  const uintptr_t low = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.r) | reinterpret_cast<uintptr_t>(a.i);
  return ((a.ldx | a.ldr | a.ldi | a.C) & (bytes / (dtype == 0 ? 4 : 2) - 1)) == 0 && low % bytes == 0;
}

int fwd_rows(int dtype) { return (dtype == 0 ? FWD<float> : FWD<bf16>)*WARPS; }
size_t entries(const GatedShape& s, int rows_) { return (size_t)((s.N + rows_ - 1) / rows_) * ((s.C + CH - 1) / CH) * s.B; }
size_t align16(size_t n) { return (n + 15) / 16 * 16; }
size_t padded(const GatedShape& s) { return (size_t)(s.C + CH - 1) / CH * CH; }
size_t chain_bytes(const GatedShape& s, size_t n) { return 4 * padded(s) + n * 96 * sizeof(u64); }
size_t records(const GatedShape& s) { return (size_t)s.B * ((s.N + KEEP - 1) / KEEP) * s.C; }

// The chain in a workspace, cleared by a launch of its own.
template <typename T>
cudaError_t chain(Chain& ch, Rows& a, char* ws, size_t n, const GatedShape& s, cudaStream_t st) {
  float* rate = reinterpret_cast<float*>(ws);
  a.rate = rate;
  ch.word = reinterpret_cast<u64*>(rate + padded(s));
  ch.err = status_word();
  const size_t most = std::max(48 * n, padded(s));
  const unsigned grid = static_cast<unsigned>(std::min<size_t>((most + 255) / 256, 8 * sm_count()));
  return launch_pdl(k_gated_start<T>, dim3(grid), dim3(256), 0, st, ch, static_cast<long>(n), rate, (const T*)a.lam, s.scale, s.C,
                    static_cast<int>(padded(s)));
}

// A kernel's dynamic shared memory, said once a device, and how many of its blocks an SM
// holds (no less than BLOCKS here; asked, because a cooperative launch of more is refused).
template <auto kernel>
cudaError_t room(size_t bytes, int* per_sm) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int n = dev < 64 ? known[dev].load(std::memory_order_acquire) : 0;
  if (n == 0) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes))) != cudaSuccess) return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, 32 * WARPS, bytes)) != cudaSuccess) return e;
    if (n < 1) return cudaErrorCooperativeLaunchTooLarge;
    if (dev < 64) known[dev].store(n, std::memory_order_release);
  }
  *per_sm = n;
  return cudaSuccess;
}

// A cooperative launch: all blocks run at once, or the launch fails.  A full grid takes every
// register of every SM: it starts once no other kernel is resident, and kernels of another
// stream run before or after it.  Blocks may start and
// ask for their first rows while k_gated_start, itself behind all that was queued before,
// still runs (27.5 us for 29.4 where tiles are few: fp32, 3 x 784 x 645, both directions).
template <auto kernel, typename... Act>
cudaError_t together(size_t tiles, size_t smem, cudaStream_t st, Act&&... args) {
  int per_sm = 0;
  const cudaError_t e = room<kernel>(smem, &per_sm);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<size_t>(tiles, (size_t)per_sm * sm_count())));
  cfg.blockDim = dim3(32 * WARPS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Act>(args)...);
}

template <typename T, int UNIT>
cudaError_t fwd(Rows a, float* h, float* kept, void* y, void* ws, const GatedShape& s, cudaStream_t st) {
  constexpr int ROWS = FWD<T> * WARPS;
  constexpr size_t stage = 3 * ROWS * CH * sizeof(T);
  a.tiles = (s.N + ROWS - 1) / ROWS;
  const size_t n = entries(s, ROWS);
  Chain ch{};
  cudaError_t e;
  if (a.tiles == 1) {  // an ordinary launch: nothing in this form of the kernel waits for the one before
    int per_sm;
    if ((e = room<k_gated_fwd<T, UNIT, false>>(stage, &per_sm)) != cudaSuccess) return e;
    k_gated_fwd<T, UNIT, false><<<static_cast<unsigned>(n), 32 * WARPS, stage, st>>>(a, ch, h, kept, (T*)y, static_cast<int>(n));
    return cudaGetLastError();
  }
  if ((e = chain<T>(ch, a, static_cast<char*>(ws), n, s, st)) != cudaSuccess) return e;
  return together<k_gated_fwd<T, UNIT, true>>(n, 2 * stage, st, a, ch, h, kept, (T*)y, static_cast<int>(n));
}

template <typename T, int UNIT>
cudaError_t bwd(Rows a, const float* kept, const void* dy, void* dx, void* dr, void* di, void* dlam, void* ws, const GatedShape& s,
                cudaStream_t st) {
  constexpr size_t stage = 4 * KEEP * CH * sizeof(T);
  a.tiles = (s.N + KEEP - 1) / KEEP;
  const size_t n = entries(s, KEEP);
  float* sums = static_cast<float*>(ws);
  Chain ch{};
  cudaError_t e;
  if (a.tiles == 1) {  // as forward
    int per_sm;
    if ((e = room<k_gated_bwd<T, UNIT, false>>(stage, &per_sm)) != cudaSuccess) return e;
    k_gated_bwd<T, UNIT, false><<<static_cast<unsigned>(n), 32 * WARPS, stage, st>>>(a, ch, (const T*)dy, kept, (T*)dx, (T*)dr, (T*)di, sums, static_cast<int>(n));
    e = cudaGetLastError();
  } else {
    if ((e = chain<T>(ch, a, static_cast<char*>(ws) + align16(4 * records(s)), n, s, st)) != cudaSuccess) return e;
    e = together<k_gated_bwd<T, UNIT, true>>(n, BACK_STAGES<T> * stage, st, a, ch, (const T*)dy, kept, (T*)dx, (T*)dr, (T*)di, sums,
                 static_cast<int>(n));
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(k_gated_lam<T>, dim3((s.C + 31) / 32), dim3(1024), 0, st, (const float*)sums, (const T*)a.lam, (T*)dlam,
                    (long)s.B * a.tiles, s.C);
}

template <typename T, bool PAIR>
cudaError_t step(Rows a, float* h, void* y, const GatedShape& s, cudaStream_t st) {
  a.groups = (s.C + 511) / 512;
  return launch_pdl(k_gated_step<T, PAIR>, dim3(a.groups * s.B), dim3(256), 0, st, a, h, (T*)y);
}

}  // namespace

size_t gated_kept_bytes(const GatedShape& s) { return 4 * records(s); }
size_t gated_ws_bytes(const GatedShape& s, bool bwd) {
  if (!bwd) return s.N > fwd_rows(s.dtype) ? chain_bytes(s, entries(s, fwd_rows(s.dtype))) : 0;
  return align16(4 * records(s)) + (s.N > KEEP ? chain_bytes(s, entries(s, KEEP)) : 0);
}

#define LA_GATED(f, ...)                                                               \
  (s.dtype == 0 ? whole(a, 0, 16) ? f<float, 16>(__VA_ARGS__) : f<float, 4>(__VA_ARGS__) \
   : whole(a, 1, 16) ? f<bf16, 16>(__VA_ARGS__)                                        \
   : whole(a, 1, 4)  ? f<bf16, 4>(__VA_ARGS__)                                         \
                     : f<bf16, 2>(__VA_ARGS__))

cudaError_t gated_fwd(const void* x, const void* r, const void* i, const void* lam, const int* lengths, float* h, float* kept, void* y,
                      void* ws, const GatedShape& s, cudaStream_t st) {
  const Rows a = rows(x, r, i, lam, lengths, s);
  return LA_GATED(fwd, a, h, kept, y, ws, s, st);
}
cudaError_t gated_bwd(const void* x, const void* r, const void* i, const void* lam, const int* lengths, const float* kept, const void* dy,
                      void* dx, void* dr, void* di, void* dlam, void* ws, const GatedShape& s, cudaStream_t st) {
  const Rows a = rows(x, r, i, lam, lengths, s);
  return LA_GATED(bwd, a, kept, dy, dx, dr, di, dlam, ws, s, st);
}
cudaError_t gated_step(const void* x, const void* r, const void* i, const void* lam, float* h, void* y, const GatedShape& s, cudaStream_t st) {
  const Rows a = rows(x, r, i, lam, nullptr, s);
  if (s.dtype == 0) return whole(a, 0, 8) ? step<float, true>(a, h, y, s, st) : step<float, false>(a, h, y, s, st);
  return whole(a, 1, 4) ? step<bf16, true>(a, h, y, s, st) : step<bf16, false>(a, h, y, s, st);
}
#undef LA_GATED

}  // namespace la
