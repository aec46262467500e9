// The selective scan on the 5th-generation tensor cores, for bf16 inputs with D
// and M in {16, 32, 64} (formulas: scan.cu).  Narrower heads ride in 64-wide
// tiles that the loads fill with zeros.
//
// Forward: chunks of 128 rows, three kernels.
//   k_sums   every chunk's own sum  F = sum_j B_j (w_j x_j)^T,
//            w_j = delta_j exp(cum_end - cum_j)
//   k_scan_carry (scan.cu)  the state before each chunk, fp32 recurrence, stored
//            in bf16 for the products that read it
//   k_out    y = P x + exp(cum) (C S_prev) + skip x,
//            P_ij = exp(cum_i - cum_j) delta_j (C_i . B_j)
// Every chunk is independent in the first and the last, so blocks need no order
// and three (k_sums) or two (k_out) share an SM: one block's loads and CUDA-core
// work cover the other's products.  A block takes one chunk and several heads of
// one group, whose B and C tiles it loads once.
// Gradients: k_sums in both directions at once, the carry of both, k_grad (one
// chunk a block again), and the sums over blocks.
//
// A chunk is one 128-row product tile.  Its states cost a head of 64 x 64 16 KB
// (fp32) and 8 KB (bf16; 16 for the gradients) written and read again, beside 32 KB
// of x and y; most of that stays in L2 for the next kernel.  Device time, L2
// flushed, 4 x 2048 rows, 32 heads of 64 x 64, 2 groups: forward 56 us (72 MB to
// read and write once: 10.6), with the final state 60, gradients 154 (110 MB: 16);
// of the gradients k_sums takes 39, the carry 22 and k_grad 90 in a profile with
// cold caches (forward: 24, 11, k_out 26).
//
// Decays: within 32 x 32 blocks off the diagonal exp(cum_i - cum_j) is a row
// factor times a column factor, both taken from the end of the column's block
// so that neither exceeds 1 (A <= 0); the diagonal blocks take one exponential
// a pair.  All exponentials are base 2, of fp32 sums.
//
// Roundings: P and the carried states to bf16 before their products (half a
// step, 2^-8, each on its own part of y), y once.  The chunk sums take w_j x_j
// as three bf16 terms (2^-24) where the final state, an fp32 output, is asked
// for, else as two (2^-16).
#include <cudaTypedefs.h>

#include "rows_map.cuh"
#include "scan.cuh"
#include "tc.cuh"
#include "tc_chunk.cuh"

namespace la {
namespace {

using namespace tc;
using namespace tcc;

constexpr int NT = 288;             // 8 compute warps, then the issuer's
constexpr int W_ISSUE = 8;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr int STILE = 64 * 64 * 2;  // one [64][64] bf16 state tile

// One chunk's gates of one head.  wp: prefix sums of log2 decays within each
// 32-row block; tot: the blocks' totals; del: delta; cf: delta exp(block end -
// cum); ew: exp(cum - block start).
struct __align__(16) Gates {
  float wp[128], del[128], cf[128], ew[128], tot[4];
  __device__ __forceinline__ float off(int q) const {  // log2 decay of the blocks before q
    return (q > 0 ? tot[0] : 0.f) + (q > 1 ? tot[1] : 0.f) + (q > 2 ? tot[2] : 0.f) + (q > 3 ? tot[3] : 0.f);
  }
  __device__ __forceinline__ float past(int q) const {  // of the blocks after q
    return (q < 3 ? tot[3] : 0.f) + (q < 2 ? tot[2] : 0.f) + (q < 1 ? tot[1] : 0.f);
  }
};

// A head's parameters, for all heads of a block.
constexpr int MAXH = 16;
struct Params {
  float A, skip, bias;
};

__device__ __forceinline__ float warp_suffix(float v) {  // inclusive, from the last lane
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float u = __shfl_down_sync(0xffffffffu, v, o);
    if (lane + o < 32) v += u;
  }
  return v;
}

// By four warps, row = 32 (warp mod 4) + lane.  ENDS: the log decay from a row to its block's
// end as a sum of its own; tot - wp keeps the roundings of two sums that may be large beside it
// (the state of a 2 x 4096-row prompt 1e-7 off instead of 3 to 12e-7, for 0.1 us of 59).
template <bool ENDS = false>
__device__ __forceinline__ void put_gates(Gates& g, float z, bool live, float A, int row) {
  const float d = live ? softplus(z) : 0.f;
  const float l = d * A * LOG2E;
  const float wp = warp_prefix(l);
  const float tot = __shfl_sync(0xffffffffu, wp, 31);
  float end = tot - wp;
  if (ENDS) {
    const float next = __shfl_down_sync(0xffffffffu, l, 1);
    end = warp_suffix((row & 31) == 31 ? 0.f : next);
  }
  g.wp[row] = wp;
  g.del[row] = d;
  g.cf[row] = d * ex2_fast(end);
  g.ew[row] = ex2_fast(wp);
  if ((row & 31) == 31) g.tot[row >> 5] = tot;
}

__device__ __forceinline__ void sync_compute() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Which rows and heads a block takes: chunk blockIdx.x, batch entry blockIdx.z,
// part p of group g's heads.
struct Share {
  int b, n0, rows, g, part, h0, nh;
  __device__ Share(const ScanShape& s, const int* lengths, int part_, int pg, int hs) {
    b = blockIdx.z;
    n0 = blockIdx.x * TC_C;
    rows = max(0, min(TC_C, valid_rows(lengths, b, s.N) - n0));
    part = part_;
    g = part / pg;
    const int hg = s.H / s.G, p = part % pg;
    h0 = g * hg + p * hs;
    nh = min(hs, hg - p * hs);
  }
  // The heads' parameters into shared memory, by threads 0 .. nh - 1 (before a block barrier).
  __device__ void params(Params* to, const bf16* A, const bf16* skip, const bf16* bias) const {
    const int i = threadIdx.x;
    if (i < nh) to[i] = Params{to_f(A[h0 + i]), par(skip, h0 + i), par(bias, h0 + i)};
  }
};

// Eight floats to a 32-byte boundary: a whole sector from one lane.
__device__ __forceinline__ void store8(float* o, const float* f) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(o), "r"(__float_as_uint(f[0])), "r"(__float_as_uint(f[1])),
               "r"(__float_as_uint(f[2])), "r"(__float_as_uint(f[3])), "r"(__float_as_uint(f[4])), "r"(__float_as_uint(f[5])),
               "r"(__float_as_uint(f[6])), "r"(__float_as_uint(f[7]))
               : "memory");
}

// Rows [rows, 128) of a swizzled [128][64] tile become zeros, by n threads.
__device__ __forceinline__ void clear_rows(uint8_t* tile, int rows, int n = 256) {
  for (int v = rows * 8 + threadIdx.x; v < TILE / 16; v += n) sts128(tile + v * 16, make_uint4(0u, 0u, 0u, 0u));
}

// The end of a block: its tensor memory is given back by the warp that took it.
__device__ __forceinline__ void leave(uint32_t tm, uint32_t cols, int issuer) {
  __syncthreads();
  tc_fence_after();
  if ((threadIdx.x >> 5) == issuer) tmem_dealloc(tm, cols);
}

#define LA_SCAN_WAITS()                                                     \
  auto wt = [&](uint64_t* bar, uint32_t parity, int code) -> bool {         \
    if (*reinterpret_cast<volatile int*>(&s_abort)) return false;           \
    if (mbar_wait(bar, parity, WAIT_NS)) return true;                       \
    *reinterpret_cast<volatile int*>(&s_abort) = 1;                         \
    fail(err, code);                                                        \
    return false;                                                           \
  };                                                                        \
  auto wtu = [&](uint64_t* bar, uint32_t parity, int code) -> bool {        \
    return __all_sync(0xffffffffu, wt(bar, parity, code));                  \
  };

struct Maps {
  CUtensorMap x, B, C, g;  // g: dy
  CUtensorMap o;           // y, or dx
  CUtensorMap S, R, Sl, Rl;  // the carried states, and what rounding them left
};

// ------------------------------------------------------------- chunk sums
// TERMS bf16 terms of the scaled operand: three where the state after the last
// row is wanted (an fp32 output: 2^-24), two for the states that products read
// in bf16 (one term would round them twice).  The first term takes x's
// place in shared memory and the third adds to the second's columns, so three
// blocks share an SM: one's load, another's conversion and a third's products
// overlap, and a head's own chain need not (two blocks of twice the buffers: 66 us
// for the 2 x 4096-row prompt, three 63; training 212 and 208).  The third term and
// the state: 4 us of 60.  Bound by latency and issue (46 % of cycles) as much as by its 67 MB of
// sums.  blockIdx.y = part, or parts + part
// for the reverse sums E = sum_i exp(cum_i) C_i dy_i^T.
constexpr int S_A = 0, S_T = TILE;  // B or C; the terms
constexpr int S_SMEM(int terms) { return (1 + terms) * TILE + 1024; }

template <int TERMS>
__global__ void __launch_bounds__(NT, 3)
    k_sums(const __grid_constant__ Maps maps, const bf16* __restrict__ dt, const bf16* __restrict__ A,
           const bf16* __restrict__ bias, const int* __restrict__ lengths, float* __restrict__ fwd, float* __restrict__ rev,
           float* __restrict__ tot, ScanShape s, int pg, int hs, int* err) {
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = align1024(smraw);
  __shared__ uint64_t bar_a, bar_x, bar_t, bar_m;
  __shared__ Gates gates[2];
  __shared__ Params par_[MAXH];
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;
  constexpr int COLS = 128;
  const int parts = s.G * pg;
  const bool back = blockIdx.y >= parts;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nch = gridDim.x;
  if (threadIdx.x == NT - 1) {
    mbar_init(&bar_a, 1);
    mbar_init(&bar_x, 1);
    mbar_init(&bar_t, 256);
    mbar_init(&bar_m, 1);
    fence_barrier_init();
    s_abort = 0;
  }
  enter(&tmem_base, COLS, warp == W_ISSUE);
  const Share w(s, lengths, back ? blockIdx.y - parts : blockIdx.y, pg, hs);
  const int DM = s.D * s.M;
  float* out = (back ? rev : fwd) + (((long)w.b * s.H + w.h0) * nch + blockIdx.x) * DM;  // head h0 + i: + i nch DM
  w.params(par_, A, nullptr, bias);
  LA_SCAN_WAITS()
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;

  if (w.rows == 0) {
    for (int i = 0; i < w.nh; ++i) {
      for (int e = threadIdx.x * 4; e < DM; e += NT * 4) *reinterpret_cast<float4*>(out + (long)i * nch * DM + e) = make_float4(0.f, 0.f, 0.f, 0.f);
      if (threadIdx.x == 0 && !back) tot[((long)w.b * s.H + w.h0 + i) * nch + blockIdx.x] = 0.f;
    }
    leave(tmem_base, COLS, W_ISSUE);
    return;
  }
  if (warp == W_ISSUE) {
    if (lane == 0) {
      const CUtensorMap* mx = back ? &maps.g : &maps.x;
      auto load = [&](int i) {
        mbar_arrive_expect_tx(&bar_x, TILE);
        tma_load_4d(sm + S_T, mx, &bar_x, 0, w.h0 + i, w.n0, w.b);
      };
      load(0);
      mbar_arrive_expect_tx(&bar_a, TILE);
      tma_load_4d(sm + S_A, back ? &maps.C : &maps.B, &bar_a, 0, w.g, w.n0, w.b);
      constexpr uint32_t ID = idesc_bf16(64, COLS, true, true), ID1 = idesc_bf16(64, 64, true, true);
      const uint64_t da = sdesc(smem_u32(sm + S_A), 16, 1024), db = sdesc(smem_u32(sm + S_T), TILE, 1024);
      int loads = 1;
      bool ok = wt(&bar_a, 0, 66);
      for (int i = 0; ok && i < w.nh; ++i) {
        if (!(ok = wt(&bar_t, i & 1, 61))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mma_bf16(tm, dadd(da, kk * 2048), dadd(db, kk * 2048), ID, kk > 0);
        if (TERMS > 2)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) mma_bf16(tm + 64, dadd(da, kk * 2048), dadd(db, 2 * TILE + kk * 2048), ID1, 1);
        mma_commit(&bar_m);
        if (i + 1 < w.nh) {
          if (!(ok = wt(&bar_m, i & 1, 67))) break;  // the terms have been read
          load(i + 1);
          ++loads;
        }
      }
      // nothing in flight at exit
      mbar_wait(&bar_x, (loads - 1) & 1, WAIT_NS);
      mbar_wait(&bar_a, 0, WAIT_NS);
      mma_commit(&bar_a);
      mbar_wait(&bar_a, 1, WAIT_NS);
    }
  } else {
    const int row = threadIdx.x & 127, half = threadIdx.x >> 7, q = row >> 5;
    const long r0 = (long)w.b * s.N + w.n0;
    auto raw = [&](int i) { return i < w.nh && row < w.rows ? to_f(dt[(r0 + row) * s.lddt + w.h0 + i]) : 0.f; };
    const int qd = warp & 3, srow = 16 * qd + lane;
    const uint32_t lq = static_cast<uint32_t>(32 * qd) << 16;
    float z = 0.f;
    if (half == 0) {
      put_gates<(TERMS > 2)>(gates[0], raw(0) + par_[0].bias, row < w.rows, par_[0].A, row);
      z = raw(1);
    }
    if (w.rows < min(TC_C, s.N - w.n0)) {  // rows past the sequence's length: not to be multiplied
      if (wtu(&bar_a, 0, 63)) clear_rows(sm + S_A, w.rows);
    }
    sync_compute();
    for (int i = 0; i < w.nh; ++i) {
      const Gates& g = gates[i & 1];
      if (threadIdx.x == 0 && !back) tot[((long)w.b * s.H + w.h0 + i) * nch + blockIdx.x] = g.off(4) * LN2;
      const bool live = row < w.rows;
      const float f = !live ? 0.f : (back ? ex2_fast(g.wp[row] + g.off(q)) : g.cf[row] * ex2_fast(g.past(q)));
      if (wtu(&bar_x, i & 1, 64)) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint8_t* at = sm + S_T + row * 128 + (((4 * half + c) ^ (row & 7)) << 4);
          const uint4 u = lds128(at);
          // a row past the length enters as zeros, whatever it holds (one weighed by 0 does not: its NaN counts)
          const uint32_t v[4] = {live ? u.x : 0u, live ? u.y : 0u, live ? u.z : 0u, live ? u.w : 0u};
          uint32_t t[TERMS][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float a = __uint_as_float(v[k] << 16) * f, b = __uint_as_float(v[k] & 0xffff0000u) * f;
#pragma unroll
            for (int j = 0; j < TERMS; ++j) {
              t[j][k] = pack_bf16(a, b);
              a -= __uint_as_float(t[j][k] << 16);
              b -= __uint_as_float(t[j][k] & 0xffff0000u);
            }
          }
#pragma unroll
          for (int j = 0; j < TERMS; ++j) sts128(at + j * TILE, make_uint4(t[j][0], t[j][1], t[j][2], t[j][3]));
        }
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_t);
      if (half == 0 && i + 1 < w.nh) {  // the next head's gates, beside this one's products
        put_gates<(TERMS > 2)>(gates[(i + 1) & 1], z + par_[i + 1].bias, row < w.rows, par_[i + 1].A, row);
        z = raw(i + 2);
      }
      if (wtu(&bar_m, i & 1, 62)) {  // the sums, and the next head's rows on their way
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float p[16], r[16];
          tmem_ld16(tm + lq + 32 * half + 16 * j, p);
          tmem_ld16(tm + lq + 64 + 32 * half + 16 * j, r);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 16; ++c) p[c] += r[c];
          const int c0 = 32 * half + 16 * j;
          if (lane < 16 && srow < s.D && c0 < s.M) {
            float* o = out + (long)i * nch * DM + srow * s.M + c0;
#pragma unroll
            for (int c = 0; c < 16; c += 8) store8(o + c, p + c);
          }
        }
      }
      sync_compute();
    }
    tc_fence_before();
  }
  leave(tm, COLS, W_ISSUE);
}

// ------------------------------------------------------------------ outputs
// A head's chain is scores, weights, P x, read-out; the next head's scores are
// issued during the read-out and a second block fills the rest.  26 us for 256
// blocks of 8 heads (55 MB read, 34 written: 2.4 times HBM's time); tensor pipe
// 21 %, issue 43 %.
constexpr int O_C = 0, O_B = TILE, O_X = 2 * TILE, O_S = 4 * TILE;  // C, B, two x stages, two state stages
constexpr int O_SMEM = 4 * TILE + 2 * STILE + 1024;
constexpr uint32_t T_A = 0, T_O = 128, T_CS = 192;  // scores (then P in place), P x, C S

__global__ void __launch_bounds__(NT, 2)
    k_out(const __grid_constant__ Maps maps, const bf16* __restrict__ dt, const bf16* __restrict__ A,
          const bf16* __restrict__ skip, const bf16* __restrict__ bias, const int* __restrict__ lengths, bf16* __restrict__ y,
          ScanShape s, int pg, int hs, int states, int* err) {
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = align1024(smraw);
  __shared__ uint64_t bar_cb, bar_x[2], bar_a, bar_p, bar_o, bar_free;
  __shared__ Gates gates[2];
  __shared__ Params par_[MAXH];
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nch = gridDim.x;
  if (threadIdx.x == NT - 1) {
    mbar_init(&bar_cb, 1);
    mbar_init(&bar_x[0], 1);
    mbar_init(&bar_x[1], 1);
    mbar_init(&bar_a, 1);
    mbar_init(&bar_p, 256);
    mbar_init(&bar_o, 1);
    mbar_init(&bar_free, 256);
    fence_barrier_init();
    s_abort = 0;
  }
  enter(&tmem_base, 256, warp == W_ISSUE);
  const Share w(s, lengths, blockIdx.y, pg, hs);
  const long r0 = (long)w.b * s.N + w.n0;
  w.params(par_, A, skip, bias);
  LA_SCAN_WAITS()
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;

  if (w.rows == 0) {  // nothing but rows past the sequence's length
    const int n = min(TC_C, s.N - w.n0), per = w.nh * s.M / 8;
    for (int e = threadIdx.x; e < n * per; e += NT)
      *reinterpret_cast<uint4*>(y + ((r0 + e / per) * s.H + w.h0) * s.M + e % per * 8) = make_uint4(0u, 0u, 0u, 0u);
    leave(tmem_base, 256, W_ISSUE);
    return;
  }
  if (warp == W_ISSUE) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&bar_cb, 2 * TILE);
      tma_load_4d(sm + O_C, &maps.C, &bar_cb, 0, w.g, w.n0, w.b);
      tma_load_4d(sm + O_B, &maps.B, &bar_cb, 0, w.g, w.n0, w.b);
      int issued = 0;
      auto load = [&](int i) {
        const int k = i & 1, h = w.h0 + i;
        mbar_arrive_expect_tx(&bar_x[k], TILE + (states ? STILE : 0));
        tma_load_4d(sm + O_X + k * TILE, &maps.x, &bar_x[k], 0, h, w.n0, w.b);
        if (states) tma_load_3d(sm + O_S + k * STILE, &maps.S, &bar_x[k], 0, 0, (w.b * s.H + h) * nch + blockIdx.x);
        ++issued;
      };
      load(0);
      if (w.nh > 1) load(1);
      constexpr uint32_t ID_A = idesc_bf16(128, 128, false, false), ID_O = idesc_bf16(128, 64, false, true);
      const uint64_t dC = sdesc(smem_u32(sm + O_C), 16, 1024), dB = sdesc(smem_u32(sm + O_B), 16, 1024);
      // The scores of head i + 1 go out as soon as P of head i has been read, beside
      // the outputs' read-out; bar_o's commit covers C S as well.
      auto scores = [&](int i) {
        if (!wt(&bar_x[i & 1], (i >> 1) & 1, 72)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_bf16(tm + T_A, dadd(dC, 32 * kk), dadd(dB, 32 * kk), ID_A, kk > 0);
        mma_commit(&bar_a);
        return true;
      };
      bool ok = wt(&bar_cb, 0, 71) && scores(0);
      for (int i = 0; ok && i < w.nh; ++i) {
        const int k = i & 1;
        const uint64_t dX = sdesc(smem_u32(sm + O_X + k * TILE), 16, 1024), dS = sdesc(smem_u32(sm + O_S + k * STILE), 16, 1024);
        if (states)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_bf16(tm + T_CS, dadd(dC, 32 * kk), dadd(dS, kk * 2048), ID_O, kk > 0);
        if (!(ok = wt(&bar_p, k, 73))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_bf16_ts(tm + T_O, tm + T_A + (kk < 4 ? 8 * kk : 32 + 8 * kk), dadd(dX, kk * 2048), ID_O, kk > 0);
        mma_commit(&bar_o);
        if (i + 1 < w.nh && !(ok = wt(&bar_o, k, 79) && scores(i + 1))) break;
        if (!(ok = wt(&bar_free, k, 74))) break;
        tc_fence_after();
        tma_store_4d(&maps.o, sm + O_X + k * TILE, 0, w.h0 + i, w.n0, w.b);  // y has taken x's place
        bulk_commit();
        if (i + 2 < w.nh) {
          bulk_wait_read();
          load(i + 2);
        }
      }
      // nothing in flight at exit: the products' last commit, loads, stores
      mma_commit(&bar_cb);
      mbar_wait(&bar_cb, 1, WAIT_NS);
      drain_loads<2>(bar_x, issued);
      bulk_wait_all();
    }
  } else {
    const int qd = warp & 3, wg = warp >> 2, row = 32 * qd + lane;
    const uint32_t lq = static_cast<uint32_t>(32 * qd) << 16;
    auto raw = [&](int i) { return i < w.nh && row < w.rows ? to_f(dt[(r0 + row) * s.lddt + w.h0 + i]) : 0.f; };
    float z = 0.f;
    if (wg == 0) {
      put_gates(gates[0], raw(0) + par_[0].bias, row < w.rows, par_[0].A, row);
      z = raw(1);
    }
    sync_compute();
    const bool cut = w.rows < min(TC_C, s.N - w.n0);
    for (int i = 0; i < w.nh; ++i) {
      const int k = i & 1;
      const Gates& g = gates[k];
      uint8_t* xt = sm + O_X + k * TILE;
      const float wp = g.wp[row], here = g.off(qd);
      if (cut && wtu(&bar_x[k], (i >> 1) & 1, 75)) clear_rows(xt, w.rows);
      if (wtu(&bar_a, k, 76)) {
        tc_fence_after();
        const uint32_t ta = tm + T_A + 64 * wg + lq;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int J = 2 * wg + j;  // a block of 32 columns
          uint32_t pk[16];
          if (J > qd) {
#pragma unroll
            for (int c = 0; c < 16; ++c) pk[c] = 0u;
          } else {
            float a[32];
            tmem_ldn<2>(ta + 32 * j, a);
            if (J < qd) {
              const float f = ex2_fast(wp + here - g.off(J + 1));
#pragma unroll
              for (int c = 0; c < 32; c += 4) {
                const float4 u = *reinterpret_cast<const float4*>(&g.cf[32 * J + c]);
                pk[c / 2] = pack_bf16(a[c] * (f * u.x), a[c + 1] * (f * u.y));
                pk[c / 2 + 1] = pack_bf16(a[c + 2] * (f * u.z), a[c + 3] * (f * u.w));
              }
            } else {
#pragma unroll
              for (int c = 0; c < 32; c += 4) {
                const float4 u = *reinterpret_cast<const float4*>(&g.wp[32 * J + c]), d = *reinterpret_cast<const float4*>(&g.del[32 * J + c]);
                // taken for masked pairs too (an overflow or NaN there goes with them) and
                // dropped by a select, not a branch
                float p0 = a[c] * (ex2_fast(wp - u.x) * d.x), p1 = a[c + 1] * (ex2_fast(wp - u.y) * d.y);
                float p2 = a[c + 2] * (ex2_fast(wp - u.z) * d.z), p3 = a[c + 3] * (ex2_fast(wp - u.w) * d.w);
                p0 = c <= lane ? p0 : 0.f, p1 = c + 1 <= lane ? p1 : 0.f;
                p2 = c + 2 <= lane ? p2 : 0.f, p3 = c + 3 <= lane ? p3 : 0.f;
                pk[c / 2] = pack_bf16(p0, p1);
                pk[c / 2 + 1] = pack_bf16(p2, p3);
              }
            }
          }
          tmem_st16u(ta + 16 * j, pk);  // over columns this warp has read
        }
        tmem_st_wait();
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_p);
      if (wg == 0 && i + 1 < w.nh) {  // the next head's gates, beside this one's products
        put_gates(gates[k ^ 1], z + par_[i + 1].bias, row < w.rows, par_[i + 1].A, row);
        z = raw(i + 2);
      }
      const float e = ex2_fast(wp + here), sk = par_[i].skip;
      const bool x_in = wtu(&bar_x[k], (i >> 1) & 1, 77), live = row < w.rows;
      if (wtu(&bar_o, k, 78) && x_in) {
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c0 = 32 * wg + 16 * j;
          float o[16], cs[16], x[16];
          tmem_ld16(tm + T_O + c0 + lq, o);
          if (states) tmem_ld16(tm + T_CS + c0 + lq, cs);
          tile_row_cols<16>(xt, row, c0, x);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float v = fmaf(sk, x[c], states ? fmaf(e, cs[c], o[c]) : o[c]);
            o[c] = live ? v : 0.f;
          }
          tile_put_cols<16>(xt, row, c0, o);
        }
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_free);
      sync_compute();  // the next head's gates are in place
    }
  }
  leave(tm, 256, W_ISSUE);
}

// ---------------------------------------------------------------- gradients
// One chunk, several heads of one group in turn.  Rows of the score tiles are
// the keys j, so that P^T and Q^T serve from tensor memory as A operands:
//   A^T = B C^T, E^T = x dy^T;  P_ij = W_ij A_ij, Q_ij = W_ij delta_j E_ij
//   du = P^T dy + f_j (B R),        f_j = exp(cum_end - cum_j)
//   dB += Q^T C + delta_j f_j (x R^T),  dC += Q B + exp(cum_i) (dy S^T)
// The carried states enter in two bf16 terms, so that what the gate's gradient is
// summed from (pair sums, x . (B R), C . (S dy), <S, R>) is accurate to 2^-16 and
// its sums over all rows, dA and ddt_bias, keep their digits where they cancel;
// x . du is the pair sum and x . (B R), without the rounded P of dx.
// dB and dC are summed over the block's heads in registers (fp32); a group's
// blocks leave fp32 partial sums that scan_groups adds up (one block: the
// gradients themselves).  The gate's gradient takes its pair sums G_ij =
// Q_ij A_ij from the fp32 scores in registers: the column sums of a 32 x 32 block
// cost 32 shuffles a warp.
//
// Sixteen compute warps, one 32 x 32 score block each (warp mod 4 is the lane
// quarter it can reach, warp / 4 the block's column), on one block an SM (all
// 512 tensor-memory columns, 193 KB of tiles).  The next head's gates and the
// last head's gate gradient are formed beside the products, the latter by the
// warps that the masked triangle leaves idle.  90 us for 128 blocks of 16 heads,
// 5.6 us a head: bound by the per-head chain and by instruction issue (50 % of
// cycles), not by a unit's rate (tensor pipe 20 %, HBM 25 %).  Column sums deferred
// past the products took 218 us and more for the training pass, a compute warp that
// also issues 229, where this took 212: they spill.
constexpr int GT = 512, NTG = GT + 32, WG_ISSUE = GT / 32;
constexpr int G_C = 0, G_B = TILE, G_X = 2 * TILE, G_Y = 4 * TILE, G_S = 6 * TILE, G_R = G_S + 4 * STILE, G_Q = G_R + 4 * STILE;
// (a stage of S or R is two tiles, its terms)
constexpr int G_SMEM = G_Q + 2 * TILE + 1024;
constexpr uint32_t TG_A = 0, TG_E = 128, TG_U = 256, TG_BR = 320, TG_B = 384, TG_C = 448;

__device__ __forceinline__ void sync_grad() { asm volatile("bar.sync 1, 512;" ::: "memory"); }

// Sum over the warp's lanes of g[c] for each of 8 columns c, to lanes c, c + 8, ... .
__device__ __forceinline__ float column_sums(float (&g)[8], int lane) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int c = 0; c < o; ++c) {
      const float keep = up ? g[c + o] : g[c], give = up ? g[c] : g[c + o];
      g[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  g[0] += __shfl_xor_sync(0xffffffffu, g[0], 8);
  return g[0] + __shfl_xor_sync(0xffffffffu, g[0], 16);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What the gate's gradient of a head is summed from, by row (and by the column
// group that formed it).
struct GateSums {
  float row[4][128], col[4][128], self[128], v[4][128], w[4][128], red[16][2];
};

__global__ void __launch_bounds__(NTG, 1)
    k_grad(const __grid_constant__ Maps maps, const bf16* __restrict__ dt, const bf16* __restrict__ A,
           const bf16* __restrict__ skip, const bf16* __restrict__ bias, const int* __restrict__ lengths,
           bf16* __restrict__ dx, bf16* __restrict__ ddt, void* dB, void* dC, float* __restrict__ pp, ScanShape s, int pg,
           int hs, int states, int* err) {
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = align1024(smraw);
  __shared__ uint64_t bar_cb, bar_in[2], bar_clear, bar_1, bar_2, bar_3, bar_4, bar_p, bar_c, bar_x, bar_free;
  __shared__ Gates gates[3];
  __shared__ Params par_[MAXH];
  __shared__ GateSums sums[2];
  __shared__ float s_tot[4][2], s_out[4][2];
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nch = gridDim.x;
  const bool direct = pg == 1;  // dB and dC themselves, else partial sums
  const int parts = s.G * pg;
  if (threadIdx.x == GT) {
    for (uint64_t* b : {&bar_cb, &bar_in[0], &bar_in[1], &bar_1, &bar_2, &bar_3, &bar_4}) mbar_init(b, 1);
    for (uint64_t* b : {&bar_clear, &bar_p, &bar_c, &bar_x, &bar_free}) mbar_init(b, GT);
    fence_barrier_init();
    s_abort = 0;
  }
  enter(&tmem_base, 512, warp == WG_ISSUE);
  const Share w(s, lengths, blockIdx.y, pg, hs);
  const long r0 = (long)w.b * s.N + w.n0;
  const int in_n = min(TC_C, s.N - w.n0);  // rows of the chunk that exist
  w.params(par_, A, skip, bias);
  LA_SCAN_WAITS()
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;
  const bool cut = w.rows < in_n;
  if (!states) {  // one chunk: the carried states are zeros, in every stage
    for (int v = threadIdx.x; v < 8 * STILE / 16; v += NTG) sts128(sm + G_S + v * 16, make_uint4(0u, 0u, 0u, 0u));
    fence_proxy_async();
    __syncthreads();
  }

  if (w.rows == 0) {  // nothing but rows past the sequence's length
    const int per = w.nh * s.M / 8;
    for (int e = threadIdx.x; e < in_n * per; e += NTG)
      *reinterpret_cast<uint4*>(dx + ((r0 + e / per) * s.H + w.h0) * s.M + e % per * 8) = make_uint4(0u, 0u, 0u, 0u);
    for (int e = threadIdx.x; e < in_n * w.nh; e += NTG) ddt[(r0 + e / w.nh) * s.H + w.h0 + e % w.nh] = from_f<bf16>(0.f);
    for (int e = threadIdx.x; e < in_n * s.D; e += NTG) {
      const long o = ((r0 + e / s.D) * parts + w.part) * s.D + e % s.D;
      if (direct) {
        static_cast<bf16*>(dB)[o] = from_f<bf16>(0.f);
        static_cast<bf16*>(dC)[o] = from_f<bf16>(0.f);
      } else {
        static_cast<float*>(dB)[o] = 0.f;
        static_cast<float*>(dC)[o] = 0.f;
      }
    }
    for (int e = threadIdx.x; e < w.nh * 3; e += NTG) pp[(((long)w.b * s.H + w.h0 + e / 3) * nch + blockIdx.x) * 3 + e % 3] = 0.f;
    leave(tmem_base, 512, WG_ISSUE);
    return;
  }
  if (warp == WG_ISSUE) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&bar_cb, 2 * TILE);
      tma_load_4d(sm + G_C, &maps.C, &bar_cb, 0, w.g, w.n0, w.b);
      tma_load_4d(sm + G_B, &maps.B, &bar_cb, 0, w.g, w.n0, w.b);
      int issued = 0;
      auto load = [&](int i) {
        const int k = i & 1, h = w.h0 + i;
        mbar_arrive_expect_tx(&bar_in[k], 2 * TILE + (states ? 4 * STILE : 0));
        tma_load_4d(sm + G_X + k * TILE, &maps.x, &bar_in[k], 0, h, w.n0, w.b);
        tma_load_4d(sm + G_Y + k * TILE, &maps.g, &bar_in[k], 0, h, w.n0, w.b);
        ++issued;
        if (!states) return;
        const int at = (w.b * s.H + h) * nch + blockIdx.x;
        tma_load_3d(sm + G_S + 2 * k * STILE, &maps.S, &bar_in[k], 0, 0, at);
        tma_load_3d(sm + G_S + (2 * k + 1) * STILE, &maps.Sl, &bar_in[k], 0, 0, at);
        tma_load_3d(sm + G_R + 2 * k * STILE, &maps.R, &bar_in[k], 0, 0, at);
        tma_load_3d(sm + G_R + (2 * k + 1) * STILE, &maps.Rl, &bar_in[k], 0, 0, at);
      };
      load(0);
      if (w.nh > 1) load(1);
      constexpr uint32_t ID_A = idesc_bf16(128, 128, false, false), ID_KM = idesc_bf16(128, 64, false, true),
                         ID_KK = idesc_bf16(128, 64, false, false), ID_MM = idesc_bf16(128, 64, true, true);
      const uint64_t dCt = sdesc(smem_u32(sm + G_C), 16, 1024), dBt = sdesc(smem_u32(sm + G_B), 16, 1024);
      const uint64_t dQ = sdesc(smem_u32(sm + G_Q), TILE, 1024);
      bool ok = wt(&bar_cb, 0, 81);
      for (int i = 0; ok && i < w.nh; ++i) {
        const int k = i & 1;
        const uint64_t dX = sdesc(smem_u32(sm + G_X + k * TILE), 16, 1024), dY = sdesc(smem_u32(sm + G_Y + k * TILE), 16, 1024);
        const uint64_t dS = sdesc(smem_u32(sm + G_S + 2 * k * STILE), 16, 1024), dR = sdesc(smem_u32(sm + G_R + 2 * k * STILE), 16, 1024);
        if (!(ok = wt(&bar_in[k], (i >> 1) & 1, 82) && (!cut || wt(&bar_clear, k, 83)))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_bf16(tm + TG_A, dadd(dBt, 32 * kk), dadd(dCt, 32 * kk), ID_A, kk > 0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_bf16(tm + TG_E, dadd(dX, 32 * kk), dadd(dY, 32 * kk), ID_A, kk > 0);
        mma_commit(&bar_1);
        if (i > 0 && !(ok = wt(&bar_free, (i - 1) & 1, 84))) break;  // the last head's accumulators have been read
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 2; ++j)  // either term of the states
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            mma_bf16(tm + TG_B, dadd(dX, 32 * kk), dadd(dR, j * STILE + 32 * kk), ID_KK, j > 0 || kk > 0);
            mma_bf16(tm + TG_C, dadd(dY, 32 * kk), dadd(dS, j * STILE + 32 * kk), ID_KK, j > 0 || kk > 0);
            mma_bf16(tm + TG_BR, dadd(dBt, 32 * kk), dadd(dR, j * STILE + kk * 2048), ID_KM, j > 0 || kk > 0);
          }
        mma_commit(&bar_2);
        if (!(ok = wt(&bar_p, k, 85))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // P^T dy
          mma_bf16_ts(tm + TG_U, tm + TG_A + 32 * (kk >> 1) + 8 * (kk & 1), dadd(dY, kk * 2048), ID_KM, kk > 0);
        mma_commit(&bar_3);
        if (!(ok = wt(&bar_c, k, 86))) break;  // x R^T and dy S^T have been read
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // Q^T C
          mma_bf16_ts(tm + TG_B, tm + TG_E + 32 * (kk >> 1) + 8 * (kk & 1), dadd(dCt, kk * 2048), ID_KM, kk > 0);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // Q B
          mma_bf16(tm + TG_C, dadd(dQ, kk * 2048), dadd(dBt, kk * 2048), ID_MM, kk > 0);
        mma_commit(&bar_4);
        if (!(ok = wt(&bar_x, k, 87))) break;
        tma_store_4d(&maps.o, sm + G_X + k * TILE, 0, w.h0 + i, w.n0, w.b);  // dx has taken x's place
        bulk_commit();
        if (!(ok = wt(&bar_4, k, 88))) break;
        if (i + 2 < w.nh) {
          bulk_wait_read();
          load(i + 2);
        }
      }
      mma_commit(&bar_cb);
      mbar_wait(&bar_cb, 1, WAIT_NS);
      drain_loads<2>(bar_in, issued);
      bulk_wait_all();
    }
  } else {
    const int qd = warp & 3, I = warp >> 2, row = 32 * qd + lane, c0 = 16 * I;
    const uint32_t lq = static_cast<uint32_t>(32 * qd) << 16;
    const bool live = row < w.rows;
    auto raw = [&](int i) { return i < w.nh && live ? to_f(dt[(r0 + row) * s.lddt + w.h0 + i]) : 0.f; };
    float z = 0.f;
    if (I == 1) {
      put_gates(gates[0], raw(0) + par_[0].bias, live, par_[0].A, row);
      z = raw(1);
    }
    // The gate's gradient of head i, row by row (sigmoid(z) = 1 - exp(-delta)), by four
    // warps whose score block the mask leaves empty, beside the next head's weights.
    const int gw = warp == 7 ? 3 : warp - 1;  // warps 1, 2, 3 and 7
    const bool gater = warp == 7 || (warp >= 1 && warp <= 3);
    auto gate_gradient = [&](int i) {
      const Gates& g = gates[i % 3];
      const GateSums& gs = sums[i & 1];
      const int t = 32 * gw + lane;
      const float del = g.del[t];
      float q = 0.f, ww = 0.f, col = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        q += gs.v[j][t] + gs.row[j][t];
        ww += gs.w[j][t];  // x_j . (B_j R) f_j
        col += gs.col[j][t];
      }
      q -= del * col;
      const float xu = col + gs.self[t] + ww;  // x_j . du_j: no rounded P in it
      ww *= del;
      const float sr = warp_sum(lane < 16 ? gs.red[lane][0] : 0.f);
      const float suf = warp_suffix(q), pre = warp_prefix(ww);
      if (lane == 0) s_tot[gw][0] = suf;
      if (lane == 31) s_tot[gw][1] = pre;
      asm volatile("bar.sync 2, 128;" ::: "memory");
      float dl = suf + (pre - ww);
      for (int j = gw + 1; j < 4; ++j) dl += s_tot[j][0];
      for (int j = 0; j < gw; ++j) dl += s_tot[j][1];
      dl = fmaf(ex2_fast(g.off(4)), sr, dl);
      const float dz = t < w.rows ? (xu + par_[i].A * dl) * -expm1f(-del) : 0.f;
      if (t < in_n) ddt[(r0 + t) * s.H + w.h0 + i] = from_f<bf16>(dz);
      const float dA = warp_sum(t < w.rows ? del * dl : 0.f), db = warp_sum(dz);
      if (lane == 0) s_out[gw][0] = dA, s_out[gw][1] = db;
      asm volatile("bar.sync 2, 128;" ::: "memory");
      if (gw == 0) {
        const float ds = warp_sum(lane < 16 ? gs.red[lane][1] : 0.f);
        if (lane == 0) {
          float* o = pp + (((long)w.b * s.H + w.h0 + i) * nch + blockIdx.x) * 3;
          o[0] = s_out[0][0] + s_out[1][0] + s_out[2][0] + s_out[3][0];
          o[1] = ds;
          o[2] = s_out[0][1] + s_out[1][1] + s_out[2][1] + s_out[3][1];
        }
      }
    };
    float aB[16], aC[16];  // dB and dC of this row, columns c0 .. c0 + 15, over the heads
#pragma unroll
    for (int c = 0; c < 16; ++c) aB[c] = aC[c] = 0.f;
    const bool cb = wtu(&bar_cb, 0, 89);
    sync_grad();
    for (int i = 0; i < w.nh; ++i) {
      const int k = i & 1;
      const Gates& g = gates[i % 3];
      GateSums& gs = sums[k];
      uint8_t *xt = sm + G_X + k * TILE, *yt = sm + G_Y + k * TILE;
      const bool in = wtu(&bar_in[k], (i >> 1) & 1, 90) && cb;
      if (cut) {
        if (in) {
          if (i == 0) {
            clear_rows(sm + G_C, w.rows, GT);
            clear_rows(sm + G_B, w.rows, GT);
          }
          clear_rows(xt, w.rows, GT);
          clear_rows(yt, w.rows, GT);
        }
        fence_proxy_async();
        mbar_arrive(&bar_clear);
      }
      const float wp = g.wp[row], del = g.del[row];
      const float tail = ex2_fast(g.tot[qd] - wp);     // from this row to its block's end
      const float fend = tail * ex2_fast(g.past(qd));  // to the chunk's end
      const float ecum = g.ew[row] * ex2_fast(g.off(qd));
      // ---- the weights on this warp's block of A^T and E^T: keys 32 qd + lane, queries 32 I + c
      if (wtu(&bar_1, k, 91)) {
        tc_fence_after();
        const uint32_t ta = tm + TG_A + 32 * I + lq, te = tm + TG_E + 32 * I + lq;
        uint8_t* qt = sm + G_Q + (I >> 1) * TILE + row * 128;
        const float fr = I > qd ? tail * ex2_fast(g.off(I) - g.off(qd + 1)) : 0.f;
        float col = 0.f, self = 0.f;  // sums over this key's pairs, without delta
#pragma unroll
        for (int o = 0; o < 4; ++o) {  // eight queries at a time
          uint32_t pw[4], qw[4];
          if (I < qd) {
#pragma unroll
            for (int c = 0; c < 4; ++c) pw[c] = qw[c] = 0u;
          } else {
            float a[8], e[8], gg[8];
            tmem_ld8(ta + 8 * o, a);
            tmem_ld8(te + 8 * o, e);
            tmem_ld_wait();
            const float4* tab = reinterpret_cast<const float4*>((I > qd ? g.ew : g.wp) + 32 * I + 8 * o);
            const float4 t0 = tab[0], t1 = tab[1];
            float tv[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
            if (I > qd) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float wt_ = tv[c] * fr;
                e[c] *= wt_;
                gg[c] = e[c] * a[c];
                e[c] *= del;
                a[c] *= wt_;
              }
            } else {
              // (the exponential of a masked pair is dropped by a select: branches around
              // them, pair by pair, took most of this stage)
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                float wt_ = ex2_fast(tv[c] - wp);
                wt_ = 8 * o + c >= lane ? wt_ : 0.f;
                e[c] *= wt_;
                gg[c] = e[c] * a[c];
                if (8 * o + c == lane) {  // a pair with itself feels no decay
                  self = gg[c];
                  gg[c] = 0.f;
                }
                e[c] *= del;
                a[c] *= wt_;
              }
            }
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
              col += gg[c] + gg[c + 1];
              pw[c / 2] = pack_bf16(a[c], a[c + 1]);
              qw[c / 2] = pack_bf16(e[c], e[c + 1]);
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) gg[c] *= del;
            const float rs = column_sums(gg, lane);
            if (lane < 8) gs.row[qd][32 * I + 8 * o + lane] = rs;
          }
          tmem_st4u(ta + 4 * o, pw);  // over columns this warp has read
          tmem_st4u(te + 4 * o, qw);
          sts128(qt + (((4 * (I & 1) + o) ^ (row & 7)) << 4), make_uint4(qw[0], qw[1], qw[2], qw[3]));
        }
        if (I < qd) gs.row[qd][32 * I + lane] = 0.f;
        gs.col[I][row] = col;
        if (I == qd) gs.self[row] = self;
        tmem_st_wait();
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_p);
      if (i > 0 && gater) gate_gradient(i - 1);
      // ---- the carried states' parts of dB and dC
      if (wtu(&bar_2, k, 92)) {
        tc_fence_after();
        float f[16], f2[16], t[16], d = 0.f;
        tmem_ld16(tm + TG_B + c0 + lq, f);
        tmem_ld16(tm + TG_C + c0 + lq, f2);
        tile_row_cols<16>(sm + G_C, row, c0, t);
        tmem_ld_wait();
        const float fb = del * fend;
#pragma unroll
        for (int c = 0; c < 16; ++c) aB[c] = fmaf(f[c], fb, aB[c]);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          f2[c] *= ecum;
          d = fmaf(f2[c], t[c], d);
          aC[c] += f2[c];
        }
        gs.v[I][row] = d;
      }
      tc_fence_before();
      mbar_arrive(&bar_c);
      if (I == 1 && i + 1 < w.nh) {  // the next head's gates, beside this one's products
        put_gates(gates[(i + 1) % 3], z + par_[i + 1].bias, live, par_[i + 1].A, row);
        z = raw(i + 2);
      }
      // <S, R> over the tiles' terms: 8 values a thread
      float sr = 0.f, dsk = 0.f;
      if (in) {
        const uint8_t *sp = sm + G_S + 2 * k * STILE + threadIdx.x * 16, *rp = sm + G_R + 2 * k * STILE + threadIdx.x * 16;
        const uint4 a0 = lds128(sp), a1 = lds128(sp + STILE), b0 = lds128(rp), b1 = lds128(rp + STILE);
        const uint32_t av[4] = {a0.x, a0.y, a0.z, a0.w}, al[4] = {a1.x, a1.y, a1.z, a1.w}, bv[4] = {b0.x, b0.y, b0.z, b0.w},
                       bl[4] = {b1.x, b1.y, b1.z, b1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sr = fmaf(__uint_as_float(av[j] << 16) + __uint_as_float(al[j] << 16), __uint_as_float(bv[j] << 16) + __uint_as_float(bl[j] << 16), sr);
          sr = fmaf(__uint_as_float(av[j] & 0xffff0000u) + __uint_as_float(al[j] & 0xffff0000u),
                    __uint_as_float(bv[j] & 0xffff0000u) + __uint_as_float(bl[j] & 0xffff0000u), sr);
        }
      }
      // ---- dx
      if (wtu(&bar_3, k, 93) && in) {
        tc_fence_after();
        float u[16], br[16], x[16], y[16], d = 0.f;
        tmem_ld16(tm + TG_U + c0 + lq, u);
        tmem_ld16(tm + TG_BR + c0 + lq, br);
        tile_row_cols<16>(xt, row, c0, x);
        tile_row_cols<16>(yt, row, c0, y);
        tmem_ld_wait();
        const float sk = par_[i].skip;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          d = fmaf(x[c], br[c], d);
          u[c] = fmaf(fend, br[c], u[c]);
          dsk = fmaf(x[c], y[c], dsk);
          u[c] = live ? fmaf(del, u[c], sk * y[c]) : 0.f;
        }
        gs.w[I][row] = fend * d;
        tile_put_cols<16>(xt, row, c0, u);  // the products that read x have been done since bar_2
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_x);
      sr = warp_sum(sr);
      dsk = warp_sum(dsk);
      if (lane == 0) gs.red[warp][0] = sr, gs.red[warp][1] = dsk;
      // ---- the pairs' parts of dB and dC
      if (wtu(&bar_4, k, 94)) {
        tc_fence_after();
        float f[16], f2[16];
        tmem_ld16(tm + TG_B + c0 + lq, f);
        tmem_ld16(tm + TG_C + c0 + lq, f2);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          aB[c] += f[c];
          aC[c] += f2[c];
        }
      }
      tc_fence_before();
      mbar_arrive(&bar_free);
      sync_grad();  // this head's sums and the next one's gates are in place
    }
    if (gater) gate_gradient(w.nh - 1);
    if (row < in_n && c0 < s.D) {
      const long o = ((r0 + row) * parts + w.part) * s.D + c0;
      if (!live) {
#pragma unroll
        for (int c = 0; c < 16; ++c) aB[c] = aC[c] = 0.f;
      }
      if (direct) {
        store_bf16<16>(static_cast<bf16*>(dB) + o, aB);
        store_bf16<16>(static_cast<bf16*>(dC) + o, aC);
      } else {
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
          *reinterpret_cast<float4*>(static_cast<float*>(dB) + o + c) = make_float4(aB[c], aB[c + 1], aB[c + 2], aB[c + 3]);
          *reinterpret_cast<float4*>(static_cast<float*>(dC) + o + c) = make_float4(aC[c], aC[c + 1], aC[c + 2], aC[c + 3]);
        }
      }
    }
  }
  leave(tm, 512, WG_ISSUE);
}

// ------------------------------------------------------------------ host

constexpr size_t LINE = 128;  // the parts of the workspace start on lines
size_t align_line(size_t n) { return (n + LINE - 1) / LINE * LINE; }
char* first_line(void* ws) { return reinterpret_cast<char*>(align_line(reinterpret_cast<size_t>(ws))); }

int chunks(const ScanShape& s) { return (s.N + TC_C - 1) / TC_C; }

// Heads a block takes in turn, from one group: the count that minimises whole
// waves of blocks times (heads + the block's fixed cost, measured at about one
// head's time).
struct Parts {
  int hs, pg;
  Parts(const ScanShape& s, int slots) {
    const int hg = s.H / s.G;
    const long units = (long)s.B * chunks(s) * s.G;
    double best = 0;
    hs = 1;
    for (int t = 1; t <= hg && t <= MAXH; ++t) {
      const long blocks = units * ((hg + t - 1) / t);
      const double cost = (double)((blocks + slots - 1) / slots) * (t + 1.0);
      if (t == 1 || cost < best) best = cost, hs = t;
    }
    pg = (hg + hs - 1) / hs;
  }
};

struct WsTC {
  size_t tot, pf, sf, sl, pr, sr, rl, pB, pC, pp, end;
  WsTC(const ScanShape& s, bool bwd) {
    const size_t n = (size_t)s.B * s.H * chunks(s), st = n * s.D * s.M;
    tot = 0;
    pf = align_line(n * 4);
    sf = pf + st * 4;
    end = align_line(sf + st * 2);
    if (bwd) {
      const int pg = Parts(s, sm_count()).pg;
      const size_t part = pg == 1 ? 0 : (size_t)s.B * s.N * s.G * pg * s.D * 4;
      sl = end;
      pr = align_line(sl + st * 2);
      sr = pr + st * 4;
      rl = align_line(sr + st * 2);
      pB = align_line(rl + st * 2);
      pC = align_line(pB + part);
      pp = align_line(pC + part);
      end = pp + align_line(n * 12);
    }
  }
};

bool row_maps(Maps& m, const ScanIn& a, const ScanShape& s) {
  return make_rows_map(&m.x, a.x, s.M, s.H, s.ldx, s.N, s.B) && make_rows_map(&m.B, a.B, s.D, s.G, s.ldb, s.N, s.B) &&
         make_rows_map(&m.C, a.C, s.D, s.G, s.ldc, s.N, s.B);
}

// The gradients' tile kernels wait for the whole of the kernel before them:
// blocks that start early fill the SMs that empty first and leave the others
// idle (training 226 us so, 238 with early starts; the forward's gain 2 to 5).
template <typename... Exp, typename... Act>
cudaError_t launch_whole(void (*kernel)(Exp...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Act&&... args) {
  kernel<<<grid, block, smem, st>>>(std::forward<Act>(args)...);
  return cudaGetLastError();
}

}  // namespace

#define LA_TRY_CUDA(x)                     \
  do {                                     \
    const cudaError_t e_ = (x);            \
    if (e_ != cudaSuccess) return e_;      \
  } while (0)

size_t scan_tc_ws_bytes(const ScanShape& s, bool bwd) { return WsTC(s, bwd).end + LINE; }

cudaError_t scan_fwd_tc(const ScanIn& a, float* S, void* y, void* ws, const ScanShape& s, cudaStream_t st) {
  const WsTC w(s, false);
  char* base = first_line(ws);
  float *tot = (float*)(base + w.tot), *pf = (float*)(base + w.pf);
  bf16* sf = (bf16*)(base + w.sf);
  const int nch = chunks(s);
  const bool states = nch > 1 || S != nullptr;
  const Parts p(s, 2 * sm_count());
  const dim3 grid(nch, s.G * p.pg, s.B);
  Maps m;
  if (!row_maps(m, a, s) || !make_rows_map(&m.o, y, s.M, s.H, (long)s.H * s.M, s.N, s.B) ||
      !make_state_map(&m.S, sf, s.M, s.D, (long)s.B * s.H * nch))
    return cudaErrorInvalidValue;
  m.g = m.x;
  m.R = m.Sl = m.Rl = m.S;
  const bf16 *dt = (const bf16*)a.dt, *A = (const bf16*)a.A, *skip = (const bf16*)a.skip, *bias = (const bf16*)a.dt_bias;
  int* err = status_word();
  if (states) {
    const Parts ps(s, 3 * sm_count());
    const dim3 sgrid(nch, s.G * ps.pg, s.B);
    const int terms = S != nullptr ? 3 : 2;
    auto sums = terms == 3 ? &k_sums<3> : &k_sums<2>;
    LA_TRY_CUDA(cudaFuncSetAttribute(sums, cudaFuncAttributeMaxDynamicSharedMemorySize, S_SMEM(terms)));
    LA_TRY_CUDA(launch_pdl(sums, sgrid, dim3(NT), S_SMEM(terms), st, m, dt, A, bias, a.lengths, pf, static_cast<float*>(nullptr), tot, s, ps.pg,
                           ps.hs, err));
    LA_TRY_CUDA(scan_carry_bf16(pf, nullptr, sf, nullptr, nullptr, nullptr, tot, S, s.B * s.H, nch, s.D * s.M, st));
  }
  LA_TRY_CUDA(cudaFuncSetAttribute(k_out, cudaFuncAttributeMaxDynamicSharedMemorySize, O_SMEM));
  return launch_pdl(k_out, grid, dim3(NT), O_SMEM, st, m, dt, A, skip, bias, a.lengths, (bf16*)y, s, p.pg, p.hs, states ? 1 : 0, err);
}

cudaError_t scan_bwd_tc(const ScanIn& a, const void* dy, const ScanGrads& d, void* ws, const ScanShape& s, cudaStream_t st) {
  const WsTC w(s, true);
  char* base = first_line(ws);
  float *tot = (float*)(base + w.tot), *pf = (float*)(base + w.pf), *pr = (float*)(base + w.pr), *pp = (float*)(base + w.pp);
  bf16 *sf = (bf16*)(base + w.sf), *sr = (bf16*)(base + w.sr), *sl = (bf16*)(base + w.sl), *rl = (bf16*)(base + w.rl);
  const int nch = chunks(s);
  const long n = (long)s.B * s.H * nch;
  Maps m;
  if (!row_maps(m, a, s) || !make_rows_map(&m.g, dy, s.M, s.H, (long)s.H * s.M, s.N, s.B) ||
      !make_rows_map(&m.o, d.x, s.M, s.H, (long)s.H * s.M, s.N, s.B) || !make_state_map(&m.S, sf, s.M, s.D, n) ||
      !make_state_map(&m.R, sr, s.M, s.D, n) || !make_state_map(&m.Sl, sl, s.M, s.D, n) || !make_state_map(&m.Rl, rl, s.M, s.D, n))
    return cudaErrorInvalidValue;
  const bf16 *dt = (const bf16*)a.dt, *A = (const bf16*)a.A, *skip = (const bf16*)a.skip, *bias = (const bf16*)a.dt_bias;
  int* err = status_word();
  const bool states = nch > 1;
  if (states) {
    const Parts ps(s, 3 * sm_count() / 2);  // either direction's share of three blocks an SM
    LA_TRY_CUDA(cudaFuncSetAttribute(k_sums<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, S_SMEM(2)));
    LA_TRY_CUDA(launch_whole(k_sums<2>, dim3(nch, 2 * s.G * ps.pg, s.B), dim3(NT), S_SMEM(2), st, m, dt, A, bias, a.lengths, pf, pr, tot, s, ps.pg, ps.hs, err));
    LA_TRY_CUDA(scan_carry_bf16(pf, pr, sf, sr, sl, rl, tot, nullptr, s.B * s.H, nch, s.D * s.M, st));
  }
  const Parts p(s, sm_count());
  const bool direct = p.pg == 1;
  LA_TRY_CUDA(cudaFuncSetAttribute(k_grad, cudaFuncAttributeMaxDynamicSharedMemorySize, G_SMEM));
  LA_TRY_CUDA(launch_whole(k_grad, dim3(nch, s.G * p.pg, s.B), dim3(NTG), G_SMEM, st, m, dt, A, skip, bias, a.lengths, (bf16*)d.x,
                         (bf16*)d.dt, direct ? d.B : static_cast<void*>(base + w.pB), direct ? d.C : static_cast<void*>(base + w.pC),
                         pp, s, p.pg, p.hs, states ? 1 : 0, err));
  if (!direct) LA_TRY_CUDA(scan_groups((float*)(base + w.pB), (float*)(base + w.pC), d.B, d.C, s, p.pg, st));
  return scan_params(pp, d.A, d.skip, d.dt_bias, s, nch, st);
}

}  // namespace la
