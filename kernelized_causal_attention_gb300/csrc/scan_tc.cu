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
// and two of them share an SM: one block's loads and CUDA-core work cover the
// other's products.  A block takes one chunk and several heads of one group,
// whose B and C tiles it loads once.
//
// Decays: within 32 x 32 blocks off the diagonal exp(cum_i - cum_j) is a row
// factor times a column factor, both taken from the end of the column's block
// so that neither exceeds 1 (A <= 0); the diagonal blocks take one exponential
// a pair.  All exponentials are base 2, of fp32 sums.
//
// Roundings: P and the carried states to bf16 before their products (half a
// step, 2^-8, each on its own part of y), y once.  The chunk sums take w_j x_j
// as two bf16 terms (2^-16), since the final state is an fp32 output.
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
// 32-row block; tot: the blocks' totals; del: delta; cf: delta exp(block end - cum).
struct Gates {
  float wp[128], del[128], cf[128], tot[4];
  __device__ __forceinline__ float off(int q) const {  // log2 decay of the blocks before q
    float s = 0.f;
    for (int p = 0; p < q; ++p) s += tot[p];
    return s;
  }
  __device__ __forceinline__ float past(int q) const {  // of the blocks after q
    float s = 0.f;
    for (int p = 3; p > q; --p) s += tot[p];
    return s;
  }
};

// By warps 0 .. 3, row = 32 warp + lane.
__device__ __forceinline__ void put_gates(Gates& g, float z, bool live, float A, int row) {
  const float d = live ? softplus(z) : 0.f;
  const float wp = warp_prefix(d * A * LOG2E);
  const float tot = __shfl_sync(0xffffffffu, wp, 31);
  g.wp[row] = wp;
  g.del[row] = d;
  g.cf[row] = d * exp2f(tot - wp);
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
};

// Rows [rows, 128) of a swizzled [128][64] tile become zeros (256 threads).
__device__ __forceinline__ void clear_rows(uint8_t* tile, int rows) {
  for (int v = rows * 8 + threadIdx.x; v < TILE / 16; v += 256) sts128(tile + v * 16, make_uint4(0u, 0u, 0u, 0u));
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
  CUtensorMap S, R;        // the carried states
};

// ------------------------------------------------------------- chunk sums
// TERMS bf16 terms of the scaled operand.  blockIdx.y = part, or parts + part
// for the reverse sums E = sum_i exp(cum_i) C_i dy_i^T.
constexpr int S_A = 0, S_X = TILE, S_T = 3 * TILE;  // B or C; two x stages; the terms
constexpr int S_SMEM(int terms) { return (3 + terms) * TILE + 1024; }

template <int TERMS>
__global__ void __launch_bounds__(NT, 2)
    k_sums(const __grid_constant__ Maps maps, const bf16* __restrict__ dt, const bf16* __restrict__ A,
           const bf16* __restrict__ bias, const int* __restrict__ lengths, float* __restrict__ fwd, float* __restrict__ rev,
           float* __restrict__ tot, ScanShape s, int pg, int hs, int* err) {
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = align1024(smraw);
  __shared__ uint64_t bar_a, bar_x[2], bar_t, bar_m, bar_fin;
  __shared__ Gates gates[2];
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;
  const int parts = s.G * pg;
  const bool back = blockIdx.y >= parts;
  const Share w(s, lengths, back ? blockIdx.y - parts : blockIdx.y, pg, hs);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nch = gridDim.x;
  const int DM = s.D * s.M;
  float* out = (back ? rev : fwd) + (((long)w.b * s.H + w.h0) * nch + blockIdx.x) * DM;  // head h0 + i: + i nch DM
  if (w.rows == 0) {
    for (int i = 0; i < w.nh; ++i) {
      for (int e = threadIdx.x * 4; e < DM; e += NT * 4) *reinterpret_cast<float4*>(out + (long)i * nch * DM + e) = make_float4(0.f, 0.f, 0.f, 0.f);
      if (threadIdx.x == 0 && !back) tot[((long)w.b * s.H + w.h0 + i) * nch + blockIdx.x] = 0.f;
    }
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(&bar_a, 1);
    mbar_init(&bar_x[0], 1);
    mbar_init(&bar_x[1], 1);
    mbar_init(&bar_t, 256);
    mbar_init(&bar_m, 1);
    mbar_init(&bar_fin, 1);
    fence_barrier_init();
    s_abort = 0;
  }
  if (warp == W_ISSUE) tmem_alloc(&tmem_base, 128);
  LA_SCAN_WAITS()
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;

  if (warp == W_ISSUE) {
    if (lane == 0) {
      const CUtensorMap* mx = back ? &maps.g : &maps.x;
      mbar_arrive_expect_tx(&bar_a, TILE);
      tma_load_4d(sm + S_A, back ? &maps.C : &maps.B, &bar_a, 0, w.g, w.n0, w.b);
      int issued = 0;
      auto load = [&](int i) {
        mbar_arrive_expect_tx(&bar_x[i & 1], TILE);
        tma_load_4d(sm + S_X + (i & 1) * TILE, mx, &bar_x[i & 1], 0, w.h0 + i, w.n0, w.b);
        ++issued;
      };
      load(0);
      if (w.nh > 1) load(1);
      constexpr uint32_t ID = idesc_bf16(64, 64, true, true);
      const uint64_t da = sdesc(smem_u32(sm + S_A), 16, 1024);
      const bool in = wt(&bar_a, 0, 66);
      for (int i = 0; in && i < w.nh; ++i) {
        if (!wt(&bar_t, i & 1, 61)) break;
        tc_fence_after();
        if (i + 2 < w.nh) load(i + 2);  // head i's stage has been read
#pragma unroll
        for (int k = 0; k < TERMS; ++k) {
          const uint64_t db = sdesc(smem_u32(sm + S_T + k * TILE), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16(tm + (i & 1) * 64, dadd(da, kk * 2048), dadd(db, kk * 2048), ID, k > 0 || kk > 0);
        }
        mma_commit(&bar_m);
      }
      // nothing in flight at exit: the products' last commit, the loads
      mma_commit(&bar_fin);
      mbar_wait(&bar_fin, 0, WAIT_NS);
      drain_loads<2>(bar_x, issued);
    }
  } else {
    const int row = threadIdx.x & 127, half = threadIdx.x >> 7, q = row >> 5;
    const long r0 = (long)w.b * s.N + w.n0;
    auto raw = [&](int i) { return i < w.nh && row < w.rows ? to_f(dt[(r0 + row) * s.lddt + w.h0 + i]) : 0.f; };
    const int qd = warp & 3, srow = 16 * qd + lane;
    const uint32_t lq = static_cast<uint32_t>(32 * qd) << 16;
    auto drain = [&](int i, bool done) {  // head i's sums, its products done
      if (done) {
        tc_fence_after();
        float f[32];
        tmem_ldn<2>(tm + (i & 1) * 64 + lq + 32 * half, f);
        if (lane < 16 && srow < s.D) {
          float* o = out + (long)i * nch * DM + srow * s.M + 32 * half;
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            if (32 * half + c < s.M) *reinterpret_cast<float4*>(o + c) = make_float4(f[c], f[c + 1], f[c + 2], f[c + 3]);
        }
      }
      tc_fence_before();
    };
    float z = half == 0 ? raw(0) : 0.f;
    if (w.rows < min(TC_C, s.N - w.n0)) {  // rows past the sequence's length: not to be multiplied
      if (wtu(&bar_a, 0, 63)) clear_rows(sm + S_A, w.rows);
    }
    for (int i = 0; i < w.nh; ++i) {
      Gates& g = gates[i & 1];
      const int h = w.h0 + i;
      if (half == 0) {
        put_gates(g, z + par(bias, h), row < w.rows, to_f(A[h]), row);
        z = raw(i + 1);
      }
      sync_compute();
      if (threadIdx.x == 0 && !back) tot[((long)w.b * s.H + h) * nch + blockIdx.x] = (g.off(4)) * LN2;
      const float f = row >= w.rows ? 0.f : (back ? exp2f(g.wp[row] + g.off(q)) : g.cf[row] * exp2f(g.past(q)));
      const bool in = wtu(&bar_x[i & 1], (i >> 1) & 1, 64);
      const bool clear = i == 0 || wtu(&bar_m, (i - 1) & 1, 65);  // the terms' tiles have been read
      if (in && clear) {
        const uint8_t* xt = sm + S_X + (i & 1) * TILE;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int o = row * 128 + (((4 * half + c) ^ (row & 7)) << 4);
          const uint4 u = lds128(xt + o);
          const uint32_t v[4] = {u.x, u.y, u.z, u.w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = f != 0.f ? __uint_as_float(v[k] << 16) * f : 0.f;
            const float b = f != 0.f ? __uint_as_float(v[k] & 0xffff0000u) * f : 0.f;
            hi[k] = pack_bf16(a, b);
            if (TERMS > 1) lo[k] = pack_bf16(a - __uint_as_float(hi[k] << 16), b - __uint_as_float(hi[k] & 0xffff0000u));
          }
          sts128(sm + S_T + o, make_uint4(hi[0], hi[1], hi[2], hi[3]));
          if (TERMS > 1) sts128(sm + S_T + TILE + o, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_t);
      if (i > 0) drain(i - 1, clear);  // (the next head's products may already be done)
    }
    drain(w.nh - 1, wtu(&bar_m, (w.nh - 1) & 1, 62));
  }
  __syncthreads();
  tc_fence_after();
  if (warp == W_ISSUE) tmem_dealloc(tm, 128);
}

// ------------------------------------------------------------------ outputs
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
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;
  const Share w(s, lengths, blockIdx.y, pg, hs);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nch = gridDim.x;
  const long r0 = (long)w.b * s.N + w.n0;
  if (w.rows == 0) {  // nothing but rows past the sequence's length
    const int n = min(TC_C, s.N - w.n0), per = w.nh * s.M / 8;
    for (int e = threadIdx.x; e < n * per; e += NT)
      *reinterpret_cast<uint4*>(y + ((r0 + e / per) * s.H + w.h0) * s.M + e % per * 8) = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  if (threadIdx.x == 0) {
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
  if (warp == W_ISSUE) tmem_alloc(&tmem_base, 256);
  LA_SCAN_WAITS()
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;

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
      bool ok = wt(&bar_cb, 0, 71);
      for (int i = 0; ok && i < w.nh; ++i) {
        const int k = i & 1;
        const uint64_t dX = sdesc(smem_u32(sm + O_X + k * TILE), 16, 1024), dS = sdesc(smem_u32(sm + O_S + k * STILE), 16, 1024);
        if (!(ok = wt(&bar_x[k], (i >> 1) & 1, 72))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_bf16(tm + T_A, dadd(dC, 32 * kk), dadd(dB, 32 * kk), ID_A, kk > 0);
        if (states)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_bf16(tm + T_CS, dadd(dC, 32 * kk), dadd(dS, kk * 2048), ID_O, kk > 0);
        mma_commit(&bar_a);
        if (!(ok = wt(&bar_p, k, 73))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_bf16_ts(tm + T_O, tm + T_A + (kk < 4 ? 8 * kk : 32 + 8 * kk), dadd(dX, kk * 2048), ID_O, kk > 0);
        mma_commit(&bar_o);
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
    float z = wg == 0 ? raw(0) : 0.f;
    const bool cut = w.rows < min(TC_C, s.N - w.n0);
    for (int i = 0; i < w.nh; ++i) {
      const int k = i & 1, h = w.h0 + i;
      Gates& g = gates[k];
      uint8_t* xt = sm + O_X + k * TILE;
      if (wg == 0) {
        put_gates(g, z + par(bias, h), row < w.rows, to_f(A[h]), row);
        z = raw(i + 1);
      }
      sync_compute();
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
              const float f = exp2f(wp + here - g.off(J + 1));
#pragma unroll
              for (int c = 0; c < 16; ++c) pk[c] = pack_bf16(a[2 * c] * (f * g.cf[32 * J + 2 * c]), a[2 * c + 1] * (f * g.cf[32 * J + 2 * c + 1]));
            } else {
#pragma unroll
              for (int c = 0; c < 32; ++c) a[c] = c <= lane ? a[c] * (exp2f(wp - g.wp[32 * J + c]) * g.del[32 * J + c]) : 0.f;
#pragma unroll
              for (int c = 0; c < 16; ++c) pk[c] = pack_bf16(a[2 * c], a[2 * c + 1]);
            }
          }
          tmem_st16u(ta + 16 * j, pk);  // over columns this warp has read
        }
        tmem_st_wait();
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_p);
      const bool x_in = wtu(&bar_x[k], (i >> 1) & 1, 77);
      if (wtu(&bar_o, k, 78) && x_in) {
        tc_fence_after();
        float o[32], cs[32], x[32];
        tmem_ldn<2>(tm + T_O + 32 * wg + lq, o);
        if (states) tmem_ldn<2>(tm + T_CS + 32 * wg + lq, cs);
        tile_row_cols<32>(xt, row, 32 * wg, x);
        const float e = exp2f(wp + here), sk = par(skip, h);
        const bool live = row < w.rows;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float v = fmaf(sk, x[c], states ? fmaf(e, cs[c], o[c]) : o[c]);
          o[c] = live ? v : 0.f;
        }
        tile_put_cols<32>(xt, row, 32 * wg, o);
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_free);
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == W_ISSUE) tmem_dealloc(tm, 256);
}

// ---------------------------------------------------------------- gradients
// One chunk, several heads of one group in turn.  Rows of the score tiles are
// the keys j, so that P^T and Q^T serve from tensor memory as A operands:
//   A^T = B C^T, E^T = x dy^T;  P_ij = W_ij A_ij, Q_ij = W_ij delta_j E_ij
//   du = P^T dy + f_j (B R),        f_j = exp(cum_end - cum_j)
//   dB += Q^T C + delta_j f_j (x R^T),  dC += Q B + exp(cum_i) (dy S^T)
// dB and dC are summed over the block's heads in registers (fp32); a group's
// blocks leave fp32 partial sums that scan_groups adds up (one block: the
// gradients themselves).  The gate's gradient takes its pair sums G_ij =
// Q_ij A_ij from the fp32 scores in registers: the column sums of a 32 x 32 block
// cost 31 shuffles a warp.
//
// Bound by the chain score products -> weights -> gradient products of one head
// at a time on one block an SM (all 512 tensor-memory columns, 166 KB of shared
// memory); the carried states' products and their read-out run beside it.
constexpr int G_C = 0, G_B = TILE, G_X = 2 * TILE, G_Y = 4 * TILE, G_S = 6 * TILE, G_R = G_S + 2 * STILE, G_Q = G_R + 2 * STILE;
constexpr int G_SMEM = G_Q + 2 * TILE + 1024;
constexpr uint32_t TG_A = 0, TG_E = 128, TG_U = 256, TG_BR = 320, TG_B = 384, TG_C = 448;

// Sum over the warp's lanes of g[c] for each column c, to lane c.
__device__ __forceinline__ float column_sums(float (&g)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int c = 0; c < o; ++c) {
      const float keep = up ? g[c + o] : g[c], give = up ? g[c] : g[c + o];
      g[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return g[0];
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_suffix(float v) {  // inclusive, from the last lane
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float u = __shfl_down_sync(0xffffffffu, v, o);
    if (lane + o < 32) v += u;
  }
  return v;
}

__global__ void __launch_bounds__(NT, 1)
    k_grad(const __grid_constant__ Maps maps, const bf16* __restrict__ dt, const bf16* __restrict__ A,
           const bf16* __restrict__ skip, const bf16* __restrict__ bias, const int* __restrict__ lengths,
           bf16* __restrict__ dx, bf16* __restrict__ ddt, void* dB, void* dC, float* __restrict__ pp, ScanShape s, int pg,
           int hs, int* err) {
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = align1024(smraw);
  __shared__ uint64_t bar_cb, bar_in[2], bar_clear, bar_1, bar_2, bar_3, bar_4, bar_p, bar_c, bar_x, bar_free;
  __shared__ Gates gates[2];
  __shared__ float s_row[4][128], s_col[2][128], s_v[2][128], s_w[2][128], s_u[2][128], s_red[8][2], s_tot[4][2], s_out[4][2];
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;
  const Share w(s, lengths, blockIdx.y, pg, hs);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nch = gridDim.x;
  const long r0 = (long)w.b * s.N + w.n0;
  const int in_n = min(TC_C, s.N - w.n0);  // rows of the chunk that exist
  const bool direct = pg == 1;             // dB and dC themselves, else partial sums
  const int parts = s.G * pg;
  if (w.rows == 0) {  // nothing but rows past the sequence's length
    const int per = w.nh * s.M / 8;
    for (int e = threadIdx.x; e < in_n * per; e += NT)
      *reinterpret_cast<uint4*>(dx + ((r0 + e / per) * s.H + w.h0) * s.M + e % per * 8) = make_uint4(0u, 0u, 0u, 0u);
    for (int e = threadIdx.x; e < in_n * w.nh; e += NT) ddt[(r0 + e / w.nh) * s.H + w.h0 + e % w.nh] = from_f<bf16>(0.f);
    for (int e = threadIdx.x; e < in_n * s.D; e += NT) {
      const long o = ((r0 + e / s.D) * parts + w.part) * s.D + e % s.D;
      if (direct) {
        static_cast<bf16*>(dB)[o] = from_f<bf16>(0.f);
        static_cast<bf16*>(dC)[o] = from_f<bf16>(0.f);
      } else {
        static_cast<float*>(dB)[o] = 0.f;
        static_cast<float*>(dC)[o] = 0.f;
      }
    }
    for (int e = threadIdx.x; e < w.nh * 3; e += NT) pp[(((long)w.b * s.H + w.h0 + e / 3) * nch + blockIdx.x) * 3 + e % 3] = 0.f;
    return;
  }
  if (threadIdx.x == 0) {
    for (uint64_t* b : {&bar_cb, &bar_in[0], &bar_in[1], &bar_1, &bar_2, &bar_3, &bar_4}) mbar_init(b, 1);
    for (uint64_t* b : {&bar_clear, &bar_p, &bar_c, &bar_x, &bar_free}) mbar_init(b, 256);
    fence_barrier_init();
    s_abort = 0;
  }
  if (warp == W_ISSUE) tmem_alloc(&tmem_base, 512);
  LA_SCAN_WAITS()
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;
  const bool cut = w.rows < in_n;

  if (warp == W_ISSUE) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&bar_cb, 2 * TILE);
      tma_load_4d(sm + G_C, &maps.C, &bar_cb, 0, w.g, w.n0, w.b);
      tma_load_4d(sm + G_B, &maps.B, &bar_cb, 0, w.g, w.n0, w.b);
      int issued = 0;
      auto load = [&](int i) {
        const int k = i & 1, h = w.h0 + i;
        mbar_arrive_expect_tx(&bar_in[k], 2 * TILE + 2 * STILE);
        tma_load_4d(sm + G_X + k * TILE, &maps.x, &bar_in[k], 0, h, w.n0, w.b);
        tma_load_4d(sm + G_Y + k * TILE, &maps.g, &bar_in[k], 0, h, w.n0, w.b);
        tma_load_3d(sm + G_S + k * STILE, &maps.S, &bar_in[k], 0, 0, (w.b * s.H + h) * nch + blockIdx.x);
        tma_load_3d(sm + G_R + k * STILE, &maps.R, &bar_in[k], 0, 0, (w.b * s.H + h) * nch + blockIdx.x);
        ++issued;
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
        const uint64_t dS = sdesc(smem_u32(sm + G_S + k * STILE), 16, 1024), dR = sdesc(smem_u32(sm + G_R + k * STILE), 16, 1024);
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
        for (int kk = 0; kk < 4; ++kk) mma_bf16(tm + TG_B, dadd(dX, 32 * kk), dadd(dR, 32 * kk), ID_KK, kk > 0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_bf16(tm + TG_C, dadd(dY, 32 * kk), dadd(dS, 32 * kk), ID_KK, kk > 0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_bf16(tm + TG_BR, dadd(dBt, 32 * kk), dadd(dR, kk * 2048), ID_KM, kk > 0);
        mma_commit(&bar_2);
        if (!(ok = wt(&bar_p, k, 85))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // P^T dy
          mma_bf16_ts(tm + TG_U, tm + TG_A + (kk < 4 ? 8 * kk : 32 + 8 * kk), dadd(dY, kk * 2048), ID_KM, kk > 0);
        mma_commit(&bar_3);
        if (!(ok = wt(&bar_c, k, 86))) break;  // x R^T and dy S^T have been read
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // Q^T C
          mma_bf16_ts(tm + TG_B, tm + TG_E + (kk < 4 ? 8 * kk : 32 + 8 * kk), dadd(dCt, kk * 2048), ID_KM, kk > 0);
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
    const int qd = warp & 3, wg = warp >> 2, row = 32 * qd + lane;
    const uint32_t lq = static_cast<uint32_t>(32 * qd) << 16;
    const bool live = row < w.rows;
    auto raw = [&](int i) { return i < w.nh && live ? to_f(dt[(r0 + row) * s.lddt + w.h0 + i]) : 0.f; };
    float z = wg == 0 ? raw(0) : 0.f;
    float aB[32], aC[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) aB[c] = aC[c] = 0.f;
    const bool cb = wtu(&bar_cb, 0, 89);
    for (int i = 0; i < w.nh; ++i) {
      const int k = i & 1, h = w.h0 + i;
      Gates& g = gates[k];
      uint8_t *xt = sm + G_X + k * TILE, *yt = sm + G_Y + k * TILE;
      const float zi = z + par(bias, h), Ah = to_f(A[h]);
      if (wg == 0) {
        put_gates(g, zi, live, Ah, row);
        z = raw(i + 1);
      }
      sync_compute();
      const bool in = wtu(&bar_in[k], (i >> 1) & 1, 90) && cb;
      if (cut) {
        if (in) {
          if (i == 0) {
            clear_rows(sm + G_C, w.rows);
            clear_rows(sm + G_B, w.rows);
          }
          clear_rows(xt, w.rows);
          clear_rows(yt, w.rows);
        }
        fence_proxy_async();
        mbar_arrive(&bar_clear);
      }
      const float wp = g.wp[row], here = g.off(qd), del = g.del[row];
      const float tail = exp2f(g.tot[qd] - wp);     // from this row to its block's end
      const float fend = tail * exp2f(g.past(qd));  // to the chunk's end
      const float ecum = exp2f(wp + here);
      // ---- the weights on A^T and E^T
      if (wtu(&bar_1, k, 91)) {
        tc_fence_after();
        const uint32_t ta = tm + TG_A + 64 * wg + lq, te = tm + TG_E + 64 * wg + lq;
        float col = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int I = 2 * wg + j;  // a block of 32 query columns
          uint32_t pw[16], qw[16];
          float rs = 0.f;
          if (I < qd) {
#pragma unroll
            for (int c = 0; c < 16; ++c) pw[c] = qw[c] = 0u;
          } else {
            float a[32], e[32];
            tmem_ldn<2>(ta + 32 * j, a);
            tmem_ldn<2>(te + 32 * j, e);
            const float fr = I > qd ? tail * exp2f(g.off(I) - g.off(qd + 1)) : 0.f;
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              float p[2], qq[2];
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const float wi = g.wp[32 * I + c + t];
                const float wt_ = I > qd ? fr * exp2f(wi) : (c + t >= lane ? exp2f(wi - wp) : 0.f);
                p[t] = wt_ * a[c + t];
                qq[t] = wt_ * del * e[c + t];
                const float gg = I == qd && c + t == lane ? 0.f : qq[t] * a[c + t];
                col += gg;
                e[c + t] = gg;
              }
              pw[c / 2] = pack_bf16(p[0], p[1]);
              qw[c / 2] = pack_bf16(qq[0], qq[1]);
            }
            rs = column_sums(e, lane);
          }
          s_row[qd][32 * I + lane] = rs;
          tmem_st16u(ta + 16 * j, pw);  // over columns this warp has read
          tmem_st16u(te + 16 * j, qw);
          uint8_t* qt = sm + G_Q + wg * TILE;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            sts128(qt + row * 128 + (((4 * j + c) ^ (row & 7)) << 4), make_uint4(qw[4 * c], qw[4 * c + 1], qw[4 * c + 2], qw[4 * c + 3]));
        }
        s_col[wg][row] = col;
        tmem_st_wait();
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_p);
      // ---- the carried states' parts of dB and dC
      if (wtu(&bar_2, k, 92)) {
        tc_fence_after();
        float f[32], t[32], d = 0.f;
        tmem_ldn<2>(tm + TG_B + 32 * wg + lq, f);
        tile_row_cols<32>(sm + G_B, row, 32 * wg, t);
        const float fb = del * fend;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          f[c] *= fb;
          d = fmaf(f[c], t[c], d);
          aB[c] += f[c];
        }
        s_w[wg][row] = d;
        d = 0.f;
        tmem_ldn<2>(tm + TG_C + 32 * wg + lq, f);
        tile_row_cols<32>(sm + G_C, row, 32 * wg, t);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          f[c] *= ecum;
          d = fmaf(f[c], t[c], d);
          aC[c] += f[c];
        }
        s_v[wg][row] = d;
      }
      tc_fence_before();
      mbar_arrive(&bar_c);
      // ---- dx
      float dsk = 0.f;
      if (wtu(&bar_3, k, 93) && in) {
        tc_fence_after();
        float u[32], x[32], y[32], d = 0.f;
        tmem_ldn<2>(tm + TG_U + 32 * wg + lq, u);
        tmem_ldn<2>(tm + TG_BR + 32 * wg + lq, x);
#pragma unroll
        for (int c = 0; c < 32; ++c) u[c] = fmaf(fend, x[c], u[c]);
        tile_row_cols<32>(xt, row, 32 * wg, x);
        tile_row_cols<32>(yt, row, 32 * wg, y);
        const float sk = par(skip, h);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          d = fmaf(x[c], u[c], d);
          dsk = fmaf(x[c], y[c], dsk);
          u[c] = live ? fmaf(del, u[c], sk * y[c]) : 0.f;
        }
        s_u[wg][row] = d;
        // <S, R> over the two bf16 tiles: 16 values a thread
        float sr = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int o = (threadIdx.x + 256 * c) * 16;
          const uint4 a = lds128(sm + G_S + k * STILE + o), b = lds128(sm + G_R + k * STILE + o);
          const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sr = fmaf(__uint_as_float(av[j] << 16), __uint_as_float(bv[j] << 16), sr);
            sr = fmaf(__uint_as_float(av[j] & 0xffff0000u), __uint_as_float(bv[j] & 0xffff0000u), sr);
          }
        }
        sr = warp_sum(sr);
        dsk = warp_sum(dsk);
        if (lane == 0) s_red[warp][0] = sr, s_red[warp][1] = dsk;
        // the products that read x have been done since bar_2 (x R^T, E^T)
        tile_put_cols<32>(xt, row, 32 * wg, u);
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_x);
      sync_compute();  // the sums of both halves are in place
      // ---- the gate's gradient: rows t of warps 0 .. 3
      if (wg == 0) {
        float q = s_v[0][row] + s_v[1][row] - (s_col[0][row] + s_col[1][row]);
#pragma unroll
        for (int j = 0; j < 4; ++j) q += s_row[j][row];
        const float ww = s_w[0][row] + s_w[1][row];
        const float suf = warp_suffix(q), pre = warp_prefix(ww);
        if (lane == 0) s_tot[qd][0] = suf;
        if (lane == 31) s_tot[qd][1] = pre;
        asm volatile("bar.sync 2, 128;" ::: "memory");
        float dl = suf + (pre - ww), sr = 0.f, ds = 0.f;
        for (int j = qd + 1; j < 4; ++j) dl += s_tot[j][0];
        for (int j = 0; j < qd; ++j) dl += s_tot[j][1];
#pragma unroll
        for (int j = 0; j < 8; ++j) sr += s_red[j][0], ds += s_red[j][1];
        dl = fmaf(exp2f(g.off(4)), sr, dl);
        const float dz = live ? (s_u[0][row] + s_u[1][row] + Ah * dl) / (1.f + expf(-zi)) : 0.f;
        if (row < in_n) ddt[(r0 + row) * s.H + h] = from_f<bf16>(dz);
        const float dA = warp_sum(live ? del * dl : 0.f), db = warp_sum(dz);
        if (lane == 0) s_out[qd][0] = dA, s_out[qd][1] = db;
        asm volatile("bar.sync 2, 128;" ::: "memory");
        if (threadIdx.x == 0) {
          float* o = pp + (((long)w.b * s.H + h) * nch + blockIdx.x) * 3;
          o[0] = s_out[0][0] + s_out[1][0] + s_out[2][0] + s_out[3][0];
          o[1] = ds;
          o[2] = s_out[0][1] + s_out[1][1] + s_out[2][1] + s_out[3][1];
        }
      }
      // ---- the pairs' parts of dB and dC
      if (wtu(&bar_4, k, 94)) {
        tc_fence_after();
        float f[32];
        tmem_ldn<2>(tm + TG_B + 32 * wg + lq, f);
#pragma unroll
        for (int c = 0; c < 32; ++c) aB[c] += f[c];
        tmem_ldn<2>(tm + TG_C + 32 * wg + lq, f);
#pragma unroll
        for (int c = 0; c < 32; ++c) aC[c] += f[c];
      }
      tc_fence_before();
      mbar_arrive(&bar_free);
    }
    if (row < in_n) {
      const long o = ((r0 + row) * parts + w.part) * s.D + 32 * wg;
#pragma unroll
      for (int c = 0; c < 32; c += 8) {
        if (32 * wg + c >= s.D) break;
        if (!live) {
#pragma unroll
          for (int j = 0; j < 8; ++j) aB[c + j] = aC[c + j] = 0.f;
        }
        if (direct) {
          store_bf16<8>(static_cast<bf16*>(dB) + o + c, aB + c);
          store_bf16<8>(static_cast<bf16*>(dC) + o + c, aC + c);
        } else {
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            *reinterpret_cast<float4*>(static_cast<float*>(dB) + o + c + j) = make_float4(aB[c + j], aB[c + j + 1], aB[c + j + 2], aB[c + j + 3]);
            *reinterpret_cast<float4*>(static_cast<float*>(dC) + o + c + j) = make_float4(aC[c + j], aC[c + j + 1], aC[c + j + 2], aC[c + j + 3]);
          }
        }
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == W_ISSUE) tmem_dealloc(tm, 512);
}

// ------------------------------------------------------------------ host

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

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
    for (int t = 1; t <= hg && t <= 16; ++t) {
      const long blocks = units * ((hg + t - 1) / t);
      const double cost = (double)((blocks + slots - 1) / slots) * (t + 1.0);
      if (t == 1 || cost < best) best = cost, hs = t;
    }
    pg = (hg + hs - 1) / hs;
  }
};

struct WsTC {
  size_t tot, pf, sf, pr, sr, pB, pC, pp, end;
  WsTC(const ScanShape& s, bool bwd) {
    const size_t n = (size_t)s.B * s.H * chunks(s), st = n * s.D * s.M;
    tot = 0;
    pf = align16(n * 4);
    sf = pf + st * 4;
    end = sf + st * 2;
    if (bwd) {
      const int pg = Parts(s, sm_count()).pg;
      const size_t part = pg == 1 ? 0 : (size_t)s.B * s.N * s.G * pg * s.D * 4;
      pr = end;
      sr = pr + st * 4;
      pB = sr + st * 2;
      pC = pB + part;
      pp = pC + part;
      end = pp + align16(n * 12);
    }
  }
};

bool row_maps(Maps& m, const ScanIn& a, const ScanShape& s) {
  return make_rows_map(&m.x, a.x, s.M, s.H, s.ldx, s.N, s.B) && make_rows_map(&m.B, a.B, s.D, s.G, s.ldb, s.N, s.B) &&
         make_rows_map(&m.C, a.C, s.D, s.G, s.ldc, s.N, s.B);
}

}  // namespace

#define LA_TRY_CUDA(x)                     \
  do {                                     \
    const cudaError_t e_ = (x);            \
    if (e_ != cudaSuccess) return e_;      \
  } while (0)

size_t scan_tc_ws_bytes(const ScanShape& s, bool bwd) { return WsTC(s, bwd).end; }

cudaError_t scan_fwd_tc(const ScanIn& a, float* S, void* y, void* ws, const ScanShape& s, cudaStream_t st) {
  const WsTC w(s, false);
  char* base = static_cast<char*>(ws);
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
  m.R = m.S;
  const bf16 *dt = (const bf16*)a.dt, *A = (const bf16*)a.A, *skip = (const bf16*)a.skip, *bias = (const bf16*)a.dt_bias;
  int* err = status_word();
  if (states) {
    LA_TRY_CUDA(cudaFuncSetAttribute(k_sums<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, S_SMEM(2)));
    k_sums<2><<<grid, NT, S_SMEM(2), st>>>(m, dt, A, bias, a.lengths, pf, nullptr, tot, s, p.pg, p.hs, err);
    LA_TRY_CUDA(cudaGetLastError());
    LA_TRY_CUDA(scan_carry_bf16(pf, nullptr, sf, nullptr, tot, S, s.B * s.H, nch, s.D * s.M, st));
  }
  LA_TRY_CUDA(cudaFuncSetAttribute(k_out, cudaFuncAttributeMaxDynamicSharedMemorySize, O_SMEM));
  k_out<<<grid, NT, O_SMEM, st>>>(m, dt, A, skip, bias, a.lengths, (bf16*)y, s, p.pg, p.hs, states ? 1 : 0, err);
  return cudaGetLastError();
}

cudaError_t scan_bwd_tc(const ScanIn& a, const void* dy, const ScanGrads& d, void* ws, const ScanShape& s, cudaStream_t st) {
  const WsTC w(s, true);
  char* base = static_cast<char*>(ws);
  float *tot = (float*)(base + w.tot), *pf = (float*)(base + w.pf), *pr = (float*)(base + w.pr), *pp = (float*)(base + w.pp);
  bf16 *sf = (bf16*)(base + w.sf), *sr = (bf16*)(base + w.sr);
  const int nch = chunks(s);
  const long n = (long)s.B * s.H * nch;
  Maps m;
  if (!row_maps(m, a, s) || !make_rows_map(&m.g, dy, s.M, s.H, (long)s.H * s.M, s.N, s.B) ||
      !make_rows_map(&m.o, d.x, s.M, s.H, (long)s.H * s.M, s.N, s.B) || !make_state_map(&m.S, sf, s.M, s.D, n) ||
      !make_state_map(&m.R, sr, s.M, s.D, n))
    return cudaErrorInvalidValue;
  const bf16 *dt = (const bf16*)a.dt, *A = (const bf16*)a.A, *skip = (const bf16*)a.skip, *bias = (const bf16*)a.dt_bias;
  int* err = status_word();
  // the sums feed bf16 gradients only: one bf16 term
  const Parts ps(s, sm_count());
  LA_TRY_CUDA(cudaFuncSetAttribute(k_sums<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, S_SMEM(1)));
  k_sums<1><<<dim3(nch, 2 * s.G * ps.pg, s.B), NT, S_SMEM(1), st>>>(m, dt, A, bias, a.lengths, pf, pr, tot, s, ps.pg, ps.hs, err);
  LA_TRY_CUDA(cudaGetLastError());
  LA_TRY_CUDA(scan_carry_bf16(pf, pr, sf, sr, tot, nullptr, s.B * s.H, nch, s.D * s.M, st));
  const Parts p(s, sm_count());
  const bool direct = p.pg == 1;
  LA_TRY_CUDA(cudaFuncSetAttribute(k_grad, cudaFuncAttributeMaxDynamicSharedMemorySize, G_SMEM));
  k_grad<<<dim3(nch, s.G * p.pg, s.B), NT, G_SMEM, st>>>(m, dt, A, skip, bias, a.lengths, (bf16*)d.x, (bf16*)d.dt,
                                                        direct ? d.B : base + w.pB, direct ? d.C : base + w.pC, pp, s, p.pg, p.hs, err);
  LA_TRY_CUDA(cudaGetLastError());
  if (!direct) LA_TRY_CUDA(scan_groups((float*)(base + w.pB), (float*)(base + w.pC), d.B, d.C, s, p.pg, st));
  return scan_params(pp, d.A, d.skip, d.dt_bias, s, nch, st);
}

}  // namespace la
