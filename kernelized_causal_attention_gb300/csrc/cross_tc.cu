// The kernelized cross attention on the 5th-generation tensor cores, for bf16
// inputs with D and M in {16, 32, 64} (formulas: cross.cu; narrower heads ride in
// zero-filled 64-wide tiles).
//
// Four tile kernels over 128-row tiles, each block walking a few tiles of one
// head with two TMA stages, two or three blocks an SM:
//   k_ksum   S += phi(k)^T v,  Z += phi(k) in fp32 on the CUDA cores
//   k_read   out = (phi(q) S) / den,  den = phi(q) . Z in fp32 on the CUDA cores
//   k_grad_q T = dout S^T;  gamma = -e (e phi(q) . T);  dq = (e T + gamma Z) phi'(q);
//            R += (e phi(q))^T dout,  r += gamma phi(q)
//   k_grad_k dk = (v R^T + r) phi'(k),  dv = phi(k) R
// and k_cross_join (cross.cu) between them.  The products are a few hundred
// cycles a tile and phi with its splits into terms about as long, so what bounds
// them is a tile's chain of load, phi, product and read-out at two or three blocks
// an SM, and the launches.  16 x 8 query heads (4 key heads) x 512 queries, 2048
// states, 64 x 64, device time with L2 flushed: forward 32 us (51 MB to read and
// write once: 7.5), gradients 42 (92 MB: 14); by kernel, cold: k_ksum 16,
// k_read 11, k_grad_q 17, k_grad_k 22, either join 5.7.
//
// What is not a bf16 input (phi, S, R) enters its products as bf16 terms: three
// (2^-24) where the sum is an fp32 output (S), elsewhere two, a = a0 + a1 to
// 2^-16, taking a0 b0 + a0 b1 + a1 b0, so that each bf16 result is rounded once.
// Z and den are plain fp32 sums.
#include "launch.h"
#include "scan.cuh"
#include "tc.cuh"
#include "tc_chunk.cuh"

namespace la {
namespace {

using namespace tc;
using namespace tcc;

constexpr int NT = 288;  // 8 compute warps, then the issuer's
constexpr int W_ISSUE = 8;
constexpr float LOG2E = 1.4426950408889634f;
constexpr int STILE = 64 * 64 * 2;

// phi by a select: a branch around the exponential would diverge at every value.  (An
// infinite exponential of x > 0 is not selected; a NaN is: a minimum would drop it.)
__device__ __forceinline__ float phif(float x) {
  const float e = ex2_fast(x * LOG2E);
  return x > 0.f ? x + 1.f : e;
}

#define LA_WAITS()                                                          \
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

__device__ __forceinline__ void sync_compute() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Thirty-two floats as bf16 terms into columns [col0, col0 + 32) of row r of
// swizzled tiles: the first at `hi`, the others at `lo` and a tile further.
template <int TERMS = 2>
__device__ __forceinline__ void put_terms(uint8_t* hi, uint8_t* lo, int r, int col0, const float* f) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int o = r * 128 + ((((col0 >> 3) + c) ^ (r & 7)) << 4);
    uint32_t t[TERMS][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a = f[8 * c + 2 * k], b = f[8 * c + 2 * k + 1];
#pragma unroll
      for (int j = 0; j < TERMS; ++j) {
        t[j][k] = pack_bf16(a, b);
        a -= __uint_as_float(t[j][k] << 16);
        b -= __uint_as_float(t[j][k] & 0xffff0000u);
      }
    }
    sts128(hi + o, make_uint4(t[0][0], t[0][1], t[0][2], t[0][3]));
#pragma unroll
    for (int j = 1; j < TERMS; ++j) sts128(lo + (j - 1) * TILE + o, make_uint4(t[j][0], t[j][1], t[j][2], t[j][3]));
  }
}

// An fp32 [D][M] state as two bf16 term tiles [64][64] (zeros past D and M), by
// the 256 compute threads.
__device__ __forceinline__ void put_state(const float* S, uint8_t* hi, uint8_t* lo, int D, int M) {
  const int d = threadIdx.x >> 2, c0 = (threadIdx.x & 3) * 16;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      const int m = c0 + 8 * c + k;
      const float4 u = d < D && m < M ? *reinterpret_cast<const float4*>(S + d * M + m) : make_float4(0.f, 0.f, 0.f, 0.f);
      f[k] = u.x, f[k + 1] = u.y, f[k + 2] = u.z, f[k + 3] = u.w;
    }
    float l[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) l[k] = f[k] - __bfloat162float(__float2bfloat16_rn(f[k]));
    st_row_chunk(hi, d, (c0 >> 3) + c, f);
    st_row_chunk(lo, d, (c0 >> 3) + c, l);
  }
}

// phi of this thread's 32 columns of a tile row; columns at or past W become 0.
__device__ __forceinline__ void phi_cols(const float* x, float* f, int col0, int W) {
#pragma unroll
  for (int c = 0; c < 32; ++c) f[c] = col0 + c < W ? phif(x[c]) : 0.f;
}

__device__ __forceinline__ float column_sums(float (&g)[32], int lane) {  // over the warp's lanes, column c to lane c
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

// The 64 x 64 accumulator at column `ta` (M = 64 layout), and the one behind it if
// TWO, to [D][M] floats at o.
template <bool TWO = false>
__device__ __forceinline__ void store_state(uint32_t ta, float* o, int D, int M, int qd, int wg, int lane) {
  float f[32];
  tmem_ldn<2>(ta + (static_cast<uint32_t>(32 * qd) << 16) + 32 * wg, f);
  if (TWO) {
    float g[32];
    tmem_ldn<2>(ta + 64 + (static_cast<uint32_t>(32 * qd) << 16) + 32 * wg, g);
#pragma unroll
    for (int c = 0; c < 32; ++c) f[c] += g[c];
  }
  const int d = 16 * qd + lane;
  if (lane < 16 && d < D) {
#pragma unroll
    for (int c = 0; c < 32; c += 4)
      if (32 * wg + c < M) *reinterpret_cast<float4*>(o + d * M + 32 * wg + c) = make_float4(f[c], f[c + 1], f[c + 2], f[c + 3]);
  }
}

// D[128 x 64] = A B with A in nA and B in two terms (K = 64): a0 b0 + a0 b1 (+ a1 b0).
template <int NA>
__device__ __forceinline__ void mma_terms(uint32_t d, uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, bool b_mn) {
  const uint32_t id = idesc_bf16(128, 64, false, b_mn);
  const uint64_t A0 = sdesc(a0, 16, 1024), A1 = sdesc(a1, 16, 1024), B0 = sdesc(b0, 16, 1024), B1 = sdesc(b1, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    const uint32_t ob = b_mn ? kk * 2048 : kk * 32;
    mma_bf16(d, dadd(A0, 32 * kk), dadd(B0, ob), id, kk > 0);
    mma_bf16(d, dadd(A0, 32 * kk), dadd(B1, ob), id, 1);
    if (NA > 1) mma_bf16(d, dadd(A1, 32 * kk), dadd(B0, ob), id, 1);
  }
}

// --------------------------------------------------------------- S and Z
constexpr int K_STAGE = 2 * TILE;  // k (then phi's first term), v
constexpr int K_T = 2 * K_STAGE;   // phi's second and third terms
constexpr int K_SMEM = K_T + 2 * TILE + 1024;

__global__ void __launch_bounds__(NT, 2)
    k_ksum(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const int* __restrict__ lengths,
           float* __restrict__ rec, int Hk, int N, int D, int M, int per, int* err) {
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = align1024(smraw);
  __shared__ uint64_t bar_in[2], bar_t[2], bar_m[2], bar_fin;
  __shared__ float s_z[4][64];
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bh = blockIdx.y;
  if (threadIdx.x == 0) {
    for (int k = 0; k < 2; ++k) {
      mbar_init(&bar_in[k], 1);
      mbar_init(&bar_t[k], 256);
      mbar_init(&bar_m[k], 1);
    }
    mbar_init(&bar_fin, 1);
    fence_barrier_init();
    s_abort = 0;
  }
  enter(&tmem_base, 128, warp == W_ISSUE);
  const int L = valid_rows(lengths, bh / Hk, N);
  const int t0 = blockIdx.x * per, nt = min(per, (L + TC_C - 1) / TC_C - t0);
  float* o = rec + (static_cast<long>(bh) * gridDim.x + blockIdx.x) * (D * M + D);
  LA_WAITS()
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;
  if (nt <= 0) {
    for (int e = threadIdx.x; e < D * M + D; e += NT) o[e] = 0.f;
  } else if (warp == W_ISSUE) {
    if (lane == 0) {
      int issued = 0;
      auto load = [&](int i) {
        uint8_t* st = sm + (i & 1) * K_STAGE;
        mbar_arrive_expect_tx(&bar_in[i & 1], 2 * TILE);
        tma_load_3d(st, &mk, &bar_in[i & 1], 0, (t0 + i) * TC_C, bh);
        tma_load_3d(st + TILE, &mv, &bar_in[i & 1], 0, (t0 + i) * TC_C, bh);
        ++issued;
      };
      load(0);
      if (nt > 1) load(1);
      constexpr uint32_t ID = idesc_bf16(64, 64, true, true);
      for (int i = 0; i < nt; ++i) {
        const int k = i & 1;
        const uint32_t st = smem_u32(sm + k * K_STAGE), v = st + TILE;
        if (!wt(&bar_t[k], (i >> 1) & 1, 111)) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 3; ++j) {  // the terms of phi(k), the first in an accumulator of its own (fewer roundings of the large sum)
          const uint64_t da = sdesc(j == 0 ? st : smem_u32(sm + K_T + (j - 1) * TILE), 16, 1024), db = sdesc(v, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) mma_bf16(tm + (j > 0 ? 64 : 0), dadd(da, kk * 2048), dadd(db, kk * 2048), ID, i > 0 || j > 1 || kk > 0);
        }
        mma_commit(&bar_m[k]);
        if (i + 2 < nt) {
          if (!wt(&bar_m[k], (i >> 1) & 1, 112)) break;
          load(i + 2);
        }
      }
      mma_commit(&bar_fin);
      mbar_wait(&bar_fin, 0, WAIT_NS);
      drain_loads<2>(bar_in, issued);
    }
  } else {
    const int qd = warp & 3, wg = warp >> 2, row = 32 * qd + lane;
    float z[32];  // this row's part of Z, over the tiles
#pragma unroll
    for (int c = 0; c < 32; ++c) z[c] = 0.f;
    for (int i = 0; i < nt; ++i) {
      const int k = i & 1, valid = L - (t0 + i) * TC_C;
      uint8_t* st = sm + k * K_STAGE;
      if (wtu(&bar_in[k], (i >> 1) & 1, 113)) {
        float x[32], f[32];
        tile_row_cols<32>(st, row, 32 * wg, x);
        phi_cols(x, f, 32 * wg, D);
        if (i > 0) wtu(&bar_m[k ^ 1], ((i - 1) >> 1) & 1, 115);  // the second and third terms have been read
        if (row >= valid) {
#pragma unroll
          for (int c = 0; c < 32; ++c) f[c] = 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c)  // a row past the length is not to be multiplied either
            sts128(st + TILE + row * 128 + (((4 * wg + c) ^ (row & 7)) << 4), make_uint4(0u, 0u, 0u, 0u));
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) z[c] += f[c];
        put_terms<3>(st, sm + K_T, row, 32 * wg, f);
      }
      fence_proxy_async();
      mbar_arrive(&bar_t[k]);
    }
    if (wtu(&bar_m[(nt - 1) & 1], ((nt - 1) >> 1) & 1, 114)) {
      tc_fence_after();
      store_state<true>(tm, o, D, M, qd, wg, lane);
    }
    tc_fence_before();
    s_z[qd][32 * wg + lane] = column_sums(z, lane);
    sync_compute();
    if (threadIdx.x < D) o[D * M + threadIdx.x] = s_z[0][threadIdx.x] + s_z[1][threadIdx.x] + s_z[2][threadIdx.x] + s_z[3][threadIdx.x];
  }
  __syncthreads();
  tc_fence_after();
  if (warp == W_ISSUE) tmem_dealloc(tm, 128);
}

// ------------------------------------------------------------------- read
constexpr int R_Q = 0, R_LO = 2 * TILE, R_S = 3 * TILE;  // two q stages, phi's second term, S in two terms
constexpr int R_SMEM = 3 * TILE + 2 * STILE + 1024;

__global__ void __launch_bounds__(NT, 3)
    k_read(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mo, const float* __restrict__ S,
           const float* __restrict__ Z, float* __restrict__ den, int H, int Hk, int N, int D, int M, int per, int* err) {
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = align1024(smraw);
  __shared__ uint64_t bar_in[2], bar_t, bar_o, bar_free;
  __shared__ float zs[64], s_den[2][128];
  __shared__ int s_some[2];  // whether Z holds anything
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bh = blockIdx.y;
  const long bhk = static_cast<long>(bh / H) * Hk + bh % H / (H / Hk);
  const int t0 = blockIdx.x * per, nt = min(per, (N + TC_C - 1) / TC_C - t0);
  if (threadIdx.x == 0) {
    mbar_init(&bar_in[0], 1);
    mbar_init(&bar_in[1], 1);
    mbar_init(&bar_t, 256);
    mbar_init(&bar_o, 1);
    mbar_init(&bar_free, 256);
    fence_barrier_init();
    s_abort = 0;
  }
  enter(&tmem_base, 64, warp == W_ISSUE);
  LA_WAITS()
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;
  if (warp == W_ISSUE) {
    if (lane == 0) {
      int issued = 0;
      auto load = [&](int i) {
        mbar_arrive_expect_tx(&bar_in[i & 1], TILE);
        tma_load_3d(sm + R_Q + (i & 1) * TILE, &mq, &bar_in[i & 1], 0, (t0 + i) * TC_C, bh);
        ++issued;
      };
      load(0);
      if (nt > 1) load(1);
      for (int i = 0; i < nt; ++i) {
        const int k = i & 1;
        uint8_t* q = sm + R_Q + k * TILE;
        if (!wt(&bar_t, k, 121)) break;
        tc_fence_after();
        mma_terms<2>(tm, smem_u32(q), smem_u32(sm + R_LO), smem_u32(sm + R_S), smem_u32(sm + R_S + STILE), true);
        mma_commit(&bar_o);
        if (!wt(&bar_free, k, 122)) break;
        tma_store_3d(&mo, q, 0, (t0 + i) * TC_C, bh);  // out has taken q's place
        bulk_commit();
        if (i + 2 < nt) {
          bulk_wait_read();
          load(i + 2);
        }
      }
      mma_commit(&bar_o);  // nothing in flight at exit
      mbar_wait(&bar_o, nt & 1, WAIT_NS);
      drain_loads<2>(bar_in, issued);
      bulk_wait_all();
    }
  } else {
    const int qd = warp & 3, wg = warp >> 2, row = 32 * qd + lane;
    put_state(S + bhk * D * M, sm + R_S, sm + R_S + STILE, D, M);
    if (threadIdx.x < 64) {
      const float z = threadIdx.x < D ? Z[bhk * D + threadIdx.x] : 0.f;
      zs[threadIdx.x] = z;
      const int any = __any_sync(0xffffffffu, z != 0.f);
      if (lane == 0) s_some[warp] = any;
    }
    sync_compute();
    const bool some = s_some[0] | s_some[1];  // no states: den = 0, whatever q holds
    for (int i = 0; i < nt; ++i) {
      const int k = i & 1, n = (t0 + i) * TC_C + row;
      uint8_t* q = sm + R_Q + k * TILE;
      if (wtu(&bar_in[k], (i >> 1) & 1, 123)) {
        float x[32], f[32], d = 0.f;
        tile_row_cols<32>(q, row, 32 * wg, x);
        phi_cols(x, f, 32 * wg, D);
#pragma unroll
        for (int c = 0; c < 32; ++c) d = fmaf(f[c], zs[32 * wg + c], d);
        s_den[wg][row] = d;
        put_terms(q, sm + R_LO, row, 32 * wg, f);
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_t);
      sync_compute();
      const float d = some ? s_den[0][row] + s_den[1][row] : 0.f;
      if (wg == 0 && n < N) den[static_cast<long>(bh) * N + n] = d;
      if (wtu(&bar_o, k, 124)) {
        tc_fence_after();
        float f[32];
        tmem_ldn<2>(tm + (static_cast<uint32_t>(32 * qd) << 16) + 32 * wg, f);
        const float e = d != 0.f ? 1.f / d : 0.f;  // no encoder states: zeros
#pragma unroll
        for (int c = 0; c < 32; ++c) f[c] = d != 0.f ? f[c] * e : 0.f;
        tile_put_cols<32>(q, row, 32 * wg, f);
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_free);
      sync_compute();  // s_den is rewritten next
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == W_ISSUE) tmem_dealloc(tm, 64);
}

// ----------------------------------------------------------- dq, R and r
constexpr int Q_STAGE = 2 * TILE;  // q (then e phi(q)'s first term, then dq), dout
constexpr int Q_LO = 2 * Q_STAGE, Q_S = Q_LO + TILE;
constexpr int Q_SMEM = Q_S + 2 * STILE + 1024;

__global__ void __launch_bounds__(NT, 2)
    k_grad_q(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
             const __grid_constant__ CUtensorMap md, const float* __restrict__ den, const float* __restrict__ S,
             const float* __restrict__ Z, float* __restrict__ rec, int H, int Hk, int N, int D, int M, int per, int* err) {
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = align1024(smraw);
  __shared__ uint64_t bar_in[2], bar_s, bar_1, bar_t, bar_2, bar_free;
  __shared__ float zs[64], s_dot[2][128], s_r[4][64];
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bh = blockIdx.y;
  const long bhk = static_cast<long>(bh / H) * Hk + bh % H / (H / Hk);
  const int t0 = blockIdx.x * per, nt = min(per, (N + TC_C - 1) / TC_C - t0);
  if (threadIdx.x == 0) {
    for (uint64_t* b : {&bar_in[0], &bar_in[1], &bar_1, &bar_2}) mbar_init(b, 1);
    for (uint64_t* b : {&bar_s, &bar_t, &bar_free}) mbar_init(b, 256);
    fence_barrier_init();
    s_abort = 0;
  }
  enter(&tmem_base, 128, warp == W_ISSUE);
  LA_WAITS()
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base, TR = tm + 64;  // T = dout S^T, R
  if (warp == W_ISSUE) {
    if (lane == 0) {
      int issued = 0;
      auto load = [&](int i) {
        uint8_t* st = sm + (i & 1) * Q_STAGE;
        mbar_arrive_expect_tx(&bar_in[i & 1], 2 * TILE);
        tma_load_3d(st, &mq, &bar_in[i & 1], 0, (t0 + i) * TC_C, bh);
        tma_load_3d(st + TILE, &mg, &bar_in[i & 1], 0, (t0 + i) * TC_C, bh);
        ++issued;
      };
      load(0);
      if (nt > 1) load(1);
      constexpr uint32_t ID_R = idesc_bf16(64, 64, true, true);
      bool ok = wt(&bar_s, 0, 131);  // S is in place
      for (int i = 0; ok && i < nt; ++i) {
        const int k = i & 1;
        const uint32_t st = smem_u32(sm + k * Q_STAGE), g = st + TILE;
        if (!(ok = wt(&bar_in[k], (i >> 1) & 1, 132))) break;
        tc_fence_after();
        mma_terms<1>(tm, g, g, smem_u32(sm + Q_S), smem_u32(sm + Q_S + STILE), false);
        mma_commit(&bar_1);
        if (!(ok = wt(&bar_t, k, 133))) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint64_t da = sdesc(j ? smem_u32(sm + Q_LO) : st, 16, 1024), db = sdesc(g, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) mma_bf16(TR, dadd(da, kk * 2048), dadd(db, kk * 2048), ID_R, i > 0 || j > 0 || kk > 0);
        }
        mma_commit(&bar_2);
        if (!(ok = wt(&bar_free, k, 134))) break;
        tc_fence_after();
        tma_store_3d(&md, sm + k * Q_STAGE, 0, (t0 + i) * TC_C, bh);  // dq has taken q's place
        bulk_commit();
        if (i + 2 < nt) {
          bulk_wait_read();
          load(i + 2);
        }
      }
      mma_commit(&bar_1);  // nothing in flight at exit
      mbar_wait(&bar_1, nt & 1, WAIT_NS);
      drain_loads<2>(bar_in, issued);
      bulk_wait_all();
    }
  } else {
    const int qd = warp & 3, wg = warp >> 2, row = 32 * qd + lane;
    const uint32_t lq = static_cast<uint32_t>(32 * qd) << 16;
    put_state(S + bhk * D * M, sm + Q_S, sm + Q_S + STILE, D, M);
    if (threadIdx.x < 64) zs[threadIdx.x] = threadIdx.x < D ? Z[bhk * D + threadIdx.x] : 0.f;
    fence_proxy_async();
    mbar_arrive(&bar_s);
    float r = 0.f;
    for (int i = 0; i < nt; ++i) {
      const int k = i & 1, n = (t0 + i) * TC_C + row;
      uint8_t* q = sm + k * Q_STAGE;
      const float dn = n < N ? den[static_cast<long>(bh) * N + n] : 0.f;
      const float e = dn != 0.f ? 1.f / dn : 0.f;
      const bool in = wtu(&bar_in[k], (i >> 1) & 1, 135);
      float f[32];  // phi(q)
      uint32_t pos = 0;  // which q are positive
      if (in) {
        float x[32];
        tile_row_cols<32>(q, row, 32 * wg, x);
        phi_cols(x, f, 32 * wg, D);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          pos |= (x[c] > 0.f ? 1u : 0u) << c;
          x[c] = f[c] * e;
        }
        put_terms(q, sm + Q_LO, row, 32 * wg, x);
      }
      fence_proxy_async();
      mbar_arrive(&bar_t);
      float t[32], dot = 0.f;
      const bool got = wtu(&bar_1, k, 136) && in;
      if (got) {
        tc_fence_after();
        tmem_ldn<2>(tm + lq + 32 * wg, t);
#pragma unroll
        for (int c = 0; c < 32; ++c) dot = fmaf(f[c], t[c], dot);
      }
      s_dot[wg][row] = dot;
      sync_compute();
      const float gam = -e * (e * (s_dot[0][row] + s_dot[1][row]));  // (e times e first leaves fp32's range from den = 5e-20 on)
      const bool done = wtu(&bar_2, k, 137);  // the products that read e phi(q) are done
      if (got && done) {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          t[c] = fmaf(e, t[c], gam * zs[32 * wg + c]) * (pos >> c & 1 ? 1.f : f[c]);
          t[c] = dn != 0.f ? t[c] : 0.f;  // no states: zeros, whatever q and dout hold
          f[c] *= gam;
        }
        tile_put_cols<32>(q, row, 32 * wg, t);
        r += column_sums(f, lane);
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_free);
      sync_compute();  // s_dot is rewritten next
    }
    s_r[qd][32 * wg + lane] = r;
    sync_compute();
    float* o = rec + (static_cast<long>(bh) * gridDim.x + blockIdx.x) * (D * M + D);
    if (threadIdx.x < D) o[D * M + threadIdx.x] = s_r[0][threadIdx.x] + s_r[1][threadIdx.x] + s_r[2][threadIdx.x] + s_r[3][threadIdx.x];
    tc_fence_after();
    store_state(TR, o, D, M, qd, wg, lane);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == W_ISSUE) tmem_dealloc(tm, 128);
}

// -------------------------------------------------------------- dk and dv
constexpr int V_STAGE = 2 * TILE;  // k (then phi's first term, then dk), v (then dv)
constexpr int V_LO = 2 * V_STAGE, V_R = V_LO + TILE;
constexpr int V_SMEM = V_R + 2 * STILE + 1024;

__global__ void __launch_bounds__(NT, 2)
    k_grad_k(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
             const __grid_constant__ CUtensorMap mdk, const __grid_constant__ CUtensorMap mdv, const int* __restrict__ lengths,
             const float* __restrict__ R, const float* __restrict__ r, bf16* __restrict__ dk, bf16* __restrict__ dv, int Hk,
             int N, int D, int M, int per, int* err) {
  extern __shared__ uint8_t smraw[];
  uint8_t* sm = align1024(smraw);
  __shared__ uint64_t bar_in[2], bar_s, bar_t, bar_2, bar_free;
  __shared__ float rs[64];
  __shared__ uint32_t tmem_base;
  __shared__ int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bh = blockIdx.y;
  if (threadIdx.x == 0) {
    for (uint64_t* b : {&bar_in[0], &bar_in[1], &bar_2}) mbar_init(b, 1);
    for (uint64_t* b : {&bar_s, &bar_t, &bar_free}) mbar_init(b, 256);
    fence_barrier_init();
    s_abort = 0;
  }
  enter(&tmem_base, 128, warp == W_ISSUE);
  const int L = valid_rows(lengths, bh / Hk, N);
  const int t0 = blockIdx.x * per, t1 = min(t0 + per, (N + TC_C - 1) / TC_C);  // tiles of this block
  const int nt = min(t1, (L + TC_C - 1) / TC_C) - t0;                          // of which hold valid rows
  {  // tiles of rows past the length: zeros
    const int n0 = (t0 + max(nt, 0)) * TC_C, n1 = min(N, t1 * TC_C);
    const long base = static_cast<long>(bh) * N + n0;
    for (int e = threadIdx.x; e < (n1 - n0) * D / 8; e += NT) *reinterpret_cast<uint4*>(dk + base * D + e * 8) = make_uint4(0u, 0u, 0u, 0u);
    for (int e = threadIdx.x; e < (n1 - n0) * M / 8; e += NT) *reinterpret_cast<uint4*>(dv + base * M + e * 8) = make_uint4(0u, 0u, 0u, 0u);
  }
  LA_WAITS()
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = tmem_base;  // v R^T, then phi(k) R at + 64
  if (nt <= 0) {
  } else if (warp == W_ISSUE) {
    if (lane == 0) {
      int issued = 0;
      auto load = [&](int i) {
        uint8_t* st = sm + (i & 1) * V_STAGE;
        mbar_arrive_expect_tx(&bar_in[i & 1], 2 * TILE);
        tma_load_3d(st, &mk, &bar_in[i & 1], 0, (t0 + i) * TC_C, bh);
        tma_load_3d(st + TILE, &mv, &bar_in[i & 1], 0, (t0 + i) * TC_C, bh);
        ++issued;
      };
      load(0);
      if (nt > 1) load(1);
      const uint32_t R0 = smem_u32(sm + V_R), R1 = R0 + STILE;
      bool ok = wt(&bar_s, 0, 141);
      for (int i = 0; ok && i < nt; ++i) {
        const int k = i & 1;
        const uint32_t st = smem_u32(sm + k * V_STAGE);
        if (!(ok = wt(&bar_in[k], (i >> 1) & 1, 142))) break;
        tc_fence_after();
        mma_terms<1>(tm, st + TILE, st + TILE, R0, R1, false);
        if (!(ok = wt(&bar_t, k, 143))) break;
        tc_fence_after();
        mma_terms<2>(tm + 64, st, smem_u32(sm + V_LO), R0, R1, true);
        mma_commit(&bar_2);
        if (!(ok = wt(&bar_free, k, 144))) break;
        tc_fence_after();
        tma_store_3d(&mdk, sm + k * V_STAGE, 0, (t0 + i) * TC_C, bh);
        tma_store_3d(&mdv, sm + k * V_STAGE + TILE, 0, (t0 + i) * TC_C, bh);
        bulk_commit();
        if (i + 2 < nt) {
          bulk_wait_read();
          load(i + 2);
        }
      }
      mma_commit(&bar_2);  // nothing in flight at exit
      mbar_wait(&bar_2, nt & 1, WAIT_NS);
      drain_loads<2>(bar_in, issued);
      bulk_wait_all();
    }
  } else {
    const int qd = warp & 3, wg = warp >> 2, row = 32 * qd + lane;
    const uint32_t lq = static_cast<uint32_t>(32 * qd) << 16;
    put_state(R + static_cast<long>(bh) * D * M, sm + V_R, sm + V_R + STILE, D, M);
    if (threadIdx.x < 64) rs[threadIdx.x] = threadIdx.x < D ? r[static_cast<long>(bh) * D + threadIdx.x] : 0.f;
    fence_proxy_async();
    mbar_arrive(&bar_s);
    sync_compute();
    for (int i = 0; i < nt; ++i) {
      const int k = i & 1;
      const bool live = (t0 + i) * TC_C + row < L;
      uint8_t* st = sm + k * V_STAGE;
      float f[32];
      uint32_t pos = 0;
      if (wtu(&bar_in[k], (i >> 1) & 1, 145)) {
        float x[32];
        tile_row_cols<32>(st, row, 32 * wg, x);
        phi_cols(x, f, 32 * wg, D);
#pragma unroll
        for (int c = 0; c < 32; ++c) pos |= (x[c] > 0.f ? 1u : 0u) << c;
        put_terms(st, sm + V_LO, row, 32 * wg, f);
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_t);
      if (wtu(&bar_2, k, 146)) {
        tc_fence_after();
        float t[32];
        tmem_ldn<2>(tm + lq + 32 * wg, t);
#pragma unroll
        for (int c = 0; c < 32; ++c) t[c] = live ? (t[c] + rs[32 * wg + c]) * (pos >> c & 1 ? 1.f : f[c]) : 0.f;
        tile_put_cols<32>(st, row, 32 * wg, t);
        tmem_ldn<2>(tm + 64 + lq + 32 * wg, t);
#pragma unroll
        for (int c = 0; c < 32; ++c) t[c] = live ? t[c] : 0.f;
        tile_put_cols<32>(st + TILE, row, 32 * wg, t);
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive(&bar_free);
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == W_ISSUE) tmem_dealloc(tm, 128);
}

// ------------------------------------------------------------------ host

// Tiles a block takes in turn: about one wave of the kernel's blocks.  (A tile a
// block and several waves measured the same within the noise and write more
// records.)
struct Walk {
  int per, nseg;
  Walk(int heads, int N, int per_sm) {
    const int tiles = (N + TC_C - 1) / TC_C, slots = per_sm * sm_count();
    per = (int)(((long)heads * tiles + slots - 1) / slots);
    if (per > tiles) per = tiles;
    nseg = (tiles + per - 1) / per;
  }
};

#define LA_TRY_CUDA(x)                     \
  do {                                     \
    const cudaError_t e_ = (x);            \
    if (e_ != cudaSuccess) return e_;      \
  } while (0)

size_t rec_bytes(const CrossShape& s) { return (size_t)(s.D * s.M + s.D) * 4; }

template <typename K>
cudaError_t room(K* k, int bytes) { return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); }

}  // namespace

size_t cross_tc_ws_bytes(const CrossShape& s, bool bwd) {
  if (!bwd) return (size_t)s.B * s.Hk * Walk(s.B * s.Hk, s.Nk, 2).nseg * rec_bytes(s);
  return ((size_t)s.B * s.H * Walk(s.B * s.H, s.Nq, 2).nseg + (size_t)s.B * s.Hk) * rec_bytes(s);
}

cudaError_t cross_fwd_tc(const void* q, const void* k, const void* v, const int* lengths, void* out, float* den, float* S,
                         float* Z, float* ws, const CrossShape& s, cudaStream_t st) {
  const Walk wk(s.B * s.Hk, s.Nk, 2), wq(s.B * s.H, s.Nq, 3);
  CUtensorMap mq, mk, mv, mo;
  if (!make_bf16_map(&mq, q, s.B * s.H, s.Nq, s.D) || !make_bf16_map(&mk, k, s.B * s.Hk, s.Nk, s.D) ||
      !make_bf16_map(&mv, v, s.B * s.Hk, s.Nk, s.M) || !make_bf16_map(&mo, out, s.B * s.H, s.Nq, s.M))
    return cudaErrorInvalidValue;
  int* err = status_word();
  LA_TRY_CUDA(room(k_ksum, K_SMEM));
  LA_TRY_CUDA(room(k_read, R_SMEM));
  LA_TRY_CUDA(launch_pdl(k_ksum, dim3(wk.nseg, s.B * s.Hk), dim3(NT), K_SMEM, st, mk, mv, lengths, ws, s.Hk, s.Nk, s.D, s.M, wk.per, err));
  LA_TRY_CUDA(cross_join(ws, S, Z, s.B * s.Hk, wk.nseg, s, st));
  return launch_pdl(k_read, dim3(wq.nseg, s.B * s.H), dim3(NT), R_SMEM, st, mq, mo, S, Z, den, s.H, s.Hk, s.Nq, s.D, s.M, wq.per, err);
}

cudaError_t cross_bwd_tc(const void* q, const void* k, const void* v, const int* lengths, const float* den, const float* S,
                         const float* Z, const void* dout, void* dq, void* dk, void* dv, float* ws, const CrossShape& s,
                         cudaStream_t st) {
  const Walk wq(s.B * s.H, s.Nq, 2), wk(s.B * s.Hk, s.Nk, 2);
  float* R = ws + (size_t)s.B * s.H * wq.nseg * (s.D * s.M + s.D);
  float* r = R + (size_t)s.B * s.Hk * s.D * s.M;
  CUtensorMap mq, mg, md, mk, mv, mdk, mdv;
  if (!make_bf16_map(&mq, q, s.B * s.H, s.Nq, s.D) || !make_bf16_map(&mg, dout, s.B * s.H, s.Nq, s.M) ||
      !make_bf16_map(&md, dq, s.B * s.H, s.Nq, s.D) || !make_bf16_map(&mk, k, s.B * s.Hk, s.Nk, s.D) ||
      !make_bf16_map(&mv, v, s.B * s.Hk, s.Nk, s.M) || !make_bf16_map(&mdk, dk, s.B * s.Hk, s.Nk, s.D) ||
      !make_bf16_map(&mdv, dv, s.B * s.Hk, s.Nk, s.M))
    return cudaErrorInvalidValue;
  int* err = status_word();
  LA_TRY_CUDA(room(k_grad_q, Q_SMEM));
  LA_TRY_CUDA(room(k_grad_k, V_SMEM));
  LA_TRY_CUDA(launch_pdl(k_grad_q, dim3(wq.nseg, s.B * s.H), dim3(NT), Q_SMEM, st, mq, mg, md, den, S, Z, ws, s.H, s.Hk, s.Nq, s.D, s.M,
                         wq.per, err));
  LA_TRY_CUDA(cross_join(ws, R, r, s.B * s.Hk, wq.nseg * (s.H / s.Hk), s, st));
  return launch_pdl(k_grad_k, dim3(wk.nseg, s.B * s.Hk), dim3(NT), V_SMEM, st, mk, mv, mdk, mdv, lengths, R, r, (bf16*)dk, (bf16*)dv,
                    s.Hk, s.Nk, s.D, s.M, wk.per, err);
}

}  // namespace la
