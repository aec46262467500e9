// Selective state space scan (the data-dependent form of the decayed causal
// recurrence): per batch entry and head, with the state S [D][M],
//   delta_t = softplus(dt_t + dt_bias),  a_t = exp(delta_t A),
//   S_t = a_t S_{t-1} + B_t (delta_t x_t)^T,   y_t = S_t^T C_t + skip x_t,
// B and C shared by the H / G heads of a group.
//
// Chunk form.  With cum_i the sum of delta A over a chunk's rows up to i and
// W_ij = exp(cum_i - cum_j) for j <= i, else 0 (u = delta x),
//   y_i = sum_j W_ij (C_i . B_j) u_j + exp(cum_i) S_prev^T C_i + skip x_i,
//   S_next = exp(cum_end) S_prev + sum_j exp(cum_end - cum_j) B_j u_j^T,
// so every chunk's own sum is formed first, the states are carried over the
// chunks, and then every chunk is independent.  Gradients, with R the gradient
// of the state after the chunk (carried from the last chunk to the first):
//   du_j = sum_i W_ij (C_i . B_j) dy_i + exp(cum_end - cum_j) R^T B_j
//   dB_j = sum_i W_ij (dy_i . u_j) C_i + exp(cum_end - cum_j) R u_j
//   dC_i = sum_j W_ij (dy_i . u_j) B_j + exp(cum_i) S_prev dy_i
//   R_prev = exp(cum_end) R + sum_i exp(cum_i) C_i dy_i^T
// and the gradient of log a_t, which every pair, carry-in and carry-out that
// spans row t feels (G_ij = W_ij (C_i . B_j)(dy_i . u_j)):
//   dl_t = sum_{i>=t, j<t} G_ij + sum_{i>=t} C_i . carry part of dC_i
//        + sum_{j<t} B_j . carry part of dB_j + exp(cum_end) <S_prev, R>.
//
// This file: the fp32 kernels (chunks of 64 rows, FFMA), the carry and the
// reductions both paths use, and the single-row step.  The fp32 chunk kernels
// are bound by the FFMA rate and their shared-memory operands: 4 x 2048 rows, 32
// heads of 64 x 64, forward 380 us, gradients 1018 (8.6 and 21.5 Gflop, 23 and 21 Tflop/s); 2 x 784 rows,
// 8 heads of 32 x 32, 36 and 50 (launches and single-chunk latency).
#include "ffma.cuh"
#include "scan.cuh"

namespace la {
namespace {

using bf16 = __nv_bfloat16;

// The log decays' prefix sums of a chunk in two floats (their difference is what
// an exponential magnifies: in one float it cost 6e-7 in y).
struct Cum {
  float hi[64], lo[64];
  __device__ __forceinline__ float decay(int i, int j) const { return expf((hi[i] - hi[j]) + (lo[i] - lo[j])); }  // j to i
  __device__ __forceinline__ float from_start(int i) const { return expf(hi[i]) * (1.f + lo[i]); }
  __device__ __forceinline__ float to_end(int j) const { return decay(63, j); }
};

// delta, cum and the raw gate's argument of a chunk's 64 rows (rows at or past
// `rows`: delta 0, cum carried on).  Threads 0 .. 63; all must call.
template <typename T>
__device__ __forceinline__ void gates(const T* dt, long lddt, int rows, float bias, float A, float* delta, Cum& cum, float* z) {
  __shared__ double first;
  const int t = threadIdx.x;
  double c = 0;
  if (t < 64) {
    float d = 0.f;
    if (t < rows) {
      const float x = to_f(dt[t * lddt]) + bias;
      if (z != nullptr) z[t] = x;
      d = softplus(x);
    } else if (z != nullptr) {
      z[t] = 0.f;
    }
    delta[t] = d;
    c = warp_prefix((double)d * (double)A);
    if (t == 31) first = c;
  }
  __syncthreads();
  if (t < 64) {
    if (t >= 32) c += first;
    cum.hi[t] = (float)c;
    cum.lo[t] = (float)(c - (double)(float)c);
  }
  __syncthreads();
}

// A chunk's own sums: F[d][m] = sum_j exp(cum_end - cum_j) delta_j B_j x_j^T
// (fwd) and, where rev is given, E[d][m] = sum_i exp(cum_i) C_i dy_i^T, and the
// chunk's log decay.  Grid (nch, BH).
template <int D, int M, typename T>
__global__ void __launch_bounds__(256)
    k_scan_sums(const T* __restrict__ x, const T* __restrict__ dt, const T* __restrict__ A, const T* __restrict__ Bm,
                const T* __restrict__ Cm, const T* __restrict__ bias, const int* __restrict__ lengths,
                const T* __restrict__ dy, float* __restrict__ fwd, float* __restrict__ rev, float* __restrict__ tot,
                ScanShape s) {
  grid_dep_enter();
  extern __shared__ float sm[];
  float* tb = sm;                  // [64][D + 4]
  float* tx = tb + 64 * (D + 4);   // [64][M + 4]
  __shared__ float delta[64];
  __shared__ Cum cum;
  const int c = blockIdx.x, bh = blockIdx.y, b = bh / s.H, h = bh % s.H, g = h / (s.H / s.G);
  const int n0 = c * FT, nch = gridDim.x;
  const int rows = max(0, min(FT, valid_rows(lengths, b, s.N) - n0));
  const long r0 = (long)b * s.N + n0;
  gates(dt + r0 * s.lddt + h, s.lddt, rows, par(bias, h), par(A, h), delta, cum, (float*)nullptr);
  if (threadIdx.x == 0) tot[(long)bh * nch + c] = cum.hi[63];
  const int tx0 = (threadIdx.x & 15) * (M / 16), ty0 = (threadIdx.x >> 4) * (D / 16);
  for (int dir = 0; dir < (rev == nullptr ? 1 : 2); ++dir) {
    Rows<T, D> bu;
    Rows<T, M> xu;
    bu.fetch((dir ? Cm + r0 * s.ldc : Bm + r0 * s.ldb) + g * D, dir ? s.ldc : s.ldb, rows);
    xu.fetch(dir ? dy + (r0 * s.H + h) * M : x + r0 * s.ldx + h * M, dir ? (long)s.H * M : s.ldx, rows);
    bu.put(tb, D + 4, nullptr);
    xu.put(tx, M + 4, nullptr);
    __syncthreads();
    for (int e = threadIdx.x; e < FT * M; e += 256) {
      const int r = e / M;
      tx[r * (M + 4) + e % M] *= dir ? cum.from_start(r) : delta[r] * cum.to_end(r);
    }
    __syncthreads();
    float acc[D / 16][M / 16];
    zero_acc(acc);
    ffma_mm(acc, tb, D + 4, tx, M + 4, FT);
    float* o = (dir ? rev : fwd) + ((long)bh * nch + c) * D * M;
#pragma unroll
    for (int r = 0; r < D / 16; ++r)
#pragma unroll
      for (int q = 0; q < M / 16; ++q) o[(ty0 + r) * M + tx0 + q] = acc[r][q];
    __syncthreads();
  }
}

__device__ __forceinline__ void put4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ float rest(float v) { return v - __bfloat162float(__float2bfloat16_rn(v)); }
__device__ __forceinline__ void put4(bf16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// One thread's chunks c0, c0 + dc, ... (n of them), four values of the state:
// run <- exp(tot) run + p[c], and before that out[c] = run where out is wanted
// (it may be p's own memory) and low[c] = what its rounding to bf16 left.  A chain
// of one fused multiply-add a chunk; the loads run eight chunks ahead of it.
template <typename O>
__device__ __forceinline__ void carry_walk(const float* p, O* out, O* low, const float* tot, long step, int c0, int dc, int n, float4& run) {
  constexpr int U = 8;
  for (int k0 = 0; k0 < n; k0 += U) {
    float4 v[U];
    float e[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (k0 + i < n) {
        const int c = c0 + (k0 + i) * dc;
        v[i] = *reinterpret_cast<const float4*>(p + c * step);
        e[i] = expf(tot[c]);
      }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (k0 + i < n) {
        if (out != nullptr) put4(out + (c0 + (k0 + i) * dc) * step, run);
        if (low != nullptr) put4(low + (c0 + (k0 + i) * dc) * step, make_float4(rest(run.x), rest(run.y), rest(run.z), rest(run.w)));
        run.x = fmaf(e[i], run.x, v[i].x);
        run.y = fmaf(e[i], run.y, v[i].y);
        run.z = fmaf(e[i], run.z, v[i].z);
        run.w = fmaf(e[i], run.w, v[i].w);
      }
  }
}

// The carry over the chunks (scan_carry): cols x segs threads, 4 cols values of one
// state, each thread row one segment of the chunks.  One segment: one walk, 128
// columns a block (32 chunks of 64 heads, DRAM-bound: 9.2 us; four segments of
// eight chunks held in registers, 12.3).  Several, for long sequences: every row
// first walks its own from zero, the starting states follow from those ends, and
// a second walk, its loads from L2, writes (512 chunks of 8 heads: 17 us, in one
// walk 65).
constexpr int CARRY_SEGS = 16;
template <typename O>
__global__ void __launch_bounds__(32 * CARRY_SEGS)
    k_scan_carry(const float* fwd, const float* rev, O* fs, O* rs, O* fl, O* rl, const float* __restrict__ tot, float* __restrict__ S,
                 int nch, int DM, int per) {
  grid_dep_enter();
  __shared__ float4 ends[CARRY_SEGS][32], start[32];
  __shared__ float decay[CARRY_SEGS];
  const int e = (blockIdx.x * blockDim.x + threadIdx.x) * 4, seg = threadIdx.y, segs = blockDim.y;
  const long bh = blockIdx.y, at = bh * nch * DM + e;
  const bool back = blockIdx.z != 0, live = e < DM;
  const float* p = (back ? rev : fwd) + at;
  O *out = (back ? rs : fs) + at, *low = fl == nullptr ? nullptr : (back ? rl : fl) + at;
  const float* tt = tot + bh * nch;
  const int first = seg * per, n = min(per, nch - first), c0 = back ? nch - 1 - first : first, dc = back ? -1 : 1;
  float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
  if (segs > 1) {
    // every segment starts from S and the last one replaces it: read before the barrier
    // (by one thread for all: past 72 registers a block an SM less, 2.5 us of training)
    if (seg == 0) start[threadIdx.x] = S != nullptr && !back && live ? *reinterpret_cast<const float4*>(S + bh * DM + e) : run;
    if (live) carry_walk(p, static_cast<O*>(nullptr), static_cast<O*>(nullptr), tt, DM, c0, dc, n, run);
    ends[seg][threadIdx.x] = run;
    float l = 0.f;
    for (int k = threadIdx.x; k < n; k += 32) l += tt[c0 + k * dc];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (threadIdx.x == 0) decay[seg] = expf(l);
    __syncthreads();
  }
  if (!live) return;
  const float* Sp = S == nullptr || back ? nullptr : S + bh * DM + e;
  const float4* from = segs > 1 ? start + threadIdx.x : reinterpret_cast<const float4*>(Sp);
  run = from != nullptr ? *from : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < seg; ++k) {
    const float f = decay[k];
    const float4 u = ends[k][threadIdx.x];
    run.x = fmaf(f, run.x, u.x), run.y = fmaf(f, run.y, u.y), run.z = fmaf(f, run.z, u.z), run.w = fmaf(f, run.w, u.w);
  }
  carry_walk(p, out, low, tt, DM, c0, dc, n, run);
  if (S != nullptr && !back && seg == segs - 1) *reinterpret_cast<float4*>(S + bh * DM + e) = run;
}

// y of one chunk and head.
template <int D, int M, typename T>
__global__ void __launch_bounds__(256)
    k_scan_out(const T* __restrict__ x, const T* __restrict__ dt, const T* __restrict__ A, const T* __restrict__ Bm,
               const T* __restrict__ Cm, const T* __restrict__ skip, const T* __restrict__ bias,
               const int* __restrict__ lengths, const float* __restrict__ prev, T* __restrict__ y, ScanShape s) {
  grid_dep_enter();
  extern __shared__ float sm[];
  float* ct = sm;                   // C^T [D][FLD]
  float* bt = ct + D * FLD;         // B^T [D][FLD]
  float* xs = bt + D * FLD;         // x   [64][M + 4]
  float* ss = xs + 64 * (M + 4);    // S_prev [D][M + 4]
  float* pt = ss + D * (M + 4);     // P^T [64][FLD]
  __shared__ float delta[64];
  __shared__ Cum cum;
  const int c = blockIdx.x, bh = blockIdx.y, b = bh / s.H, h = bh % s.H, g = h / (s.H / s.G);
  const int n0 = c * FT, nch = gridDim.x;
  const int rows = max(0, min(FT, valid_rows(lengths, b, s.N) - n0));
  const long r0 = (long)b * s.N + n0;
  Rows<T, D> cu, bu;
  Rows<T, M> xu;
  State<D, M, false> su;
  cu.fetch(Cm + r0 * s.ldc + g * D, s.ldc, rows);
  bu.fetch(Bm + r0 * s.ldb + g * D, s.ldb, rows);
  xu.fetch(x + r0 * s.ldx + h * M, s.ldx, rows);
  if (prev != nullptr) su.fetch(prev + ((long)bh * nch + c) * D * M);
  cu.put(nullptr, 0, ct);
  bu.put(nullptr, 0, bt);
  xu.put(xs, M + 4, nullptr);
  if (prev != nullptr) su.put(ss, nullptr);
  gates(dt + r0 * s.lddt + h, s.lddt, rows, par(bias, h), par(A, h), delta, cum, (float*)nullptr);
  const int i0 = (threadIdx.x >> 4) * 4, j0 = (threadIdx.x & 15) * 4, m0 = (threadIdx.x & 15) * (M / 16);
  {
    float a[4][4];
    zero_acc(a);
    ffma_mm(a, ct, FLD, bt, FLD, D);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = i0 + r, j = j0 + q;
        pt[j * FLD + i] = j <= i ? a[r][q] * delta[j] * cum.decay(i, j) : 0.f;
      }
  }
  __syncthreads();
  float acc[4][M / 16];
  zero_acc(acc);
  if (prev != nullptr) {
    ffma_mm(acc, ct, FLD, ss, M + 4, D);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int q = 0; q < M / 16; ++q) acc[r][q] *= cum.from_start(i0 + r);
  }
  ffma_mm(acc, pt, FLD, xs, M + 4, FT);
  const float sk = par(skip, h);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + r;
    if (n0 + i >= s.N) break;
#pragma unroll
    for (int q = 0; q < M / 16; ++q) acc[r][q] = i < rows ? fmaf(sk, xs[i * (M + 4) + m0 + q], acc[r][q]) : 0.f;
    store_cols(y + ((r0 + i) * s.H + h) * M + m0, acc[r]);
  }
}

// A sum in two floats: s + c to about 2^-45 (Knuth's exact addition), in plain
// instructions (fp64 ones took a fifth of k_scan_grad's time).
struct Two {
  float s = 0.f, c = 0.f;
  __device__ __forceinline__ void add(float g) {
    const float t = __fadd_rn(s, g), z = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(g, z)));
    s = t;
  }
  __device__ __forceinline__ void add(float g, float gc) { add(g), c += gc; }
  __device__ __forceinline__ void add_xor(int o) {
    const float u = __shfl_xor_sync(0xffffffffu, s, o), uc = __shfl_xor_sync(0xffffffffu, c, o);
    add(u, uc);
  }
};

// k_scan_grad's shared memory (floats): what the head sizes need, so that two
// blocks share an SM up to 32 x 32 and one above.
template <int D, int M>
struct GradTiles {
  static constexpr int ct = 0, bt = ct + 64 * FLD, cn = bt + D * FLD, bn = cn + 64 * (D + 4), xt = bn + 64 * (D + 4),
                       gt = xt + M * FLD, gn = gt + M * FLD, qn = gn + 64 * (M + 4), rn = qn + 64 * FLD,
                       rt = rn + D * (M + 4), st = rt + M * (D + 4), end = st + M * (D + 4);
};

// Gradients of one chunk and head: dx, ddt, this head's dB and dC (fp32, one
// partial a head) and the chunk's parameter sums.
template <int D, int M, typename T>
__global__ void __launch_bounds__(256)
    k_scan_grad(const T* __restrict__ x, const T* __restrict__ dt, const T* __restrict__ A, const T* __restrict__ Bm,
                const T* __restrict__ Cm, const T* __restrict__ skip, const T* __restrict__ bias,
                const int* __restrict__ lengths, const T* __restrict__ dy, const float* __restrict__ prev,
                const float* __restrict__ next, T* __restrict__ dx, T* __restrict__ ddt, float* __restrict__ pB,
                float* __restrict__ pC, float* __restrict__ pp, ScanShape s) {
  grid_dep_enter();
  extern __shared__ float sm[];
  using L = GradTiles<D, M>;
  float* ct = sm + L::ct;  // C^T, then Q^T
  float* bt = sm + L::bt;  // B^T
  float* cn = sm + L::cn;  // C
  float* bn = sm + L::bn;  // B
  float* xt = sm + L::xt;  // x^T
  float* gt = sm + L::gt;  // dy^T
  float* gn = sm + L::gn;  // dy
  float* qn = sm + L::qn;  // Q, then P
  float* rn = sm + L::rn;  // R
  float* rt = sm + L::rt;  // R^T
  float* st = sm + L::st;  // S_prev^T
  __shared__ Cum cum;
  __shared__ float delta[64], z[64], v[64], w[64], xdu[64], red[8];
  __shared__ float2 rowg[64], colg[8][64];
  __shared__ float s_next[3], s_last;
  const int c = blockIdx.x, bh = blockIdx.y, b = bh / s.H, h = bh % s.H, g = h / (s.H / s.G);
  const int n0 = c * FT, nch = gridDim.x;
  const int rows = max(0, min(FT, valid_rows(lengths, b, s.N) - n0));
  const long r0 = (long)b * s.N + n0;
  Rows<T, D> cu, bu;
  Rows<T, M> xu, gu;
  cu.fetch(Cm + r0 * s.ldc + g * D, s.ldc, rows);
  bu.fetch(Bm + r0 * s.ldb + g * D, s.ldb, rows);
  xu.fetch(x + r0 * s.ldx + h * M, s.ldx, rows);
  gu.fetch(dy + (r0 * s.H + h) * M, (long)s.H * M, rows);
  cu.put(cn, D + 4, ct);
  bu.put(bn, D + 4, bt);
  xu.put(nullptr, 0, xt);
  gu.put(gn, M + 4, gt);
  const float* Sp = prev + ((long)bh * nch + c) * D * M;
  const float* Rp = next + ((long)bh * nch + c) * D * M;
  State<D, M, true> su, ru;
  su.fetch(Sp);
  ru.fetch(Rp);
  su.put(nullptr, st);
  ru.put(rn, rt);
  float sr = 0.f;
  for (int e = threadIdx.x; e < D * M; e += 256) sr = fmaf(Sp[e], Rp[e], sr);
  const float Ah = par(A, h), sk = par(skip, h);
  gates(dt + r0 * s.lddt + h, s.lddt, rows, par(bias, h), Ah, delta, cum, z);
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15, i0 = ty * 4, j0 = tx * 4;
  float p[4][4];  // P, until Q has been read
  {
    float a[4][4], e[4][4];
    zero_acc(a);
    zero_acc(e);
    ffma_mm(a, ct, FLD, bt, FLD, D);
    ffma_mm(e, gt, FLD, xt, FLD, M);
    __syncthreads();  // C^T has been read: Q^T takes its place
    // Row and column sums of the same G are subtracted below: in two floats what they
    // share cancels, in one it left 3e-6 in dA
    Two rs[4], cs[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = i0 + r, j = j0 + q;
        const float wt = j <= i ? cum.decay(i, j) : 0.f;
        p[r][q] = wt * a[r][q];
        const float qq = wt * delta[j] * e[r][q];
        qn[i * FLD + j] = qq;
        ct[j * FLD + i] = qq;
        const float gg = j < i ? __fmul_rn(qq, a[r][q]) : 0.f;  // a pair with itself feels no decay
        rs[r].add(gg);
        cs[q].add(gg);
      }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) rs[r].add_xor(o);
      if (tx == 0) rowg[i0 + r] = make_float2(rs[r].s, rs[r].c);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      cs[q].add_xor(16);
      if ((ty & 1) == 0) colg[ty >> 1][j0 + q] = make_float2(cs[q].s, cs[q].c);
    }
  }
  __syncthreads();
  const long prow = (r0 * s.H + h) * D;  // this head's partial of row n0
  {
    // dC
    constexpr int CC = D / 16;
    const int d0 = tx * CC;
    float acc[4][CC];
    zero_acc(acc);
    ffma_mm(acc, gt, FLD, st, D + 4, M);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float f = cum.from_start(i0 + r);
      float t = 0.f;
#pragma unroll
      for (int q = 0; q < CC; ++q) {
        acc[r][q] *= f;
        t = fmaf(acc[r][q], cn[(i0 + r) * (D + 4) + d0 + q], t);
      }
      t = row_sum(t);
      if (tx == 0) v[i0 + r] = t;
    }
    ffma_mm(acc, ct, FLD, bn, D + 4, FT);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n0 + i0 + r < s.N) store_cols(pC + prow + (long)(i0 + r) * s.H * D + d0, acc[r]);
    // dB
    zero_acc(acc);
    ffma_mm(acc, xt, FLD, rt, D + 4, M);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float f = delta[i0 + r] * cum.to_end(i0 + r);
      float t = 0.f;
#pragma unroll
      for (int q = 0; q < CC; ++q) {
        acc[r][q] *= f;
        t = fmaf(acc[r][q], bn[(i0 + r) * (D + 4) + d0 + q], t);
      }
      t = row_sum(t);
      if (tx == 0) w[i0 + r] = t;
    }
    ffma_mm(acc, qn, FLD, cn, D + 4, FT);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n0 + i0 + r < s.N) store_cols(pB + prow + (long)(i0 + r) * s.H * D + d0, acc[r]);
  }
  __syncthreads();  // Q has been read: P takes its place
#pragma unroll
  for (int r = 0; r < 4; ++r) *reinterpret_cast<float4*>(qn + (i0 + r) * FLD + j0) = make_float4(p[r][0], p[r][1], p[r][2], p[r][3]);
  __syncthreads();
  float dskip = 0.f;
  {
    // dx
    constexpr int CC = M / 16;
    const int m0 = tx * CC;
    float acc[4][CC];
    zero_acc(acc);
    ffma_mm(acc, bt, FLD, rn, M + 4, D);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int q = 0; q < CC; ++q) acc[r][q] *= cum.to_end(i0 + r);
    ffma_mm(acc, qn, FLD, gn, M + 4, FT);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int j = i0 + r;
      float t = 0.f;
#pragma unroll
      for (int q = 0; q < CC; ++q) {
        const float xv = xt[(m0 + q) * FLD + j], gv = gn[j * (M + 4) + m0 + q];
        t = fmaf(acc[r][q], xv, t);
        dskip = fmaf(gv, xv, dskip);
        acc[r][q] = fmaf(acc[r][q], delta[j], sk * gv);
      }
      t = row_sum(t);
      if (tx == 0) xdu[j] = t;
      if (n0 + j < s.N) store_cols(dx + ((r0 + j) * s.H + h) * M + m0, acc[r]);
    }
  }
  sr = block_sum(sr, red);
  dskip = block_sum(dskip, red);
  // dl: sums over the rows from t on, and over those before t
  const int t = threadIdx.x, lane = t & 31;
  Two pairs;
  float from = 0.f, upto = 0.f, before = 0.f;
  if (t < 64) {
    pairs.add(rowg[t].x, rowg[t].y);
#pragma unroll
    for (int q = 0; q < 8; ++q) pairs.add(-colg[q][t].x, -colg[q][t].y);
    from = v[t];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float ps = __shfl_down_sync(0xffffffffu, pairs.s, o), pc = __shfl_down_sync(0xffffffffu, pairs.c, o);
      const float f = __shfl_down_sync(0xffffffffu, from, o);
      if (lane + o < 32) pairs.add(ps, pc), from += f;
    }
    upto = warp_prefix(w[t]);
    before = __shfl_up_sync(0xffffffffu, upto, 1);
    if (lane == 0) before = 0.f;
    if (t == 31) s_last = upto;
    if (t == 32) s_next[0] = pairs.s, s_next[1] = pairs.c, s_next[2] = from;
  }
  __syncthreads();
  float dA = 0.f, db = 0.f;
  if (t < 64) {
    if (t < 32)
      pairs.add(s_next[0], s_next[1]), from += s_next[2];
    else
      before += s_last;
    const float dl = fmaf(cum.from_start(63), sr, from + before) + (pairs.s + pairs.c);
    const float dd = xdu[t] + Ah * dl;
    const float dz = t < rows ? dd / (1.f + expf(-z[t])) : 0.f;
    if (n0 + t < s.N) ddt[(r0 + t) * s.H + h] = from_f<T>(dz);
    dA = delta[t] * dl;
    db = dz;
  }
  dA = block_sum(dA, red);
  db = block_sum(db, red);
  if (t == 0) {
    float* o = pp + ((long)bh * nch + c) * 3;
    o[0] = dA, o[1] = dskip, o[2] = db;
  }
}

// One head's parameter gradients: a block sums its B x nch chunks in a fixed order.
template <typename T>
__global__ void __launch_bounds__(256)
    k_scan_params(const float* __restrict__ pp, T* dA, T* dskip, T* dbias, int B, int H, int nch) {
  grid_dep_enter();
  __shared__ float red[8];
  const int h = blockIdx.x;
  float a[3] = {0.f, 0.f, 0.f};
  for (long i = threadIdx.x; i < (long)B * nch; i += 256) {
    const float* p = pp + ((i / nch * H + h) * nch + i % nch) * 3;
    a[0] += p[0], a[1] += p[1], a[2] += p[2];
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const float t = block_sum(a[k], red);
    if (threadIdx.x == 0) {
      T* o = k == 0 ? dA : (k == 1 ? dskip : dbias);
      if (o != nullptr) o[h] = from_f<T>(t);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256)
    k_scan_groups(const float* __restrict__ pB, const float* __restrict__ pC, T* __restrict__ dB, T* __restrict__ dC, long n,
                  int pg, int D4) {
  grid_dep_enter();
  const long e = (long)blockIdx.x * 256 + threadIdx.x;
  if (e >= n) return;
  const long row = e / D4;  // (b, n, g)
  const int d = (int)(e % D4);
  const float4* p = reinterpret_cast<const float4*>(blockIdx.y ? pC : pB) + row * pg * D4 + d;
  float4 s = p[0];
  for (int i = 1; i < pg; ++i) {
    const float4 u = p[(long)i * D4];
    s.x += u.x, s.y += u.y, s.z += u.z, s.w += u.w;
  }
  const float f[4] = {s.x, s.y, s.z, s.w};
  store_cols((blockIdx.y ? dC : dB) + e * 4, f);
}

// One row for each stream: the state is read and written once (the traffic
// that bounds the step), the read-out folded into the same pass.  Every thread
// holds float4 columns of rows rg, rg + RG, ... .  8192 states of 64 x 64 (271 MB):
// 43.0 us, 6.3 TB/s; a handful of streams cost a launch.
template <int D, int M, typename T>
__global__ void __launch_bounds__(256)
    k_scan_step(const T* __restrict__ x, const T* __restrict__ dt, const T* __restrict__ A, const T* __restrict__ Bm,
                const T* __restrict__ Cm, const T* __restrict__ skip, const T* __restrict__ bias, float* __restrict__ S,
                T* __restrict__ y, ScanShape s) {
  constexpr int M4 = M / 4, RG = 256 / M4, RPT = (D + RG - 1) / RG;
  __shared__ float sb[D], sc[D], su[M];
  __shared__ float4 red[RG < D ? RG : D][M4];
  const long bh = blockIdx.x;
  const int b = (int)(bh / s.H), h = (int)(bh % s.H), g = h / (s.H / s.G), t = threadIdx.x;
  const int c4 = t % M4, rg = t / M4;
  float4* Sh = reinterpret_cast<float4*>(S + bh * D * M);
  float4 r[RPT];
#pragma unroll
  for (int k = 0; k < RPT; ++k)
    if (rg + k * RG < D) r[k] = Sh[(rg + k * RG) * M4 + c4];
  const float delta = softplus(to_f(dt[(long)b * s.lddt + h]) + par(bias, h));
  const float a = expf(delta * par(A, h));
  if (t < D) {
    sb[t] = to_f(Bm[(long)b * s.ldb + g * D + t]);
    sc[t] = to_f(Cm[(long)b * s.ldc + g * D + t]);
  }
  if (t < M) su[t] = to_f(x[(long)b * s.ldx + h * M + t]);
  __syncthreads();
  float u[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = delta * su[4 * c4 + i];
#pragma unroll
  for (int k = 0; k < RPT; ++k) {
    const int d = rg + k * RG;
    if (d < D) {
      const float bd = sb[d], cd = sc[d];
      r[k].x = fmaf(a, r[k].x, bd * u[0]);
      r[k].y = fmaf(a, r[k].y, bd * u[1]);
      r[k].z = fmaf(a, r[k].z, bd * u[2]);
      r[k].w = fmaf(a, r[k].w, bd * u[3]);
      Sh[d * M4 + c4] = r[k];
      acc[0] = fmaf(cd, r[k].x, acc[0]);
      acc[1] = fmaf(cd, r[k].y, acc[1]);
      acc[2] = fmaf(cd, r[k].z, acc[2]);
      acc[3] = fmaf(cd, r[k].w, acc[3]);
    }
  }
  if (rg < D) red[rg][c4] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  if (t < M) {
    float o = par(skip, h) * su[t];
    for (int k = 0; k < (RG < D ? RG : D); ++k) o += reinterpret_cast<const float*>(red[k])[t];
    y[bh * M + t] = from_f<T>(o);
  }
}

template <typename K>
cudaError_t smem(K* k, size_t bytes) {
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

// The workspace of the fp32 path (bytes from its start).
struct WsCC {
  size_t tot, fwd, rev, pB, pC, pp, end;
  WsCC(const ScanShape& s, bool bwd) {
    const size_t BH = (size_t)s.B * s.H, nch = (s.N + FT - 1) / FT, st = BH * nch * s.D * s.M * 4;
    tot = 0;
    fwd = align16(BH * nch * 4);
    rev = fwd + st;
    end = rev;
    if (bwd) {
      const size_t part = (size_t)s.B * s.N * s.H * s.D * 4;
      pB = rev + st;
      pC = pB + part;
      pp = pC + part;
      end = pp + align16(BH * nch * 12);
    }
  }
};

}  // namespace

#define LA_TRY_CUDA(x)                     \
  do {                                     \
    const cudaError_t e_ = (x);            \
    if (e_ != cudaSuccess) return e_;      \
  } while (0)

size_t scan_cc_ws_bytes(const ScanShape& s, bool bwd) { return WsCC(s, bwd).end; }

template <typename O>
static cudaError_t carry(const float* fwd, const float* rev, O* fs, O* rs, O* fl, O* rl, const float* tot, float* S, int BH, int nch, int DM,
                         cudaStream_t st) {
  const int segs = nch <= 64 ? 1 : CARRY_SEGS, per = (nch + segs - 1) / segs, cols = segs == 1 ? 128 : 32;
  const dim3 grid((DM / 4 + cols - 1) / cols, BH, rev == nullptr ? 1 : 2), block(cols, (nch + per - 1) / per);
  return launch_pdl(k_scan_carry<O>, grid, block, 0, st, fwd, rev, fs, rs, fl, rl, tot, S, nch, DM, per);
}

cudaError_t scan_carry(float* fwd, float* rev, const float* tot, float* S, int BH, int nch, int DM, cudaStream_t st) {
  float* none = nullptr;
  return carry(fwd, rev, fwd, rev, none, none, tot, S, BH, nch, DM, st);
}

cudaError_t scan_carry_bf16(const float* fwd, const float* rev, void* fs, void* rs, void* fl, void* rl, const float* tot,
                            float* S, int BH, int nch, int DM, cudaStream_t st) {
  return carry(fwd, rev, (bf16*)fs, (bf16*)rs, (bf16*)fl, (bf16*)rl, tot, S, BH, nch, DM, st);
}

cudaError_t scan_params(const float* pp, void* dA, void* dskip, void* dbias, const ScanShape& s, int nch, cudaStream_t st) {
  if (s.dtype == 0)
    return launch_pdl(k_scan_params<float>, dim3(s.H), dim3(256), 0, st, pp, (float*)dA, (float*)dskip, (float*)dbias, s.B, s.H, nch);
  return launch_pdl(k_scan_params<bf16>, dim3(s.H), dim3(256), 0, st, pp, (bf16*)dA, (bf16*)dskip, (bf16*)dbias, s.B, s.H, nch);
}

cudaError_t scan_groups(const float* pB, const float* pC, void* dB, void* dC, const ScanShape& s, int pg, cudaStream_t st) {
  const long n = (long)s.B * s.N * s.G * (s.D / 4);
  const dim3 grid((unsigned)((n + 255) / 256), 2);
  if (s.dtype == 0)
    return launch_pdl(k_scan_groups<float>, grid, dim3(256), 0, st, pB, pC, (float*)dB, (float*)dC, n, pg, s.D / 4);
  return launch_pdl(k_scan_groups<bf16>, grid, dim3(256), 0, st, pB, pC, (bf16*)dB, (bf16*)dC, n, pg, s.D / 4);
}

cudaError_t scan_fwd_cc(const ScanIn& a, float* S, void* y, void* ws_, const ScanShape& s, cudaStream_t st) {
  using T = float;
  char* ws = static_cast<char*>(ws_);
  const WsCC w(s, false);
  const int nch = (s.N + FT - 1) / FT, BH = s.B * s.H;
  float *tot = (float*)(ws + w.tot), *fwd = (float*)(ws + w.fwd), *none = nullptr;
  const bool states = nch > 1 || S != nullptr;
  const dim3 grid(nch, BH), block(256);
  const T *x = (const T*)a.x, *dt = (const T*)a.dt, *A = (const T*)a.A, *Bm = (const T*)a.B, *Cm = (const T*)a.C,
          *skip = (const T*)a.skip, *bias = (const T*)a.dt_bias, *dy = nullptr;
  LA_DISPATCH_DM(s.D, s.M, {
    if (states) {
      constexpr size_t b1 = 64 * (D_ + M_ + 8) * 4;
      LA_TRY_CUDA(launch_pdl(k_scan_sums<D_, M_, T>, grid, block, b1, st, x, dt, A, Bm, Cm, bias, a.lengths, dy, fwd, none, tot, s));
      LA_TRY_CUDA(scan_carry(fwd, nullptr, tot, S, BH, nch, D_ * M_, st));
    }
    constexpr size_t b2 = (2 * D_ * FLD + 64 * (M_ + 4) + D_ * (M_ + 4) + 64 * FLD) * 4;
    LA_TRY_CUDA(smem(&k_scan_out<D_, M_, T>, b2));
    return launch_pdl(k_scan_out<D_, M_, T>, grid, block, b2, st, x, dt, A, Bm, Cm, skip, bias, a.lengths,
                      (const float*)(states ? fwd : nullptr), (T*)y, s);
  });
  return cudaErrorInvalidValue;
}

cudaError_t scan_bwd_cc(const ScanIn& a, const void* dy_, const ScanGrads& d, void* ws_, const ScanShape& s, cudaStream_t st) {
  using T = float;
  char* ws = static_cast<char*>(ws_);
  const WsCC w(s, true);
  const int nch = (s.N + FT - 1) / FT, BH = s.B * s.H;
  float *tot = (float*)(ws + w.tot), *fwd = (float*)(ws + w.fwd), *rev = (float*)(ws + w.rev), *pB = (float*)(ws + w.pB),
        *pC = (float*)(ws + w.pC), *pp = (float*)(ws + w.pp);
  const dim3 grid(nch, BH), block(256);
  const T *x = (const T*)a.x, *dt = (const T*)a.dt, *A = (const T*)a.A, *Bm = (const T*)a.B, *Cm = (const T*)a.C,
          *skip = (const T*)a.skip, *bias = (const T*)a.dt_bias, *dy = (const T*)dy_;
  LA_DISPATCH_DM(s.D, s.M, {
    constexpr size_t b1 = 64 * (D_ + M_ + 8) * 4;
    LA_TRY_CUDA(launch_pdl(k_scan_sums<D_, M_, T>, grid, block, b1, st, x, dt, A, Bm, Cm, bias, a.lengths, dy, fwd, rev, tot, s));
    LA_TRY_CUDA(scan_carry(fwd, rev, tot, nullptr, BH, nch, D_ * M_, st));
    constexpr size_t b2 = GradTiles<D_, M_>::end * 4;
    LA_TRY_CUDA(smem(&k_scan_grad<D_, M_, T>, b2));
    LA_TRY_CUDA(launch_pdl(k_scan_grad<D_, M_, T>, grid, block, b2, st, x, dt, A, Bm, Cm, skip, bias, a.lengths, dy,
                           (const float*)fwd, (const float*)rev, (T*)d.x, (T*)d.dt, pB, pC, pp, s));
  });
  LA_TRY_CUDA(scan_groups(pB, pC, d.B, d.C, s, s.H / s.G, st));
  return scan_params(pp, d.A, d.skip, d.dt_bias, s, nch, st);
}

template <typename T>
static cudaError_t step(const ScanIn& a, float* S, void* y, const ScanShape& s, cudaStream_t st) {
  LA_DISPATCH_DM(s.D, s.M, (k_scan_step<D_, M_, T><<<s.B * s.H, 256, 0, st>>>((const T*)a.x, (const T*)a.dt, (const T*)a.A,
                                                                             (const T*)a.B, (const T*)a.C, (const T*)a.skip,
                                                                             (const T*)a.dt_bias, S, (T*)y, s)));
  return cudaGetLastError();
}

cudaError_t scan_step(const ScanIn& a, float* S, void* y, const ScanShape& s, cudaStream_t st) {
  return s.dtype == 0 ? step<float>(a, S, y, s, st) : step<bf16>(a, S, y, s, st);
}

}  // namespace la
