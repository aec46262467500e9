// Kernelized cross attention: queries of one sequence against the states of
// another, of its own length ("Linear Attention/zh", kernel reformulation, with
// keys and values from an encoder).  Per batch entry and key head,
//   S = sum_{j<L_b} phi(k_j) v_j^T,  Z = sum_{j<L_b} phi(k_j),
// and for each of the H / Hk query heads that share it
//   out_i = S^T phi(q_i) / den_i,  den_i = phi(q_i) . Z;  L_b = 0 gives zeros (of den and
//   the gradients too), whatever q and dout hold.
// Gradients, with e_i = 1 / den_i and gamma_i = -e_i (dout_i . out_i):
//   dphi(q_i) = e_i S dout_i + gamma_i Z,   dout_i . out_i = e_i phi(q_i) . (S dout_i)
//   R = sum_i e_i phi(q_i) dout_i^T,  r = sum_i gamma_i phi(q_i)   (over the query heads too)
//   dphi(k_j) = R v_j + r,   dv_j = R^T phi(k_j),   j < L_b.
// S and Z are what a decoder keeps of its encoder: a single token then reads
// them alone (k_cross_step), whatever the encoder's length.
//
// This file (bf16 prompts and training: cross_tc.cu): the fp32 kernels (64-row
// tiles, FFMA), the sums over partial records, and the single-token read.  The
// fp32 tile kernels are bound by the FFMA rate and their shared-memory operands:
// 16 x 8 query heads (4 key heads) x 512 queries, 2048 states, 64 x 64: forward
// 89 us, gradients 169 (1.6 and 3.2 Gflop, 18 to 19 Tflop/s).
#include "ffma.cuh"
#include "scan.cuh"

namespace la {
namespace {

using bf16 = __nv_bfloat16;

// phi of a natural [64][W] tile in place; rows at or past `rows` become zero.
template <int W>
__device__ __forceinline__ void phi_nat(float* t, int rows) {
  for (int e = threadIdx.x; e < FT * W; e += 256) {
    float& v = t[e / W * (W + 4) + e % W];
    v = e / W < rows ? phi(v) : 0.f;
  }
}

// Partial S and Z of one segment of tiles into rec[bhk][seg] (D M values, then D).
template <int D, int M, typename T>
__global__ void __launch_bounds__(256)
    k_cross_sums(const T* __restrict__ k, const T* __restrict__ v, const int* __restrict__ lengths, float* __restrict__ rec,
                 int Hk, int N, int per) {
  grid_dep_enter();
  extern __shared__ float sm[];
  float* kt = sm;                 // phi(k) [64][D + 4]
  float* vt = kt + 64 * (D + 4);  // v [64][M + 4]
  const int seg = blockIdx.x, bh = blockIdx.y;
  const int L = valid_rows(lengths, bh / Hk, N);
  float acc[D / 16][M / 16], z = 0.f;
  zero_acc(acc);
  for (int c = seg * per; c < (seg + 1) * per; ++c) {
    const int rows = min(FT, L - c * FT);
    if (rows <= 0) break;
    const long r0 = (long)bh * N + (long)c * FT;
    Rows<T, D> ku;
    Rows<T, M> vu;
    __syncthreads();
    ku.fetch(k + r0 * D, D, rows);
    vu.fetch(v + r0 * M, M, rows);
    ku.put(kt, D + 4, nullptr);
    vu.put(vt, M + 4, nullptr);
    __syncthreads();
    phi_nat<D>(kt, rows);
    __syncthreads();
    ffma_mm(acc, kt, D + 4, vt, M + 4, FT);
    if (threadIdx.x < D)
      for (int r = 0; r < FT; ++r) z += kt[r * (D + 4) + threadIdx.x];
  }
  float* o = rec + ((long)bh * gridDim.x + seg) * (D * M + D);
  const int d0 = (threadIdx.x >> 4) * (D / 16), m0 = (threadIdx.x & 15) * (M / 16);
#pragma unroll
  for (int r = 0; r < D / 16; ++r)
#pragma unroll
    for (int q = 0; q < M / 16; ++q) o[(d0 + r) * M + m0 + q] = acc[r][q];
  if (threadIdx.x < D) o[D * M + threadIdx.x] = z;
}

// S and Z (or R and r) of every key head: the sum of its records, in order.  A
// launch of its own (4 to 6 us cold): summing the records in each block that reads
// them, 4 to 13 of them, took longer (bf16 forward 32.8 us against 31.7; fp32, at
// the sizes above and before the tile loads were gathered, 145 against 99).
__global__ void __launch_bounds__(256)
    k_cross_join(const float* __restrict__ rec, float* __restrict__ S, float* __restrict__ Z, int nrec, int DM, int D) {
  grid_dep_enter();
  const int e = (blockIdx.x * 256 + threadIdx.x) * 4;
  const long bh = blockIdx.y;
  if (e >= DM + D) return;
  const float4* p = reinterpret_cast<const float4*>(rec + bh * nrec * (DM + D) + e);
  const long step = (DM + D) / 4;
  float4 s = p[0];
#pragma unroll 8
  for (int i = 1; i < nrec; ++i) {
    const float4 u = p[i * step];
    s.x += u.x, s.y += u.y, s.z += u.z, s.w += u.w;
  }
  *reinterpret_cast<float4*>(e < DM ? S + bh * DM + e : Z + bh * D + (e - DM)) = s;
}

// out and den of 64 queries of one head.
template <int D, int M, typename T>
__global__ void __launch_bounds__(256)
    k_cross_read(const T* __restrict__ q, const float* __restrict__ S, const float* __restrict__ Z, T* __restrict__ out,
                 float* __restrict__ den, int H, int Hk, int N) {
  grid_dep_enter();
  extern __shared__ float sm[];
  float* qt = sm;             // phi(q)^T [D][FLD]
  float* ss = qt + D * FLD;   // S [D][M + 4]
  __shared__ float zs[D], ds[64];
  const int n0 = blockIdx.x * FT, bh = blockIdx.y, rows = min(FT, N - n0);
  const long bhk = (long)(bh / H) * Hk + bh % H / (H / Hk), r0 = (long)bh * N + n0;
  Rows<T, D> qu;
  State<D, M, false> su;
  qu.fetch(q + r0 * D, D, rows);
  su.fetch(S + bhk * D * M);
  qu.put(nullptr, 0, qt);
  su.put(ss, nullptr);
  if (threadIdx.x < D) zs[threadIdx.x] = Z[bhk * D + threadIdx.x];
  __syncthreads();
  for (int e = threadIdx.x; e < D * 64; e += 256) qt[e / 64 * FLD + e % 64] = phi(qt[e / 64 * FLD + e % 64]);
  __syncthreads();
  if (threadIdx.x < 64) {
    float s = 0.f;
    bool some = false;  // no states: Z = 0, and den = 0 whatever q holds
    for (int d = 0; d < D; ++d) s = fmaf(qt[d * FLD + threadIdx.x], zs[d], s), some |= zs[d] != 0.f;
    s = some ? s : 0.f;
    ds[threadIdx.x] = s;
    if (threadIdx.x < rows) den[r0 + threadIdx.x] = s;
  }
  __syncthreads();
  float acc[4][M / 16];
  zero_acc(acc);
  ffma_mm(acc, qt, FLD, ss, M + 4, D);
  const int i0 = (threadIdx.x >> 4) * 4, m0 = (threadIdx.x & 15) * (M / 16);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (i0 + r >= rows) break;
    const float d = ds[i0 + r];
#pragma unroll
    for (int c = 0; c < M / 16; ++c) acc[r][c] = d != 0.f ? acc[r][c] / d : 0.f;
    store_cols(out + (r0 + i0 + r) * M + m0, acc[r]);
  }
}

// dq of a segment of query tiles, and the segment's partial R and r.
template <int D, int M, typename T>
__global__ void __launch_bounds__(256)
    k_cross_grad_q(const T* __restrict__ q, const float* __restrict__ den, const T* __restrict__ dout,
                   const float* __restrict__ S, const float* __restrict__ Z, T* __restrict__ dq,
                   float* __restrict__ rec, int H, int Hk, int N, int per) {
  grid_dep_enter();
  extern __shared__ float sm[];
  float* qn = sm;                   // q, then e phi(q) [64][D + 4]
  float* gt = qn + 64 * (D + 4);    // dout^T [M][FLD]
  float* gn = gt + M * FLD;         // dout [64][M + 4]
  float* st = gn + 64 * (M + 4);    // S^T [M][D + 4]
  __shared__ float zs[D], es[64], gs[64];
  const int seg = blockIdx.x, bh = blockIdx.y;
  const long bhk = (long)(bh / H) * Hk + bh % H / (H / Hk);
  State<D, M, true> su;
  su.fetch(S + bhk * D * M);
  su.put(nullptr, st);
  if (threadIdx.x < D) zs[threadIdx.x] = Z[bhk * D + threadIdx.x];
  float R[D / 16][M / 16], rr = 0.f;
  zero_acc(R);
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  constexpr int CC = D / 16;
  for (int c = seg * per; c < (seg + 1) * per && c * FT < N; ++c) {
    const int rows = min(FT, N - c * FT);
    const long r0 = (long)bh * N + (long)c * FT;
    Rows<T, D> qu;
    Rows<T, M> gu;
    __syncthreads();
    qu.fetch(q + r0 * D, D, rows);
    gu.fetch(dout + r0 * M, M, rows);
    const float d = (threadIdx.x & 63) < rows ? den[r0 + (threadIdx.x & 63)] : 0.f;
    if (d == 0.f) qu.clear(), gu.clear();  // no states: zeros, whatever q and dout hold
    qu.put(qn, D + 4, nullptr);
    gu.put(gn, M + 4, gt);
    if (threadIdx.x < 64) es[threadIdx.x] = d != 0.f ? 1.f / d : 0.f;
    __syncthreads();
    float acc[4][CC];
    zero_acc(acc);
    ffma_mm(acc, gt, FLD, st, D + 4, M);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = ty * 4 + r;
      const float e = es[i];
      // dout_i . out_i = e phi(q_i) . (S dout_i): out itself, rounded, is not read
      float x[CC], f[CC], t = 0.f;
#pragma unroll
      for (int k = 0; k < CC; ++k) {
        x[k] = qn[i * (D + 4) + tx * CC + k];
        f[k] = i < rows ? phi(x[k]) : 0.f;
        t = fmaf(f[k], acc[r][k], t);
      }
      const float g = -e * (e * row_sum(t));  // (e times e first leaves fp32's range from den = 5e-20 on)
      if (tx == 0) gs[i] = g;
#pragma unroll
      for (int k = 0; k < CC; ++k) {
        acc[r][k] = fmaf(e, acc[r][k], g * zs[tx * CC + k]) * (x[k] > 0.f ? 1.f : f[k]);
        qn[i * (D + 4) + tx * CC + k] = f[k];
      }
      if (i < rows) store_cols(dq + (r0 + i) * D + tx * CC, acc[r]);
    }
    __syncthreads();
    if (threadIdx.x < D)
      for (int i = 0; i < FT; ++i) rr = fmaf(gs[i], qn[i * (D + 4) + threadIdx.x], rr);
    __syncthreads();
    for (int e = threadIdx.x; e < FT * D; e += 256) qn[e / D * (D + 4) + e % D] *= es[e / D];
    __syncthreads();
    ffma_mm(R, qn, D + 4, gn, M + 4, FT);
  }
  // records of one key head are neighbours: its query heads' segments in turn
  float* o = rec + ((long)bh * gridDim.x + seg) * (D * M + D);
  const int d0 = ty * (D / 16), m0 = tx * (M / 16);
#pragma unroll
  for (int r = 0; r < D / 16; ++r)
#pragma unroll
    for (int k = 0; k < M / 16; ++k) o[(d0 + r) * M + m0 + k] = R[r][k];
  if (threadIdx.x < D) o[D * M + threadIdx.x] = rr;
}

// dk and dv of 64 encoder states of one key head.
template <int D, int M, typename T>
__global__ void __launch_bounds__(256)
    k_cross_grad_k(const T* __restrict__ k, const T* __restrict__ v, const int* __restrict__ lengths,
                   const float* __restrict__ R, const float* __restrict__ r, T* __restrict__ dk, T* __restrict__ dv, int Hk,
                   int N) {
  grid_dep_enter();
  extern __shared__ float sm[];
  float* kt = sm;                  // k^T, then phi(k)^T [D][FLD]
  float* vt = kt + D * FLD;        // v^T [M][FLD]
  float* rn = vt + M * FLD;        // R [D][M + 4]
  float* rt = rn + D * (M + 4);    // R^T [M][D + 4]
  __shared__ float rs[D];
  const int n0 = blockIdx.x * FT, bh = blockIdx.y;
  const int rows = min(FT, max(0, valid_rows(lengths, bh / Hk, N) - n0));
  const long r0 = (long)bh * N + n0;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  Rows<T, D> ku;
  Rows<T, M> vu;
  State<D, M, true> ru;
  ku.fetch(k + r0 * D, D, rows);
  ku.put(nullptr, 0, kt);
  vu.fetch(v + r0 * M, M, rows);
  vu.put(nullptr, 0, vt);
  ru.fetch(R + (long)bh * D * M);
  ru.put(rn, rt);
  if (threadIdx.x < D) rs[threadIdx.x] = r[(long)bh * D + threadIdx.x];
  __syncthreads();
  constexpr int CK = D / 16, CV = M / 16;
  float acc[4][CK], o[4][CV];
  zero_acc(acc);
  ffma_mm(acc, vt, FLD, rt, D + 4, M);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < CK; ++c) {
      float& kv = kt[(tx * CK + c) * FLD + ty * 4 + i];
      const float x = kv, f = phi(x);
      acc[i][c] = (acc[i][c] + rs[tx * CK + c]) * (x > 0.f ? 1.f : f);
      kv = f;
    }
  __syncthreads();
  zero_acc(o);
  ffma_mm(o, kt, FLD, rn, M + 4, D);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = ty * 4 + i;
    if (n0 + j >= N) break;
    if (j >= rows) {
#pragma unroll
      for (int c = 0; c < CK; ++c) acc[i][c] = 0.f;
#pragma unroll
      for (int c = 0; c < CV; ++c) o[i][c] = 0.f;
    }
    store_cols(dk + (r0 + j) * D + tx * CK, acc[i]);
    store_cols(dv + (r0 + j) * M + tx * CV, o[i]);
  }
}

// One token for each stream: y = S^T phi(q) / phi(q) . Z for the query heads of
// one key head, whose state is read once.  Bound by that read: 16,384 states of
// 64 x 64 (277 MB) in 42.9 us, 6.45 TB/s.
template <int D, int M, typename T>
__global__ void __launch_bounds__(256)
    k_cross_step(const T* __restrict__ q, const float* __restrict__ S, const float* __restrict__ Z, T* __restrict__ y,
                 int per) {
  constexpr int M4 = M / 4, RG = 256 / M4, RPT = (D + RG - 1) / RG, RR = RG < D ? RG : D;
  __shared__ float sq[D], sden[2];
  __shared__ float4 red[RR][M4];
  const long bhk = blockIdx.x;
  const int t = threadIdx.x, c4 = t % M4, rg = t / M4;
  const float4* Sh = reinterpret_cast<const float4*>(S + bhk * D * M);
  float4 r[RPT];
#pragma unroll
  for (int k = 0; k < RPT; ++k)
    if (rg + k * RG < D) r[k] = Sh[(rg + k * RG) * M4 + c4];
  const float z = t < D ? Z[bhk * D + t] : 0.f;
  for (int i = 0; i < per; ++i) {
    const long bh = bhk * per + i;
    float dp = 0.f;
    if (t < D) {
      const float f = phi(to_f(q[bh * D + t]));
      sq[t] = f;
      dp = z != 0.f ? f * z : 0.f;  // Z = 0: den = 0, whatever q holds
    }
    if (t < 64) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dp += __shfl_xor_sync(0xffffffffu, dp, o);
      if ((t & 31) == 0) sden[t >> 5] = dp;
    }
    __syncthreads();
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < RPT; ++k)
      if (rg + k * RG < D) {
        const float f = sq[rg + k * RG];
        a.x = fmaf(f, r[k].x, a.x);
        a.y = fmaf(f, r[k].y, a.y);
        a.z = fmaf(f, r[k].z, a.z);
        a.w = fmaf(f, r[k].w, a.w);
      }
    if (rg < D) red[rg][c4] = a;
    __syncthreads();
    if (t < M) {
      const float den = sden[0] + sden[1];
      float o = 0.f;
#pragma unroll 8
      for (int k = 0; k < RR; ++k) o += reinterpret_cast<const float*>(red[k])[t];
      y[bh * M + t] = from_f<T>(den != 0.f ? o / den : 0.f);
    }
    __syncthreads();
  }
}

template <typename K>
cudaError_t smem(K* k, size_t bytes) {
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// Tiles a block takes in turn: as many blocks as fill the SMs four times over, so
// that a short last wave costs a quarter of what one wave's would.
struct Split {
  int per, nseg;
  Split(int heads, int N, int rows) {
    const int tiles = (N + rows - 1) / rows;
    int want = (4 * sm_count() + heads - 1) / heads;
    want = want < 1 ? 1 : (want > tiles ? tiles : want);
    per = (tiles + want - 1) / want;
    nseg = (tiles + per - 1) / per;
  }
};

size_t rec_bytes(const CrossShape& s) { return (size_t)(s.D * s.M + s.D) * 4; }

#define LA_TRY_CUDA(x)                     \
  do {                                     \
    const cudaError_t e_ = (x);            \
    if (e_ != cudaSuccess) return e_;      \
  } while (0)

}  // namespace

cudaError_t cross_join(const float* rec, float* S, float* Z, int heads, int nrec, const CrossShape& s, cudaStream_t st) {
  const int DM = s.D * s.M;
  return launch_pdl(k_cross_join, dim3(((DM + s.D) / 4 + 255) / 256, heads), dim3(256), 0, st, rec, S, Z, nrec, DM, s.D);
}

namespace {

cudaError_t fwd(const void* q, const void* k, const void* v, const int* lengths, void* out, float* den, float* S, float* Z,
                float* ws, const CrossShape& s, cudaStream_t st) {
  const Split p(s.B * s.Hk, s.Nk, FT);
  LA_DISPATCH_DM(s.D, s.M, {
    constexpr size_t b1 = 64 * (D_ + M_ + 8) * 4;
    LA_TRY_CUDA(launch_pdl(k_cross_sums<D_, M_, float>, dim3(p.nseg, s.B * s.Hk), dim3(256), b1, st, (const float*)k, (const float*)v,
                           lengths, ws, s.Hk, s.Nk, p.per));
    LA_TRY_CUDA(cross_join(ws, S, Z, s.B * s.Hk, p.nseg, s, st));
    constexpr size_t b2 = (D_ * FLD + D_ * (M_ + 4)) * 4;
    LA_TRY_CUDA(launch_pdl(k_cross_read<D_, M_, float>, dim3((s.Nq + FT - 1) / FT, s.B * s.H), dim3(256), b2, st, (const float*)q,
                           (const float*)S, (const float*)Z, (float*)out, den, s.H, s.Hk, s.Nq));
  });
  return cudaGetLastError();
}

cudaError_t bwd(const void* q, const void* k, const void* v, const int* lengths, const float* den,
                const float* S, const float* Z, const void* dout, void* dq, void* dk, void* dv, float* ws,
                const CrossShape& s, cudaStream_t st) {
  const Split p(s.B * s.H, s.Nq, FT);
  float* R = ws + (size_t)s.B * s.H * p.nseg * (s.D * s.M + s.D);
  float* r = R + (size_t)s.B * s.Hk * s.D * s.M;
  LA_DISPATCH_DM(s.D, s.M, {
    constexpr size_t b1 = (64 * (D_ + 4) + M_ * FLD + 64 * (M_ + 4) + M_ * (D_ + 4)) * 4;
    LA_TRY_CUDA(smem(&k_cross_grad_q<D_, M_, float>, b1));
    LA_TRY_CUDA(launch_pdl(k_cross_grad_q<D_, M_, float>, dim3(p.nseg, s.B * s.H), dim3(256), b1, st, (const float*)q, den,
                           (const float*)dout, S, Z, (float*)dq, ws, s.H, s.Hk, s.Nq, p.per));
    LA_TRY_CUDA(cross_join(ws, R, r, s.B * s.Hk, p.nseg * (s.H / s.Hk), s, st));
    constexpr size_t b2 = (D_ * FLD + M_ * FLD + D_ * (M_ + 4) + M_ * (D_ + 4)) * 4;
    LA_TRY_CUDA(smem(&k_cross_grad_k<D_, M_, float>, b2));
    LA_TRY_CUDA(launch_pdl(k_cross_grad_k<D_, M_, float>, dim3((s.Nk + FT - 1) / FT, s.B * s.Hk), dim3(256), b2, st, (const float*)k,
                           (const float*)v, lengths, (const float*)R, (const float*)r, (float*)dk, (float*)dv, s.Hk, s.Nk));
  });
  return cudaGetLastError();
}

template <typename T>
cudaError_t step(const void* q, const float* S, const float* Z, void* y, const CrossShape& s, cudaStream_t st) {
  LA_DISPATCH_DM(s.D, s.M, (k_cross_step<D_, M_, T><<<s.B * s.Hk, 256, 0, st>>>((const T*)q, S, Z, (T*)y, s.H / s.Hk)));
  return cudaGetLastError();
}

}  // namespace

size_t cross_ws_bytes(const CrossShape& s, bool bwd) {
  if (s.dtype != 0) return cross_tc_ws_bytes(s, bwd);
  if (!bwd) return (size_t)s.B * s.Hk * Split(s.B * s.Hk, s.Nk, FT).nseg * rec_bytes(s);
  return ((size_t)s.B * s.H * Split(s.B * s.H, s.Nq, FT).nseg + (size_t)s.B * s.Hk) * rec_bytes(s);
}

cudaError_t cross_fwd(const void* q, const void* k, const void* v, const int* lengths, void* out, float* den, float* S,
                      float* Z, float* ws, const CrossShape& s, cudaStream_t st) {
  return s.dtype == 0 ? fwd(q, k, v, lengths, out, den, S, Z, ws, s, st)
                      : cross_fwd_tc(q, k, v, lengths, out, den, S, Z, ws, s, st);
}

cudaError_t cross_bwd(const void* q, const void* k, const void* v, const int* lengths, const float* den, const float* S,
                      const float* Z, const void* dout, void* dq, void* dk, void* dv, float* ws, const CrossShape& s,
                      cudaStream_t st) {
  return s.dtype == 0 ? bwd(q, k, v, lengths, den, S, Z, dout, dq, dk, dv, ws, s, st)
                      : cross_bwd_tc(q, k, v, lengths, den, S, Z, dout, dq, dk, dv, ws, s, st);
}

cudaError_t cross_step(const void* q, const float* S, const float* Z, void* y, const CrossShape& s, cudaStream_t st) {
  return s.dtype == 0 ? step<float>(q, S, Z, y, s, st) : step<bf16>(q, S, Z, y, s, st);
}

}  // namespace la
