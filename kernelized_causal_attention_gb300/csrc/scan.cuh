// Shared by the convolution's, the scan's and the cross attention's kernels:
// the start of a dependent kernel, the gate, valid rows, the carry and the sums.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "tc_chunk.cuh"

namespace la {

// For kernels launched with launch_pdl: the next kernel may start as blocks
// leave, and nothing before this in the stream is still running once it returns.
__device__ __forceinline__ void grid_dep_enter() {
  tcc::grid_dep_launch();
  tcc::grid_dep_wait();
}

// The same for a kernel that takes tensor memory, by one warp: only once the
// kernel before is done, and the next kernel may start only once every block has
// it.  A block that held tensor memory while it waited for a kernel one of whose
// blocks still asked for some could keep both waiting.
__device__ __forceinline__ void enter(uint32_t* base, uint32_t cols, bool allocates) {
  tcc::grid_dep_wait();
  if (allocates) {
    tc::tmem_alloc(base, cols);
    tcc::grid_dep_launch();
  }
}

// The hardware's base-2 exponential and reciprocal (relative error about 2^-22,
// results below 2^-126 are zero): one instruction each, for values that are
// rounded to bf16 or weigh terms that are.
__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// softplus(x) = log(1 + exp(x)), written so that neither branch overflows.
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

__device__ __forceinline__ int valid_rows(const int* lengths, int b, int N) {
  return lengths == nullptr ? N : min(max(lengths[b], 0), N);
}

// Element h of a per-head parameter vector that may be absent.
template <typename T>
__device__ __forceinline__ float par(const T* p, int h) { return p == nullptr ? 0.f : to_f(p[h]); }

// Inclusive prefix sum over a warp.
template <typename F>
__device__ __forceinline__ F warp_prefix(F v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const F u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The carry over the chunks: fwd (and rev) hold [BH][nch][D M] chunk sums, tot
// [BH][nch] the chunks' log decays.  On return fwd[c] holds the state before
// chunk c and rev[c] the state gradient after it; S, if given, is the state to
// start from and becomes the last one.
cudaError_t scan_carry(float* fwd, float* rev, const float* tot, float* S, int BH, int nch, int DM, cudaStream_t st);
// The same, with the carried states rounded to bf16 into fs (and rs), and what
// that left, rounded, into fl and rl if given.
cudaError_t scan_carry_bf16(const float* fwd, const float* rev, void* fs, void* rs, void* fl, void* rl, const float* tot,
                            float* S, int BH, int nch, int DM, cudaStream_t st);

// Sums the per-chunk parameter gradients pp[BH][nch][3] (A, skip, dt_bias) over
// the batch and the chunks, in a fixed order.
cudaError_t scan_params(const float* pp, void* dA, void* dskip, void* dbias, const ScanShape& s, int nch, cudaStream_t st);

// dB and dC from fp32 partial sums [B N][parts][D] each (parts per group
// neighbouring, parts = G pg): pg partials a value, summed in order.
cudaError_t scan_groups(const float* pB, const float* pC, void* dB, void* dC, const ScanShape& s, int pg, cudaStream_t st);

}  // namespace la
