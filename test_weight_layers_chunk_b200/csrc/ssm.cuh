// Shared pieces of the state-space scan kernels.
//
//   S_t = exp(dt_t A) S_{t-1} + dt_t v_t k_t^T,    y_t = S_t q_t + D v_t
//
// per (batch row, head), S [P][N]; q and k are shared by the heads of a group.
// Over a chunk of Q tokens, with c_t = sum_{s<=t} dt_s A (from the chunk's
// start), the state S at its start and eta_s = dt_s:
//   y_t   = e^{c_t} S q_t + sum_{s<=t} e^{c_t-c_s} eta_s (q_t.k_s) v_s + D v_t
//   S_end = e^{c_Q} S + sum_s e^{c_Q-c_s} eta_s v_s k_s^T
// and, for the gradient X of S_end and dy_t:
//   dS   = e^{c_Q} X + sum_t e^{c_t} dy_t q_t^T
//   dv_s = eta_s (sum_{t>=s} e^{c_t-c_s} (q_t.k_s) dy_t + e^{c_Q-c_s} X k_s) + D dy_s
//   dq_t = sum_{s<=t} e^{c_t-c_s} eta_s (dy_t.v_s) k_s + e^{c_t} S^T dy_t
//   dk_s = sum_{t>=s} e^{c_t-c_s} eta_s (dy_t.v_s) q_t + e^{c_Q-c_s} eta_s X^T v_s
// The gradient of log decay r sums every (source s, reader t) pair whose path
// passes r, with Z_ts = e^{c_t-c_s} eta_s (q_t.k_s) (dy_t.v_s):
//   dl_r = sum_{s<r<=t} Z_ts + sum_{t>=r} e^{c_t} q_t.(S^T dy_t)
//        + sum_{s<r} e^{c_Q-c_s} eta_s k_s.(X^T v_s) + e^{c_Q} <S, X>
// and the sum over s<r<=t is a suffix sum of (row sums - column sums) of Z off
// its diagonal. ddt_r = A dl_r + sum_{t>=r} Z_tr / eta_r + e^{c_Q-c_r} k_r.(X^T v_r).
#pragma once
#include "seq_ops.h"

namespace e2ttt {

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The logarithms c_t in units of log2, each as an fp32 value and what that
// rounding left: c reaches hundreds within a chunk, where one fp32 value would
// be off by 1e-5 while the decay between neighbouring tokens is near one.
struct ChunkLogs {
  float* hi;   // [Q]
  float* lo;   // [Q]
  float* eta;  // [Q]
  __device__ __forceinline__ float decay(int t, int s) const {  // e^{c_t - c_s}
    return ex2((hi[t] - hi[s]) + (lo[t] - lo[s]));
  }
  __device__ __forceinline__ float from_start(int t) const { return ex2(hi[t] + lo[t]); }
  __device__ __forceinline__ float to_end(int s) const {
    return ex2((hi[Q1] - hi[s]) + (lo[Q1] - lo[s]));
  }
  int Q1;  // Q - 1
};

// One warp fills the logs of a chunk of Q <= 128 tokens (a multiple of 32), of
// which the first `n` exist; the others have eta = 0 and change nothing.
__device__ __forceinline__ void fill_chunk_logs(const ChunkLogs& L, const float* dt, float A, int n) {
  const int lane = threadIdx.x & 31, Q = L.Q1 + 1, per = Q / 32;
  const double Al = (double)A * 1.4426950408889634;
  double run[4];
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < per) {
      const int t = lane * per + i;
      const float e = t < n ? dt[t] : 0.f;
      L.eta[t] = e;
      sum += e * Al;
      run[i] = sum;
    }
  }
  double pre = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(~0u, pre, o);
    if (lane >= o) pre += u;
  }
  pre -= sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < per) {
      const int t = lane * per + i;
      const double c = pre + run[i];
      const float h = (float)c;
      L.hi[t] = h;
      L.lo[t] = (float)(c - (double)h);
    }
  }
}

// A chunk's part of dA = sum_r eta_r dl_r, by one warp (lane l has the tokens l K ..
// l K + K - 1), with dl_r = sum_{t>=r} a_t + sum_{s<r} b_s + through. Summed the
// other way round, with E_t = eta_1 + .. + eta_t, it is
//   sum_t a_t E_t + sum_s b_s (E_Q - E_s) + through E_Q,
// in fp64: the chunks' parts cancel to a few hundredths of their size.
template <int K>
__device__ __forceinline__ double decay_gradient(const float (&a)[K], const float (&b)[K], const float* eta,
                                                 float through, int lane) {
  double E[K], run = 0.0;
#pragma unroll
  for (int i = 0; i < K; ++i) E[i] = run += eta[i];
  double pre = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(~0u, pre, o);
    pre += lane >= o ? u : 0.0;
  }
  const double all = __shfl_sync(~0u, pre, 31);
  pre -= run;
  double sum = lane == 0 ? through * all : 0.0;
#pragma unroll
  for (int i = 0; i < K; ++i) sum += a[i] * (pre + E[i]) + b[i] * (all - (pre + E[i]));
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  return sum;
}

__device__ __forceinline__ int ssm_row_length(const int* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

}  // namespace e2ttt
