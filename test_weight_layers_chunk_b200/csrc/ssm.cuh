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

// 2^x to about one unit of fp32, for an exponent in fp64: 2^x = 2^n e^{f ln 2} with n
// the nearest whole number and |f| <= 1/2, by the exponential series to the eighth
// power (what is left out is below 2e-10).
__device__ __forceinline__ float exp2_rounded(double x) {
  x = x < -200.0 ? -200.0 : x > 200.0 ? 200.0 : x;  // 2^x is zero or infinite beyond; a NaN stays one
  const double n = rint(x);
  const float f = (float)(x - n) * 0.69314718055994531f;
  float p = 1.0f / 40320.0f;
  p = fmaf(p, f, 1.0f / 5040.0f);
  p = fmaf(p, f, 1.0f / 720.0f);
  p = fmaf(p, f, 1.0f / 120.0f);
  p = fmaf(p, f, 1.0f / 24.0f);
  p = fmaf(p, f, 1.0f / 6.0f);
  p = fmaf(p, f, 0.5f);
  p = fmaf(p, f, 1.0f);
  p = fmaf(p, f, 1.0f);
  // the exponent in two halves, each within range
  const int e = (int)n, h = e / 2;
  return p * __int_as_float((h + 127) << 23) * __int_as_float((e - h + 127) << 23);
}

// What a chunk's decays are made of, [kLogRows][Q]: the logarithms c_t in units of
// log2, each as an fp32 value and what that rounding left (c reaches hundreds within
// a chunk, where one fp32 value would be off by 1e-5 while the decay between
// neighbouring tokens is near one); eta_t; and, computed from fp64 logarithms since
// the states carry them along the whole row, e^{c_t}, e^{c_Q-c_t}, and e^{c_r-c_t} with r
// the last token of t's block of 32.
constexpr int kLogRows = 6;
struct ChunkLogs {
  float *hi, *lo, *eta, *start, *end, *tail;
  int Q1;  // Q - 1
  __device__ __forceinline__ ChunkLogs(float* p, int Q)
      : hi(p), lo(p + Q), eta(p + 2 * Q), start(p + 3 * Q), end(p + 4 * Q), tail(p + 5 * Q), Q1(Q - 1) {}
  __device__ __forceinline__ float decay(int t, int s) const {  // e^{c_t - c_s}
    return ex2((hi[t] - hi[s]) + (lo[t] - lo[s]));
  }
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
  const double last = __shfl_sync(~0u, pre, 31), block = __shfl_sync(~0u, pre, lane | (32 / per - 1));
  pre -= sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < per) {
      const int t = lane * per + i;
      const double c = pre + run[i];
      const float h = (float)c;
      L.hi[t] = h;
      L.lo[t] = (float)(c - (double)h);
      L.start[t] = exp2_rounded(c);
      L.end[t] = exp2_rounded(last - c);
      L.tail[t] = exp2_rounded(block - c);
    }
  }
}

// A chunk's part of dA = sum_r eta_r dl_r, by one warp (lane l has the tokens l K ..
// l K + K - 1, K = Q / 32). Summed by what passes over r instead, with E_t = eta_1 +
// .. + eta_t, it is
//   sum_{s<t} Z_ts (E_t - E_s) + sum_t in_t E_t + sum_s out_s (E_Q - E_s) + through E_Q
// (in, out: the terms of readers and of sources beside the chunk's own pairs). The
// pairs come as sums over blocks of 32 tokens, rows(c, t) over the sources in block
// c and cols(d, s) over the readers in block d: with E counted from the end of an
// earlier block, or within one from its start, little of them cancels. In fp64, as
// the chunks' parts cancel to a few hundredths of their size.
template <int K, class Rows, class Cols>
__device__ __forceinline__ double decay_gradient(Rows rows, Cols cols, const double (&in)[K],
                                                 const double (&out)[K], const float* eta, double through,
                                                 int lane) {
  constexpr int kLanes = 32 / K;  // lanes of a block
  const int mine = lane / kLanes;
  double E[K], run = 0.0, ends[K];
#pragma unroll
  for (int i = 0; i < K; ++i) E[i] = run += eta[i];
  double pre = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(~0u, pre, o);
    pre += lane >= o ? u : 0.0;
  }
#pragma unroll
  for (int c = 0; c < K; ++c) ends[c] = __shfl_sync(~0u, pre, (c + 1) * kLanes - 1);
  pre -= run;
  double first = 0.0, last = 0.0;
#pragma unroll
  for (int c = 0; c < K; ++c) {
    first = c + 1 == mine ? ends[c] : first;
    last = c == mine ? ends[c] : last;
  }
  double sum = lane == 0 ? through * ends[K - 1] : 0.0;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const double e = pre + E[i];
    sum += in[i] * e + out[i] * (ends[K - 1] - e);
#pragma unroll
    for (int c = 0; c < K; ++c) {
      if (c <= mine) sum += (double)rows(c, i) * (e - (c < mine ? ends[c] : first));
      if (c >= mine) sum += (double)eta[i] * cols(c, i) * (c > mine ? last - e : first - e);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  return sum;
}

__device__ __forceinline__ int ssm_row_length(const int* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

}  // namespace e2ttt
