// State-space scan, fp32 CUDA-core kernels for every size and type, and the
// passes over chunk states that all forms share. The mathematics is in ssm.cuh.
//
// A chunk's work is a handful of small matrix products, done here from shared
// memory by 16 x 16 threads with 4 x 4 results each; chunks meet only in their
// states, which one elementwise pass carries along the tokens.
#include <type_traits>

#include "ssm.cuh"
#include "trace.h"

namespace e2ttt {
namespace {

constexpr int kT = 256;

// acc[i][j] += sum_k A(m_i, k) B(k, n_j), m_i = ty + 16 i, n_j = n0 + tx + 16 j
// clamped to nmax. A at a + m*am + k*ak, B at b + k*bk + n*bn.
template <int R>
__device__ __forceinline__ void tile_mm(float (&acc)[R][4], const float* a, int am, int ak,
                                        const float* b, int bk, int bn, int K, int n0, int nmax) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int no[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) no[j] = min(n0 + tx + 16 * j, nmax) * bn;
  for (int k = 0; k < K; ++k) {
    float x[R], y[4];
#pragma unroll
    for (int i = 0; i < R; ++i) x[i] = a[(ty + 16 * i) * am + k * ak];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = b[k * bk + no[j]];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
  }
}
template <int R>
__device__ __forceinline__ void clear(float (&acc)[R][4]) {
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
}
// Sum over the 16 threads that share ty.
__device__ __forceinline__ float row_sum16(float x) {
#pragma unroll
  for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// rows x cols of src (row pitch `ld`) to dst (row pitch `pitch`), as fp32; rows
// from n on and columns from cols to cpad are zero.
template <typename T>
__device__ __forceinline__ void load_tile(float* dst, int pitch, const T* src, long long ld, int rows,
                                          int n, int cols, int cpad) {
  for (int i = threadIdx.x; i < rows * cpad; i += kT) {
    const int r = i / cpad, c = i - r * cpad;
    dst[r * pitch + c] = r < n && c < cols ? to_f<T>(src[(long long)r * ld + c]) : 0.f;
  }
}

struct Where {
  int b, h, g, pt, c, bh, t0, n, p0, np;
};
__device__ __forceinline__ Where where(const SsmDims& s, const int* lengths) {
  Where w;
  w.bh = blockIdx.y;
  w.b = w.bh / s.H;
  w.h = w.bh - w.b * s.H;
  w.g = w.h / (s.H / s.G);
  w.c = blockIdx.x;
  w.pt = blockIdx.z;
  w.t0 = w.c * s.Q;
  w.n = min(max(ssm_row_length(lengths, w.b, s.T) - w.t0, 0), s.Q);
  w.p0 = w.pt * kSsmPT;
  w.np = min(kSsmPT, s.P - w.p0);
  return w;
}

__device__ __forceinline__ ChunkLogs chunk_logs(float* p, int Q) {
  ChunkLogs L;
  L.hi = p;
  L.lo = p + Q;
  L.eta = p + 2 * Q;
  L.Q1 = Q - 1;
  return L;
}

// states[c][bh] = the chunk's own contribution to its end state
//   REV 0: sum_s e^{c_Q-c_s} eta_s x_s y_s^T  (x = v, y = k)
//   REV 1: sum_t e^{c_t} x_t y_t^T            (x = dy, y = q; the adjoint)
// and decay[c][bh] = e^{c_Q}.
template <typename T, int REV>
__global__ void __launch_bounds__(kT)
    chunk_state_kernel(SsmDims s, const T* __restrict__ x, const T* __restrict__ y,
                       const float* __restrict__ dt, const float* __restrict__ A,
                       const int* __restrict__ lengths, float* __restrict__ states,
                       float* __restrict__ decay, int* __restrict__ status) {
  extern __shared__ float sm[];
  const Where w = where(s, lengths);
  if (blockIdx.x + blockIdx.y + blockIdx.z + threadIdx.x == 0) *status = 0;  // nothing here waits
  const int Q = s.Q, N = s.N, XP = kSsmPT + 1, NP = N + 1;
  const ChunkLogs L = chunk_logs(sm, Q);
  float* xs = sm + 3 * Q;
  float* ys = xs + Q * XP;
  if (threadIdx.x < 32) fill_chunk_logs(L, dt + (long long)w.bh * s.T + w.t0, A[w.h], w.n);
  load_tile<T>(ys, NP, y + (((long long)w.b * s.G + w.g) * s.T + w.t0) * N, N, Q, w.n, N, N);
  load_tile<T>(xs, XP, x + ((long long)w.bh * s.T + w.t0) * s.P + w.p0, s.P, Q, w.n, w.np, kSsmPT);
  __syncthreads();
  for (int i = threadIdx.x; i < Q * kSsmPT; i += kT) {
    const int t = i / kSsmPT, p = i - t * kSsmPT;
    xs[t * XP + p] *= REV ? L.from_start(t) : L.to_end(t) * L.eta[t];
  }
  if (threadIdx.x == 0 && w.pt == 0)
    decay[(long long)w.c * s.B * s.H + w.bh] = L.from_start(Q - 1);
  __syncthreads();
  float* out = states + (((long long)w.c * s.B * s.H + w.bh) * s.P + w.p0) * N;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int n0 = 0; n0 < N; n0 += 64) {
    float acc[4][4];
    clear(acc);
    tile_mm<4>(acc, xs, 1, XP, ys, NP, 1, Q, n0, N - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = ty + 16 * i, n = n0 + tx + 16 * j;
        if (p < w.np && n < N) out[(long long)p * N + n] = acc[i][j];
      }
  }
}

// Turns the chunks' own contributions into the states at their starts (REV 0,
// from `first`) or the gradients at their ends (REV 1, from the last chunk
// back); `last` gets what is left after the last one. `copy`, where given, takes
// them rounded to bf16 (what the outputs' products read), and without `keep` the
// fp32 ones are not written. Elementwise along the chunks, bound by the states'
// bytes; V is float4 where rows and pointers allow.
__device__ __forceinline__ void store_bf16(bf16* p, float x) { *p = from_f<bf16>(x); }
__device__ __forceinline__ void store_bf16(bf16* p, const float4& x) {
  __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  *reinterpret_cast<uint2*>(p) = uint2{*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b)};
}
__device__ __forceinline__ void decay_add(float& run, float d, float own) { run = fmaf(d, run, own); }
__device__ __forceinline__ void decay_add(float4& run, float d, const float4& own) {
  run = float4{fmaf(d, run.x, own.x), fmaf(d, run.y, own.y), fmaf(d, run.z, own.z), fmaf(d, run.w, own.w)};
}
constexpr int kCarryBatch = 8;  // chunks whose loads are in flight together
template <typename V, int REV>
__global__ void __launch_bounds__(kT)
    carry_kernel(int NC, int BH, long long PN, const V* __restrict__ first,
                 const float* __restrict__ decay, V* __restrict__ states, V* __restrict__ last,
                 bf16* __restrict__ copy, bool keep) {
  constexpr int W = sizeof(V) / sizeof(float);
  const int bh = blockIdx.y;
  const long long i = (long long)blockIdx.x * kT + threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  if (i >= PN) return;
  V run = first ? first[bh * PN + i] : V{};
  constexpr int U = kCarryBatch;
  for (int c0 = 0; c0 < NC; c0 += U) {
    V own[U];
    float d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = REV ? NC - 1 - (c0 + u) : c0 + u;
      if (c0 + u < NC) {
        own[u] = __ldcs(states + ((long long)c * BH + bh) * PN + i);
        d[u] = decay[(long long)c * BH + bh];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = REV ? NC - 1 - (c0 + u) : c0 + u;
      if (c0 + u < NC) {
        const long long at = ((long long)c * BH + bh) * PN + i;
        if (keep) __stcs(states + at, run);
        if (copy) store_bf16(copy + at * W, run);
        decay_add(run, d[u], own[u]);
      }
    }
  }
  if (last) last[bh * PN + i] = run;
}

// y of one chunk from the state at its start.
template <typename T, int R>  // R = Q / 16
__global__ void __launch_bounds__(kT)
    chunk_out_kernel(SsmDims s, const T* __restrict__ q, const T* __restrict__ k,
                     const T* __restrict__ v, const float* __restrict__ dt,
                     const float* __restrict__ A, const float* __restrict__ D,
                     const int* __restrict__ lengths, const float* __restrict__ states,
                     T* __restrict__ y) {
  extern __shared__ float sm[];
  const Where w = where(s, lengths);
  const int Q = s.Q, N = s.N, XP = kSsmPT + 1, NP = N + 1, QP = Q + 1;
  const ChunkLogs L = chunk_logs(sm, Q);
  float* qs = sm + 3 * Q;
  float* ks = qs + Q * NP;  // then the state [PT][NP]
  float* xs = ks + (Q > kSsmPT ? Q : kSsmPT) * NP;
  float* ws = xs + Q * XP;
  if (threadIdx.x < 32) fill_chunk_logs(L, dt + (long long)w.bh * s.T + w.t0, A[w.h], w.n);
  const long long qo = (((long long)w.b * s.G + w.g) * s.T + w.t0) * N;
  load_tile<T>(qs, NP, q + qo, N, Q, w.n, N, N);
  load_tile<T>(ks, NP, k + qo, N, Q, w.n, N, N);
  load_tile<T>(xs, XP, v + ((long long)w.bh * s.T + w.t0) * s.P + w.p0, s.P, Q, w.n, w.np, kSsmPT);
  __syncthreads();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[R][4];
  clear(acc);
  tile_mm<R>(acc, qs, NP, 1, ks, 1, NP, N, 0, Q - 1);
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = ty + 16 * i, u = tx + 16 * j;
      if (u < Q) ws[t * QP + u] = u <= t ? acc[i][j] * L.decay(t, u) * L.eta[u] : 0.f;
    }
  __syncthreads();
  load_tile<float>(ks, NP, states + (((long long)w.c * s.B * s.H + w.bh) * s.P + w.p0) * N, N, kSsmPT,
                   w.np, N, N);
  __syncthreads();
  clear(acc);
  tile_mm<R>(acc, qs, NP, 1, ks, 1, NP, N, 0, kSsmPT - 1);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float f = L.from_start(ty + 16 * i);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] *= f;
  }
  tile_mm<R>(acc, ws, QP, 1, xs, XP, 1, Q, 0, kSsmPT - 1);
  const float Dh = D ? D[w.h] : 0.f;
  T* out = y + ((long long)w.bh * s.T + w.t0) * s.P + w.p0;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = ty + 16 * i, p = tx + 16 * j;
      if (w.t0 + t < s.T && p < w.np)
        out[(long long)t * s.P + p] =
            from_f<T>(t < w.n ? fmaf(Dh, xs[t * XP + p], acc[i][j]) : 0.f);
    }
}

// Sum over the block to thread 0, in a fixed order.
__device__ __forceinline__ float block_sum0(float x, float* scratch) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.f;
  if (threadIdx.x == 0)
    for (int i = 0; i < kT / 32; ++i) x += scratch[i];
  return x;
}

// All gradients of one chunk from the state at its start and the gradient of the
// state at its end. dq, dk per head and tile of state rows (fp32 partial sums
// [B*H*NPT][T][N]), ddt per tile ([NPT][B*H][T]), dA and dD per chunk and tile
// ([NC][NPT][B*H]).
template <typename T, int R>
__global__ void __launch_bounds__(kT)
    chunk_grad_kernel(SsmDims s, const T* __restrict__ q, const T* __restrict__ k,
                      const T* __restrict__ v, const float* __restrict__ dt,
                      const float* __restrict__ A, const float* __restrict__ D,
                      const int* __restrict__ lengths, const float* __restrict__ states,
                      const float* __restrict__ ends, const T* __restrict__ dy,
                      float* __restrict__ dqp, float* __restrict__ dkp, T* __restrict__ dv,
                      float* __restrict__ ddtp, float* __restrict__ dAp, float* __restrict__ dDp) {
  extern __shared__ float sm[];
  const Where w = where(s, lengths);
  const int Q = s.Q, N = s.N, XP = kSsmPT + 1, NP = N + 1, QP = Q + 1;
  const ChunkLogs L = chunk_logs(sm, Q);
  float* dots = sm + 3 * Q;  // [6][Q]: row sums, column sums, readers', sources', deta, K's diagonal
  float* scratch = dots + 6 * Q;
  float* qs = scratch + 16;
  float* ks = qs + Q * NP;
  float* Ss = ks + Q * NP;
  float* Xs = Ss + kSsmPT * NP;
  float* xs = Xs + kSsmPT * NP;
  float* gs = xs + Q * XP;
  float* Ws = gs + Q * XP;  // e^{c_t-c_s} (q_t.k_s)
  float* Ks = Ws + Q * QP;  // e^{c_t-c_s} eta_s (dy_t.v_s)
  float* cz = Ks + Q * QP;  // [2][16][Q]: column sums by thread row, of Z off its diagonal and of deta
  if (threadIdx.x < 32) fill_chunk_logs(L, dt + (long long)w.bh * s.T + w.t0, A[w.h], w.n);
  const long long qo = (((long long)w.b * s.G + w.g) * s.T + w.t0) * N;
  const long long vo = ((long long)w.bh * s.T + w.t0) * s.P + w.p0;
  const long long so = (((long long)w.c * s.B * s.H + w.bh) * s.P + w.p0) * N;
  load_tile<T>(qs, NP, q + qo, N, Q, w.n, N, N);
  load_tile<T>(ks, NP, k + qo, N, Q, w.n, N, N);
  load_tile<T>(xs, XP, v + vo, s.P, Q, w.n, w.np, kSsmPT);
  load_tile<T>(gs, XP, dy + vo, s.P, Q, w.n, w.np, kSsmPT);
  load_tile<float>(Ss, NP, states + so, N, kSsmPT, w.np, N, N);
  load_tile<float>(Xs, NP, ends + so, N, kSsmPT, w.np, N, N);
  __syncthreads();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  {
    float m[R][4], kk[R][4];
    clear(m);
    clear(kk);
    tile_mm<R>(m, qs, NP, 1, ks, 1, NP, N, 0, Q - 1);
    tile_mm<R>(kk, gs, XP, 1, xs, 1, XP, kSsmPT, 0, Q - 1);
    float colz[4] = {}, cold[4] = {};
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int t = ty + 16 * i;
      float rows = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int u = tx + 16 * j;
        if (u >= Q) continue;
        const float e = u <= t ? L.decay(t, u) : 0.f;
        const float a = u <= t ? e * m[i][j] : 0.f;
        const float b = u <= t ? e * L.eta[u] * kk[i][j] : 0.f;
        Ws[t * QP + u] = a;
        Ks[t * QP + u] = b;
        const float r = a * kk[i][j], z = u < t ? r * L.eta[u] : 0.f;
        rows += z;
        colz[j] += z;
        cold[j] += r;
        if (u == t) dots[5 * Q + t] = kk[i][j];
      }
      rows = row_sum16(rows);
      if (tx == 0) dots[t] = rows;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int u = tx + 16 * j;
      if (u >= Q) continue;
      cz[ty * Q + u] = colz[j];
      cz[(16 + ty) * Q + u] = cold[j];
    }
  }
  __syncthreads();
  for (int u = threadIdx.x; u < Q; u += kT) {
    float z = 0.f, de = 0.f;
    for (int i = 0; i < 16; ++i) {
      z += cz[i * Q + u];
      de += cz[(16 + i) * Q + u];
    }
    dots[Q + u] = z;
    dots[4 * Q + u] = de;
  }
  // dv
  {
    float acc[R][4];
    clear(acc);
    tile_mm<R>(acc, ks, NP, 1, Xs, 1, NP, N, 0, kSsmPT - 1);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float f = L.to_end(ty + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] *= f;
    }
    tile_mm<R>(acc, Ws, 1, QP, gs, XP, 1, Q, 0, kSsmPT - 1);
    const float Dh = D ? D[w.h] : 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = ty + 16 * i, p = tx + 16 * j;
        if (w.t0 + t < s.T && p < w.np)
          dv[vo + (long long)t * s.P + p] =
              from_f<T>(t < w.n ? fmaf(L.eta[t], acc[i][j], Dh * gs[t * XP + p]) : 0.f);
      }
  }
  // dq, dk and the dots of their state parts
  const long long po = (((long long)w.bh * s.NPT + w.pt) * s.T + w.t0) * N;
  float rd[R], sd[R];
#pragma unroll
  for (int i = 0; i < R; ++i) rd[i] = sd[i] = 0.f;
  for (int n0 = 0; n0 < N; n0 += 64) {
    float acc[R][4];
    clear(acc);
    tile_mm<R>(acc, gs, XP, 1, Ss, NP, 1, kSsmPT, n0, N - 1);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int t = ty + 16 * i;
      const float f = L.from_start(t);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx + 16 * j;
        acc[i][j] *= f;
        if (n < N) rd[i] = fmaf(acc[i][j], qs[t * NP + n], rd[i]);
      }
    }
    tile_mm<R>(acc, Ks, QP, 1, ks, NP, 1, Q, n0, N - 1);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = ty + 16 * i, n = n0 + tx + 16 * j;
        if (w.t0 + t < s.T && n < N) dqp[po + (long long)t * N + n] = t < w.n ? acc[i][j] : 0.f;
      }
    clear(acc);
    tile_mm<R>(acc, xs, XP, 1, Xs, NP, 1, kSsmPT, n0, N - 1);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int t = ty + 16 * i;
      const float f = L.to_end(t);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx + 16 * j;
        acc[i][j] *= f;
        if (n < N) sd[i] = fmaf(acc[i][j], ks[t * NP + n], sd[i]);
        acc[i][j] *= L.eta[t];
      }
    }
    tile_mm<R>(acc, Ks, 1, QP, qs, NP, 1, Q, n0, N - 1);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = ty + 16 * i, n = n0 + tx + 16 * j;
        if (w.t0 + t < s.T && n < N) dkp[po + (long long)t * N + n] = t < w.n ? acc[i][j] : 0.f;
      }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float a = row_sum16(rd[i]), b = row_sum16(sd[i]);
    if (tx == 0) {
      dots[2 * Q + ty + 16 * i] = a;
      dots[3 * Q + ty + 16 * i] = b;
    }
  }
  // e^{c_Q} <S, X>
  float ip = 0.f;
  for (int i = threadIdx.x; i < kSsmPT * N; i += kT) {
    const int p = i / N, n = i - p * N;
    ip = fmaf(Ss[p * NP + n], Xs[p * NP + n], ip);
  }
  ip = block_sum0(ip, scratch);
  if (threadIdx.x == 0) {
    const float* rows = dots;
    const float *cols = dots + Q, *rdr = dots + 2 * Q, *src = dots + 3 * Q, *de = dots + 4 * Q,
                *kd = dots + 5 * Q;
    const double through = (double)L.from_start(Q - 1) * ip;
    double before = 0.0;  // sources before r, read after the chunk
    for (int r = 0; r < Q; ++r) before += (double)L.eta[r] * src[r];
    double after = 0.0, dA = 0.0, dD = 0.0;
    const float Ah = A[w.h];
    float* out = ddtp + ((long long)w.pt * s.B * s.H + w.bh) * s.T + w.t0;
    for (int r = Q - 1; r >= 0; --r) {
      before -= (double)L.eta[r] * src[r];
      after += (double)rows[r] - cols[r] + rdr[r];
      const double dl = after + before + through;
      dA += L.eta[r] * dl;
      dD += kd[r];
      if (w.t0 + r < s.T) out[r] = r < w.n ? (float)(Ah * dl + de[r] + src[r]) : 0.f;
    }
    const long long o = ((long long)w.c * s.NPT + w.pt) * s.B * s.H + w.bh;
    dAp[o] = (float)dA;
    dDp[o] = (float)dD;
  }
}

// out[b][g][i] = sum over the group's parts, in order: dq (blockIdx.z 0) and dk
// (1), V values at a time; the blocks of blockIdx.z 2 take dA and dD.
template <typename T, int V>
__device__ __forceinline__ void group_sum(const float* part, int parts, long long row, T* out) {
  const long long i = ((long long)blockIdx.x * kT + threadIdx.x) * V;
  if (i >= row) return;
  const float* p = part + (long long)blockIdx.y * parts * row + i;
  float a[V] = {};
#pragma unroll 8
  for (int j = 0; j < parts; ++j) {
    float x[V];
    if constexpr (V == 4) {
      const float4 f = __ldcs(reinterpret_cast<const float4*>(p));
      x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
    } else {
      x[0] = *p;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) a[e] += x[e];
    p += row;
  }
  T* o = out + (long long)blockIdx.y * row + i;
  if constexpr (V == 4 && sizeof(T) == 2) {
    store_bf16(reinterpret_cast<bf16*>(o), float4{a[0], a[1], a[2], a[3]});
  } else if constexpr (V == 4) {
    *reinterpret_cast<float4*>(o) = float4{a[0], a[1], a[2], a[3]};
  } else {
    *o = from_f<T>(a[0]);
  }
}
// dA[h], dD[h]: sums of part [rows][H], one block per head, in a fixed order.
__device__ void head_sum(const float* dAp, const float* dDp, int rows, int H, int h, float* dA, float* dD) {
  __shared__ double s[2][kT / 32];
  double a[2] = {0.0, 0.0};
  for (int i = threadIdx.x; i < rows; i += kT) {
    a[0] += dAp[(long long)i * H + h];
    a[1] += dDp[(long long)i * H + h];
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
#pragma unroll
    for (int o = 16; o; o >>= 1) a[w] += __shfl_xor_sync(~0u, a[w], o);
    if ((threadIdx.x & 31) == 0) s[w][threadIdx.x >> 5] = a[w];
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    double sum = 0.0;
    for (int i = 0; i < kT / 32; ++i) sum += s[threadIdx.x][i];
    float* out = threadIdx.x ? dD : dA;
    if (out) out[h] = (float)sum;
  }
}
// blockIdx.z: 0 and 1 dq and dk, 2 the heads' sums (blockIdx.z starts at 2 where
// dq and dk are there already).
template <typename T, int V>
__global__ void __launch_bounds__(kT)
    grad_sums_kernel(const float* __restrict__ dqp, const float* __restrict__ dkp, int parts,
                     long long row, T* __restrict__ dq, T* __restrict__ dk,
                     const float* __restrict__ dAp, const float* __restrict__ dDp, int rows, int H,
                     float* __restrict__ dA, float* __restrict__ dD, int z0) {
  griddep_wait();
  const int z = blockIdx.z + z0;
  if (z == 0) return group_sum<T, V>(dqp, parts, row, dq);
  if (z == 1) return group_sum<T, V>(dkp, parts, row, dk);
  for (int h = blockIdx.y * gridDim.x + blockIdx.x; h < H; h += gridDim.x * gridDim.y) {
    head_sum(dAp, dDp, rows, H, h, dA, dD);
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kT) tile_sum_kernel(const float* __restrict__ part, int tiles,
                                                      long long n, float* __restrict__ out) {
  const long long i = (long long)blockIdx.x * kT + threadIdx.x;
  griddep_wait();
  if (i >= n) return;
  float a = 0.f;
  for (int j = 0; j < tiles; ++j) a += part[(long long)j * n + i];
  out[i] = a;
}

// One token: S = e^{dt A} S + dt v k^T in place, y = S q + D v. Bound by HBM: S
// is read and written once. kLanes lanes share a state row; each loads all its
// pieces of the row before it stores any, so that a warp has whole rows in flight.
//   VEC: 8 lanes a row and PIECES float4 a lane (N <= 32 PIECES, a multiple of 4)
//   else 32 lanes a row, single values
template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&f)[4]);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
template <>
__device__ __forceinline__ void load4<bf16>(const bf16* p, float (&f)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xffff0000u);
  f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xffff0000u);
}
template <typename T, int PIECES>  // PIECES 0: single values
__global__ void __launch_bounds__(kT)
    ssm_step_kernel(SsmDims s, const T* __restrict__ q, const T* __restrict__ k,
                    const T* __restrict__ v, const float* __restrict__ dt,
                    const float* __restrict__ A, const float* __restrict__ D,
                    float* __restrict__ S, T* __restrict__ y) {
  constexpr int kLanes = PIECES ? 8 : 32;
  const int bh = blockIdx.y, b = bh / s.H, h = bh - b * s.H, g = h / (s.H / s.G);
  const int p = blockIdx.x * (kT / kLanes) + threadIdx.x / kLanes, l = threadIdx.x % kLanes;
  const bool on = p < s.P;
  float* row = S + ((long long)bh * s.P + p) * s.N;
  const T* qr = q + ((long long)b * s.G + g) * s.N;
  const T* kr = k + ((long long)b * s.G + g) * s.N;
  float acc = 0.f, x = 0.f;
  if constexpr (PIECES > 0) {
    float4 r[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int n = (i * kLanes + l) * 4;
      if (on && n < s.N) r[i] = __ldcs(reinterpret_cast<const float4*>(row + n));
    }
    const float e = dt[bh], dec = ex2(e * A[h] * 1.44269504f);
    x = on ? to_f<T>(v[(long long)bh * s.P + p]) : 0.f;
    const float ex = e * x;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int n = (i * kLanes + l) * 4;
      if (on && n < s.N) {
        float kf[4], qf[4];
        load4<T>(kr + n, kf);
        load4<T>(qr + n, qf);
        r[i].x = fmaf(dec, r[i].x, ex * kf[0]);
        r[i].y = fmaf(dec, r[i].y, ex * kf[1]);
        r[i].z = fmaf(dec, r[i].z, ex * kf[2]);
        r[i].w = fmaf(dec, r[i].w, ex * kf[3]);
        __stcs(reinterpret_cast<float4*>(row + n), r[i]);
        acc = fmaf(r[i].x, qf[0], acc);
        acc = fmaf(r[i].y, qf[1], acc);
        acc = fmaf(r[i].z, qf[2], acc);
        acc = fmaf(r[i].w, qf[3], acc);
      }
    }
  } else {
    const float e = dt[bh], dec = ex2(e * A[h] * 1.44269504f);
    x = on ? to_f<T>(v[(long long)bh * s.P + p]) : 0.f;
    const float ex = e * x;
    float r[8];  // N <= 256
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (on && i * 32 + l < s.N) r[i] = row[i * 32 + l];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = i * 32 + l;
      if (on && n < s.N) {
        r[i] = fmaf(dec, r[i], ex * to_f<T>(kr[n]));
        row[n] = r[i];
        acc = fmaf(r[i], to_f<T>(qr[n]), acc);
      }
    }
  }
#pragma unroll
  for (int o = kLanes / 2; o; o >>= 1) acc += __shfl_xor_sync(~0u, acc, o);
  if (on && l == 0) y[(long long)bh * s.P + p] = from_f<T>(D ? fmaf(D[h], x, acc) : acc);
}

size_t state_smem(const SsmDims& s) {
  return sizeof(float) * (3 * s.Q + (size_t)s.Q * (kSsmPT + 1) + (size_t)s.Q * (s.N + 1));
}
size_t out_smem(const SsmDims& s) {
  return sizeof(float) * (3 * s.Q + (size_t)(s.Q + (s.Q > kSsmPT ? s.Q : kSsmPT)) * (s.N + 1) +
                          (size_t)s.Q * (kSsmPT + 1) + (size_t)s.Q * (s.Q + 1));
}
size_t grad_smem(const SsmDims& s) {
  return sizeof(float) * (9 * s.Q + 16 + (size_t)2 * (s.Q + kSsmPT) * (s.N + 1) +
                          (size_t)2 * s.Q * (kSsmPT + 1) + (size_t)2 * s.Q * (s.Q + 1) +
                          (size_t)32 * s.Q);
}

template <class F>
cudaError_t allow_smem(F* f, size_t bytes) {
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Cuts up the backward's workspace (or, of a null one, only measures it).
size_t cut_bwd(const SsmDims& s, char* ws, float* ddt, SsmBwdScratch* w) {
  size_t o = 0;
  const size_t f = sizeof(float), BH = (size_t)s.B * s.H;
  auto take = [&](size_t n) {
    char* p = ws + o;
    o = up256(o + n);
    return (float*)p;
  };
  // One part per head and state tile on CUDA cores; none where the tensor cores'
  // only part is the result.
  const size_t parts = s.tc ? ssm_tc_grad_parts(s) : (size_t)s.H / s.G * s.NPT;
  const size_t sums = s.tc && parts == 1 ? 0 : parts * s.B * s.G * s.T * s.N * f;
  w->status = (int*)take(256);
  w->ends = take(s.NC * BH * s.P * s.N * f);
  w->decay = take(s.NC * BH * f);
  w->logs = take(s.tc ? ssm_tc_logs_bytes(s) : 0);
  w->dq = take(sums);
  w->dk = take(sums);
  w->ddt = s.NPT > 1 ? take(s.NPT * BH * s.T * f) : ddt;
  w->dA = take((size_t)s.NC * s.NPT * BH * f);
  w->dD = take((size_t)s.NC * s.NPT * BH * f);
  return o;
}

template <typename T>
cudaError_t fwd_t(const SsmFwdArgs& a) {
  const SsmDims& s = a.s;
  const dim3 grid(s.NC, s.B * s.H, s.NPT);
  cudaError_t e;
  {
    E2TTT_TRACE("ssm_chunk_state", a.st);
    if ((e = allow_smem(chunk_state_kernel<T, 0>, state_smem(s))) != cudaSuccess) return e;
    chunk_state_kernel<T, 0><<<grid, kT, state_smem(s), a.st>>>(
        s, (const T*)a.v, (const T*)a.k, a.dt, a.A, a.lengths, a.states, a.decay, a.status);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = ssm_carry(s, false, a.S0, a.decay, a.states, a.S_end, nullptr, true, a.st)) != cudaSuccess) return e;
  E2TTT_TRACE("ssm_chunk_out", a.st);
  auto kern = chunk_out_kernel<T, 2>;
  if constexpr (std::is_same<T, float>::value)  // bf16 with so few columns runs on the tensor cores
    if (s.Q == 64) kern = chunk_out_kernel<T, 4>;
  if ((e = allow_smem(kern, out_smem(s))) != cudaSuccess) return e;
  kern<<<grid, kT, out_smem(s), a.st>>>(s, (const T*)a.q, (const T*)a.k, (const T*)a.v, a.dt, a.A,
                                        a.D, a.lengths, a.states, (T*)a.y);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_t(const SsmBwdArgs& a, const SsmBwdScratch& w) {
  const SsmDims& s = a.s;
  const dim3 grid(s.NC, s.B * s.H, s.NPT);
  cudaError_t e;
  {
    E2TTT_TRACE("ssm_chunk_dstate", a.st);
    if ((e = allow_smem(chunk_state_kernel<T, 1>, state_smem(s))) != cudaSuccess) return e;
    chunk_state_kernel<T, 1><<<grid, kT, state_smem(s), a.st>>>(
        s, (const T*)a.dy, (const T*)a.q, a.dt, a.A, a.lengths, w.ends, w.decay, w.status);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = ssm_carry(s, true, a.dS_end, w.decay, w.ends, a.dS0, nullptr, true, a.st)) != cudaSuccess) return e;
  {
    E2TTT_TRACE("ssm_chunk_grad", a.st);
    auto kern = chunk_grad_kernel<T, 2>;
    if constexpr (std::is_same<T, float>::value)  // bf16 with so few columns runs on the tensor cores
      if (s.Q == 64) kern = chunk_grad_kernel<T, 4>;
    if ((e = allow_smem(kern, grad_smem(s))) != cudaSuccess) return e;
    kern<<<grid, kT, grad_smem(s), a.st>>>(s, (const T*)a.q, (const T*)a.k, (const T*)a.v, a.dt, a.A,
                                           a.D, a.lengths, a.states, w.ends, (const T*)a.dy, w.dq, w.dk,
                                           (T*)a.dv, w.ddt, w.dA, w.dD);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return ssm_grad_sums(a, w, s.H / s.G * s.NPT);
}

}  // namespace

cudaError_t ssm_carry(const SsmDims& s, bool back, const float* first, const float* decay,
                      float* states, float* last, void* copy, bool keep, cudaStream_t st) {
  const int BH = s.B * s.H;
  const long long PN = (long long)s.P * s.N;
  E2TTT_TRACE(back ? "ssm_carry_back" : "ssm_carry", st);
  if (PN % 4 == 0 && !(((uintptr_t)first | (uintptr_t)states | (uintptr_t)last) & 15)) {
    const dim3 grid((unsigned)((PN / 4 + kT - 1) / kT), BH);
    return launch_pdl(back ? carry_kernel<float4, 1> : carry_kernel<float4, 0>, grid, dim3(kT), 0, st, s.NC, BH,
                      PN / 4, (const float4*)first, decay, (float4*)states, (float4*)last, (bf16*)copy, keep);
  }
  const dim3 grid((unsigned)((PN + kT - 1) / kT), BH);
  return launch_pdl(back ? carry_kernel<float, 1> : carry_kernel<float, 0>, grid, dim3(kT), 0, st, s.NC, BH, PN,
                    first, decay, states, last, (bf16*)copy, keep);
}

template <typename T>
static cudaError_t grad_sums_t(const SsmBwdArgs& a, const SsmBwdScratch& w, int parts) {
  const SsmDims& s = a.s;
  const long long row = (long long)s.T * s.N;
  const bool vec = s.N % 4 == 0 && !(((uintptr_t)a.dq | (uintptr_t)a.dk) & (4 * sizeof(T) - 1));
  const bool direct = s.tc && parts == 1;  // dq and dk are there
  const long long per = kT * (vec ? 4 : 1);
  const dim3 grid = direct ? dim3(s.H, 1, 1) : dim3((unsigned)((row + per - 1) / per), s.B * s.G, 3);
  E2TTT_TRACE("ssm_grad_sums", a.st);
  return launch_pdl(vec ? grad_sums_kernel<T, 4> : grad_sums_kernel<T, 1>, grid, dim3(kT), 0, a.st,
                    (const float*)w.dq, (const float*)w.dk, parts, row, (T*)a.dq, (T*)a.dk, (const float*)w.dA,
                    (const float*)w.dD, s.NC * s.NPT * s.B, s.H, a.dA, a.dD, direct ? 2 : 0);
}
cudaError_t ssm_grad_sums(const SsmBwdArgs& a, const SsmBwdScratch& w, int parts) {
  const SsmDims& s = a.s;
  if (s.NPT > 1) {
    const long long n = (long long)s.B * s.H * s.T;
    E2TTT_TRACE("ssm_tile_sum", a.st);
    const cudaError_t e = launch_pdl(tile_sum_kernel, dim3((unsigned)((n + kT - 1) / kT)), dim3(kT), 0, a.st,
                                     (const float*)w.ddt, s.NPT, n, a.ddt);
    if (e != cudaSuccess) return e;
  }
  return s.bf16_act ? grad_sums_t<bf16>(a, w, parts) : grad_sums_t<float>(a, w, parts);
}

size_t ssm_bwd_workspace_bytes(const SsmDims& s) {
  SsmBwdScratch w;
  return cut_bwd(s, nullptr, nullptr, &w);
}
cudaError_t ssm_fwd(const SsmFwdArgs& a) { return a.s.bf16_act ? fwd_t<bf16>(a) : fwd_t<float>(a); }
cudaError_t ssm_bwd(const SsmBwdArgs& a) {
  SsmBwdScratch w;
  cut_bwd(a.s, (char*)a.ws, a.ddt, &w);
  if (a.s.tc) return ssm_tc_bwd(a, w);
  return a.s.bf16_act ? bwd_t<bf16>(a, w) : bwd_t<float>(a, w);
}

template <typename T>
static cudaError_t step_t(const SsmStepArgs& a) {
  const SsmDims& s = a.s;
  const uintptr_t qk = (uintptr_t)a.q | (uintptr_t)a.k;
  const bool vec = s.N % 4 == 0 && !((uintptr_t)a.S & 15) && !(qk & (4 * sizeof(T) - 1));
  const int pieces = !vec ? 0 : s.N <= 64 ? 2 : s.N <= 128 ? 4 : 8;
  auto kern = pieces == 0   ? ssm_step_kernel<T, 0>
              : pieces == 2 ? ssm_step_kernel<T, 2>
              : pieces == 4 ? ssm_step_kernel<T, 4>
                            : ssm_step_kernel<T, 8>;
  const int rows = kT / (vec ? 8 : 32);
  E2TTT_TRACE("ssm_step", a.st);
  kern<<<dim3((s.P + rows - 1) / rows, s.B * s.H), kT, 0, a.st>>>(
      s, (const T*)a.q, (const T*)a.k, (const T*)a.v, a.dt, a.A, a.D, a.S, (T*)a.y);
  return cudaGetLastError();
}
cudaError_t ssm_step(const SsmStepArgs& a) { return a.s.bf16_act ? step_t<bf16>(a) : step_t<float>(a); }

}  // namespace e2ttt
