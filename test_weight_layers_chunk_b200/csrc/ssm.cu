// State-space scan for every size and type, its single-token form, and the passes over
// chunk states that all forms share. The mathematics is in ssm.cuh.
//
// A chunk's work is a handful of small matrix products from shared memory; chunks
// meet only in their states, which one elementwise pass carries along the tokens.
// 2 x 16 heads x 2048 tokens, 64 x 128 states, fp32: forward 196 us, backward 507; 64 x
// 256 states in bf16: 476 and 1094 (fp32 490 and 1100: the products are the same). Bound
// by the products' instructions: each warp splits its operands again, and q k^T is made
// again for each head and tile of state rows.
#include "ssm.cuh"
#include "trace.h"

namespace e2ttt {
namespace {

constexpr int kT = 256;

// Products of fp32 tiles in shared memory on the warps' tensor instructions
// (m16n8k8, tf32): each operand enters as two tf32 terms, a = a0 + a1 to 22 bits,
// and a b = a0 b0 + a0 b1 + a1 b0 (what is left out is 2^-22 of it at most). Against
// plain fp32 multiply-adds from shared memory this reads each operand value once per 16
// or 8 results instead of once per 4 (training step of 2 x 6 heads x 509 tokens, 48 x
// 40 states: 99 -> 72 us). There, and for 8 heads x 1000 tokens of 64 x 128 states, y, S
// and the gradients are off from 64-bit ones by 0.6 to 1.6 times what fp32 matrix
// products of the same chunk form are (2-norms of 0.5 to 2.4e-7), dA by 2 to 3 times
// (4 to 6e-7).
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// The block's 8 warps share a result of R * 16 rows x 64 columns: R warps down, W
// = 8 / R across, each 16 rows by R * 8 columns. Result e of column tile j of a
// thread is at row() + 8 (e >> 1), col(j) + (e & 1).
template <int R>
struct Tile {
  static constexpr int W = 8 / R;
  float v[R][4];
  static __device__ __forceinline__ int row() { return (threadIdx.x >> 5) % R * 16 + (threadIdx.x & 31) / 4; }
  static __device__ __forceinline__ int across() { return (threadIdx.x >> 5) / R; }
  static __device__ __forceinline__ int col(int j) { return across() * R * 8 + j * 8 + (threadIdx.x & 3) * 2; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j][e] = 0.f;
  }
  // += sum_k A(m, k) B(k, n0 + n): A at a + m*am + k*ak, B at b + k*bk + n*bn, for
  // K a multiple of 8 (zeros where the data ends) and columns up to nmax (clamped).
  __device__ __forceinline__ void mm(const float* a, int am, int ak, const float* b, int bk, int bn, int K,
                                     int n0, int nmax) {
    const int q = threadIdx.x & 3, r = (threadIdx.x & 31) / 4;
    const float* a0 = a + row() * am + q * ak;
    const float* b0[R];
#pragma unroll
    for (int j = 0; j < R; ++j) b0[j] = b + min(n0 + across() * R * 8 + j * 8 + r, nmax) * bn + q * bk;
#pragma unroll 2
    for (int k = 0; k < K; k += 8) {
      uint32_t ah[4], al[4];
      split_tf32(a0[k * ak], ah[0], al[0]);
      split_tf32(a0[k * ak + 8 * am], ah[1], al[1]);
      split_tf32(a0[(k + 4) * ak], ah[2], al[2]);
      split_tf32(a0[(k + 4) * ak + 8 * am], ah[3], al[3]);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        uint32_t bh[2], bl[2];
        split_tf32(b0[j][k * bk], bh[0], bl[0]);
        split_tf32(b0[j][(k + 4) * bk], bh[1], bl[1]);
        // Eight products at a time from zero, then added with rounding: the tensor
        // instructions' own additions cut off, which over a long sum would lean one way.
        float t[4] = {};
        mma_tf32(t, al, bh);
        mma_tf32(t, ah, bl);
        mma_tf32(t, ah, bh);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][e] += t[e];
      }
    }
  }
};
// Sum over the four threads that share a row.
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(~0u, x, 1);
  return x + __shfl_xor_sync(~0u, x, 2);
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

// State columns as the products contract them: a multiple of 8, zeros beyond N. A
// row's pitch is 4 more, so that the 8 rows and 4 columns that a warp reads at
// once fall into 32 different banks.
__host__ __device__ __forceinline__ int pad8(int n) { return (n + 7) & ~7; }
constexpr int kXP = kSsmPT + 4;

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
  const int Q = s.Q, N = s.N, XP = kXP, NP = pad8(N) + 4;
  const ChunkLogs L(sm, Q);
  float* xs = sm + kLogRows * Q;
  float* ys = xs + Q * XP;
  if (threadIdx.x < 32) fill_chunk_logs(L, dt + (long long)w.bh * s.T + w.t0, A[w.h], w.n);
  load_tile<T>(ys, NP, y + (((long long)w.b * s.G + w.g) * s.T + w.t0) * N, N, Q, w.n, N, pad8(N));
  load_tile<T>(xs, XP, x + ((long long)w.bh * s.T + w.t0) * s.P + w.p0, s.P, Q, w.n, w.np, kSsmPT);
  __syncthreads();
  for (int i = threadIdx.x; i < Q * kSsmPT; i += kT) {
    const int t = i / kSsmPT, p = i - t * kSsmPT;
    xs[t * XP + p] *= REV ? L.start[t] : L.end[t] * L.eta[t];
  }
  if (threadIdx.x == 0 && w.pt == 0)
    decay[(long long)w.c * s.B * s.H + w.bh] = L.start[Q - 1];
  __syncthreads();
  float* out = states + (((long long)w.c * s.B * s.H + w.bh) * s.P + w.p0) * N;
  for (int n0 = 0; n0 < N; n0 += 64) {
    Tile<4> acc;
    acc.clear();
    acc.mm(xs, 1, XP, ys, NP, 1, Q, n0, N - 1);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = acc.row() + 8 * (e >> 1), n = n0 + acc.col(j) + (e & 1);
        if (p < w.np && n < N) out[(long long)p * N + n] = acc.v[j][e];
      }
  }
}

// Turns the chunks' own contributions into the states at their starts (REV 0,
// from `first`) or the gradients at their ends (REV 1, from the last chunk
// back); `last` gets what is left after the last one. `copy`, where given, takes
// them rounded to bf16 (what the outputs' products read), and without `keep` the
// fp32 ones are not written. Elementwise along the chunks; V is float4 where rows and
// pointers allow. 14 to 18 us for 16 chunks of 128 heads' 64 x 128 states with only the
// copy written (101 MB, DRAM 50 %), 31 to 35 us with both (168 MB, 28 %): bound by the
// latency of its loads (long scoreboard, 22 % of the warps' places taken). But 4 or 16
// chunks in flight or more blocks on an SM cost up to half more on long rows.
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
  constexpr int W = sizeof(V) / sizeof(float), U = kCarryBatch;
  const int bh = blockIdx.y;
  const long long i = (long long)blockIdx.x * kT + threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  if (i >= PN) return;
  V run = first ? first[bh * PN + i] : V{};
  // this element in the first chunk of the walk, and the way to the next one
  const long long step = (REV ? -1 : 1) * (long long)BH * PN, start = (REV ? NC - 1LL : 0) * BH;
  V* p = states + (start + bh) * PN + i;
  bf16* to = copy ? copy + ((start + bh) * PN + i) * W : nullptr;
  const float* d = decay + start + bh;
  const int dstep = REV ? -BH : BH;
  int c = 0;
  for (; c + U <= NC; c += U) {
    V own[U];
    float e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      own[u] = __ldcs(p + u * step);
      e[u] = d[u * (long long)dstep];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (keep) __stcs(p, run);
      if (to) {
        store_bf16(to, run);
        to += step * W;
      }
      decay_add(run, e[u], own[u]);
      p += step;
      d += dstep;
    }
  }
  for (; c < NC; ++c) {
    const V own = *p;
    if (keep) __stcs(p, run);
    if (to) {
      store_bf16(to, run);
      to += step * W;
    }
    decay_add(run, *d, own);
    p += step;
    d += dstep;
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
  const int Q = s.Q, N = s.N, XP = kXP, NP = pad8(N) + 4, QP = Q + 4;
  const ChunkLogs L(sm, Q);
  float* qs = sm + kLogRows * Q;
  float* ks = qs + Q * NP;  // then the state [PT][NP]
  float* xs = ks + (Q > kSsmPT ? Q : kSsmPT) * NP;
  float* ws = xs + Q * XP;
  if (threadIdx.x < 32) fill_chunk_logs(L, dt + (long long)w.bh * s.T + w.t0, A[w.h], w.n);
  const long long qo = (((long long)w.b * s.G + w.g) * s.T + w.t0) * N;
  load_tile<T>(qs, NP, q + qo, N, Q, w.n, N, pad8(N));
  load_tile<T>(ks, NP, k + qo, N, Q, w.n, N, pad8(N));
  load_tile<T>(xs, XP, v + ((long long)w.bh * s.T + w.t0) * s.P + w.p0, s.P, Q, w.n, w.np, kSsmPT);
  __syncthreads();
  const int NK = pad8(N);
  Tile<R> acc;
  acc.clear();
  acc.mm(qs, NP, 1, ks, 1, NP, NK, 0, Q - 1);
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = acc.row() + 8 * (e >> 1), u = acc.col(j) + (e & 1);
      const float x = acc.v[j][e] * (L.decay(t, min(u, Q - 1)) * L.eta[min(u, Q - 1)]);
      if (u < Q) ws[t * QP + u] = u <= t ? x : 0.f;
    }
  __syncthreads();
  load_tile<float>(ks, NP, states + (((long long)w.c * s.B * s.H + w.bh) * s.P + w.p0) * N, N, kSsmPT,
                   w.np, N, NK);
  __syncthreads();
  acc.clear();
  acc.mm(qs, NP, 1, ks, 1, NP, NK, 0, kSsmPT - 1);
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc.v[j][e] *= L.start[acc.row() + 8 * (e >> 1)];
  acc.mm(ws, QP, 1, xs, XP, 1, Q, 0, kSsmPT - 1);
  const float Dh = D ? D[w.h] : 0.f;
  T* out = y + ((long long)w.bh * s.T + w.t0) * s.P + w.p0;
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = acc.row() + 8 * (e >> 1), p = acc.col(j) + (e & 1);
      const float o = fmaf(Dh, xs[t * XP + min(p, kSsmPT - 1)], acc.v[j][e]);
      if (w.t0 + t < s.T && p < w.np) out[(long long)t * s.P + p] = from_f<T>(t < w.n ? o : 0.f);
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
                      float* __restrict__ ddtp, double* __restrict__ dAp, double* __restrict__ dDp) {
  extern __shared__ float sm[];
  const Where w = where(s, lengths);
  const int Q = s.Q, N = s.N, XP = kXP, NP = pad8(N) + 4, QP = Q + 4;
  const ChunkLogs L(sm, Q);
  // [3][Q]: row sums of Z off its diagonal, column sums of Z / eta off it, and the
  // diagonal of Z / eta
  float* dots = sm + kLogRows * Q;
  float* scratch = dots + 3 * Q;  // doubles too: Q is even
  float* qs = scratch + 16;
  float* ks = qs + Q * NP;
  float* Ss = ks + Q * NP;
  float* Xs = Ss + kSsmPT * NP;
  float* xs = Xs + kSsmPT * NP;
  float* gs = xs + Q * XP;
  float* Ws = gs + Q * XP;  // e^{c_t-c_s} (q_t.k_s)
  float* Ks = Ws + Q * QP;  // e^{c_t-c_s} eta_s (dy_t.v_s)
  float* cz = Ks + Q * QP;       // [8][Q]: sums by warp
  float* parts = cz + 8 * Q;     // [2][R / 2][Q]: rows' and columns' sums by blocks of 32
  if (threadIdx.x < 32) fill_chunk_logs(L, dt + (long long)w.bh * s.T + w.t0, A[w.h], w.n);
  const long long qo = (((long long)w.b * s.G + w.g) * s.T + w.t0) * N;
  const long long vo = ((long long)w.bh * s.T + w.t0) * s.P + w.p0;
  const long long so = (((long long)w.c * s.B * s.H + w.bh) * s.P + w.p0) * N;
  load_tile<T>(qs, NP, q + qo, N, Q, w.n, N, pad8(N));
  load_tile<T>(ks, NP, k + qo, N, Q, w.n, N, pad8(N));
  load_tile<T>(xs, XP, v + vo, s.P, Q, w.n, w.np, kSsmPT);
  load_tile<T>(gs, XP, dy + vo, s.P, Q, w.n, w.np, kSsmPT);
  load_tile<float>(Ss, NP, states + so, N, kSsmPT, w.np, N, pad8(N));
  load_tile<float>(Xs, NP, ends + so, N, kSsmPT, w.np, N, pad8(N));
  __syncthreads();
  const int NK = pad8(N);
  {
    Tile<R> m, kk;
    m.clear();
    kk.clear();
    m.mm(qs, NP, 1, ks, 1, NP, NK, 0, Q - 1);
    kk.mm(gs, XP, 1, xs, 1, XP, kSsmPT, 0, Q - 1);
    float rows[2] = {};
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = m.row() + 8 * (e >> 1), u = m.col(j) + (e & 1), uc = min(u, Q - 1);
        const float d = L.decay(t, uc), eta = L.eta[uc];
        const float a = u <= t ? d * m.v[j][e] : 0.f;
        const float r = u <= t ? a * kk.v[j][e] : 0.f;
        if (u < Q) {
          Ws[t * QP + u] = a;
          Ks[t * QP + u] = u <= t ? d * eta * kk.v[j][e] : 0.f;
          if (u == t) dots[2 * Q + t] = r;
        }
        m.v[j][e] = u < t && u < Q ? r : 0.f;  // Z / eta off the diagonal
        rows[e >> 1] = fmaf(m.v[j][e], eta, rows[e >> 1]);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rows[i] = quad_sum(rows[i]);
      if ((threadIdx.x & 3) == 0) cz[m.across() * Q + m.row() + 8 * i] = rows[i];
    }
    // column sums: over the 8 rows that a thread's column has in the warp, twice
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float c = m.v[j][e] + m.v[j][e + 2];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) c += __shfl_xor_sync(~0u, c, o);
        const int u = m.col(j) + e;
        if ((threadIdx.x & 31) < 4 && u < Q) cz[(4 + (threadIdx.x >> 5) % R) * Q + u] = c;
      }
  }
  __syncthreads();
  for (int u = threadIdx.x; u < Q; u += kT) {
    // by blocks of 32 tokens (a warp's share is R * 8 columns, 16 rows), then in all
    constexpr int K = R / 2, kAcross = Tile<R>::W / K;
    float z = 0.f, c = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float zk = 0.f;
#pragma unroll
      for (int i = 0; i < kAcross; ++i) zk += R * 8 * (k * kAcross + i) < Q ? cz[(k * kAcross + i) * Q + u] : 0.f;
      const float ck = cz[(4 + 2 * k) * Q + u] + cz[(5 + 2 * k) * Q + u];
      parts[k * Q + u] = zk;
      parts[(K + k) * Q + u] = ck;
      z += zk;
      c += ck;
    }
    dots[u] = z;
    dots[Q + u] = c;
  }
  // dv
  {
    Tile<R> acc;
    acc.clear();
    acc.mm(ks, NP, 1, Xs, 1, NP, NK, 0, kSsmPT - 1);
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc.v[j][e] *= L.end[acc.row() + 8 * (e >> 1)];
    acc.mm(Ws, 1, QP, gs, XP, 1, Q, 0, kSsmPT - 1);
    const float Dh = D ? D[w.h] : 0.f;
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = acc.row() + 8 * (e >> 1), p = acc.col(j) + (e & 1);
        const float o = fmaf(L.eta[t], acc.v[j][e], Dh * gs[t * XP + min(p, kSsmPT - 1)]);
        if (w.t0 + t < s.T && p < w.np) dv[vo + (long long)t * s.P + p] = from_f<T>(t < w.n ? o : 0.f);
      }
  }
  // dq, dk and the dots of their state parts
  const long long po = (((long long)w.bh * s.NPT + w.pt) * s.T + w.t0) * N;
  float dot[2][2] = {};  // of dq, dk; of this thread's two rows
  for (int n0 = 0; n0 < N; n0 += 64) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const float* mine = which ? ks : qs;
      float* out = which ? dkp : dqp;
      Tile<R> acc;
      acc.clear();
      acc.mm(which ? xs : gs, XP, 1, which ? Xs : Ss, NP, 1, kSsmPT, n0, N - 1);
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = acc.row() + 8 * (e >> 1), n = n0 + acc.col(j) + (e & 1);
          const float x = acc.v[j][e] * (which ? L.end[t] : L.start[t]);
          dot[which][e >> 1] = fmaf(n < N ? x : 0.f, mine[t * NP + min(n, N - 1)], dot[which][e >> 1]);
          acc.v[j][e] = which ? x * L.eta[t] : x;
        }
      if (which)
        acc.mm(Ks, 1, QP, qs, NP, 1, Q, n0, N - 1);
      else
        acc.mm(Ks, QP, 1, ks, NP, 1, Q, n0, N - 1);
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = acc.row() + 8 * (e >> 1), n = n0 + acc.col(j) + (e & 1);
          if (w.t0 + t < s.T && n < N) out[po + (long long)t * N + n] = t < w.n ? acc.v[j][e] : 0.f;
        }
    }
  }
  __syncthreads();  // the column sums' scratch has been read
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float x = quad_sum(dot[which][i]);
      if ((threadIdx.x & 3) == 0)
        cz[(which * 4 + Tile<R>::across()) * Q + Tile<R>::row() + 8 * i] = x;
    }
  // e^{c_Q} <S, X>
  float ip = 0.f;
  for (int i = threadIdx.x; i < kSsmPT * N; i += kT) {
    const int p = i / N, n = i - p * N;
    ip = fmaf(Ss[p * NP + n], Xs[p * NP + n], ip);
  }
  ip = block_sum0(ip, scratch);
  // dD = sum dy v: fp64, as over a row it may cancel to almost nothing
  double dsum = 0.0;
  for (int i = threadIdx.x; i < Q * kSsmPT; i += kT) {
    const int t = i / kSsmPT, p = i - t * kSsmPT;
    dsum += (double)gs[t * XP + p] * xs[t * XP + p];
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) dsum += __shfl_xor_sync(~0u, dsum, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) reinterpret_cast<double*>(scratch)[threadIdx.x >> 5] = dsum;
  __syncthreads();
  if (threadIdx.x < 32) {
    // ddt, dA, dD: lane l has the tokens l * K .. l * K + K - 1
    constexpr int K = R / 2;  // Q / 32
    const int lane = threadIdx.x;
    double in4[K], out4[K];
    float a4[K], b4[K], src[K], as = 0.f, bs = 0.f;
    double dD = 0.0;
    for (int i = 0; i < kT / 32; ++i) dD += reinterpret_cast<const double*>(scratch)[i];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int r = lane * K + i;
      float rd = 0.f;
      src[i] = 0.f;
      for (int x = 0; x < Tile<R>::W; ++x) {
        rd += cz[x * Q + r];
        src[i] += cz[(4 + x) * Q + r];
      }
      in4[i] = rd;
      out4[i] = (double)L.eta[r] * src[i];
      a4[i] = (dots[r] - L.eta[r] * dots[Q + r]) + rd;
      b4[i] = (float)out4[i];
      as += a4[i];
      bs += b4[i];
    }
    float after = as, before = bs;  // of this lane's tokens on; up to them
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float x = __shfl_down_sync(~0u, after, d), y = __shfl_up_sync(~0u, before, d);
      after += lane + d < 32 ? x : 0.f;
      before += lane >= d ? y : 0.f;
    }
    // exclusive of this lane's own, without taking them off again
    after = __shfl_down_sync(~0u, after, 1);
    before = __shfl_up_sync(~0u, before, 1);
    after = lane < 31 ? after : 0.f;
    before = lane > 0 ? before : 0.f;
    ip = __shfl_sync(~0u, ip, 0);
    const float through = L.start[Q - 1] * ip, Ah = A[w.h];
    const double dA = decay_gradient<K>([&](int c, int i) { return parts[c * Q + lane * K + i]; },
                                        [&](int d, int i) { return parts[(K + d) * Q + lane * K + i]; }, in4, out4,
                                        L.eta + lane * K, (double)L.start[Q - 1] * ip, lane);
    float dl[K];
#pragma unroll
    for (int i = K - 1; i >= 0; --i) dl[i] = after += a4[i];
    float* out = ddtp + ((long long)w.pt * s.B * s.H + w.bh) * s.T + w.t0;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int r = lane * K + i;
      dl[i] += before + through;
      before += b4[i];
      const float x = fmaf(Ah, dl[i], dots[Q + r] + dots[2 * Q + r] + src[i]);
      if (w.t0 + r < s.T) out[r] = r < w.n ? x : 0.f;
    }
    if (lane == 0) {
      const long long o = ((long long)w.c * s.NPT + w.pt) * s.B * s.H + w.bh;
      dAp[o] = dA;
      dDp[o] = dD;
    }
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
__device__ void head_sum(const double* dAp, const double* dDp, int rows, int H, int h, float* dA, float* dD) {
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
                     const double* __restrict__ dAp, const double* __restrict__ dDp, int rows, int H,
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
// pieces of the row before it stores any, so that a warp has whole rows in flight:
// 25.1 us for 64 x 32 heads of 64 x 128 (5360 GB/s, 83 % of a copy); value by value it
// took 55, and with the decay in a single fp32 value 24.6.
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
// e^{dt A} by its first 24 bits, cut off, and what that leaves (never negative, so that
// an infinite state keeps its sign). A state takes one of these for each token, over
// thousands of them: rounded to fp32 the decay itself would be off by 2^-25 the same way
// every time, 2^-25 / |dt A| of the state in the end. Formed as 1 + (e^x - 1), whose
// second part has 24 bits of its own; below -1/2 the memory is too short to need it. (By
// an exponential in fp64 a step of 64 x 32 heads took 28.7 us instead of 25.1.)
struct StepDecay {
  float hi, lo;
  __device__ __forceinline__ StepDecay(float dt, float A) {
    const float x = dt * A;
    if (fabsf(x) < 0.5f) {
      const float m = expm1f(x);
      hi = __fadd_rz(1.f, m);
      lo = m - (hi - 1.f);  // exact
    } else {
      hi = expf(x);
      lo = 0.f;
    }
  }
  // the decayed state, and what the token adds: one rounding at the state's size
  __device__ __forceinline__ float operator()(float S, float add) const {
    return fmaf(hi, S, lo > 0.f ? fmaf(lo, S, add) : add);
  }
};
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
    const float e = dt[bh];
    const StepDecay dec(e, A[h]);
    x = on ? to_f<T>(v[(long long)bh * s.P + p]) : 0.f;
    const float ex = e * x;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int n = (i * kLanes + l) * 4;
      if (on && n < s.N) {
        float kf[4], qf[4];
        load4<T>(kr + n, kf);
        load4<T>(qr + n, qf);
        r[i].x = dec(r[i].x, ex * kf[0]);
        r[i].y = dec(r[i].y, ex * kf[1]);
        r[i].z = dec(r[i].z, ex * kf[2]);
        r[i].w = dec(r[i].w, ex * kf[3]);
        __stcs(reinterpret_cast<float4*>(row + n), r[i]);
        acc = fmaf(r[i].x, qf[0], acc);
        acc = fmaf(r[i].y, qf[1], acc);
        acc = fmaf(r[i].z, qf[2], acc);
        acc = fmaf(r[i].w, qf[3], acc);
      }
    }
  } else {
    const float e = dt[bh];
    const StepDecay dec(e, A[h]);
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
        r[i] = dec(r[i], ex * to_f<T>(kr[n]));
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
  return sizeof(float) * (kLogRows * s.Q + (size_t)s.Q * kXP + (size_t)s.Q * (pad8(s.N) + 4));
}
size_t out_smem(const SsmDims& s) {
  return sizeof(float) * (kLogRows * s.Q + (size_t)(s.Q + (s.Q > kSsmPT ? s.Q : kSsmPT)) * (pad8(s.N) + 4) +
                          (size_t)s.Q * kXP + (size_t)s.Q * (s.Q + 4));
}
size_t grad_smem(const SsmDims& s) {
  return sizeof(float) * ((kLogRows + 3) * s.Q + 16 + (size_t)2 * (s.Q + kSsmPT) * (pad8(s.N) + 4) +
                          (size_t)2 * s.Q * kXP + (size_t)2 * s.Q * (s.Q + 4) +
                          (size_t)12 * s.Q);
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
  // One part per head and state tile here; none where the tcgen05 kernels' only part
  // is the result.
  const size_t parts = s.tc ? ssm_tc_grad_parts(s) : (size_t)s.H / s.G * s.NPT;
  const size_t sums = s.tc && parts == 1 ? 0 : parts * s.B * s.G * s.T * s.N * f;
  w->status = (int*)take(256);
  w->ends = take(s.NC * BH * s.P * s.N * f);
  w->decay = take(s.NC * BH * f);
  w->logs = take(s.tc ? ssm_tc_logs_bytes(s) : 0);
  w->dq = take(sums);
  w->dk = take(sums);
  w->ddt = s.NPT > 1 ? take(s.NPT * BH * s.T * f) : ddt;
  w->dA = (double*)take((size_t)s.NC * s.NPT * BH * sizeof(double));
  w->dD = (double*)take((size_t)s.NC * s.NPT * BH * sizeof(double));
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
  auto kern = s.Q == 64 ? chunk_out_kernel<T, 4> : chunk_out_kernel<T, 2>;
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
    auto kern = s.Q == 64 ? chunk_grad_kernel<T, 4> : chunk_grad_kernel<T, 2>;
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
                    (const float*)w.dq, (const float*)w.dk, parts, row, (T*)a.dq, (T*)a.dk, (const double*)w.dA,
                    (const double*)w.dD, s.NC * s.NPT * s.B, s.H, a.dA, a.dD, direct ? 2 : 0);
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
