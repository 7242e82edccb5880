// Short causal depthwise convolution over tokens, its gradients, and its form
// for single tokens.
//
//   z_t = bias + sum_{j<W} w_j x_{t-(W-1)+j},   y_t = z_t or silu(z_t)
//
// per (batch row, head, channel), with x before the first token taken from
// `state` (the W-1 inputs before it) or zero. Adjoint, with dz_t = dy_t y'(z_t):
//   dx_t = sum_j w_j dz_{t+(W-1)-j},  dw_j = sum_t dz_t x_{t-(W-1)+j},  dbias = sum_t dz_t.
//
// Bound by HBM: the forward reads x and writes y once, the backward reads x and
// dy and writes dx. A thread owns one 16-byte vector of channels and walks a run
// of R consecutive tokens with the last W inputs (and, backward, the last W dz)
// in registers, so a run re-reads only the W-1 tokens before it (and the
// backward the W-1 after it), which the neighbouring run has just brought into
// L1/L2. Threads of a warp cover consecutive channels, then consecutive runs.
#include "seq_ops.h"
#include "trace.h"

namespace e2ttt {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxW = 8;

// 1 / (1 + exp(-z)); exp overflows to infinity for z << 0, whose reciprocal is 0.
__device__ __forceinline__ float sigmoid_fast(float z) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * z));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

template <typename T, int VEC> struct VecOf;
template <> struct VecOf<bf16, 8> { typedef uint4 type; };
template <> struct VecOf<float, 4> { typedef uint4 type; };
template <> struct VecOf<bf16, 1> { typedef unsigned short type; };
template <> struct VecOf<float, 1> { typedef unsigned int type; };

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const typename VecOf<T, VEC>::type& r, float (&f)[VEC]) {
  const T* p = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int i = 0; i < VEC; ++i) f[i] = to_f<T>(p[i]);
}
template <typename T, int VEC>
__device__ __forceinline__ typename VecOf<T, VEC>::type pack(const float (&f)[VEC]) {
  typename VecOf<T, VEC>::type r;
  T* p = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int i = 0; i < VEC; ++i) p[i] = from_f<T>(f[i]);
  return r;
}

struct Geo {
  int H, T, d, nvec, nvt, rows;  // vectors per token, vectors per block, runs per block
  int runs;                      // runs of R tokens in T
  int R;
  bool silu;
};

__device__ __forceinline__ int row_length(const int* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

// Input at position i of the sequence [state; x[0..len)] (i = 0 is the oldest
// history row), zero outside it.
template <typename T, int VEC>
__device__ __forceinline__ void load_seq(const T* xrow, const T* srow, int i, int W1, int len,
                                         int d, int c0, float (&f)[VEC]) {
  typedef typename VecOf<T, VEC>::type V;
  const T* p = nullptr;
  if (i >= W1) {
    if (i - W1 < len) p = xrow + (long long)(i - W1) * d + c0;
  } else if (srow && i >= 0) {
    p = srow + (long long)i * d + c0;
  }
  if (p) {
    unpack<T, VEC>(*reinterpret_cast<const V*>(p), f);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = 0.f;
  }
}

template <typename T, int W, int VEC>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(Geo g, const T* __restrict__ x,
                                                            const float* __restrict__ w,
                                                            const float* __restrict__ bias,
                                                            const T* __restrict__ state,
                                                            const int* __restrict__ lengths,
                                                            T* __restrict__ y,
                                                            T* __restrict__ state_end) {
  typedef typename VecOf<T, VEC>::type V;
  constexpr int W1 = W - 1;
  const int bh = blockIdx.y, h = bh % g.H;
  const int vi = blockIdx.z * g.nvt + threadIdx.x % g.nvt;
  const int run = blockIdx.x * g.rows + threadIdx.x / g.nvt;
  if (vi >= g.nvec || run >= g.runs) return;
  const int c0 = vi * VEC, len = row_length(lengths, bh / g.H, g.T);
  const T* xrow = x + (long long)bh * g.T * g.d;
  T* yrow = y + (long long)bh * g.T * g.d;
  const T* srow = state ? state + (long long)bh * W1 * g.d : nullptr;

  float wr[W][VEC], br[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    br[e] = bias ? bias[h * g.d + c0 + e] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) wr[j][e] = w[((long long)h * g.d + c0 + e) * W + j];
  }
  const int t0 = run * g.R, t1 = min(t0 + g.R, g.T);
  float win[W][VEC];  // the W inputs that end at the current token
#pragma unroll
  for (int j = 0; j < W1; ++j) load_seq<T, VEC>(xrow, srow, t0 + j, W1, len, g.d, c0, win[j]);

  constexpr int BATCH = 8;
  for (int tb = t0; tb < t1; tb += BATCH) {
    V raw[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      raw[i] = V{};
      if (tb + i < t1 && tb + i < len)
        raw[i] = *reinterpret_cast<const V*>(xrow + (long long)(tb + i) * g.d + c0);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int t = tb + i;
      unpack<T, VEC>(raw[i], win[W1]);
      float o[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float z = br[e];
#pragma unroll
        for (int j = 0; j < W; ++j) z = fmaf(wr[j][e], win[j][e], z);
        z = g.silu ? z * sigmoid_fast(z) : z;
        o[e] = t < len ? z : 0.f;
      }
      if (t < t1) *reinterpret_cast<V*>(yrow + (long long)t * g.d + c0) = pack<T, VEC>(o);
#pragma unroll
      for (int j = 0; j < W1; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) win[j][e] = win[j + 1][e];
    }
  }
  if (state_end && run == 0) {
#pragma unroll
    for (int j = 0; j < W1; ++j) {
      float f[VEC];
      load_seq<T, VEC>(xrow, srow, len + j, W1, len, g.d, c0, f);
      *reinterpret_cast<V*>(state_end + ((long long)bh * W1 + j) * g.d + c0) = pack<T, VEC>(f);
    }
  }
}

// part [B * gridDim.x][H][W + 1][d]: this block's sums of dz x (taps 0..W-1) and dz.
template <typename T, int W, int VEC>
__global__ void __launch_bounds__(kThreads)
    conv_bwd_kernel(Geo g, const T* __restrict__ x, const float* __restrict__ w,
                    const float* __restrict__ bias, const T* __restrict__ state,
                    const int* __restrict__ lengths, const T* __restrict__ dy,
                    const T* __restrict__ dstate_end, T* __restrict__ dx, T* __restrict__ dstate,
                    float* __restrict__ part) {
  typedef typename VecOf<T, VEC>::type V;
  constexpr int W1 = W - 1;
  extern __shared__ float sums[];  // [blockDim.x][VEC]
  const int bh = blockIdx.y, h = bh % g.H, b = bh / g.H;
  const int vl = threadIdx.x % g.nvt, vi = blockIdx.z * g.nvt + vl, c0 = vi * VEC;
  const bool on = vi < g.nvec;
  const int len = row_length(lengths, b, g.T);
  const T* xrow = x + (long long)bh * g.T * g.d;
  const T* dyrow = dy + (long long)bh * g.T * g.d;
  T* dxrow = dx + (long long)bh * g.T * g.d;
  const T* srow = state ? state + (long long)bh * W1 * g.d : nullptr;

  float wr[W][VEC], br[VEC], dw[W][VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    br[e] = on && bias ? bias[h * g.d + c0 + e] : 0.f;
    db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      wr[j][e] = on ? w[((long long)h * g.d + c0 + e) * W + j] : 0.f;
      dw[j][e] = 0.f;
    }
  }
  for (int run = blockIdx.x * g.rows + threadIdx.x / g.nvt; on && run < g.runs;
       run += gridDim.x * g.rows) {
    const int t0 = run * g.R, t1 = min(t0 + g.R, g.T);
    float win[W][VEC], dz[W][VEC];  // dz[j]: of the token j before the current one
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) dz[j][e] = 0.f;
#pragma unroll
    for (int j = 0; j < W1; ++j) load_seq<T, VEC>(xrow, srow, t0 + j, W1, len, g.d, c0, win[j]);
    constexpr int BATCH = 4;
    for (int tb = t0; tb < t1 + W1; tb += BATCH) {
      V rx[BATCH], rd[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        rx[i] = V{};
        rd[i] = V{};
        if (tb + i < t1 + W1 && tb + i < len) {
          rx[i] = *reinterpret_cast<const V*>(xrow + (long long)(tb + i) * g.d + c0);
          rd[i] = *reinterpret_cast<const V*>(dyrow + (long long)(tb + i) * g.d + c0);
        }
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int s = tb + i;
        float gy[VEC], o[VEC];
        unpack<T, VEC>(rx[i], win[W1]);
        unpack<T, VEC>(rd[i], gy);
        const bool mine = s < t1;  // its sums belong to this run
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float z = br[e];
#pragma unroll
          for (int j = 0; j < W; ++j) z = fmaf(wr[j][e], win[j][e], z);
          float f = 1.f;
          if (g.silu) {
            const float sg = sigmoid_fast(z);
            f = sg * fmaf(z, 1.f - sg, 1.f);
          }
          dz[0][e] = s < len ? gy[e] * f : 0.f;
          const float own = mine ? dz[0][e] : 0.f;
          db[e] += own;
#pragma unroll
          for (int j = 0; j < W; ++j) dw[j][e] = fmaf(own, win[j][e], dw[j][e]);
          o[e] = 0.f;
#pragma unroll
          for (int j = 0; j < W; ++j) o[e] = fmaf(wr[j][e], dz[j][e], o[e]);
        }
        // o is the gradient of sequence position s (x of token s - W1, or history row s)
        const int t = s - W1;
        if (s < t1 + W1 && (t >= t0 || (t < 0 && run == 0))) {
          const int je = s - len;  // which row of state_end this input is, if any
          if (dstate_end && je >= 0 && je < W1) {
            float f[VEC];
            unpack<T, VEC>(*reinterpret_cast<const V*>(
                               dstate_end + ((long long)bh * W1 + je) * g.d + c0), f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] += f[e];
          }
          if (t >= len) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = 0.f;
          }
          if (t >= 0)
            *reinterpret_cast<V*>(dxrow + (long long)t * g.d + c0) = pack<T, VEC>(o);
          else if (dstate)
            *reinterpret_cast<V*>(dstate + ((long long)bh * W1 + s) * g.d + c0) = pack<T, VEC>(o);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
#pragma unroll
          for (int j = 0; j < W1; ++j) win[j][e] = win[j + 1][e];
#pragma unroll
          for (int j = W1; j > 0; --j) dz[j][e] = dz[j - 1][e];
        }
      }
    }
  }
  // Sums over this block's runs, one tap at a time, in the order of the runs.
  const long long slot = ((long long)b * gridDim.x + blockIdx.x) * g.H + h;
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) sums[threadIdx.x * VEC + e] = j < W ? dw[j < W ? j : 0][e] : db[e];
    __syncthreads();
    for (int i = threadIdx.x; i < g.nvt * VEC; i += blockDim.x) {
      const int c = blockIdx.z * g.nvt * VEC + i;
      if (c >= g.d) continue;
      float s = 0.f;
      for (int r = 0; r < g.rows; ++r) s += sums[r * g.nvt * VEC + i];
      part[(slot * (W + 1) + j) * g.d + c] = s;
    }
  }
}

// dw [H][d][W], dbias [H][d]: sums of `n` partial rows, in order. A block's 8
// warps share the rows of 32 channels.
template <int W>
__global__ void __launch_bounds__(256) conv_sum_kernel(const float* __restrict__ part, int n, int H,
                                                       int d, float* __restrict__ dw,
                                                       float* __restrict__ dbias) {
  __shared__ float s[8][32];
  const int c = blockIdx.x * 32 + threadIdx.x % 32, way = threadIdx.x / 32;
  const int j = blockIdx.y, h = blockIdx.z;
  float a = 0.f;
  if (c < d)
#pragma unroll 4
    for (int i = way; i < n; i += 8) a += part[(((long long)i * H + h) * (W + 1) + j) * d + c];
  s[way][threadIdx.x % 32] = a;
  __syncthreads();
  if (way == 0 && c < d) {
    for (int i = 1; i < 8; ++i) a += s[i][threadIdx.x];
    if (j < W)
      dw[((long long)h * d + c) * W + j] = a;
    else if (dbias)
      dbias[(long long)h * d + c] = a;
  }
}

template <typename T, int W, int VEC>
__global__ void __launch_bounds__(kThreads)
    conv_step_kernel(int BH, int H, int d, bool silu, const T* __restrict__ x,
                     const float* __restrict__ w, const float* __restrict__ bias,
                     T* __restrict__ state, T* __restrict__ y) {
  typedef typename VecOf<T, VEC>::type V;
  constexpr int W1 = W - 1;
  const int nvec = d / VEC;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (id >= (long long)BH * nvec) return;
  const int bh = (int)(id / nvec), c0 = (int)(id % nvec) * VEC, h = bh % H;
  T* srow = state + (long long)bh * W1 * d + c0;
  V raw[W];
#pragma unroll
  for (int j = 0; j < W1; ++j) raw[j] = *reinterpret_cast<const V*>(srow + (long long)j * d);
  raw[W1] = *reinterpret_cast<const V*>(x + (long long)bh * d + c0);
  float o[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) o[e] = bias ? bias[h * d + c0 + e] : 0.f;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    float f[VEC];
    unpack<T, VEC>(raw[j], f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = fmaf(w[((long long)h * d + c0 + e) * W + j], f[e], o[e]);
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) o[e] = silu ? o[e] * sigmoid_fast(o[e]) : o[e];
  *reinterpret_cast<V*>(y + (long long)bh * d + c0) = pack<T, VEC>(o);
#pragma unroll
  for (int j = 0; j < W1; ++j) *reinterpret_cast<V*>(srow + (long long)j * d) = raw[j + 1];
}

Geo geometry(const ConvDims& s, int vec) {
  Geo g{};
  g.H = s.H;
  g.T = s.T;
  g.d = s.d;
  g.silu = s.silu;
  g.nvec = s.d / vec;
  g.nvt = g.nvec < kThreads ? g.nvec : kThreads;
  g.rows = kThreads / g.nvt;
  g.R = 16;
  g.runs = (s.T + g.R - 1) / g.R;
  return g;
}

// Blocks along the tokens of one (batch row, head) in the backward: every block
// leaves one partial row per head, so long rows are looped over rather than
// spread over more than what fills the GPU.
int bwd_blocks_x(const ConvDims& s, const Geo& g) {
  const int tiles = (g.runs + g.rows - 1) / g.rows;
  const long long want = (148LL * 8 + (long long)s.B * s.H - 1) / ((long long)s.B * s.H);
  return (int)(tiles < want ? tiles : want);
}

template <typename T, int W, int VEC>
cudaError_t fwd_t(const ConvArgs& a, void* y, void* state_end) {
  const Geo g = geometry(a.s, VEC);
  dim3 grid((g.runs + g.rows - 1) / g.rows, a.s.B * a.s.H, (g.nvec + g.nvt - 1) / g.nvt);
  E2TTT_TRACE("conv_fwd", a.st);
  conv_fwd_kernel<T, W, VEC><<<grid, g.nvt * g.rows, 0, a.st>>>(
      g, (const T*)a.x, a.w, a.bias, (const T*)a.state, a.lengths, (T*)y, (T*)state_end);
  return cudaGetLastError();
}

template <typename T, int W, int VEC>
cudaError_t bwd_t(const ConvArgs& a, const void* dy, const void* dstate_end, void* dx, float* dw,
                  float* dbias, void* dstate, void* ws) {
  const Geo g = geometry(a.s, VEC);
  const int gx = bwd_blocks_x(a.s, g);
  dim3 grid(gx, a.s.B * a.s.H, (g.nvec + g.nvt - 1) / g.nvt);
  const int threads = g.nvt * g.rows;
  {
    E2TTT_TRACE("conv_bwd", a.st);
    conv_bwd_kernel<T, W, VEC><<<grid, threads, threads * VEC * sizeof(float), a.st>>>(
        g, (const T*)a.x, a.w, a.bias, (const T*)a.state, a.lengths, (const T*)dy,
        (const T*)dstate_end, (T*)dx, (T*)dstate, (float*)ws);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  E2TTT_TRACE("conv_sum", a.st);
  conv_sum_kernel<W><<<dim3((a.s.d + 31) / 32, W + 1, a.s.H), 256, 0, a.st>>>(
      (const float*)ws, a.s.B * gx, a.s.H, a.s.d, dw, dbias);
  return cudaGetLastError();
}

template <typename T, int W, int VEC>
cudaError_t step_t(const ConvArgs& a, void* state, void* y) {
  const long long n = (long long)a.s.B * a.s.H * (a.s.d / VEC);
  E2TTT_TRACE("conv_step", a.st);
  conv_step_kernel<T, W, VEC><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, a.st>>>(
      a.s.B * a.s.H, a.s.H, a.s.d, a.s.silu, (const T*)a.x, a.w, a.bias, (T*)state, (T*)y);
  return cudaGetLastError();
}

// The instantiations: activation type, width, vectors or single channels.
#define CONV_WIDTHS(F, T, VEC, ...)                    \
  switch (a.s.W) {                                     \
    case 1: return F<T, 1, VEC>(__VA_ARGS__);          \
    case 2: return F<T, 2, VEC>(__VA_ARGS__);          \
    case 3: return F<T, 3, VEC>(__VA_ARGS__);          \
    case 4: return F<T, 4, VEC>(__VA_ARGS__);          \
    case 5: return F<T, 5, VEC>(__VA_ARGS__);          \
    case 6: return F<T, 6, VEC>(__VA_ARGS__);          \
    case 7: return F<T, 7, VEC>(__VA_ARGS__);          \
    case 8: return F<T, 8, VEC>(__VA_ARGS__);          \
  }                                                    \
  return cudaErrorInvalidValue;
#define CONV_DISPATCH(F, ...)                          \
  if (a.s.bf16_act) {                                  \
    if (a.vec) { CONV_WIDTHS(F, bf16, 8, __VA_ARGS__) } \
    CONV_WIDTHS(F, bf16, 1, __VA_ARGS__)               \
  }                                                    \
  if (a.vec) { CONV_WIDTHS(F, float, 4, __VA_ARGS__) } \
  CONV_WIDTHS(F, float, 1, __VA_ARGS__)

}  // namespace

size_t conv_bwd_workspace_bytes(const ConvDims& s) {
  // whichever of the vector and single-channel forms runs (alignment decides at the call)
  size_t most = 0;
  for (int vec : {1, s.bf16_act ? 8 : 4}) {
    if (s.d % vec) continue;
    const size_t n = (size_t)s.B * bwd_blocks_x(s, geometry(s, vec)) * s.H * (s.W + 1) * s.d * sizeof(float);
    if (n > most) most = n;
  }
  return most;
}

cudaError_t conv_fwd(const ConvArgs& a, void* y, void* state_end) {
  CONV_DISPATCH(fwd_t, a, y, state_end)
}
cudaError_t conv_bwd(const ConvArgs& a, const void* dy, const void* dstate_end, void* dx, float* dw,
                     float* dbias, void* dstate, void* ws) {
  CONV_DISPATCH(bwd_t, a, dy, dstate_end, dx, dw, dbias, dstate, ws)
}
cudaError_t conv_step(const ConvArgs& a, void* state, void* y) {
  CONV_DISPATCH(step_t, a, state, y)
}

}  // namespace e2ttt
