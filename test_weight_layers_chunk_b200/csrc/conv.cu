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
// dy and writes dx. A thread owns four consecutive channels and walks a run
// of R consecutive tokens with the last W inputs (and, backward, the last W dz)
// in registers, so a run re-reads only the W-1 tokens before it (and the
// backward the W-1 after it), which the neighbouring run has just brought into
// L1/L2. Threads of a warp cover consecutive channels, then consecutive runs.
// 4 x 8 heads x 2048 tokens x 256 channels, W = 4, bf16 with silu: forward 18 us
// (67 MB), backward 34 us with its sums (101 MB), where the bytes take 10 and 16; fp32:
// 26 and 44 us, where they take 21 and 31. No unit is full (bf16: MUFU 51 and 28 % busy
// with two operations an element, issue 45 and 44 %, DRAM 21 and 26 %): with 37 and 21 %
// of the warps' places taken, what is left is latency that they do not cover. Packed
// fp32 pairs, whole batches without predicates and asynchronous copies brought them
// from 40 and 97 us; eight channels a thread needed too many registers.
#include "seq_ops.h"
#include "trace.h"

namespace e2ttt {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxW = 8;

// Pairs of fp32 values, for the packed fp32 instructions: one issue for two
// channels, each rounded as by itself.
typedef float2 F2;
__device__ __forceinline__ unsigned long long bits(F2 a) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ F2 pair(unsigned long long b) {
  F2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return pair(r);
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return pair(r);
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return pair(r);
}
__device__ __forceinline__ F2 both(float x) { return F2{x, x}; }
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 1 / (1 + exp(-z)); exp overflows to infinity for z << 0, whose reciprocal is 0.
__device__ __forceinline__ F2 sigmoid2(F2 z) {
  const F2 a = mul2(z, both(-1.4426950408889634f));
  const F2 b = add2(F2{ex2(a.x), ex2(a.y)}, both(1.0f));
  return F2{rcp(b.x), rcp(b.y)};
}

template <typename T, int VEC> struct VecOf;
template <> struct VecOf<bf16, 4> { typedef uint2 type; };
template <> struct VecOf<float, 4> { typedef uint4 type; };
template <> struct VecOf<bf16, 1> { typedef unsigned short type; };
template <> struct VecOf<float, 1> { typedef unsigned int type; };

// A thread's VEC channels as NP pairs (one channel: a pair with a spare half).
template <typename T, int VEC>
__device__ __forceinline__ void unpack(const typename VecOf<T, VEC>::type& r, F2 (&f)[(VEC + 1) / 2]) {
  const T* p = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int i = 0; i < (VEC + 1) / 2; ++i) f[i] = F2{to_f<T>(p[2 * i]), VEC > 1 ? to_f<T>(p[VEC > 1 ? 2 * i + 1 : 0]) : 0.f};
}
template <typename T, int VEC>
__device__ __forceinline__ typename VecOf<T, VEC>::type pack(const F2 (&f)[(VEC + 1) / 2]) {
  typename VecOf<T, VEC>::type r;
  T* p = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int i = 0; i < (VEC + 1) / 2; ++i) {
    p[2 * i] = from_f<T>(f[i].x);
    if (VEC > 1) p[VEC > 1 ? 2 * i + 1 : 0] = from_f<T>(f[i].y);
  }
  return r;
}
template <int NP>
__device__ __forceinline__ void zero(F2 (&f)[NP]) {
#pragma unroll
  for (int i = 0; i < NP; ++i) f[i] = both(0.f);
}

struct Geo {
  int H, T, d, nvec, nvt, rows;  // vectors per token, vectors per block, runs per block
  int runs;                      // runs of R tokens in T
  int R;
};

__device__ __forceinline__ int row_length(const int* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

// The W taps of VEC consecutive channels: contiguous in memory, read as 16-byte
// vectors where the first one is aligned.
template <int W, int VEC>
__device__ __forceinline__ void load_taps(const float* w, F2 (&wr)[W][(VEC + 1) / 2]) {
  float flat[W * VEC];
  if (VEC > 1 && (((uintptr_t)w) & 15) == 0) {
#pragma unroll
    for (int i = 0; i < W * VEC / 4; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(w + 4 * i);
      flat[4 * i] = v.x, flat[4 * i + 1] = v.y, flat[4 * i + 2] = v.z, flat[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < W * VEC; ++i) flat[i] = w[i];
  }
#pragma unroll
  for (int i = 0; i < (VEC + 1) / 2; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j)
      wr[j][i] = F2{flat[2 * i * W + j], VEC > 1 ? flat[(VEC > 1 ? 2 * i + 1 : 0) * W + j] : 0.f};
}
template <int VEC>
__device__ __forceinline__ void load_bias(const float* bias, F2 (&br)[(VEC + 1) / 2]) {
#pragma unroll
  for (int i = 0; i < (VEC + 1) / 2; ++i)
    br[i] = bias ? F2{bias[2 * i], VEC > 1 ? bias[VEC > 1 ? 2 * i + 1 : 0] : 0.f} : both(0.f);
}

// Input at position i of the sequence [state; x[0..len)] (i = 0 is the oldest
// history row), zero outside it.
template <typename T, int VEC>
__device__ __forceinline__ void load_seq(const T* xrow, const T* srow, int i, int W1, int len,
                                         int d, int c0, F2 (&f)[(VEC + 1) / 2]) {
  typedef typename VecOf<T, VEC>::type V;
  const T* p = nullptr;
  if (i >= W1) {
    if (i - W1 < len) p = xrow + (long long)(i - W1) * d + c0;
  } else if (srow && i >= 0) {
    p = srow + (long long)i * d + c0;
  }
  if (p)
    unpack<T, VEC>(*reinterpret_cast<const V*>(p), f);
  else
    zero(f);
}

constexpr int kBatch = 4;   // tokens that are computed together

// A thread's own ring of raw rows in shared memory, filled by asynchronous copies
// several batches ahead without holding registers; no other thread reads it, so it
// needs no barrier. Single channels of two bytes are too small for such copies and
// are loaded when they are needed.
template <typename T, int VEC, int STREAMS>
struct Ring {
  typedef typename VecOf<T, VEC>::type V;
  static constexpr bool kAsync = sizeof(V) >= 4;
  // Batches whose loads are in flight beyond the current one (two of 16 bytes keep a
  // block's ring within the 48 KB that need no asking for).
  static constexpr int kAhead = sizeof(V) == 16 ? 2 : 3, kRing = kAhead + 1;
  V* slots;  // [kRing][STREAMS][kBatch][threads]
  int threads;
  __device__ __forceinline__ V* slot(int batch, int stream, int i) const {
    return slots + (((batch % kRing) * STREAMS + stream) * kBatch + i) * threads + threadIdx.x;
  }
  // Rows p, p + d, .. of one batch.
  __device__ __forceinline__ void copy(int batch, int stream, const T* p, int d) const {
    if constexpr (kAsync) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(slot(batch, stream, i));
        if constexpr (sizeof(V) == 16)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
        else
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(p), "n"(sizeof(V)) : "memory");
        p += d;
      }
    }
  }
  // Ends one batch of copies (an empty one too: the groups are counted).
  __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // The batch that was committed kAhead batches before the last one has landed.
  __device__ __forceinline__ void landed() const { asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory"); }
  __device__ __forceinline__ void read(V (&raw)[kBatch], int batch, int stream, const T* p, int d) const {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if constexpr (kAsync)
        raw[i] = *slot(batch, stream, i);
      else
        raw[i] = *reinterpret_cast<const V*>(p);
      p += d;
    }
  }
};

template <typename T, int W, int VEC, bool SILU>
__global__ void __launch_bounds__(kThreads, W <= 4 ? 4 : 2) conv_fwd_kernel(Geo g, const T* __restrict__ x,
                                                            const float* __restrict__ w,
                                                            const float* __restrict__ bias,
                                                            const T* __restrict__ state,
                                                            const int* __restrict__ lengths,
                                                            T* __restrict__ y,
                                                            T* __restrict__ state_end) {
  typedef typename VecOf<T, VEC>::type V;
  constexpr int W1 = W - 1, NP = (VEC + 1) / 2;
  const int bh = blockIdx.y, h = bh % g.H;
  const int vi = blockIdx.z * g.nvt + threadIdx.x % g.nvt;
  const int run = blockIdx.x * g.rows + threadIdx.x / g.nvt;
  if (vi >= g.nvec || run >= g.runs) return;
  const int c0 = vi * VEC, len = row_length(lengths, bh / g.H, g.T);
  const T* xrow = x + (long long)bh * g.T * g.d;
  T* yrow = y + (long long)bh * g.T * g.d;
  const T* srow = state ? state + (long long)bh * W1 * g.d : nullptr;
  const int t0 = run * g.R, t1 = min(t0 + g.R, g.T), end = min(t1, len);
  const int full = end > t0 ? (end - t0) / kBatch : 0;  // whole batches of tokens that exist

  const T* xp = xrow + (long long)t0 * g.d + c0;
  T* yp = yrow + (long long)t0 * g.d + c0;
  extern __shared__ __align__(16) uint8_t ring_bytes[];
  typedef Ring<T, VEC, 1> R;
  constexpr int kAhead = R::kAhead;
  const R ring{reinterpret_cast<V*>(ring_bytes), (int)blockDim.x};
  const long long step = (long long)kBatch * g.d;
#pragma unroll
  for (int n = 0; n < kAhead; ++n) {
    if (n < full) ring.copy(n, 0, xp + n * step, g.d);
    ring.commit();
  }
  F2 wr[W][NP], br[NP];
  load_taps<W, VEC>(w + ((long long)h * g.d + c0) * W, wr);
  load_bias<VEC>(bias ? bias + h * g.d + c0 : nullptr, br);
  F2 win[W][NP];  // the W inputs that end at the current token
#pragma unroll
  for (int j = 0; j < W1; ++j) load_seq<T, VEC>(xrow, srow, t0 + j, W1, len, g.d, c0, win[j]);

  auto token = [&](const V& raw, F2(&o)[NP]) {
    unpack<T, VEC>(raw, win[W1]);
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      F2 z = br[e];
#pragma unroll
      for (int j = 0; j < W; ++j) z = fma2(wr[j][e], win[j][e], z);
      o[e] = SILU ? mul2(z, sigmoid2(z)) : z;
#pragma unroll
      for (int j = 0; j < W1; ++j) win[j][e] = win[j + 1][e];
    }
  };
#pragma unroll 1
  for (int n = 0; n < full; ++n) {
    if (n + kAhead < full) ring.copy(n + kAhead, 0, xp + kAhead * step, g.d);
    ring.commit();
    ring.landed();
    V raw[kBatch];
    ring.read(raw, n, 0, xp, g.d);
    xp += step;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      F2 o[NP];
      token(raw[i], o);
      *reinterpret_cast<V*>(yp) = pack<T, VEC>(o);
      yp += g.d;
    }
  }
#pragma unroll 1
  for (int t = t0 + full * kBatch; t < t1; ++t) {
    F2 o[NP];
    V raw{};
    if (t < end) raw = *reinterpret_cast<const V*>(xp);
    token(raw, o);
    if (t >= end) zero(o);
    *reinterpret_cast<V*>(yp) = pack<T, VEC>(o);
    xp += g.d;
    yp += g.d;
  }
  if (state_end && run == 0) {
#pragma unroll
    for (int j = 0; j < W1; ++j) {
      F2 f[NP];
      load_seq<T, VEC>(xrow, srow, len + j, W1, len, g.d, c0, f);
      *reinterpret_cast<V*>(state_end + ((long long)bh * W1 + j) * g.d + c0) = pack<T, VEC>(f);
    }
  }
}

// part [B * gridDim.x][H][W + 1][d]: this block's sums of dz x (taps 0..W-1) and dz.
// A run's walk goes W - 1 tokens past its end: their dz reach back into it.
template <typename T, int W, int VEC, bool SILU>
__global__ void __launch_bounds__(kThreads, W <= 4 ? 2 : 1)
    conv_bwd_kernel(Geo g, const T* __restrict__ x, const float* __restrict__ w,
                    const float* __restrict__ bias, const T* __restrict__ state,
                    const int* __restrict__ lengths, const T* __restrict__ dy,
                    const T* __restrict__ dstate_end, T* __restrict__ dx, T* __restrict__ dstate,
                    float* __restrict__ part) {
  typedef typename VecOf<T, VEC>::type V;
  constexpr int W1 = W - 1, NP = (VEC + 1) / 2;
  extern __shared__ __align__(16) uint8_t ring_bytes[];
  float* sums = reinterpret_cast<float*>(ring_bytes);  // [blockDim.x][VEC], after the runs
  typedef Ring<T, VEC, 2> R;
  constexpr int kAhead = R::kAhead;
  const R ring{reinterpret_cast<V*>(ring_bytes), (int)blockDim.x};
  const long long step = (long long)kBatch * g.d;
  const int bh = blockIdx.y, h = bh % g.H, b = bh / g.H;
  const int vl = threadIdx.x % g.nvt, vi = blockIdx.z * g.nvt + vl, c0 = vi * VEC;
  const bool on = vi < g.nvec;
  const int len = row_length(lengths, b, g.T);
  const T* xrow = x + (long long)bh * g.T * g.d;
  const T* dyrow = dy + (long long)bh * g.T * g.d;
  T* dxrow = dx + (long long)bh * g.T * g.d;
  const T* srow = state ? state + (long long)bh * W1 * g.d : nullptr;

  F2 wr[W][NP], br[NP], dw[W][NP], db[NP];
  if (on) {
    load_taps<W, VEC>(w + ((long long)h * g.d + c0) * W, wr);
    load_bias<VEC>(bias ? bias + h * g.d + c0 : nullptr, br);
  }
  zero(db);
#pragma unroll
  for (int j = 0; j < W; ++j) zero(dw[j]);
#pragma unroll 1
  for (int run = blockIdx.x * g.rows + threadIdx.x / g.nvt; on && run < g.runs;
       run += gridDim.x * g.rows) {
    const int t0 = run * g.R, t1 = min(t0 + g.R, g.T), last = t1 + W1;
    const int end = min(t1, len), full = end > t0 ? (end - t0) / kBatch : 0;
    const T* xp = xrow + (long long)t0 * g.d + c0;
    const T* gp = dyrow + (long long)t0 * g.d + c0;
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      if (n < full) {
        ring.copy(n, 0, xp + n * step, g.d);
        ring.copy(n, 1, gp + n * step, g.d);
      }
      ring.commit();
    }
    F2 win[W][NP], dz[W][NP];  // dz[j]: of the token j before the current one
#pragma unroll
    for (int j = 0; j < W; ++j) zero(dz[j]);
#pragma unroll
    for (int j = 0; j < W1; ++j) load_seq<T, VEC>(xrow, srow, t0 + j, W1, len, g.d, c0, win[j]);

    // One token s: its dz, its sums (`mine`: it belongs to this run), and the
    // gradient o of sequence position s (x of token s - W1, or history row s).
    auto token = [&](const V& rx, const V& rd, bool mine, F2(&o)[NP]) {
      F2 gy[NP];
      unpack<T, VEC>(rx, win[W1]);
      unpack<T, VEC>(rd, gy);
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        if constexpr (SILU) {
          F2 z = br[e];
#pragma unroll
          for (int j = 0; j < W; ++j) z = fma2(wr[j][e], win[j][e], z);
          const F2 sg = sigmoid2(z);
          const F2 f = fma2(z, fma2(sg, both(-1.f), both(1.f)), both(1.f));  // y' = sg (1 + z (1 - sg))
          dz[0][e] = mul2(gy[e], mul2(sg, f));
        } else {
          dz[0][e] = gy[e];
        }
        if (mine) {
          db[e] = add2(db[e], dz[0][e]);
#pragma unroll
          for (int j = 0; j < W; ++j) dw[j][e] = fma2(dz[0][e], win[j][e], dw[j][e]);
        }
        o[e] = mul2(wr[0][e], dz[0][e]);
#pragma unroll
        for (int j = 1; j < W; ++j) o[e] = fma2(wr[j][e], dz[j][e], o[e]);
#pragma unroll
        for (int j = 0; j < W1; ++j) win[j][e] = win[j + 1][e];
#pragma unroll
        for (int j = W1; j > 0; --j) dz[j][e] = dz[j - 1][e];
      }
    };
    T* op = dxrow + (long long)(t0 - W1) * g.d + c0;  // where token s's o goes
#pragma unroll 1
    for (int n = 0; n < full; ++n) {
      if (n + kAhead < full) {
        ring.copy(n + kAhead, 0, xp + kAhead * step, g.d);
        ring.copy(n + kAhead, 1, gp + kAhead * step, g.d);
      }
      ring.commit();
      ring.landed();
      V rx[kBatch], rd[kBatch];
      ring.read(rx, n, 0, xp, g.d);
      ring.read(rd, n, 1, gp, g.d);
      xp += step;
      gp += step;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        F2 o[NP];
        token(rx[i], rd[i], true, o);
        if (n * kBatch + i >= W1)
          *reinterpret_cast<V*>(op) = pack<T, VEC>(o);
        else if (run == 0 && dstate)
          *reinterpret_cast<V*>(dstate + ((long long)bh * W1 + n * kBatch + i) * g.d + c0) = pack<T, VEC>(o);
        op += g.d;
      }
    }
    int s = t0 + full * kBatch;
    if (s == t1 && last <= len && full * kBatch >= W1) {
      // the tokens past the run, all there
#pragma unroll
      for (int i = 0; i < W1; ++i) {
        F2 o[NP];
        token(*reinterpret_cast<const V*>(xp), *reinterpret_cast<const V*>(gp), false, o);
        *reinterpret_cast<V*>(op) = pack<T, VEC>(o);
        xp += g.d;
        gp += g.d;
        op += g.d;
      }
    } else {
#pragma unroll 1
      for (; s < last; ++s) {
        const int t = s - W1;
        F2 o[NP];
        V vx{}, vd{};
        if (s < len) {
          vx = *reinterpret_cast<const V*>(xp);
          vd = *reinterpret_cast<const V*>(gp);
        }
        token(vx, vd, s < t1, o);
        const int je = s - len;  // which row of state_end this input is, if any
        if (dstate_end && je >= 0 && je < W1) {
          F2 f[NP];
          unpack<T, VEC>(*reinterpret_cast<const V*>(dstate_end + ((long long)bh * W1 + je) * g.d + c0), f);
#pragma unroll
          for (int e = 0; e < NP; ++e) o[e] = add2(o[e], f[e]);
        }
        if (t >= len) zero(o);
        if (t >= t0)
          *reinterpret_cast<V*>(op) = pack<T, VEC>(o);
        else if (run == 0 && dstate)
          *reinterpret_cast<V*>(dstate + ((long long)bh * W1 + s) * g.d + c0) = pack<T, VEC>(o);
        xp += g.d;
        gp += g.d;
        op += g.d;
      }
    }
  }
  // Sums over this block's runs, one tap at a time, in the order of the runs.
  const long long slot = ((long long)b * gridDim.x + blockIdx.x) * g.H + h;
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const F2 v = j < W ? dw[j < W ? j : 0][e] : db[e];
      sums[threadIdx.x * VEC + 2 * e] = v.x;
      if (VEC > 1) sums[threadIdx.x * VEC + 2 * e + 1] = v.y;
    }
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
// warps share the rows of 32 channels. Resets the workspace's status word: nothing waits.
template <int W>
__global__ void __launch_bounds__(256) conv_sum_kernel(const float* __restrict__ part, int n, int H,
                                                       int d, float* __restrict__ dw,
                                                       float* __restrict__ dbias, int* __restrict__ status) {
  __shared__ float s[8][32];
  if (blockIdx.x + blockIdx.y + blockIdx.z + threadIdx.x == 0) *status = 0;
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
  constexpr int W1 = W - 1, NP = (VEC + 1) / 2;
  const int nvec = d / VEC;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (id >= (long long)BH * nvec) return;
  const int bh = (int)(id / nvec), c0 = (int)(id % nvec) * VEC, h = bh % H;
  T* srow = state + (long long)bh * W1 * d + c0;
  V raw[W];
#pragma unroll
  for (int j = 0; j < W1; ++j) raw[j] = *reinterpret_cast<const V*>(srow + (long long)j * d);
  raw[W1] = *reinterpret_cast<const V*>(x + (long long)bh * d + c0);
  F2 wr[W][NP], o[NP];
  load_taps<W, VEC>(w + ((long long)h * d + c0) * W, wr);
  load_bias<VEC>(bias ? bias + h * d + c0 : nullptr, o);
#pragma unroll
  for (int j = 0; j < W; ++j) {
    F2 f[NP];
    unpack<T, VEC>(raw[j], f);
#pragma unroll
    for (int e = 0; e < NP; ++e) o[e] = fma2(wr[j][e], f[e], o[e]);
  }
#pragma unroll
  for (int e = 0; e < NP; ++e) o[e] = silu ? mul2(o[e], sigmoid2(o[e])) : o[e];
  *reinterpret_cast<V*>(y + (long long)bh * d + c0) = pack<T, VEC>(o);
#pragma unroll
  for (int j = 0; j < W1; ++j) *reinterpret_cast<V*>(srow + (long long)j * d) = raw[j + 1];
}

Geo geometry(const ConvDims& s, int vec, bool back) {
  Geo g{};
  g.H = s.H;
  g.T = s.T;
  g.d = s.d;
  g.nvec = s.d / vec;
  g.nvt = g.nvec < kThreads ? g.nvec : kThreads;
  g.rows = kThreads / g.nvt;
  // Long runs re-read and recompute less (W - 1 tokens a run, which the backward
  // walks twice); short ones give more threads. The longest that still gives every
  // SM 768 threads, in the backward (half as many fit) 384.
  g.R = back ? 64 : 32;
  const long long enough = (long long)kPlannedSms * (back ? 384 : 768);
  while (g.R > 8 && (long long)s.B * s.H * g.nvec * ((s.T + g.R - 1) / g.R) < enough) g.R /= 2;
  g.runs = (s.T + g.R - 1) / g.R;
  return g;
}

// Blocks along the tokens of one (batch row, head) in the backward: every block
// leaves one partial row per head, so long rows are looped over rather than
// spread over more than what fills the GPU.
int bwd_blocks_x(const ConvDims& s, const Geo& g) {
  const int tiles = (g.runs + g.rows - 1) / g.rows;
  const long long want = (kPlannedSms * 8LL + (long long)s.B * s.H - 1) / ((long long)s.B * s.H);
  return (int)(tiles < want ? tiles : want);
}

// Shared memory of a block: its ring, or the sums that follow it.
template <typename T, int VEC, int STREAMS>
size_t ring_bytes(int threads) {
  typedef Ring<T, VEC, STREAMS> R;
  const size_t ring = R::kAsync ? sizeof(typename R::V) * R::kRing * STREAMS * kBatch * threads : 0;
  const size_t sums = sizeof(float) * VEC * threads;
  return ring > sums ? ring : sums;
}

template <class F>
cudaError_t allow_smem(F* f, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int W, int VEC>
cudaError_t fwd_t(const ConvArgs& a, void* y, void* state_end) {
  const Geo g = geometry(a.s, VEC, false);
  dim3 grid((g.runs + g.rows - 1) / g.rows, a.s.B * a.s.H, (g.nvec + g.nvt - 1) / g.nvt);
  E2TTT_TRACE("conv_fwd", a.st);
  auto kern = a.s.silu ? conv_fwd_kernel<T, W, VEC, true> : conv_fwd_kernel<T, W, VEC, false>;
  const int threads = g.nvt * g.rows;
  const size_t smem = ring_bytes<T, VEC, 1>(threads);
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, threads, smem, a.st>>>(
      g, (const T*)a.x, a.w, a.bias, (const T*)a.state, a.lengths, (T*)y, (T*)state_end);
  return cudaGetLastError();
}

template <typename T, int W, int VEC>
cudaError_t bwd_t(const ConvArgs& a, const void* dy, const void* dstate_end, void* dx, float* dw,
                  float* dbias, void* dstate, void* ws) {
  const Geo g = geometry(a.s, VEC, true);
  const int gx = bwd_blocks_x(a.s, g);
  dim3 grid(gx, a.s.B * a.s.H, (g.nvec + g.nvt - 1) / g.nvt);
  const int threads = g.nvt * g.rows;
  float* part = (float*)((char*)ws + kStatusBytes);
  {
    E2TTT_TRACE("conv_bwd", a.st);
    auto kern = a.s.silu ? conv_bwd_kernel<T, W, VEC, true> : conv_bwd_kernel<T, W, VEC, false>;
    const size_t smem = ring_bytes<T, VEC, 2>(threads);
    cudaError_t e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    kern<<<grid, threads, smem, a.st>>>(
        g, (const T*)a.x, a.w, a.bias, (const T*)a.state, a.lengths, (const T*)dy,
        (const T*)dstate_end, (T*)dx, (T*)dstate, part);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  E2TTT_TRACE("conv_sum", a.st);
  conv_sum_kernel<W><<<dim3((a.s.d + 31) / 32, W + 1, a.s.H), 256, 0, a.st>>>(
      part, a.s.B * gx, a.s.H, a.s.d, dw, dbias, (int*)ws);
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
    if (a.vec) { CONV_WIDTHS(F, bf16, 4, __VA_ARGS__) } \
    CONV_WIDTHS(F, bf16, 1, __VA_ARGS__)               \
  }                                                    \
  if (a.vec) { CONV_WIDTHS(F, float, 4, __VA_ARGS__) } \
  CONV_WIDTHS(F, float, 1, __VA_ARGS__)

}  // namespace

size_t conv_bwd_workspace_bytes(const ConvDims& s) {
  // whichever of the vector and single-channel forms runs (alignment decides at the call)
  size_t most = 0;
  for (int vec : {1, 4}) {
    if (s.d % vec) continue;
    const size_t n = (size_t)s.B * bwd_blocks_x(s, geometry(s, vec, true)) * s.H * (s.W + 1) * s.d * sizeof(float);
    if (n > most) most = n;
  }
  return kStatusBytes + most;
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
