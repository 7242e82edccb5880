// State-space scan on the tensor cores (bf16 activations, at most 128 state
// columns; any alignment, odd sizes padded with zeros in shared memory). The
// mathematics is in ssm.cuh; chunks are of 128 tokens, so that every product of
// a chunk is one 128-row tcgen05 tile with its accumulator in tensor memory.
//
// A matrix lies in shared memory as columns of 64 bf16 (128-byte rows, 128-byte
// swizzle). The same bytes serve as a K-major operand (its columns contracted)
// and as an MN-major one (its rows contracted), so nothing is transposed.
//
// Precision. Inputs are bf16 and enter the products as they are. What is not an
// input is rounded once to bf16 where its product ends in a bf16 result (the
// decayed scores, the state in y and dv); where the product ends in an fp32
// result (the states, and the dots behind ddt and dA) it enters as three bf16
// terms that together hold all 24 bits of it, each with a product of its own.
#include <atomic>
#include <initializer_list>

#include "ssm.cuh"
#include "tc_gemm2.cuh"
#include "trace.h"

namespace e2ttt {
namespace {

using tc2::idesc;
using tc2::smem_u32;

constexpr int kQ = kSsmTcChunk;  // tokens per chunk
constexpr int kThreads = 512;    // 16 warps: tensor-memory lanes 32 (w & 3), a share of the columns each
constexpr int kPT = kSsmPT;

// Byte offset of 16-byte piece `j` (8 columns) of row r in a tile of ROWS rows.
template <int ROWS>
__device__ __forceinline__ uint32_t piece(int r, int j) {
  return (uint32_t)((j >> 3) * ROWS * 128 + r * 128 + (((j & 7) ^ (r & 7)) << 4));
}

// Descriptor of such a tile: `mn` for the MN-major reading (64-column blocks
// ROWS * 128 bytes apart).
template <int ROWS>
__device__ __forceinline__ uint64_t tile_desc(const uint8_t* p, bool mn) {
  uint64_t d = (uint64_t)((smem_u32(p) & 0x3FFFFu) >> 4);
  d |= (uint64_t)(mn ? (ROWS * 128) >> 4 : 1) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// Start-address advance of contraction step k (16 deep), in 16-byte units.
template <int ROWS, bool MN>
__device__ __forceinline__ uint32_t step_off(int k) {
  return MN ? (uint32_t)(k * 2048) >> 4 : (uint32_t)((k >> 2) * ROWS * 128 + (k & 3) * 32) >> 4;
}
// acc[128][N] (+)= A B over `steps` steps of 16; A of AROWS stored rows, B of BROWS.
template <int AROWS, bool AMN, int BROWS, bool BMN, int N>
__device__ __forceinline__ void mma(uint32_t acc, const uint8_t* a, const uint8_t* b, int steps,
                                    bool add) {
  const uint64_t da = tile_desc<AROWS>(a, AMN), db = tile_desc<BROWS>(b, BMN);
  constexpr uint32_t id = idesc(128, N, AMN, BMN);
  for (int k = 0; k < steps; ++k)
    tc::mma_bf16(acc, da + step_off<AROWS, AMN>(k), db + step_off<BROWS, BMN>(k), id, add || k);
}

// The waits that the failure-detection test hook (e2ttt_test_stall_next_scan) can make
// block (0, 0, 0) of the next launch that has them take for run out.
enum Stall : int { kNone, kStates, kScores, kRows, kOutputs, kDots, kPairs, kResults };
__device__ __forceinline__ bool stalled(int stall, int at) {
  return stall == at && blockIdx.x + blockIdx.y + blockIdx.z == 0;
}

// The waits of one block on its MMAs: one mbarrier, one phase per commit.
struct Mmas {
  uint64_t* bar;
  uint32_t phase;
  int* status;
  // True (for the whole block) once the last commit has completed; false, with
  // the status word set, where a thread waited about a second without it.
  __device__ __forceinline__ bool wait(bool stall) {
    const bool ok = tc::mbar_wait(bar, phase) && !stall;
    const bool all = __syncthreads_and(ok);
    if (!all) {  // whichever thread it was
      if (threadIdx.x == 0) atomicExch(status, tc2::kErrMma);
      // once more, so that the MMAs do not outlive their memory
      (void)tc::mbar_wait(bar, phase);
    }
    phase ^= 1u;
    tc::tc_fence_after();
    return all;
  }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Eight consecutive values of a row of `cols` from column c on, zeros beyond.
__device__ __forceinline__ uint4 load8(const bf16* row, int c, int cols) {
  uint4 r{0, 0, 0, 0};
  bf16* p = reinterpret_cast<bf16*>(&r);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < cols) p[i] = row[c + i];
  return r;
}

// Rows [0, n) of src (pitch ld, `cols` columns) into a tile of ROWS rows and
// BLOCKS 64-column blocks; everything else is zero. VEC: 16-byte copies apply.
template <int ROWS, int BLOCKS, bool VEC>
__device__ __forceinline__ void load_rows(uint8_t* tile, const bf16* src, long long ld, int n, int cols) {
  constexpr int kPer = BLOCKS * 8, kStep = kThreads / kPer;  // pieces in a row, rows at a time
  static_assert(kStep % 8 == 0 && ROWS % kStep == 0, "a thread's rows share their swizzle");
  const int j = threadIdx.x % kPer, r0 = threadIdx.x / kPer;
  const int left = j * 8 < cols ? n - r0 : 0;
  const bf16* p = src + r0 * ld + j * 8;
  uint8_t* dst = tile + piece<ROWS>(r0, j);
#pragma unroll
  for (int i = 0; i < ROWS / kStep; ++i) {
    const bool on = i * kStep < left;
    if constexpr (VEC)
      cp16(smem_u32(dst) + i * kStep * 128, on ? p : src, on);
    else
      *reinterpret_cast<uint4*>(dst + i * kStep * 128) =
          on ? load8(src + (long long)(r0 + i * kStep) * ld, j * 8, cols) : uint4{0, 0, 0, 0};
    p += kStep * ld;
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float lo_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Eight values to a row of which `left` columns remain.
template <bool VEC>
__device__ __forceinline__ void store8(bf16* out, const uint4& w, int left) {
  if constexpr (VEC) {
    if (left >= 8) *reinterpret_cast<uint4*>(out) = w;  // rows are whole pieces
  } else {
    const bf16* e = reinterpret_cast<const bf16*>(&w);
    for (int j = 0; j < 8 && j < left; ++j) out[j] = e[j];
  }
}

// Eight fp32 values of a row of which `left` remain (at most 0: none), zeros beyond.
template <bool VEC>
__device__ __forceinline__ void load8f(float (&f)[8], const float* p, int left) {
  if constexpr (VEC) {  // rows are whole pieces
    float4 a{0, 0, 0, 0}, b{0, 0, 0, 0};
    if (left > 0) {
      a = *reinterpret_cast<const float4*>(p);
      b = *reinterpret_cast<const float4*>(p + 4);
    }
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e < left ? p[e] : 0.f;
  }
}

// f as three bf16 terms that add up to it exactly (above the smallest exponents): each
// is what the ones before leave, cut off to its first eight bits, so that it is the
// upper half of a word as it stands. ROUND: the first term is f rounded to bf16, for a
// product that takes it alone (cut off, it would be 0.28 % too small on average);
// what that leaves has at most 16 bits for the other two.
template <bool ROUND = false>
__device__ __forceinline__ void split3(const float (&f)[8], uint4 (&t)[3]) {
  uint32_t* o[3] = {&t[0].x, &t[1].x, &t[2].x};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = f[2 * i], b = f[2 * i + 1];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const uint32_t w = ROUND && j == 0 ? pack2(a, b) : __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
      o[j][i] = w;
      a -= lo_f(w);
      b -= hi_f(w);
    }
  }
}

// Floats of a chunk's logs, which logs_kernel writes once per call to
// [B*H][NC][kLogRows][kQ].
constexpr int kLogs = kLogRows * kQ;

// One block per (chunk, batch row and head), one thread per token: its logs (see
// ChunkLogs) and the chunk's decay e^{c_Q}; resets the status word of the launches
// that follow.
__global__ void __launch_bounds__(kQ)
    logs_kernel(SsmDims s, const float* __restrict__ dt, const float* __restrict__ A,
                const int* __restrict__ lengths, float* __restrict__ logs,
                float* __restrict__ decay, int* __restrict__ status) {
  __shared__ double sums[kQ / 32];
  const int t = threadIdx.x, w = t >> 5, lane = t & 31, c = blockIdx.x, bh = blockIdx.y, b = bh / s.H;
  griddep_wait();
  griddep_launch_dependents();
  if (c == 0 && bh == 0 && t == 0) *status = 0;
  const int n = min(max(ssm_row_length(lengths, b, s.T) - c * kQ, 0), kQ);
  const float eta = t < n ? dt[(long long)bh * s.T + c * kQ + t] : 0.f;
  double x = eta * ((double)A[bh - b * s.H] * 1.4426950408889634);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(~0u, x, o);
    x += lane >= o ? u : 0.0;
  }
  if (lane == 31) sums[w] = x;
  __syncthreads();
  double before = 0.0, all = 0.0;
#pragma unroll
  for (int i = 0; i < kQ / 32; ++i) {
    before += i < w ? sums[i] : 0.0;
    all += sums[i];
  }
  x += before;
  const float hi = (float)x;
  float* out = logs + ((long long)bh * s.NC + c) * kLogs + t;
  out[0] = hi;
  out[kQ] = (float)(x - (double)hi);
  out[2 * kQ] = eta;
  out[3 * kQ] = exp2_rounded(x);
  out[4 * kQ] = exp2_rounded(all - x);
  out[5 * kQ] = exp2_rounded(before + sums[w] - x);
  if (t == 0) decay[(long long)c * s.B * s.H + bh] = exp2_rounded(all);
}

__device__ __forceinline__ void load_logs(const ChunkLogs& L, const float* logs, int bh, int NC, int c) {
  const float4* p = reinterpret_cast<const float4*>(logs + ((long long)bh * NC + c) * kLogs);
  if (threadIdx.x < kLogs / 4) reinterpret_cast<float4*>(L.hi)[threadIdx.x] = p[threadIdx.x];
}

// Set-up and tear-down that every kernel shares: an mbarrier and `COLS` columns
// of tensor memory.
template <int COLS>
__device__ __forceinline__ uint32_t block_begin(uint64_t* bar, uint32_t* slot) {
  if (threadIdx.x == 0) {
    tc::mbar_init(bar, 1);
    tc::fence_mbar_init();
  }
  if (threadIdx.x < 32) {
    tc::tmem_alloc(slot, COLS);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  return *slot;
}
template <int COLS>
__device__ __forceinline__ void block_end(uint32_t tmem) {
  cp_wait();  // (left over only where a wait gave up)
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (threadIdx.x < 32) tc::tmem_dealloc(tmem, COLS);
}
// Shared-memory writes of this thread become visible to the MMAs; then the block meets.
__device__ __forceinline__ void publish() {
  tc::fence_async_smem();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
}

// 16 columns of this thread's lane from each of N places.
template <int N>
__device__ __forceinline__ void tmem_ld16(const uint32_t (&at)[N], float (&x)[N][16]) {
  uint32_t r[N][16];
#pragma unroll
  for (int n = 0; n < N; ++n)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[n][0]), "=r"(r[n][1]), "=r"(r[n][2]), "=r"(r[n][3]), "=r"(r[n][4]), "=r"(r[n][5]),
          "=r"(r[n][6]), "=r"(r[n][7]), "=r"(r[n][8]), "=r"(r[n][9]), "=r"(r[n][10]), "=r"(r[n][11]),
          "=r"(r[n][12]), "=r"(r[n][13]), "=r"(r[n][14]), "=r"(r[n][15])
        : "r"(at[n])
        : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      asm volatile("" : "+r"(r[n][i]));  // no use of it moves before the wait
      x[n][i] = __uint_as_float(r[n][i]);
    }
}

// 16 columns of this thread's lane, to tensor memory (complete on return).
__device__ __forceinline__ void tmem_st16(uint32_t at, const float (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), "f"(x[8]),
      "f"(x[9]), "f"(x[10]), "f"(x[11]), "f"(x[12]), "f"(x[13]), "f"(x[14]), "f"(x[15])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint8_t* align1k(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// ------------------------------------------------------------------ two streams of heads
// The chunk-state and output kernels take one chunk of one group and a run of
// its items (a head, and a tile of 64 state rows where there are several). The
// tile that all heads share is loaded once; two groups of 256 threads then take
// the items in turn, each with its own buffers, accumulators and barriers, so
// that one group's MMAs and loads run under the other's arithmetic. A row (token)
// has two threads, one for each half of its columns.
constexpr int kHalf = kThreads / 2;

__device__ __forceinline__ void group_sync(int wg) { asm volatile("bar.sync %0, 256;" ::"r"(wg + 1) : "memory"); }
// Whether `ok` holds for all of the group's threads.
__device__ __forceinline__ bool group_and(int wg, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(wg + 1), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}
// Shared-memory writes of the group become visible to the MMAs; the group meets.
__device__ __forceinline__ void group_publish(int wg) {
  tc::fence_async_smem();
  tc::tc_fence_before();
  group_sync(wg);
  tc::tc_fence_after();
}
// Mmas::wait() for a group of 256 threads with an mbarrier of its own.
struct GroupMmas {
  uint64_t* bar;
  uint32_t phase;
  int* status;
  int wg;
  __device__ __forceinline__ bool wait(bool stall, bool so_far = true) {
    const bool ok = tc::mbar_wait(bar, phase) && so_far && !(stall && threadIdx.x == kHalf - 1);
    if (!ok) atomicExch(status, tc2::kErrMma);
    const bool all = group_and(wg, ok);
    if (!all) (void)tc::mbar_wait(bar, phase);
    phase ^= 1u;
    tc::tc_fence_after();
    return all;
  }
};

// Rows of one item by the threads of a group (cp.async where VEC).
template <int ROWS, int BLOCKS, bool VEC>
__device__ __forceinline__ void group_load_rows(uint8_t* tile, const bf16* src, long long ld, int n, int cols) {
  constexpr int kPer = BLOCKS * 8, kStep = kHalf / kPer;
  static_assert(kStep % 8 == 0 && ROWS % kStep == 0, "a thread's rows share their swizzle");
  const int tid = threadIdx.x % kHalf, j = tid % kPer, r0 = tid / kPer;
  const int left = j * 8 < cols ? n - r0 : 0;
  const bf16* p = src + r0 * ld + j * 8;
  uint8_t* dst = tile + piece<ROWS>(r0, j);
#pragma unroll
  for (int i = 0; i < ROWS / kStep; ++i) {
    const bool on = i * kStep < left;
    if constexpr (VEC)
      cp16(smem_u32(dst) + i * kStep * 128, on ? p : src, on);
    else
      *reinterpret_cast<uint4*>(dst + i * kStep * 128) =
          on ? load8(src + (long long)(r0 + i * kStep) * ld, j * 8, cols) : uint4{0, 0, 0, 0};
    p += kStep * ld;
  }
}

struct Items {
  int b, g, c, t0, n, i0, i1, HG, NPT;
  __device__ __forceinline__ int head(int it) const { return g * HG + (NPT == 1 ? it : it / NPT); }
  __device__ __forceinline__ int first_row(int it) const { return NPT == 1 ? 0 : it % NPT * kPT; }
};
__device__ __forceinline__ Items block_items(const SsmDims& s, const int* lengths, int per) {
  Items m;
  m.c = blockIdx.x;
  m.b = blockIdx.y / s.G;
  m.g = blockIdx.y - m.b * s.G;
  m.HG = s.H / s.G;
  m.NPT = s.NPT;
  m.t0 = m.c * kQ;
  m.n = min(max(ssm_row_length(lengths, m.b, s.T) - m.t0, 0), kQ);
  m.i0 = blockIdx.z * per;
  m.i1 = min(m.HG * s.NPT, m.i0 + per);
  return m;
}

// ------------------------------------------------------------------ chunk states
// states[c][bh][p][n] = sum_s w_s x_s[p] y_s[n]: with REV 0 x = v, y = k,
// w_s = e^{c_Q-c_s} eta_s; with REV 1 x = dy, y = q, w_t = e^{c_t}. D[n][p] on
// the tensor cores: y contracted over its rows (128 state columns as rows of the
// tile), against the three terms of w x side by side, so that y is read once for
// all three (N = 192: 80 cycles of shared-memory reads a step instead of 144).
// 33 us for 128 heads x 2048 tokens (64 x 128 states), where its bytes take 15: a
// chain of short steps in two streams. Results gathered in shared memory for one
// bulk copy took 41 us, three streams with one accumulator 35.
template <int REV, bool VEC>
__global__ void __launch_bounds__(kThreads, 1)
    state_kernel(SsmDims s, const bf16* __restrict__ x, const bf16* __restrict__ y,
                 const float* __restrict__ logs, const int* __restrict__ lengths,
                 float* __restrict__ states, int per, int* __restrict__ status, int stall) {
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bar, gbar[2];
  __shared__ uint32_t slot;
  uint8_t* ys = align1k(raw);  // [kQ][128]
  const int wg = threadIdx.x / kHalf, t = threadIdx.x % kQ, half = threadIdx.x / kQ & 1, quad = t >> 5;
  uint8_t* xs = ys + kQ * 256 + wg * 3 * kQ * 128;  // three of [kQ][64]
  if (threadIdx.x == 0)
    for (int i = 0; i < 2; ++i) tc::mbar_init(&gbar[i], 1);
  const uint32_t tmem = block_begin<512>(&bar, &slot) + wg * 192;
  griddep_wait();
  griddep_launch_dependents();
  const Items m = block_items(s, lengths, per);
  load_rows<kQ, 2, VEC>(ys, y + (((long long)m.b * s.G + m.g) * s.T + m.t0) * s.N, s.N, m.n, s.N);
  uint4 xv[4];
  float w = 0.f;
  // This thread's row of the item, and its token's weight.
  auto fetch = [&](int it) {
    const int h = m.head(it), p0 = m.first_row(it), bh = m.b * s.H + h;
    const int np = min(kPT, s.P - p0);
    const bf16* xr = x + ((long long)bh * s.T + m.t0 + t) * s.P + p0;
    const float* lg = logs + ((long long)bh * s.NC + m.c) * kLogs + t;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = half * 32 + j * 8;
      xv[j] = uint4{0, 0, 0, 0};
      if (t < m.n && col < np) xv[j] = VEC ? *reinterpret_cast<const uint4*>(xr + col) : load8(xr, col, np);
    }
    w = REV ? lg[3 * kQ] : lg[4 * kQ] * lg[2 * kQ];
  };
  int it = m.i0 + wg;
  if (it < m.i1) fetch(it);
  cp_wait();
  publish();
  GroupMmas done{&gbar[wg], 0u, status, wg};
#pragma unroll 1
  for (; it < m.i1; it += 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t* u = &xv[j].x;
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = w * lo_f(u[i]);
        f[2 * i + 1] = w * hi_f(u[i]);
      }
      uint4 term[3];
      split3(f, term);
#pragma unroll
      for (int i = 0; i < 3; ++i) *reinterpret_cast<uint4*>(xs + i * kQ * 128 + piece<kQ>(t, half * 4 + j)) = term[i];
    }
    group_publish(wg);
    if (threadIdx.x % kHalf == 0) {
      mma<kQ, true, kQ, true, 192>(tmem, ys, xs, kQ / 16, false);
      tc::mma_commit(&gbar[wg]);
    }
    if (it + 2 < m.i1) fetch(it + 2);
    if (!done.wait(stalled(stall, kStates))) break;
    const int h = m.head(it), p0 = m.first_row(it), bh = m.b * s.H + h;
    const int np = min(kPT, s.P - p0);
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    float* out = states + (((long long)m.c * s.B * s.H + bh) * s.P + p0 + half * 32) * s.N + t;
    if (quad * 32 < s.N) {
#pragma unroll
      for (int cb = half * 32; cb < half * 32 + 32; cb += 16) {
        float ld[3][16];
        tmem_ld16<3>({lanes + cb, lanes + 64 + cb, lanes + 128 + cb}, ld);
        const int left = t < s.N ? np - cb : 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (j < left) *out = ld[0][j] + (ld[1][j] + ld[2][j]);
          out += s.N;
        }
      }
    }
    tc::tc_fence_before();
    group_sync(wg);  // the accumulators are read before the next item's MMAs write them
    tc::tc_fence_after();
  }
  block_end<512>(tmem - wg * 192);
}

// ------------------------------------------------------------------ outputs
// The scores q k^T are the same for all heads of a group: they are made once and
// stay in tensor memory. An item turns them into its decayed scores W,
//   W_ts = e^{c_t-c_s} eta_s q_t.k_s, s <= t
// the decay taken exactly within the row's own block of 32 tokens, and as
// e^{c_t-c_r} e^{c_r-c_s} with r the last token of an earlier block (two factors
// that are both at most one for a decaying state), so that only a quarter of the
// decays takes an exponential each. A token's own term, W_tt v_t, joins D v_t in
// fp32 instead: where it is most of y_t, y_t then has no rounding but its last.
// 32 us for 128 heads x 2048 tokens (64 x 128 states; its bytes take 16); with a
// chunk's q k^T made again for every head and loads by all threads it was 72.
struct OutMaps {
  CUtensorMap v, y, S;  // [B*H][T][P] (boxes of 128 x 64), and [NC*B*H][P][N] (64 x 64)
};
template <int NB, bool VEC>
__global__ void __launch_bounds__(kThreads, 1)
    out_kernel(SsmDims s, const bf16* __restrict__ q, const bf16* __restrict__ k,
               const bf16* __restrict__ v, const float* __restrict__ logs,
               const float* __restrict__ D, const int* __restrict__ lengths,
               const bf16* __restrict__ states, bf16* __restrict__ y, int per,
               int* __restrict__ status, int stall, const __grid_constant__ OutMaps maps) {
  extern __shared__ uint8_t raw[];
  __shared__ __align__(16) float slog[2][kLogs], own[kQ];
  __shared__ uint64_t bar, gbar[2], sbar[2], full[2];
  __shared__ uint32_t slot;
  const int wg = threadIdx.x / kHalf, t = threadIdx.x % kQ, half = threadIdx.x / kQ & 1, quad = t >> 5;
  const bool leader = threadIdx.x % kHalf == 0;
  uint8_t* qs = align1k(raw);               // [kQ][NB * 64]
  uint8_t* ks = qs + NB * kQ * 128;         // [kQ][NB * 64], then group 0's scores
  uint8_t* Ws = ks + wg * kQ * 256;         // [kQ][kQ]
  uint8_t* Ss = ks + 2 * kQ * 256 + wg * NB * kPT * 128;                        // [64][NB * 64]
  uint8_t* vs = ks + 2 * kQ * 256 + 2 * NB * kPT * 128 + wg * 2 * kQ * 128;     // two of [kQ][64]
  if (threadIdx.x == 0)
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&gbar[i], 1);
      tc::mbar_init(&sbar[i], 1);
      tc::mbar_init(&full[i], 1);
    }
  const uint32_t tmem = block_begin<512>(&bar, &slot);
  griddep_wait();
  griddep_launch_dependents();
  const Items m = block_items(s, lengths, per);
  const long long qo = (((long long)m.b * s.G + m.g) * s.T + m.t0) * s.N;
  load_rows<kQ, NB, VEC>(qs, q + qo, s.N, m.n, s.N);
  load_rows<kQ, NB, VEC>(ks, k + qo, s.N, m.n, s.N);
  float hi = 0.f, lo = 0.f, eta = 0.f, start = 0.f, tail = 0.f;
  auto fetch_logs = [&](int it) {
    const float* lg = logs + ((long long)(m.b * s.H + m.head(it)) * s.NC + m.c) * kLogs + t;
    hi = lg[0];
    lo = lg[kQ];
    eta = lg[2 * kQ];
    start = lg[3 * kQ];
    tail = lg[5 * kQ];
  };
  // An item's state and rows: by TMA where a row of the tile is either a token that
  // exists or beyond T (which reads as zero), else by the group's threads.
  const bool tma = VEC && m.n == min(kQ, s.T - m.t0);
  auto fetch_state = [&](int it) {
    const int bh = m.b * s.H + m.head(it), p0 = m.first_row(it);
    if (tma) {
      if (leader)
        for (int i = 0; i < NB; ++i)
          tc::tma_load_3d(Ss + i * kPT * 128, &maps.S, &full[wg], i * 64, p0, m.c * s.B * s.H + bh);
    } else {
      group_load_rows<kPT, NB, VEC>(Ss, states + (((long long)m.c * s.B * s.H + bh) * s.P + p0) * s.N, s.N,
                                    min(kPT, s.P - p0), s.N);
    }
  };
  auto fetch_rows = [&](int it, int buf) {
    const int bh = m.b * s.H + m.head(it), p0 = m.first_row(it);
    if (tma) {
      if (leader) {
        tc::mbar_expect_tx(&full[wg], kQ * 128 + NB * kPT * 128);  // of the state too
        tc::tma_load_3d(vs + buf * kQ * 128, &maps.v, &full[wg], p0, m.t0, bh);
      }
    } else {
      group_load_rows<kQ, 1, VEC>(vs + buf * kQ * 128, v + ((long long)bh * s.T + m.t0) * s.P + p0, s.P, m.n,
                                  min(kPT, s.P - p0));
    }
  };
  int it = m.i0 + wg;
  if (it < m.i1) {
    fetch_logs(it);
    fetch_rows(it, 0);
    fetch_state(it);
  }
  cp_wait();
  publish();
  const int nsteps = (s.N + 15) / 16;
  Mmas first{&bar, 0u, status};
  if (threadIdx.x == 0) {
    mma<kQ, false, kQ, false, 128>(tmem, qs, ks, nsteps, false);
    tc::mma_commit(&bar);
  }
  const uint32_t kYi = 128 + wg * 128, kYd = kYi + 64;
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
  if (first.wait(stalled(stall, kScores) && threadIdx.x == kThreads - 1)) {
    // q_t.k_t; the scores above the diagonal blocks are zero for every item
    if (wg == 0 && half == 0) {
      float a[32], x = 0.f;
      tc::tmem_ld32(lanes + quad * 32, a);
#pragma unroll
      for (int i = 0; i < 32; ++i) x = t == quad * 32 + i ? a[i] : x;
      own[t] = x;
    }
    __syncthreads();
    for (int cb = half; cb < 4; cb += 2)
      if (cb > quad)
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(Ws + piece<kQ>(t, cb * 4 + i)) = uint4{0, 0, 0, 0};
    GroupMmas done{&gbar[wg], 0u, status, wg};
    const ChunkLogs L(slog[wg], kQ);  // tail here with eta
    int buf = 0;
    uint32_t phase = 0;  // of the loads and of the state's product
    bool lead_ok = true, gave_up = false;
#pragma unroll 1
    for (; it < m.i1; it += 2, buf ^= 1) {
      const int h = m.head(it), p0 = m.first_row(it), bh = m.b * s.H + h;
      const int np = min(kPT, s.P - p0);
      if (half == 0) {
        L.hi[t] = hi;
        L.lo[t] = lo;
        L.eta[t] = eta;
        L.tail[t] = tail * eta;
      }
      const float f = start, thi = hi, tlo = lo;
      cp_wait();
      group_publish(wg);  // the item's logs, and what the threads loaded, are there
      if (leader) {
        lead_ok = !tma || (tc::mbar_wait(&full[wg], phase) && !stalled(stall, kRows));
        mma<kQ, false, kPT, false, 64>(tmem + kYi, qs, Ss, nsteps, false);
        tc::mma_commit(&sbar[wg]);
      }
      const bool more = it + 2 < m.i1 && lead_ok;  // (on giving up no load is added to one that has not landed)
      if (more) {
        fetch_logs(it + 2);
        if (tma && leader) tc::bulk_wait_read<0>();  // that buffer's y is on its way
        fetch_rows(it + 2, buf ^ 1);
      }
#pragma unroll 1
      for (int cb = half; cb < quad; cb += 2) {
        float a[32];
        tc::tmem_ld32(lanes + cb * 32, a);
        const float row = ex2((thi - L.hi[cb * 32 + 31]) + (tlo - L.lo[cb * 32 + 31]));
        uint4 o[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 w = *reinterpret_cast<const float4*>(L.tail + cb * 32 + i * 4);
          uint32_t* ow = &o[i >> 1].x + (i & 1) * 2;
          ow[0] = pack2(a[i * 4] * (row * w.x), a[i * 4 + 1] * (row * w.y));
          ow[1] = pack2(a[i * 4 + 2] * (row * w.z), a[i * 4 + 3] * (row * w.w));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(Ws + piece<kQ>(t, cb * 4 + i)) = o[i];
      }
      if ((quad & 1) == half) {
        float a[32];
        tc::tmem_ld32(lanes + quad * 32, a);
        uint4 o[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int u = quad * 32 + i * 4, d = t - u;
          const float4 uh = *reinterpret_cast<const float4*>(L.hi + u);
          const float4 ul = *reinterpret_cast<const float4*>(L.lo + u);
          const float4 ue = *reinterpret_cast<const float4*>(L.eta + u);
          // (all lanes compute, then the later tokens' are dropped: no branches)
          const float w0 = a[i * 4] * (ex2((thi - uh.x) + (tlo - ul.x)) * ue.x);
          const float w1 = a[i * 4 + 1] * (ex2((thi - uh.y) + (tlo - ul.y)) * ue.y);
          const float w2 = a[i * 4 + 2] * (ex2((thi - uh.z) + (tlo - ul.z)) * ue.z);
          const float w3 = a[i * 4 + 3] * (ex2((thi - uh.w) + (tlo - ul.w)) * ue.w);
          uint32_t* ow = &o[i >> 1].x + (i & 1) * 2;
          ow[0] = pack2(d > 0 ? w0 : 0.f, d > 1 ? w1 : 0.f);
          ow[1] = pack2(d > 2 ? w2 : 0.f, d > 3 ? w3 : 0.f);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(Ws + piece<kQ>(t, quad * 4 + i)) = o[i];
      }
      group_publish(wg);
      uint8_t* vb = vs + buf * kQ * 128;
      if (leader) {
        mma<kQ, false, kQ, true, 64>(tmem + kYd, Ws, vb, kQ / 16, false);
        tc::mma_commit(&gbar[wg]);
      }
      if (!tma || leader) lead_ok = tc::mbar_wait(&sbar[wg], phase) && lead_ok;  // the state's tile is free
      if (more) fetch_state(it + 2);
      if (!done.wait(stalled(stall, kOutputs), lead_ok)) {
        gave_up = true;
        break;
      }
      // (v has landed: the leader saw it before the group last met)
      phase ^= 1u;
      const float Dh = fmaf(own[t], L.eta[t], D ? D[h] : 0.f);
      {
        float yi[32], yd[32];
        tc::tmem_ld32(lanes + kYi + half * 32, yi);
        tc::tmem_ld32(lanes + kYd + half * 32, yd);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4* at = reinterpret_cast<uint4*>(vb + piece<kQ>(t, half * 4 + i));
          const uint4 xv = *at;
          const uint32_t* xu = &xv.x;
          uint4 o;
          uint32_t* ou = &o.x;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int a = i * 8 + e * 2;
            const float y0 = fmaf(f, yi[a], yd[a]) + Dh * lo_f(xu[e]);
            const float y1 = fmaf(f, yi[a + 1], yd[a + 1]) + Dh * hi_f(xu[e]);
            const uint32_t p = pack2(y0, y1);
            ou[e] = t < m.n ? p : 0u;
          }
          *at = o;  // y takes the place of v
        }
      }
      if constexpr (VEC) {
        group_publish(wg);
        if (leader) {  // rows beyond T and columns beyond P are not written
          tc::tma_store_3d(&maps.y, vb, p0, m.t0, bh);
          tc::bulk_commit();
          if (!tma) tc::bulk_wait_read<0>();
        }
        if (!tma) group_sync(wg);
      } else {
        tc::tc_fence_before();
        group_sync(wg);
        tc::tc_fence_after();
        // whole rows to memory: eight threads a row
        const int j = t & 7, r0 = threadIdx.x % kHalf >> 3;
        bf16* out = y + ((long long)bh * s.T + m.t0 + r0) * s.P + p0 + j * 8;
        for (int i = 0; i < 4; ++i)
          if (m.t0 + r0 + i * 32 < s.T)
            store8<VEC>(out + i * 32 * (long long)s.P,
                        *reinterpret_cast<const uint4*>(vb + piece<kQ>(r0, j) + i * 32 * 128), np - j * 8);
      }
    }
    if (leader) {
      tc::bulk_wait_all();
      if (tma && gave_up)  // no load of ours may outlive the block
        for (uint32_t i = 0; i < 2; ++i) (void)tc::mbar_wait(&full[wg], phase ^ i);
    }
  } else if (tma && leader && it < m.i1) {
    (void)tc::mbar_wait(&full[wg], 0u);
  }
  block_end<512>(tmem);
}

// ------------------------------------------------------------------ gradients
// 16 columns of one value per (row = lane, column): the sum over the warp's
// lanes of column `lane & 15`, to that lane.
__device__ __forceinline__ float column_sums(float (&v)[16], int lane) {
#pragma unroll
  for (int o = 8; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float send = up ? v[i] : v[i + o];
      const float keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(~0u, send, o);
    }
  return v[0] + __shfl_xor_sync(~0u, v[0], 16);
}
struct GradOut {
  float *dq, *dk;    // [B*G][parts][T][N]: sums over a part's heads, fp32
  bf16 *dq16, *dk16; // the results themselves, where there is one part
  bf16* dv;
  float* ddt;
  double *dA, *dD;
};

// All gradients of one chunk for a run of heads of one group (and their tiles of
// 64 state rows: `items`). dq and dk add up over the items in tensor memory: the
// products with the decayed scores by the MMAs, the states' parts, whose rows are
// scaled item by item, by loads and stores between them. (In registers they
// would not fit beside the rest: with most of the SM's L1 taken as shared memory,
// spilled registers go to L2.)
//   tensor memory: [0, 256) scratch (S^T dy | X^T v; then q k^T | dy v^T; then the
//   two parts of dv), [256, 384) dq, [384, 512) dk
//   shared memory: q, k; v of the item, dy of this and of the next; S and X in
//   three terms, later overwritten by the two score matrices (X's first term stays)
// What the next item reads comes in under this one: its S and X to registers once
// the last products are issued, its v and dy once the scores are made.
// 214 us for 128 heads x 2048 tokens (64 x 128 states), some 20000 cycles an item, of
// which the MMAs are 4100: one chain of steps, since a second stream's tiles do not
// fit. v, dy and dv by TMA took 218 us (more registers spilled), 256 threads with dq
// and dk in registers 268.
template <int NB, bool VEC>
__global__ void __launch_bounds__(kThreads, 1)
    grad_kernel(SsmDims s, const bf16* __restrict__ q, const bf16* __restrict__ k,
                const bf16* __restrict__ v, const bf16* __restrict__ dy,
                const float* __restrict__ logs, const float* __restrict__ A,
                const float* __restrict__ D, const int* __restrict__ lengths,
                const float* __restrict__ states, const float* __restrict__ ends, GradOut o,
                int per, int* __restrict__ status, int stall) {
  constexpr int kTerm = NB * kPT * 128;  // bytes of one term of a state
  extern __shared__ uint8_t raw[];
  __shared__ __align__(16) float slog[kLogs];
  __shared__ float rows[4][kQ], cols[4][kQ], rdr[4][kQ], src[4][kQ], diag[2][kQ], owned[kQ],
      warp_ip[kThreads / 32];
  __shared__ int lost;  // the wait that the test hook makes this block lose
  __shared__ double warp_d[kThreads / 32];
  __shared__ uint64_t bar;
  __shared__ uint32_t slot;
  uint8_t* qs = align1k(raw);
  uint8_t* ks = qs + NB * kQ * 128;
  uint8_t* vs = ks + NB * kQ * 128;
  uint8_t* gb = vs + kQ * 128;       // two of [kQ][64]: dy, by turns
  uint8_t* W1 = gb + 2 * kQ * 128;   // e^{c_t-c_s} q_t.k_s, [t][s]
  uint8_t* W2 = W1 + kQ * 256;       // e^{c_t-c_s} eta_s dy_t.v_s
  uint8_t* Xs = W2 + kQ * 256;       // X, first term
  uint8_t* St = W1;                  // S, three terms, and X's second and third, under W1 and W2
  const int c = blockIdx.x, bg = blockIdx.y, b = bg / s.G, g = bg - b * s.G, split = blockIdx.z;
  const int HG = s.H / s.G, items = HG * s.NPT, BH = s.B * s.H, t0 = c * kQ;
  const ChunkLogs L(slog, kQ);
  if (threadIdx.x == 0) lost = stalled(stall, stall) ? stall : kNone;
  const uint32_t tmem = block_begin<512>(&bar, &slot);
  griddep_wait();
  griddep_launch_dependents();
  const int n = min(max(ssm_row_length(lengths, b, s.T) - t0, 0), kQ);
  const long long qo = ((long long)bg * s.T + t0) * s.N;
  load_rows<kQ, NB, VEC>(qs, q + qo, s.N, n, s.N);
  load_rows<kQ, NB, VEC>(ks, k + qo, s.N, n, s.N);
  // A row (token) has four threads, one for each quarter of its columns.
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3, part = warp >> 2;
  const int t = quad * 32 + lane;
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
  constexpr uint32_t kDq = 256, kDk = 384;
  constexpr int HC = NB * 16;  // a thread's columns of dq and dk: [part * HC, part * HC + HC)
  const int nsteps = (s.N + 15) / 16;
  Mmas done{&bar, 0u, status};
  bool ok = true;
  if (part == quad) owned[t] = 0.f;  // sum over the items of eta_t dy_t.v_t, by the row's diagonal block's thread

  const int i0 = split * per, i1 = min(items, i0 + per);
  auto head = [&](int it) { return g * HG + (s.NPT == 1 ? it : it / s.NPT); };
  auto tile = [&](int it) { return s.NPT == 1 ? 0 : it % s.NPT; };
  auto fetch_rows = [&](int it, int buf) {
    const int p0 = tile(it) * kPT, np = min(kPT, s.P - p0);
    const long long vo = ((long long)(b * s.H + head(it)) * s.T + t0) * s.P + p0;
    load_rows<kQ, 1, VEC>(vs, v + vo, s.P, n, np);
    load_rows<kQ, 1, VEC>(gb + buf * kQ * 128, dy + vo, s.P, n, np);
  };
  constexpr int kPer = NB * 8, kStep = kThreads / kPer, kIt = kPT / kStep;
  float Sf[kIt][8], Xf[kIt][8];
  auto fetch_states = [&](int it) {
    const int p0 = tile(it) * kPT, np = min(kPT, s.P - p0), j = threadIdx.x % kPer, r0 = threadIdx.x / kPer;
    const long long so = (((long long)c * BH + b * s.H + head(it)) * s.P + p0 + r0) * s.N + j * 8;
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const int left = r0 + i * kStep < np ? s.N - j * 8 : 0;
      load8f<VEC>(Sf[i], states + so + (long long)i * kStep * s.N, left);
      load8f<VEC>(Xf[i], ends + so + (long long)i * kStep * s.N, left);
    }
  };
  fetch_rows(i0, 0);
  fetch_states(i0);
#pragma unroll 1
  for (int it = i0; it < i1 && ok; ++it) {
    const int h = head(it), pt = tile(it), bh = b * s.H + h;
    const int p0 = pt * kPT, np = min(kPT, s.P - p0);
    const long long vo = ((long long)bh * s.T + t0) * s.P + p0;
    uint8_t* gs = gb + ((it - i0) & 1) * kQ * 128;
    load_logs(L, logs, bh, s.NC, c);
    // S and X, as three terms each, and <S, X>
    {
      const int j = threadIdx.x % kPer, r0 = threadIdx.x / kPer;
      float ip = 0.f;
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) ip = fmaf(Sf[i][e], Xf[i][e], ip);
        const uint32_t at = piece<kPT>(r0 + i * kStep, j);
        uint4 term[3];
        split3(Sf[i], term);
#pragma unroll
        for (int m = 0; m < 3; ++m) *reinterpret_cast<uint4*>(St + m * kTerm + at) = term[m];
        split3<true>(Xf[i], term);  // dv takes the first one alone
        *reinterpret_cast<uint4*>(Xs + at) = term[0];
        *reinterpret_cast<uint4*>(St + 3 * kTerm + at) = term[1];
        *reinterpret_cast<uint4*>((NB == 1 ? St + 4 * kTerm : Xs + kTerm) + at) = term[2];
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) ip += __shfl_xor_sync(~0u, ip, d);
      if (lane == 0) warp_ip[warp] = ip;
    }
    cp_wait();
    publish();
    if (threadIdx.x == 0) {
      const uint8_t* x2 = NB == 1 ? St + 4 * kTerm : Xs + kTerm;
      // the small terms first: the accumulator's cut-off bits then are the first term's alone
      for (int m = 2; m >= 0; --m) mma<kQ, false, kPT, true, NB * 64>(tmem, gs, St + m * kTerm, kPT / 16, m < 2);
      mma<kQ, false, kPT, true, NB * 64>(tmem + 128, vs, x2, kPT / 16, false);
      mma<kQ, false, kPT, true, NB * 64>(tmem + 128, vs, St + 3 * kTerm, kPT / 16, true);
      mma<kQ, false, kPT, true, NB * 64>(tmem + 128, vs, Xs, kPT / 16, true);
      tc::mma_commit(&bar);
    }
    {
      // dD = sum dy v: products of bf16 are exact in fp32; over a row the sum may
      // cancel to almost nothing, so beyond a thread's 16 it is in fp64
      float x = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t at = piece<kQ>(t, part * 2 + j);
        const uint4 rv = *reinterpret_cast<const uint4*>(vs + at), rg = *reinterpret_cast<const uint4*>(gs + at);
        const uint32_t *uv = &rv.x, *ug = &rg.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x = fmaf(lo_f(uv[i]), lo_f(ug[i]), fmaf(hi_f(uv[i]), hi_f(ug[i]), x));
      }
      double sum = x;
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
      if (lane == 0) warp_d[warp] = sum;
    }
    if (!(ok = done.wait(lost == kDots))) break;
    // the states' parts of dq and dk, and their dots with q and k
    {
      const float f = L.start[t], e = L.end[t], ee = e * L.eta[t];
      const bool add = it > i0;
      float rd = 0.f, sd = 0.f;
#pragma unroll
      for (int cb = 0; cb < NB; ++cb) {
        const uint32_t col = lanes + part * HC + cb * 16;
        float ld[4][16];
        tmem_ld16<4>({col, col + 128, col + kDq, col + kDk}, ld);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t at = piece<kQ>(t, (part * HC + cb * 16) / 8 + j);
          const uint4 rq = *reinterpret_cast<const uint4*>(qs + at), rk = *reinterpret_cast<const uint4*>(ks + at);
          const uint32_t *uq = &rq.x, *uk = &rk.x;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c0 = j * 8 + i * 2;
            rd = fmaf(ld[0][c0], lo_f(uq[i]), rd);
            sd = fmaf(ld[1][c0], lo_f(uk[i]), sd);
            rd = fmaf(ld[0][c0 + 1], hi_f(uq[i]), rd);
            sd = fmaf(ld[1][c0 + 1], hi_f(uk[i]), sd);
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          ld[2][i] = fmaf(ld[0][i], f, add ? ld[2][i] : 0.f);
          ld[3][i] = fmaf(ld[1][i], ee, add ? ld[3][i] : 0.f);
        }
        tmem_st16(col + kDq, ld[2]);
        tmem_st16(col + kDk, ld[3]);
      }
      rdr[part][t] = rd * f;
      src[part][t] = sd * e;
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (threadIdx.x == 0) {
      mma<kQ, false, kQ, false, 128>(tmem, qs, ks, nsteps, false);
      mma<kQ, false, kQ, false, 128>(tmem + 128, gs, vs, kPT / 16, false);
      tc::mma_commit(&bar);
    }
    if (!(ok = done.wait(lost == kPairs))) break;
    if (it + 1 < i1) fetch_rows(it + 1, (it - i0 + 1) & 1);  // v has done its part
    // the decayed scores, and the row and column sums of Z off its diagonal
    float zrow = 0.f, dr = 0.f, dd = 0.f, dm = 0.f;
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const int u0 = part * 32 + sub * 16;
      uint4 o1[2] = {}, o2[2] = {};
      if (part <= quad) {
        float ld[2][16], off[16];
        tmem_ld16<2>({lanes + u0, lanes + 128 + u0}, ld);
        float(&m)[16] = ld[0], (&kk)[16] = ld[1];
        float e[16], h[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v4 = *reinterpret_cast<const float4*>(L.eta + u0 + i * 4);
          h[i * 4] = v4.x, h[i * 4 + 1] = v4.y, h[i * 4 + 2] = v4.z, h[i * 4 + 3] = v4.w;
        }
        if (part < quad) {
          const float row = L.decay(t, part * 32 + 31);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 v4 = *reinterpret_cast<const float4*>(L.tail + u0 + i * 4);
            e[i * 4] = row * v4.x, e[i * 4 + 1] = row * v4.y, e[i * 4 + 2] = row * v4.z, e[i * 4 + 3] = row * v4.w;
          }
        } else {
          const float thi = L.hi[t], tlo = L.lo[t];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 a4 = *reinterpret_cast<const float4*>(L.hi + u0 + i * 4);
            const float4 b4 = *reinterpret_cast<const float4*>(L.lo + u0 + i * 4);
            e[i * 4] = ex2((thi - a4.x) + (tlo - b4.x));
            e[i * 4 + 1] = ex2((thi - a4.y) + (tlo - b4.y));
            e[i * 4 + 2] = ex2((thi - a4.z) + (tlo - b4.z));
            e[i * 4 + 3] = ex2((thi - a4.w) + (tlo - b4.w));
          }
          // the later tokens' are dropped (all lanes compute: no branches)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int u = u0 + i;
            e[i] = u <= t ? e[i] : 0.f;
            m[i] = u <= t ? m[i] : 0.f;
            kk[i] = u <= t ? kk[i] : 0.f;
          }
        }
        // q_t.k_t, the same for every item (before the decay, whose NaN would be one head's)
        if (part == quad && it == i0)
#pragma unroll
          for (int i = 0; i < 16; ++i) dm = u0 + i == t ? m[i] : dm;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          m[i] *= e[i];
          off[i] = m[i] * kk[i];
        }
        if (part == quad)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const bool on = u0 + i == t;
            dr = on ? off[i] : dr;
            dd = on ? kk[i] : dd;
            kk[i] = on ? 0.f : kk[i];  // joins dq and dk in fp32, at the end
            m[i] = on ? 0.f : m[i];  // joins D in fp32
            off[i] = on ? 0.f : off[i];
          }
#pragma unroll
        for (int i = 0; i < 16; ++i) kk[i] *= e[i] * h[i];
#pragma unroll
        for (int i = 0; i < 16; ++i) zrow = fmaf(off[i], h[i], zrow);
        uint32_t *w1 = &o1[0].x, *w2 = &o2[0].x;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w1[i] = pack2(m[2 * i], m[2 * i + 1]);
          w2[i] = pack2(kk[2 * i], kk[2 * i + 1]);
        }
        const float sum = column_sums(off, lane);
        if (lane < 16) cols[quad][u0 + lane] = sum;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<uint4*>(W1 + piece<kQ>(t, u0 / 8 + i)) = o1[i];
        *reinterpret_cast<uint4*>(W2 + piece<kQ>(t, u0 / 8 + i)) = o2[i];
      }
    }
    rows[part][t] = zrow;
    if (part == quad) {  // the quarter that holds this row's diagonal block
      diag[0][t] = dr;
      owned[t] = fmaf(dd, L.eta[t], owned[t]);
      if (it == i0) diag[1][t] = dm;
    }
    publish();
    if (threadIdx.x == 0) {
      mma<kQ, true, kQ, true, 64>(tmem, W1, gs, kQ / 16, false);
      mma<kQ, false, kPT, false, 64>(tmem + 64, ks, Xs, nsteps, false);
      mma<kQ, false, kQ, true, NB * 64>(tmem + kDq, W2, ks, kQ / 16, true);
      mma<kQ, true, kQ, true, NB * 64>(tmem + kDk, W2, qs, kQ / 16, true);
      tc::mma_commit(&bar);
    }
    if (it + 1 < i1) fetch_states(it + 1);
    if (warp >= kThreads / 32 - 2) {
      // Two warps make ddt, and dA and dD, while the MMAs run: lane l has the tokens
      // 4 l .. 4 l + 3.
      const bool for_dt = warp == kThreads / 32 - 1;
      float ip = lane < kThreads / 32 ? warp_ip[lane] : 0.f;
#pragma unroll
      for (int d = kThreads / 64; d; d >>= 1) ip += __shfl_xor_sync(~0u, ip, d);
      ip = __shfl_sync(~0u, ip, 0);
      float in4[4], src4[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = lane * 4 + i;
        in4[i] = (rdr[0][r] + rdr[1][r]) + (rdr[2][r] + rdr[3][r]);
        src4[i] = (src[0][r] + src[1][r]) + (src[2][r] + src[3][r]);
      }
      if (for_dt) {
        float a4[4], b4[4], off4[4], as = 0.f, bs = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = lane * 4 + i;
          float off = 0.f;
#pragma unroll
          for (int qd = 0; qd < 4; ++qd) off += qd >= r >> 5 ? cols[qd][r] : 0.f;
          off4[i] = off;
          a4[i] = ((rows[0][r] + rows[1][r]) + (rows[2][r] + rows[3][r]) - L.eta[r] * off) + in4[i];
          b4[i] = L.eta[r] * src4[i];
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
        const float through = L.start[kQ - 1] * ip, Ah = A[h];
        float dl[4];
#pragma unroll
        for (int i = 3; i >= 0; --i) dl[i] = after += a4[i];
        float* out = o.ddt + ((long long)pt * BH + bh) * s.T + t0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = lane * 4 + i;
          dl[i] += before + through;
          before += b4[i];
          const float x = fmaf(Ah, dl[i], off4[i] + diag[0][r] + src4[i]);
          if (t0 + r < s.T) out[r] = r < n ? x : 0.f;
        }
      } else {
        double in[4], out[4], dsum = lane < kThreads / 32 ? warp_d[lane] : 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = lane * 4 + i;
          in[i] = in4[i];
          out[i] = (double)L.eta[r] * src4[i];
        }
        const double dA = decay_gradient<4>([&](int cb, int i) { return rows[cb][lane * 4 + i]; },
                                            [&](int qd, int i) { return cols[qd][lane * 4 + i]; }, in, out,
                                            L.eta + lane * 4, (double)L.start[kQ - 1] * ip, lane);
#pragma unroll
        for (int d = 16; d; d >>= 1) dsum += __shfl_xor_sync(~0u, dsum, d);
        if (lane == 0) {
          const long long at = ((long long)c * s.NPT + pt) * BH + bh;
          o.dA[at] = dA;
          o.dD[at] = dsum;
        }
      }
      __syncwarp();
    }
    if (!(ok = done.wait(lost == kResults))) break;
    {
      float ld[2][16];
      tmem_ld16<2>({lanes + part * 16, lanes + 64 + part * 16}, ld);
      float(&a1)[16] = ld[0], (&a2)[16] = ld[1];
      const float e = L.end[t], eta = L.eta[t], Dh = fmaf(eta, diag[1][t], D ? D[h] : 0.f);
      bf16* out = o.dv + vo + (long long)t * s.P + part * 16;
      if (t0 + t < s.T)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 r = *reinterpret_cast<const uint4*>(gs + piece<kQ>(t, part * 2 + i));
          const uint32_t* u = &r.x;
          uint4 w;
          uint32_t* wu = &w.x;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int x = i * 8 + j * 2;
            const float d0 = fmaf(eta, fmaf(e, a2[x], a1[x]), Dh * lo_f(u[j]));
            const float d1 = fmaf(eta, fmaf(e, a2[x + 1], a1[x + 1]), Dh * hi_f(u[j]));
            const uint32_t p = pack2(d0, d1);
            wu[j] = t < n ? p : 0u;
          }
          store8<VEC>(out + i * 8, w, np - (part * 16 + i * 8));
        }
    }
    tc::tc_fence_before();
    __syncthreads();  // the item's tiles, logs and sums are free for the next one
    tc::tc_fence_after();
  }
  // A token's own terms, eta_t (dy_t.v_t) k_t and q_t, are added in fp32.
  __syncthreads();
  if (ok) {
    const int parts = gridDim.z;
    const float own = owned[t];
    const bool there = t0 + t < s.T;
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
      for (int cb = 0; cb < NB; ++cb) {
        float ld[1][16];
        tmem_ld16<1>({lanes + (which ? kDk : kDq) + part * HC + cb * 16}, ld);
        float(&a)[16] = ld[0];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 r = *reinterpret_cast<const uint4*>((which ? qs : ks) +
                                                          piece<kQ>(t, (part * HC + cb * 16) / 8 + j));
          const uint32_t* u = &r.x;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int x = j * 8 + i * 2;
            const float x0 = fmaf(own, lo_f(u[i]), a[x]), x1 = fmaf(own, hi_f(u[i]), a[x + 1]);
            a[x] = t < n ? x0 : 0.f;
            a[x + 1] = t < n ? x1 : 0.f;
          }
        }
        const int col = part * HC + cb * 16;
        if (!there) continue;
        if (parts == 1) {
          bf16* out = (which ? o.dk16 : o.dq16) + qo + (long long)t * s.N + col;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            store8<VEC>(out + i * 8,
                        uint4{pack2(a[i * 8], a[i * 8 + 1]), pack2(a[i * 8 + 2], a[i * 8 + 3]),
                              pack2(a[i * 8 + 4], a[i * 8 + 5]), pack2(a[i * 8 + 6], a[i * 8 + 7])},
                        s.N - col - i * 8);
        } else {
          float* out = (which ? o.dk : o.dq) + (((long long)bg * parts + split) * s.T + t0 + t) * s.N + col;
          if (s.N % 4 == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (col + i * 4 < s.N)
                *reinterpret_cast<float4*>(out + i * 4) = float4{a[i * 4], a[i * 4 + 1], a[i * 4 + 2], a[i * 4 + 3]};
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (col + i < s.N) out[i] = a[i];
          }
        }
      }
  }
  block_end<512>(tmem);
}

size_t state_smem() { return 1024 + kQ * 256 + 2 * 3 * kQ * 128; }
template <int NB>
size_t out_smem() {
  return 1024 + NB * kQ * 128 + 2 * kQ * 256 + 2 * NB * kPT * 128 + 4 * kQ * 128;
}

template <int NB>
size_t grad_smem() {
  return 1024 + 2 * NB * kQ * 128 + 3 * kQ * 128 + 2 * kQ * 256 + (NB == 1 ? 1 : 2) * NB * kPT * 128;
}

// How many blocks share the items of a group's chunk: of all ways, the one whose
// waves of blocks, each of `fixed` + its longest stream of items, end first. `part`
// is what one block more adds in memory traffic. All in units of an item's time.
int item_parts(const SsmDims& s, int streams, double fixed, double part) {
  const long long items = (long long)s.H / s.G * s.NPT, base = (long long)s.B * s.G * s.NC;
  int best = 1;
  double cost = 1e300;
  for (long long ns = 1; ns <= items; ++ns) {
    const long long per = (items + ns - 1) / ns;
    if ((items + per - 1) / per != ns) continue;
    const double c = (double)((base * ns + kPlannedSms - 1) / kPlannedSms) * ((per + streams - 1) / streams + fixed) +
                     part * ns * base / kPlannedSms;
    if (c < cost) cost = c, best = (int)ns;
  }
  return best;
}
// The gradients: q, k and the results weigh about a third of an item; every part
// more is one more fp32 copy of dq and dk to write and add up. Against every other split
// of eight shapes (8 to 64 heads in 1 to 8 groups, 300 to 16384 tokens) the forward's is
// within 1 % of the best one, the gradients' within 9 % (13 parts where 10 were best for
// 2 x 64 heads x 2048 tokens, 277 us against 254, and 8 where 1 was for 32 x 16384).
int grad_parts(const SsmDims& s) { return item_parts(s, 1, 0.35, 0.04); }

dim3 item_grid(const SsmDims& s, int parts, int* per) {
  const long long items = (long long)s.H / s.G * s.NPT;
  *per = (int)((items + parts - 1) / parts);
  return dim3(s.NC, s.B * s.G, parts);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiledFn>(ptr);
  }();
  return fn;
}
// Matrices [count][rows][cols] of bf16 in boxes of box_rows x 64, 128-byte swizzle;
// what lies outside a matrix reads as zero and is not written.
bool tile_map(CUtensorMap* m, const void* base, uint64_t count, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cols, rows, count}, strides[2] = {cols * 2, rows * cols * 2};
  const cuuint32_t box[3] = {64, box_rows, 1}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class F>
cudaError_t allow_smem(F* f, size_t bytes) {
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// The wait that the test hook has armed, for a launch that has waits first .. last.
std::atomic<int> g_stall{kNone};
int take_stall(int first, int last) {
  int armed = g_stall.load(std::memory_order_relaxed);
  return armed >= first && armed <= last && g_stall.compare_exchange_strong(armed, kNone) ? armed : kNone;
}

bool vectors(const SsmDims& s, std::initializer_list<const void*> ps) {
  if (s.N % 8 || s.P % 8) return false;
  for (const void* p : ps)
    if ((uintptr_t)p & 15) return false;
  return true;
}

}  // namespace

void arm_scan_stall(int wait) { g_stall.store(wait >= kStates && wait <= kResults ? wait : kNone); }

size_t ssm_tc_logs_bytes(const SsmDims& s) {
  return (size_t)s.B * s.H * s.NC * kLogs * sizeof(float);
}

int ssm_tc_grad_parts(const SsmDims& s) { return grad_parts(s); }

cudaError_t ssm_tc_bwd(const SsmBwdArgs& a, const SsmBwdScratch& w) {
  const SsmDims& s = a.s;
  const int BH = s.B * s.H, parts = grad_parts(s);
  int per = 0;
  const bool vec = vectors(s, {a.q, a.k, a.v, a.dy, a.dq, a.dk, a.dv, a.states});
  cudaError_t e;
  {
    E2TTT_TRACE("ssm_logs", a.st);
    e = launch_pdl(logs_kernel, dim3(s.NC, BH), dim3(kQ), 0, a.st, s, a.dt, a.A, a.lengths, w.logs,
                   w.decay, w.status);
    if (e != cudaSuccess) return e;
  }
  {
    E2TTT_TRACE("ssm_chunk_dstate", a.st);
    auto kern = vec ? state_kernel<1, true> : state_kernel<1, false>;
    if ((e = allow_smem(kern, state_smem())) != cudaSuccess) return e;
    const dim3 grid = item_grid(s, item_parts(s, 2, 1.5, 0), &per);
    e = launch_pdl(kern, grid, dim3(kThreads), state_smem(), a.st, s, (const bf16*)a.dy, (const bf16*)a.q,
                   (const float*)w.logs, a.lengths, w.ends, per, w.status, take_stall(kStates, kStates));
    if (e != cudaSuccess) return e;
  }
  if ((e = ssm_carry(s, true, a.dS_end, w.decay, w.ends, a.dS0, nullptr, true, a.st)) != cudaSuccess) return e;
  {
    E2TTT_TRACE("ssm_chunk_grad", a.st);
    auto kern = s.N <= 64 ? (vec ? grad_kernel<1, true> : grad_kernel<1, false>)
                          : (vec ? grad_kernel<2, true> : grad_kernel<2, false>);
    const size_t smem = s.N <= 64 ? grad_smem<1>() : grad_smem<2>();
    if ((e = allow_smem(kern, smem)) != cudaSuccess) return e;
    const GradOut o{w.dq, w.dk, (bf16*)a.dq, (bf16*)a.dk, (bf16*)a.dv, w.ddt, w.dA, w.dD};
    const dim3 grid = item_grid(s, parts, &per);
    e = launch_pdl(kern, grid, dim3(kThreads), smem, a.st, s, (const bf16*)a.q,
                   (const bf16*)a.k, (const bf16*)a.v, (const bf16*)a.dy, (const float*)w.logs, a.A, a.D, a.lengths,
                   a.states, (const float*)w.ends, o, per, w.status, take_stall(kDots, kResults));
    if (e != cudaSuccess) return e;
  }
  return ssm_grad_sums(a, w, parts);
}

cudaError_t ssm_tc_fwd(const SsmFwdArgs& a) {
  const SsmDims& s = a.s;
  const int BH = s.B * s.H;
  int per = 0;
  const bool vec = vectors(s, {a.q, a.k, a.v, a.y});
  cudaError_t e;
  {
    E2TTT_TRACE("ssm_logs", a.st);
    e = launch_pdl(logs_kernel, dim3(s.NC, BH), dim3(kQ), 0, a.st, s, a.dt, a.A, a.lengths, a.logs,
                   a.decay, a.status);
    if (e != cudaSuccess) return e;
  }
  {
    E2TTT_TRACE("ssm_chunk_state", a.st);
    auto kern = vec ? state_kernel<0, true> : state_kernel<0, false>;
    if ((e = allow_smem(kern, state_smem())) != cudaSuccess) return e;
    const dim3 grid = item_grid(s, item_parts(s, 2, 1.5, 0), &per);
    e = launch_pdl(kern, grid, dim3(kThreads), state_smem(), a.st, s, (const bf16*)a.v, (const bf16*)a.k,
                   (const float*)a.logs, a.lengths, a.states, per, a.status, take_stall(kStates, kStates));
    if (e != cudaSuccess) return e;
  }
  if ((e = ssm_carry(s, false, a.S0, a.decay, a.states, a.S_end, a.starts, a.keep, a.st)) != cudaSuccess) return e;
  E2TTT_TRACE("ssm_chunk_out", a.st);
  auto kern = s.N <= 64 ? (vec ? out_kernel<1, true> : out_kernel<1, false>)
                        : (vec ? out_kernel<2, true> : out_kernel<2, false>);
  const size_t smem = s.N <= 64 ? out_smem<1>() : out_smem<2>();
  if ((e = allow_smem(kern, smem)) != cudaSuccess) return e;
  const dim3 grid = item_grid(s, item_parts(s, 2, 1.5, 0), &per);
  OutMaps maps = {};
  if (vec && !(tile_map(&maps.v, a.v, BH, s.T, s.P, kQ) && tile_map(&maps.y, a.y, BH, s.T, s.P, kQ) &&
               tile_map(&maps.S, a.starts, (uint64_t)s.NC * BH, s.P, s.N, kPT)))
    return cudaErrorNotSupported;
  return launch_pdl(kern, grid, dim3(kThreads), smem, a.st, s, (const bf16*)a.q, (const bf16*)a.k,
                    (const bf16*)a.v, (const float*)a.logs, a.D, a.lengths, (const bf16*)a.starts,
                    (bf16*)a.y, per, a.status, take_stall(kScores, kOutputs), maps);
}

}  // namespace e2ttt
