// Global 2-norm of many gradient tensors and their clipping by it:
//   norm = sqrt(sum over tensors and elements of g^2),
//   out  = g min(1, max_norm / (norm + 1e-6)).
//
// Bound by HBM: the norm reads every gradient once; the clip reads them again
// and writes them, and reads nothing where the norm is within max_norm and the
// clip is in place. The tensors are cut into pieces of kPieceBytes; block i
// takes an equal range of the pieces of the whole list, so one launch serves
// many small tensors as well as a few large ones (the list travels as a kernel
// parameter, kMany tensors to a launch). Squares are summed in fp32 over one
// 16-byte vector, then in fp64, to one partial per block; the clip's blocks each
// add up all partials themselves, in the same order, so no block waits for
// another and results repeat bit for bit. A block of either pass has the same
// range of pieces and the clip walks it backwards, so that what the norm read
// last is still in L2. 63M values of both types in 97 us: two reads and a write of
// 188 MB at 5.85 TB/s. Asking L2 to hold 32 to 96 MB between the passes gained nothing.
#include "seq_ops.h"
#include "trace.h"

namespace e2ttt {
namespace {

constexpr int kThreads = 256;
// Pieces of equal bytes, so that the blocks' shares are alike whatever the types.
constexpr int kPieceBytes = 32768;
template <typename T> constexpr int kPiece = kPieceBytes / sizeof(T);
constexpr int kFew = 32, kMany = 480;

struct Item {
  const void* g;
  void* out;
  unsigned long long n;
  unsigned first;  // its first piece in the launch's list
  unsigned act;    // 1: bf16
};
template <int MAX>
struct List {
  Item t[MAX];
  int count;
  unsigned pieces;
};

// The tensor that piece `p` belongs to (first <= p, the last such one).
template <int MAX>
__device__ __forceinline__ int find(const List<MAX>& l, unsigned p) {
  int lo = 0, hi = l.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.t[mid].first <= p) lo = mid; else hi = mid;
  }
  return lo;
}

// First piece of block b's range.
__device__ __forceinline__ unsigned range_start(unsigned pieces, unsigned b) {
  return (unsigned)((unsigned long long)pieces * b / gridDim.x);
}

template <typename T> struct Wide { static constexpr int N = 16 / sizeof(T); };

// Sum of squares of one vector in fp32, and whether that neither overflowed nor
// lost small values; where it did, the squares are taken again in fp64.
template <typename T>
__device__ __forceinline__ float squares(const uint4& raw) {
  const T* p = reinterpret_cast<const T*>(&raw);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < Wide<T>::N; ++i) s = fmaf(to_f<T>(p[i]), to_f<T>(p[i]), s);
  return s;
}
__device__ __forceinline__ bool fits(float s) { return s > 1e-24f && s < 1e37f; }
// Zeros of either sign throughout, whose sum is exact: whole rows of a gradient are zero
// where a token or an expert was not used.
template <typename T>
__device__ __forceinline__ bool zeros(const uint4& raw) {
  return ((raw.x | raw.y | raw.z | raw.w) & (sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu)) == 0;
}
template <typename T>
__device__ __forceinline__ double square1(T v) {
  const double x = to_f<T>(v);
  return x * x;
}

template <typename T>
__device__ double piece_squares(const Item& it, unsigned piece) {
  constexpr int N = Wide<T>::N;
  const unsigned long long beg = (unsigned long long)piece * kPiece<T>;
  const int n = (int)(it.n - beg < kPiece<T> ? it.n - beg : kPiece<T>);
  const T* g = (const T*)it.g + beg;
  double a = 0.0;
  // elements before the first 16-byte boundary, whole vectors, the rest
  const int head = min(n, (int)(((16 - ((uintptr_t)g & 15)) & 15) / sizeof(T)));
  const int nv = (n - head) / N;
  const uint4* v = reinterpret_cast<const uint4*>(g + head);
  if ((int)threadIdx.x < head) a += square1<T>(g[threadIdx.x]);
  constexpr int U = 8;
  for (int i = threadIdx.x; i < nv; i += kThreads * U) {
    uint4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = i + u * kThreads < nv ? v[i + u * kThreads] : uint4{0, 0, 0, 0};
    float q[U];
    bool all = true;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      q[u] = squares<T>(r[u]);
      all = all && (fits(q[u]) || zeros<T>(r[u]));  // (those past the end are zeros)
    }
    if (all) {
#pragma unroll
      for (int u = 0; u < U; ++u) a += q[u];
    } else {
      for (int u = 0; u < U && i + u * kThreads < nv; ++u)
        for (int e = 0; e < N; ++e) a += square1<T>(g[head + (long long)(i + u * kThreads) * N + e]);
    }
  }
  for (int i = head + nv * N + threadIdx.x; i < n; i += kThreads) a += square1<T>(g[i]);
  return a;
}

// Sum over the block, to every thread, in a fixed order.
__device__ __forceinline__ double block_sum(double a) {
  __shared__ double s[kThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(~0u, a, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = a;
  __syncthreads();
  a = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) a += s[i];
  return a;
}

__device__ __forceinline__ double partials_sum(const double* part, int n) {
  double a = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) a += part[i];
  return block_sum(a);
}

template <int MAX>
__global__ void __launch_bounds__(kThreads, 4)
    grad_squares_kernel(const __grid_constant__ List<MAX> l, double* __restrict__ part) {
  double a = 0.0;
  const unsigned p0 = range_start(l.pieces, blockIdx.x), p1 = range_start(l.pieces, blockIdx.x + 1);
  int i = p0 < p1 ? find(l, p0) : 0;
  for (unsigned p = p0; p < p1; ++p) {
    while (i + 1 < l.count && l.t[i + 1].first <= p) ++i;
    const Item& it = l.t[i];
    a += it.act ? piece_squares<bf16>(it, p - it.first) : piece_squares<float>(it, p - it.first);
  }
  a = block_sum(a);
  if (threadIdx.x == 0) part[blockIdx.x] = a;
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const double* __restrict__ part, int n,
                                                             float* __restrict__ norm, int* __restrict__ status) {
  const double s = partials_sum(part, n);
  if (threadIdx.x == 0) *norm = (float)sqrt(s), *status = 0;
}

template <typename T>
__device__ void piece_scale(const Item& it, unsigned piece, float scale) {
  constexpr int N = Wide<T>::N;
  const unsigned long long beg = (unsigned long long)piece * kPiece<T>;
  const int n = (int)(it.n - beg < kPiece<T> ? it.n - beg : kPiece<T>);
  const T* g = (const T*)it.g + beg;
  T* o = (T*)it.out + beg;
  const bool same = (((uintptr_t)g ^ (uintptr_t)o) & 15) == 0;
  const int head = same ? min(n, (int)(((16 - ((uintptr_t)g & 15)) & 15) / sizeof(T))) : n;
  const int nv = (n - head) / N;
  for (int i = threadIdx.x; i < head; i += kThreads) o[i] = from_f<T>(to_f<T>(g[i]) * scale);
  const uint4* v = reinterpret_cast<const uint4*>(g + head);
  uint4* w = reinterpret_cast<uint4*>(o + head);
  constexpr int U = 4;
  for (int i = threadIdx.x; i < nv; i += kThreads * U) {
    uint4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * kThreads < nv) r[u] = __ldcs(v + i + u * kThreads);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      T* p = reinterpret_cast<T*>(&r[u]);
#pragma unroll
      for (int e = 0; e < N; ++e) p[e] = from_f<T>(to_f<T>(p[e]) * scale);
      if (i + u * kThreads < nv) __stcs(w + i + u * kThreads, r[u]);
    }
  }
  for (int i = head + nv * N + threadIdx.x; i < n; i += kThreads)
    o[i] = from_f<T>(to_f<T>(g[i]) * scale);
}

template <int MAX>
__global__ void __launch_bounds__(kThreads, 4)
    grad_clip_kernel(const __grid_constant__ List<MAX> l, const double* __restrict__ part, int n,
                     float max_norm, float* __restrict__ norm, int* __restrict__ status) {
  const float total = (float)sqrt(partials_sum(part, n));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = total, *status = 0;
  const float c = max_norm / (total + 1e-6f);
  const float scale = c > 1.f ? 1.f : c;  // a NaN norm scales by NaN
  const unsigned p0 = range_start(l.pieces, blockIdx.x), p1 = range_start(l.pieces, blockIdx.x + 1);
  int i = p0 < p1 ? find(l, p1 - 1) : 0;
  for (unsigned p = p1; p-- > p0;) {
    while (l.t[i].first > p) --i;
    const Item& it = l.t[i];
    if (scale == 1.f && it.g == it.out) continue;
    if (it.act)
      piece_scale<bf16>(it, p - it.first, scale);
    else
      piece_scale<float>(it, p - it.first, scale);
  }
}

// Fills `l` with up to MAX non-empty tensors from index `at` on; returns the
// index after the last one taken.
template <int MAX>
int take(const GradList& g, int at, List<MAX>* l) {
  l->count = 0;
  l->pieces = 0;
  for (; at < g.count && l->count < MAX; ++at) {
    if (!g.n[at]) continue;
    const int each = g.act[at] == 1 ? kPiece<bf16> : kPiece<float>;
    const unsigned long long pieces = (g.n[at] + each - 1) / each;
    if (l->count && pieces + l->pieces > 0x7fffffffull) break;
    l->t[l->count++] = Item{g.g[at], g.out && g.out[at] ? g.out[at] : const_cast<void*>(g.g[at]),
                            (unsigned long long)g.n[at], l->pieces, (unsigned)(g.act[at] == 1)};
    l->pieces += (unsigned)pieces;
  }
  return at;
}

template <int MAX>
cudaError_t squares_t(const GradList& g, double* part, int* parts, cudaStream_t st) {
  List<MAX> l;
  *parts = 0;
  for (int at = 0; at < g.count;) {
    at = take(g, at, &l);
    if (!l.count) break;
    int blocks = sm_count() * 4;
    if (blocks > kGradBlocksMax) blocks = kGradBlocksMax;
    if ((unsigned)blocks > l.pieces) blocks = (int)l.pieces;
    E2TTT_TRACE("grad_squares", st);
    grad_squares_kernel<MAX><<<blocks, kThreads, 0, st>>>(l, part + *parts);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    *parts += blocks;
  }
  return cudaSuccess;
}

template <int MAX>
cudaError_t clip_t(const GradList& g, const double* part, int parts, float max_norm, float* norm,
                   int* status, cudaStream_t st) {
  List<MAX> l;
  for (int at = 0; at < g.count;) {
    at = take(g, at, &l);
    if (!l.count) break;
    int blocks = sm_count() * 4;
    if ((unsigned)blocks > l.pieces) blocks = (int)l.pieces;
    E2TTT_TRACE("grad_clip", st);
    grad_clip_kernel<MAX><<<blocks, kThreads, 0, st>>>(l, part, parts, max_norm, norm, status);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    norm = nullptr;  // the first launch writes it
  }
  return cudaSuccess;
}

double* partials(void* ws) { return (double*)((char*)ws + kStatusBytes); }

cudaError_t squares_of(const GradList& g, double* part, int* parts, cudaStream_t st) {
  return g.count <= kFew ? squares_t<kFew>(g, part, parts, st) : squares_t<kMany>(g, part, parts, st);
}

}  // namespace

size_t grad_workspace_bytes(int count) {
  return kStatusBytes + (size_t)((count + kMany - 1) / kMany + 1) * kGradBlocksMax * sizeof(double);
}

cudaError_t grad_norm(const GradList& g, float* norm, void* ws, cudaStream_t st) {
  int parts = 0;
  const cudaError_t e = squares_of(g, partials(ws), &parts, st);
  if (e != cudaSuccess) return e;
  E2TTT_TRACE("grad_norm", st);
  grad_norm_kernel<<<1, kThreads, 0, st>>>(partials(ws), parts, norm, (int*)ws);
  return cudaGetLastError();
}

cudaError_t grad_clip(const GradList& g, float max_norm, float* norm, void* ws, cudaStream_t st) {
  int parts = 0;
  bool any = false;
  for (int i = 0; i < g.count; ++i) any = any || g.n[i];
  if (!any) return grad_norm(g, norm, ws, st);
  const cudaError_t e = squares_of(g, partials(ws), &parts, st);
  if (e != cudaSuccess) return e;
  return g.count <= kFew ? clip_t<kFew>(g, partials(ws), parts, max_norm, norm, (int*)ws, st)
                         : clip_t<kMany>(g, partials(ws), parts, max_norm, norm, (int*)ws, st);
}

}  // namespace e2ttt
