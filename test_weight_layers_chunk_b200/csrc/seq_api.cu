// C entry points of the short convolution, the state-space scan and the gradient
// norm: argument checks and workspace layout. See include/e2ttt.h.
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "checks.h"
#include "seq_ops.h"

namespace e2ttt {

int sm_count() {
  thread_local int dev = -1, sms = 0;
  int now = -1;
  if (cudaGetDevice(&now) != cudaSuccess) return 148;
  if (now != dev) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, now) != cudaSuccess) return 148;
    dev = now;
  }
  return sms;
}

namespace {

#define TRY(call)                              \
  do {                                         \
    const e2ttt_status st_ = (call);           \
    if (st_ != E2TTT_OK) return st_;           \
  } while (0)

e2ttt_status check_ws(const char* who, const void* ws, size_t have, size_t need) {
  if (!ws) return failf(E2TTT_ERR_INVALID_ARG, "%s: workspace is NULL (needs %zu bytes)", who, need);
  if (have < need)
    return failf(E2TTT_ERR_INVALID_ARG, "%s: workspace too small: %zu < %zu bytes", who, have, need);
  if ((uintptr_t)ws & 255)
    return failf(E2TTT_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  return E2TTT_OK;
}

e2ttt_status check_run(cudaError_t e, const char* who) {
  return e == cudaSuccess ? E2TTT_OK : fail_cuda(e, who);
}

// ------------------------------------------------------------------ convolution
e2ttt_status conv_dims(const char* who, const e2ttt_conv_shape* s, ConvDims* d) {
  if (!s) return failf(E2TTT_ERR_INVALID_ARG, "%s: shape is NULL", who);
  if (s->B < 1 || s->H < 1 || s->T < 1 || s->d < 1 || s->W < 1)
    return failf(E2TTT_ERR_INVALID_ARG, "%s: sizes must be >= 1 (B=%d H=%d T=%d d=%d W=%d)", who, s->B,
                 s->H, s->T, s->d, s->W);
  if (s->W > 8) return failf(E2TTT_ERR_INVALID_ARG, "%s: W must be <= 8", who);
  if (s->act != E2TTT_F32 && s->act != E2TTT_BF16)
    return failf(E2TTT_ERR_INVALID_ARG, "%s: unknown activation dtype", who);
  if (s->silu != 0 && s->silu != 1) return failf(E2TTT_ERR_INVALID_ARG, "%s: silu must be 0 or 1", who);
  if ((long long)s->B * s->H > 65535)
    return failf(E2TTT_ERR_INVALID_ARG, "%s: B*H must be <= 65535", who);
  if (s->T > (1 << 24)) return failf(E2TTT_ERR_INVALID_ARG, "%s: T must be <= 2^24", who);
  if (s->d > (1 << 20) || (long long)s->H * s->d * s->W >= (1LL << 31))
    return failf(E2TTT_ERR_INVALID_ARG, "%s: d must be <= 2^20 and H*d*W < 2^31", who);
  *d = ConvDims{s->B, s->H, s->T, s->d, s->W, s->act == E2TTT_BF16, s->silu == 1};
  return E2TTT_OK;
}

struct ConvBytes {
  size_t es, x, w, b, st, len;
};
ConvBytes conv_bytes(const ConvDims& d) {
  const size_t es = d.bf16_act ? 2 : 4, rows = (size_t)d.B * d.H, hd = (size_t)d.H * d.d;
  return ConvBytes{es, rows * d.T * d.d * es, hd * d.W * 4, hd * 4, rows * (d.W - 1) * d.d * es,
                   (size_t)d.B * 4};
}

// Whether four channels at a time can be read and written as one vector.
bool conv_vectors(const ConvDims& d, std::initializer_list<const void*> ps) {
  return d.d % 4 == 0 && all_aligned(d.bf16_act ? 8 : 16, ps);
}

// ------------------------------------------------------------------ scan
e2ttt_status ssm_dims(const char* who, const e2ttt_ssm_shape* s, SsmDims* d) {
  if (!s) return failf(E2TTT_ERR_INVALID_ARG, "%s: shape is NULL", who);
  if (s->B < 1 || s->H < 1 || s->G < 1 || s->T < 1 || s->d_k < 1 || s->d_v < 1)
    return failf(E2TTT_ERR_INVALID_ARG, "%s: sizes must be >= 1 (B=%d H=%d G=%d T=%d d_k=%d d_v=%d)",
                 who, s->B, s->H, s->G, s->T, s->d_k, s->d_v);
  if (s->H % s->G) return failf(E2TTT_ERR_INVALID_ARG, "%s: H=%d is not a multiple of G=%d", who, s->H, s->G);
  if (s->act != E2TTT_F32 && s->act != E2TTT_BF16)
    return failf(E2TTT_ERR_INVALID_ARG, "%s: unknown activation dtype", who);
  if (s->d_k > 256 || s->d_v > 1024)
    return failf(E2TTT_ERR_INVALID_ARG, "%s: d_k must be <= 256 and d_v <= 1024", who);
  if ((long long)s->B * s->H > 65535)
    return failf(E2TTT_ERR_INVALID_ARG, "%s: B*H must be <= 65535", who);
  if (s->T > (1 << 24)) return failf(E2TTT_ERR_INVALID_ARG, "%s: T must be <= 2^24", who);
  d->B = s->B;
  d->H = s->H;
  d->G = s->G;
  d->T = s->T;
  d->N = s->d_k;
  d->P = s->d_v;
  d->bf16_act = s->act == E2TTT_BF16;
  d->tc = d->bf16_act && s->d_k <= 128;
  // mma.sync (ssm.cu): 64 tokens to a chunk; with more than 128 state columns the
  // backward's tiles of 64 tokens would not fit an SM's shared memory.
  d->Q = d->tc ? kSsmTcChunk : s->d_k <= 128 ? 64 : 32;
  d->NC = (s->T + d->Q - 1) / d->Q;
  d->NPT = (s->d_v + kSsmPT - 1) / kSsmPT;
  if ((long long)d->NC * s->B * s->H * d->NPT >= (1LL << 31))
    return failf(E2TTT_ERR_INVALID_ARG, "%s: too many chunks: ceil(T/%d)*B*H*ceil(d_v/64) must be < 2^31", who, d->Q);
  return E2TTT_OK;
}

struct SsmBytes {
  size_t es, qk, v, dt, head, S, len, saved;
};
SsmBytes ssm_bytes(const SsmDims& d) {
  const size_t es = d.bf16_act ? 2 : 4, bh = (size_t)d.B * d.H;
  const size_t S = bh * d.P * d.N * 4;
  return SsmBytes{es, (size_t)d.B * d.G * d.T * d.N * es, bh * d.T * d.P * es, bh * d.T * 4,
                  (size_t)d.H * 4, S, (size_t)d.B * 4, S * d.NC};
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Forward scratch: status word, the chunks' decays, their logarithms (tensor
// cores), their start states in bf16 (tensor cores) and their states (in
// saved_states where given).
struct SsmFwdWs {
  size_t decay, logs, starts, states, total;
};
SsmFwdWs ssm_fwd_layout(const SsmDims& d) {
  SsmFwdWs L{};
  L.decay = 256;
  L.logs = L.decay + up256((size_t)d.NC * d.B * d.H * 4);
  L.starts = L.logs + (d.tc ? up256(ssm_tc_logs_bytes(d)) : 0);
  L.states = L.starts + (d.tc ? up256(ssm_bytes(d).saved / 2) : 0);
  L.total = L.states + up256(ssm_bytes(d).saved);
  return L;
}

// ------------------------------------------------------------------ gradients
// No output may meet another output or a gradient other than its own in place.
e2ttt_status check_grads(const char* who, const void* const* g, void* const* out, const size_t* n,
                         const int* act, int count, const void* norm, const void* ws, size_t wsn) {
  if (count < 0 || (count && (!g || !n || !act)))
    return failf(E2TTT_ERR_INVALID_ARG, "%s: count is negative or a list is NULL", who);
  struct End {
    uintptr_t beg, end;
    int written;
  };
  std::vector<End> all;
  all.reserve((size_t)count * 2 + 2);
  for (int i = 0; i < count; ++i) {
    if (act[i] != E2TTT_F32 && act[i] != E2TTT_BF16)
      return failf(E2TTT_ERR_INVALID_ARG, "%s: tensor %d: unknown dtype", who, i);
    if (!n[i]) continue;
    const size_t es = act[i] == E2TTT_BF16 ? 2 : 4;
    if (!g[i]) return failf(E2TTT_ERR_INVALID_ARG, "%s: gradient %d is NULL", who, i);
    if (n[i] > (size_t(1) << 40))
      return failf(E2TTT_ERR_INVALID_ARG, "%s: gradient %d has more than 2^40 elements", who, i);
    void* o = out ? out[i] : nullptr;
    if (((uintptr_t)g[i] | (uintptr_t)o) & (es - 1))
      return failf(E2TTT_ERR_INVALID_ARG, "%s: tensor %d must be aligned to its elements", who, i);
    const bool in_place = !o || o == g[i];
    all.push_back(End{(uintptr_t)g[i], (uintptr_t)g[i] + n[i] * es, out && in_place});
    if (!in_place) all.push_back(End{(uintptr_t)o, (uintptr_t)o + n[i] * es, 1});
  }
  all.push_back(End{(uintptr_t)norm, (uintptr_t)norm + 4, 1});
  all.push_back(End{(uintptr_t)ws, (uintptr_t)ws + wsn, 1});
  // sorted by start, a range that meets an earlier one meets the furthest end so
  // far, or the furthest end of a written one
  std::sort(all.begin(), all.end(), [](const End& a, const End& b) { return a.beg < b.beg; });
  uintptr_t any = 0, written = 0;
  for (const End& e : all) {
    if ((e.written && e.beg < any) || e.beg < written)
      return failf(E2TTT_ERR_INVALID_ARG, "%s: an output overlaps another tensor of the call", who);
    any = std::max(any, e.end);
    if (e.written) written = std::max(written, e.end);
  }
  return E2TTT_OK;
}

}  // namespace
}  // namespace e2ttt

using namespace e2ttt;

// Every entry point: no exception leaves it.
#define GUARD(who, ...)                                                     \
  try {                                                                      \
    set_last_error("");                                                      \
    __VA_ARGS__                                                                     \
  } catch (...) {                                                            \
    return failf(E2TTT_ERR_CUDA, "%s: out of host memory", who);             \
  }

extern "C" {

size_t e2ttt_short_conv_workspace_bytes(const e2ttt_conv_shape* s) {
  ConvDims d;
  if (conv_dims("e2ttt_short_conv_workspace_bytes", s, &d) != E2TTT_OK) return 0;
  return conv_bwd_workspace_bytes(d);
}

e2ttt_status e2ttt_short_conv_fwd(const e2ttt_conv_shape* s, const void* x, const float* w,
                                  const float* bias, const void* state, const int* lengths,
                                  void* y, void* state_end, void* stream) {
  static const char* who = "e2ttt_short_conv_fwd";
  GUARD(who, {
    ConvDims d;
    TRY(conv_dims(who, s, &d));
    if (!x || !w || !y)
      return failf(E2TTT_ERR_INVALID_ARG, "%s: x, w and y must not be NULL", who);
    const ConvBytes n = conv_bytes(d);
    TRY(check_aligned(who, n.es, {{x, 0, "x"}, {state, 0, "state"}, {y, 0, "y"}, {state_end, 0, "state_end"}}));
    TRY(check_aligned(who, 4, {{w, 0, "w"}, {bias, 0, "bias"}, {lengths, 0, "lengths"}}));
    TRY(check_spans(who, {{x, n.x, "x"}, {w, n.w, "w"}, {bias, n.b, "bias"}, {state, n.st, "state"},
                          {lengths, n.len, "lengths"}},
                    {{y, n.x, "y"}, {state_end, n.st, "state_end"}}));
    const bool vec = conv_vectors(d, {x, state, y, state_end});
    ConvArgs a{d, x, w, bias, state, lengths, vec, (cudaStream_t)stream};
    return check_run(conv_fwd(a, y, d.W > 1 ? state_end : nullptr), who);
  })
}

e2ttt_status e2ttt_short_conv_bwd(const e2ttt_conv_shape* s, const void* x, const float* w,
                                  const float* bias, const void* state, const int* lengths,
                                  const void* dy, const void* dstate_end, void* dx, float* dw,
                                  float* dbias, void* dstate, void* ws, size_t ws_bytes,
                                  void* stream) {
  static const char* who = "e2ttt_short_conv_bwd";
  GUARD(who, {
    ConvDims d;
    TRY(conv_dims(who, s, &d));
    if (!x || !w || !dy || !dx || !dw)
      return failf(E2TTT_ERR_INVALID_ARG, "%s: x, w, dy, dx and dw must not be NULL", who);
    const ConvBytes n = conv_bytes(d);
    const size_t need = conv_bwd_workspace_bytes(d);
    TRY(check_ws(who, ws, ws_bytes, need));
    TRY(check_aligned(who, n.es, {{x, 0, "x"}, {state, 0, "state"}, {dy, 0, "dy"},
                                  {dstate_end, 0, "dstate_end"}, {dx, 0, "dx"}, {dstate, 0, "dstate"}}));
    TRY(check_aligned(who, 4, {{w, 0, "w"}, {bias, 0, "bias"}, {lengths, 0, "lengths"}, {dw, 0, "dw"},
                               {dbias, 0, "dbias"}}));
    TRY(check_spans(who, {{x, n.x, "x"}, {w, n.w, "w"}, {bias, n.b, "bias"}, {state, n.st, "state"},
                          {lengths, n.len, "lengths"}, {dy, n.x, "dy"}, {dstate_end, n.st, "dstate_end"}},
                    {{dx, n.x, "dx"}, {dw, n.w, "dw"}, {dbias, n.b, "dbias"}, {dstate, n.st, "dstate"},
                     {ws, need, "workspace"}}));
    const bool vec = conv_vectors(d, {x, state, dy, dstate_end, dx, dstate});
    ConvArgs a{d, x, w, bias, state, lengths, vec, (cudaStream_t)stream};
    return check_run(conv_bwd(a, dy, d.W > 1 ? dstate_end : nullptr, dx, dw, dbias,
                              d.W > 1 ? dstate : nullptr, ws), who);
  })
}

e2ttt_status e2ttt_short_conv_step(const e2ttt_conv_shape* s, const void* x, const float* w,
                                   const float* bias, void* state, void* y, void* stream) {
  static const char* who = "e2ttt_short_conv_step";
  GUARD(who, {
    ConvDims d;
    TRY(conv_dims(who, s, &d));
    if (d.T != 1) return failf(E2TTT_ERR_INVALID_ARG, "%s: T must be 1", who);
    if (!x || !w || !y || (!state && d.W > 1))
      return failf(E2TTT_ERR_INVALID_ARG, "%s: x, w, state and y must not be NULL", who);
    const ConvBytes n = conv_bytes(d);
    TRY(check_aligned(who, n.es, {{x, 0, "x"}, {state, 0, "state"}, {y, 0, "y"}}));
    TRY(check_aligned(who, 4, {{w, 0, "w"}, {bias, 0, "bias"}}));
    TRY(check_spans(who, {{x, n.x, "x"}, {w, n.w, "w"}, {bias, n.b, "bias"}},
                    {{state, n.st, "state"}, {y, n.x, "y"}}));
    const bool vec = conv_vectors(d, {x, state, y});
    ConvArgs a{d, x, w, bias, nullptr, nullptr, vec, (cudaStream_t)stream};
    return check_run(conv_step(a, state, y), who);
  })
}

size_t e2ttt_ssm_workspace_bytes(const e2ttt_ssm_shape* s, int for_bwd) {
  SsmDims d;
  if (ssm_dims("e2ttt_ssm_workspace_bytes", s, &d) != E2TTT_OK) return 0;
  return for_bwd ? ssm_bwd_workspace_bytes(d) : ssm_fwd_layout(d).total;
}

size_t e2ttt_ssm_saved_bytes(const e2ttt_ssm_shape* s) {
  SsmDims d;
  if (ssm_dims("e2ttt_ssm_saved_bytes", s, &d) != E2TTT_OK) return 0;
  return ssm_bytes(d).saved;
}

e2ttt_status e2ttt_ssm_scan_fwd(const e2ttt_ssm_shape* s, const void* q, const void* k,
                                const void* v, const float* dt, const float* A, const float* D,
                                const float* S0, const int* lengths, void* y, float* S_end,
                                float* saved, void* ws, size_t ws_bytes, void* stream) {
  static const char* who = "e2ttt_ssm_scan_fwd";
  GUARD(who, {
    SsmDims d;
    TRY(ssm_dims(who, s, &d));
    if (!q || !k || !v || !dt || !A || !y || !S_end)
      return failf(E2TTT_ERR_INVALID_ARG, "%s: q, k, v, dt, A, y and S_end must not be NULL", who);
    const SsmBytes n = ssm_bytes(d);
    const SsmFwdWs lay = ssm_fwd_layout(d);
    const size_t need = lay.total;
    TRY(check_ws(who, ws, ws_bytes, need));
    TRY(check_aligned(who, n.es, {{q, 0, "q"}, {k, 0, "k"}, {v, 0, "v"}, {y, 0, "y"}}));
    TRY(check_aligned(who, 4, {{dt, 0, "dt"}, {A, 0, "A"}, {D, 0, "D"}, {S0, 0, "S0"},
                               {lengths, 0, "lengths"}, {S_end, 0, "S_end"}, {saved, 0, "saved_states"}}));
    TRY(check_spans(who, {{q, n.qk, "q"}, {k, n.qk, "k"}, {v, n.v, "v"}, {dt, n.dt, "dt"}, {A, n.head, "A"},
                          {D, n.head, "D"}, {S0, n.S, "S0"}, {lengths, n.len, "lengths"}},
                    {{y, n.v, "y"}, {S_end, n.S, "S_end"}, {saved, n.saved, "saved_states"},
                     {ws, need, "workspace"}}));
    char* w = (char*)ws;
    SsmFwdArgs a{d, q, k, v, dt, A, D, S0, lengths, y, S_end, saved ? saved : (float*)(w + lay.states),
                 (float*)(w + lay.decay), (float*)(w + lay.logs), w + lay.starts, saved != nullptr, (int*)w,
                 (cudaStream_t)stream};
    return check_run(d.tc ? ssm_tc_fwd(a) : ssm_fwd(a), who);
  })
}

e2ttt_status e2ttt_ssm_scan_bwd(const e2ttt_ssm_shape* s, const void* q, const void* k,
                                const void* v, const float* dt, const float* A, const float* D,
                                const int* lengths, const float* saved, const void* dy,
                                const float* dS_end, void* dq, void* dk, void* dv, float* ddt,
                                float* dA, float* dD, float* dS0, void* ws, size_t ws_bytes,
                                void* stream) {
  static const char* who = "e2ttt_ssm_scan_bwd";
  GUARD(who, {
    SsmDims d;
    TRY(ssm_dims(who, s, &d));
    if (!q || !k || !v || !dt || !A || !saved || !dy || !dq || !dk || !dv || !ddt || !dA)
      return failf(E2TTT_ERR_INVALID_ARG,
                   "%s: only D, lengths, dS_end, dD and dS0 may be NULL", who);
    if ((D == nullptr) != (dD == nullptr))
      return failf(E2TTT_ERR_INVALID_ARG, "%s: dD must be NULL exactly where D is", who);
    const SsmBytes n = ssm_bytes(d);
    const size_t need = ssm_bwd_workspace_bytes(d);
    TRY(check_ws(who, ws, ws_bytes, need));
    TRY(check_aligned(who, n.es, {{q, 0, "q"}, {k, 0, "k"}, {v, 0, "v"}, {dy, 0, "dy"}, {dq, 0, "dq"},
                                  {dk, 0, "dk"}, {dv, 0, "dv"}}));
    TRY(check_aligned(who, 4, {{dt, 0, "dt"}, {A, 0, "A"}, {D, 0, "D"}, {lengths, 0, "lengths"},
                               {saved, 0, "saved_states"}, {dS_end, 0, "dS_end"}, {ddt, 0, "ddt"},
                               {dA, 0, "dA"}, {dD, 0, "dD"}, {dS0, 0, "dS0"}}));
    TRY(check_spans(who, {{q, n.qk, "q"}, {k, n.qk, "k"}, {v, n.v, "v"}, {dt, n.dt, "dt"}, {A, n.head, "A"},
                          {D, n.head, "D"}, {lengths, n.len, "lengths"}, {saved, n.saved, "saved_states"},
                          {dy, n.v, "dy"}, {dS_end, n.S, "dS_end"}},
                    {{dq, n.qk, "dq"}, {dk, n.qk, "dk"}, {dv, n.v, "dv"}, {ddt, n.dt, "ddt"},
                     {dA, n.head, "dA"}, {dD, n.head, "dD"}, {dS0, n.S, "dS0"}, {ws, need, "workspace"}}));
    SsmBwdArgs a{d, q, k, v, dt, A, D, lengths, saved, dy, dS_end, dq, dk, dv, ddt, dA, dD, dS0, ws,
                 (cudaStream_t)stream};
    return check_run(ssm_bwd(a), who);
  })
}

e2ttt_status e2ttt_ssm_step(const e2ttt_ssm_shape* s, const void* q, const void* k, const void* v,
                            const float* dt, const float* A, const float* D, float* S, void* y,
                            void* stream) {
  static const char* who = "e2ttt_ssm_step";
  GUARD(who, {
    SsmDims d;
    TRY(ssm_dims(who, s, &d));
    if (d.T != 1) return failf(E2TTT_ERR_INVALID_ARG, "%s: T must be 1", who);
    if (!q || !k || !v || !dt || !A || !S || !y)
      return failf(E2TTT_ERR_INVALID_ARG, "%s: only D may be NULL", who);
    const SsmBytes n = ssm_bytes(d);
    TRY(check_aligned(who, n.es, {{q, 0, "q"}, {k, 0, "k"}, {v, 0, "v"}, {y, 0, "y"}}));
    TRY(check_aligned(who, 4, {{dt, 0, "dt"}, {A, 0, "A"}, {D, 0, "D"}, {S, 0, "S"}}));
    TRY(check_spans(who, {{q, n.qk, "q"}, {k, n.qk, "k"}, {v, n.v, "v"}, {dt, n.dt, "dt"}, {A, n.head, "A"},
                          {D, n.head, "D"}},
                    {{S, n.S, "S"}, {y, n.v, "y"}}));
    SsmStepArgs a{d, q, k, v, dt, A, D, S, y, (cudaStream_t)stream};
    return check_run(ssm_step(a), who);
  })
}

void e2ttt_test_stall_next_scan(int wait) { arm_scan_stall(wait); }

size_t e2ttt_grad_workspace_bytes(int count) { return count < 0 ? 0 : grad_workspace_bytes(count); }

e2ttt_status e2ttt_grad_norm(const void* const* g, const size_t* n, const int* act, int count,
                             float* norm, void* ws, size_t ws_bytes, void* stream) {
  static const char* who = "e2ttt_grad_norm";
  GUARD(who, {
    if (!norm || ((uintptr_t)norm & 3))
      return failf(E2TTT_ERR_INVALID_ARG, "%s: norm is NULL or unaligned", who);
    const size_t need = e2ttt_grad_workspace_bytes(count);
    TRY(check_ws(who, ws, ws_bytes, need));
    TRY(check_grads(who, g, nullptr, n, act, count, norm, ws, need));
    return check_run(grad_norm(GradList{g, nullptr, n, act, count}, norm, ws, (cudaStream_t)stream), who);
  })
}

e2ttt_status e2ttt_clip_grad_norm(const void* const* g, void* const* out, const size_t* n,
                                  const int* act, int count, float max_norm, float* norm, void* ws,
                                  size_t ws_bytes, void* stream) {
  static const char* who = "e2ttt_clip_grad_norm";
  GUARD(who, {
    if (!norm || ((uintptr_t)norm & 3))
      return failf(E2TTT_ERR_INVALID_ARG, "%s: norm is NULL or unaligned", who);
    if (!(max_norm >= 0.f) || isinf(max_norm))
      return failf(E2TTT_ERR_INVALID_ARG, "%s: max_norm must be finite and >= 0", who);
    const size_t need = e2ttt_grad_workspace_bytes(count);
    TRY(check_ws(who, ws, ws_bytes, need));
    void* none = nullptr;
    std::vector<void*> in_place;
    if (!out && count > 0) {
      in_place.assign((size_t)count, none);
      out = in_place.data();
    }
    TRY(check_grads(who, g, out, n, act, count, norm, ws, need));
    return check_run(grad_clip(GradList{g, out, n, act, count}, max_norm, norm, ws, (cudaStream_t)stream), who);
  })
}

}  // extern "C"
