// Internal interfaces of the operators around a recurrent layer: the short
// causal convolution (conv.cu), the state-space scan (ssm.cu, ssm_tc.cu) and
// the gradient norm (grad_norm.cu). Their C entry points are in seq_api.cu.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace e2ttt {

// A workspace starts with its status word (e2ttt_workspace_status), which every call resets.
constexpr size_t kStatusBytes = 256;

// Number of SMs of the current device (asked once per device and thread).
int sm_count();
// The SMs that work is split for where the split sets a workspace's size or the order of
// sums: a B200's, not asked, so that both depend on the shape alone.
constexpr int kPlannedSms = 148;

// ------------------------------------------------------------------ convolution
struct ConvDims {
  int B, H, T, d, W;
  bool bf16_act, silu;
};
struct ConvArgs {
  ConvDims s;
  const void* x;
  const float *w, *bias;  // bias may be NULL
  const void* state;      // may be NULL: zeros
  const int* lengths;     // may be NULL: T everywhere
  bool vec;               // vectors of 4 channels apply: row size and every pointer
  cudaStream_t st;
};
size_t conv_bwd_workspace_bytes(const ConvDims& s);
cudaError_t conv_fwd(const ConvArgs& a, void* y, void* state_end);
cudaError_t conv_bwd(const ConvArgs& a, const void* dy, const void* dstate_end, void* dx, float* dw,
                     float* dbias, void* dstate, void* ws);
cudaError_t conv_step(const ConvArgs& a, void* state, void* y);

// ------------------------------------------------------------------ scan
struct SsmDims {
  int B, H, G, T;
  int N, P;      // state columns (d_k) and rows (d_v)
  int Q, NC;     // tokens per chunk, chunks
  int NPT;       // tiles of kSsmPT state rows
  bool bf16_act;
  bool tc;       // chunks run on the tcgen05 kernels (ssm_tc.cu)
};
constexpr int kSsmPT = 64;
constexpr int kSsmTcChunk = 128;  // tokens per chunk on the tensor cores

struct SsmFwdArgs {
  SsmDims s;
  const void *q, *k, *v;
  const float *dt, *A, *D, *S0;
  const int* lengths;
  void* y;
  float* S_end;
  float* states;  // [NC][B*H][P][N]: saved_states or workspace
  float* decay;   // [NC][B*H] workspace
  float* logs;    // tensor cores: the chunks' logarithms, workspace
  void* starts;   // tensor cores: the chunks' start states in bf16, workspace
  bool keep;      // the fp32 states are wanted (saved_states)
  int* status;    // device status word of the bounded waits
  cudaStream_t st;
};
cudaError_t ssm_fwd(const SsmFwdArgs& a);     // tf32 pairs on mma.sync, any shape
cudaError_t ssm_tc_fwd(const SsmFwdArgs& a);  // tcgen05 kernels, shapes with tc set
size_t ssm_tc_logs_bytes(const SsmDims& s);
// Test hook behind e2ttt_test_stall_next_scan.
void arm_scan_stall(int wait);
// The states' passage along the chunks (back: their adjoint's, from the end),
// from `first` (NULL: zero); what is left after the last chunk goes to `last`, a
// bf16 copy of the states to `copy` (may be NULL); without `keep` only that.
cudaError_t ssm_carry(const SsmDims& s, bool back, const float* first, const float* decay,
                      float* states, float* last, void* copy, bool keep, cudaStream_t st);

struct SsmBwdArgs {
  SsmDims s;
  const void *q, *k, *v;
  const float *dt, *A, *D;
  const int* lengths;
  const float* states;  // from the forward
  const void* dy;
  const float* dS_end;
  void *dq, *dk, *dv;
  float *ddt, *dA, *dD, *dS0;
  void* ws;
  cudaStream_t st;
};
// The backward's workspace, cut up.
struct SsmBwdScratch {
  int* status;
  float *ends, *decay, *logs;  // [NC][B*H][P][N], [NC][B*H], the chunks' logarithms (tensor cores)
  float *dq, *dk;              // [B*G][parts][T][N] sums over part of a group's heads
  float* ddt;                  // [NPT][B*H][T]; the output itself where NPT is 1
  double *dA, *dD;             // [NC][NPT][B*H]; the parts cancel
};
size_t ssm_bwd_workspace_bytes(const SsmDims& s);
cudaError_t ssm_bwd(const SsmBwdArgs& a);
cudaError_t ssm_tc_bwd(const SsmBwdArgs& a, const SsmBwdScratch& w);
int ssm_tc_grad_parts(const SsmDims& s);
// dq, dk (where there are several parts), ddt, dA and dD from their parts.
cudaError_t ssm_grad_sums(const SsmBwdArgs& a, const SsmBwdScratch& w, int parts);

struct SsmStepArgs {
  SsmDims s;
  const void *q, *k, *v;
  const float *dt, *A, *D;
  float* S;
  void* y;
  cudaStream_t st;
};
cudaError_t ssm_step(const SsmStepArgs& a);

// ------------------------------------------------------------------ gradient norm
struct GradList {
  const void* const* g;
  void* const* out;  // NULL: in place
  const size_t* n;
  const int* act;
  int count;
};
constexpr int kGradBlocksMax = 1024;
size_t grad_workspace_bytes(int count);
cudaError_t grad_norm(const GradList& l, float* norm, void* ws, cudaStream_t st);
cudaError_t grad_clip(const GradList& l, float max_norm, float* norm, void* ws, cudaStream_t st);

}  // namespace e2ttt
