// Host side of the gated delta rule: the checked arguments of a call and the
// launchers of its kernels.
#pragma once

#include <cuda_runtime.h>

#include "ttt_delta.h"

namespace ttt {

struct DeltaArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  const float* S0;          // or NULL
  const int* seq_starts;    // or NULL
  int n_seq, B, Hk, Hv, N, dk, dv;
  int bf16;
  float scale;
  delta_rule_layout lay;    // filled in for dense calls too
  void* out;
  float* S_final;           // or NULL
  void* workspace;
  int* status;
  unsigned long long wait_ns;
  cudaStream_t stream;
};

struct DeltaStepArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  float* state;
  const int* slots;         // or NULL
  int n_slots, B, Hk, Hv, dk, dv;
  int bf16;
  float scale;
  delta_rule_layout lay;
  void* out;
  int* status;
  cudaStream_t stream;
};

// Token by token in fp32: every type, size and stride.  Returns a ttt_status.
int delta_rule_recurrent(const DeltaArgs& a);

// Chunks of 64 tokens on the tensor cores (bf16, d_k <= 128, aligned strides).
// Returns 1 where it does not apply, else a ttt_status.
int delta_rule_chunk_launch(const DeltaArgs& a);
// Test hook: see ttt_selftest_withhold_delta.
void delta_rule_withhold(int kernel);
// Workspace bytes of such a call (0 where it never applies).
size_t delta_rule_chunk_workspace(int B, int Hv, int N, int dk, int dv, int n_seq);

int delta_rule_step_launch(const DeltaStepArgs& a);

struct BlockNormArgs {
  const void* y;
  const float* w;
  const void* gate;
  const void* residual;
  const float* scale;
  const float* w_next;
  long long rows;
  int D, group;
  int io_bf16, stream_bf16;
  int act;
  float eps;
  block_norm_strides st;
  void* out;
  void* h;
  cudaStream_t stream;
};

int block_norm_launch(const BlockNormArgs& a);

}  // namespace ttt
