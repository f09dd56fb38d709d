// Host side of the fixed-state mixers (window attention, selective scan, short
// convolution): the checked arguments of a call and the launchers of its kernels.
#pragma once

#include <cuda_runtime.h>

#include "ttt_mixers.h"

namespace ttt {

struct WindowArgs {
  const void* q;
  const void* k;
  const void* v;
  void* cache_k;            // or NULL, as
  void* cache_v;
  const int* slots;         // or NULL
  const int* past;          // or NULL
  const int* seq_starts;    // or NULL
  int n_slots, n_seq, B, Hq, Hk, N, d, window, sinks;
  int bf16;
  float scale;
  window_attention_layout lay;   // filled in for dense calls too
  void* out;
  int* status;
  unsigned long long wait_ns;
  cudaStream_t stream;
};

// Every type, size and stride, in fp32.  Returns a ttt_status.
int window_attention_simt(const WindowArgs& a);
// On the tensor cores (bf16, d <= 128, aligned strides, scale > 0).  Returns 1 where it
// does not apply, else a ttt_status.
int window_attention_tc(const WindowArgs& a);
// Test hook: see ttt_selftest_withhold_window.
void window_attention_withhold(int what);
// The new keys and values into the caches, behind the attention.
int window_attention_store(const WindowArgs& a);

struct WindowStepArgs {
  const void* q;
  const void* k;
  const void* v;
  void* cache_k;
  void* cache_v;
  const int* positions;
  const int* slots;         // or NULL
  int n_slots, B, Hq, Hk, d, window, sinks;
  int bf16;
  float scale;
  window_attention_layout lay;
  void* out;
  int* status;
  cudaStream_t stream;
};

int window_attention_step_launch(const WindowStepArgs& a);

struct ScanArgs {
  const void* x;
  const void* dt;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* Dx;          // or NULL
  const float* dt_bias;     // or NULL
  const void* z;            // or NULL
  const float* state_in;    // or NULL
  const int* seq_starts;    // or NULL
  int n_seq, B, N, D, S, G;
  int bf16, softplus;
  selective_scan_layout lay;
  void* out;
  float* state_out;         // or NULL
  void* workspace;
  int* status;
  cudaStream_t stream;
};

size_t selective_scan_workspace(int B, int N, int D, int S, int G, int n_seq, int bf16);
int selective_scan_launch(const ScanArgs& a);

struct ScanStepArgs {
  const void* x;
  const void* dt;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* Dx;
  const float* dt_bias;
  const void* z;
  float* state;
  const int* slots;
  int n_slots, B, D, S, G;
  int bf16, softplus;
  selective_scan_layout lay;
  void* out;
  int* status;
  cudaStream_t stream;
};

int selective_scan_step_launch(const ScanStepArgs& a);

struct ConvArgs {
  const void* x;
  const float* w;
  const float* bias;        // or NULL
  const void* state_in;     // or NULL
  const int* seq_starts;    // or NULL
  int n_seq, B, N, D, W;
  int bf16, silu;
  short_conv_layout lay;
  void* out;
  void* state_out;          // or NULL
  int* status;
  cudaStream_t stream;
};

int short_conv_launch(const ConvArgs& a);

struct ConvStepArgs {
  const void* x;
  const float* w;
  const float* bias;
  void* state;
  const int* slots;
  int n_slots, B, D, W;
  int bf16, silu;
  short_conv_layout lay;
  void* out;
  int* status;
  cudaStream_t stream;
};

int short_conv_step_launch(const ConvStepArgs& a);

}  // namespace ttt
