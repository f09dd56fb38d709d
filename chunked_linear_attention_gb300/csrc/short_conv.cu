// The short causal convolution, per channel y_t = bias + sum_j w_j x_{t - W + 1 + j} with
// an optional SiLU: whole sequences, and single tokens on a pool of states.
//
// Bound by HBM: each input is read once and each output written once, W products an
// element.
#include <climits>

#include "mixers.cuh"
#include "mixers.h"
#include "prof.h"

namespace ttt {

namespace {

struct ConvParams {
  const void* x;
  const float* w;
  const float* bias;
  const void* state_in;
  const int* starts;
  void* out;
  void* state_out;
  int* status;
  int n_seq, N, D, vecs, tiles;
  long long units;       // batch x tiles x vecs
  int silu;
  short_conv_layout lay;
};

// ------------------------------------------------------------ whole sequences
// A thread has E neighbouring channels (16 bytes) of TT tokens, the last W - 1 inputs in
// registers; neighbouring threads have neighbouring channels.  The inputs before its first
// token are read again, from the L2.
constexpr int kConvTokens = 16;

template <typename T, int W, int E, bool VEC>
__global__ void __launch_bounds__(128) short_conv_kernel(const __grid_constant__ ConvParams p) {
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0 && p.starts) check_starts(p.starts, p.n_seq, p.N, p.status);
  const long long u = blockIdx.x * 128ll + threadIdx.x;
  if (u >= p.units) return;
  const int c = (int)(u % p.vecs) * E;
  const long long bt = u / p.vecs;
  const int tile = (int)(bt % p.tiles), b = (int)(bt / p.tiles);
  const int n = VEC ? E : min(E, p.D - c);
  float w[W][E], bias[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    bias[e] = p.bias && e < n ? p.bias[c + e] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][e] = e < n ? p.w[(long long)(c + e) * W + j] : 0.f;
  }
  const T* x = static_cast<const T*>(p.x) + b * p.lay.x.batch + c;
  T* out = static_cast<T*>(p.out) + b * p.lay.out.batch + c;
  const T* sin = static_cast<const T*>(p.state_in);
  T* sout = static_cast<T*>(p.state_out);

  // input `row` of a sequence's state (0: the oldest) before its first token
  auto from_state = [&](int seq, int row, float (&v)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.f;
    if (sin) load_row<T, E, VEC>(sin + ((long long)seq * (W - 1) + row) * p.D + c, n, v);
  };
  auto input = [&](const TokenSeq& s, int t, float (&v)[E]) {   // token t, perhaps before t0
    if (t >= s.t0) load_row<T, E, VEC>(x + t * p.lay.x.token, n, v);
    else from_state(s.seq, W - 1 + (t - s.t0), v);
  };

  // the states of empty sequences, spread over the tiles
  if (sout && p.starts)
    for (int s = tile; s < p.n_seq; s += p.tiles)
      if (p.starts[s] == p.starts[s + 1])
        for (int r = 0; r < W - 1; ++r) {
          float v[E];
          from_state(s, r, v);
          store_row<T, E, VEC>(sout + ((long long)s * (W - 1) + r) * p.D + c, n, v);
        }

  const int end = min((tile + 1) * kConvTokens, p.N);
  int t = tile * kConvTokens;
  while (t < end) {
    const TokenSeq s = token_seq(p.starts, p.n_seq, b, p.N, t);
    if (s.seq < 0) {   // tokens of no sequence
      ++t;
      continue;
    }
    float h[W - 1][E];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) input(s, t - (W - 1) + j, h[j]);
    const int stop = min(end, s.t1);
#pragma unroll 4
    for (; t < stop; ++t) {
      float v[E], y[E];
      load_row<T, E, VEC>(x + t * p.lay.x.token, n, v);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float a = bias[e];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) a = fmaf(w[j][e], h[j][e], a);
        a = fmaf(w[W - 1][e], v[e], a);
        y[e] = p.silu ? silu_f(a) : a;
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) h[j][e] = h[j + 1][e];
        h[W - 2][e] = v[e];
      }
      store_row<T, E, VEC>(out + t * p.lay.out.token, n, y);
    }
    if (sout && stop == s.t1) {
#pragma unroll
      for (int r = 0; r < W - 1; ++r)
        store_row<T, E, VEC>(sout + ((long long)s.seq * (W - 1) + r) * p.D + c, n, h[r]);
    }
  }
}

bool wide(const void* x, int bytes) { return (reinterpret_cast<uintptr_t>(x) & (bytes - 1)) == 0; }

template <typename T, int W>
int conv_w(const ConvArgs& a, ConvParams p) {
  constexpr int E = 16 / sizeof(T);
  const bool vec = a.D % E == 0 && wide(a.x, 16) && wide(a.out, 16) && wide(a.state_in, 16) &&
                   wide(a.state_out, 16) && a.lay.x.batch % E == 0 && a.lay.x.token % E == 0 &&
                   a.lay.out.batch % E == 0 && a.lay.out.token % E == 0;
  const int per = vec ? E : 1;
  p.vecs = (a.D + per - 1) / per;
  p.tiles = (a.N + kConvTokens - 1) / kConvTokens;
  p.units = (long long)a.B * p.tiles * p.vecs;
  const long long grid = (p.units + 127) / 128;
  if (grid > INT_MAX) return TTT_ERR_UNSUPPORTED;
  const double n = (double)a.B * a.N * a.D;
  ProfScope ps(PT_CONV, a.stream, 2.0 * n * W, 2.0 * n * sizeof(T));
  const cudaError_t e =
      vec ? launch_behind(short_conv_kernel<T, W, E, true>, (unsigned)grid, 128, 0, a.stream, p)
          : launch_behind(short_conv_kernel<T, W, 1, false>, (unsigned)grid, 128, 0, a.stream, p);
  return e == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

template <typename T>
int conv_t(const ConvArgs& a, const ConvParams& p) {
  switch (a.W) {
    case 2: return conv_w<T, 2>(a, p);
    case 3: return conv_w<T, 3>(a, p);
    case 4: return conv_w<T, 4>(a, p);
    case 5: return conv_w<T, 5>(a, p);
    case 6: return conv_w<T, 6>(a, p);
    case 7: return conv_w<T, 7>(a, p);
    default: return conv_w<T, 8>(a, p);
  }
}

// ------------------------------------------------------------ single tokens
struct ConvStepParams {
  const void* x;
  const float* w;
  const float* bias;
  void* state;
  const int* slots;
  void* out;
  int* status;
  int n_slots, D, W, silu;
  short_conv_layout lay;
};

// One CTA: 128 E channels of one row.
template <typename T, int E, bool VEC>
__global__ void __launch_bounds__(128) conv_step_kernel(const __grid_constant__ ConvStepParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.y, c = (blockIdx.x * 128 + threadIdx.x) * E;
  const int slot = row_slot(p.slots, p.n_slots, b, p.status);
  if (c >= p.D) return;
  const int n = VEC ? E : min(E, p.D - c);
  T* out = static_cast<T*>(p.out) + b * p.lay.out.batch + c;
  float y[E];
  if (slot < 0) {
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = 0.f;
    store_row<T, E, VEC>(out, n, y);
    return;
  }
  float v[E];
  load_row<T, E, VEC>(static_cast<const T*>(p.x) + b * p.lay.x.batch + c, n, v);
  const float* w = p.w + (long long)c * p.W;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    y[e] = p.bias && e < n ? p.bias[c + e] : 0.f;
    if (e < n) y[e] = fmaf(w[e * p.W + p.W - 1], v[e], y[e]);
  }
  T* st = static_cast<T*>(p.state) + (long long)slot * (p.W - 1) * p.D + c;
  for (int j = 0; j < p.W - 1; ++j) {
    float h[E];
    load_row<T, E, VEC>(st + (long long)j * p.D, n, h);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e < n) y[e] = fmaf(w[e * p.W + j], h[e], y[e]);
    if (j > 0) store_row<T, E, VEC>(st + (long long)(j - 1) * p.D, n, h);
  }
  store_row<T, E, VEC>(st + (long long)(p.W - 2) * p.D, n, v);
  if (p.silu) {
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = silu_f(y[e]);
  }
  store_row<T, E, VEC>(out, n, y);
}

template <typename T>
int conv_step_t(const ConvStepArgs& a, const ConvStepParams& p) {
  constexpr int E = 8 / sizeof(T);
  const bool vec = a.D % E == 0 && wide(a.x, 8) && wide(a.out, 8) && wide(a.state, 8) &&
                   a.lay.x.batch % E == 0 && a.lay.out.batch % E == 0;
  const int per = 128 * (vec ? E : 1);
  const dim3 grid((a.D + per - 1) / per, a.B);
  const double n = (double)a.B * a.D;
  ProfScope ps(PT_CONV_STEP, a.stream, 2.0 * n * a.W, 2.0 * n * a.W * sizeof(T));
  const cudaError_t e = vec ? launch_grid(conv_step_kernel<T, E, true>, grid, 128, 0, a.stream, p)
                            : launch_grid(conv_step_kernel<T, 1, false>, grid, 128, 0, a.stream, p);
  return e == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

}  // namespace

int short_conv_launch(const ConvArgs& a) {
  ConvParams p{};
  p.x = a.x; p.w = a.w; p.bias = a.bias; p.state_in = a.state_in;
  p.starts = a.seq_starts;
  p.out = a.out;
  p.state_out = a.state_out;
  p.status = a.status;
  p.n_seq = a.n_seq; p.N = a.N; p.D = a.D;
  p.silu = a.silu;
  p.lay = a.lay;
  return a.bf16 ? conv_t<__nv_bfloat16>(a, p) : conv_t<float>(a, p);
}

int short_conv_step_launch(const ConvStepArgs& a) {
  ConvStepParams p{};
  p.x = a.x; p.w = a.w; p.bias = a.bias; p.state = a.state;
  p.slots = a.slots;
  p.out = a.out;
  p.status = a.status;
  p.n_slots = a.n_slots; p.D = a.D; p.W = a.W; p.silu = a.silu;
  p.lay = a.lay;
  return a.bf16 ? conv_step_t<__nv_bfloat16>(a, p) : conv_step_t<float>(a, p);
}

}  // namespace ttt
