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
  int n_seq, N, D, vecs, tiles, tokens;
  long long units;       // batch x tiles x vecs
  int silu;
  short_conv_layout lay;
};

// ------------------------------------------------------------ whole sequences
// A thread has E neighbouring channels of up to 64 tokens, the last W - 1 inputs in
// registers; neighbouring threads have neighbouring channels.  The inputs before its first
// token are read again, from the L2.  Eight tokens are worked on while the next eight are on
// their way; channels go in pairs through the packed fp32 instructions.  What is in flight
// decides: with eight bf16 channels a thread (16 bytes an access, 159 registers) 2 x 32768
// tokens of 1536 channels take 108 us, with four (8 bytes) and four tokens 88, and eight
// tokens 76; the filters spilled to local memory for more blocks cost far more.
constexpr int kConvGroup = 8;

template <typename T, int W, int E, bool VEC>
__global__ void __launch_bounds__(128) short_conv_kernel(const __grid_constant__ ConvParams p) {
  constexpr int P = (E + 1) / 2, U = kConvGroup;   // pairs of channels
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0 && p.starts) check_starts(p.starts, p.n_seq, p.N, p.status);
  const long long u = blockIdx.x * 128ll + threadIdx.x;
  if (u >= p.units) return;
  const int bt = (int)(u / p.vecs), c = (int)(u - (long long)bt * p.vecs) * E;
  const int b = bt / p.tiles, tile = bt - b * p.tiles;
  const int n = VEC ? E : min(E, p.D - c);
  F2 w[W][P], bias[P];
#pragma unroll
  for (int e = 0; e < P; ++e) {
    float v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = p.bias && 2 * e + i < n ? p.bias[c + 2 * e + i] : 0.f;
    bias[e] = pack2(v[0], v[1]);
#pragma unroll
    for (int j = 0; j < W; ++j) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[i] = 2 * e + i < n ? p.w[(long long)(c + 2 * e + i) * W + j] : 0.f;
      w[j][e] = pack2(v[0], v[1]);
    }
  }
  const T* x = static_cast<const T*>(p.x) + b * p.lay.x.batch + c;
  T* out = static_cast<T*>(p.out) + b * p.lay.out.batch + c;
  const T* sin = static_cast<const T*>(p.state_in);
  T* sout = static_cast<T*>(p.state_out);
  using V = Pack<T, E>;

  auto zero = [&](V& v) {
#pragma unroll
    for (int e = 0; e < E; ++e) v.v[e] = from_f<T>(0.f);
  };
  // input `row` of a sequence's state (0: the oldest) before its first token
  auto from_state = [&](int seq, int row, V& v) {
    zero(v);
    if (sin) load_pack<T, E, VEC>(sin + ((long long)seq * (W - 1) + row) * p.D + c, n, v);
  };
  auto to_state = [&](int seq, int row, const V& v) {
    T* to = sout + ((long long)seq * (W - 1) + row) * p.D + c;
    if constexpr (VEC) {
      *reinterpret_cast<V*>(to) = v;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e < n) to[e] = v.v[e];
    }
  };
  auto input = [&](const TokenSeq& s, int t, V& v) {   // token t, perhaps before t0
    if (t >= s.t0) load_pack<T, E, VEC>(x + t * p.lay.x.token, n, v);
    else from_state(s.seq, W - 1 + (t - s.t0), v);
  };
  auto pairs = [&](const V& q, F2 (&v)[P]) {
    float f[E];
    pack_f(q, f);
#pragma unroll
    for (int e = 0; e < P; ++e) v[e] = pack2(f[2 * e], 2 * e + 1 < E ? f[2 * e + 1] : 0.f);
  };
  const F2 l2e = pack2(-1.44269504088896341f, -1.44269504088896341f), ones = pack2(1.f, 1.f);
  // one output from the W inputs that end with its token
  auto one = [&](const F2 (*h)[P], T* to) {
    float y[E];
#pragma unroll
    for (int e = 0; e < P; ++e) {
      F2 a = bias[e];
#pragma unroll
      for (int j = 0; j < W; ++j) a = fma2(w[j][e], h[j][e], a);
      if (p.silu) {   // a / (1 + e^-a)
        float e0, e1;
        unpack2(mul2(a, l2e), e0, e1);
        unpack2(add2(pack2(ex2(e0), ex2(e1)), ones), e0, e1);
        a = mul2(a, pack2(rcp_f(e0), rcp_f(e1)));
      }
      float a0, a1;
      unpack2(a, a0, a1);
      y[2 * e] = a0;
      if (2 * e + 1 < E) y[2 * e + 1] = a1;
    }
    store_row<T, E, VEC>(to, n, y);
  };

  // the states of empty sequences, spread over the tiles
  if (sout && p.starts)
    for (int s = tile; s < p.n_seq; s += p.tiles)
      if (p.starts[s] == p.starts[s + 1])
        for (int r = 0; r < W - 1; ++r) {
          V v;
          from_state(s, r, v);
          to_state(s, r, v);
        }

  const int end = min((tile + 1) * p.tokens, p.N);
  int t = tile * p.tokens;
  while (t < end) {
    const TokenSeq s = token_seq(p.starts, p.n_seq, b, p.N, t);
    if (s.seq < 0) {   // tokens of no sequence
      ++t;
      continue;
    }
    F2 h[W - 1 + U][P];   // inputs t - W + 1 .. t + U - 1
    V q[U];
    const int stop = min(end, s.t1);
    const T* xt = x + t * p.lay.x.token;
    T* ot = out + t * p.lay.out.token;
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (t + i < stop) load_pack<T, E, VEC>(xt + i * p.lay.x.token, n, q[i]);
    {
      V v[W - 1];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) input(s, t - (W - 1) + j, v[j]);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) pairs(v[j], h[j]);
    }
#pragma unroll 1
    while (t < stop) {
      const int m = min(U, stop - t);
#pragma unroll
      for (int i = 0; i < U; ++i) pairs(q[i], h[W - 1 + i]);
      xt += U * p.lay.x.token;
      if (t + 2 * U <= stop) {
#pragma unroll
        for (int i = 0; i < U; ++i) load_pack<T, E, VEC>(xt + i * p.lay.x.token, n, q[i]);
      } else {
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (t + U + i < stop) load_pack<T, E, VEC>(xt + i * p.lay.x.token, n, q[i]);
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (i < m) one(h + i, ot + i * p.lay.out.token);
      ot += U * p.lay.out.token;
      t += m;
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < P; ++e) h[j][e] = h[j + U][e];
    }
    if (sout && stop == s.t1) {
#pragma unroll
      for (int r = 0; r < W - 1; ++r) {
        V v;
        input(s, s.t1 - (W - 1) + r, v);
        to_state(s.seq, r, v);
      }
    }
  }
}

bool wide(const void* x, int bytes) { return (reinterpret_cast<uintptr_t>(x) & (bytes - 1)) == 0; }

template <typename T, int W>
int conv_w(const ConvArgs& a, ConvParams p) {
  constexpr int E = 4, bytes = E * sizeof(T);
  const bool vec = a.D % E == 0 && wide(a.x, bytes) && wide(a.out, bytes) &&
                   wide(a.state_in, bytes) && wide(a.state_out, bytes) && a.lay.x.batch % E == 0 && a.lay.x.token % E == 0 &&
                   a.lay.out.batch % E == 0 && a.lay.out.token % E == 0;
  const int per = vec ? E : 1;
  p.vecs = (a.D + per - 1) / per;
  // long tiles read few inputs twice, short ones fill the card: as long as there are 1024
  // threads for every SM (20011 tokens of 1000 channels: 64 tokens 34.8 us, 32 33.0)
  p.tokens = 64;
  while (p.tokens > 8 && (long long)a.B * ((a.N + p.tokens - 1) / p.tokens) * p.vecs < 152 * 1024)
    p.tokens /= 2;
  p.tiles = (a.N + p.tokens - 1) / p.tokens;
  p.units = (long long)a.B * p.tiles * p.vecs;
  const long long grid = (p.units + 127) / 128;
  if (grid > INT_MAX || (long long)a.B * p.tiles > INT_MAX) return TTT_ERR_UNSUPPORTED;
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
  int n_slots, B, D, silu;
  short_conv_layout lay;
};

// One CTA: 128 E channels of R rows, whose states and inputs are on their way together; the
// filters, in registers, serve all of them.
template <typename T, int W, int E, int R, bool VEC>
__global__ void __launch_bounds__(128) conv_step_kernel(const __grid_constant__ ConvStepParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int b0 = blockIdx.y * R, c = (blockIdx.x * 128 + threadIdx.x) * E;
  const int n = VEC ? (c < p.D ? E : 0) : max(0, min(E, p.D - c));
  int slot[R];
  read_slots<R>(p.slots, b0, p.B, slot);
  using V = Pack<T, E>;
  V h[R][W - 1], x[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (n == 0 || slot[i] < 0 || slot[i] >= p.n_slots) continue;
    load_pack<T, E, VEC>(static_cast<const T*>(p.x) + (b0 + i) * p.lay.x.batch + c, n, x[i]);
    const T* st = static_cast<const T*>(p.state) + (long long)slot[i] * (W - 1) * p.D + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_pack<T, E, VEC>(st + (long long)j * p.D, n, h[i][j]);
  }
  float w[E * W], bias[E];
  const float* from = p.w + (long long)c * W;
  if constexpr (VEC) {
    constexpr int P = E * W % 4 == 0 ? 4 : 2;
    using Q = Pack<float, P>;
    if (n > 0) {
#pragma unroll
      for (int e = 0; e < E * W; e += P) {
        const Q q = *reinterpret_cast<const Q*>(from + e);
#pragma unroll
        for (int k = 0; k < P; ++k) w[e + k] = q.v[k];
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < E * W; ++e) w[e] = e < n * W ? from[e] : 0.f;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) bias[e] = p.bias && e < n ? p.bias[c + e] : 0.f;
  drop_bad_slots<R>(p.slots, p.n_slots, b0, p.B, p.status, slot);
  if (n == 0) return;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (b0 + i >= p.B) return;
    T* out = static_cast<T*>(p.out) + (b0 + i) * p.lay.out.batch + c;
    float y[E], v[E];
    if (slot[i] < 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = 0.f;
      store_row<T, E, VEC>(out, n, y);
      continue;
    }
    pack_f(x[i], v);
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = fmaf(w[e * W + W - 1], v[e], bias[e]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      pack_f(h[i][j], v);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = fmaf(w[e * W + j], v[e], y[e]);
    }
    if (p.silu) {
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = silu_f(y[e]);
    }
    store_row<T, E, VEC>(out, n, y);
    T* st = static_cast<T*>(p.state) + (long long)slot[i] * (W - 1) * p.D + c;
#pragma unroll
    for (int j = 1; j < W; ++j) {
      const V& q = j < W - 1 ? h[i][j] : x[i];
      if constexpr (VEC) {
        *reinterpret_cast<V*>(st + (long long)(j - 1) * p.D) = q;
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (e < n) st[(long long)(j - 1) * p.D + e] = q.v[e];
      }
    }
  }
}

template <typename T, int W>
int conv_step_w(const ConvStepArgs& a, const ConvStepParams& p) {
  constexpr int E = 8 / sizeof(T);
  const bool vec = a.D % E == 0 && wide(a.x, 8) && wide(a.out, 8) && wide(a.state, 8) &&
                   wide(a.w, 16) && a.lay.x.batch % E == 0 && a.lay.out.batch % E == 0;
  const int per = 128 * (vec ? E : 1);
  const unsigned blocks = (a.D + per - 1) / per;
  // four rows a thread where every SM gets a block all the same (512 rows of 4096 channels
  // 7.4 us, one row a thread 9.1; 128 rows 3.8 and 4.0)
  const bool four = vec && (long long)blocks * ((a.B + 3) / 4) >= 152;
  const dim3 grid(blocks, four ? (a.B + 3) / 4 : a.B);
  const double n = (double)a.B * a.D;
  ProfScope ps(PT_CONV_STEP, a.stream, 2.0 * n * W, 2.0 * n * W * sizeof(T));
  void (*kern)(ConvStepParams) = four  ? conv_step_kernel<T, W, E, 4, true>
                                 : vec ? conv_step_kernel<T, W, E, 1, true>
                                       : conv_step_kernel<T, W, 1, 1, false>;
  return launch_grid(kern, grid, 128, 0, a.stream, p) == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

template <typename T>
int conv_step_t(const ConvStepArgs& a, const ConvStepParams& p) {
  switch (a.W) {
    case 2: return conv_step_w<T, 2>(a, p);
    case 3: return conv_step_w<T, 3>(a, p);
    case 4: return conv_step_w<T, 4>(a, p);
    case 5: return conv_step_w<T, 5>(a, p);
    case 6: return conv_step_w<T, 6>(a, p);
    case 7: return conv_step_w<T, 7>(a, p);
    default: return conv_step_w<T, 8>(a, p);
  }
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
  p.n_slots = a.n_slots; p.B = a.B; p.D = a.D; p.silu = a.silu;
  p.lay = a.lay;
  return a.bf16 ? conv_step_t<__nv_bfloat16>(a, p) : conv_step_t<float>(a, p);
}

}  // namespace ttt
