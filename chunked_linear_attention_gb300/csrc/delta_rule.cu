// The gated delta rule token by token in fp32, for every type, size and
// stride: the whole-sequence form where the tensor-core kernel does not apply,
// and the single-token form on a pool of states.
//
// A row of the state S [d_v, d_k] only meets its own value, so rows are
// independent: S_i <- a S_i + u_i k^T with u_i = beta (v_i - a S_i k).  L lanes
// hold one row, E elements each, and the state stays in registers over the
// tokens.  With S the state before the token, both products of a token are
// taken from it at once, S k and S q (o = scale (a S q + u (k . q))), so a
// token costs one butterfly over L lanes and not two in a row.
#include <type_traits>

#include "delta_tc.cuh"
#include "prof.h"

namespace ttt {

namespace {

constexpr int kStatusArg = -8;  // TTT_ERR_ARG

// Element e of lane l in a row: groups of four neighbours per lane (16-byte
// accesses, 16 L bytes in one piece per access of the L lanes).
template <int L>
__device__ __forceinline__ int elem(int l, int e) {
  return (e >> 2) * (4 * L) + l * 4 + (e & 3);
}

template <int L>
__device__ __forceinline__ float sum_lanes(float x) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The tokens of sequence s: [t0, t0 + len).  Bad bounds give an empty
// sequence and TTT_ERR_ARG.
__device__ __forceinline__ void seq_range(const int* starts, int s, int N, int* status, int& t0,
                                          int& len) {
  const int a = starts[s], b = starts[s + 1];
  const bool ok = a >= 0 && a <= b && b <= N;
  if (!ok) report_status(status, kStatusArg);
  t0 = ok ? a : 0;
  len = ok ? b - a : 0;
}

// Numbers one at a time, or two in one register for the packed instructions.
__device__ __forceinline__ float fma_(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ F2 fma_(F2 a, F2 b, F2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float mul_(float a, float b) { return a * b; }
__device__ __forceinline__ F2 mul_(F2 a, F2 b) { return mul2(a, b); }
__device__ __forceinline__ void all_(float& v, float x) { v = x; }
__device__ __forceinline__ void all_(F2& v, float x) { v = pack2(x, x); }
__device__ __forceinline__ float sum_(const float (&a)[4]) { return (a[0] + a[1]) + (a[2] + a[3]); }
__device__ __forceinline__ float sum_(const F2 (&a)[2]) {
  float x, y;
  unpack2(add2(a[0], a[1]), x, y);
  return x + y;
}
__device__ __forceinline__ void four(float* v, const float* p) {
  *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ void four(F2* v, const float* p) {
  const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(p);
  v[0] = x.x;
  v[1] = x.y;
}

// ------------------------------------------------------------ whole sequences
// One CTA: 16 rows of one (sequence, head): four warps compute, four more bring
// the next TT tokens' k, q, v (as fp32), decay, beta and k . q into the other half
// of the shared memory.  Bound by the chain of a token (two dot products, a
// butterfly, the update), hidden in part by the other CTA of the SM: in fp32 B 4,
// H 4, 8192 tokens take 1.61 ms at d 128 (0.20 us a token; 128 CTAs, so most
// SMs hold one), 256 tokens of one head 31 us at d 32 and 58 at d 128.  With d_k of
// 256, two CTAs per SM (128 registers) take 0.86 ms for 2048 tokens (before the packed
// instructions 1.00, and one CTA 1.34); of 512, four rows a thread 1.04 ms for 512 tokens
// and two 1.5 (held to registers for one block by the launch bounds, 1.60).
constexpr int kRecWarps = 4;

struct RecParams {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  const float* S0;
  const int* starts;
  void* out;
  float* S_final;
  int* status;
  int Hk, Hv, N, dk, dv, row_tiles;
  float scale;
  delta_rule_layout lay;
};

template <typename T, int L, int E, int R, int TT>
__global__ void __launch_bounds__(256, R < 4 ? 2 : 0)
    delta_recurrent_kernel(const __grid_constant__ RecParams p) {
  constexpr int W = L * E;                         // padded d_k
  constexpr int ROWS = kRecWarps * (32 / L) * R;   // rows of this CTA
  constexpr int TOK = 2 * W + ROWS + 4;            // floats per staged token
  extern __shared__ __align__(16) float stage[];   // [2][TT][TOK]
  pdl_launch_dependents();
  pdl_wait();
  const int tile = blockIdx.x % p.row_tiles;
  const int sh = blockIdx.x / p.row_tiles;
  const int h = sh % p.Hv, s = sh / p.Hv;
  const int hk = h / (p.Hv / p.Hk);
  int t0 = 0, len = p.N;
  long long batch = s;
  if (p.starts) {
    seq_range(p.starts, s, p.N, p.status, t0, len);
    batch = 0;
  }
  const T* q = static_cast<const T*>(p.q) + batch * p.lay.q.batch + hk * p.lay.q.head +
               t0 * p.lay.q.token;
  const T* k = static_cast<const T*>(p.k) + batch * p.lay.k.batch + hk * p.lay.k.head +
               t0 * p.lay.k.token;
  const T* v = static_cast<const T*>(p.v) + batch * p.lay.v.batch + h * p.lay.v.head +
               t0 * p.lay.v.token;
  const float* g = p.g + batch * p.lay.g.batch + h * p.lay.g.head + t0 * p.lay.g.token;
  const float* be = p.beta + batch * p.lay.beta.batch + h * p.lay.beta.head + t0 * p.lay.beta.token;
  T* out = static_cast<T*>(p.out) + batch * p.lay.out.batch + h * p.lay.out.head +
           t0 * p.lay.out.token;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = tile * ROWS;
  const int ntile = (len + TT - 1) / TT;

  // by the loader warps: all of a warp's tokens are on their way before the first
  // is put down (one after the other, a tile waited for four trips to memory)
  constexpr int TPW = TT / kRecWarps, KE = W / 32, VE = (ROWS + 31) / 32;
  auto load = [&](int it, int buf) {
    float kv[TPW][KE], qv[TPW][KE], vv[TPW][VE], gv[TPW], bv[TPW];
#pragma unroll
    for (int x = 0; x < TPW; ++x) {
      const int t = it * TT + x * kRecWarps + warp - kRecWarps;
      const bool in = t < len;
#pragma unroll
      for (int e = 0; e < KE; ++e) {
        const int c = 32 * e + lane;
        kv[x][e] = in && c < p.dk ? to_f<T>(k[t * p.lay.k.token + c]) : 0.f;
        qv[x][e] = in && c < p.dk ? to_f<T>(q[t * p.lay.q.token + c]) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int c = 32 * e + lane;
        vv[x][e] = in && c < ROWS && row0 + c < p.dv ? to_f<T>(v[t * p.lay.v.token + row0 + c]) : 0.f;
      }
      gv[x] = in ? g[t * p.lay.g.token] : 0.f;
      bv[x] = in ? be[t * p.lay.beta.token] : 0.f;
    }
#pragma unroll
    for (int x = 0; x < TPW; ++x) {
      float* d = stage + (buf * TT + x * kRecWarps + warp - kRecWarps) * TOK;
      float kq = 0.f;
#pragma unroll
      for (int e = 0; e < KE; ++e) {
        d[32 * e + lane] = kv[x][e];
        d[W + 32 * e + lane] = qv[x][e];
        kq = fmaf(kv[x][e], qv[x][e], kq);
      }
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (32 * e + lane < ROWS) d[2 * W + 32 * e + lane] = vv[x][e];
      kq = sum_lanes<32>(kq);
      if (lane == 0)
        *reinterpret_cast<float4*>(d + 2 * W + ROWS) = make_float4(expf(gv[x]), bv[x], kq, 0.f);
    }
  };

  const int l = lane % L;
  // Packed from 8 elements a lane on (64 heads, 4096 tokens: d 128 2.49 -> 2.26 ms, d 64 825
  // -> 792 us; with 4, 64 heads of d 32 and 2048 tokens, 236 -> 244 us).
  using V = std::conditional_t<(E >= 8), F2, float>;
  constexpr int PW = sizeof(V) / 4, NA = 4 / PW;
  V S[R][E / PW];
  int row[R];
  bool mine[R];   // this lane stores the row's outputs
  T* op = out + row0 + warp * R * (32 / L) + lane / L;
  const long long sbase = (long long)sh * p.dv * p.dk;
  if (warp < kRecWarps) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      row[r] = (warp * R + r) * (32 / L) + lane / L;
      mine[r] = l == 0 && row0 + row[r] < p.dv;
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = elem<L>(l, e + i);
          s[i] = p.S0 && row0 + row[r] < p.dv && c < p.dk
                     ? p.S0[sbase + (long long)(row0 + row[r]) * p.dk + c]
                     : 0.f;
        }
        if constexpr (PW == 2) {
          S[r][e / 2] = pack2(s[0], s[1]);
          S[r][e / 2 + 1] = pack2(s[2], s[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) S[r][e + i] = s[i];
        }
      }
    }
  } else if (ntile > 0) {
    load(0, 0);
  }
  __syncthreads();
  for (int it = 0; it < ntile; ++it) {
    const int buf = it & 1;
    if (warp >= kRecWarps) {
      if (it + 1 < ntile) load(it + 1, buf ^ 1);
    } else {
      const int n = min(TT, len - it * TT);
      // a token's operands are read while the one before it is worked on
      V kk[E / PW], qq[E / PW];
      float vv[R];
      float4 f;
      const float* d = stage + buf * TT * TOK;
      auto fetch = [&]() {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          four(&kk[e / PW], d + elem<L>(l, e));
          four(&qq[e / PW], d + W + elem<L>(l, e));
        }
#pragma unroll
        for (int r = 0; r < R; ++r) vv[r] = d[2 * W + row[r]];
        f = *reinterpret_cast<const float4*>(d + 2 * W + ROWS);   // decay, beta, k . q
        d += TOK;
      };
      fetch();
#pragma unroll 2
      for (int j = 0; j < n; ++j) {
        V k0[E / PW];
        float v0[R], sk[R], sq[R];
        const float4 f0 = f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          v0[r] = vv[r];
          V a[NA] = {}, c[NA] = {};   // short chains
#pragma unroll
          for (int e = 0; e < E / PW; ++e) {
            a[e % NA] = fma_(S[r][e], kk[e], a[e % NA]);
            c[e % NA] = fma_(S[r][e], qq[e], c[e % NA]);
          }
          sk[r] = sum_(a);
          sq[r] = sum_(c);
        }
#pragma unroll
        for (int e = 0; e < E / PW; ++e) k0[e] = kk[e];
        if (j + 1 < n) fetch();
#pragma unroll
        for (int r = 0; r < R; ++r) {
          sk[r] = sum_lanes<L>(sk[r]);
          sq[r] = sum_lanes<L>(sq[r]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float u = f0.y * (v0[r] - f0.x * sk[r]);
          V uu, decay;
          all_(uu, u);
          all_(decay, f0.x);
#pragma unroll
          for (int e = 0; e < E / PW; ++e) S[r][e] = fma_(uu, k0[e], mul_(decay, S[r][e]));
          if (mine[r]) op[32 / L * r] = from_f<T>(p.scale * fmaf(u, f0.z, f0.x * sq[r]));
        }
        op += p.lay.out.token;
      }
    }
    __syncthreads();
  }
  if (warp < kRecWarps && p.S_final) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < E; e += PW) {
        float s[PW];
        if constexpr (PW == 2) unpack2(S[r][e / 2], s[0], s[1]);
        else s[0] = S[r][e];
#pragma unroll
        for (int i = 0; i < PW; ++i) {
          const int c = elem<L>(l, e + i);
          if (row0 + row[r] < p.dv && c < p.dk)
            p.S_final[sbase + (long long)(row0 + row[r]) * p.dk + c] = s[i];
        }
      }
  }
}

template <typename T, int L, int E, int R, int TT>
int launch_recurrent(const DeltaArgs& a, RecParams p) {
  constexpr int ROWS = kRecWarps * (32 / L) * R;
  constexpr int smem = 2 * TT * (2 * L * E + ROWS + 4) * 4;
  auto kern = delta_recurrent_kernel<T, L, E, R, TT>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TTT_ERR_CUDA;
  p.row_tiles = (a.dv + ROWS - 1) / ROWS;
  const long long grid = (long long)a.n_seq * a.Hv * p.row_tiles;
  const double tok = (double)a.B * a.N;
  ProfScope ps(PT_DELTA_RECURRENT, a.stream, 7.0 * tok * a.Hv * a.dk * a.dv,
               tok * (a.bf16 ? 2 : 4) * 2.0 * (a.Hk * a.dk + a.Hv * a.dv));
  return launch_behind(kern, (unsigned)grid, 256, smem, a.stream, p) == cudaSuccess ? TTT_OK
                                                                                    : TTT_ERR_CUDA;
}

template <typename T>
int recurrent_t(const DeltaArgs& a, const RecParams& p) {
  if (a.dk <= 32) return launch_recurrent<T, 8, 4, 1, 16>(a, p);
  if (a.dk <= 64) return launch_recurrent<T, 8, 8, 1, 16>(a, p);
  if (a.dk <= 128) return launch_recurrent<T, 8, 16, 1, 16>(a, p);
  if (a.dk <= 256) return launch_recurrent<T, 16, 16, 2, 8>(a, p);
  return launch_recurrent<T, 32, 16, 4, 8>(a, p);
}

// ------------------------------------------------------------ single tokens
struct StepParams {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  float* state;
  const int* slots;
  void* out;
  int* status;
  int n_slots, Hk, Hv, dk, dv, row_tiles;
  float scale;
  delta_rule_layout lay;
};

constexpr int kStepThreads = 128;

// One CTA: 4 (32 / L) R rows of one (row of the batch, head).  The state is
// read and written once, each thread's R E elements all in flight together; the
// bound is HBM (the states' bytes twice).  Heads of 128 x 128: 256 rows of 32
// heads 163 us (6.6 TB/s, 99% of a measured copy), 56 rows of 16 heads 20.4 us
// (5.8 TB/s: beginning and end are a part of it), one row of 4 heads 4 us.
// R: 128 bytes in flight a thread and more (at d_k 128 R = 1 took 177 us, 4 167; at 64
// one row 115 us for 512 rows of 32 heads, two 89, four 84; at 32 one 53, two 35, four
// 41; at 256 and 512 one row 177 and 178 us, two 164).
template <typename T, int L, int E, int R, bool VEC>
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(
    const __grid_constant__ StepParams p) {
  constexpr int ROWS = (kStepThreads / L) * R;
  pdl_launch_dependents();
  pdl_wait();
  const int tile = blockIdx.x % p.row_tiles;
  const int bh = blockIdx.x / p.row_tiles;
  const int h = bh % p.Hv, b = bh / p.Hv;
  const int hk = h / (p.Hv / p.Hk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % L;
  const int row0 = tile * ROWS;
  T* out = static_cast<T*>(p.out) + b * p.lay.out.batch + h * p.lay.out.head;
  int slot = b;
  bool live = true;
  if (p.slots) {
    slot = p.slots[b];
    bool taken = slot >= p.n_slots;
    for (int i = threadIdx.x; i < b; i += kStepThreads) taken |= p.slots[i] == slot;
    const bool bad = __syncthreads_or(taken) && slot >= 0;
    if (bad && threadIdx.x == 0) report_status(p.status, kStatusArg);
    live = slot >= 0 && !bad;
  }
  if (!live) {
    for (int r = threadIdx.x; r < ROWS; r += kStepThreads)
      if (row0 + r < p.dv) out[row0 + r] = from_f<T>(0.f);
    return;
  }
  float* S = p.state + ((long long)slot * p.Hv + h) * p.dv * p.dk;
  const T* q = static_cast<const T*>(p.q) + b * p.lay.q.batch + hk * p.lay.q.head;
  const T* k = static_cast<const T*>(p.k) + b * p.lay.k.batch + hk * p.lay.k.head;
  const T* v = static_cast<const T*>(p.v) + b * p.lay.v.batch + h * p.lay.v.head;
  float s[R][E];
  int row[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    row[r] = row0 + (warp * R + r) * (32 / L) + lane / L;
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const int c = elem<L>(l, e);
      const float* src = S + (long long)row[r] * p.dk + c;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row[r] < p.dv) {
        if (VEC) {
          if (c < p.dk) x = __ldcs(reinterpret_cast<const float4*>(src));
        } else {
          if (c < p.dk) x.x = src[0];
          if (c + 1 < p.dk) x.y = src[1];
          if (c + 2 < p.dk) x.z = src[2];
          if (c + 3 < p.dk) x.w = src[3];
        }
      }
      s[r][e] = x.x; s[r][e + 1] = x.y; s[r][e + 2] = x.z; s[r][e + 3] = x.w;
    }
  }
  float kk[E], qq[E], vv[R], kq = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = elem<L>(l, e);
    kk[e] = c < p.dk ? to_f<T>(k[c]) : 0.f;
    qq[e] = c < p.dk ? to_f<T>(q[c]) : 0.f;
    kq = fmaf(kk[e], qq[e], kq);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) vv[r] = row[r] < p.dv ? to_f<T>(v[row[r]]) : 0.f;
  const float a = expf(p.g[b * p.lay.g.batch + h * p.lay.g.head]);
  const float be = p.beta[b * p.lay.beta.batch + h * p.lay.beta.head];
  kq = sum_lanes<L>(kq);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float sk = 0.f, sq = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      sk = fmaf(s[r][e], kk[e], sk);
      sq = fmaf(s[r][e], qq[e], sq);
    }
    sk = sum_lanes<L>(sk);
    sq = sum_lanes<L>(sq);
    const float u = be * (vv[r] - a * sk);
    if (row[r] >= p.dv) continue;
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const int c = elem<L>(l, e);
      float* dst = S + (long long)row[r] * p.dk + c;
      float4 x;
      x.x = fmaf(u, kk[e], a * s[r][e]);
      x.y = fmaf(u, kk[e + 1], a * s[r][e + 1]);
      x.z = fmaf(u, kk[e + 2], a * s[r][e + 2]);
      x.w = fmaf(u, kk[e + 3], a * s[r][e + 3]);
      if (VEC) {
        if (c < p.dk) __stcs(reinterpret_cast<float4*>(dst), x);
      } else {
        if (c < p.dk) dst[0] = x.x;
        if (c + 1 < p.dk) dst[1] = x.y;
        if (c + 2 < p.dk) dst[2] = x.z;
        if (c + 3 < p.dk) dst[3] = x.w;
      }
    }
    if (l == 0) out[row[r]] = from_f<T>(p.scale * fmaf(u, kq, a * sq));
  }
}

template <typename T, int L, int E, int R, bool VEC>
int launch_step(const DeltaStepArgs& a, StepParams p) {
  constexpr int ROWS = (kStepThreads / L) * R;
  p.row_tiles = (a.dv + ROWS - 1) / ROWS;
  const double heads = (double)a.B * a.Hv;
  ProfScope ps(PT_DELTA_STEP, a.stream, 7.0 * heads * a.dk * a.dv, 8.0 * heads * a.dk * a.dv);
  return launch_behind(delta_step_kernel<T, L, E, R, VEC>, (unsigned)(a.B * a.Hv * p.row_tiles),
                       kStepThreads, 0, a.stream, p) == cudaSuccess
             ? TTT_OK
             : TTT_ERR_CUDA;
}

template <typename T, bool VEC>
int step_t(const DeltaStepArgs& a, const StepParams& p) {
  if (a.dk <= 32) return launch_step<T, 8, 4, 2, VEC>(a, p);
  if (a.dk <= 64) return launch_step<T, 8, 8, 4, VEC>(a, p);
  if (a.dk <= 128) return launch_step<T, 8, 16, 2, VEC>(a, p);
  if (a.dk <= 256) return launch_step<T, 16, 16, 2, VEC>(a, p);
  return launch_step<T, 32, 16, 2, VEC>(a, p);
}

}  // namespace

int delta_rule_recurrent(const DeltaArgs& a) {
  RecParams p{};
  p.q = a.q; p.k = a.k; p.v = a.v; p.g = a.g; p.beta = a.beta; p.S0 = a.S0;
  p.starts = a.seq_starts;
  p.out = a.out;
  p.S_final = a.S_final;
  p.status = a.status;
  p.Hk = a.Hk; p.Hv = a.Hv; p.N = a.N; p.dk = a.dk; p.dv = a.dv;
  p.scale = a.scale;
  p.lay = a.lay;
  return a.bf16 ? recurrent_t<__nv_bfloat16>(a, p) : recurrent_t<float>(a, p);
}

int delta_rule_step_launch(const DeltaStepArgs& a) {
  StepParams p{};
  p.q = a.q; p.k = a.k; p.v = a.v; p.g = a.g; p.beta = a.beta;
  p.state = a.state;
  p.slots = a.slots;
  p.out = a.out;
  p.status = a.status;
  p.n_slots = a.n_slots; p.Hk = a.Hk; p.Hv = a.Hv; p.dk = a.dk; p.dv = a.dv;
  p.scale = a.scale;
  p.lay = a.lay;
  const bool vec = a.dk % 4 == 0;
  if (a.bf16)
    return vec ? step_t<__nv_bfloat16, true>(a, p) : step_t<__nv_bfloat16, false>(a, p);
  return vec ? step_t<float, true>(a, p) : step_t<float, false>(a, p);
}

}  // namespace ttt
