// Device helpers of the fixed-state mixers: packed sequences on the token axis
// and slots of a pool.
#pragma once

#include "common.cuh"
#include "delta_tc.cuh"

namespace ttt {

constexpr int kStatusBadArg = -8;  // TTT_ERR_ARG

// The sequence of one token.
struct TokenSeq {
  int seq, t0, t1;   // seq -1: the token is in none
};

// Sequence of token t of batch b.  Any content of `starts` gives a sequence that
// holds t within [0, N), or none.
__device__ __forceinline__ TokenSeq token_seq(const int* starts, int n_seq, int b, int N, int t) {
  TokenSeq r;
  if (!starts) {
    r.seq = b;
    r.t0 = 0;
    r.t1 = N;
    return r;
  }
  int lo = 0, hi = n_seq;   // the last entry that is not behind t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= t) lo = mid;
    else hi = mid;
  }
  r.seq = lo;
  r.t0 = starts[lo];
  r.t1 = starts[lo + 1];
  if (r.t0 < 0 || r.t0 > t || r.t1 <= t || r.t1 > N) r.seq = -1;
  return r;
}

// By all threads of one block: reports entries that do not ascend within 0..N.
__device__ __forceinline__ void check_starts(const int* starts, int n_seq, int N, int* status) {
  bool bad = false;
  for (int i = threadIdx.x; i < n_seq; i += blockDim.x) {
    const int a = starts[i], e = starts[i + 1];
    bad |= a < 0 || e < a || e > N;
  }
  if (bad) report_status(status, kStatusBadArg);
}

// By all threads of a block: the slot of row b of a single-token call, -1 for an idle
// row, for a slot outside the pool and for one that an earlier row uses (reported).
__device__ __forceinline__ int row_slot(const int* slots, int n_slots, int b, int* status) {
  if (!slots) return b;
  const int slot = slots[b];
  bool taken = slot >= n_slots;
  if (slot >= 0)
    for (int i = threadIdx.x; i < b; i += blockDim.x) taken |= slots[i] == slot;
  const bool bad = __syncthreads_or(taken) && slot >= 0;
  if (bad && threadIdx.x == 0) report_status(status, kStatusBadArg);
  return bad ? -1 : slot;
}

// The same for rows b0 .. b0 + R - 1 of one block, in two parts: what a thread reads from the
// pool between them (of slots inside it) is on its way meanwhile.
template <int R>
__device__ __forceinline__ void read_slots(const int* slots, int b0, int B, int (&slot)[R]) {
#pragma unroll
  for (int i = 0; i < R; ++i) slot[i] = b0 + i < B ? (slots ? slots[b0 + i] : b0 + i) : -1;
}
template <int R>
__device__ __forceinline__ void drop_bad_slots(const int* slots, int n_slots, int b0, int B,
                                               int* status, int (&slot)[R]) {
  if (!slots) return;
  __shared__ unsigned taken;
  if (threadIdx.x == 0) taken = 0u;
  __syncthreads();
  unsigned bad = 0u;
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (slot[i] >= n_slots) bad |= 1u << i;
  for (int e = threadIdx.x; e < min(b0 + R - 1, B); e += blockDim.x) {
    const int other = slots[e];
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (slot[i] >= 0 && other == slot[i] && e < b0 + i) bad |= 1u << i;
  }
  if (bad) atomicOr(&taken, bad);
  __syncthreads();
  if (taken && threadIdx.x == 0) report_status(status, kStatusBadArg);
#pragma unroll
  for (int i = 0; i < R; ++i)
    if ((taken >> i) & 1) slot[i] = -1;
}

// e^x through the base-2 exponential: off by 2^-22 and |x| 2^-24 (the product's rounding).
__device__ __forceinline__ float exp_f(float x) { return ex2(x * 1.44269504088896341f); }

// 1 / x for x in [1, 2^126); 0 above.
__device__ __forceinline__ float rcp_f(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log(1 + e^x), from log1p(u) = 2 atanh(u / (2 + u)) with u = e^-|x| in (0, 1]: the series
// in s = u / (2 + u) <= 1/3 ends at s^11, whose first missing term is at most 1/9^6 / 13 =
// 1.4e-7 of the sum.  Two at a time, for the packed instructions.
__device__ __forceinline__ void softplus2(float& x0, float& x1) {
  const float u0 = exp_f(-fabsf(x0)), u1 = exp_f(-fabsf(x1));
  const F2 s = pack2(u0 * rcp_f(2.f + u0), u1 * rcp_f(2.f + u1)), t = mul2(s, s);
  auto all = [](float v) { return pack2(v, v); };
  F2 p = all(1.f / 11.f);
  p = fma2(p, t, all(1.f / 9.f));
  p = fma2(p, t, all(1.f / 7.f));
  p = fma2(p, t, all(1.f / 5.f));
  p = fma2(p, t, all(1.f / 3.f));
  p = fma2(p, t, all(1.f));
  p = mul2(p, add2(s, s));
  float y0, y1;
  unpack2(p, y0, y1);
  x0 = fmaxf(x0, 0.f) + y0;
  x1 = fmaxf(x1, 0.f) + y1;
}

// x sigmoid(x).  Where e^-x passes 2^126 (x < -87) it is 0; x = -inf gives NaN, as the
// product -inf * 0 does.
__device__ __forceinline__ float silu_f(float x) { return x * rcp_f(1.f + exp_f(-x)); }

// E neighbouring elements as they are; VEC: by one access (aligned to it).
template <typename T, int E>
struct alignas(sizeof(T) * E) Pack {
  T v[E];
};
template <typename T, int E, bool VEC>
__device__ __forceinline__ void load_pack(const T* p, int n, Pack<T, E>& v) {
  if constexpr (VEC) {
    v = *reinterpret_cast<const Pack<T, E>*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) v.v[i] = i < n ? p[i] : from_f<T>(0.f);
  }
}

// A pack as fp32 (two bf16 numbers of a word: the upper one is its own fp32 number).
template <typename T, int E>
__device__ __forceinline__ void pack_f(const Pack<T, E>& q, float (&v)[E]) {
  if constexpr (sizeof(T) == 2 && E % 2 == 0) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&q);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = to_f<T>(q.v[i]);
  }
}

// E neighbouring elements as fp32, and back; VEC: by one access (aligned to it).
template <typename T, int E, bool VEC>
__device__ __forceinline__ void load_row(const T* p, int n, float (&v)[E]) {
  if constexpr (VEC && sizeof(T) * E == 16) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const T* t = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = to_f<T>(t[i]);
  } else if constexpr (VEC && sizeof(T) * E == 8) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    const T* t = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = to_f<T>(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = i < n ? to_f<T>(p[i]) : 0.f;
  }
}
template <typename T, int E, bool VEC>
__device__ __forceinline__ void store_row(T* p, int n, const float (&v)[E]) {
  if constexpr (VEC && sizeof(T) * E == 16) {
    uint4 w;
    T* t = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int i = 0; i < E; ++i) t[i] = from_f<T>(v[i]);
    *reinterpret_cast<uint4*>(p) = w;
  } else if constexpr (VEC && sizeof(T) * E == 8) {
    uint2 w;
    T* t = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int i = 0; i < E; ++i) t[i] = from_f<T>(v[i]);
    *reinterpret_cast<uint2*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < n) p[i] = from_f<T>(v[i]);
  }
}

// launch_behind (delta_tc.cuh) with a grid of several dimensions, and clusters of
// `cluster` blocks along x.
template <typename P>
cudaError_t launch_grid(void (*kern)(P), dim3 grid, unsigned block, size_t smem,
                        cudaStream_t stream, const P& params, unsigned cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, params);
}

}  // namespace ttt
