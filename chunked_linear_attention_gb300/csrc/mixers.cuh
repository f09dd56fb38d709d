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

// log(1 + e^x), from log1p(u) = 2 atanh(u / (2 + u)) with u = e^-|x| in (0, 1]: the series
// in s = u / (2 + u) <= 1/3 ends at s^15, whose first missing term is 1/9^8 / 17 = 1.4e-9
// of the sum, below half a step of fp32.
__device__ __forceinline__ float softplus_f(float x) {
  const float u = expf(-fabsf(x));
  const float s = __fdividef(u, 2.f + u), t = s * s;
  float p = 1.f / 15.f;
  p = fmaf(p, t, 1.f / 13.f);
  p = fmaf(p, t, 1.f / 11.f);
  p = fmaf(p, t, 1.f / 9.f);
  p = fmaf(p, t, 1.f / 7.f);
  p = fmaf(p, t, 1.f / 5.f);
  p = fmaf(p, t, 1.f / 3.f);
  p = fmaf(p, t, 1.f);
  return fmaxf(x, 0.f) + 2.f * s * p;
}

// x sigmoid(x).  Where e^-x passes 2^126 (x < -87) the fast quotient is 0; x = -inf gives
// NaN, as the product -inf * 0 does.
__device__ __forceinline__ float silu_f(float x) { return __fdividef(x, 1.f + expf(-x)); }

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
