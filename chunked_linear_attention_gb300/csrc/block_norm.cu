// The norms around a block (block_norm_forward) in one pass over each row.
//
//   n = y / sqrt(mean_group(y^2) + eps) w;  r = residual + scale n act(gate);
//   h = r / sqrt(mean_row(r^2) + eps) w_next
//
// One CTA per row; a thread owns VPT pieces of VEC neighbouring elements, keeps
// them in registers as fp32 between the two means and the stores, so every
// tensor moves once and the kernel is bound by HBM.  A group's mean: the
// squares are summed within a piece, by a butterfly over the P lanes that the
// group's pieces fill in whole (P = the largest power of two that divides the
// group's pieces, at most 32), and the group's few remaining partial sums
// through shared memory, always in the same order.
#include "common.cuh"
#include "delta_rule.h"
#include "prof.h"

namespace ttt {

namespace {

struct NormParams {
  const void* y;
  const float* w;
  const void* gate;
  const void* residual;
  const float* scale;
  const float* w_next;
  void* out;
  void* h;
  int D, group, act;
  int pieces;        // D / VEC
  int gpieces;       // group / VEC
  int P;             // lanes of a group's butterfly
  float eps;
  block_norm_strides st;
};

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[VEC]) {
  if constexpr (VEC == 8 && sizeof(T) == 2) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  } else if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 f = __ldcs(reinterpret_cast<const float4*>(p) + i);
      x[4 * i] = f.x; x[4 * i + 1] = f.y; x[4 * i + 2] = f.z; x[4 * i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = to_f<T>(p[i]);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[VEC]) {
  if constexpr (VEC == 8 && sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 r = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  } else if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __stcs(reinterpret_cast<float4*>(p) + i,
             make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = from_f<T>(x[i]);
  }
}

// Weights: read by every row, so kept in the caches.
template <int VEC>
__device__ __forceinline__ void load_w(const float* p, float (&x)[VEC]) {
  if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
      x[4 * i] = f.x; x[4 * i + 1] = f.y; x[4 * i + 2] = f.z; x[4 * i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = __ldg(p + i);
  }
}

template <typename T, typename TS, int VEC, int VPT>
__global__ void __launch_bounds__(1024) block_norm_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ float part[];   // [pieces / P] group partials, then [32] row partials
  const long long row = blockIdx.x;
  const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31;
  const T* y = static_cast<const T*>(p.y) + row * p.st.y;
  const T* z = static_cast<const T*>(p.gate) + row * p.st.gate;
  const TS* x = static_cast<const TS*>(p.residual) + row * p.st.residual;
  float m[VPT][VEC], gate[VPT][VEC], res[VPT][VEC];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * nt + tid) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) m[i][j] = gate[i][j] = res[i][j] = 0.f;
    if (c < p.D) {
      load_vec<T, VEC>(y + c, m[i]);
      if (p.act) load_vec<T, VEC>(z + c, gate[i]);
      if (p.residual) load_vec<TS, VEC>(x + c, res[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VEC; ++j) ss = fmaf(m[i][j], m[i][j], ss);
    for (int o = p.P >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const int piece = i * nt + tid;
    if (piece < p.pieces && (piece & (p.P - 1)) == 0) part[piece / p.P] = ss;
  }
  __syncthreads();
  const int per = p.gpieces / p.P;   // partials of a group
  float rr = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int piece = i * nt + tid, c = piece * VEC;
    if (c < p.D) {
      const int grp = piece / p.gpieces;
      float ss = 0.f;
      for (int j = 0; j < per; ++j) ss += part[grp * per + j];
      const float inv = rsqrtf(ss / (float)p.group + p.eps);
      float w[VEC];
      if (p.w) {
        load_w<VEC>(p.w + (c - grp * p.group), w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) m[i][j] *= inv * w[j];
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) m[i][j] *= inv;
      }
      if (p.act) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float sg = sigmoid_precise(gate[i][j]);
          m[i][j] *= p.act == BLOCK_GATE_SILU ? gate[i][j] * sg : sg;
        }
      }
      if (p.scale) {
        load_w<VEC>(p.scale + c, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) m[i][j] *= w[j];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        m[i][j] += res[i][j];
        rr = fmaf(m[i][j], m[i][j], rr);
      }
      store_vec<TS, VEC>(static_cast<TS*>(p.out) + row * p.st.out + c, m[i]);
    }
  }
  if (!p.w_next) return;
  float* rpart = part + p.pieces / p.P;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) rr += __shfl_xor_sync(0xffffffffu, rr, o);
  if (lane == 0) rpart[warp] = rr;
  __syncthreads();
  float tot = 0.f;
  for (int j = 0; j < (nt >> 5); ++j) tot += rpart[j];
  const float inv = rsqrtf(tot / (float)p.D + p.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * nt + tid) * VEC;
    if (c < p.D) {
      float w[VEC];
      load_w<VEC>(p.w_next + c, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) m[i][j] *= inv * w[j];
      store_vec<T, VEC>(static_cast<T*>(p.h) + row * p.st.h + c, m[i]);
    }
  }
}

template <typename T, typename TS, int VEC, int VPT>
int launch_norm(const BlockNormArgs& a, NormParams p) {
  p.pieces = a.D / VEC;
  p.gpieces = a.group / VEC;
  p.P = 1;
  while (p.P < 32 && p.gpieces % (2 * p.P) == 0) p.P *= 2;
  const int nt = ((p.pieces + VPT - 1) / VPT + 31) / 32 * 32;
  const int smem = (p.pieces / p.P + 32) * 4;
  auto kern = block_norm_kernel<T, TS, VEC, VPT>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TTT_ERR_CUDA;
  const double n = (double)a.rows * a.D;
  ProfScope ps(PT_BLOCK_NORM, a.stream, 0.0,
               n * (sizeof(T) * (1 + (a.gate ? 1 : 0) + (a.h ? 1 : 0)) +
                    sizeof(TS) * (1 + (a.residual ? 1 : 0))));
  kern<<<(unsigned)a.rows, nt, smem, a.stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

template <typename T, typename TS>
int norm_t(const BlockNormArgs& a, const NormParams& p) {
  auto al = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  const bool wide = a.D % 8 == 0 && a.group % 8 == 0 && al(a.y) && al(a.w) && al(a.gate) &&
                    al(a.residual) && al(a.scale) && al(a.w_next) && al(a.out) && al(a.h) &&
                    a.st.y % 8 == 0 && a.st.gate % 8 == 0 && a.st.residual % 8 == 0 &&
                    a.st.out % 8 == 0 && a.st.h % 8 == 0;
  if (wide) {
    if (a.D <= 8192) return launch_norm<T, TS, 8, 1>(a, p);
    return launch_norm<T, TS, 8, 2>(a, p);
  }
  if (a.D <= 1024) return launch_norm<T, TS, 1, 1>(a, p);
  if (a.D <= 4096) return launch_norm<T, TS, 1, 4>(a, p);
  return launch_norm<T, TS, 1, 16>(a, p);
}

}  // namespace

int block_norm_launch(const BlockNormArgs& a) {
  NormParams p{};
  p.y = a.y; p.w = a.w; p.gate = a.gate; p.residual = a.residual;
  p.scale = a.scale; p.w_next = a.w_next; p.out = a.out; p.h = a.h;
  p.D = a.D; p.group = a.group; p.act = a.act; p.eps = a.eps;
  p.st = a.st;
  using B = __nv_bfloat16;
  if (a.io_bf16) return a.stream_bf16 ? norm_t<B, B>(a, p) : norm_t<B, float>(a, p);
  return a.stream_bf16 ? norm_t<float, B>(a, p) : norm_t<float, float>(a, p);
}

}  // namespace ttt
