// The norms around a block (block_norm_forward) in one pass over each row.
//
//   n = y / sqrt(mean_group(y^2) + eps) w;  r = residual + scale n act(gate);
//   h = r / sqrt(mean_row(r^2) + eps) w_next
//
// A thread owns VPT pieces of VEC neighbouring elements, the same ones in every
// row that its CTA takes, so the weights are read once; the next row's loads are
// issued before the present row's arithmetic.  A row stays in registers as fp32
// between the two means and the stores: every tensor moves once, and the bound is
// HBM.  A group's mean: the squares are summed within a piece, by a butterfly over
// the P lanes that the group's pieces fill in whole (P = the largest power of two
// that divides the group's pieces, at most 32), and the group's few remaining
// partial sums through shared memory, always in the same order.
//
// Measured: 65536 rows of 1536 with four gated groups, bf16, 101 us (6.0 TB/s, 89%
// of a measured copy; one row per CTA, with the weights read anew for each, took
// 197: its instructions, and not HBM, were the bound); 20011 rows of 1536 with gate,
// fp32 residual and both norms 67 us (6.4 TB/s); a single row 4 us.  Longer rows
// reach 3.7 to 4.9 TB/s (fewer CTAs per SM to run past each other's barriers), ones
// of unaligned length 1.2 to 1.7 (an element per access, and issue is the bound).
#include <atomic>

#include "delta_tc.cuh"
#include "prof.h"

namespace ttt {

namespace {

// Threads of a CTA, at most: 256 for rows of up to 2048 elements, a piece per thread
// (three CTAs per SM and their loads in flight); 768 for longer ones, 512 with two
// pieces or (unaligned rows of up to 2048) four elements each; 1024 where a thread
// cannot hold the weights and the next row.
template <int VEC, int VPT, int PARTS, bool KEEP>
constexpr int kMaxThreads = !KEEP ? 1024 : VEC == 1 || VPT > 1 ? 512 : PARTS >= 0 ? 256 : 768;
// CTAs per SM to leave registers for: four where at most gate or residual is there
// besides y, all bf16 (four gated groups of 1536: 103 us, with three 112).
template <int PARTS, int BYTES>
constexpr int kMinCtas = PARTS < 0                                             ? 1
                         : BYTES == 4 && (PARTS == 0 || PARTS == 2 || PARTS == 4) ? 4
                                                                               : 3;

// Partial sums of a group up to which every thread adds them up for itself; of more
// a warp makes one first (21816 rows of 1538 in two groups 366 us; rows of 1537 whose
// partial sums every thread added up took 6.1 ms).
constexpr int kFew = 16;

struct NormParams {
  const void* y;
  const float* w;
  const void* gate;
  const void* residual;
  const float* scale;
  const float* w_next;
  void* out;
  void* h;
  long long rows;
  int D, group, act;
  int pieces;        // D / VEC
  int gpieces;       // group / VEC
  int P;             // lanes of a group's butterfly
  int nt;            // threads per row
  int np;            // places of the groups' partial sums
  float eps;
  block_norm_strides st;
};

// VEC elements as they are loaded.
template <typename T, int VEC>
struct Raw {
  T x[VEC];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = p[i];
  }
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = to_f<T>(x[i]);
  }
};
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<float, 8> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

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

// A weight's elements, or ones.
template <int VEC>
__device__ __forceinline__ void load_w(const float* p, bool there, float (&x)[VEC]) {
  if (!there) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = 1.f;
  } else if constexpr (VEC == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 f = reinterpret_cast<const float4*>(p)[i];
      x[4 * i] = f.x; x[4 * i + 1] = f.y; x[4 * i + 2] = f.z; x[4 * i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = p[i];
  }
}

// sigmoid(x) from the hardware exponential and reciprocal (2^-22 each; the
// exponent's own rounding adds |x| 2^-24): the exact division would cost more
// than the loads.  Saturates to 0 and 1.
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sigmoid_fast(float x) {
  return rcp_fast(1.f + ex2(x * -1.4426950408889634f));
}

// A piece's arithmetic; PACK: eight numbers, two at a time by the packed instructions
// (65536 rows of 1536, gated groups: 102.6 -> 100.8 us; kernels short of registers lose by
// it, 6710 rows of 5000 167 -> 190).
template <bool PACK, int VEC>
__device__ __forceinline__ float sum_squares(const float (&m)[VEC], float s) {
  if constexpr (PACK) {
    F2 a = pack2(s, 0.f);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const F2 x = pack2(m[j], m[j + 1]);
      a = fma2(x, x, a);
    }
    float x, y;
    unpack2(a, x, y);
    return x + y;
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) s = fmaf(m[j], m[j], s);
    return s;
  }
}
// m *= c w
template <bool PACK, int VEC>
__device__ __forceinline__ void scale_by(float (&m)[VEC], float c, const float (&w)[VEC]) {
  if constexpr (PACK) {
#pragma unroll
    for (int j = 0; j < 8; j += 2)
      unpack2(mul2(pack2(m[j], m[j + 1]), mul2(pack2(c, c), pack2(w[j], w[j + 1]))), m[j], m[j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) m[j] *= c * w[j];
  }
}
// m *= sigmoid(z), or z sigmoid(z)
template <bool PACK, int VEC>
__device__ __forceinline__ void gate_by(float (&m)[VEC], const float (&z)[VEC], bool silu) {
  if constexpr (PACK) {
    constexpr float kC = -1.4426950408889634f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const F2 zz = pack2(z[j], z[j + 1]);
      float a, b;
      unpack2(mul2(zz, pack2(kC, kC)), a, b);
      unpack2(add2(pack2(ex2(a), ex2(b)), pack2(1.f, 1.f)), a, b);
      F2 g = pack2(rcp_fast(a), rcp_fast(b));
      if (silu) g = mul2(g, zz);
      unpack2(mul2(pack2(m[j], m[j + 1]), g), m[j], m[j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) m[j] *= silu ? z[j] * sigmoid_fast(z[j]) : sigmoid_fast(z[j]);
  }
}

// PARTS: which of gate (4), residual (2) and next norm (1) are there; -1: the
// call says (wide or unaligned rows, which need no variant for each).
template <typename T, typename TS, int VEC, int VPT, int PARTS, bool KEEP>
__global__ void __launch_bounds__(kMaxThreads<VEC, VPT, PARTS, KEEP>, kMinCtas<PARTS, sizeof(T) + sizeof(TS)>)
    block_norm_kernel(const __grid_constant__ NormParams p) {
  const bool GATE = PARTS < 0 ? p.gate != nullptr : (PARTS & 4) != 0;
  const bool RES = PARTS < 0 ? p.residual != nullptr : (PARTS & 2) != 0;
  const bool NEXT = PARTS < 0 ? p.h != nullptr : (PARTS & 1) != 0;
  // for each row of the CTA: [2][pieces / P] group partials, [2][nt / 32] row partials
  extern __shared__ float smem[];
  pdl_launch_dependents();
  pdl_wait();
  const int ty = threadIdx.x / p.nt, tid = threadIdx.x - ty * p.nt, ny = blockDim.x / p.nt;
  const int warp = tid >> 5, lane = tid & 31, nw = p.nt >> 5, np = p.np;
  float* part = smem + ty * 2 * (np + nw);
  float* rpart = part + 2 * np;
  constexpr bool PACK = VEC == 8 && PARTS >= 0;
  // one group: each warp makes a partial sum, whatever the group's length
  const bool one = PARTS < 0 && p.gpieces == p.pieces;
  const int per = one ? nw : p.gpieces / p.P;   // partials of a group
  const bool many = PARTS < 0 && !one && per > kFew;
  const float inv_g = 1.f / (float)p.group, inv_d = 1.f / (float)p.D;
  // Piece i of this thread: its first column, that in its group, its group's first
  // partial sum, and the partial sum that it writes itself (or -1).
  struct Piece {
    int col, wcol, first, slot;
  };
  int me = tid;
  auto place = [&](int i) {
    const int piece = i * p.nt + me, grp = piece / p.gpieces;
    Piece c;
    c.col = piece * VEC;
    c.wcol = c.col - grp * p.group;
    c.first = grp * per;
    c.slot = piece < p.pieces && piece % p.P == 0 ? piece / p.P : -1;
    return c;
  };
  auto weights = [&](const Piece& c, float (&x)[VEC]) {
    const bool in = c.col < p.D;
    float a[VEC];
    load_w<VEC>(p.w + c.wcol, in && p.w, x);
    load_w<VEC>(p.scale + c.col, in && p.scale, a);
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] *= a[j];
  };
  // Weights are read once, and the next row ahead, where the registers hold both;
  // else the weights come from the caches row by row, gate and residual G pieces at
  // a time when they are needed, and the CTA's many threads hide the loads (all of
  // it held, 700 bytes a thread were spilled).
  constexpr int G = KEEP ? VPT : VEC == 1 ? 4 : 1;
  static_assert(VPT % G == 0, "whole groups");
  float w[KEEP ? VPT : 1][VEC], wn[KEEP ? VPT : 1][VEC];   // w: times the residual scale
  Piece held[KEEP ? VPT : 1] = {};
  auto at = [&](int i) { return KEEP ? held[KEEP ? i : 0] : place(i); };
  auto col = [&](int i) { return KEEP ? held[KEEP ? i : 0].col : (i * p.nt + me) * VEC; };
  if (KEEP) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      held[KEEP ? i : 0] = place(i);
      weights(held[KEEP ? i : 0], w[KEEP ? i : 0]);
      if (NEXT) load_w<VEC>(p.w_next + col(i), col(i) < p.D, wn[KEEP ? i : 0]);
    }
  }
  // rows move by whole CTAs: pointers advance, nothing is multiplied per row (short
  // of registers: multiplied)
  long long row = (long long)blockIdx.x * ny + ty;
  const long long step = (long long)gridDim.x * ny;
  const T *py, *pz;
  const TS* px;
  TS* po;
  T* ph;
  auto point = [&]() {
    py = static_cast<const T*>(p.y) + row * p.st.y;
    pz = static_cast<const T*>(p.gate) + row * p.st.gate;
    px = static_cast<const TS*>(p.residual) + row * p.st.residual;
    po = static_cast<TS*>(p.out) + row * p.st.out;
    ph = static_cast<T*>(p.h) + row * p.st.h;
  };
  point();
  const long long sy = step * p.st.y, sz = step * p.st.gate, sx = step * p.st.residual;
  const long long so = step * p.st.out, shh = step * p.st.h;
  Raw<T, VEC> ry[VPT], rz[G];
  Raw<TS, VEC> rx[G];
  auto load_y = [&]() {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (col(i) < p.D) ry[i].load(py + col(i));
  };
  auto load_zx = [&](int i0) {
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (col(i0 + i) < p.D) {
        if (GATE) rz[i].load(pz + col(i0 + i));
        if (RES) rx[i].load(px + col(i0 + i));
      }
  };
  auto load = [&]() {
    load_y();
    load_zx(0);
    py += sy;
    if (GATE) pz += sz;
    if (RES) px += sx;
  };
  if (KEEP && row < p.rows) load();
  int buf = 0;
  for (long long r0 = (long long)blockIdx.x * ny; r0 < p.rows; r0 += step, row += step, buf ^= 1) {
    const bool live = row < p.rows;   // the CTA's rows meet at its barriers
    float m[VPT][VEC], z[G][VEC], x[G][VEC];
    if (!KEEP) {
      asm volatile("" : "+r"(me));   // places and pointers anew in each row: no room to hold them
      point();
      if (live) load_y();
    }
    auto get_zx = [&]() {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        if (GATE) rz[i].get(z[i]);
        if (RES) rx[i].get(x[i]);
      }
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) ry[i].get(m[i]);
    if (KEEP) get_zx();
    if (KEEP && row + step < p.rows) load();
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float ss = sum_squares<PACK>(m[i], 0.f);
      if (one) {
        all += col(i) < p.D ? ss : 0.f;
        continue;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < p.P) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const int slot = at(i).slot;
      if (slot >= 0) part[buf * np + slot] = ss;
    }
    if (one) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      if (lane == 0) part[buf * np + warp] = all;
    }
    __syncthreads();
    if (many) {   // a warp per group; its sum takes the place of its first partial
      for (int g = warp; g * p.gpieces < p.pieces; g += nw) {
        float* q = part + buf * np + g * per;
        float s4[4] = {0.f, 0.f, 0.f, 0.f};   // of at most 16384 terms, 128 each
        for (int j = lane; j < per; j += 128) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j + 32 * e < per) s4[e] += q[j + 32 * e];
        }
        float ss = (s4[0] + s4[1]) + (s4[2] + s4[3]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        __syncwarp();
        if (lane == 0) q[0] = ss;
      }
      __syncthreads();
    }
    float rr = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (!live) continue;
      if (!KEEP && i % G == 0) {
        load_zx(i);
        get_zx();
      }
      const Piece c = at(i);
      if (c.col >= p.D) continue;
      float ss = 0.f;
      for (int j = 0; j < (many ? 1 : per); ++j) ss += part[buf * np + c.first + j];
      const float inv = rsqrtf(fmaf(ss, inv_g, p.eps));
      float f[VEC];
      if (KEEP) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] = w[KEEP ? i : 0][j];
      } else {
        weights(c, f);
      }
      scale_by<PACK>(m[i], inv, f);
      if (GATE) {
        if (p.act == BLOCK_GATE_SILU) gate_by<PACK>(m[i], z[i % G], true);
        else gate_by<PACK>(m[i], z[i % G], false);
      }
      if (RES) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) m[i][j] += x[i % G][j];
      }
      if (NEXT) rr = sum_squares<PACK>(m[i], rr);
      store_vec<TS, VEC>(po + c.col, m[i]);
    }
    if (KEEP) po += so;
    if (NEXT) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) rr += __shfl_xor_sync(0xffffffffu, rr, o);
      if (lane == 0) rpart[buf * nw + warp] = rr;
      __syncthreads();
      float tot = 0.f;
      for (int j = 0; j < nw; ++j) tot += rpart[buf * nw + j];
      const float inv = rsqrtf(fmaf(tot, inv_d, p.eps));
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (!live || col(i) >= p.D) continue;
        float f[VEC];
        if (KEEP) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) f[j] = wn[KEEP ? i : 0][j];
        } else {
          load_w<VEC>(p.w_next + col(i), true, f);
        }
        scale_by<PACK>(m[i], inv, f);
        store_vec<T, VEC>(ph + col(i), m[i]);
      }
      if (KEEP) ph += shh;
    }
  }
}

template <typename T, typename TS, int VEC, int VPT, int PARTS, bool KEEP>
int launch_parts(const BlockNormArgs& a, NormParams p) {
  auto kern = block_norm_kernel<T, TS, VEC, VPT, PARTS, KEEP>;
  static std::atomic<int> known{0};   // the kernel's registers, once a call has found them
  int regs = known.load(std::memory_order_relaxed);
  if (regs == 0) {
    cudaFuncAttributes at;
    if (cudaFuncGetAttributes(&at, kern) != cudaSuccess) return TTT_ERR_CUDA;
    regs = at.numRegs;
    known.store(regs, std::memory_order_relaxed);
  }
  p.pieces = a.D / VEC;
  p.gpieces = a.group / VEC;
  p.P = 1;
  while (p.P < 32 && p.gpieces % (2 * p.P) == 0) p.P *= 2;
  p.nt = ((p.pieces + VPT - 1) / VPT + 31) / 32 * 32;
  // rows per CTA: up to 256 threads; CTAs: what the SMs hold of them at once, so
  // that all run to the end together
  const int ny = p.nt >= 256 ? 1 : 256 / p.nt, threads = p.nt * ny;
  p.np = PARTS < 0 && p.gpieces == p.pieces ? p.nt / 32 : p.pieces / p.P;
  const int smem = ny * 2 * (p.np + p.nt / 32) * 4;
  // always the limit of the longest rows (of unaligned groups, a partial sum an element):
  // one call's own size could be below what another host thread is about to launch with
  constexpr int kMostSmem = 2 * (16384 + 32) * 4;
  if (smem > 48 * 1024 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMostSmem) != cudaSuccess)
    return TTT_ERR_CUDA;
  int per_sm = 65536 / ((regs + 7) / 8 * 8 * threads);
  per_sm = per_sm < 1 ? 1 : per_sm > 2048 / threads ? 2048 / threads : per_sm;
  const double n = (double)a.rows * a.D;
  ProfScope ps(PT_BLOCK_NORM, a.stream, 0.0,
               n * (sizeof(T) * (1 + (a.gate ? 1 : 0) + (a.h ? 1 : 0)) +
                    sizeof(TS) * (1 + (a.residual ? 1 : 0))));
  const long long ctas = (a.rows + ny - 1) / ny, most = 152ll * per_sm;
  return launch_behind(kern, (unsigned)(ctas < most ? ctas : most), threads, smem, a.stream, p) ==
                 cudaSuccess
             ? TTT_OK
             : TTT_ERR_CUDA;
}

template <typename T, typename TS>
int launch_narrow(const BlockNormArgs& a, const NormParams& p) {
  switch ((a.gate ? 4 : 0) | (a.residual ? 2 : 0) | (a.h ? 1 : 0)) {
    case 0: return launch_parts<T, TS, 8, 1, 0, true>(a, p);
    case 1: return launch_parts<T, TS, 8, 1, 1, true>(a, p);
    case 2: return launch_parts<T, TS, 8, 1, 2, true>(a, p);
    case 3: return launch_parts<T, TS, 8, 1, 3, true>(a, p);
    case 4: return launch_parts<T, TS, 8, 1, 4, true>(a, p);
    case 5: return launch_parts<T, TS, 8, 1, 5, true>(a, p);
    case 6: return launch_parts<T, TS, 8, 1, 6, true>(a, p);
    default: return launch_parts<T, TS, 8, 1, 7, true>(a, p);
  }
}

template <typename T, typename TS>
int norm_t(const BlockNormArgs& a, const NormParams& p) {
  auto al = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  const bool wide = a.D % 8 == 0 && a.group % 8 == 0 && al(a.y) && al(a.w) && al(a.gate) &&
                    al(a.residual) && al(a.scale) && al(a.w_next) && al(a.out) && al(a.h) &&
                    a.st.y % 8 == 0 && a.st.gate % 8 == 0 && a.st.residual % 8 == 0 &&
                    a.st.out % 8 == 0 && a.st.h % 8 == 0;
  if (wide) {
    int pieces = a.group / 8;   // of a group, and of a butterfly's sum: see launch_parts
    for (int i = 0; i < 5 && pieces % 2 == 0; ++i) pieces /= 2;
    if (a.D <= 8 * 256 && pieces <= kFew) return launch_narrow<T, TS>(a, p);
    if (a.D <= 8 * 256) return launch_parts<T, TS, 8, 1, -1, true>(a, p);
    // two pieces a thread where two CTAs of them fit an SM (rows of 4096 in bf16, two
    // norms, gate and residual: 77 us for 8192 rows, 97 with one piece; of 6144, one
    // CTA, 115 against 104), and where little is held ahead
    if (a.D <= 8 * 512 || (a.D <= 8 * 1024 && sizeof(T) + sizeof(TS) == 4))
      return launch_parts<T, TS, 8, 2, -1, true>(a, p);
    if (a.D <= 8 * 768) return launch_parts<T, TS, 8, 1, -1, true>(a, p);
    return launch_parts<T, TS, 8, 2, -1, false>(a, p);
  }
  if (a.D <= 4 * 512) return launch_parts<T, TS, 1, 4, -1, true>(a, p);
  return launch_parts<T, TS, 1, 16, -1, false>(a, p);
}

}  // namespace

int block_norm_launch(const BlockNormArgs& a) {
  NormParams p{};
  p.y = a.y; p.w = a.w; p.gate = a.gate; p.residual = a.residual;
  p.scale = a.scale; p.w_next = a.w_next; p.out = a.out; p.h = a.h;
  p.rows = a.rows;
  p.D = a.D; p.group = a.group; p.act = a.act; p.eps = a.eps;
  p.st = a.st;
  using B = __nv_bfloat16;
  if (a.io_bf16) return a.stream_bf16 ? norm_t<B, B>(a, p) : norm_t<B, float>(a, p);
  return a.stream_bf16 ? norm_t<float, B>(a, p) : norm_t<float, float>(a, p);
}

}  // namespace ttt
