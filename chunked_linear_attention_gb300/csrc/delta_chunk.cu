// The gated delta rule over whole sequences on the tensor cores: chunks of 64
// tokens, d_k <= 128, 128 rows of the state per CTA.
//
// With G the running sum of g inside a chunk, D_ij = exp(G_i - G_j) (i >= j) and
// S the state before the chunk, the 64 rank-one updates of a chunk are
//     A_ij = beta_i D_ij k_i . k_j  (i > j),   T = (1 + A)^-1 diag(beta)
//     X    = T (V - e^G o K S^T)               (the corrected values)
//     O    = scale (e^G o Q S^T + (D o Q K^T) X)
//     S   <- e^{G_63} S + X^T (e^{G_63 - G} o K)
// Everything with the state is kept transposed (rows of S = TMEM lanes = d_v), so
// that S, K S^T and X are TMEM operands of the next product and never visit
// shared memory; q, k, v are used as TMA left them.
//
// Precision: inputs are bf16, but the state that a prompt leaves behind is read
// for thousands of tokens, so no intermediate is rounded to bf16.  Each is held
// as a pair hi + lo of bf16 numbers (16 bits of significand); products of a pair
// with an input take two MMAs, of two pairs three (lo lo is left out).  Sums are
// fp32 and the state itself stays in fp32 registers.
//
// Roles (640 threads, one CTA per SM, persistent over (sequence, head, d_v tile)):
//   warp 0      TMA: q, k, v of the coming chunks, three stages.
//   warp 1      all tcgen05 MMAs.
//   warp 2      the chunk's decay factors and beta; zeroes the rows behind a
//               sequence's end, so that other sequences' values cannot reach it.
//   warps 4-7   D o Q K^T and T: 16 x 16 diagonal blocks of 1 + A are inverted by
//               substitution, one per warp, and joined to 64 x 64 by products
//               T_21 = -T_22 A_21 T_11 on 16 x 16 blocks in registers (mma.sync
//               tf32, each operand as two parts, so fp32 accuracy; a tcgen05
//               product is at least 64 rows).
//   warps 8-15  the chain S -> K S^T -> X -> S.
//   warps 16-19 the outputs.
#include <cuda.h>

#include <mutex>

#include "builder.h"
#include "common.cuh"
#include "delta_rule.h"
#include "prof.h"

namespace ttt {

namespace {

constexpr int kC = 64;                  // tokens per chunk
constexpr int kThreads = 640;
constexpr int kStages = 3;
constexpr int kBlk = 8192;              // 64 rows of 64 bf16
constexpr int kStageBytes = 6 * kBlk;   // Q0 K0 Q1 K1 V0 V1 (column blocks of 64)
constexpr int kTPBytes = 4 * kBlk;      // P hi, P lo, T hi, T lo (T's first fp32 A, then T)

struct Scal {
  float eg[kC];     // exp(G_i)
  float er[kC];     // exp(G_63 - G_j)
  float beta[kC];
  float gl[kC];     // running sum of g log2(e) inside each block of 16
  float el[kC];     // exp2(blk - gl): decay from token j to the end of its block
  float blk[4];     // each block's sum of g log2(e)
  float eall;       // exp(G_63)
  float pad[3];
};

struct Bars {
  uint64_t full[kStages], ready[kStages], empty[kStages];
  uint64_t tp_ready[2], tp_free[2];
  uint64_t d1_full, d1_free, ks_full, y_ready, x_full, xs_ready, ds_full, x_ready, s_ready;
  uint64_t o_full, o_free;
  uint32_t tmem;
};

constexpr int kSmem = kStages * kStageBytes + 2 * kTPBytes + kStages * (int)sizeof(Scal) +
                      (int)sizeof(Bars) + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");

// TMEM columns
constexpr uint32_t kD1 = 0;      // 64: rows 0-63 Q K^T, rows 64-127 K K^T
constexpr uint32_t kQS = 64;     // 64: S Q^T
constexpr uint32_t kKS = 128;    // 64: S K^T, then its pair in the same columns
constexpr uint32_t kDS = 128;    // 128: X^T K (after K S^T is used up)
constexpr uint32_t kSh = 256;    // 64 + 64: S, hi and lo
constexpr uint32_t kX = 384;     // 64: X, then its pair
constexpr uint32_t kO = 448;     // 64: P X

struct ChunkParams {
  CUtensorMap q, k, v;
  const float* g;
  const float* beta;
  const float* S0;
  const int* starts;
  __nv_bfloat16* out;
  float* S_final;
  int* status;
  unsigned long long wait_ns;
  delta_rule_stride sg, sb, so;
  int Hk, Hv, N, dk, dv, tiles, items;
  float scale;
};

struct Item {
  int seq, h, tile, batch, t0, len;
};

__device__ __forceinline__ Item get_item(const ChunkParams& p, int i) {
  Item it;
  it.tile = i % p.tiles;
  const int sh = i / p.tiles;
  it.h = sh % p.Hv;
  it.seq = sh / p.Hv;
  it.batch = it.seq;
  it.t0 = 0;
  it.len = p.N;
  if (p.starts) {
    const int a = p.starts[it.seq], b = p.starts[it.seq + 1];
    const bool ok = a >= 0 && a <= b && b <= p.N;
    if (!ok) report_status(p.status, -8);
    it.batch = 0;
    it.t0 = ok ? a : 0;
    it.len = ok ? b - a : 0;
  }
  return it;
}

__device__ __forceinline__ int chunks(const Item& it) { return (it.len + kC - 1) / kC; }

// ---------------------------------------------------------------- wrappers
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// D[tmem] (+)= A[tmem] B[smem], issued by one elected lane of the warp.
__device__ __forceinline__ void umma_ts_w(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&w)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]),
      "r"(w[8]), "r"(w[9]), "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

template <int R>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// (a, b) as a pair of packed bf16 pairs: a ~ hi.x + lo.x, b ~ hi.y + lo.y, each
// off by at most 2^-17 of its value.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const float ra = a - __uint_as_float(hi << 16);
  const float rb = b - __uint_as_float(hi & 0xffff0000u);
  const __nv_bfloat162 l = __floats2bfloat162_rn(ra, rb);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- 16 x 16 blocks
// Element (i, j) of the fp32 scratch: rows of 64, groups of four neighbours
// exchanged by the row, so that rows, columns and fragments meet no bank twice.
__device__ __forceinline__ int at(int i, int j) {
  return i * 64 + ((((j >> 2) ^ i) & 15) << 2) + (j & 3);
}

struct Frag {
  uint32_t hi[4], lo[4];
};

// x = hi + lo with hi a tf32 number; lo's bits below tf32 are dropped by the MMA
// (2^-21 of x).
__device__ __forceinline__ void tf32_parts(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma3(float (&c)[4], const Frag& a, float x0, float x1) {
  uint32_t h0, l0, h1, l1;
  tf32_parts(x0, h0, l0);
  tf32_parts(x1, h1, l1);
  mma_tf32(c, a.lo, h0, h1);
  mma_tf32(c, a.hi, l0, l1);
  mma_tf32(c, a.hi, h0, h1);
}

// c[2] (a 16 x 16 block, two tiles of 8 columns) += M(i0.., k0..) M(k0.., j0..)
__device__ __forceinline__ void block_mm(float (&c)[2][4], const float* M, int i0, int k0, int j0,
                                         int g, int t) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    Frag a;
    const int k = k0 + 8 * s;
    tf32_parts(M[at(i0 + g, k + t)], a.hi[0], a.lo[0]);
    tf32_parts(M[at(i0 + g + 8, k + t)], a.hi[1], a.lo[1]);
    tf32_parts(M[at(i0 + g, k + t + 4)], a.hi[2], a.lo[2]);
    tf32_parts(M[at(i0 + g + 8, k + t + 4)], a.hi[3], a.lo[3]);
#pragma unroll
    for (int n = 0; n < 2; ++n)
      mma3(c[n], a, M[at(k + t, j0 + 8 * n + g)], M[at(k + t + 4, j0 + 8 * n + g)]);
  }
}

// c (tile n of 8 columns) += W M(k0.., j0 + 8 n..), W a block in accumulator
// form: its columns 2t and 2t + 1 take the operand's places t and t + 4.
__device__ __forceinline__ void block_wm(float (&c)[4], const float (&w)[2][4], const float* M,
                                         int k0, int j, int g, int t) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    Frag a;
    tf32_parts(w[s][0], a.hi[0], a.lo[0]);
    tf32_parts(w[s][2], a.hi[1], a.lo[1]);
    tf32_parts(w[s][1], a.hi[2], a.lo[2]);
    tf32_parts(w[s][3], a.hi[3], a.lo[3]);
    const int k = k0 + 8 * s + 2 * t;
    mma3(c, a, M[at(k, j + g)], M[at(k + 1, j + g)]);
  }
}

__device__ __forceinline__ void put_neg(float* M, const float (&c)[4], int i0, int j0, int g,
                                        int t) {
  *reinterpret_cast<float2*>(&M[at(i0 + g, j0 + 2 * t)]) = make_float2(-c[0], -c[1]);
  *reinterpret_cast<float2*>(&M[at(i0 + g + 8, j0 + 2 * t)]) = make_float2(-c[2], -c[3]);
}

// ---------------------------------------------------------------- the kernel
__global__ void __launch_bounds__(kThreads, 1)
    delta_chunk_kernel(const __grid_constant__ ChunkParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* tp = smem + kStages * kStageBytes;
  Scal* scal = reinterpret_cast<Scal*>(tp + 2 * kTPBytes);
  Bars* B = reinterpret_cast<Bars*>(scal + kStages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned long long lim = p.wait_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&B->full[s], 1);
      mbar_init(&B->ready[s], 1);
      mbar_init(&B->empty[s], 1 + 8 + 4 + 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&B->tp_ready[b], 4);
      mbar_init(&B->tp_free[b], 1);
    }
    mbar_init(&B->d1_full, 1);
    mbar_init(&B->d1_free, 4);
    mbar_init(&B->ks_full, 1);
    mbar_init(&B->y_ready, 8);
    mbar_init(&B->x_full, 1);
    mbar_init(&B->xs_ready, 8);
    mbar_init(&B->ds_full, 1);
    mbar_init(&B->x_ready, 8);
    mbar_init(&B->s_ready, 8);
    mbar_init(&B->o_full, 1);
    mbar_init(&B->o_free, 4);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&B->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem;
  bool ok = true;   // after a wait that ran out: no more waiting, run to the end
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = mbar_wait_w(bar, parity, p.status, lim);
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp < 4) {
    regs_dec<56>();
    if (warp == 0) {
      int n = 0;
      for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
        const Item it = get_item(p, i);
        const int hk = it.h / (p.Hv / p.Hk), nc = chunks(it);
        for (int c = 0; c < nc && ok; ++c, ++n) {
          const int s = n % kStages;
          wait(&B->empty[s], ((n / kStages) & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) {
            uint8_t* st = smem + s * kStageBytes;
            const int t = it.t0 + c * kC;
            mbar_arrive_expect_tx(&B->full[s], kStageBytes);
            for (int b = 0; b < 2; ++b) {
              tma_load_4d(st + (2 * b + 1) * kBlk, &p.k, 64 * b, t, hk, it.batch, &B->full[s]);
              tma_load_4d(st + 2 * b * kBlk, &p.q, 64 * b, t, hk, it.batch, &B->full[s]);
            }
            for (int b = 0; b < 2; ++b)
              tma_load_4d(st + (4 + b) * kBlk, &p.v, 128 * it.tile + 64 * b, t, it.h, it.batch,
                          &B->full[s]);
          }
          __syncwarp();
        }
      }
      if (!ok)   // copies still on their way into this CTA's shared memory
        for (int m = n > kStages ? n - kStages : 0; m < n; ++m)
          mbar_wait_w(&B->full[m % kStages], (m / kStages) & 1, p.status, lim);
    } else if (warp == 1) {
      int total = 0;
      for (int i = blockIdx.x; i < p.items; i += gridDim.x) total += chunks(get_item(p, i));
      const uint32_t base = smem_u32(smem), tpb = smem_u32(tp);
      const uint32_t id64 = idesc_bf16_f32(64, 0, 0);        // both K-major
      const uint32_t id64m = idesc_bf16_f32(64, 1, 0);       // A = V^T, MN-major
      const uint32_t id128 = idesc_bf16_f32(128, 0, 1);      // B = K^T, MN-major
      auto issue_d1 = [&](int n) {   // [Q; K] K^T
        const uint32_t st = base + (n % kStages) * kStageBytes;
        const uint64_t a = smem_desc_sw128(st, 16, 1024), b = smem_desc_sw128(st + kBlk, 16, 1024);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t o = (k >> 2) * (2 * kBlk / 16) + (k & 3) * 2;
          umma_bf16_w(tmem + kD1, a + o, b + o, id64, k != 0);
        }
        umma_commit_w(&B->d1_full);
      };
      if (total > 0) {
        wait(&B->ready[0], 0);
        tc_fence_after();
        issue_d1(0);
      }
      for (int n = 0; n < total && ok; ++n) {
        const uint32_t st = base + (n % kStages) * kStageBytes;
        const uint32_t tb = tpb + (n & 1) * kTPBytes;
        const uint32_t ph = n & 1;
        // S K^T, S Q^T
        wait(&B->s_ready, ph);
        tc_fence_after();
        const uint64_t kd = smem_desc_sw128(st + kBlk, 16, 1024);
        const uint64_t qd = smem_desc_sw128(st, 16, 1024);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          umma_ts_w(tmem + kKS, tmem + kSh + (k >> 3) * 64 + (k & 7) * 8,
                    kd + ((k >> 2) & 1) * (2 * kBlk / 16) + (k & 3) * 2, id64, k != 0);
        umma_commit_w(&B->ks_full);
        wait(&B->o_free, ph ^ 1);
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 16; ++k)
          umma_ts_w(tmem + kQS, tmem + kSh + (k >> 3) * 64 + (k & 7) * 8,
                    qd + ((k >> 2) & 1) * (2 * kBlk / 16) + (k & 3) * 2, id64, k != 0);
        // X = T V + T (-e^G K S^T)
        wait(&B->tp_ready[ph], (n >> 1) & 1);
        if (n > 0) wait(&B->o_full, ph ^ 1);   // P X of the chunk before has read X
        tc_fence_after();
        const uint64_t vd = smem_desc_sw128(st + 4 * kBlk, kBlk, 1024);
        const uint64_t th = smem_desc_sw128(tb + 2 * kBlk, 16, 1024);
        const uint64_t tl = smem_desc_sw128(tb + 3 * kBlk, 16, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          umma_bf16_w(tmem + kX, vd + k * 128, tl + k * 2, id64m, k != 0);
          umma_bf16_w(tmem + kX, vd + k * 128, th + k * 2, id64m, 1);
        }
        wait(&B->y_ready, ph);
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t y = tmem + kKS + (k >> 1) * 32 + (k & 1) * 8;
          umma_ts_w(tmem + kX, y + 16, th + k * 2, id64, 1);
          umma_ts_w(tmem + kX, y, tl + k * 2, id64, 1);
          umma_ts_w(tmem + kX, y, th + k * 2, id64, 1);
        }
        umma_commit_w(&B->x_full);
        // the next chunk's products with itself
        if (n + 1 < total) {
          wait(&B->ready[(n + 1) % kStages], ((n + 1) / kStages) & 1);
          wait(&B->d1_free, ph);
          tc_fence_after();
          issue_d1(n + 1);
        }
        // X^T K
        wait(&B->xs_ready, ph);
        tc_fence_after();
        const uint64_t km = smem_desc_sw128(st + kBlk, 2 * kBlk, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = tmem + kX + (k >> 1) * 32 + (k & 1) * 8;
          umma_ts_w(tmem + kDS, x + 16, km + k * 128, id128, k != 0);
          umma_ts_w(tmem + kDS, x, km + k * 128, id128, 1);
        }
        umma_commit_w(&B->ds_full);
        // P X
        wait(&B->x_ready, ph);
        tc_fence_after();
        const uint64_t pH = smem_desc_sw128(tb, 16, 1024);
        const uint64_t pL = smem_desc_sw128(tb + kBlk, 16, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = tmem + kX + (k >> 1) * 32 + (k & 1) * 8;
          umma_ts_w(tmem + kO, x + 16, pH + k * 2, id64, k != 0);
          umma_ts_w(tmem + kO, x, pL + k * 2, id64, 1);
          umma_ts_w(tmem + kO, x, pH + k * 2, id64, 1);
        }
        umma_commit_w(&B->o_full);
        umma_commit_w(&B->tp_free[ph]);
        umma_commit_w(&B->empty[n % kStages]);
      }
      // every arrival on this CTA's barriers has landed before it ends
      if (total > 0) wait(&B->empty[(total - 1) % kStages], ((total - 1) / kStages) & 1);
    } else if (warp == 2) {
      constexpr float kLog2e = 1.4426950408889634f;
      int n = 0;
      for (int i = blockIdx.x; i < p.items; i += gridDim.x) {
        const Item it = get_item(p, i);
        const float* g = p.g + it.batch * p.sg.batch + it.h * p.sg.head + it.t0 * p.sg.token;
        const float* be = p.beta + it.batch * p.sb.batch + it.h * p.sb.head + it.t0 * p.sb.token;
        const int nc = chunks(it);
        float gv[2], bv[2], gn[2], bn[2];
        auto load = [&](int c, float (&x)[2], float (&y)[2]) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = c * kC + 32 * e + lane;
            x[e] = t < it.len ? g[t * p.sg.token] : 0.f;
            y[e] = t < it.len ? be[t * p.sb.token] : 0.f;
          }
        };
        if (nc > 0) load(0, gn, bn);
        for (int c = 0; c < nc; ++c, ++n) {
          const int s = n % kStages;
          gv[0] = gn[0]; gv[1] = gn[1]; bv[0] = bn[0]; bv[1] = bn[1];
          if (c + 1 < nc) load(c + 1, gn, bn);
          // full: the stage was empty, and so were its factors
          wait(&B->full[s], (n / kStages) & 1);
          Scal& sc = scal[s];
          float gl[2], tot[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // exp(-104) is zero in fp32: -inf becomes a number that can be subtracted
            float x = fmaxf(gv[e], -104.f);
            if (gv[e] != gv[e]) x = gv[e];
            x *= kLog2e;
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) {
              const float y = __shfl_up_sync(0xffffffffu, x, o, 16);
              if ((lane & 15) >= o) x += y;
            }
            gl[e] = x;
            tot[e] = __shfl_sync(0xffffffffu, x, 15, 16);   // this lane's block
          }
          float blk[4];
          blk[0] = __shfl_sync(0xffffffffu, tot[0], 0);
          blk[1] = __shfl_sync(0xffffffffu, tot[0], 16);
          blk[2] = __shfl_sync(0xffffffffu, tot[1], 0);
          blk[3] = __shfl_sync(0xffffffffu, tot[1], 16);
          const bool up = lane >= 16;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = 32 * e + lane;
            const float before = e == 0 ? (up ? blk[0] : 0.f)
                                        : (up ? blk[0] + blk[1] + blk[2] : blk[0] + blk[1]);
            const float after = e == 0 ? (up ? blk[2] + blk[3] : blk[1] + blk[2] + blk[3])
                                       : (up ? 0.f : blk[3]);
            const float rest = tot[e] - gl[e];
            sc.eg[j] = ex2(gl[e] + before);
            sc.er[j] = ex2(rest + after);
            sc.beta[j] = bv[e];
            sc.gl[j] = gl[e];
            sc.el[j] = ex2(rest);
          }
          if (lane == 0) {
            sc.blk[0] = blk[0]; sc.blk[1] = blk[1]; sc.blk[2] = blk[2]; sc.blk[3] = blk[3];
            sc.eall = ex2(blk[0] + blk[1] + blk[2] + blk[3]);
          }
          const int valid = min(kC, it.len - c * kC);
          if (valid < kC) {
            const uint32_t st = smem_u32(smem + s * kStageBytes) + valid * 128;
            const int pieces = (kC - valid) * 8;
            for (int b = 0; b < 6; ++b)
              for (int x = lane; x < pieces; x += 32)
                sts128(st + b * kBlk + x * 16, make_uint4(0, 0, 0, 0));
            fence_proxy_async_smem();
          }
          arrive(&B->ready[s]);
        }
      }
    }
  } else if (warp < 8) {
    // ---- P = scale D o Q K^T and T
    regs_dec<88>();
    const int q4 = warp & 3, half = q4 & 1, tid = threadIdx.x - 128;
    const int g8 = lane >> 2, t4 = lane & 3;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const int row = half * 32 + lane, I = row >> 4;
    int total = 0;
    for (int i = blockIdx.x; i < p.items; i += gridDim.x) total += chunks(get_item(p, i));
    for (int n = 0; n < total; ++n) {
      const int s = n % kStages;
      const Scal& sc = scal[s];
      uint8_t* buf = tp + (n & 1) * kTPBytes;
      float* M = reinterpret_cast<float*>(buf + 2 * kBlk);
      wait(&B->ready[s], (n / kStages) & 1);
      const float gli = sc.gl[row];
      const float mul = q4 < 2 ? p.scale : sc.beta[row];
      float f[3];
      {
        float e = gli;
#pragma unroll
        for (int J = 2; J >= 0; --J) {
          f[J] = 0.f;
          if (J < I) {
            f[J] = mul * ex2(e);
            e += sc.blk[J];
          }
        }
      }
      wait(&B->tp_free[n & 1], ((n >> 1) & 1) ^ 1);
      wait(&B->d1_full, n & 1);
      tc_fence_after();
#pragma unroll
      for (int J = 0; J < 4; ++J) {
        float x[16];
        if (J <= 2 * half + 1) {
          tmem_ld16(tmem + kD1 + lane_off + 16 * J, x);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int j = 16 * J + e;
            float d = 0.f;
            if (J >= 2 * half) d = j <= row ? mul * ex2(gli - sc.gl[j]) : 0.f;
            if (J < 3 && J < I) d = f[J < 3 ? J : 0] * sc.el[j];
            // a product of rows that do not meet here may be anything: no 0 * inf
            x[e] = j <= row ? x[e] * d : 0.f;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0.f;
        }
        if (q4 < 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split2(x[8 * h + 2 * e], x[8 * h + 2 * e + 1], hi[e], lo[e]);
            const uint32_t o =
                smem_u32(buf) + row * 128 + (((2 * J + h) ^ (row & 7)) << 4);
            sts128(o, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            sts128(o + kBlk, make_uint4(lo[0], lo[1], lo[2], lo[3]));
          }
        } else if (J <= 2 * half + 1) {
#pragma unroll
          for (int h = 0; h < 4; ++h)
            *reinterpret_cast<float4*>(&M[at(row, 16 * J + 4 * h)]) =
                make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
        }
      }
      tc_fence_before();
      arrive(&B->d1_free);
      named_bar_sync(1, 128);
      {   // T of this warp's diagonal block, column lane & 15 in registers
        const int b0 = 16 * q4, c = lane & 15;
        float x[16];
        x[0] = c == 0 ? 1.f : 0.f;
#pragma unroll
        for (int i = 1; i < 16; ++i) {
          float a[16];
#pragma unroll
          for (int m = 0; m <= (i - 1) / 4; ++m)
            *reinterpret_cast<float4*>(&a[4 * m]) =
                *reinterpret_cast<const float4*>(&M[at(b0 + i, b0 + 4 * m)]);
          float v0 = c == i ? 1.f : 0.f, v1 = 0.f;
#pragma unroll
          for (int l = 0; l < i; ++l) {
            if (l & 1) v1 = fmaf(-a[l], x[l], v1);
            else v0 = fmaf(-a[l], x[l], v0);
          }
          x[i] = v0 + v1;
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
          for (int i = 0; i < 16; ++i) M[at(b0 + i, b0 + c)] = x[i];
        }
      }
      named_bar_sync(1, 128);
      {   // T_10 and T_32: two warps each, eight columns a warp
        const int J = q4 & 2, I1 = J + 1, col = 8 * (q4 & 1);
        float w[2][4] = {}, r[4] = {};
        block_mm(w, M, 16 * I1, 16 * I1, 16 * J, g8, t4);
        block_wm(r, w, M, 16 * J, 16 * J + col, g8, t4);
        named_bar_sync(1, 128);
        put_neg(M, r, 16 * I1, 16 * J + col, g8, t4);
      }
      named_bar_sync(1, 128);
      {   // the lower left quarter: block (I2, J2) of it
        const int I2 = 2 + (q4 >> 1), J2 = q4 & 1;
        float w1[2][4] = {}, w0[2][4] = {}, r[2][4] = {};
        for (int m = 2; m <= I2; ++m) {
          block_mm(w1, M, 16 * I2, 16 * m, 16, g8, t4);
          if (J2 == 0) block_mm(w0, M, 16 * I2, 16 * m, 0, g8, t4);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          block_wm(r[c], w1, M, 16, 16 * J2 + 8 * c, g8, t4);
          if (J2 == 0) block_wm(r[c], w0, M, 0, 8 * c, g8, t4);
        }
        named_bar_sync(1, 128);
#pragma unroll
        for (int c = 0; c < 2; ++c) put_neg(M, r[c], 16 * I2, 16 * J2 + 8 * c, g8, t4);
      }
      named_bar_sync(1, 128);
      {   // T diag(beta) as a pair, over the scratch
        const int i = tid >> 1, j0 = 32 * (tid & 1);
        float x[32];
#pragma unroll
        for (int m = 0; m < 8; ++m)
          *reinterpret_cast<float4*>(&x[4 * m]) =
              *reinterpret_cast<const float4*>(&M[at(i, j0 + 4 * m)]);
#pragma unroll
        for (int m = 0; m < 32; ++m) x[m] = j0 + m <= i ? x[m] * sc.beta[j0 + m] : 0.f;
        named_bar_sync(1, 128);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(x[8 * h + 2 * e], x[8 * h + 2 * e + 1], hi[e], lo[e]);
          const uint32_t o =
              smem_u32(M) + i * 128 + (((j0 / 8 + h) ^ (i & 7)) << 4);
          sts128(o, make_uint4(hi[0], hi[1], hi[2], hi[3]));
          sts128(o + kBlk, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
      }
      fence_proxy_async_smem();
      arrive(&B->tp_ready[n & 1]);
      arrive(&B->empty[s]);
    }
  } else if (warp < 16) {
    // ---- the chain: rows 32 q4 + lane, half of the columns
    regs_inc<136>();
    const int q4 = warp & 3, half = (warp - 8) >> 2;
    const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
    int n = 0;
    for (int i = blockIdx.x; i < p.items; i += gridDim.x) {
      const Item it = get_item(p, i);
      const int nc = chunks(it);
      const int row = 128 * it.tile + 32 * q4 + lane;
      const long long so = (((long long)it.seq * p.Hv + it.h) * p.dv + row) * p.dk + 64 * half;
      float S[64];
#pragma unroll
      for (int c = 0; c < 64; c += 4) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.S0 && row < p.dv && 64 * half + c < p.dk)
          x = *reinterpret_cast<const float4*>(p.S0 + so + c);
        S[c] = x.x; S[c + 1] = x.y; S[c + 2] = x.z; S[c + 3] = x.w;
      }
      auto put_S = [&]() {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            split2(S[32 * b + 2 * e], S[32 * b + 2 * e + 1], hi[e], lo[e]);
          tmem_st16(tl + kSh + 32 * half + 16 * b, hi);
          tmem_st16(tl + kSh + 64 + 32 * half + 16 * b, lo);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(&B->s_ready);
      };
      if (nc > 0) put_S();
      for (int c = 0; c < nc; ++c, ++n) {
        const int s = n % kStages;
        const uint32_t ph = n & 1;
        const Scal& sc = scal[s];
        float x[32];
        uint32_t xh[16], xl[16];
        wait(&B->ready[s], (n / kStages) & 1);
        wait(&B->ks_full, ph);
        tc_fence_after();
        tmem_ld32(tl + kKS + 32 * half, x);
        tmem_wait32(x);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 f = *reinterpret_cast<const float2*>(&sc.eg[32 * half + 2 * e]);
          split2(-f.x * x[2 * e], -f.y * x[2 * e + 1], xh[e], xl[e]);
        }
        tmem_st16(tl + kKS + 32 * half, xh);
        tmem_st16(tl + kKS + 32 * half + 16, xl);
        tmem_wait_st();
        tc_fence_before();
        arrive(&B->y_ready);

        wait(&B->x_full, ph);
        tc_fence_after();
        tmem_ld32(tl + kX + 32 * half, x);
        tmem_wait32(x);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 f = *reinterpret_cast<const float2*>(&sc.er[32 * half + 2 * e]);
          split2(f.x * x[2 * e], f.y * x[2 * e + 1], xh[e], xl[e]);
        }
        tmem_st16(tl + kX + 32 * half, xh);
        tmem_st16(tl + kX + 32 * half + 16, xl);
        tmem_wait_st();
        tc_fence_before();
        arrive(&B->xs_ready);
#pragma unroll
        for (int e = 0; e < 16; ++e) split2(x[2 * e], x[2 * e + 1], xh[e], xl[e]);
        const float eall = sc.eall;
        arrive(&B->empty[s]);

        wait(&B->ds_full, ph);
        tc_fence_after();
        tmem_st16(tl + kX + 32 * half, xh);
        tmem_st16(tl + kX + 32 * half + 16, xl);
        tmem_wait_st();
        tc_fence_before();
        arrive(&B->x_ready);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          tmem_ld32(tl + kDS + 64 * half + 32 * b, x);
          tmem_wait32(x);
#pragma unroll
          for (int e = 0; e < 32; ++e) S[32 * b + e] = fmaf(eall, S[32 * b + e], x[e]);
        }
        if (c + 1 < nc) put_S();
      }
      if (ok && p.S_final && row < p.dv) {
#pragma unroll
        for (int c = 0; c < 64; c += 4)
          if (64 * half + c < p.dk)
            *reinterpret_cast<float4*>(p.S_final + so + c) =
                make_float4(S[c], S[c + 1], S[c + 2], S[c + 3]);
      }
    }
  } else {
    // ---- outputs
    regs_dec<64>();
    const int q4 = warp & 3;
    const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
    int n = 0;
    for (int i = blockIdx.x; i < p.items; i += gridDim.x) {
      const Item it = get_item(p, i);
      const int nc = chunks(it);
      const int col = 128 * it.tile + 32 * q4 + lane;
      __nv_bfloat16* out = p.out + it.batch * p.so.batch + it.h * p.so.head +
                           it.t0 * p.so.token + col;
      for (int c = 0; c < nc; ++c, ++n) {
        const int s = n % kStages;
        const Scal& sc = scal[s];
        wait(&B->ready[s], (n / kStages) & 1);
        wait(&B->o_full, n & 1);
        tc_fence_after();
        const int valid = ok && col < p.dv ? min(kC, it.len - c * kC) : 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          float x[16], y[16];
          tmem_ld16_nowait(tl + kQS + 16 * b, x);
          tmem_ld16_nowait(tl + kO + 16 * b, y);
          tmem_wait_bind(x);
          tmem_wait_bind(y);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int t = 16 * b + e;
            if (t < valid)
              out[(long long)(c * kC + t) * p.so.token] =
                  __float2bfloat16_rn(fmaf(p.scale * sc.eg[t], x[e], y[e]));
          }
        }
        tc_fence_before();
        arrive(&B->o_free);
        arrive(&B->empty[s]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

int g_ready[64] = {0};   // 0 unknown, 1 usable, 2 not usable
int g_sms[64] = {0};
std::mutex g_mu;

// One-time setup of the current device; the number of SMs, 0 if not usable.
int prepare() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_ready[dev] == 0) {
    g_ready[dev] = 2;
    if (cudaFuncSetAttribute(delta_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmem) == cudaSuccess &&
        cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
      g_ready[dev] = 1;
    cudaGetLastError();
  }
  return g_ready[dev] == 1 ? g_sms[dev] : 0;
}

// [B, H, N, d] bf16 with the given strides as a map of 64 x 64 boxes.
bool make_map(CUtensorMap* m, const void* ptr, const delta_rule_stride& s, int B, int H, int N,
              int d) {
  const unsigned long long dims[4] = {(unsigned long long)d, (unsigned long long)N,
                                      (unsigned long long)H, (unsigned long long)B};
  // the stride of a dimension of one element is never used: give a valid one
  auto bytes = [](long long x, int n) { return n > 1 ? (unsigned long long)x * 2 : 16ull; };
  const unsigned long long st[3] = {bytes(s.token, N), bytes(s.head, H), bytes(s.batch, B)};
  for (unsigned long long x : st)
    if (x == 0 || x % 16 != 0 || x >= (1ull << 40)) return false;
  if ((reinterpret_cast<uintptr_t>(ptr) & 15) != 0 || d % 8 != 0) return false;
  const unsigned box[4] = {64, kC, 1, 1};
  return encode_bf16_4d(m, ptr, dims, st, box);
}

}  // namespace

int delta_rule_chunk_launch(const DeltaArgs& a) {
  if (!a.bf16 || a.dk > 128) return 1;
  ChunkParams p;
  if (!make_map(&p.q, a.q, a.lay.q, a.B, a.Hk, a.N, a.dk) ||
      !make_map(&p.k, a.k, a.lay.k, a.B, a.Hk, a.N, a.dk) ||
      !make_map(&p.v, a.v, a.lay.v, a.B, a.Hv, a.N, a.dv))
    return 1;
  const int sms = prepare();
  if (!sms) return TTT_ERR_CUDA;
  p.g = a.g; p.beta = a.beta; p.S0 = a.S0; p.starts = a.seq_starts;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.S_final = a.S_final;
  p.status = a.status;
  p.wait_ns = a.wait_ns;
  p.sg = a.lay.g; p.sb = a.lay.beta; p.so = a.lay.out;
  p.Hk = a.Hk; p.Hv = a.Hv; p.N = a.N; p.dk = a.dk; p.dv = a.dv;
  p.tiles = (a.dv + 127) / 128;
  p.items = a.n_seq * a.Hv * p.tiles;
  p.scale = a.scale;
  const double tok = (double)a.B * a.N;
  ProfScope ps(PT_DELTA_CHUNK, a.stream, 7.0 * tok * a.Hv * a.dk * a.dv,
               tok * 4.0 * (a.Hk * a.dk + a.Hv * a.dv));
  delta_chunk_kernel<<<p.items < sms ? p.items : sms, kThreads, kSmem, a.stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

}  // namespace ttt
