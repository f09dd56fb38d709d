// What the tensor-core kernels of the gated delta rule share: the records that
// one writes and the other reads, and small device helpers.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "delta_rule.h"

namespace ttt {

constexpr int kC = 64;       // tokens per chunk
constexpr int kBlk = 8192;   // 64 rows of 64 bf16, 128-byte swizzled

// Record of one (chunk, value head): four 64 x 64 bf16 tiles as the MMAs read
// them (rows i, columns j, 128-byte swizzled): T diag(beta) hi and lo,
// scale D o Q K^T hi and lo.
constexpr int kRecBytes = 4 * kBlk;

struct RecScal {
  float neg[kC];   // -exp(G_i)
  float er[kC];    // exp(G_63 - G_j)
  float eall;      // exp(G_63)
  float pad[3];
};
static_assert(sizeof(RecScal) % 16 == 0, "bulk copies move 16 bytes");

// Token range of a sequence, and the number of its first chunk's records.  For
// packed sequences both come from a plan that one block makes beforehand.
struct SeqPlan {
  int t0, len, chunk0, pad;
};

// Segment j of n of a sequence: the chunks that one CTA walks.
struct SegPlan {
  int seq, j, n;
  int chunks;   // of each segment but a sequence's last
};

__host__ __device__ __forceinline__ int n_chunks(int len) {
  return len / kC + (len % kC != 0);   // len + 63 may pass 31 bits
}

__device__ __forceinline__ SeqPlan seq_plan(const SeqPlan* plan, int seq, int N) {
  if (plan) return plan[seq];
  SeqPlan s;
  s.t0 = 0;
  s.len = N;
  s.chunk0 = seq * n_chunks(N);
  s.pad = 0;
  return s;
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ bool elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}"
               : "=r"(r));
  return r != 0;
}

// Bounded wait, by every lane for itself (a vote after each wait would double its
// 45 cycles, and a chunk's chain holds a dozen of them in turn).  After one that ran
// out (ok false) a lane's waits return at once and its role runs to its end.  It stores
// nothing any more, and gives back no shared memory that copies or products may still be
// using: it arrives on none of the barriers that say that copies have landed or that a
// stage is free, and commits no products.  (Not issuing them cost 2.5% of a call,
// not arriving anywhere 0.6%.)  What it hands on otherwise is garbage that other roles may
// store; the status word says that the results are void.  Loops bring `ok` together once
// an iteration (together()), before anything that the whole warp must do together depends
// on it.  Before the CTA ends, the roles that issue copies and products wait for their last
// ones, for those that they were for may have given up.
__device__ __forceinline__ void wait_w(bool& ok, uint64_t* bar, uint32_t parity, int* status,
                                       unsigned long long lim) {
  if (!ok || mbar_try_wait(bar, parity)) return;
  unsigned long long since = 0;
  while (!mbar_try_wait_sleep(bar, parity, 1000000u)) {
    const unsigned long long now = global_ns();
    if (since == 0) since = now;
    if (now - since > lim) {
      report_status(status, kStatusTimeout);
      ok = false;
      return;
    }
  }
}
__device__ __forceinline__ bool together(bool ok) { return __all_sync(0xffffffffu, ok); }

// Two fp32 values in one 64-bit register, for the packed fp32 instructions.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pack2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(F2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 sub2(F2 a, F2 b) {
  F2 r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// (a, b) as a pair of packed bf16 pairs: a ~ hi.x + lo.x, b ~ hi.y + lo.y, each
// off by at most 2^-17 of its value.
__device__ __forceinline__ void split2(F2 v, uint32_t& hi, uint32_t& lo) {
  float a, b;
  unpack2(v, a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const F2 r = sub2(v, pack2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)));
  unpack2(r, a, b);
  const __nv_bfloat162 l = __floats2bfloat162_rn(a, b);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- host side
// Launch that may begin while the kernel before it in the stream still runs: its
// prologue (barriers, TMEM, tensor maps) overlaps that kernel's end.  The kernel
// calls pdl_wait() before it touches memory.  A kernel that uses TMEM lets the next
// one begin (pdl_launch_dependents) only once it holds its own: a CTA of the next kernel
// keeps what it allocates until this kernel has ended, so that a CTA of this one that
// came to the same SM with its allocation still ahead would wait for ever.  Short launches
// in a row gain their launch's latency too: 56 tokens of 16 heads 24.6 -> 22.5 us, 20011
// rows of 1536 69.6 -> 67.5.
template <typename P>
cudaError_t launch_behind(void (*kern)(P), unsigned grid, unsigned block, size_t smem,
                          cudaStream_t stream, const P& params) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, params);
}

// [B, H, N, d] bf16 with the given strides as a map of 64 x 64 boxes; false
// where TMA cannot take it.
bool delta_map(CUtensorMap* m, const void* ptr, const delta_rule_stride& s, int B, int H, int N,
               int d);

struct PrepParams {
  CUtensorMap q, k;
  const float* g;
  const float* beta;
  const SeqPlan* plan;     // or NULL
  int n_seq;
  int Hk, Hv, N, dk;
  delta_rule_stride sg, sb;
  float scale;
  uint8_t* rec;            // [chunk][Hv] records
  RecScal* scal;           // [chunk][Hv]
  int* status;
  unsigned long long wait_ns;
  int withhold;            // test hook: the first CTA's loads are not issued
};

// One-time kernel attributes of the current device.
cudaError_t prepare_delta_prep();
// The records of every chunk; `chunks` is the number of chunk places.
cudaError_t launch_delta_prep(const PrepParams& p, int chunks, cudaStream_t stream);

}  // namespace ttt
