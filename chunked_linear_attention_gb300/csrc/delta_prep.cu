// First kernel of the tensor-core delta rule: what a chunk of 64 tokens needs that
// does not depend on the state, for all chunks at once.  One CTA takes a (chunk,
// key head): Q K^T and K K^T in one MMA (M = 128: the rows of Q, then of K), then
// for each value head of the key head, with G the running sum of g inside the
// chunk and D_ij = exp(G_i - G_j),
//     P_ij = scale D_ij q_i . k_j  (i >= j)
//     T    = (1 + A)^-1 diag(beta),  A_ij = beta_i D_ij k_i . k_j  (i > j)
// each as a pair of bf16 tiles in the layout of the second kernel's MMAs.
//
// The inverse: the four 16 x 16 diagonal blocks by substitution, two of them a warp, a
// column per lane; then joined, T_21 = -T_22 A_21 T_11, first to 32 and then to
// 64, by products of 16 x 16 blocks on mma.sync tf32 with both operands in two
// parts (fp32 accuracy; the smallest tcgen05 product has 64 rows).
//
// D is never formed from differences of rounded sums (behind a few tokens that clear the
// state a sum inside a block of 16 reaches 1e3, and its last bit 1e-4): inside a block
// the running sum is a pair of fp32 numbers, whose differences keep the small g between
// two tokens; from a token to its block's end the small g are summed for themselves,
// from the end on; and blocks are joined by factors that are at most 1 where g <= 0.
//
// Bound by instruction issue and shared memory (issue 48%, l1tex 61%, DRAM 34%): the
// decays, the substitution and the pairs cost about 7400 warp instructions per
// record.  2048 records (B 4, H 4, 8192 tokens) take 33 us, 8192 (131072 tokens of 4
// heads) 101 us, against 80 for the bytes (32 and 98 with the running sum in one number;
// its differences by packed instructions, at more registers, took 34).  Six
// CTAs per SM, so that one's substitution runs beside another's products; T's tiles lie
// over the scratch, and the record over q and k, to make room for them.
#include "delta_tc.cuh"
#include "prof.h"

namespace ttt {

namespace {

// ---------------------------------------------------------------- 16 x 16 blocks
// The fp32 scratch of A and T: the ten 16 x 16 blocks (I, J <= I) one behind the
// other, rows of 16 floats 20 apart (so that the fragments' and the rows'
// accesses spread over the banks).
constexpr int kRowF = 20, kBlockF = 16 * kRowF;
static_assert(10 * kBlockF * 4 <= 2 * kBlk, "scratch");

__device__ __forceinline__ int block_at(int I, int J) { return (I * (I + 1) / 2 + J) * kBlockF; }

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

// c (16 rows, NT tiles of 8 columns) += A B for 16 x 16 blocks A and B (B from
// its first column on): three tf32 products of the parts.  The order of the
// summation index is free: places t and t + 4 of a step of eight take columns
// (rows of B) 2t and 2t + 1.
template <int NT>
__device__ __forceinline__ void block_mm(float (&c)[NT][4], const float* A, const float* B,
                                         int lane) {
  const int g = lane >> 2, t = lane & 3;
  const float* a = A + g * kRowF + 2 * t;
  const float* b = B + 2 * t * kRowF + g;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const float2 u = *reinterpret_cast<const float2*>(a + 8 * s);
    const float2 v = *reinterpret_cast<const float2*>(a + 8 * s + 8 * kRowF);
    uint32_t ah[4], al[4];
    tf32_parts(u.x, ah[0], al[0]);
    tf32_parts(v.x, ah[1], al[1]);
    tf32_parts(u.y, ah[2], al[2]);
    tf32_parts(v.y, ah[3], al[3]);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t h0, l0, h1, l1;
      tf32_parts(b[8 * s * kRowF + 8 * n], h0, l0);
      tf32_parts(b[(8 * s + 1) * kRowF + 8 * n], h1, l1);
      mma_tf32(c[n], al, h0, h1);
      mma_tf32(c[n], ah, l0, l1);
      mma_tf32(c[n], ah, h0, h1);
    }
  }
}

template <int NT>
__device__ __forceinline__ void block_put(float* M, const float (&c)[NT][4], float sign, int lane) {
  float* m = M + (lane >> 2) * kRowF + 2 * (lane & 3);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    *reinterpret_cast<float2*>(m + 8 * n) = make_float2(sign * c[n][0], sign * c[n][1]);
    *reinterpret_cast<float2*>(m + 8 * n + 8 * kRowF) = make_float2(sign * c[n][2], sign * c[n][3]);
  }
}

// ---------------------------------------------------------------- the kernel
constexpr int kPThreads = 128;
constexpr uint32_t kPCols = 64;

struct PrepShared {
  float beta[kC];
  float2 gl[kC];   // running sum of g log2(e) inside each block of 16, and what its
                   // roundings left out
  float el[kC];    // decay from token j to the end of its block
  float blk[4];    // each block's sum of g log2(e)
  RecScal scal;
  uint64_t full, done;
  uint32_t tmem;
};
// Q0 K0 Q1 K1 (column blocks of 64), then the four tiles of a record
constexpr int kPSmem = 4 * kBlk + (int)sizeof(PrepShared) + 1024;

__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

__global__ void __launch_bounds__(kPThreads, 6)
    delta_prep_kernel(const __grid_constant__ PrepParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tile =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  PrepShared& sh = *reinterpret_cast<PrepShared*>(tile + 4 * kBlk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.x % p.Hk, place = blockIdx.x / p.Hk;
  if (p.plan) pdl_wait();   // the plan is the kernel before
  // the chunk at this place
  int seq, c;
  if (p.plan) {   // last sequence whose first chunk is not behind the place
    int lo = 0, hi = p.n_seq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.plan[mid].chunk0 <= place) lo = mid;
      else hi = mid - 1;
    }
    seq = lo;
    c = place - p.plan[lo].chunk0;
  } else {
    const int nc = n_chunks(p.N);
    seq = place / nc;
    c = place - seq * nc;
  }
  const SeqPlan sp = seq_plan(p.plan, seq, p.N);
  const int valid = min(kC, sp.len - c * kC);
  if (valid <= 0) return;
  const int batch = p.plan ? 0 : seq, t0 = sp.t0 + c * kC;
  const int group = p.Hv / p.Hk;
  bool ok = true;

  if (tid == 0) {
    mbar_init(&sh.full, 1);
    mbar_init(&sh.done, 1);
    fence_mbar_init();
    const int blocks = p.withhold && blockIdx.x == 0 ? 0 : p.dk > 64 ? 2 : 1;
    if (blocks) mbar_arrive_expect_tx(&sh.full, 2 * blocks * kBlk);
    for (int b = 0; b < blocks; ++b) {
      tma_load_4d(tile + 2 * b * kBlk, &p.q, 64 * b, t0, hk, batch, &sh.full);
      tma_load_4d(tile + (2 * b + 1) * kBlk, &p.k, 64 * b, t0, hk, batch, &sh.full);
    }
  }
  if (warp == 1) tmem_alloc(&sh.tmem, kPCols);
  // this head's g and beta: warp 3 (beside warp 0's wait for the tiles), tokens lane
  // and lane + 32
  float gv[2] = {0.f, 0.f}, bv[2] = {0.f, 0.f};
  auto load_gates = [&](int h) {
    const float* g = p.g + batch * p.sg.batch + h * p.sg.head + t0 * p.sg.token;
    const float* be = p.beta + batch * p.sb.batch + h * p.sb.head + t0 * p.sb.token;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = 32 * e + lane;
      gv[e] = t < valid ? g[t * p.sg.token] : 0.f;
      bv[e] = t < valid ? be[t * p.sb.token] : 0.f;
    }
  };
  if (warp == 3) load_gates(hk * group);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_launch_dependents();   // (with TMEM in hand: see launch_behind)
  if (warp == 0 || valid < kC) wait_w(ok, &sh.full, 0, p.status, p.wait_ns);
  if (valid < kC) {   // rows behind the sequence's end: other tokens, or none
    const int pieces = (kC - valid) * 8;
    for (int b = 0; b < 4; ++b)
      for (int x = tid; x < pieces; x += kPThreads)
        sts128(smem_u32(tile) + b * kBlk + valid * 128 + x * 16, make_uint4(0, 0, 0, 0));
    fence_proxy_async_smem();
    __syncthreads();
  }
  if (warp == 0) {
    const uint64_t a = smem_desc_sw128(smem_u32(tile), 16, 1024);
    const uint64_t b = smem_desc_sw128(smem_u32(tile) + kBlk, 16, 1024);
    const uint32_t id = idesc_bf16_f32(64, 0, 0);
    if (elect_lane()) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (!ok || (k == 4 && p.dk <= 64)) break;
        const uint32_t o = (k >> 2) * (2 * kBlk / 16) + (k & 3) * 2;
        umma_bf16(tmem, a + o, b + o, id, k != 0);
      }
      umma_commit(&sh.done);
    }
    __syncwarp();
  }

  const int half = warp & 1, row = half * 32 + lane, I = row >> 4;
  const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
  float* M = reinterpret_cast<float*>(tile);   // over the room of T's tiles
#pragma unroll 1
  for (int hg = 0; hg < group; ++hg) {
    const int h = hk * group + hg;
    if (warp == 3) {
      constexpr float kLog2e = 1.4426950408889634f;
      float gl[2], rest[2], tot[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // exp(-104) is zero in fp32: -inf becomes a number that can be subtracted
        const float x0 = (gv[e] < -104.f ? -104.f : gv[e]) * kLog2e;
        float x = x0, r = 0.f;   // the sum up to this token
        float z = __shfl_down_sync(0xffffffffu, x0, 1, 16);   // and of the tokens behind it
        if ((lane & 15) == 15) z = 0.f;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
          const float y = __shfl_up_sync(0xffffffffu, x, o, 16);
          const float s = __shfl_up_sync(0xffffffffu, r, o, 16);
          const float w = __shfl_down_sync(0xffffffffu, z, o, 16);
          if ((lane & 15) >= o) {   // two numbers as their sum and its rounding error
            const float sum = __fadd_rn(x, y), part = __fsub_rn(sum, x);
            r += s + __fadd_rn(__fsub_rn(x, __fsub_rn(sum, part)), __fsub_rn(y, part));
            x = sum;
          }
          if ((lane & 15) + o < 16) z += w;
        }
        gl[e] = x;
        rest[e] = z;
        sh.gl[32 * e + lane] = make_float2(x, r);
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
        sh.scal.neg[j] = -ex2(gl[e] + before);
        sh.scal.er[j] = ex2(rest[e] + after);
        sh.beta[j] = bv[e];
        sh.el[j] = ex2(rest[e]);
      }
      if (lane == 0) {
#pragma unroll
        for (int b = 0; b < 4; ++b) sh.blk[b] = blk[b];
        sh.scal.eall = ex2(blk[0] + blk[1] + blk[2] + blk[3]);
      }
      if (hg + 1 < group) load_gates(h + 1);
    }
    if (hg == 0) {
      wait_w(ok, &sh.done, 0, p.status, p.wait_ns);   // the tiles' room is free for the record
      tc_fence_after();
    }
    __syncthreads();
    const float gli = sh.gl[row].x;
    const float mul = warp < 2 ? p.scale : sh.beta[row];
    float decay = gli;   // log2 of the decay from the end of block J to the row
    const uint32_t prow = smem_u32(tile) + 2 * kBlk + row * 128;
#pragma unroll 1
    for (int J = 3; J >= 0; --J) {
      if (J > 2 * half + 1) {   // behind the diagonal for all of the warp
        if (warp < 2) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const uint32_t o = prow + (((2 * J + b) ^ (row & 7)) << 4);
            sts128(o, make_uint4(0, 0, 0, 0));
            sts128(o + kBlk, make_uint4(0, 0, 0, 0));
          }
        }
        continue;
      }
      float x[16];
      F2 y[8];
      tmem_ld16_nowait(tmem + lane_off + 16 * J, x);
      float f = 0.f;
      if (J < I) {
        f = mul * ex2(decay);
        decay += sh.blk[J];
      }
      const F2 f2 = pack2(f, f);
      const ulonglong2* el2 = reinterpret_cast<const ulonglong2*>(&sh.el[16 * J]);
      F2 d[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const ulonglong2 w = el2[e];
        d[2 * e] = mul2(f2, w.x);
        d[2 * e + 1] = mul2(f2, w.y);
      }
      if (J >= 2 * half) {   // lanes with their diagonal here, or (J > I) nothing
        const float4* gl2 = reinterpret_cast<const float4*>(&sh.gl[16 * J]);
        const int last = row - 16 * J;   // last column of the row's part
        if (J >= I) {
          const float gri = sh.gl[row].y;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 w = gl2[e];
            d[e] = pack2(mul * ex2((gli - w.x) + (gri - w.y)),
                         mul * ex2((gli - w.z) + (gri - w.w)));
          }
        }
        tmem_wait_bind(x);
        // a product behind the diagonal may be anything, and so may its decay
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float a, b;
          unpack2(mul2(pack2(x[2 * e], x[2 * e + 1]), d[e]), a, b);
          y[e] = pack2(2 * e <= last ? a : 0.f, 2 * e + 1 <= last ? b : 0.f);
        }
      } else {
        tmem_wait_bind(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = mul2(pack2(x[2 * e], x[2 * e + 1]), d[e]);
      }
      if (warp < 2) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(y[4 * b + e], hi[e], lo[e]);
          const uint32_t o = prow + (((2 * J + b) ^ (row & 7)) << 4);
          sts128(o, make_uint4(hi[0], hi[1], hi[2], hi[3]));
          sts128(o + kBlk, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
      } else if (J <= I) {
        ulonglong2* m = reinterpret_cast<ulonglong2*>(M + block_at(I, J) + (row & 15) * kRowF);
#pragma unroll
        for (int b = 0; b < 4; ++b) m[b] = make_ulonglong2(y[2 * b], y[2 * b + 1]);
      }
    }
    // T of the diagonal blocks, by the warps that have just written them (two blocks
    // each, a column per lane), while the others are at P's pairs
    if (warp >= 2) {
      __syncwarp();
      const int col = lane & 15, blk = 2 * half + (lane >> 4);
      float* m = M + block_at(blk, blk);
      float x[16];
      x[0] = col == 0 ? 1.f : 0.f;
#pragma unroll
      for (int i = 1; i < 16; ++i) {
        float a[16];
#pragma unroll
        for (int e = 0; e <= (i - 1) / 4; ++e)
          *reinterpret_cast<float4*>(&a[4 * e]) =
              *reinterpret_cast<const float4*>(m + i * kRowF + 4 * e);
        float v0 = col == i ? 1.f : 0.f, v1 = 0.f;
#pragma unroll
        for (int l = 0; l < i; ++l) {
          if (l & 1) v1 = fmaf(-a[l], x[l], v1);
          else v0 = fmaf(-a[l], x[l], v0);
        }
        x[i] = v0 + v1;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) m[i * kRowF + col] = x[i];
    }
    __syncthreads();
    {   // T_10 and T_32: two warps each, eight columns a warp; W = T_11 A_10 first
      const int J = warp & 2, I1 = J + 1, col = 8 * (warp & 1);
      float* a = M + block_at(I1, J);
      float w[1][4] = {}, r[1][4] = {};
      block_mm<1>(w, M + block_at(I1, I1), a + col, lane);
      __syncthreads();
      block_put<1>(a + col, w, 1.f, lane);
      __syncthreads();
      block_mm<1>(r, a, M + block_at(J, J) + col, lane);
      __syncthreads();
      block_put<1>(a + col, r, -1.f, lane);
    }
    __syncthreads();
    {   // the lower left quarter, block (I2, J2) of it: W = T_BB A_BA, then -W T_AA
      const int I2 = 2 + (warp >> 1), J2 = warp & 1;
      float* o = M + block_at(I2, J2);
      float w[2][4] = {}, r[2][4] = {};
#pragma unroll 1
      for (int m = 2; m <= I2; ++m)
        block_mm<2>(w, M + block_at(I2, m), M + block_at(m, J2), lane);
      __syncthreads();
      block_put<2>(o, w, 1.f, lane);
      __syncthreads();
#pragma unroll 1
      for (int m = J2; m < 2; ++m)
        block_mm<2>(r, M + block_at(I2, m), M + block_at(m, J2), lane);
      __syncthreads();
      block_put<2>(o, r, -1.f, lane);
    }
    __syncthreads();
    {   // T diag(beta) as a pair, over the scratch: the warp's 16 rows, two blocks of
        // 16 columns at a time (the first two are all that the upper rows have)
      const int r = lane & 15, i = 16 * warp + r, hf = lane >> 4;
      F2 x[2][8];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int J = 2 * b + hf;
        if (2 * b > warp) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (J <= warp) {
            v = *reinterpret_cast<const float4*>(M + block_at(warp, J) + r * kRowF + 4 * e);
            const float4 be = *reinterpret_cast<const float4*>(&sh.beta[16 * J + 4 * e]);
            const int j = 16 * J + 4 * e;
            v.x = j <= i ? v.x * be.x : 0.f;
            v.y = j + 1 <= i ? v.y * be.y : 0.f;
            v.z = j + 2 <= i ? v.z * be.z : 0.f;
            v.w = j + 3 <= i ? v.w * be.w : 0.f;
          }
          x[b][2 * e] = pack2(v.x, v.y);
          x[b][2 * e + 1] = pack2(v.z, v.w);
        }
      }
      __syncthreads();
      const uint32_t trow = smem_u32(tile) + i * 128;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
          if (2 * b <= warp) {
#pragma unroll
            for (int e = 0; e < 4; ++e) split2(x[b][4 * q + e], hi[e], lo[e]);
          }
          const uint32_t o = trow + (((4 * b + 2 * hf + q) ^ (i & 7)) << 4);
          sts128(o, make_uint4(hi[0], hi[1], hi[2], hi[3]));
          sts128(o + kBlk, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
      }
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0 && ok) {
      const long long r = (long long)place * p.Hv + h;
      bulk_store(p.rec + r * kRecBytes, smem_u32(tile), kRecBytes);
      bulk_store(p.scal + r, smem_u32(&sh.scal), sizeof(RecScal));
      bulk_commit_group();
    }
    if (hg + 1 < group && tid == 0) bulk_wait_read();   // the next one takes its room
    __syncthreads();
  }
  if (tid == 0) bulk_wait_all();
  if (!ok) {   // the loads and the products may still be on their way
    ok = true;
    wait_w(ok, &sh.full, 0, p.status, p.wait_ns);
    ok = true;
    wait_w(ok, &sh.done, 0, p.status, p.wait_ns);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kPCols);
  }
}

}  // namespace

cudaError_t prepare_delta_prep() {
  return cudaFuncSetAttribute(delta_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem);
}

cudaError_t launch_delta_prep(const PrepParams& p, int chunks, cudaStream_t stream) {
  const double rec = (double)chunks * p.Hv;
  ProfScope ps(PT_DELTA_PREP, stream, 2.0 * 128 * 64 * 128 * (double)chunks * p.Hk,
               rec * (kRecBytes + sizeof(RecScal)) + 32768.0 * chunks * p.Hk);
  if (p.plan)
    return launch_behind(delta_prep_kernel, (unsigned)(chunks * p.Hk), kPThreads, kPSmem, stream, p);
  delta_prep_kernel<<<(unsigned)(chunks * p.Hk), kPThreads, kPSmem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace ttt
