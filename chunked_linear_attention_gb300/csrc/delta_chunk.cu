// The gated delta rule over whole sequences on the tensor cores: chunks of 64
// tokens, d_k <= 128, 128 rows of the state per CTA.
//
// With G the running sum of g inside a chunk, D_ij = exp(G_i - G_j) (i >= j) and
// S the state before the chunk, the 64 rank-one updates of a chunk are
//     A_ij = beta_i D_ij k_i . k_j  (i > j),   T = (1 + A)^-1 diag(beta)
//     X    = T (V - e^G o K S^T)               (the corrected values)
//     O    = scale (e^G o Q S^T + (D o Q K^T) X)
//     S   <- e^{G_63} S + X^T (e^{G_63 - G} o K)
// delta_prep.cu makes T and D o Q K^T for all chunks at once; here the state runs
// over the chunks.  Everything with the state is kept transposed (rows of S =
// TMEM lanes = d_v), so that S, K S^T and X are TMEM operands of the next product
// and never visit shared memory; q, k, v are used as TMA left them.
//
// Precision: inputs are bf16, but the state that a prompt leaves behind is read
// for thousands of tokens, so no intermediate is rounded to bf16.  Each is held
// as a pair hi + lo of bf16 numbers (16 bits of significand); products of a pair
// with an input take two MMAs, of two pairs three (lo lo is left out).  Sums are
// fp32 and the state itself stays in fp32 registers.
//
// Few long sequences would leave most of the card idle (a chunk follows the one
// before), so they are cut into segments.  A segment maps its start state to
// S P + L; L and P (the rule run on a zero state, and on the unit matrix with
// v = 0) are computed for all segments at once, the start states follow by
// S_{j+1} = S_j P_j + L_j, and all segments run at once.
//
// What bounds it: a chunk's four products follow one another (S K^T, X, X^T K, and
// the state's next pairs), with a conversion by the warps between any two.  A step
// takes 2.25 us, of which the tensor pipe works 47% (2690 cycles of products, in
// pairs); one more order of products to fill the gaps (two MMA warps, other
// hand-overs) was slower.  B 4, H 4, 8192 tokens, d 128: 138 us (prep 33, L and P
// 54, join 14, outputs 47, their ends overlapping), token by token 1.6 ms; one
// sequence of 131072 tokens, 4 heads: 425 us (101, 157, 42, 136).
//
// Roles (512 threads, one CTA per SM, persistent over (segment, head, d_v tile)):
//   warp 0      TMA: q, k, v in three stages, the chunk's records in two.
//   warp 1      all MMAs.
//   warp 2      zeroes the rows behind a sequence's end, so that other
//               sequences' values cannot reach it.
//   warps 4-11  the chain S -> K S^T -> X -> S: warp w has rows 32 (w % 4) .. and half
//               of the columns, and hands them to the MMAs 16 at a time.
//   warps 12-15 the outputs.
#include <atomic>
#include <mutex>

#include "builder.h"
#include "delta_tc.cuh"
#include "prof.h"

namespace ttt {

namespace {

constexpr int kStages = 3;
constexpr int kStageBytes = 6 * kBlk;   // Q0 K0 Q1 K1 V0 V1 (column blocks of 64)

struct Bars {
  uint64_t full[kStages], ready[kStages], empty[kStages];
  uint64_t t_full[2], t_free[2], p_full[2], p_free[2];
  uint64_t ks_full, x_full, ds_full, x_ready;
  uint64_t y_ready[2], xs_ready[2], s_ready[4];
  uint64_t o_full, o_free, done;
  uint32_t tmem;
};

constexpr int kOutBytes = 4 * 32 * 64;
constexpr int kSmem = kStages * kStageBytes + 2 * kRecBytes + 4 * (int)sizeof(RecScal) +
                      kOutBytes + (int)sizeof(Bars) + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");

// TMEM columns
constexpr uint32_t kXu = 0;      // 64: X as a pair
constexpr uint32_t kQS = 64;     // 64: S Q^T
constexpr uint32_t kKS = 128;    // 64: S K^T, then its pair in the same columns
constexpr uint32_t kDS = 128;    // 128: X^T K (after K S^T is used up)
constexpr uint32_t kSh = 256;    // 128: S, for each 16 of d_k 8 columns of hi and 8 of lo
constexpr uint32_t kX = 384;     // 64: X, then e^{G_63 - G} X as a pair
constexpr uint32_t kO = 448;     // 64: P X

constexpr int kPBytes = 65536;
constexpr int kStateFloats = 128 * 128;   // a tile of the state between the kernels

struct ScanParams {
  CUtensorMap q, k, v;
  const SeqPlan* plan;     // packed sequences, or NULL
  const SegPlan* segs;     // likewise, as are
  const int* order;        // the segments' places, a sequence's last ones at the end,
  const int* counts;       // and how many are not a last one, all, and sequences of several
  const uint8_t* rec;
  const RecScal* scal;
  const float* S0;
  const float* Sseg;       // [segment][Hv][tile] start states of the segments
  float* S_final;
  float* L;                // [segment][Hv][tile] (the carry pass)
  uint8_t* P;              // [segment][Hv]: 128 x 128 pairs, as the join's operand tiles
  __nv_bfloat16* out;
  int* status;
  unsigned long long wait_ns;
  delta_rule_stride so;
  int Hk, Hv, N, dk, dv, tiles;
  int seqs, seg_chunks, seg_n;   // not packed: chunks per segment; segments per sequence
  float scale;
  int wide_out;            // rows of out can be stored 16 bytes at a time
  int withhold;            // test hook: the first CTA's second chunk is never ready
};

struct Item {
  int h, tile, batch, t0, len, chunk0;
  const float* from;       // start state [dv][dk] of this head, or NULL
  const float* from_tile;  // or a tile as the join left it
  float* to;               // end state, or NULL
};

// The k-th segment: whole ones first, so that a round of the SMs is of one length;
// the last ones of the sequences (of any length) behind them.
__device__ __forceinline__ SegPlan get_segment(const ScanParams& p, int k, int& place) {
  if (p.segs) {
    place = p.order[k];
    return p.segs[place];
  }
  const int whole = p.seqs * (p.seg_n - 1);
  SegPlan sg;
  sg.n = p.seg_n;
  sg.chunks = p.seg_chunks;
  if (k < whole) {
    sg.seq = k / (p.seg_n - 1);
    sg.j = k - sg.seq * (p.seg_n - 1);
  } else {
    sg.seq = k - whole;
    sg.j = p.seg_n - 1;
  }
  place = sg.seq * p.seg_n + sg.j;
  return sg;
}

// Items of the carry pass (no last segments) and of the outputs' pass.
__device__ __forceinline__ int n_items(const ScanParams& p, bool carry) {
  const int n = p.counts ? p.counts[carry ? 0 : 1] : carry ? p.seqs * (p.seg_n - 1) : p.seqs * p.seg_n;
  return n * p.Hv * p.tiles;
}

// A CTA's items are its places in rounds that go to and fro over the CTAs, so that with
// long items first no CTA gets the longest of every round (24 sequences of 20011
// tokens, 8 heads: 6 us).  The distance to the second item; this and the next one are
// two rounds together.
__device__ __forceinline__ int first_hop() { return 2 * (gridDim.x - 1 - blockIdx.x) + 1; }

// The tokens of a segment, in an item.
__device__ __forceinline__ void set_range(const ScanParams& p, const SegPlan& sg, Item& it) {
  const SeqPlan sp = seq_plan(p.plan, sg.seq, p.N);
  const int before = sg.j * sg.chunks;
  it.batch = p.plan ? 0 : sg.seq;
  it.t0 = sp.t0 + before * kC;
  it.len = sg.j == sg.n - 1 ? sp.len - before * kC : sg.chunks * kC;
  it.chunk0 = sp.chunk0 + before;
}

__device__ __forceinline__ Item get_item(const ScanParams& p, int i) {
  Item it;
  it.tile = i % p.tiles;
  const int sh = i / p.tiles;
  it.h = sh % p.Hv;
  int place;
  const SegPlan sg = get_segment(p, sh / p.Hv, place);
  set_range(p, sg, it);
  it.from = it.from_tile = nullptr;
  it.to = nullptr;
  const long long one = (long long)p.dv * p.dk;
  const long long sqh = (long long)sg.seq * p.Hv + it.h;
  // a sequence of several segments has its S0 from the join too: S_final may be S0,
  // and the last segment's CTA may be done before the first one's has begun
  if (sg.n > 1 && (sg.j > 0 || p.S0))
    it.from_tile =
        p.Sseg + (((long long)place * p.Hv + it.h) * p.tiles + it.tile) * kStateFloats;
  else if (p.S0) it.from = p.S0 + sqh * one;
  if (sg.j == sg.n - 1 && p.S_final) it.to = p.S_final + sqh * one;
  return it;
}

// ---------------------------------------------------------------- wrappers
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* w) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
               "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&w)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// After a wait that ran out: the MMAs that this warp has issued are waited for
// before their TMEM is given back.
__device__ __forceinline__ void drain_mmas(uint64_t* bar, bool el, int* status,
                                           unsigned long long lim) {
  if (el) umma_commit(bar);
  __syncwarp();
  mbar_wait_w(bar, 0, status, lim);
}

template <int R>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// A 128 x 128 state between the kernels, in the order of the threads that hold it
// (row 32 q4 + lane, 64 columns from 64 half, four at a time): a warp's access is
// 512 bytes in one piece, where rows of d_k numbers would be 32 pieces of 16 bytes
// (the join step took 5 us that way).  The float4 of columns 4 c ..:
__device__ __forceinline__ long long state_at(int q4, int half, int c, int lane) {
  return ((q4 * 2 + half) * 16 + c) * 32 + lane;
}

// (C float4 of a row from column 4 C half on: half a row of 8 C columns)
template <int C>
__device__ __forceinline__ void load_state(const float* tile, int q4, int half, int lane,
                                           F2 (&S)[2 * C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int x = C * half + c;
    const ulonglong2 w =
        reinterpret_cast<const ulonglong2*>(tile)[state_at(q4, x >> 4, x & 15, lane)];
    S[2 * c] = w.x;
    S[2 * c + 1] = w.y;
  }
}

template <int C>
__device__ __forceinline__ void store_state(float* tile, int q4, int half, int lane,
                                            const F2 (&S)[2 * C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int x = C * half + c;
    reinterpret_cast<ulonglong2*>(tile)[state_at(q4, x >> 4, x & 15, lane)] =
        make_ulonglong2(S[2 * c], S[2 * c + 1]);
  }
}

// 4 C columns of one row of a user's state (rows of dk numbers, dk a multiple of 8),
// 32 bytes at a time (16 where the tensor begins in the middle of 32); columns from
// dk on are zero.
__device__ __forceinline__ bool at_32(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 31) == 0;
}
template <int C>
__device__ __forceinline__ void load_row(const float* from, int cols, F2 (&S)[2 * C]) {
#pragma unroll
  for (int c = 0; c < C / 2; ++c) {
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (8 * c < cols) {
      if (at_32(from)) {
        ldg256(from + 8 * c, w);
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 x = reinterpret_cast<const uint4*>(from)[2 * c + e];
          w[4 * e] = x.x; w[4 * e + 1] = x.y; w[4 * e + 2] = x.z; w[4 * e + 3] = x.w;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      S[4 * c + e] = pack2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
  }
}
template <int C>
__device__ __forceinline__ void store_row(float* to, int cols, const F2 (&S)[2 * C]) {
#pragma unroll
  for (int c = 0; c < C / 2; ++c) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, b;
      unpack2(S[4 * c + e], a, b);
      w[2 * e] = __float_as_uint(a);
      w[2 * e + 1] = __float_as_uint(b);
    }
    if (8 * c < cols) {
      if (at_32(to)) {
        stg256(to + 8 * c, w);
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          reinterpret_cast<uint4*>(to)[2 * c + e] =
              make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
      }
    }
  }
}

// 16 tokens' values of a row, each times f[token], as pairs at TMEM columns taddr
// (8 of hi, 8 of lo: the operand of one MMA each).
__device__ __forceinline__ void put_scaled(uint32_t taddr, const float (&x)[16], const float* f) {
  uint32_t hi[8], lo[8];
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(f + 2 * e);
    split2(mul2(w.x, pack2(x[2 * e], x[2 * e + 1])), hi[e], lo[e]);
    split2(mul2(w.y, pack2(x[2 * e + 2], x[2 * e + 3])), hi[e + 1], lo[e + 1]);
  }
  tmem_st8(taddr, hi);
  tmem_st8(taddr + 8, lo);
}

// put_scaled with half of the registers at a time.
__device__ __forceinline__ void put_scaled_lean(uint32_t taddr, const float (&x)[16],
                                                const float* f) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(f + 8 * h + 2 * e);
      const int c = 8 * h + 2 * e;
      split2(mul2(w.x, pack2(x[c], x[c + 1])), hi[e], lo[e]);
      split2(mul2(w.y, pack2(x[c + 2], x[c + 3])), hi[e + 1], lo[e + 1]);
    }
    tmem_st4(taddr + 4 * h, hi);
    tmem_st4(taddr + 8 + 4 * h, lo);
  }
}

// The same without a factor.
__device__ __forceinline__ void put_pairs(uint32_t taddr, const float (&x)[16]) {
  uint32_t hi[8], lo[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) split2(pack2(x[2 * e], x[2 * e + 1]), hi[e], lo[e]);
  tmem_st8(taddr, hi);
  tmem_st8(taddr + 8, lo);
}

// 16 TMEM lanes by 16 columns: v[4 b + 2 r + c] is lane lane / 4 + 8 r, column
// 8 b + 2 (lane % 4) + c.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                 "=f"(v[6]), "=f"(v[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_frag(float (&v)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7])
               :
               : "memory");
}
// Four 8 x 8 matrices of 16-bit elements, stored transposed; lane i gives the
// address of row i % 8 (of the stored form) of matrix i / 8.
__device__ __forceinline__ void stmatrix4_t(uint32_t saddr, const uint32_t (&w)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}

// ---------------------------------------------------------------- the kernel
// DK: 128, or 64 for d_k up to 64: a step's state, its pairs and its products with k and
// q are half as many columns (B 2, 32 heads of d 64, 4096 tokens: 132 us, with 128
// columns 153; the carry pass of 4 heads, 131072 tokens: 128 and 154).
template <int DK>
__global__ void __launch_bounds__(512, 1)
    delta_scan_kernel(const __grid_constant__ ScanParams p) {
  constexpr int HC = DK / 2, NB = HC / 16, QK = DK / 64;   // columns of half a row; in 16s; blocks
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* rec = smem + kStages * kStageBytes;
  RecScal* scal = reinterpret_cast<RecScal*>(rec + 2 * kRecBytes);
  uint8_t* obuf = reinterpret_cast<uint8_t*>(scal + 4);   // outputs on their way
  Bars* B = reinterpret_cast<Bars*>(obuf + kOutBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&B->full[s], 1);
      mbar_init(&B->ready[s], 1);
      mbar_init(&B->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&B->t_full[b], 1);
      mbar_init(&B->t_free[b], 1);
      mbar_init(&B->p_full[b], 1);
      mbar_init(&B->p_free[b], 1);
    }
    mbar_init(&B->ks_full, 1);
    mbar_init(&B->x_full, 1);
    mbar_init(&B->ds_full, 1);
    mbar_init(&B->x_ready, 8);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&B->y_ready[b], 8);
      mbar_init(&B->xs_ready[b], 8);
    }
    for (int b = 0; b < NB; ++b) mbar_init(&B->s_ready[b], 8);
    mbar_init(&B->o_full, 1);
    mbar_init(&B->o_free, 4);
    mbar_init(&B->done, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&B->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem;
  pdl_launch_dependents();   // (with TMEM in hand: see launch_behind)
  pdl_wait();
  const int items = n_items(p, false);
  bool ok = true;   // after a wait that ran out: no more waiting, run to the end
  auto wait = [&](uint64_t* bar, uint32_t parity) { wait_w(ok, bar, parity, p.status, p.wait_ns); };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  // (see wait_w)
  auto arrive_if = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(bar);
  };
  auto commit = [&](uint64_t* bar) {
    if (ok) umma_commit(bar);
  };

  if (warp < 4) {
    regs_dec<64>();
    if (warp == 0) {
      int n = 0;
      for (int i = blockIdx.x, hop = first_hop(); i < items && (ok = together(ok));
           i += hop, hop = 2 * gridDim.x - hop) {
        const Item it = get_item(p, i);
        const int hk = it.h / (p.Hv / p.Hk), nc = n_chunks(it.len);
        for (int c = 0; c < nc && (ok = together(ok)); ++c, ++n) {
          const int s = n % kStages, r = n & 1;
          wait(&B->empty[s], ((n / kStages) & 1) ^ 1);
          if (!(ok = together(ok))) break;
          if (lane == 0) {
            uint8_t* st = smem + s * kStageBytes;
            const int t = it.t0 + c * kC;
            mbar_arrive_expect_tx(&B->full[s], (2 * QK + 2) * kBlk);
            for (int b = 0; b < QK; ++b) {
              tma_load_4d(st + (2 * b + 1) * kBlk, &p.k, 64 * b, t, hk, it.batch, &B->full[s]);
              tma_load_4d(st + 2 * b * kBlk, &p.q, 64 * b, t, hk, it.batch, &B->full[s]);
            }
            for (int b = 0; b < 2; ++b)
              tma_load_4d(st + (4 + b) * kBlk, &p.v, 128 * it.tile + 64 * b, t, it.h, it.batch,
                          &B->full[s]);
          }
          __syncwarp();
          // T's two tiles are used up long before the chunk's outputs: a record's
          // halves come and go on their own.  The factors' four places need no
          // barrier: at T(n) the outputs of chunk n - 4 have been read.
          const long long x = (long long)(it.chunk0 + c) * p.Hv + it.h;
          wait(&B->t_free[r], ((n >> 1) & 1) ^ 1);
          if (lane == 0 && ok) {
            mbar_arrive_expect_tx(&B->t_full[r], kRecBytes / 2 + sizeof(RecScal));
            bulk_load_g2s(rec + r * kRecBytes, p.rec + x * kRecBytes, kRecBytes / 2, &B->t_full[r]);
            bulk_load_g2s(scal + (n & 3), p.scal + x, sizeof(RecScal), &B->t_full[r]);
          }
          __syncwarp();
          wait(&B->p_free[r], ((n >> 1) & 1) ^ 1);
          if (lane == 0 && ok) {
            mbar_arrive_expect_tx(&B->p_full[r], kRecBytes / 2);
            bulk_load_g2s(rec + r * kRecBytes + kRecBytes / 2, p.rec + x * kRecBytes + kRecBytes / 2,
                          kRecBytes / 2, &B->p_full[r]);
          }
          __syncwarp();
        }
      }
      {   // copies still on their way into this CTA's shared memory
        ok = together(ok);
        for (int m = n > kStages ? n - kStages : 0; m < n; ++m)
          mbar_wait_w(&B->full[m % kStages], (m / kStages) & 1, p.status, p.wait_ns);
        for (int m = n > 2 ? n - 2 : 0; m < n; ++m) {
          mbar_wait_w(&B->t_full[m & 1], (m >> 1) & 1, p.status, p.wait_ns);
          mbar_wait_w(&B->p_full[m & 1], (m >> 1) & 1, p.status, p.wait_ns);
        }
      }
    } else if (warp == 1) {
      const bool el = elect_lane();
      const uint32_t base = smem_u32(smem), recb = smem_u32(rec);
      const uint32_t id64 = idesc_bf16_f32(64, 0, 0);        // both K-major
      const uint32_t id64m = idesc_bf16_f32(64, 1, 0);       // A = V^T, MN-major
      const uint32_t idk = idesc_bf16_f32(DK, 0, 1);         // B = K^T, MN-major
      int n = 0;
      for (int i = blockIdx.x, hop = first_hop(); i < items && (ok = together(ok));
           i += hop, hop = 2 * gridDim.x - hop) {
        const Item it = get_item(p, i);
        const int nc = n_chunks(it.len);
        for (int c = 0; c < nc && (ok = together(ok)); ++c, ++n) {
          const uint32_t st = base + (n % kStages) * kStageBytes;
          const uint32_t rb = recb + (n & 1) * kRecBytes;
          const uint32_t ph = n & 1;
          const uint64_t th = smem_desc_sw128(rb, 16, 1024);
          const uint64_t tl = smem_desc_sw128(rb + kBlk, 16, 1024);
          // S K^T
          wait(&B->ready[n % kStages], (n / kStages) & 1);
          const uint64_t kd = smem_desc_sw128(st + kBlk, 16, 1024);
#pragma unroll
          for (int b = 0; b < NB; ++b) {   // 16 of each half of d_k at a time
            wait(&B->s_ready[b], ph);
            tc_fence_after();
            if (el) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t a = tmem + kSh + HC * h + 16 * b;
                const uint64_t kb = kd + (DK == 128 ? h * (2 * kBlk / 16) : h * 4) + b * 2;
                umma_ts(tmem + kKS, a + 8, kb, id64, b + h != 0);
                umma_ts(tmem + kKS, a, kb, id64, 1);
              }
              if (b == NB - 1) commit(&B->ks_full);
            }
            __syncwarp();
          }
          // T V, while S K^T is converted (the pairs of S that the chain has made say
          // that the chunk before is done with X's columns)
          wait(&B->t_full[ph], (n >> 1) & 1);
          tc_fence_after();
          if (el) {
            const uint64_t vd = smem_desc_sw128(st + 4 * kBlk, kBlk, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              umma_bf16(tmem + kX, vd + k * 128, tl + k * 2, id64m, k != 0);
              umma_bf16(tmem + kX, vd + k * 128, th + k * 2, id64m, 1);
            }
          }
          __syncwarp();
          // X += T (-e^G K S^T)
#pragma unroll
          for (int b = 0; b < 2; ++b) {   // 16 of each half of the tokens at a time
            wait(&B->y_ready[b], ph);
            tc_fence_after();
            if (el) {
#pragma unroll
              for (int k = b; k < 4; k += 2) {
                const uint32_t y = tmem + kKS + k * 16;
                umma_ts(tmem + kX, y + 8, th + k * 2, id64, 1);
                umma_ts(tmem + kX, y, tl + k * 2, id64, 1);
                umma_ts(tmem + kX, y, th + k * 2, id64, 1);
              }
              if (b == 1) {
                commit(&B->x_full);
                commit(&B->t_free[ph]);
              }
            }
            __syncwarp();
          }
          // S Q^T
          wait(&B->o_free, ph ^ 1);
          tc_fence_after();
          if (el) {
            const uint64_t qd = smem_desc_sw128(st, 16, 1024);
#pragma unroll 4
            for (int k = 0; k < DK / 8; ++k)
              umma_ts(tmem + kQS, tmem + kSh + (k >> 1) * 16 + (k & 1) * 8,
                      qd + (k >> 3) * (2 * kBlk / 16) + ((k >> 1) & 3) * 2, id64, k != 0);
          }
          __syncwarp();
          // X^T K
          const uint64_t km = smem_desc_sw128(st + kBlk, 2 * kBlk, 1024);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            wait(&B->xs_ready[b], ph);
            tc_fence_after();
            if (el) {
#pragma unroll
              for (int k = b; k < 4; k += 2) {
                const uint32_t x = tmem + kX + k * 16;
                umma_ts(tmem + kDS, x + 8, km + k * 128, idk, k != 0);
                umma_ts(tmem + kDS, x, km + k * 128, idk, 1);
              }
              if (b == 1) {
                commit(&B->ds_full);
                commit(&B->empty[n % kStages]);
              }
            }
            __syncwarp();
          }
          // P X
          wait(&B->x_ready, ph);
          wait(&B->p_full[ph], (n >> 1) & 1);
          tc_fence_after();
          if (el) {
            const uint64_t pH = smem_desc_sw128(rb + 2 * kBlk, 16, 1024);
            const uint64_t pL = smem_desc_sw128(rb + 3 * kBlk, 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t x = tmem + kXu + k * 16;
              umma_ts(tmem + kO, x + 8, pH + k * 2, id64, k != 0);
              umma_ts(tmem + kO, x, pL + k * 2, id64, 1);
              umma_ts(tmem + kO, x, pH + k * 2, id64, 1);
            }
            commit(&B->o_full);
            commit(&B->p_free[ph]);
          }
          __syncwarp();
        }
      }
      ok = together(ok);
      if (n > 0) {   // every arrival on this CTA's barriers has landed before it ends
        wait(&B->empty[(n - 1) % kStages], ((n - 1) / kStages) & 1);
        wait(&B->t_free[(n - 1) & 1], ((n - 1) >> 1) & 1);
        wait(&B->p_free[(n - 1) & 1], ((n - 1) >> 1) & 1);
      }
      if (!together(ok)) drain_mmas(&B->done, el, p.status, p.wait_ns);
    } else if (warp == 2) {
      int n = 0;
      for (int i = blockIdx.x, hop = first_hop(); i < items; i += hop, hop = 2 * gridDim.x - hop) {
        const Item it = get_item(p, i);
        const int nc = n_chunks(it.len);
        for (int c = 0; c < nc; ++c, ++n) {
          const int s = n % kStages;
          wait(&B->full[s], (n / kStages) & 1);
          const int valid = min(kC, it.len - c * kC);
          if (valid < kC) {
            const uint32_t st = smem_u32(smem + s * kStageBytes) + valid * 128;
            const int pieces = (kC - valid) * 8;
            for (int b = 0; b < 6; ++b)
              for (int x = lane; x < pieces && (b < 2 * QK || b >= 4); x += 32)
                sts128(st + b * kBlk + x * 16, make_uint4(0, 0, 0, 0));
            fence_proxy_async_smem();
          }
          if (!(p.withhold && blockIdx.x == 0 && n == 1)) arrive_if(&B->ready[s]);
        }
      }
    }
  } else if (warp < 12) {
    // ---- the chain: rows 32 q4 + lane, half of the columns
    regs_inc<168>();
    const int q4 = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
    int n = 0;
    for (int i = blockIdx.x, hop = first_hop(); i < items; i += hop, hop = 2 * gridDim.x - hop) {
      const Item it = get_item(p, i);
      const int nc = n_chunks(it.len);
      const int row = 128 * it.tile + 32 * q4 + lane;
      const long long so = (long long)row * p.dk + HC * half;
      F2 S[HC / 2];
      if (it.from_tile) {
        load_state<HC / 4>(it.from_tile, q4, half, lane, S);
      } else {
        load_row<HC / 4>(it.from + so, it.from && row < p.dv ? p.dk - HC * half : 0, S);
      }
      auto put_S = [&]() {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) split2(S[8 * b + e], hi[e], lo[e]);
          tmem_st8(tl + kSh + HC * half + 16 * b, hi);
          tmem_st8(tl + kSh + HC * half + 16 * b + 8, lo);
          tmem_wait_st();
          tc_fence_before();
          arrive(&B->s_ready[b]);
        }
      };
#pragma unroll 1
      for (int c = 0; c < nc; ++c, ++n) {
        const uint32_t ph = n & 1;
        put_S();
        const RecScal& sc = scal[n & 3];
        float x[2][16];
        wait(&B->t_full[ph], (n >> 1) & 1);
        wait(&B->ks_full, ph);
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t a = tl + kKS + 32 * half + 16 * b;
          tmem_ld16_nowait(a, x[b]);
          tmem_wait_bind(x[b]);
          put_scaled(a, x[b], &sc.neg[32 * half + 16 * b]);
          tmem_wait_st();
          tc_fence_before();
          arrive(&B->y_ready[b]);
        }

        wait(&B->x_full, ph);
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t a = tl + kX + 32 * half + 16 * b;
          tmem_ld16_nowait(a, x[b]);
          tmem_wait_bind(x[b]);
          put_scaled(a, x[b], &sc.er[32 * half + 16 * b]);
          tmem_wait_st();
          tc_fence_before();
          arrive(&B->xs_ready[b]);
        }
        const F2 eall = pack2(sc.eall, sc.eall);
        if (n > 0) wait(&B->o_full, ph ^ 1);   // P X of the chunk before has read X
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < 2; ++b) put_pairs(tl + kXu + 32 * half + 16 * b, x[b]);
        tmem_wait_st();
        tc_fence_before();
        arrive(&B->x_ready);

        wait(&B->ds_full, ph);
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          tmem_ld16_nowait(tl + kDS + HC * half + 16 * b, x[0]);
          tmem_wait_bind(x[0]);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            S[8 * b + e] = fma2(eall, S[8 * b + e], pack2(x[0][2 * e], x[0][2 * e + 1]));
        }
      }
      if (ok && it.to && row < p.dv) store_row<HC / 4>(it.to + so, p.dk - HC * half, S);
    }
  } else {
    // ---- outputs
    regs_dec<104>();
    const int q4 = warp & 3;
    const float nscale = -p.scale;
    const F2 nscale2 = pack2(nscale, nscale);
    const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
    // this warp's 32 tokens x 32 rows of d_v, 64 bytes a token, the 16-byte pieces
    // of a token exchanged by its number
    uint8_t* ob = obuf + q4 * 2048;
    const uint32_t obs = smem_u32(ob);
    int n = 0;
    for (int i = blockIdx.x, hop = first_hop(); i < items; i += hop, hop = 2 * gridDim.x - hop) {
      const Item it = get_item(p, i);
      const int nc = n_chunks(it.len);
      const int col = 128 * it.tile + 32 * q4;
      __nv_bfloat16* out = p.out + it.batch * p.so.batch + it.h * p.so.head +
                           it.t0 * p.so.token + col;
#pragma unroll 1
      for (int c = 0; c < nc; ++c, ++n) {
        const RecScal& sc = scal[n & 3];
        wait(&B->o_full, n & 1);
        tc_fence_after();
        const int valid = ok ? min(kC, it.len - c * kC) : 0;
#pragma unroll 1
        for (int th = 0; th < 2; ++th) {   // 32 tokens at a time
#pragma unroll 2
          for (int b = 0; b < 4; ++b) {    // 16 rows (b & 1) by 16 tokens (b >> 1)
            float x[8], y[8];
            const int t0 = 32 * th + 16 * (b >> 1);
            const uint32_t ta = tl + ((uint32_t)(16 * (b & 1)) << 16) + t0;
            tmem_ld_frag(ta + kQS, x);
            tmem_ld_frag(ta + kO, y);
            uint32_t w[4];
            F2 f[2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
              f[t] = mul2(nscale2,
                          *reinterpret_cast<const F2*>(&sc.neg[t0 + 8 * t + 2 * (lane & 3)]));
            tmem_wait_frag(x);
            tmem_wait_frag(y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {   // tokens 8 (e >> 1) .., rows 8 (e & 1) ..
              const F2 o =
                  fma2(f[e >> 1], pack2(x[2 * e], x[2 * e + 1]), pack2(y[2 * e], y[2 * e + 1]));
              float o0, o1;
              unpack2(o, o0, o1);
              const __nv_bfloat162 r = __floats2bfloat162_rn(o0, o1);
              w[e] = *reinterpret_cast<const uint32_t*>(&r);
            }
            const int t = 16 * (b >> 1) + 8 * (lane >> 4) + (lane & 7);
            const int piece = 2 * (b & 1) + ((lane >> 3) & 1);
            stmatrix4_t(obs + t * 64 + ((piece ^ ((t >> 1) & 3)) << 4), w);
          }
          if (th == 1) {
            tc_fence_before();
            arrive(&B->o_free);
          } else {
            __syncwarp();
          }
          __nv_bfloat16* dst = out + (long long)(c * kC + 32 * th) * p.so.token;
          const int here = valid - 32 * th;
          if (p.wide_out) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int t = 8 * b + (lane >> 2), piece = lane & 3;
              const uint4 w = lds128(obs + t * 64 + ((piece ^ ((t >> 1) & 3)) << 4));
              if (t < here && col + 8 * piece < p.dv)
                *reinterpret_cast<uint4*>(dst + (long long)t * p.so.token + 8 * piece) = w;
            }
          } else {
            const int last = here < 32 ? here : 32;
#pragma unroll 1
            for (int t = 0; t < last; ++t) {
              const __nv_bfloat16 o = *reinterpret_cast<const __nv_bfloat16*>(
                  ob + t * 64 + (((lane >> 3) ^ ((t >> 1) & 3)) << 4) + 2 * (lane & 7));
              if (col + lane < p.dv) dst[(long long)t * p.so.token + lane] = o;
            }
          }
          __syncwarp();
        }
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

// ---------------------------------------------------------------- L and P of the segments
// The chain without outputs, for two units at once: a unit is 128 rows of L (start
// state zero) or the rows of P (start state the unit matrix, v = 0).  The units of
// a (segment, head) share k and T, and while one unit's products run, the other's
// results are converted: the chain's steps wait on one another, and a single one
// leaves the tensor cores idle most of the time (a chunk of two units takes 2.65 us,
// one of one unit with outputs 2.25).
//
// 256 TMEM columns per unit: S as pairs and later X^T K in the same 128 (S itself
// is in registers, and its pairs are used up by then; both take 16 columns per 16
// of d_k), S K^T and its pairs in 64, X and its pairs in 64.
// Warps 4-11 and 12-19 are the units' chains: rows 32 (w % 4) .., half of the columns.
constexpr int kCarryStages = 4;
constexpr int kCarryBytes = 6 * kBlk;   // K0 K1 V0 V1, T hi, T lo
constexpr uint32_t kUnitCols = 256, kUA = 128, kUX = 192;

struct CarryBars {
  uint64_t full[kCarryStages], ready[kCarryStages], empty[kCarryStages];
  uint64_t ks_full[2], y_ready[2], x_full[2], xs_ready[2], ds_full[2], s_ready[2];
  uint64_t done;
  uint32_t tmem;
};
constexpr int kCarrySmem = kCarryStages * (kCarryBytes + (int)sizeof(RecScal)) +
                           (int)sizeof(CarryBars) + 1024;
static_assert(kCarrySmem <= 227 * 1024, "shared memory");

// Unit 0: a tile of L; unit 1: P, beside the first tile.
struct CarryItem {
  Item it;
  long long sgh;           // (segment, head)
};

__device__ __forceinline__ CarryItem get_carry(const ScanParams& p, int i) {
  CarryItem c;
  c.it.tile = i % p.tiles;
  const int sh = i / p.tiles;
  c.it.h = sh % p.Hv;
  int place;
  const SegPlan sg = get_segment(p, sh / p.Hv, place);
  set_range(p, sg, c.it);
  c.sgh = (long long)place * p.Hv + c.it.h;
  return c;
}

template <int DK>
__global__ void __launch_bounds__(640, 1)
    delta_carry_kernel(const __grid_constant__ ScanParams p) {
  constexpr int HC = DK / 2, QK = DK / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  RecScal* scal = reinterpret_cast<RecScal*>(smem + kCarryStages * kCarryBytes);
  CarryBars* B = reinterpret_cast<CarryBars*>(scal + kCarryStages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kCarryStages; ++s) {
      mbar_init(&B->full[s], 1);
      mbar_init(&B->ready[s], 1);
      mbar_init(&B->empty[s], 1 + 16);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&B->ks_full[u], 1);
      mbar_init(&B->y_ready[u], 8);
      mbar_init(&B->x_full[u], 1);
      mbar_init(&B->xs_ready[u], 8);
      mbar_init(&B->ds_full[u], 1);
      mbar_init(&B->s_ready[u], 8);
    }
    mbar_init(&B->done, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&B->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem;
  pdl_launch_dependents();   // (with TMEM in hand: see launch_behind)
  pdl_wait();
  const int items = n_items(p, true);
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) { wait_w(ok, bar, parity, p.status, p.wait_ns); };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  // (see wait_w)
  auto arrive_if = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(bar);
  };
  auto commit = [&](uint64_t* bar) {
    if (ok) umma_commit(bar);
  };

  if (warp < 4) {
    regs_dec<64>();
    if (warp == 0) {
      int n = 0;
      for (int i = blockIdx.x, hop = first_hop(); i < items && (ok = together(ok));
           i += hop, hop = 2 * gridDim.x - hop) {
        const CarryItem ci = get_carry(p, i);
        const int hk = ci.it.h / (p.Hv / p.Hk), nc = n_chunks(ci.it.len);
        for (int c = 0; c < nc; ++c, ++n) {
          const int s = n % kCarryStages;
          wait(&B->empty[s], ((n / kCarryStages) & 1) ^ 1);
          if (!(ok = together(ok))) break;
          if (lane == 0) {
            uint8_t* st = smem + s * kCarryBytes;
            const int t = ci.it.t0 + c * kC;
            const long long x = (long long)(ci.it.chunk0 + c) * p.Hv + ci.it.h;
            mbar_arrive_expect_tx(&B->full[s], (4 + QK) * kBlk + sizeof(RecScal));
            for (int b = 0; b < QK; ++b)
              tma_load_4d(st + b * kBlk, &p.k, 64 * b, t, hk, ci.it.batch, &B->full[s]);
            for (int b = 0; b < 2; ++b)
              tma_load_4d(st + (2 + b) * kBlk, &p.v, 128 * ci.it.tile + 64 * b, t, ci.it.h,
                          ci.it.batch, &B->full[s]);
            bulk_load_g2s(st + 4 * kBlk, p.rec + x * kRecBytes, 2 * kBlk, &B->full[s]);
            bulk_load_g2s(scal + s, p.scal + x, sizeof(RecScal), &B->full[s]);
          }
          __syncwarp();
        }
      }
      ok = together(ok);   // copies still on their way into this CTA's shared memory
      for (int m = n > kCarryStages ? n - kCarryStages : 0; m < n; ++m)
        mbar_wait_w(&B->full[m % kCarryStages], (m / kCarryStages) & 1, p.status, p.wait_ns);
    } else if (warp == 1) {
      const bool el = elect_lane();
      const uint32_t base = smem_u32(smem);
      const uint32_t id64 = idesc_bf16_f32(64, 0, 0);
      const uint32_t id64m = idesc_bf16_f32(64, 1, 0);
      const uint32_t idk = idesc_bf16_f32(DK, 0, 1);
      int n = 0;
      uint32_t nu1 = 0;   // chunks of unit 1
      for (int i = blockIdx.x, hop = first_hop(); i < items && (ok = together(ok));
           i += hop, hop = 2 * gridDim.x - hop) {
        const CarryItem ci = get_carry(p, i);
        const int nc = n_chunks(ci.it.len), units = ci.it.tile == 0 ? 2 : 1;
        for (int c = 0; c < nc && (ok = together(ok)); ++c, ++n) {
          const int s = n % kCarryStages;
          const uint32_t st = base + s * kCarryBytes;
          const uint64_t th = smem_desc_sw128(st + 4 * kBlk, 16, 1024);
          const uint64_t tl = smem_desc_sw128(st + 5 * kBlk, 16, 1024);
          const uint32_t ph[2] = {(uint32_t)n & 1, nu1 & 1};
          wait(&B->ready[s], (n / kCarryStages) & 1);
          // T V, once the chunk before is done with X's columns (behind S K^T, as in the
          // outputs' pass, it is slower here: the other unit's products wait then)
          if (n > 0) wait(&B->ds_full[0], ph[0] ^ 1);
          tc_fence_after();
          if (el) {
            const uint64_t vd = smem_desc_sw128(st + 2 * kBlk, kBlk, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              umma_bf16(tmem + kUX, vd + k * 128, tl + k * 2, id64m, k != 0);
              umma_bf16(tmem + kUX, vd + k * 128, th + k * 2, id64m, 1);
            }
          }
          __syncwarp();
#pragma unroll
          for (int u = 0; u < 2; ++u) {   // S K^T
            if (u >= units) break;
            const uint32_t d = tmem + u * kUnitCols;
            wait(&B->s_ready[u], ph[u]);
            tc_fence_after();
            if (el) {
              const uint64_t kd = smem_desc_sw128(st, 16, 1024);
#pragma unroll
              for (int k = 0; k < DK / 16; ++k) {
                const uint64_t b = kd + (k >> 2) * (kBlk / 16) + (k & 3) * 2;
                umma_ts(d + kUA, d + 16 * k + 8, b, id64, k != 0);
                umma_ts(d + kUA, d + 16 * k, b, id64, 1);
              }
              commit(&B->ks_full[u]);
            }
            __syncwarp();
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {   // X += T (-e^G K S^T)
            if (u >= units) break;
            const uint32_t d = tmem + u * kUnitCols;
            wait(&B->y_ready[u], ph[u]);
            tc_fence_after();
            if (el) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t y = d + kUA + 16 * k;
                umma_ts(d + kUX, y + 8, th + k * 2, id64, u == 0 || k != 0);
                umma_ts(d + kUX, y, tl + k * 2, id64, 1);
                umma_ts(d + kUX, y, th + k * 2, id64, 1);
              }
              commit(&B->x_full[u]);
            }
            __syncwarp();
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {   // X^T K
            if (u >= units) break;
            const uint32_t d = tmem + u * kUnitCols;
            wait(&B->xs_ready[u], ph[u]);
            tc_fence_after();
            if (el) {
              const uint64_t km = smem_desc_sw128(st, kBlk, 1024);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t x = d + kUX + 16 * k;
                umma_ts(d, x + 8, km + k * 128, idk, k != 0);
                umma_ts(d, x, km + k * 128, idk, 1);
              }
              commit(&B->ds_full[u]);
              if (u == units - 1) commit(&B->empty[s]);
            }
            __syncwarp();
          }
          if (units == 2) ++nu1;
        }
      }
      ok = together(ok);
      if (n > 0)   // every arrival on this CTA's barriers has landed before it ends
        wait(&B->empty[(n - 1) % kCarryStages], ((n - 1) / kCarryStages) & 1);
      if (!together(ok)) drain_mmas(&B->done, el, p.status, p.wait_ns);
    } else if (warp == 2) {
      int n = 0;
      for (int i = blockIdx.x, hop = first_hop(); i < items; i += hop, hop = 2 * gridDim.x - hop) {
        const CarryItem ci = get_carry(p, i);
        const int nc = n_chunks(ci.it.len);
        // (segments before a sequence's last one hold whole chunks: nothing to zero)
        for (int c = 0; c < nc; ++c, ++n) {
          wait(&B->full[n % kCarryStages], (n / kCarryStages) & 1);
          if (!(p.withhold && blockIdx.x == 0 && n == 1)) arrive_if(&B->ready[n % kCarryStages]);
        }
      }
    }
  } else {
    regs_inc<104>();
    const int q4 = warp & 3, half = ((warp - 4) >> 2) & 1, u = (warp - 4) >> 3;
    const uint32_t d = tmem + u * kUnitCols + ((uint32_t)(q4 * 32) << 16);
    int n = 0;
    uint32_t m = 0;   // chunks of this unit
    for (int i = blockIdx.x, hop = first_hop(); i < items; i += hop, hop = 2 * gridDim.x - hop) {
      const CarryItem ci = get_carry(p, i);
      const int nc = n_chunks(ci.it.len);
      if (u == 1 && ci.it.tile != 0) {   // no unit here: pass the stages on
        for (int c = 0; c < nc; ++c, ++n) {
          wait(&B->ready[n % kCarryStages], (n / kCarryStages) & 1);
          arrive_if(&B->empty[n % kCarryStages]);
        }
        continue;
      }
      const bool is_p = u == 1;
      const int row = 32 * q4 + lane;
      F2 S[HC / 2];
      {
        const int one = is_p ? row - HC * half : -1;   // this row's column of the unit matrix
#pragma unroll
        for (int c = 0; c < HC / 2; ++c)
          S[c] = pack2(one == 2 * c ? 1.f : 0.f, one == 2 * c + 1 ? 1.f : 0.f);
      }
      auto put_S = [&]() {
#pragma unroll
        for (int b = 0; b < HC / 8; ++b) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(S[4 * b + e], hi[e], lo[e]);
          tmem_st4(d + HC * half + 16 * (b >> 1) + 4 * (b & 1), hi);
          tmem_st4(d + HC * half + 16 * (b >> 1) + 8 + 4 * (b & 1), lo);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(&B->s_ready[u]);
      };
      put_S();
#pragma unroll 1
      for (int c = 0; c < nc; ++c, ++n, ++m) {
        const int s = n % kCarryStages;
        const uint32_t ph = m & 1;
        const RecScal& sc = scal[s];
        wait(&B->ready[s], (n / kCarryStages) & 1);
        wait(&B->ks_full[u], ph);
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t a = d + kUA + 32 * half + 16 * b;
          float x[16];
          tmem_ld16_nowait(a, x);
          tmem_wait_bind(x);
          put_scaled_lean(a, x, &sc.neg[32 * half + 16 * b]);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(&B->y_ready[u]);

        wait(&B->x_full[u], ph);
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t a = d + kUX + 32 * half + 16 * b;
          float x[16];
          tmem_ld16_nowait(a, x);
          tmem_wait_bind(x);
          put_scaled_lean(a, x, &sc.er[32 * half + 16 * b]);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(&B->xs_ready[u]);
        const F2 eall = pack2(sc.eall, sc.eall);
        arrive_if(&B->empty[s]);

        wait(&B->ds_full[u], ph);
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < HC / 16; ++b) {
          float x[16];
          tmem_ld16_nowait(d + HC * half + 16 * b, x);
          tmem_wait_bind(x);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            S[8 * b + e] = fma2(eall, S[8 * b + e], pack2(x[2 * e], x[2 * e + 1]));
        }
        if (c + 1 < nc) put_S();
      }
      if (!ok) continue;
      // (d_k up to 64: what the join reads behind column 64 is zero)
      if (is_p) {   // row of the join's operand tiles: 64 columns a block, hi then lo
        uint8_t* to = p.P + ci.sgh * kPBytes + row * 128;
#pragma unroll
        for (int c = 0; c < HC / 8; ++c) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split2(S[4 * c + e], hi[e], lo[e]);
          const int x = HC / 8 * half + c;
          const int o = (x >> 3) * 16384 + (((x & 7) ^ (row & 7)) << 4);
          *reinterpret_cast<uint4*>(to + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(to + kPBytes / 2 + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          if (DK == 64) {
            *reinterpret_cast<uint4*>(to + 16384 + o) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(to + kPBytes / 2 + 16384 + o) = make_uint4(0, 0, 0, 0);
          }
        }
      } else {
        float* to = p.L + (ci.sgh * p.tiles + ci.it.tile) * kStateFloats;
        store_state<HC / 4>(to, q4, half, lane, S);
        if (DK == 64) {
#pragma unroll
          for (int c = 0; c < HC / 2; ++c) S[c] = 0;
          store_state<HC / 4>(to, q4, 2 + half, lane, S);
        }
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

// ---------------------------------------------------------------- plan of packed sequences
constexpr int kPlanThreads = 256;

// Sum of x over the block's threads before this one; `total` over all.
template <typename I>
__device__ __forceinline__ I block_before(I x, I* part, I& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  I s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();
  if (lane == 31) part[warp] = s;
  __syncthreads();
  I before = 0;
  total = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  return before + s - x;
}

// Chunks per segment, for lengths that only the device knows: the cheapest of 64
// choices from `least` (what the workspace has places for) to the longest sequence, by
// the measured times of make_plan.  nc: this thread's sequence (of at most
// kPlanThreads); units: heads by tiles of d_v.  (8000 tokens in 24 sequences, 16 heads:
// 174 to 183 us with the host's cut, 115 to 157 so; 20011 tokens, 24 sequences, 8 heads:
// 173 to 189 and 144 to 181; the plan takes 8.7 us.)
__device__ __forceinline__ int choose_segments(int nc, int n_seq, int least, int units) {
  constexpr int kChoices = 64;
  constexpr float kSms = 152.f;
  __shared__ int len[kPlanThreads];
  __shared__ float cost[kChoices];
  __shared__ int longest;
  const int lane = threadIdx.x & 31;
  auto choice = [&](int c) {
    const int most = max(longest, least);
    if (c == kChoices - 1) return most;
    const float x = c < 16 ? (float)(least + c) : (float)(least + 16) * exp2f((c - 16) * 0.125f);
    return x < (float)most ? (int)x : most;
  };
  len[threadIdx.x] = nc;
  if (threadIdx.x == 0) longest = 0;
  __syncthreads();
  atomicMax(&longest, nc);
  __syncthreads();
  // eight lanes a choice
#pragma unroll 1
  for (int c = threadIdx.x >> 3; c < kChoices; c += kPlanThreads / 8) {
    const int lc = choice(c);
    float whole = 0.f, left = 0.f, hops = 0.f, most = 0.f;
    for (int s = lane & 7; s < n_seq; s += 8) {
      const int before = max(0, (len[s] - 1) / lc);   // segments before the last one
      const float l = (float)(len[s] - before * lc);
      whole += (float)before;
      left += l + 0.6f;
      hops = fmaxf(hops, (float)before);
      most = fmaxf(most, l);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      whole += __shfl_xor_sync(0xffffffffu, whole, o);
      left += __shfl_xor_sync(0xffffffffu, left, o);
      hops = fmaxf(hops, __shfl_xor_sync(0xffffffffu, hops, o));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    if ((lane & 7) == 0) {
      const float items = whole * units, rounds = ceilf(items / kSms), step = (float)(lc + 1);
      // last segments that find no free SM in the round that the whole ones begin
      const float room = rounds * kSms - items, last = (float)n_seq * units;
      const float behind = items > 0.f && last > room ? fminf(lc, most) * (1.f - room / last) : 0.f;
      const float mean = (items * step + left * units) / kSms;
      // a join's step is 8 CTAs' work, and they take one item after the other
      const float join = fmaxf(hops, 8.f * items / kSms + 0.5f * hops);
      const float steps = fmaxf(fmaxf(rounds * step + behind, 1.03f * mean + 0.5f), most + 0.6f);
      cost[c] = 1.f + 2.25f * steps +
                (items > 0.f ? 5.f + 2.65f * rounds * step + 5.f + join : 4.f);
    }
  }
  __syncthreads();
  int best = cost[lane + 32] < cost[lane] ? lane + 32 : lane;   // by every warp for itself
  float low = cost[best];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, low, o);
    const int c = __shfl_xor_sync(0xffffffffu, best, o);
    if (x < low || (x == low && c < best)) {
      low = x;
      best = c;
    }
  }
  return choice(best);
}

__global__ void __launch_bounds__(kPlanThreads)
    delta_plan_kernel(const int* starts, int n_seq, int N, int chunks, int least, bool split,
                      int units, SeqPlan* plan, SegPlan* segs, int* order, int* joins, int* counts,
                      int* status) {
  __shared__ int part[kPlanThreads / 32];
  __shared__ long long wide_part[kPlanThreads / 32];
  pdl_launch_dependents();
  auto bounds = [&](int s, int& t0, int& len) {
    const int a = starts[s], b = starts[s + 1];
    const bool good = a >= 0 && a <= b && b <= N;
    t0 = good ? a : 0;
    len = good ? b - a : 0;
    return good;
  };
  const bool few = n_seq <= kPlanThreads;   // a thread per sequence
  int t0 = 0, len = 0, seg_chunks = least;
  bool good = true;
  if ((int)threadIdx.x < n_seq) good = bounds(threadIdx.x, t0, len);
  if (split && few) seg_chunks = choose_segments(n_chunks(len), n_seq, least, units);
  int last = -1, left = 0;   // this thread's sequence's last segment and its chunks
  // (sequences that overlap may hold more chunks together than an int can count)
  long long chunk0 = 0;
  int seg0 = 0, join0 = 0;
  for (int s0 = 0; s0 < n_seq; s0 += kPlanThreads) {
    const int s = s0 + (int)threadIdx.x;
    int nc = 0, ns = 0;
    if (s < n_seq) {
      if (s0 > 0) good = bounds(s, t0, len);
      if (!good) report_status(status, -8);
      nc = n_chunks(len);
      ns = max(1, (nc + seg_chunks - 1) / seg_chunks);
    }
    long long tc;
    int ts;
    const long long cb = chunk0 + block_before<long long>(nc, wide_part, tc);
    // bounds that ascend fit always; sequences that overlap (bad bounds between
    // them) may hold more chunks than there are places: those stay empty, and begin
    // behind the last place (the chunks' kernel searches ascending first chunks)
    const bool fits = cb + nc <= chunks;
    if (!fits && s < n_seq) {
      len = 0;
      ns = 1;
    }
    const int sb = seg0 + block_before(ns, part, ts);
    int tj;
    const int jb = join0 + block_before(ns > 1 ? 1 : 0, part, tj);
    if (ns > 1) joins[jb] = sb;   // the place of its first segment
    join0 += tj;
    if (s < n_seq) {
      last = sb + ns - 1;
      left = n_chunks(len) - (ns - 1) * seg_chunks;
      plan[s] = SeqPlan{t0, len, fits ? (int)cb : chunks, 0};
      for (int j = 0; j < ns; ++j) {
        segs[sb + j] = SegPlan{s, j, ns, seg_chunks};
        if (j + 1 < ns) order[sb - s + j] = sb + j;   // s last ones are before it
      }
    }
    chunk0 += tc;
    seg0 += ts;
  }
  // The last segments, behind the whole ones, long ones first: the short ones fill up
  // the rounds.  (Order among equals does not matter to any result.)
  __shared__ int count[kPlanThreads], base[kPlanThreads];
  count[threadIdx.x] = 0;
  __syncthreads();   // segs and plan are written
  const int whole = seg0 - n_seq;
  auto bin = [](int chunks) { return kPlanThreads - 1 - min(chunks, kPlanThreads - 1); };
  auto chunks_of = [&](const SegPlan& sg) {
    return n_chunks(plan[sg.seq].len) - sg.j * seg_chunks;
  };
  if (few) {
    if (last >= 0) atomicAdd(&count[bin(left)], 1);
  } else {
    for (int i = (int)threadIdx.x; i < seg0; i += kPlanThreads) {
      const SegPlan sg = segs[i];
      if (sg.j == sg.n - 1) atomicAdd(&count[bin(chunks_of(sg))], 1);
    }
  }
  __syncthreads();
  int all;
  base[threadIdx.x] = block_before(count[threadIdx.x], part, all);
  __syncthreads();
  if (few) {
    if (last >= 0) order[whole + atomicAdd(&base[bin(left)], 1)] = last;
  } else {
    for (int i = (int)threadIdx.x; i < seg0; i += kPlanThreads) {
      const SegPlan sg = segs[i];
      if (sg.j == sg.n - 1) order[whole + atomicAdd(&base[bin(chunks_of(sg))], 1)] = i;
    }
  }
  if (threadIdx.x == 0) {
    counts[0] = whole;
    counts[1] = seg0;
    counts[2] = join0;
  }
}

// ---------------------------------------------------------------- start states of the segments
// S_{j+1} = S_j P_j + L_j: a CTA takes 128 rows of the state of one (sequence, head)
// through all segments, S as pairs in TMEM, P_j as pairs from the carry pass (64 KB
// by bulk copy, the next one on its way), three products, L_j added in fp32.  For
// sequences of one length (packed ones go by rows, below).
// Warps 0-7: rows 32 (w % 4) .., half of the columns; warp 8: copies and MMAs.
// (A step in fp32 on the CUDA cores took 16 SMs 2.5 us.)
constexpr int kJoinThreads = 288;
constexpr int kJoinSmem = 2 * kPBytes + 256 + 1024;

struct JoinBars {
  uint64_t full[2], s_ready, d_full;
  uint32_t tmem;
};

struct JoinParams {
  const SegPlan* segs;
  const int* joins;
  const int* counts;
  int seqs, seg_n;
  const float* S0;
  const float* L;
  const uint8_t* P;
  float* Sseg;
  int* status;
  unsigned long long wait_ns;
  int Hv, dk, dv, tiles;
  int withhold;            // test hook: the first CTA's second step is never ready
};

__global__ void __launch_bounds__(kJoinThreads, 1)
    delta_join_kernel(const __grid_constant__ JoinParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  JoinBars* B = reinterpret_cast<JoinBars*>(smem + 2 * kPBytes);
  const int tile = blockIdx.x % p.tiles, x = blockIdx.x / p.tiles;
  const int h = x % p.Hv, seq = x / p.Hv, n = p.seg_n, seg0 = seq * n;
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&B->full[0], 1);
    mbar_init(&B->full[1], 1);
    mbar_init(&B->s_ready, 8);
    mbar_init(&B->d_full, 1);
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(&B->tmem, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem;   // 128 columns of S's pairs, 128 of the product
  pdl_launch_dependents();
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) { wait_w(ok, bar, parity, p.status, p.wait_ns); };
  if (warp == 8) {
    const bool el = elect_lane();
    const uint32_t id = idesc_bf16_f32(128, 0, 1);   // B = P, MN-major
    auto load = [&](int j) {
      mbar_arrive_expect_tx(&B->full[j & 1], kPBytes);
      bulk_load_g2s(smem + (j & 1) * kPBytes, p.P + ((long long)(seg0 + j) * p.Hv + h) * kPBytes,
                    kPBytes, &B->full[j & 1]);
    };
    int loaded = 0;
    for (; loaded < 2 && loaded + 1 < n; ++loaded)
      if (el) load(loaded);
    int j = 0;
    for (; j + 1 < n && ok; ++j) {
      const uint32_t pb = smem_u32(smem) + (j & 1) * kPBytes;
      wait(&B->full[j & 1], (j >> 1) & 1);
      wait(&B->s_ready, j & 1);
      if (!(ok = together(ok))) break;
      tc_fence_after();
      if (el) {
        const uint64_t ph = smem_desc_sw128(pb, 16384, 1024);
        const uint64_t pl = smem_desc_sw128(pb + kPBytes / 2, 16384, 1024);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          umma_ts(tmem + 128, tmem + 16 * m + 8, ph + m * 128, id, m != 0);
          umma_ts(tmem + 128, tmem + 16 * m, pl + m * 128, id, 1);
          umma_ts(tmem + 128, tmem + 16 * m, ph + m * 128, id, 1);
        }
        umma_commit(&B->d_full);
      }
      __syncwarp();
      wait(&B->d_full, j & 1);
      ok = together(ok);
      if (ok && loaded + 1 < n) {
        if (el) load(loaded);
        ++loaded;
      }
      __syncwarp();
    }
    if (!ok)   // copies still on their way into this CTA's shared memory
      for (; j < loaded; ++j) mbar_wait_w(&B->full[j & 1], (j >> 1) & 1, p.status, p.wait_ns);
  } else {
    const int q4 = warp & 3, half = warp >> 2;
    const int row = 128 * tile + 32 * q4 + lane;
    const uint32_t t = tmem + ((uint32_t)(q4 * 32) << 16) + 64 * half;
    F2 S[32], L[32];
    load_row<16>(p.S0 + (((long long)seq * p.Hv + h) * p.dv + row) * p.dk + 64 * half,
             p.S0 && row < p.dv ? p.dk - 64 * half : 0, S);
    auto place = [&](int j) { return (((long long)(seg0 + j) * p.Hv + h) * p.tiles + tile) * kStateFloats; };
#pragma unroll 1
    for (int j = 0; j + 1 < n; ++j) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split2(S[8 * b + e], hi[e], lo[e]);
        tmem_st8(t + 16 * b, hi);
        tmem_st8(t + 16 * b + 8, lo);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      const bool withheld = p.withhold && blockIdx.x == 0 && warp == 0 && j == 1;
      if (lane == 0 && ok && !withheld) mbar_arrive(&B->s_ready);
      // beside the product: its 128 KB through the load-store units take as long
      load_state<16>(p.L + place(j), q4, half, lane, L);
      if (ok && (j > 0 || p.S0)) store_state<16>(p.Sseg + place(j), q4, half, lane, S);
      wait(&B->d_full, j & 1);
      tc_fence_after();
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        float d[16];
        tmem_ld16_nowait(t + 128 + 16 * b, d);
        tmem_wait_bind(d);
#pragma unroll
        for (int e = 0; e < 8; ++e) S[8 * b + e] = add2(L[8 * b + e], pack2(d[2 * e], d[2 * e + 1]));
      }
    }
    if (ok) store_state<16>(p.Sseg + place(n - 1), q4, half, lane, S);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// The same for few heads: a CTA takes 16 MT rows, so that a head's step is spread over
// 8 / MT SMs (one SM moves 192 KB in a step above).  Warp w makes columns 16 w .. of the
// next state from S's pairs in shared memory and P's, on mma.sync (tcgen05 has no
// product of 16 rows), and keeps them as fp32; P in three places, two ahead.  A step
// takes 0.95 to 1.05 us (MT = 2: 1.8), bound by the reads of shared memory (the load-store
// pipe 65% busy, the tensor pipe 35%); on the CUDA cores four rows took 1.0, eight 1.8.
constexpr int kRowsThreads = 256;
constexpr int kRowsStages = 3;
constexpr int kRowStride = 136;   // of the pairs' rows: eight of them in eight bank groups

template <int MT>
struct RowsShared {
  uint8_t P[kRowsStages][kPBytes];
  __nv_bfloat16 A[2][2][16 * MT * kRowStride];   // [step & 1][hi, lo]
  uint64_t full[kRowsStages];
};
static_assert(sizeof(RowsShared<2>) <= 227 * 1024, "shared memory");

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int MT>
__global__ void __launch_bounds__(kRowsThreads, 1)
    delta_join_rows_kernel(const __grid_constant__ JoinParams p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  RowsShared<MT>& sh = *reinterpret_cast<RowsShared<MT>*>(smem_raw);
  constexpr int kParts = 8 / MT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int s = 0; s < kRowsStages; ++s) mbar_init(&sh.full[s], 1);
    fence_mbar_init();
  }
  pdl_wait();
  bool ok = true;
  // operand addresses of this lane
  const uint32_t a_at = ((lane & 7) + 8 * ((lane >> 3) & 1)) * kRowStride * 2 + 16 * (lane >> 4);
  const int b_row = (lane & 7) + 8 * ((lane >> 3) & 1), b_chunk = 2 * (warp & 3) + (lane >> 4);
  const uint32_t b_at = (warp >> 2) * 16384 + b_row * 128 + ((b_chunk ^ (b_row & 7)) << 4);
  auto at = [&](int row, int col) {   // in a tile between the kernels
    return (int)state_at(row >> 5, col >> 6, (col & 63) >> 2, row & 31) * 4 + (col & 3);
  };
  const bool small = p.dk <= 64;
  const int items = (p.counts ? p.counts[2] : p.seqs) * p.Hv * p.tiles * kParts;
  int done = 0;     // steps of the items before
  int loaded = 0;   // of P, in all, by thread 0
#pragma unroll 1
  for (int i = blockIdx.x; i < items; i += gridDim.x) {
    const int row0 = 16 * MT * (i % kParts), x = i / kParts;
    const int tile = x % p.tiles, h = x / p.tiles % p.Hv, k0 = x / p.tiles / p.Hv;
    const int seg0 = p.segs ? p.joins[k0] : k0 * p.seg_n;
    const int seq = p.segs ? p.segs[seg0].seq : k0, n = p.segs ? p.segs[seg0].n : p.seg_n;
    auto load = [&](int j) {   // d_k up to 64: the first quarter of hi and of lo
      uint64_t* bar = &sh.full[loaded % kRowsStages];
      uint8_t* to = sh.P[loaded % kRowsStages];
      const uint8_t* from = p.P + ((long long)(seg0 + j) * p.Hv + h) * kPBytes;
      if (p.withhold && blockIdx.x == 0 && loaded == 1) {
        ++loaded;
        return;
      }
      mbar_arrive_expect_tx(bar, small ? 2 * kBlk : kPBytes);
      if (small) {
        bulk_load_g2s(to, from, kBlk, bar);
        bulk_load_g2s(to + kPBytes / 2, from + kPBytes / 2, kBlk, bar);
      } else {
        bulk_load_g2s(to, from, kPBytes, bar);
      }
      ++loaded;
    };
    __syncthreads();   // everyone is done with the item before, and sees the barriers
    if (tid == 0 && ok) {
      if (done > 0) fence_proxy_async_smem();
      while (loaded < done + kRowsStages && loaded + 1 < done + n) load(loaded - done);
    }
    auto place = [&](int j) {
      return (((long long)(seg0 + j) * p.Hv + h) * p.tiles + tile) * kStateFloats;
    };
    // this thread's numbers: rows r, r + 8 of each 16, two columns of each 8
    const int r = row0 + (lane >> 2), c = 16 * warp + 2 * (lane & 3);
    F2 S[MT][2][2];   // [16 rows][8 columns][8 rows]
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = r + 16 * m + 8 * e, col = c + 8 * t, grow = 128 * tile + row;
          float2 s = make_float2(0.f, 0.f);
          if (p.S0 && grow < p.dv && col < p.dk)   // (d_k is even)
            s = *reinterpret_cast<const float2*>(
                p.S0 + (((long long)seq * p.Hv + h) * p.dv + grow) * p.dk + col);
          S[m][t][e] = pack2(s.x, s.y);
          if (p.S0) *reinterpret_cast<F2*>(p.Sseg + place(0) + at(row, col)) = S[m][t][e];
        }
#pragma unroll 1
    for (int j = 0; j + 1 < n; ++j, ++done) {
      F2 L[MT][2][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = r + 16 * m + 8 * e, col = c + 8 * t;
            L[m][t][e] = *reinterpret_cast<const F2*>(p.L + place(j) + at(row, col));
            uint32_t hi, lo;
            split2(S[m][t][e], hi, lo);
            const int o = (row - row0) * kRowStride + col;
            *reinterpret_cast<uint32_t*>(&sh.A[done & 1][0][o]) = hi;
            *reinterpret_cast<uint32_t*>(&sh.A[done & 1][1][o]) = lo;
          }
      __syncthreads();
      // everyone is done with the step before: its P's place takes the next one
      if (tid == 0 && ok && j > 0 && loaded - done + j + 1 < n) {
        fence_proxy_async_smem();
        load(loaded - done + j);
      }
      wait_w(ok, &sh.full[done % kRowsStages], (done / kRowsStages) & 1, p.status, p.wait_ns);
      const uint32_t P = smem_u32(sh.P[done % kRowsStages]) + b_at;
      const uint32_t Ah = smem_u32(sh.A[done & 1][0]) + a_at, Al = smem_u32(sh.A[done & 1][1]) + a_at;
      float acc[MT][2][3][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][t][q][e] = 0.f;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (small && (k == 4 || warp >= 4)) break;   // zeros
        uint32_t bh[4], bl[4];
        ldmatrix4_t(bh, P + k * 16 * 128);
        ldmatrix4_t(bl, P + kPBytes / 2 + k * 16 * 128);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t ah[4], al[4];
          ldmatrix4(ah, Ah + (16 * m * kRowStride + 16 * k) * 2);
          ldmatrix4(al, Al + (16 * m * kRowStride + 16 * k) * 2);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            mma_bf16(acc[m][t][0], al, bh[2 * t], bh[2 * t + 1]);
            mma_bf16(acc[m][t][1], ah, bl[2 * t], bl[2 * t + 1]);
            mma_bf16(acc[m][t][2], ah, bh[2 * t], bh[2 * t + 1]);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float(&q)[3][4] = acc[m][t];
            const F2 low =
                add2(pack2(q[0][2 * e], q[0][2 * e + 1]), pack2(q[1][2 * e], q[1][2 * e + 1]));
            S[m][t][e] = add2(L[m][t][e], add2(low, pack2(q[2][2 * e], q[2][2 * e + 1])));
            if (ok)
              *reinterpret_cast<F2*>(p.Sseg + place(j + 1) + at(r + 16 * m + 8 * e, c + 8 * t)) =
                  S[m][t][e];
          }
    }
  }
  // copies still on their way into this CTA's shared memory
  if (tid == 0 && !ok)
    for (int j = loaded > kRowsStages ? loaded - kRowsStages : 0; j < loaded; ++j)
      mbar_wait(&sh.full[j % kRowsStages], (j / kRowsStages) & 1, p.status, p.wait_ns);
}

template <int MT>
cudaError_t launch_rows(const JoinParams& j, int sms, cudaStream_t stream) {
  const long long items = (long long)j.seqs * j.Hv * j.tiles * (8 / MT);
  return launch_behind(delta_join_rows_kernel<MT>, (unsigned)(items < sms ? items : sms),
                       kRowsThreads, sizeof(RowsShared<MT>), stream, j);
}

std::atomic<int> g_withhold{0};   // test hook: 1 prep, 2 L and P, 3 join, 4 outputs

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
    auto room = [](auto kern, size_t bytes) {
      return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) ==
             cudaSuccess;
    };
    if (room(delta_scan_kernel<64>, kSmem) && room(delta_scan_kernel<128>, kSmem) &&
        room(delta_carry_kernel<64>, kCarrySmem) && room(delta_carry_kernel<128>, kCarrySmem) &&
        room(delta_join_kernel, kJoinSmem) &&
        room(delta_join_rows_kernel<1>, sizeof(RowsShared<1>)) &&
        room(delta_join_rows_kernel<2>, sizeof(RowsShared<2>)) &&
        prepare_delta_prep() == cudaSuccess &&
        cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
      g_ready[dev] = 1;
    cudaGetLastError();
  }
  return g_ready[dev] == 1 ? g_sms[dev] : 0;
}

constexpr int kSms = 152;   // for the plan of a call, which must not need a device

// How a call is cut, and where its workspace holds what.
struct Plan {
  int chunks;        // places of records per head
  int seg_chunks, seg_n, seg_places;
  bool split;
  size_t plan, segs, lists, scal, rec, L, P, Sseg, total;
};

Plan make_plan(int B, int Hv, int N, int dk, int dv, int n_seq, bool packed) {
  Plan p;
  const int tiles = (dv + 127) / 128;
  const int nc = n_chunks(N);
  p.chunks = packed ? N / kC + n_seq : B * nc;
  // Chunks per segment, from measured times in us: a step with outputs 2.25 and one
  // of L and P 2.65, on one SM; a join step 1.0 with 16 rows per CTA, 1.8 with 32, 2.3 by
  // tiles; beginnings 1 (most of it beside the kernel before), 5, 5 and, by tiles, 10.
  // 1024 tokens take 41.0 us in segments and 47.4 whole with 4 heads, 55.2 and 53.5 with
  // 32; 4096 tokens 82 (nine segments) and 100 (five) with 16 heads, 181 and 191 (whole)
  // with 48.
  const long long units = (long long)(packed ? 1 : B) * Hv * tiles;
  const double join = packed || units * 8 <= kSms ? 1.0 : units * 4 <= kSms ? 1.8 : 2.3;
  auto rounds = [](double items) { return (double)(long long)((items + kSms - 1) / kSms); };
  double best = 0.0;
  p.seg_chunks = nc;
  for (int n = 1; n <= 128 && n <= nc; ++n) {
    const int lc = (nc + n - 1) / n;
    double t, hops = n - 1;
    if (!packed) {   // sequences of one length: whole rounds of the SMs
      t = 1.0 + 2.25 * rounds((double)units * n) * (lc + 1);
      if (n > 1) t += 5.0 + 2.65 * rounds((double)units * (n - 1)) * (lc + 1);
    } else {
      // lengths unknown: of n_seq sequences half a segment is left over each, and the
      // longest is about four times the mean.  The plan kernel sees them and may cut
      // longer segments (choose_segments); the workspace holds the ones of this cut.
      const double longest = n_seq > 4 ? 4.0 * nc / n_seq : nc;
      double whole = (double)nc / lc - 0.5 * n_seq;
      hops = longest / lc;
      if (whole < hops) whole = hops;
      if (hops < 1.0) whole = 0.0;
      const double left = longest < lc ? longest : 0.75 * lc + 1.5;
      t = 1.0 + 2.25 * (rounds(units * whole) * (lc + 1) + rounds((double)units * n_seq) * left);
      if (whole > 0.0) t += 5.0 + 2.65 * rounds(units * whole) * (lc + 1);
    }
    if (hops >= 1.0) t += (join > 2.0 ? 10.0 : 5.0) + join * hops;
    if (n == 1 || t < best) {
      best = t;
      p.seg_chunks = lc;
    }
  }
  p.seg_n = (nc + p.seg_chunks - 1) / p.seg_chunks;
  p.split = p.seg_n > 1;
  p.seg_places = packed ? p.chunks / p.seg_chunks + n_seq : B * p.seg_n;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  p.plan = take(packed ? (size_t)n_seq * sizeof(SeqPlan) : 0);
  p.segs = take(packed ? (size_t)p.seg_places * sizeof(SegPlan) : 0);
  p.lists = take(packed ? ((size_t)p.seg_places + n_seq + 4) * sizeof(int) : 0);
  p.scal = take((size_t)p.chunks * Hv * sizeof(RecScal));
  p.rec = take((size_t)p.chunks * Hv * kRecBytes);
  const size_t sh = p.split ? (size_t)p.seg_places * Hv : 0;
  p.L = take(sh * tiles * kStateFloats * 4);
  p.P = take(sh * kPBytes);
  p.Sseg = take(sh * tiles * kStateFloats * 4);
  p.total = off;
  return p;
}

}  // namespace

bool delta_map(CUtensorMap* m, const void* ptr, const delta_rule_stride& s, int B, int H, int N,
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

void delta_rule_withhold(int kernel) { g_withhold.store(kernel); }

size_t delta_rule_chunk_workspace(int B, int Hv, int N, int dk, int dv, int n_seq) {
  if (dk > 128 || dk % 8 != 0 || dv % 8 != 0) return 0;
  size_t need = 0;
  if (B == 1) need = make_plan(B, Hv, N, dk, dv, n_seq, true).total;
  if (n_seq == B) {
    const size_t dense = make_plan(B, Hv, N, dk, dv, n_seq, false).total;
    need = dense > need ? dense : need;
  }
  return need;
}

int delta_rule_chunk_launch(const DeltaArgs& a) {
  if (!a.bf16 || a.dk > 128) return 1;
  // A few tokens of a few heads are done sooner token by token, in one launch (16
  // heads: 32 tokens 14.4 us, here 16.4; 48 tokens 16.4 and 16.5; 64 tokens 20.5 and
  // 16.4; with more CTAs than SMs it is slower from 16 tokens on).
  if (a.N <= 40 && (long long)a.n_seq * a.Hv * ((a.dv + 15) / 16) <= kSms) return 1;
  PrepParams r;
  ScanParams p;
  if (!delta_map(&p.q, a.q, a.lay.q, a.B, a.Hk, a.N, a.dk) ||
      !delta_map(&p.k, a.k, a.lay.k, a.B, a.Hk, a.N, a.dk) ||
      !delta_map(&p.v, a.v, a.lay.v, a.B, a.Hv, a.N, a.dv))
    return 1;
  const int sms = prepare();
  if (!sms) return TTT_ERR_CUDA;
  const bool packed = a.seq_starts != nullptr;
  const Plan pl = make_plan(a.B, a.Hv, a.N, a.dk, a.dv, a.n_seq, packed);
  char* ws = static_cast<char*>(a.workspace);
  SeqPlan* plan = packed ? reinterpret_cast<SeqPlan*>(ws + pl.plan) : nullptr;
  SegPlan* segs = packed ? reinterpret_cast<SegPlan*>(ws + pl.segs) : nullptr;

  r.q = p.q; r.k = p.k;
  r.g = a.g; r.beta = a.beta;
  r.plan = plan;
  r.n_seq = a.n_seq;
  r.Hk = a.Hk; r.Hv = a.Hv; r.N = a.N; r.dk = a.dk;
  r.sg = a.lay.g; r.sb = a.lay.beta;
  r.scale = a.scale;
  r.rec = reinterpret_cast<uint8_t*>(ws + pl.rec);
  r.scal = reinterpret_cast<RecScal*>(ws + pl.scal);
  r.status = a.status;
  r.wait_ns = a.wait_ns;
  const int withhold = g_withhold.load(std::memory_order_relaxed);
  r.withhold = withhold == 1;

  p.plan = plan;
  p.segs = segs;
  int* counts = packed ? reinterpret_cast<int*>(ws + pl.lists) : nullptr;
  int* joins = packed ? counts + 4 : nullptr;
  int* order = packed ? joins + a.n_seq : nullptr;
  p.counts = counts;
  p.order = order;
  p.seqs = a.n_seq;
  p.rec = r.rec;
  p.scal = r.scal;
  p.S0 = a.S0;
  p.S_final = a.S_final;
  p.L = reinterpret_cast<float*>(ws + pl.L);
  p.P = reinterpret_cast<uint8_t*>(ws + pl.P);
  float* Sseg = reinterpret_cast<float*>(ws + pl.Sseg);
  p.Sseg = Sseg;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.status = a.status;
  p.wait_ns = a.wait_ns;
  p.so = a.lay.out;
  p.Hk = a.Hk; p.Hv = a.Hv; p.N = a.N; p.dk = a.dk; p.dv = a.dv;
  p.tiles = (a.dv + 127) / 128;
  p.seg_chunks = pl.seg_chunks;
  p.seg_n = pl.seg_n;
  p.scale = a.scale;
  p.wide_out = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && a.lay.out.batch % 8 == 0 &&
               a.lay.out.head % 8 == 0 && a.lay.out.token % 8 == 0;

  const double tok = (double)a.B * a.N;
  if (packed) {
    ProfScope ps(PT_DELTA_PLAN, a.stream, 0.0, 20.0 * a.n_seq);
    delta_plan_kernel<<<1, kPlanThreads, 0, a.stream>>>(a.seq_starts, a.n_seq, a.N, pl.chunks,
                                                        pl.seg_chunks, pl.split, a.Hv * p.tiles,
                                                        plan, segs, order, joins, counts, a.status);
    if (cudaGetLastError() != cudaSuccess) return TTT_ERR_CUDA;
  }
  if (launch_delta_prep(r, pl.chunks, a.stream) != cudaSuccess) return TTT_ERR_CUDA;
  if (pl.split) {
    {
      p.withhold = withhold == 2;
      const int items = (packed ? pl.seg_places : a.B * (pl.seg_n - 1)) * a.Hv * p.tiles;
      ProfScope ps(PT_DELTA_CARRY, a.stream, 5.0 * tok * a.Hv * a.dk * (a.dv + a.dk),
                   tok * 2.0 * (a.Hk * a.dk + a.Hv * a.dv));
      if (launch_behind(a.dk > 64 ? delta_carry_kernel<128> : delta_carry_kernel<64>, items < sms ? items : sms, 640, kCarrySmem, a.stream, p) !=
          cudaSuccess)
        return TTT_ERR_CUDA;
    }
    JoinParams j;
    j.segs = segs;
    j.joins = joins;
    j.counts = counts;
    j.seqs = a.n_seq;
    j.seg_n = pl.seg_n;
    j.S0 = a.S0;
    j.L = p.L;
    j.P = p.P;
    j.Sseg = Sseg;
    j.status = a.status;
    j.wait_ns = a.wait_ns;
    j.Hv = a.Hv; j.dk = a.dk; j.dv = a.dv;
    j.tiles = p.tiles;
    j.withhold = withhold == 3;
    const double states = (double)pl.seg_places * a.Hv * a.dk;
    ProfScope ps(PT_DELTA_JOIN, a.stream, 2.0 * states * a.dk * a.dv,
                 4.0 * states * (a.dk + 2 * a.dv));
    // by rows where that still fits the card at once, and for packed sequences, of which
    // a few long ones have most of the steps (5 sequences of 20011 tokens, 8 heads: 173 to
    // 177 us, by tiles 185 to 199; 64 sequences of 30000, 4 heads: 111 to 150 and 113 to 147)
    const long long tiles = (long long)a.n_seq * a.Hv * p.tiles;
    const cudaError_t e =
        packed || tiles * 8 <= sms ? launch_rows<1>(j, sms, a.stream)
        : tiles * 4 <= sms         ? launch_rows<2>(j, sms, a.stream)
                                       : launch_behind(delta_join_kernel, (unsigned)tiles, kJoinThreads,
                                                       kJoinSmem, a.stream, j);
    if (e != cudaSuccess) return TTT_ERR_CUDA;
  }
  const int items = pl.seg_places * a.Hv * p.tiles;
  p.withhold = withhold == 4;
  ProfScope ps(PT_DELTA_CHUNK, a.stream, 7.0 * tok * a.Hv * a.dk * a.dv,
               tok * 4.0 * (a.Hk * a.dk + a.Hv * a.dv));
  return launch_behind(a.dk > 64 ? delta_scan_kernel<128> : delta_scan_kernel<64>, items < sms ? items : sms, 512, kSmem, a.stream, p) ==
                 cudaSuccess
             ? TTT_OK
             : TTT_ERR_CUDA;
}

}  // namespace ttt
