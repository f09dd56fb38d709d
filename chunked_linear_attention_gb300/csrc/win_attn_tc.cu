// Window attention on the tensor cores: bf16, d <= 128.
//
// A block has 256 queries of one head, as two tiles of 128 rows that share the key tiles
// of 64 (win_attn.cuh has the list).  Per key tile and query tile
//     S = Q K^T      (128 x 64, fp32 in TMEM)
//     P = exp2(c S - c m),  l += sum P     (c = scale log2 e; one thread per row)
//     O += P V       (P as bf16 in the TMEM columns that S had)
// with m the row's largest score so far.  O and l are only rescaled, in TMEM, when that has
// grown by more than 8 / c since the last time: until then the weights are at most 2^8 too
// large, and so are their sums.  P is rounded to bf16 (2^-8 of each weight) as the operand
// of the second product; l sums what was not rounded.  As pairs hi + lo of bf16 numbers, with
// twice the second products, outputs are off by 1.7e-3 in the norm where they are by 1.8e-3 now
// (the outputs' own rounding is 1.7e-3), and the case below takes 1013 us for 770.
//
// S lies in two buffers a query tile: while the rows make the weights of one, the products
// fill the other.  Key tiles of 128 with one buffer leave a tile's products and rows waiting
// for one another (2 x 32768 tokens of 12 heads of 128 on 4 key heads, window 2048: 800 us,
// with a product warp for both query tiles 764); of 64 with one product warp 1080 (2780 clocks
// an entry of its own instructions), with one a query tile 780 - 795, and the packed and
// ragged prompts gain 9% from the smaller tiles.  With the rows' products and sums in the packed
// fp32 instructions 761 (heads of 64: 615, without 662); over inputs that pass the L2 767.
//
// What bounds it: 2 x 32768 tokens as above run at 1.04 PFLOP/s of visible pairs, 54% of the
// tensor cores' measured rate.  Per pair of query tiles and 64 keys the products take 1280 clocks (S 384
// each, N 64 being bound by the operands' shared memory, and O 256) and the exponentials 512
// (32 a clock); the rest are the hand-overs and the rows' other instructions: scores from TMEM
// and weights into it, maxima, sums, conversions.
//
// A value that a query does not see still meets its weight 0 in P V, where NaN or
// infinity would spoil the row.  So rows with outputs that are not finite are made again, in
// fp32, from the keys that they see alone (which leaves what is really NaN or infinite): by all
// the block's warps, behind its last item, when no role waits for another.
//
// Roles (384 threads, one block per SM, persistent over (tile pair, head)):
//   warp 0      TMA: Q, and K and V of a key tile together through a ring.
//   warps 1, 3  the products of the first and of the second query tile.
//   warp 2      the list of key tiles, for all others.
//   warps 4-7   rows of the first tile, warps 8-11 of the second: softmax, rescaling,
//               outputs.
#include <atomic>
#include <mutex>

#include "builder.h"
#include "prof.h"
#include "win_rows.cuh"

namespace ttt {

namespace {

constexpr int kM = 128;                  // rows of a tile
constexpr int kKeys = 64;                // keys of a key tile
constexpr int kThreads = 384;

template <int DP>
struct Plan {
  static constexpr int kQ = kM * DP * 2;                     // bytes of a tile of Q
  static constexpr int kKv = kKeys * DP * 2;                 // of K or V
  static constexpr int kStages = 64 * 1024 / kKv;            // of a K and a V each
  static constexpr int kStaging = 8 * 32 * 128;              // 32 rows of 64 outputs a warp
  static constexpr int kSmem = 2 * kQ + 2 * kStages * kKv + kStaging + 1024 + 1024;
};
constexpr int kMostStages = Plan<64>::kStages;
static_assert(Plan<128>::kSmem <= 227 * 1024 && Plan<64>::kSmem <= 227 * 1024, "shared memory");

// What the list warp tells the others: one entry per key tile that either query tile needs.
enum : int {
  kNeed = 1,      // << t: query tile t needs the key tile
  kWhole = 4,     // << t: all its queries see all of it
  kCache = 16,    // the key tile lies in a cache
  kTileEntry = 32,
  kLast = 64,     // of its item
  kStop = 128     // of the block (without kTileEntry: there was none)
};
struct Entry {
  int flags;
  int base, end;       // the key tile: see WinTile
  int i0, b, h;        // the item
  int seq, slot, count, past, head;   // a cache
  int pad;
};
static_assert(sizeof(Entry) == 48, "read 16 bytes at a time");
constexpr int kEntries = 8;
constexpr int kReaders = 11;   // the loads' thread, the products' two warps, eight row warps

struct Bars {
  uint64_t e_full[kEntries], e_free[kEntries];
  uint64_t q_full, q_free;
  uint64_t full[kMostStages], empty[kMostStages];
  uint64_t s_full[2][2], p_full[2][2];   // by query tile and buffer
  uint64_t pv_done[2], o_full[2], o_free[2];
  uint64_t done[2];
  uint32_t tmem;
  int spoiled;   // a row has outputs that are not finite
  int failed;    // a wait ran out
  alignas(16) Entry entry[kEntries];
};
static_assert(sizeof(Bars) <= 1024, "control region");

struct TcParams {
  CUtensorMap q, k, v, ck, cv;
  WinParams w;
  int tiles;            // pairs of query tiles of the token axis
  unsigned items;       // (batch, tile pair, head)
  int wide_out;         // rows of out can be stored 16 bytes at a time
};

// The queries a .. e - 1 of one tile: which key tiles they need, and see in whole.
struct SubTile {
  int a, e, lo, s0, s1;
  int lo_last;   // first key of the last query's window
};

__device__ __noinline__ SubTile sub_tile(const WinParams& p, int b, int a, int e) {
  SubTile s;
  s.a = a;
  s.e = min(e, p.N);
  const WinRow r = win_row(p, b, a);
  s.lo = r.i >= 0 ? r.lo : max(0, a - p.window + 1);
  s.s0 = r.i >= 0 ? r.t0 : 0;
  s.s1 = r.i >= 0 ? r.sink1 : 0;
  s.lo_last = s.a < s.e ? win_row(p, b, s.e - 1).lo : 0;
  return s;
}

__device__ __forceinline__ bool needs(const SubTile& s, const WinTile& t) {
  if (s.a >= s.e) return false;
  if (t.seq >= 0) return max(s.a, t.c.i0) < min(s.e, t.c.i1);
  return t.base < s.e &&
         (t.base + kKeys > s.lo || (t.base < s.s1 && t.base + kKeys > s.s0));
}

// The windows of a tile's queries begin one behind another, so that the last one's and the
// first query bound them all.
__device__ __forceinline__ bool sees_whole(const SubTile& s, const WinTile& t) {
  return t.seq < 0 && t.base >= s.lo_last && t.base + kKeys - 1 <= s.a && t.base + kKeys <= t.end;
}

struct Item {
  int b, h, i0;
};
__device__ __forceinline__ Item get_item(const TcParams& p, unsigned n) {
  Item it;
  const unsigned r = n / (unsigned)p.w.Hq;
  it.h = (int)(n - r * (unsigned)p.w.Hq);
  it.b = (int)(r / (unsigned)p.tiles);
  it.i0 = (int)(r - (unsigned)it.b * (unsigned)p.tiles) * 2 * kM;
  return it;
}

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

// Bounded waits whose slow part is a call: the code that every tile runs has to stay in the
// instruction cache (with everything in line, a third of the time went into fetching it).
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, int* status,
                                       unsigned long long lim) {
  return mbar_wait(bar, parity, status, lim);
}
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, int* status,
                                         unsigned long long lim) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, status, lim);
}
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, int* status,
                                         unsigned long long lim) {
  return __all_sync(0xffffffffu, wait_one(bar, parity, status, lim));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&x);
}

// Bits of the columns x0 .. x1 - 1 among the 32 from `at` on.
__device__ __forceinline__ uint32_t span_bits(int x0, int x1, int at) {
  const int lo = max(x0 - at, 0), hi = min(x1 - at, 32);
  if (lo >= hi) return 0u;
  return (0xffffffffu >> (32 - hi)) & (0xffffffffu << lo);
}

// The entries, read by a whole warp (by one thread: ALONE).
template <bool ALONE>
struct Reader {
  int n;
  __device__ __forceinline__ bool wait(Bars* B, int* status, unsigned long long lim) {
    uint64_t* bar = &B->e_full[n % kEntries];
    const uint32_t ph = (n / kEntries) & 1;
    return ALONE ? wait_one(bar, ph, status, lim) : wait_all(bar, ph, status, lim);
  }
  // 16 bytes of the entry
  __device__ __forceinline__ void part(Bars* B, Entry& e, int i) {
    reinterpret_cast<int4*>(&e)[i] = reinterpret_cast<const int4*>(&B->entry[n % kEntries])[i];
  }
  __device__ __forceinline__ void done(Bars* B) {
    if (!ALONE) __syncwarp();
    if (ALONE || (threadIdx.x & 31) == 0) mbar_arrive(&B->e_free[n % kEntries]);
    ++n;
  }
};

// The spoiled rows of the block's items again.
template <int DP>
__device__ __noinline__ void mend_rows(const TcParams& tp, uint8_t* smem) {
  static_assert(simt_smem<DP, kM>() <= 2 * Plan<DP>::kQ + 2 * Plan<DP>::kStages * Plan<DP>::kKv,
                "in the place of the queries' and keys' tiles");
  for (unsigned item = blockIdx.x; item < tp.items; item += gridDim.x) {
    const Item it = get_item(tp, item);
    for (int t = 0; t < 2; ++t) {
      const int i0 = it.i0 + t * kM;
      __syncthreads();
      if (i0 < tp.w.N)
        window_rows<__nv_bfloat16, DP, kM, true, kThreads / 32, true>(
            tp.w, it.b, it.h, i0, reinterpret_cast<float*>(smem));
    }
  }
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) window_tc_kernel(const __grid_constant__ TcParams tp) {
  using PL = Plan<DP>;
  constexpr int NS = PL::kStages, QB = PL::kQ, TB = PL::kKv, NB = DP / 64;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* Q = smem;
  uint8_t* ring = smem + 2 * QB;
  uint8_t* staging = ring + 2 * NS * TB;
  Bars* B = reinterpret_cast<Bars*>(staging + PL::kStaging);
  const WinParams& p = tp.w;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned long long lim = p.wait_ns;

  if (tid == 0) {
    mbar_init(&B->q_full, 1);
    mbar_init(&B->q_free, 2);   // by the products of both query tiles, as are K and V
    for (int s = 0; s < kEntries; ++s) {
      mbar_init(&B->e_full[s], 1);
      mbar_init(&B->e_free[s], kReaders);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&B->full[s], 1);
      mbar_init(&B->empty[s], 2);
    }
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&B->s_full[t][i], 1);
        mbar_init(&B->p_full[t][i], 4);   // a lane of each warp
      }
      mbar_init(&B->pv_done[t], 1);
      mbar_init(&B->o_full[t], 1);
      mbar_init(&B->o_free[t], 4);
    }
    mbar_init(&B->done[0], 1);
    mbar_init(&B->done[1], 1);
    B->spoiled = B->failed = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&B->tmem, 512);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem;
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      int fills = 0, q_loads = 0;
      bool ok = true, first = true;   // first key tile of an item
      Reader<true> rd{0};
      Entry e;
      while (ok) {
        ok = rd.wait(B, p.status, lim);
        if (!ok) break;
        for (int i = 0; i < 3; ++i) rd.part(B, e, i);
        rd.done(B);
        if (!(e.flags & kTileEntry)) break;
        const int hk = e.h / (p.Hq / p.Hk), s = fills % NS;
        const bool c = e.flags & kCache;
        const CUtensorMap *mk = c ? &tp.ck : &tp.k, *mv = c ? &tp.cv : &tp.v;
        const int w = c ? e.slot : e.b;
        if (p.withhold == 1 && blockIdx.x == 0 && fills == 1) break;
        ok = wait_one(&B->empty[s], ((fills / NS) & 1) ^ 1, p.status, lim);
        if (!ok) break;
        mbar_arrive_expect_tx(&B->full[s], 2 * TB);
        uint8_t* st = ring + s * 2 * TB;
#pragma unroll
        for (int x = 0; x < NB; ++x)
          tma_load_4d(st + x * (kKeys * 128), mk, x * 64, e.base, hk, w, &B->full[s]);
#pragma unroll
        for (int x = 0; x < NB; ++x)
          tma_load_4d(st + TB + x * (kKeys * 128), mv, x * 64, e.base, hk, w, &B->full[s]);
        ++fills;
        if (first) {   // the first keys do not wait for the last item's queries
          ok = wait_one(&B->q_free, (q_loads & 1) ^ 1, p.status, lim);
          if (!ok) break;
          mbar_arrive_expect_tx(&B->q_full, 2 * QB);
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int x = 0; x < NB; ++x)
              tma_load_4d(Q + t * QB + x * (kM * 128), &tp.q, x * 64, e.i0 + t * kM, e.h, e.b, &B->q_full);
          ++q_loads;
        }
        first = e.flags & kLast;
        if (e.flags & kStop) break;
      }
      if (!ok) {   // what is on its way lands before the block ends
        B->failed = 1;
        if (q_loads) wait_one(&B->q_full, (q_loads - 1) & 1, p.status, lim);
        for (int k = 1; k <= NS && k <= fills; ++k)
          wait_one(&B->full[(fills - k) % NS], ((fills - k) / NS) & 1, p.status, lim);
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == 3) {
    // ---------------------------------------------------------------- products
    // A warp for each query tile, so that neither waits for the other's weights (one warp for
    // both took longer over its entries, waits and instructions than the products themselves).
    // S of the tile's key tile j, then O of j - 2: the scores lie in two buffers, so that the
    // rows find the next ones when they are done with a tile.
    const int u = warp >> 1;
    const uint32_t Su = tmem + u * kM, Ou = tmem + 256 + u * kM;
    const uint32_t id_s = idesc_bf16_f32(kKeys, 0, 0), id_o = idesc_bf16_f32(DP, 0, 1);
    const uint64_t qd = smem_desc_sw128(smem_u32(Q + u * QB), 16, 1024);
    const uint64_t kd = smem_desc_sw128(smem_u32(ring), 16, 1024);
    const uint64_t vd = smem_desc_sw128(smem_u32(ring + TB), kKeys * 128, 1024);
    int items = 0;                      // with key tiles
    uint32_t ns = 0, np = 0, no = 0;    // scores made, weights taken; parity of the outputs begun
    bool ok = true;
    bool inside = false, begun = false; // an item; its outputs
    int v0 = -1, v1 = -1;               // stages whose V await their weights
    Reader<false> rd{0};
    auto outputs = [&]() {   // O += P V for v0
      if (!begun) {
        ok = ok && wait_all(&B->o_free[u], no ^ 1, p.status, lim);
        no ^= 1;
      }
      const uint32_t buf = np & 1;
      ok = ok && wait_all(&B->p_full[u][buf], (np >> 1) & 1, p.status, lim);
      if (!ok) return;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < kKeys / 16; ++k)
        umma_ts_w(Ou, Su + buf * kKeys + k * 8, vd + v0 * (2 * TB >> 4) + k * 128, id_o, begun || k != 0);
      umma_commit_w(&B->pv_done[u]);
      ++np;
      begun = true;
    };
    while (ok) {
      // a stage that is full has an entry (the loads' thread read it before): what is left to
      // wait for is the first, for there may be none
      const int ks = rd.n % NS;
      if (rd.n == 0) {
        ok = rd.wait(B, p.status, lim);
        if (!ok || !(B->entry[0].flags & kTileEntry)) break;
      }
      ok = wait_all(&B->full[ks], (rd.n / NS) & 1, p.status, lim);
      if (!ok) break;
      const int flags = *reinterpret_cast<volatile int*>(&B->entry[rd.n % kEntries].flags);
      rd.done(B);
      if (!inside) {
        ok = wait_all(&B->q_full, items & 1, p.status, lim);
        if (!ok) break;
        ++items;
        inside = true;
      }
      tc_fence_after();
      const bool mine = flags & (kNeed << u);
      if (mine) {
        if (v0 >= 0) outputs();
        if (!ok) break;
        const uint32_t buf = ns & 1;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)   // S = Q K^T
          umma_bf16_w(Su + buf * kKeys, qd + (k >> 2) * (kM * 8) + (k & 3) * 2,
                      kd + ks * (2 * TB >> 4) + (k >> 2) * (kKeys * 8) + (k & 3) * 2, id_s, k != 0);
        umma_commit_w(&B->s_full[u][buf]);
        ++ns;
        if (v0 >= 0) umma_commit_w(&B->empty[v0]);
        v0 = v1;
        v1 = ks;
        if (!(flags & kLast)) continue;
      }
      // another's key tile or an item's end: what awaits its weights goes first, for its stage
      // may be in the way of the tiles to come
#pragma unroll 1
      for (int i = 0; i < 2 && ok; ++i) {
        if (v0 >= 0) {
          outputs();
          if (ok) umma_commit_w(&B->empty[v0]);
        }
        v0 = v1;
        v1 = -1;
      }
      if (!ok) break;
      if (!mine) {
        if (lane == 0) mbar_arrive(&B->empty[ks]);
        __syncwarp();
      }
      if (flags & kLast) {
        umma_commit_w(&B->q_free);
        if (begun) umma_commit_w(&B->o_full[u]);
        inside = begun = false;
      }
      if (flags & kStop) break;
    }
    if (!ok) {   // the products under way end before their TMEM is given back
      B->failed = 1;
      umma_commit_w(&B->done[u]);
      wait_all(&B->done[u], 0, p.status, lim);
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- the list
    if (blockIdx.x == 0 && p.starts) {   // reports bounds that are none
      bool bad = false;
      for (int i = lane; i < p.n_seq; i += 32) {
        const int a = p.starts[i], e = p.starts[i + 1];
        bad |= a < 0 || e < a || e > p.N;
      }
      if (bad) report_status(p.status, kStatusBadArg);
    }
    if (lane == 0) {
      int n = 0;
      bool ok = true;
      auto put = [&](const Entry& e) {
        const int s = n % kEntries;
        ok = ok && wait_one(&B->e_free[s], ((n / kEntries) & 1) ^ 1, p.status, lim);
        if (!ok) return;
        const int4* src = reinterpret_cast<const int4*>(&e);
        int4* dst = reinterpret_cast<int4*>(&B->entry[s]);
        dst[0] = src[0];
        dst[1] = src[1];
        dst[2] = src[2];
        mbar_arrive(&B->e_full[s]);
        ++n;
      };
      Entry e = {}, held = {};   // an entry is held back until it is known whether it is a last
      bool holds = false;
      for (unsigned item = blockIdx.x; item < tp.items && ok; item += gridDim.x) {
        const Item it = get_item(tp, item);
        e.b = it.b;
        e.h = it.h;
        e.i0 = it.i0;
        const SubTile s0 = sub_tile(p, it.b, it.i0, it.i0 + kM);
        const SubTile s1 = sub_tile(p, it.b, it.i0 + kM, it.i0 + 2 * kM);
        WinList<kKeys> w = win_list<kKeys>(p, it.b, it.i0, it.i0 + 2 * kM);
        WinTile t;
        bool first = true;
        while (ok && win_next(p, w, t)) {
          const bool n0 = needs(s0, t), n1 = needs(s1, t);
          if (!n0 && !n1) continue;
          if (holds) {
            if (first) held.flags |= kLast;
            put(held);
          }
          first = false;
          e.flags = kTileEntry | (n0 ? kNeed : 0) | (n1 ? kNeed << 1 : 0) |
                    (sees_whole(s0, t) ? kWhole : 0) | (sees_whole(s1, t) ? kWhole << 1 : 0);
          e.base = t.base;
          e.end = t.end;
          if (t.seq >= 0) {
            e.flags |= kCache;
            e.seq = t.seq;
            e.slot = t.c.slot;
            e.count = t.c.count;
            e.past = t.c.past;
            e.head = t.c.head;
          }
          held = e;
          holds = true;
        }
      }
      held.flags |= kLast | kStop;
      put(held);
      if (!ok) B->failed = 1;
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- rows
    const int t = (warp - 4) >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t S = tmem + t * kM + lanes, O = tmem + 256 + t * kM + lanes;
    const float c = p.scale, grow = 8.f / c;
    uint8_t* stage = staging + (warp - 4) * (32 * 128);
    int ns = 0, no = 0;
    bool ok = true, begun = false;   // begun: in this item
    float m = -INFINITY, l = 0.f;   // the row's reference and sum
    int ib = 0, ih = 0, i0 = 0;
    WinRow row;
    row.i = -1;
    bool live = false;
    auto rescale = [&](float to) {
      const float f = to > m ? ex2((m - to) * c) : 1.f;
      m = to;
      l *= f;
      if (!begun) return;
#pragma unroll 1   // rare: what is run for every tile has to stay in the instruction cache
      for (int x = 0; x < DP / 16; ++x) {
        float o[16];
        tmem_ld16_nowait(O + 16 * x, o);
        tmem_wait_bind(o);
        uint32_t ow[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) ow[e] = __float_as_uint(o[e] * f);
        tmem_st16(O + 16 * x, ow);
      }
    };
    Reader<false> rd{0};
    Entry e;
    while (ok) {
      ok = rd.wait(B, p.status, lim);
      if (!ok) break;
      rd.part(B, e, 0);
      if (!begun || (e.flags & kCache)) {
        rd.part(B, e, 1);
        rd.part(B, e, 2);
      }
      rd.done(B);
      if (e.flags & (kNeed << t)) {
        if (!begun) {
          ib = e.b;
          ih = e.h;
          i0 = e.i0;
          m = -INFINITY;
          l = 0.f;
          row = win_row(p, ib, i0 + t * kM + r);
          live = row.i >= 0;
          if (!live) {   // stored nowhere: sees what there is
            row.i = 0x7ffffffe;
            row.lo = row.t0 = row.sink1 = 0;
          }
        }
        const int buf = ns & 1;
        const uint32_t Sb = S + buf * kKeys;
        ok = wait_all(&B->s_full[t][buf], (ns >> 1) & 1, p.status, lim);
        if (!ok) break;
        tc_fence_after();
        float s[2][32];
        tmem_ld32(Sb, s[0]);
        tmem_ld32(Sb + 32, s[1]);
        tmem_wait32(s[0]);
        tmem_wait32(s[1]);
        if (!(e.flags & (kWhole << t))) {
          // up to three spans of columns that the row sees
          int a0, a1, b0, b1, c0 = 0, c1 = 0;
          if (!(e.flags & kCache)) {
            const int top = min(row.i + 1, e.end);
            a0 = row.lo - e.base;
            a1 = top - e.base;
            b0 = row.t0 - e.base;
            b1 = min(row.sink1, top) - e.base;
          } else {
            // places of the ring up to the head are of the newest lap, the others of the one
            // before
            const int x = row.wlo - e.past + e.head, sk = p.sinks;
            a0 = -e.base;
            a1 = min(sk, e.count) - e.base;
            b0 = sk + max(x, 0) - e.base;
            b1 = min(sk + e.head, e.count) - e.base;
            c0 = sk + max(x + p.window, e.head) - e.base;
            c1 = e.count - e.base;
            if (row.seq != e.seq) a1 = b1 = c1 = -1;
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t bits = span_bits(a0, a1, 32 * x) | span_bits(b0, b1, 32 * x) |
                                  span_bits(c0, c1, 32 * x);
            if (!__all_sync(0xffffffffu, bits == 0xffffffffu)) {
#pragma unroll
              for (int y = 0; y < 32; ++y) s[x][y] = bits & (1u << y) ? s[x][y] : -INFINITY;
            }
          }
        }
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < 32; y += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) tops[i] = max3(tops[i], s[x][y + 2 * i], s[x][y + 2 * i + 1]);
        const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
        if (__any_sync(0xffffffffu, top > m + grow)) {
          // the outputs so far are those of all tiles before this one
          if (begun) {
            ok = wait_all(&B->pv_done[t], (ns - 1) & 1, p.status, lim);
            if (!ok) break;
            tc_fence_after();
          }
          rescale(top > m + grow ? top : m);
        }
        ++ns;
        begun = true;
        F2 sum0 = pack2(0.f, 0.f), sum1 = sum0;
        const float mc = m == -INFINITY ? 0.f : m * c;
        const F2 cc = pack2(c, c), mm = pack2(-mc, -mc);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t pw[16];
#pragma unroll
          for (int y = 0; y < 32; y += 4) {
            float v0, v1, v2, v3;
            unpack2(fma2(pack2(s[x][y], s[x][y + 1]), cc, mm), v0, v1);
            unpack2(fma2(pack2(s[x][y + 2], s[x][y + 3]), cc, mm), v2, v3);
            v0 = ex2(v0);
            v1 = ex2(v1);
            v2 = ex2(v2);
            v3 = ex2(v3);
            sum0 = add2(sum0, pack2(v0, v1));
            sum1 = add2(sum1, pack2(v2, v3));
            pw[y / 2] = bf16_pair(v0, v1);
            pw[y / 2 + 1] = bf16_pair(v2, v3);
          }
          tmem_st16(Sb + 16 * x, pw);
        }
        float l0, l1;
        unpack2(add2(sum0, sum1), l0, l1);
        l += l0 + l1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        const bool kept = p.withhold == 2 && blockIdx.x == 0 && t == 0 && ns == 2;
        if (lane == 0 && !kept) mbar_arrive(&B->p_full[t][buf]);
      }
      if ((e.flags & kLast) && begun) {
        begun = false;
        ok = wait_all(&B->o_full[t], no & 1, p.status, lim);
        if (!ok) break;
        ++no;
        tc_fence_after();
        const float f = 1.f / l;
        const int first = i0 + t * kM + (r & ~31);   // the warp's rows
        const unsigned rows = __ballot_sync(0xffffffffu, live);
        __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + ib * p.lay.out.batch +
                            ih * p.lay.out.head + (first + (lane >> 3)) * p.lay.out.token +
                            (lane & 7) * 8;
        const long long step = 4 * p.lay.out.token;
        bool fine = true;
#pragma unroll 1
        for (int y = 0; y < NB; ++y) {   // 64 columns, through shared memory: whole lines are stored
          __syncwarp();
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            float o[16];
            tmem_ld16_nowait(O + 64 * y + 16 * x, o);
            tmem_wait_bind(o);
            uint32_t ow[8];
            float big = 0.f;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              o[i] *= f;
              o[i + 1] *= f;
              big = fmaf(o[i], 0.f, fmaf(o[i + 1], 0.f, big));   // NaN if any is not finite
              ow[i / 2] = bf16_pair(o[i], o[i + 1]);
            }
            fine = fine && big == 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              *reinterpret_cast<uint4*>(stage + lane * 128 + (((2 * x + i) ^ (lane & 7)) << 4)) =
                  make_uint4(ow[4 * i], ow[4 * i + 1], ow[4 * i + 2], ow[4 * i + 3]);
          }
          __syncwarp();
          if (y == NB - 1) {   // the outputs are read: the next item's products may begin
            tc_fence_before();
            if (lane == 0) mbar_arrive(&B->o_free[t]);
          }
          if (64 * y + (lane & 7) * 8 < p.d) {
            __nv_bfloat16* at = to + 64 * y;
#pragma unroll 2
            for (int n = lane >> 3; n < 32; n += 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(stage + n * 128 + (((lane & 7) ^ (n & 7)) << 4));
              if ((rows >> n) & 1) {
                if (tp.wide_out) {
                  *reinterpret_cast<uint4*>(at) = v;
                } else {
                  const __nv_bfloat16* w8 = reinterpret_cast<const __nv_bfloat16*>(&v);
#pragma unroll
                  for (int j = 0; j < 8; ++j) at[j] = w8[j];
                }
              }
              at += step;
            }
          }
        }
        // (a row whose weights are NaN, or all 0, is NaN by what it sees: nothing to mend)
        if (live && !fine && l > 0.f) B->spoiled = 1;
      }
      if (e.flags & kStop) break;
    }
    if (!ok) B->failed = 1;
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (B->spoiled && !B->failed) mend_rows<DP>(tp, smem);
}

std::atomic<int> g_withhold{0};

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
    g_sms[dev] = device_sm_count();
    if (cudaFuncSetAttribute(window_tc_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Plan<64>::kSmem) == cudaSuccess &&
        cudaFuncSetAttribute(window_tc_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Plan<128>::kSmem) == cudaSuccess && g_sms[dev] > 0)
      g_ready[dev] = 1;
  }
  return g_ready[dev] == 1 ? g_sms[dev] : 0;
}

// [B, H, N, d] with the given strides as a map of 64 x `rows` boxes; false where TMA cannot
// take it.
bool win_map(CUtensorMap* m, const void* ptr, const delta_rule_stride& s, long long B, long long H,
             long long N, int d, unsigned rows) {
  const unsigned long long dims[4] = {(unsigned long long)d, (unsigned long long)N,
                                      (unsigned long long)H, (unsigned long long)B};
  // the stride of a dimension of one element is never used: give a valid one
  auto bytes = [](long long x, long long n) { return n > 1 ? (unsigned long long)x * 2 : 16ull; };
  const unsigned long long st[3] = {bytes(s.token, N), bytes(s.head, H), bytes(s.batch, B)};
  for (unsigned long long x : st)
    if (x == 0 || x % 16 != 0 || x >= (1ull << 40)) return false;
  if ((reinterpret_cast<uintptr_t>(ptr) & 15) != 0 || d % 8 != 0) return false;
  const unsigned box[4] = {64, rows, 1, 1};
  return encode_bf16_4d(m, ptr, dims, st, box);
}

}  // namespace

void window_attention_withhold(int what) { g_withhold.store(what); }

int window_attention_tc(const WindowArgs& a) {
  if (!a.bf16 || a.d > 128 || a.d % 8 != 0 || !(a.scale > 0.f)) return 1;
  TcParams p;
  if (!win_map(&p.q, a.q, a.lay.q, a.B, a.Hq, a.N, a.d, kM) ||
      !win_map(&p.k, a.k, a.lay.k, a.B, a.Hk, a.N, a.d, kKeys) ||
      !win_map(&p.v, a.v, a.lay.v, a.B, a.Hk, a.N, a.d, kKeys))
    return 1;
  if (a.past) {
    const long long places = (long long)a.window + a.sinks;
    const delta_rule_stride s = {(long long)a.Hk * places * a.d, places * a.d, a.d};
    if (!win_map(&p.ck, a.cache_k, s, a.n_slots, a.Hk, places, a.d, kKeys) ||
        !win_map(&p.cv, a.cache_v, s, a.n_slots, a.Hk, places, a.d, kKeys))
      return 1;
  } else {
    p.ck = p.k;
    p.cv = p.v;
  }
  const int sms = prepare();
  if (!sms) return TTT_ERR_CUDA;
  p.w = win_params(a);
  p.w.withhold = g_withhold.load();
  p.tiles = (a.N + 2 * kM - 1) / (2 * kM);
  const long long items = (long long)a.B * p.tiles * a.Hq;
  if (items > 0x7fffffff) return 1;
  p.items = (unsigned)items;
  p.wide_out = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && a.lay.out.batch % 8 == 0 &&
               a.lay.out.head % 8 == 0 && a.lay.out.token % 8 == 0;
  const unsigned grid = (unsigned)(items < sms ? items : sms);
  const double tok = (double)a.B * a.N;
  const double seen = a.N < (double)a.window + a.sinks ? a.N * 0.5 : (double)a.window + a.sinks;
  ProfScope ps(PT_WIN_TC, a.stream, 4.0 * tok * a.Hq * a.d * seen, tok * 4.0 * a.d * (a.Hq + a.Hk));
  const cudaError_t e =
      a.d <= 64 ? launch_behind(window_tc_kernel<64>, grid, kThreads, Plan<64>::kSmem, a.stream, p)
                : launch_behind(window_tc_kernel<128>, grid, kThreads, Plan<128>::kSmem, a.stream, p);
  return e == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

}  // namespace ttt
