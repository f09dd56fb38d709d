// The selective state space scan: whole sequences, and single tokens on a pool of
// states.  Per channel, with a state h of S numbers and r = softplus(dt + bias),
//     h <- exp(r A) h + r x B_t,   y_t = (C_t . h + Dx x) z sigmoid(z).
//
// The channels are independent; so are the numbers of a state until y sums over them.
// A thread holds CPT neighbouring channels x SPT numbers of the state, and L lanes one
// channel's state.  Per token four warps run the recurrence on r, r x, B and C as fp32 in
// shared memory; four others bring the next tile of them there and turn the last tile's sums
// into outputs (one kind of warp for both, 1048 us where this takes 838).  With A' = A
// log2(e) each element of the state costs one base-2 exponential and four fp32 operations,
// issued in pairs.
//
// What bounds it: issue.  2 x 32768 tokens of 1536 x 16, bf16: 828 us, the carry 330 of them;
// the exponentials of both passes alone would take 344 us (32 a clock and SM), the bytes of
// the output pass 119.  A (token, channel) takes 84 lane-instructions of the carry and 124 of
// the outputs, and 62% of the clocks issue one a scheduler.
//
// Few long sequences would leave most of the card idle (a token follows the one
// before), so the token axis is cut into segments.  A segment maps the state that it
// begins with to exp(R A) h + l, with R the sum of its r and l its end state from
// zero; the carry pass finds l and R for all segments at once, the join pass the states at
// the segments' starts one after the other, and the output pass runs all segments at
// once.  The carry makes every exponential twice; it is taken where the channels alone
// do not fill the card (scan_shape).
//
// Packed sequences lie on the token axis as they are: a segment in which a sequence
// begins ends with a state that knows nothing of what came before the segment.
#include <climits>

#include "mixers.cuh"
#include "mixers.h"
#include "prof.h"

namespace ttt {

namespace {

constexpr int kScanThreads = 128;
constexpr int kScanSms = 152;
constexpr float kLog2e = 1.44269504088896341f;

struct ScanParams {
  const void* x;
  const void* dt;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* Dx;
  const float* dt_bias;
  const void* z;
  const float* state_in;
  const int* starts;
  void* out;
  float* state_out;
  float* seg_state;    // [B][segs][D][S]: end states from zero, then start states
  float* seg_sum;      // [B][segs][D]: sums of r, for exp(R A)
  int* seg_new;        // [B][segs]: a sequence begins, or a token is in none, in the segment
  int* status;
  int n_seq, N, D, S, G, segs, seg_tokens, blocks;   // channel blocks per group
  int softplus;
  selective_scan_layout lay;
};

template <int L>
__device__ __forceinline__ float sum_over(float x) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sums of CPT channels over L lanes, spread over the lanes where there are four channels:
// each step sends the half that the other lane goes on with.  Lane l ends with
// `kept` channels from own_first on (all lanes above the fourth hold copies).
template <int CPT, int L>
struct LaneSums {
  static constexpr int kept = CPT == 1 || L >= 4 ? 1 : CPT / L;
  __device__ static __forceinline__ int own_first(int l) {
    if (CPT == 1 || L == 1) return 0;
    return L == 2 ? 2 * l : 2 * (l & 1) + ((l >> 1) & 1);
  }
  __device__ static __forceinline__ bool writes(int l) { return CPT == 1 ? l == 0 : l < 4; }
  __device__ static __forceinline__ void sum(const float (&v)[CPT], int l, float (&y)[kept]) {
    if constexpr (CPT == 1) {
      y[0] = sum_over<L>(v[0]);
    } else if constexpr (L == 1) {
#pragma unroll
      for (int i = 0; i < CPT; ++i) y[i] = v[i];
    } else {
      const bool hi = l & 1;
      const float a = (hi ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 1);
      const float c = (hi ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 1);
      if constexpr (L == 2) {
        y[0] = a;
        y[1] = c;
      } else {
        const bool up = l & 2;
        float s = (up ? c : a) + __shfl_xor_sync(0xffffffffu, up ? a : c, 2);
#pragma unroll
        for (int o = 4; o < L; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        y[0] = s;
      }
    }
  }
};

// Tokens of a tile, and bytes of shared memory: two tiles of r and r x, B and C.
template <int CPT, int L>
constexpr int scan_tile() {
  return kScanThreads / L * CPT > 256 ? 8 : 16;
}
template <int CPT, int SPT, int L, bool CARRY>
constexpr int scan_smem() {
  return 2 * scan_tile<CPT, L>() * (kScanThreads / L * CPT * 8 + (CARRY ? 1 : 2) * SPT * L * 4);
}

// The tiles of a segment: tokens t .. t + m - 1 of one sequence.
struct ScanTile {
  int t, m, seq;    // m 0: no more
  bool first, last; // of the sequence
};

struct ScanTiles {
  int t, end;
  TokenSeq sq;
  bool fresh;       // the state knows nothing of what came before the segment
};

template <int TILE>
__device__ __forceinline__ ScanTile next_tile(const ScanParams& p, ScanTiles& w, int b) {
  ScanTile r;
  r.t = w.t;
  r.m = 0;
  r.seq = -1;
  r.first = r.last = false;
  while (w.t < w.end) {
    if (w.t >= w.sq.t1) {
      w.sq = token_seq(p.starts, p.n_seq, b, p.N, w.t);
      if (w.sq.seq < 0) {
        w.sq.t1 = 0;
        w.fresh = true;
        // before the first and behind the last sequence in one go
        if (w.t < p.starts[0]) w.t = min(w.end, p.starts[0]);
        else if (w.t >= p.starts[p.n_seq]) w.t = w.end;
        else ++w.t;
        continue;
      }
    }
    r.t = w.t;
    r.seq = w.sq.seq;
    r.m = min(TILE, min(w.end, w.sq.t1) - w.t);
    r.first = w.t == w.sq.t0;
    w.fresh |= r.first;
    w.t += r.m;
    r.last = w.t == w.sq.t1;
    break;
  }
  return r;
}

// One CTA: CH channels of one segment.  Four warps run the recurrence on a tile in shared
// memory; four more bring the next tile's r, r x, B and C meanwhile, and turn the last tile's
// sums into outputs.
template <typename T, int CPT, int SPT, int L, bool CARRY, bool VEC>
__global__ void __launch_bounds__(2 * kScanThreads, CPT == 1 ? 3 : 2) selective_scan_kernel(
    const __grid_constant__ ScanParams p) {
  constexpr int SP = SPT * L;                      // padded S
  constexpr int CH = kScanThreads / L * CPT;       // channels of this CTA
  constexpr int kTile = scan_tile<CPT, L>();
  constexpr int NV = CH / CPT, STEP = kScanThreads / NV;   // groups of CPT channels; rows at once
  constexpr int ROWS = kTile / STEP > 0 ? kTile / STEP : 1;
  // of them at a time: registers
  constexpr int kMost = VEC && sizeof(T) == 2 ? (CARRY ? 4 : 2) : CPT == 1 ? 4 : 1;
  constexpr int RB = ROWS < kMost ? ROWS : kMost;
  using Sums = LaneSums<CPT, L>;
  constexpr int BC = (CARRY ? 1 : 2) * SP;
  extern __shared__ __align__(16) float sm[];
  float2* ru = reinterpret_cast<float2*>(sm);      // [2][kTile][CH]: r and r x, then y in r's place
  float* bc = sm + 2 * kTile * CH * 2;             // [2][kTile][B, C][SP]
  pdl_launch_dependents();
  pdl_wait();
  const int seg = blockIdx.x, b = blockIdx.z;
  const int g = blockIdx.y / p.blocks, blk = blockIdx.y % p.blocks;
  const int Dg = p.D / p.G, tid = threadIdx.x % kScanThreads, l = tid % L;
  const bool loads = threadIdx.x >= kScanThreads;
  if (seg == 0 && blockIdx.y == 0 && b == 0 && p.starts && !CARRY)
    check_starts(p.starts, p.n_seq, p.N, p.status);
  const long long one = (long long)p.D * p.S;
  ScanTiles w;
  w.t = (int)((long long)seg * p.seg_tokens);
  w.end = (int)min((long long)seg * p.seg_tokens + p.seg_tokens, (long long)p.N);
  w.sq.t1 = 0;
  w.fresh = false;

  // registers of a block: 256 x 128 at launch, more for the warps with the states
  constexpr int kFew = 96, kMany = 152;
  static_assert(kFew + kMany <= 2 * 128, "registers at launch");
  if (loads) {
    if constexpr (CPT > 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFew));
    const int vl = tid % NV * CPT, vg = blk * CH + vl, row0 = tid / NV;
    const int vn = max(0, min(CPT, Dg - vg)), vc = g * Dg + vg;
    const T* x = static_cast<const T*>(p.x) + b * p.lay.x.batch + vc;
    const T* dt = static_cast<const T*>(p.dt) + b * p.lay.dt.batch + vc;
    const T* z = CARRY || !p.z ? nullptr : static_cast<const T*>(p.z) + b * p.lay.z.batch + vc;
    T* out = static_cast<T*>(p.out) + b * p.lay.out.batch + vc;
    const T* Bm = static_cast<const T*>(p.Bm) + b * p.lay.B.batch + (long long)g * p.S;
    const T* Cm = static_cast<const T*>(p.Cm) + b * p.lay.C.batch + (long long)g * p.S;
    float bias[CPT], dx[CPT];
#pragma unroll
    for (int e = 0; e < CPT; ++e) {
      bias[e] = p.dt_bias && e < vn ? p.dt_bias[vc + e] : 0.f;
      dx[e] = !CARRY && p.Dx && e < vn ? p.Dx[vc + e] : 0.f;
    }
    // A turn finishes the tile `done` and puts the tile `next` in its place: a thread has the
    // same rows and channels of both.  What it needs is on its way one part of a turn ahead.
    using V = Pack<T, CPT>;
    struct Part {
      V xd[RB], zd[RB], xn[RB], rn[RB];
    };
    // (the rows of a part lie STEP tokens apart)
    const long long dx_ = STEP * p.lay.x.token, ddt = STEP * p.lay.dt.token,
                    dz = STEP * p.lay.z.token, dout = STEP * p.lay.out.token;
    auto fetch = [&](const ScanTile& done, const ScanTile& next, int i0, Part& q) {
      const int r0 = row0 + i0 * STEP;
      const int nd = CARRY || vn <= 0 ? 0 : done.m, nn = vn <= 0 ? 0 : next.m;
      const T* a = x + (done.t + r0) * p.lay.x.token;
      const T* c = z + (done.t + r0) * p.lay.z.token;
      const T* d = x + (next.t + r0) * p.lay.x.token;
      const T* e = dt + (next.t + r0) * p.lay.dt.token;
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        if (!CARRY && r0 + i * STEP < nd) {
          load_pack<T, CPT, VEC>(a, vn, q.xd[i]);
          if (z) load_pack<T, CPT, VEC>(c, vn, q.zd[i]);
        }
        if (r0 + i * STEP < nn) {
          load_pack<T, CPT, VEC>(d, vn, q.xn[i]);
          load_pack<T, CPT, VEC>(e, vn, q.rn[i]);
        }
        a += dx_;
        c += dz;
        d += dx_;
        e += ddt;
      }
    };
    auto use = [&](const ScanTile& done, const ScanTile& next, float2* my, int i0, const Part& q) {
      const int r0 = row0 + i0 * STEP;
      const int nd = CARRY || vn <= 0 ? 0 : done.m, nn = vn <= 0 ? 0 : next.m;
      T* o = out + (done.t + r0) * p.lay.out.token;
      float2* at = my + r0 * CH;
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        if (!CARRY && r0 + i * STEP < nd) {
          float y[CPT];
#pragma unroll
          for (int e = 0; e < CPT; e += 2) {
            if constexpr (CPT > 1) {
              const float4 v = *reinterpret_cast<const float4*>(at + e);
              y[e] = v.x;
              y[e + 1] = v.z;
            } else {
              y[e] = at[e].x;
            }
          }
          float xv[CPT], zv[CPT];
          pack_f(q.xd[i], xv);
          if (z) pack_f(q.zd[i], zv);
#pragma unroll
          for (int e = 0; e < CPT; ++e) {
            y[e] = fmaf(dx[e], xv[e], y[e]);
            if (z) y[e] *= silu_f(zv[e]);
          }
          store_row<T, CPT, VEC>(o, vn, y);
        }
        if (r0 + i * STEP < nn) {
          float r[CPT + 1], xv[CPT], rv[CPT];
          pack_f(q.xn[i], xv);
          pack_f(q.rn[i], rv);
#pragma unroll
          for (int e = 0; e < CPT; ++e) r[e] = rv[e] + bias[e];
          r[CPT] = 0.f;
          if (p.softplus) {
#pragma unroll
            for (int e = 0; e < CPT; e += 2) softplus2(r[e], r[e + 1]);
          }
          if constexpr (CPT > 1) {
#pragma unroll
            for (int e = 0; e < CPT; e += 2)
              *reinterpret_cast<float4*>(at + e) =
                  make_float4(r[e], r[e] * xv[e], r[e + 1], r[e + 1] * xv[e + 1]);
          } else {
            at[0] = make_float2(r[0], r[0] * xv[0]);
          }
        }
        o += dout;
        at += STEP * CH;
      }
    };
    // B and C of a tile, a turn ahead too where they are few
    constexpr int NBC = (kTile * SP + kScanThreads - 1) / kScanThreads;
    constexpr bool AHEAD = NBC <= 4;
    T bq[AHEAD ? NBC : 1], cq[AHEAD ? NBC : 1];
    auto fetch_bc = [&](const ScanTile& next) {
      if constexpr (AHEAD) {
#pragma unroll
        for (int i = 0; i < NBC; ++i) {
          const int e = tid + i * kScanThreads, j = e / SP, s = e % SP;
          bq[i] = cq[i] = from_f<T>(0.f);
          if (j < next.m && s < p.S) {
            bq[i] = Bm[(next.t + j) * p.lay.B.token + s];
            if (!CARRY) cq[i] = Cm[(next.t + j) * p.lay.C.token + s];
          }
        }
      }
    };
    // the turn's parts, with the first one of the turn after it (done2, next2) fetched last
    auto turn = [&](const ScanTile& done, const ScanTile& next, const ScanTile& done2,
                    const ScanTile& next2, int buf, Part& q) {
      float2* my = ru + buf * kTile * CH + vl;
      float* mb = bc + buf * kTile * BC;
      if constexpr (AHEAD) {
#pragma unroll
        for (int i = 0; i < NBC; ++i) {
          const int e = tid + i * kScanThreads, j = e / SP, s = e % SP;
          if (j < kTile) {
            mb[j * BC + s] = to_f<T>(bq[i]);
            if (!CARRY) mb[j * BC + SP + s] = to_f<T>(cq[i]);
          }
        }
        fetch_bc(next2);
      } else {
        for (int e = tid; e < next.m * SP; e += kScanThreads) {
          const int j = e / SP, s = e % SP;
          mb[j * BC + s] = s < p.S ? to_f<T>(Bm[(next.t + j) * p.lay.B.token + s]) : 0.f;
          if (!CARRY)
            mb[j * BC + SP + s] = s < p.S ? to_f<T>(Cm[(next.t + j) * p.lay.C.token + s]) : 0.f;
        }
      }
#pragma unroll 1
      for (int i0 = 0; i0 < ROWS; i0 += RB) {
        Part f;
        const bool more = i0 + RB < ROWS;
        fetch(more ? done : done2, more ? next : next2, more ? i0 + RB : 0, f);
        use(done, next, my, i0, q);
        q = f;
      }
    };
    ScanTile none;
    none.t = none.m = 0;
    ScanTile prev = none, cur = next_tile<kTile>(p, w, b), nxt = next_tile<kTile>(p, w, b);
    Part q;
    fetch(none, cur, 0, q);
    fetch_bc(cur);
    turn(none, cur, none, nxt, 0, q);
    __syncthreads();
    for (int k = 0; cur.m > 0; ++k) {
      const ScanTile nx2 = next_tile<kTile>(p, w, b);
      turn(prev, nxt, cur, nx2, (k + 1) & 1, q);
      __syncthreads();
      prev = cur;
      cur = nxt;
      nxt = nx2;
      if (cur.m == 0 && !CARRY) turn(prev, none, none, none, k & 1, q);
    }
    return;
  }

  if constexpr (CPT > 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMany));
  const int cl = tid / L * CPT, cg = blk * CH + cl;
  const int n = max(0, min(CPT, Dg - cg));
  const int c = g * Dg + (n > 0 ? cg : 0);   // idle threads run along and store nothing
  F2 A[CPT][SPT / 2], h[CPT][SPT / 2];
  float sum[CPT];
#pragma unroll
  for (int e = 0; e < CPT; ++e) {
    sum[e] = 0.f;
#pragma unroll
    for (int s = 0; s < SPT; s += 2) {
      float a[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        a[i] = e < n && l * SPT + s + i < p.S
                   ? p.A[(long long)(c + e) * p.S + l * SPT + s + i] * kLog2e : 0.f;
      A[e][s / 2] = pack2(a[0], a[1]);
    }
  }
  auto load_state = [&](const float* src) {   // [D][S] of one sequence or segment, or NULL
#pragma unroll
    for (int e = 0; e < CPT; ++e)
#pragma unroll
      for (int s = 0; s < SPT; s += 2) {
        float v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          v[i] = src && e < n && l * SPT + s + i < p.S
                     ? src[(long long)(c + e) * p.S + l * SPT + s + i] : 0.f;
        h[e][s / 2] = pack2(v[0], v[1]);
      }
  };
  auto store_state = [&](float* dst) {
#pragma unroll
    for (int e = 0; e < CPT; ++e)
#pragma unroll
      for (int s = 0; s < SPT; s += 2) {
        float v[2];
        unpack2(h[e][s / 2], v[0], v[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (e < n && l * SPT + s + i < p.S)
            dst[(long long)(c + e) * p.S + l * SPT + s + i] = v[i];
      }
  };
  // the states of empty sequences, spread over the segments
  if (!CARRY && p.state_out && p.starts)
    for (int s = seg; s < p.n_seq; s += p.segs)
      if (p.starts[s] == p.starts[s + 1]) {
        load_state(p.state_in ? p.state_in + s * one : nullptr);
        store_state(p.state_out + s * one);
      }
  if (!CARRY && seg > 0) load_state(p.seg_state + ((long long)b * p.segs + seg) * one);
  else load_state(nullptr);
  ScanTile cur = next_tile<kTile>(p, w, b);
  __syncthreads();
  for (int k = 0; cur.m > 0; ++k) {
    const ScanTile nxt = next_tile<kTile>(p, w, b);
    if (cur.first) load_state(p.state_in ? p.state_in + cur.seq * one : nullptr);
    float2* my = ru + (k & 1) * kTile * CH + cl;
    const float* bj = bc + (k & 1) * kTile * BC + l * SPT;
#pragma unroll 1
    for (int j = 0; j < cur.m; ++j, my += CH, bj += BC) {
      float2 q[CPT];
#pragma unroll
      for (int e = 0; e < CPT; e += 2) {
        if constexpr (CPT > 1) {
          const float4 v = *reinterpret_cast<const float4*>(my + e);
          q[e] = make_float2(v.x, v.y);
          q[e + 1] = make_float2(v.z, v.w);
        } else {
          q[e] = my[e];
        }
      }
      F2 acc[CPT];
#pragma unroll
      for (int e = 0; e < CPT; ++e) acc[e] = 0ull;
#pragma unroll
      for (int s = 0; s < SPT / 2; s += 2) {
        const ulonglong2 Bv = *reinterpret_cast<const ulonglong2*>(bj + 2 * s);
        ulonglong2 Cv = make_ulonglong2(0ull, 0ull);
        if (!CARRY) Cv = *reinterpret_cast<const ulonglong2*>(bj + SP + 2 * s);
#pragma unroll
        for (int e = 0; e < CPT; ++e) {
          const F2 rr = pack2(q[e].x, q[e].x), uu = pack2(q[e].y, q[e].y);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float a0, a1;
            unpack2(mul2(rr, A[e][s + i]), a0, a1);
            h[e][s + i] = fma2(pack2(ex2(a0), ex2(a1)), h[e][s + i], mul2(uu, i ? Bv.y : Bv.x));
            if (!CARRY) acc[e] = fma2(i ? Cv.y : Cv.x, h[e][s + i], acc[e]);
          }
        }
      }
      if (CARRY) {
#pragma unroll
        for (int e = 0; e < CPT; ++e) sum[e] += q[e].x;
      } else {
        float v[CPT], y[Sums::kept];
#pragma unroll
        for (int e = 0; e < CPT; ++e) {
          float a0, a1;
          unpack2(acc[e], a0, a1);
          v[e] = a0 + a1;
        }
        Sums::sum(v, l, y);
        if (Sums::writes(l)) {
#pragma unroll
          for (int e = 0; e < Sums::kept; ++e) my[Sums::own_first(l) + e].x = y[e];
        }
      }
    }
    if (!CARRY && p.state_out && cur.last) store_state(p.state_out + cur.seq * one);
    __syncthreads();
    cur = nxt;
  }
  if (CARRY) {
    const long long at = (long long)b * p.segs + seg;
    store_state(p.seg_state + at * one);
    if (l == 0) {
#pragma unroll
      for (int e = 0; e < CPT; ++e)
        if (e < n) p.seg_sum[at * p.D + c + e] = sum[e];
    }
    if (blockIdx.y == 0 && tid == 0) p.seg_new[at] = w.fresh;
  }
}

// The factor 2^e of a state behind a segment, in parts: whole^3 last.  Where 2^e is no normal number
// (|e| above 126) 2^e h may be one all the same, so h takes a quarter of e at a time, which covers
// all factors that lead from an fp32 number to another (|e| up to 277).  The parts are never 0 nor
// infinite: what is NaN or infinite in h stays, and 0 stays 0, as token by token.  No branch: the
// states follow one another (24 packed sequences 210 us, 214 with the rare cases in branches).
struct SegmentFactor {
  float whole, last;
};
__device__ __forceinline__ SegmentFactor segment_factor(float e) {
  const bool parts = fabsf(e) > 126.f;
  const float f = ex2(fminf(fmaxf(parts ? 0.25f * e : e, -126.f), 127.f));
  return {parts ? f : 1.f, f};
}

// The start states of the segments 1, 2, ..: one thread per number of the state.
__global__ void __launch_bounds__(256) scan_join_kernel(const __grid_constant__ ScanParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const long long one = (long long)p.D * p.S;
  const long long i = blockIdx.x * 256ll + threadIdx.x;
  if (i >= one) return;
  const int b = blockIdx.y;
  const float A = p.A[i] * kLog2e;
  float* st = p.seg_state + (long long)b * p.segs * one + i;
  const float* sum = p.seg_sum + (long long)b * p.segs * p.D + i / p.S;
  const int* fresh = p.seg_new + (long long)b * p.segs;
  float h = 0.f;
  constexpr int U = 16;   // segments whose numbers are on their way together, behind U others
  struct Part {
    float l[U], r[U];
    int fresh[U];
  };
  auto fetch = [&](int j, Part& q) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const bool in = j + k < p.segs - 1;
      q.l[k] = in ? st[(j + k) * one] : 0.f;
      q.r[k] = in ? sum[(long long)(j + k) * p.D] : 0.f;
      q.fresh[k] = in ? fresh[j + k] : 1;
    }
  };
  Part q;
  fetch(0, q);
  for (int j = 0; j < p.segs - 1; j += U) {
    Part next;
    fetch(j + U, next);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (j + k >= p.segs - 1) break;
      if (j + k > 0) st[(j + k) * one] = h;
      const SegmentFactor f = segment_factor(A == 0.f ? 0.f : A * q.r[k]);
      h = q.fresh[k] ? q.l[k] : fmaf(h * f.whole * f.whole * f.whole, f.last, q.l[k]);
    }
    q = next;
  }
  st[(p.segs - 1) * one] = h;
}

struct ScanShape {
  int cpt, spt, lanes;   // a thread's channels and numbers, lanes per channel
  int segs, seg_tokens, blocks;
};

ScanShape scan_shape(int B, int N, int D, int S, int G) {
  ScanShape s;
  // Many channels and tokens: four channels a thread, so that each number of B and C from
  // shared memory serves four.  Otherwise one channel over S / 4 lanes, so that a token takes
  // little time.  (S 16, 2048 tokens of 1536 channels: 60 us against 90; 1024 of 1024: 46
  // and 39.  Groups of 64 channels leave half of the first kind's threads idle: 8192 tokens
  // of 24 groups 401 us against 324.)
  const long long work = (long long)B * N * D;
  const bool wide = work >= 1 << 21 && D / G >= 128;
  s.cpt = wide ? 4 : 1;
  s.spt = wide ? 8 : 4;
  s.lanes = 1;
  while (s.spt * s.lanes < S) s.lanes *= 2;
  const int ch = kScanThreads / s.lanes * s.cpt;
  s.blocks = (D / G + ch - 1) / ch;
  // One round of CTAs, two on every SM, and segments of whole tiles.  The carry costs 2/3 of an
  // output pass, so that two segments of half the length pay already (25 sequences of 8000 x
  // 1536: 2457 us, whole 2697), but for the launches and the join: 64 tokens of 512 channels
  // 9.1 us in four segments, 8.9 whole and in one launch; 128 tokens 9.5 and 15.7; 192 tokens
  // of 4096 channels 27.4 in two, 26.6 whole, 256 34.0 and 34.5.
  const long long ctas = (long long)B * G * s.blocks, room = 2 * kScanSms;
  long long segs = room / ctas;
  const long long most = (N + 15) / 16;
  if (segs > most) segs = most;
  if (segs < 1 || N < 96 || (segs == 2 && N < 256)) segs = 1;
  s.seg_tokens = (int)(((N + segs - 1) / segs + 15) / 16 * 16);   // whole tiles
  s.segs = (N + s.seg_tokens - 1) / s.seg_tokens;
  return s;
}

template <typename P>
cudaError_t scan_launch(void (*kern)(P), dim3 grid, int smem, cudaStream_t stream, const P& p) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return launch_grid(kern, grid, 2 * kScanThreads, smem, stream, p);
}

template <typename T, int CPT, int SPT, int L>
int launch_scan(const ScanArgs& a, ScanParams p, const ScanShape& s) {
  constexpr int E = CPT;
  const unsigned bytes = E * sizeof(T);
  auto ok = [&](const void* ptr, const mixer_stride& st) {
    return (reinterpret_cast<uintptr_t>(ptr) & (bytes - 1)) == 0 && st.batch % E == 0 &&
           st.token % E == 0;
  };
  const bool vec = CPT > 1 && (a.D / a.G) % E == 0 && ok(a.x, a.lay.x) && ok(a.dt, a.lay.dt) &&
                   (!a.z || ok(a.z, a.lay.z)) && ok(a.out, a.lay.out);
  const double n = (double)a.B * a.N * a.D;
  if (s.segs > 1) {
    {
      ProfScope ps(PT_SCAN_CARRY, a.stream, 4.0 * n * a.S, 2.0 * n * sizeof(T));
      const dim3 grid(s.segs - 1, a.G * s.blocks, a.B);
      const cudaError_t e =
          vec ? scan_launch(selective_scan_kernel<T, CPT, SPT, L, true, CPT != 1>, grid, scan_smem<CPT, SPT, L, true>(), a.stream, p)
              : scan_launch(selective_scan_kernel<T, CPT, SPT, L, true, false>, grid, scan_smem<CPT, SPT, L, true>(), a.stream, p);
      if (e != cudaSuccess) return TTT_ERR_CUDA;
    }
    const long long one = (long long)a.D * a.S;
    ProfScope ps(PT_SCAN_JOIN, a.stream, 2.0 * a.B * s.segs * one, 8.0 * a.B * s.segs * one);
    if (launch_grid(scan_join_kernel, dim3((unsigned)((one + 255) / 256), a.B), 256, 0, a.stream, p) != cudaSuccess)
      return TTT_ERR_CUDA;
  }
  ProfScope ps(PT_SCAN, a.stream, 6.0 * n * a.S, (a.z ? 4.0 : 3.0) * n * sizeof(T));
  const dim3 grid(s.segs, a.G * s.blocks, a.B);
  const cudaError_t e =
      vec ? scan_launch(selective_scan_kernel<T, CPT, SPT, L, false, CPT != 1>, grid, scan_smem<CPT, SPT, L, false>(), a.stream, p)
          : scan_launch(selective_scan_kernel<T, CPT, SPT, L, false, false>, grid, scan_smem<CPT, SPT, L, false>(), a.stream, p);
  return e == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

template <typename T, int CPT, int SPT>
int scan_lanes(const ScanArgs& a, const ScanParams& p, const ScanShape& s) {
  if (s.lanes == 1) return launch_scan<T, CPT, SPT, 1>(a, p, s);
  if (s.lanes == 2) return launch_scan<T, CPT, SPT, 2>(a, p, s);
  if (s.lanes == 4) return launch_scan<T, CPT, SPT, 4>(a, p, s);
  if (s.lanes == 8) return launch_scan<T, CPT, SPT, 8>(a, p, s);
  if (s.lanes == 16) return launch_scan<T, CPT, SPT, 16>(a, p, s);
  if constexpr (SPT == 4) return launch_scan<T, CPT, SPT, 32>(a, p, s);
  return TTT_ERR_UNSUPPORTED;
}

template <typename T>
int scan_t(const ScanArgs& a, const ScanParams& p, const ScanShape& s) {
  return s.cpt == 1 ? scan_lanes<T, 1, 4>(a, p, s) : scan_lanes<T, 4, 8>(a, p, s);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// ------------------------------------------------------------ single tokens
struct ScanStepParams {
  const void* x;
  const void* dt;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* Dx;
  const float* dt_bias;
  const void* z;
  float* state;
  const int* slots;
  void* out;
  int* status;
  int n_slots, B, D, S, G, softplus;
  selective_scan_layout lay;
};

// L lanes a channel, each K pieces of four numbers of its state, R rows of the batch a thread.
// 245 rows of 4096 x 16 over states that pass the L2: 32.5 us, 4.2 TB/s of 6.8, bound by the loads'
// latency and by issue (55%); with the states of one call in the L2 25 us, 1000 rows 122 us, as
// below.  Both what is on its way and the instructions count: the step, the gate, the skip and the sum over the lanes are for a
// channel, so that one piece a lane (four rows a thread: 34 and 174 us) makes them twice as
// often; two pieces and four rows 29 and 143, four pieces of one lane 32 and 132.  With 64
// numbers four pieces and one row are ahead (1000 rows of 2048: 192 us, two pieces and two
// rows 229).
enum ScanPieces { kAnySize, kPieces, kAllPieces };   // S: any; a multiple of 4; 4 L K
template <typename T, int L, int K, int R, ScanPieces P>
__global__ void __launch_bounds__(128) scan_step_kernel(const __grid_constant__ ScanStepParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int b0 = blockIdx.y * R, l = threadIdx.x % L;
  const int c = blockIdx.x * (128 / L) + threadIdx.x / L;
  const bool in = c < p.D;
  int slot[R];
  read_slots<R>(p.slots, b0, p.B, slot);
  // everything is on its way before the slots are compared with other rows'
  const int g = in ? c / (p.D / p.G) : 0;
  constexpr bool VEC = P != kAnySize;
  // numbers 4 (l + L k) .. + 3 of the state, `n` of them below S
  auto first = [&](int k) { return 4 * (l + L * k); };
  auto n = [&](int k) { return P == kAllPieces ? 4 : in ? max(0, min(4, p.S - first(k))) : 0; };
  float h[R][K][4], a[K][4];
  float xv[R], r[R], zv[R];
  Pack<T, 4> Bq[R][K], Cq[R][K];
  auto load_bc = [&](int i) {
    const T* Bm = static_cast<const T*>(p.Bm) + (b0 + i) * p.lay.B.batch + (long long)g * p.S;
    const T* Cm = static_cast<const T*>(p.Cm) + (b0 + i) * p.lay.C.batch + (long long)g * p.S;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (n(k) == 0) continue;
      load_pack<T, 4, VEC>(Bm + first(k), n(k), Bq[i][k]);
      load_pack<T, 4, VEC>(Cm + first(k), n(k), Cq[i][k]);
    }
  };
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int b = b0 + i;
    xv[i] = r[i] = zv[i] = 0.f;
    if (slot[i] < 0 || slot[i] >= p.n_slots) continue;
    const float* st = p.state + ((long long)slot[i] * p.D + c) * p.S;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (n(k) > 0) load_row<float, 4, VEC>(st + first(k), n(k), h[i][k]);
    load_bc(i);
    if (in) {
      xv[i] = to_f<T>(static_cast<const T*>(p.x)[b * p.lay.x.batch + c]);
      r[i] = to_f<T>(static_cast<const T*>(p.dt)[b * p.lay.dt.batch + c]);
      if (p.z) zv[i] = to_f<T>(static_cast<const T*>(p.z)[b * p.lay.z.batch + c]);
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (n(k) > 0) load_row<float, 4, VEC>(p.A + (long long)c * p.S + first(k), n(k), a[k]);
  const float bias = in && p.dt_bias ? p.dt_bias[c] : 0.f, dx = in && p.Dx ? p.Dx[c] : 0.f;
  drop_bad_slots<R>(p.slots, p.n_slots, b0, p.B, p.status, slot);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int b = b0 + i;
    if (b >= p.B) break;
    T* out = static_cast<T*>(p.out) + b * p.lay.out.batch + c;
    if (slot[i] < 0) {
      if (in && l == 0) *out = from_f<T>(0.f);
      continue;
    }
    float rr = r[i] + bias, acc = 0.f;
    if (p.softplus) {
      float none = 0.f;
      softplus2(rr, none);
    }
    float* st = p.state + ((long long)slot[i] * p.D + c) * p.S;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (n(k) == 0) continue;
      float Bv[4], Cv[4];
      pack_f(Bq[i][k], Bv);
      pack_f(Cq[i][k], Cv);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[i][k][e] = fmaf(ex2(rr * (a[k][e] * kLog2e)), h[i][k][e], rr * xv[i] * Bv[e]);
        acc = fmaf(Cv[e], h[i][k][e], acc);
      }
      store_row<float, 4, VEC>(st + first(k), n(k), h[i][k]);
    }
    acc = sum_over<L>(acc);
    if (in && l == 0) {
      acc = fmaf(dx, xv[i], acc);
      if (p.z) acc *= silu_f(zv[i]);
      *out = from_f<T>(acc);
    }
  }
}

template <typename T, int L, int K>
int launch_scan_step(const ScanStepArgs& a, const ScanStepParams& p) {
  const int per = 128 / L;
  const double n = (double)a.B * a.D * a.S;
  ProfScope ps(PT_SCAN_STEP, a.stream, 6.0 * n, 8.0 * n);
  // four numbers lie in one 16-byte piece where S is a multiple of 4; those of B and C too
  auto ok = [](const void* x, unsigned bytes) { return (reinterpret_cast<uintptr_t>(x) & (bytes - 1)) == 0; };
  const bool vec = a.S % 4 == 0 && ok(a.state, 16) && ok(a.A, 16) &&
                   ok(a.Bm, 4 * sizeof(T)) && ok(a.Cm, 4 * sizeof(T)) && a.lay.B.batch % 4 == 0 &&
                   a.lay.C.batch % 4 == 0;
  const bool all = vec && a.S == 4 * L * K && a.D % per == 0;
  // several rows a thread where that leaves every SM four blocks (states of 4096 x 16: 32
  // rows 4.4 us, one row a thread 5.2; 8 rows 3.4 and 2.9)
  constexpr int M = K == 1 ? 4 : K == 2 ? 2 : 1;
  const int R = (long long)((a.D + per - 1) / per) * ((a.B + M - 1) / M) >= 4 * kScanSms ? M : 1;
  const dim3 grid((a.D + per - 1) / per, (a.B + R - 1) / R);
  void (*kern)(ScanStepParams) = all   ? scan_step_kernel<T, L, K, 1, kAllPieces>
                                 : vec ? scan_step_kernel<T, L, K, 1, kPieces>
                                       : scan_step_kernel<T, L, K, 1, kAnySize>;
  if constexpr (M > 1) {
    if (R == M)
      kern = all   ? scan_step_kernel<T, L, K, M, kAllPieces>
             : vec ? scan_step_kernel<T, L, K, M, kPieces>
                   : scan_step_kernel<T, L, K, M, kAnySize>;
  }
  return launch_grid(kern, grid, 128, 0, a.stream, p) == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

template <typename T>
int scan_step_t(const ScanStepArgs& a, const ScanStepParams& p) {
  if (a.S <= 4) return launch_scan_step<T, 1, 1>(a, p);
  if (a.S <= 8) return launch_scan_step<T, 1, 2>(a, p);
  if (a.S <= 16) return launch_scan_step<T, 2, 2>(a, p);
  if (a.S <= 32) return launch_scan_step<T, 4, 2>(a, p);
  if (a.S <= 64) return launch_scan_step<T, 4, 4>(a, p);
  return launch_scan_step<T, 8, 4>(a, p);
}

}  // namespace

size_t selective_scan_workspace(int B, int N, int D, int S, int G, int n_seq, int bf16) {
  (void)n_seq;
  (void)bf16;
  const ScanShape s = scan_shape(B, N, D, S, G);
  if (s.segs == 1) return 0;
  const size_t k = (size_t)B * s.segs;
  return align256(k * D * S * 4) + align256(k * D * 4) + align256(k * 4);
}

int selective_scan_launch(const ScanArgs& a) {
  const ScanShape s = scan_shape(a.B, a.N, a.D, a.S, a.G);
  ScanParams p{};
  p.x = a.x; p.dt = a.dt; p.A = a.A; p.Bm = a.Bm; p.Cm = a.Cm; p.Dx = a.Dx;
  p.dt_bias = a.dt_bias; p.z = a.z; p.state_in = a.state_in;
  p.starts = a.seq_starts;
  p.out = a.out;
  p.state_out = a.state_out;
  p.status = a.status;
  p.n_seq = a.n_seq; p.N = a.N; p.D = a.D; p.S = a.S; p.G = a.G;
  p.segs = s.segs; p.seg_tokens = s.seg_tokens; p.blocks = s.blocks;
  p.softplus = a.softplus;
  p.lay = a.lay;
  char* ws = static_cast<char*>(a.workspace);
  const size_t k = (size_t)a.B * s.segs;
  p.seg_state = reinterpret_cast<float*>(ws);
  ws += align256(k * a.D * a.S * 4);
  p.seg_sum = reinterpret_cast<float*>(ws);
  ws += align256(k * a.D * 4);
  p.seg_new = reinterpret_cast<int*>(ws);
  return a.bf16 ? scan_t<__nv_bfloat16>(a, p, s) : scan_t<float>(a, p, s);
}

int selective_scan_step_launch(const ScanStepArgs& a) {
  ScanStepParams p{};
  p.x = a.x; p.dt = a.dt; p.A = a.A; p.Bm = a.Bm; p.Cm = a.Cm; p.Dx = a.Dx;
  p.dt_bias = a.dt_bias; p.z = a.z; p.state = a.state;
  p.slots = a.slots;
  p.out = a.out;
  p.status = a.status;
  p.n_slots = a.n_slots; p.B = a.B; p.D = a.D; p.S = a.S; p.G = a.G;
  p.softplus = a.softplus;
  p.lay = a.lay;
  return a.bf16 ? scan_step_t<__nv_bfloat16>(a, p) : scan_step_t<float>(a, p);
}

}  // namespace ttt
