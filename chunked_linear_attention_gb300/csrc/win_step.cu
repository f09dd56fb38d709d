// Window attention for one token of each of B sequences, on their caches.
//
// What a token sees lies in the first min(t + 1, sinks + window) places of its slot, in
// some order; a softmax does not mind the order.  So the step writes the token's key and
// value to their place and takes the places as one list, split over the blocks of a
// cluster; a block takes several query heads of a key head together and keeps running
// maxima and sums, which warps and blocks join at the end through (distributed) shared
// memory.  In fp32 (and for rows that are not in 16-byte pieces) a warp reads several keys
// at once, DP / 8 lanes a key, 8 dimensions a lane; bf16 goes to the tensor cores, below.  The new token's
// row is taken from its inputs, never from the place that is being written.
//
// Bound by HBM where a block takes all query heads of its key head, up to eight on the tensor
// cores and four in fp32: keys and values once.  250 rows, 32 query heads on 8 key heads of 128,
// 2048 + 4 places, bf16: 303 us, 6.9 TB/s; fp32 with 64 rows 192 us, 5.6 TB/s.  More heads are
// taken in parts, by neighbouring blocks that each read the cache: fp32 with 64 heads on 8 324
// us, with 128 565.
#include <cooperative_groups.h>

#include "mixers.cuh"
#include "mixers.h"
#include "prof.h"

namespace ttt {

namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kStepSms = 152;

struct WinStepParams {
  const void* q;
  const void* k;
  const void* v;
  void* cache_k;
  void* cache_v;
  const int* positions;
  const int* slots;
  void* out;
  int* status;
  int n_slots, Hq, Hk, d, window, sinks, chunks, splits;
  float scale;
  window_attention_layout lay;
};

// A block's part of the work.
template <typename T>
struct StepRowT {
  int b, h0, heads, split, from, to, own;
  const T* kn;
  const T* vn;
  const T* ck;
  const T* cv;
};

// False for an idle row (the same in the whole cluster), whose outputs are set to zero.
// Otherwise the new key and value are on their way to their place.
template <typename T>
__device__ __forceinline__ bool step_row(const WinStepParams& p, int G, StepRowT<T>& r) {
  r.split = blockIdx.x % p.splits;   // rank in the cluster
  const int chunk = blockIdx.x / p.splits % p.chunks;
  const int hk = blockIdx.x / p.splits / p.chunks;
  r.b = blockIdx.y;
  const int group = p.Hq / p.Hk, tid = threadIdx.x;
  r.h0 = hk * group + chunk * G;
  r.heads = min(G, group - chunk * G);
  int slot = row_slot(p.slots, p.n_slots, r.b, p.status);
  const int t = slot >= 0 ? p.positions[r.b] : 0;
  if (t < 0) {
    if (tid == 0) report_status(p.status, kStatusBadArg);
    slot = -1;
  }
  if (slot < 0) {
    T* out = static_cast<T*>(p.out) + r.b * p.lay.out.batch + r.h0 * p.lay.out.head;
    if (r.split == 0)
      for (int e = tid; e < r.heads * p.d; e += blockDim.x)
        out[e / p.d * p.lay.out.head + e % p.d] = from_f<T>(0.f);
    return false;
  }
  const int places = p.sinks + p.window;
  const int count = t < places ? t + 1 : places;
  r.own = t < p.sinks ? t : p.sinks + (t - p.sinks) % p.window;
  r.kn = static_cast<const T*>(p.k) + r.b * p.lay.k.batch + hk * p.lay.k.head;
  r.vn = static_cast<const T*>(p.v) + r.b * p.lay.v.batch + hk * p.lay.v.head;
  const long long at = ((long long)slot * p.Hk + hk) * places * p.d;
  T* ck = static_cast<T*>(p.cache_k) + at;
  T* cv = static_cast<T*>(p.cache_v) + at;
  if (r.split == 0 && chunk == 0)
    for (int e = tid; e < p.d; e += blockDim.x) {
      ck[(long long)r.own * p.d + e] = r.kn[e];
      cv[(long long)r.own * p.d + e] = r.vn[e];
    }
  r.ck = ck;
  r.cv = cv;
  r.from = (int)((long long)count * r.split / p.splits);
  r.to = (int)((long long)count * (r.split + 1) / p.splits);
  return true;
}

// The warps' sums, then the cluster's blocks' (a part of the outputs each).
template <typename T, int DP, int G, int NW>
__device__ __forceinline__ void step_join(const WinStepParams& p, const StepRowT<T>& r,
                                          float (&acc_s)[NW][G][DP], float (&m_s)[NW][G],
                                          float (&l_s)[NW][G], float (&acc_b)[G][DP],
                                          float (&m_b)[G], float (&l_b)[G]) {
  const int tid = threadIdx.x;
  T* out = static_cast<T*>(p.out) + r.b * p.lay.out.batch + r.h0 * p.lay.out.head;
  __syncthreads();
  for (int e = tid; e < r.heads * DP; e += NW * 32) {
    const int g = e / DP, x = e % DP;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, m_s[w][g]);
    const float base = top == -INFINITY ? 0.f : top;
    float a = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = ex2(m_s[w][g] - base);
      a = fmaf(f, acc_s[w][g][x], a);
      sum = fmaf(f, l_s[w][g], sum);
    }
    if (p.splits == 1) {
      if (x < p.d) out[g * p.lay.out.head + x] = from_f<T>(a / sum);
    } else {
      acc_b[g][x] = a;
      if (x == 0) {
        m_b[g] = top;
        l_b[g] = sum;
      }
    }
  }
  if (p.splits == 1) return;
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  for (int e = r.split * NW * 32 + tid; e < r.heads * p.d; e += p.splits * NW * 32) {
    const int g = e / p.d, x = e % p.d;
    float top = -INFINITY;
    for (int i = 0; i < p.splits; ++i) top = fmaxf(top, *cl.map_shared_rank(&m_b[g], i));
    const float base = top == -INFINITY ? 0.f : top;
    float a = 0.f, sum = 0.f;
    for (int i = 0; i < p.splits; ++i) {
      const float f = ex2(*cl.map_shared_rank(&m_b[g], i) - base);
      a = fmaf(f, *cl.map_shared_rank(&acc_b[g][x], i), a);
      sum = fmaf(f, *cl.map_shared_rank(&l_b[g], i), sum);
    }
    out[g * p.lay.out.head + x] = from_f<T>(a / sum);
  }
  cl.sync();   // no block ends while another reads from it
}

// Two blocks on an SM: with four query heads and four keys of a lane on their way the registers
// are for one, and 64 rows of fp32 as above take 217 us; two keys and two blocks 192.
template <typename T, int DP, int G, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, 2) window_step_kernel(
    const __grid_constant__ WinStepParams p) {
  constexpr int LPK = DP / 8;        // lanes per key
  constexpr int KPW = 32 / LPK;      // keys a warp reads at once
  constexpr int U = G == 4 ? 2 : 4;  // keys of a lane on their way together
  __shared__ float acc_s[kWarps][G][DP];
  __shared__ float m_s[kWarps][G], l_s[kWarps][G];
  __shared__ float acc_b[G][DP], m_b[G], l_b[G];   // of this block
  pdl_launch_dependents();
  pdl_wait();
  StepRowT<T> row;
  if (!step_row<T>(p, G, row)) return;
  const int b = row.b, h0 = row.h0, heads = row.heads, own = row.own, from = row.from, to = row.to;
  const T *kn = row.kn, *vn = row.vn, *ck = row.ck, *cv = row.cv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ld = lane % LPK, lk = lane / LPK;
  // this lane's 8 dimensions
  const int c = ld * 8, n = VEC ? (c < p.d ? 8 : 0) : max(0, min(8, p.d - c));
  float q[G][8], acc[G][8], m[G], l[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      acc[g][e] = 0.f;
      q[g][e] = g < heads && e < n ? to_f<T>(static_cast<const T*>(p.q)[b * p.lay.q.batch +
                                         (h0 + g) * p.lay.q.head + c + e]) * p.scale : 0.f;
    }
  }
  // 8 numbers of a row: two 16-byte pieces in fp32
  auto row8 = [&](const T* x, float (&f)[8]) {
    if constexpr (VEC && sizeof(T) == 4) {
      const float4 a = n ? *reinterpret_cast<const float4*>(x + c) : make_float4(0, 0, 0, 0);
      const float4 e = n ? *reinterpret_cast<const float4*>(x + c + 4) : make_float4(0, 0, 0, 0);
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
      f[4] = e.x; f[5] = e.y; f[6] = e.z; f[7] = e.w;
    } else if constexpr (VEC) {
      const uint4 w = n ? *reinterpret_cast<const uint4*>(x + c) : make_uint4(0, 0, 0, 0);
      const T* y = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = to_f<T>(y[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = e < n ? to_f<T>(x[c + e]) : 0.f;
    }
  };
  for (int j0 = from + warp * KPW * U; j0 < to; j0 += kWarps * KPW * U) {
    float kr[U][8], vr[U][8], s[U][G];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * KPW + lk;
      const int jj = j < to ? j : from;   // read along, counted as -inf below
      row8(jj == own ? kn : ck + (long long)jj * p.d, kr[u]);
      row8(jj == own ? vn : cv + (long long)jj * p.d, vr[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float a = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) a = fmaf(q[g][e], kr[u][e], a);
#pragma unroll
        for (int o = LPK / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        s[u][g] = j0 + u * KPW + lk < to ? a : -INFINITY;
      }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float top = m[g];
#pragma unroll
      for (int u = 0; u < U; ++u) top = fmaxf(top, s[u][g]);
      const float base = top == -INFINITY ? 0.f : top;
      const float f = ex2(m[g] - base);
      m[g] = top;
      l[g] *= f;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[g][e] *= f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = ex2(s[u][g] - base);
        const bool in = j0 + u * KPW + lk < to;
        l[g] += w;
        if (in) {
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[g][e] = fmaf(w, vr[u][e], acc[g][e]);
        }
      }
    }
  }
  // the key lanes of a warp
#pragma unroll
  for (int g = 0; g < G; ++g) {
#pragma unroll
    for (int o = LPK; o < 32; o <<= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m[g], o);
      const float lo = __shfl_xor_sync(0xffffffffu, l[g], o);
      const float top = fmaxf(m[g], mo), base = top == -INFINITY ? 0.f : top;
      const float fa = ex2(m[g] - base), fb = ex2(mo - base);
      l[g] = l[g] * fa + lo * fb;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        acc[g][e] = acc[g][e] * fa + __shfl_xor_sync(0xffffffffu, acc[g][e], o) * fb;
      m[g] = top;
    }
    if (lk == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) acc_s[warp][g][c + e] = acc[g][e];
      if (ld == 0) {
        m_s[warp][g] = m[g];
        l_s[warp][g] = l[g];
      }
    }
  }
  step_join<T, DP, G, kWarps>(p, row, acc_s, m_s, l_s, acc_b, m_b, l_b);
}

// ------------------------------------------------------------ bf16 on the tensor cores
// With several query heads a key head the products above take longer than the keys and
// values (8 FMA and their reduction for each number read; the 250 rows above took 667 us):
// for bf16 they go through the warp-wide matrix instruction, 16 keys at a time.
//   S [heads x keys] = Q K^T: rows are the heads (8 at most; the other 8 rows are idle).  A
//       lane reads 16 bytes of a key and uses them as the two operands' halves of two
//       products: the dimensions of a product are those that its lanes have read.
//   O [heads x d] = P V: the weights as a pair hi + lo of bf16 numbers (off by 2^-17), hi in
//       rows 0 - 7 and lo in rows 8 - 15, so that one product takes both.  A lane reads 16
//       bytes of four values' rows and pairs those of neighbouring keys.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}

// Keys and values come to shared memory by asynchronous copies, kStepStages tiles of 16 a
// warp, so that a warp has two on their way while it works on one (loaded into registers
// where they are used, an iteration waited for memory: 16 rows of 8 key heads and 2052
// places took 35 us, 27 with the copies).  A row's 16-byte pieces lie at their number xor the row's, so that the
// lanes of a read fall on different banks.
constexpr int kStepStages = 3;

template <int DP, int NW>
constexpr int step_smem() {
  return NW * kStepStages * 2 * 16 * DP * 2;
}

template <int DP, int NW>
__global__ void __launch_bounds__(NW * 32) window_step_mma_kernel(
    const __grid_constant__ WinStepParams p) {
  using T = __nv_bfloat16;
  constexpr int G = 8, H = DP / 64;   // heads; halves of 64 dimensions
  constexpr int kTileB = 16 * DP * 2, kPer = DP / 8;   // bytes of a tile; pieces of a row
  extern __shared__ __align__(128) uint8_t ring[];
  static_assert(NW * kStepStages * 2 * kTileB >= NW * G * DP * 4, "the sums take the ring's place");
  float(&acc_s)[NW][G][DP] = *reinterpret_cast<float(*)[NW][G][DP]>(ring);
  __shared__ float m_s[NW][G], l_s[NW][G];
  __shared__ float acc_b[G][DP], m_b[G], l_b[G];   // of this block
  pdl_launch_dependents();
  pdl_wait();
  StepRowT<T> r;
  if (!step_row<T>(p, G, r)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  // this lane's dimensions of head g: 32 i + 8 q4 ..
  uint4 q[2 * H];
#pragma unroll
  for (int i = 0; i < 2 * H; ++i) {
    q[i] = make_uint4(0u, 0u, 0u, 0u);
    const int c = 32 * i + 8 * q4;
    if (g < r.heads && c < p.d) {
      const T* src = static_cast<const T*>(p.q) + r.b * p.lay.q.batch + (r.h0 + g) * p.lay.q.head + c;
      uint16_t w[8];   // rows of q at any address
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = reinterpret_cast<const uint16_t*>(src)[e];
      q[i] = make_uint4(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16,
                        w[4] | (uint32_t)w[5] << 16, w[6] | (uint32_t)w[7] << 16);
    }
  }
  float acc[H][8][4], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int y = 0; y < H; ++y)
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[y][n][e] = 0.f;

  uint8_t* mine = ring + warp * kStepStages * 2 * kTileB;
  const uint32_t mine_s = smem_u32(mine);
  const int first = r.from + warp * 16, step = NW * 16;
  // the tile of places j0 .. j0 + 15 to a stage; zeros behind the last place and dimension
  auto fetch = [&](int j0, int stage) {
    const uint32_t to = mine_s + stage * 2 * kTileB;
    if (j0 < r.to) {
#pragma unroll
      for (int x = 0; x < 16 * kPer / 32; ++x) {
        const int e = x * 32 + lane, row = e / kPer, c = e % kPer, j = j0 + row;
        const bool in = j < r.to && c * 8 < p.d, own = j == r.own;
        const long long at = in ? (long long)j * p.d + c * 8 : 0;
        const uint32_t dst = to + row * (DP * 2) + ((c ^ (row & 7)) << 4);
        copy16(dst, own && in ? r.kn + c * 8 : r.ck + at, in);
        copy16(dst + kTileB, own && in ? r.vn + c * 8 : r.cv + at, in);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int x = 0; x < kStepStages - 1; ++x) fetch(first + x * step, x);
  int stage = 0;
  for (int j0 = first; j0 < r.to; j0 += step) {
    int ahead = stage + kStepStages - 1;
    if (ahead >= kStepStages) ahead -= kStepStages;
    fetch(j0 + (kStepStages - 1) * step, ahead);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStepStages - 1) : "memory");
    __syncwarp();
    const uint32_t ks = mine_s + stage * 2 * kTileB, vs = ks + kTileB;
    if (++stage == kStepStages) stage = 0;
    uint4 k[2][2 * H], v[H][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)      // key j0 + 8 t + g
#pragma unroll
      for (int i = 0; i < 2 * H; ++i)
        k[t][i] = lds128(ks + (8 * t + g) * (DP * 2) + (((4 * i + q4) ^ g) << 4));
#pragma unroll
    for (int t = 0; t < 4; ++t) {    // keys j0 + 2 q4, + 1, + 8, + 9
      const int row = 2 * q4 + (t & 1) + 4 * (t & 2);
#pragma unroll
      for (int y = 0; y < H; ++y)
        v[y][t] = lds128(vs + row * (DP * 2) + (((8 * y + g) ^ (row & 7)) << 4));
    }
    __syncwarp();   // read before the stage is filled again
    float s[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * H; ++i) {
        mma16816(s[t], q[i].x, 0u, q[i].y, 0u, k[t][i].x, k[t][i].y);
        mma16816(s[t], q[i].z, 0u, q[i].w, 0u, k[t][i].z, k[t][i].w);
      }
    }
    // head g, keys j0 + 2 q4, + 1, + 8, + 9
    float x[4];
    float top = m;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = j0 + 2 * q4 + (e & 1) + 4 * (e & 2);
      x[e] = j < r.to ? s[e >> 1][e & 1] * p.scale : -INFINITY;
      top = fmaxf(top, x[e]);
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float base = top == -INFINITY ? 0.f : top;
    if (__any_sync(0xffffffffu, top > m)) {
      const float f = ex2(m - base);
      l *= f;
#pragma unroll
      for (int y = 0; y < H; ++y)
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[y][n][e] *= f;
    }
    m = top;
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = ex2(x[e] - base);
      l += x[e];
    }
    split2(pack2(x[0], x[1]), hi[0], lo[0]);
    split2(pack2(x[2], x[3]), hi[1], lo[1]);
#pragma unroll
    for (int y = 0; y < H; ++y)
#pragma unroll
      for (int n = 0; n < 8; n += 2) {
        // dimensions 64 y + 8 g + n, + 1 of the four keys
        auto word = [&](const uint4& w) { return n < 2 ? w.x : n < 4 ? w.y : n < 6 ? w.z : w.w; };
        const uint32_t a = word(v[y][0]), b = word(v[y][1]), c = word(v[y][2]), d = word(v[y][3]);
        mma16816(acc[y][n], hi[0], lo[0], hi[1], lo[1], __byte_perm(a, b, 0x5410),
                 __byte_perm(c, d, 0x5410));
        mma16816(acc[y][n + 1], hi[0], lo[0], hi[1], lo[1], __byte_perm(a, b, 0x7632),
                 __byte_perm(c, d, 0x7632));
      }
  }
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();   // the ring is done with
  // the sums of hi and of lo; column 2 q4 + e of the products with n has dimension
  // 64 y + 8 (2 q4 + e) + n
#pragma unroll
  for (int y = 0; y < H; ++y)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int n = 0; n < 8; n += 4)
        *reinterpret_cast<float4*>(&acc_s[warp][g][64 * y + 8 * (2 * q4 + e) + n]) = make_float4(
            acc[y][n][e] + acc[y][n][e + 2], acc[y][n + 1][e] + acc[y][n + 1][e + 2],
            acc[y][n + 2][e] + acc[y][n + 2][e + 2], acc[y][n + 3][e] + acc[y][n + 3][e + 2]);
  if (q4 == 0) {
    m_s[warp][g] = m;
    l_s[warp][g] = l;
  }
  step_join<T, DP, G, NW>(p, r, acc_s, m_s, l_s, acc_b, m_b, l_b);
}

// G: query heads that a block takes together.
template <typename T>
int win_step_go(const WindowStepArgs& a, WinStepParams p, int G, int warps, int smem,
                void (*kern)(WinStepParams)) {
  // static arrays of up to 8 KB count towards the 48 KB that need no leave
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TTT_ERR_CUDA;
  p.chunks = (a.Hq / a.Hk + G - 1) / G;
  // as many blocks as two a SM, and none with less than 128 places (up to four a SM: 8, 16
  // and 32 rows of 8 key heads and 2052 places 20, 32 and 53 us, by this rule 15, 27 and 45)
  const long long ctas = (long long)a.B * a.Hk * p.chunks, places = (long long)a.window + a.sinks;
  p.splits = 1;
  while (p.splits < 8 && ctas * p.splits * 2 <= 2 * kStepSms && places / (p.splits * 2) >= 128)
    p.splits *= 2;
  const double pairs = (double)a.B * places;
  ProfScope ps(PT_WIN_STEP, a.stream, 4.0 * pairs * a.Hq * a.d, 2.0 * pairs * a.Hk * a.d * sizeof(T));
  const dim3 grid((unsigned)(a.Hk * p.chunks * p.splits), a.B);
  const cudaError_t e = launch_grid(kern, grid, warps * 32, smem, a.stream, p, p.splits);
  return e == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

// Rows of 8 numbers, 16 bytes at a time: the caches are dense and 16-byte aligned.
template <typename T>
bool rows_of_8(const WindowStepArgs& a) {
  constexpr int per = 16 / sizeof(T);
  auto ok = [&](const void* x, const delta_rule_stride& s) {
    return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && s.batch % per == 0 && s.head % per == 0;
  };
  return a.d % 8 == 0 && ok(a.k, a.lay.k) && ok(a.v, a.lay.v);
}

template <typename T, int DP, int G>
int launch_win_step(const WindowStepArgs& a, const WinStepParams& p) {
  return win_step_go<T>(a, p, G, kWarps, 0,
                        rows_of_8<T>(a) ? window_step_kernel<T, DP, G, true>
                                        : window_step_kernel<T, DP, G, false>);
}

template <typename T, int DP>
int step_g(const WindowStepArgs& a, const WinStepParams& p) {
  const int group = a.Hq / a.Hk;
  if (group == 1) return launch_win_step<T, DP, 1>(a, p);
  if (group == 2) return launch_win_step<T, DP, 2>(a, p);
  return launch_win_step<T, DP, 4>(a, p);
}

template <typename T>
int step_d(const WindowStepArgs& a, const WinStepParams& p) {
  if constexpr (sizeof(T) == 2) {
    if (a.d <= 128 && rows_of_8<T>(a)) {
      // a warp takes 16 places at a time: four warps a block, or two where there are many
      // blocks with few places (2048 blocks: 64 places 34 us with four, 26 with two; 200: 60
      // and 53; 600: 112 and 111; 64 blocks with 128 places 5.4 and 6.9)
      const long long ctas = (long long)a.B * a.Hk * ((a.Hq / a.Hk + 7) / 8);
      const bool few = (long long)a.window + a.sinks <= 512 && ctas >= 4 * kStepSms;
      if (a.d <= 64)
        return few ? win_step_go<T>(a, p, 8, 2, step_smem<64, 2>(), window_step_mma_kernel<64, 2>)
                   : win_step_go<T>(a, p, 8, 4, step_smem<64, 4>(), window_step_mma_kernel<64, 4>);
      return few ? win_step_go<T>(a, p, 8, 2, step_smem<128, 2>(), window_step_mma_kernel<128, 2>)
                 : win_step_go<T>(a, p, 8, 4, step_smem<128, 4>(), window_step_mma_kernel<128, 4>);
    }
  }
  if (a.d <= 64) return step_g<T, 64>(a, p);
  if (a.d <= 128) return step_g<T, 128>(a, p);
  return step_g<T, 256>(a, p);
}

}  // namespace

int window_attention_step_launch(const WindowStepArgs& a) {
  WinStepParams p{};
  p.q = a.q; p.k = a.k; p.v = a.v;
  p.cache_k = a.cache_k; p.cache_v = a.cache_v;
  p.positions = a.positions;
  p.slots = a.slots;
  p.out = a.out;
  p.status = a.status;
  p.n_slots = a.n_slots; p.Hq = a.Hq; p.Hk = a.Hk; p.d = a.d; p.window = a.window; p.sinks = a.sinks;
  p.scale = a.scale * 1.44269504088896341f;
  p.lay = a.lay;
  return a.bf16 ? step_d<__nv_bfloat16>(a, p) : step_d<float>(a, p);
}

}  // namespace ttt
