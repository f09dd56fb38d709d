// Rows of the window attention in fp32, for every type, size and stride, by one block.
#pragma once

#include "win_attn.cuh"

namespace ttt {

// QT queries of one head, from i0 on, against key tiles of 64, two threads a query.  A thread
// holds 8 x 4 scores and 8 rows x DP / 16 columns of the output, with a running maximum and
// sum of the softmax per row, so that each score is made once.  Bound by the shared memory's
// words per product (12 for 32, in the scores and, at d 64, in the outputs): two thirds of
// the fp32 pipe at best.  16384 tokens, 8 heads, window 1024: heads of 64 0.97 ms (34
// TFLOP/s), of 128 1.89 ms; with 4 x 4 scores a thread (8 words for 16) and every score masked
// by itself 1.36 and 3.21.  2048 tokens with a window of 512 are 256 blocks of few warps: 126
// us, by 256 threads a block 116.
constexpr int kKT = 64, kPad = 4;

// Bytes of shared memory.
template <int DP, int QT>
constexpr int simt_smem() {
  return (DP * (QT + kPad) + DP * (kKT + kPad) + kKT * DP + kKT * (QT + kPad)) * 4 +
         QT * (int)sizeof(WinRow);
}

// All of the block's WARPS warps bring the tiles, the first QT / 16 do the rest.  SPOILED: only
// rows whose outputs are not finite are stored, and nothing is done where there are none.
template <typename T, int DP, int QT, bool VEC, int WARPS, bool SPOILED>
__device__ __forceinline__ void window_rows(const WinParams& p, int b, int h, int i0, float* sm) {
  constexpr int NC = DP / 64;                  // 4 NC columns of the output a thread
  constexpr int kQT = QT;
  float* Qt = sm;                              // [DP][kQT + kPad]
  float* Kt = Qt + DP * (kQT + kPad);          // [DP][kKT + kPad]
  float* V = Kt + DP * (kKT + kPad);           // [kKT][DP]
  float* Pt = V + kKT * DP;                    // [kKT][kQT + kPad]
  WinRow* rows = reinterpret_cast<WinRow*>(Pt + kKT * (kQT + kPad));
  const int hk = h / (p.Hq / p.Hk);
  const int tid = threadIdx.x, lane = tid & 31, tx = tid & 15, ty = tid >> 4;
  const bool works = WARPS == QT / 16 || tid < 2 * QT;
  const T* q = static_cast<const T*>(p.q) + b * p.lay.q.batch + h * p.lay.q.head;
  const T* k = static_cast<const T*>(p.k) + b * p.lay.k.batch + hk * p.lay.k.head;
  const T* v = static_cast<const T*>(p.v) + b * p.lay.v.batch + hk * p.lay.v.head;
  T* out = static_cast<T*>(p.out) + b * p.lay.out.batch + h * p.lay.out.head;
  if (tid < kQT) rows[tid] = win_row(p, b, i0 + tid);
  if (SPOILED) {
    __syncthreads();
    bool any = false;
    for (int r = tid >> 5; r < kQT; r += WARPS) {
      const int i = rows[r].i;
      if (i < 0) continue;
      bool fine = true;
      for (int c = lane; c < p.d; c += 32) fine = fine && isfinite(to_f<T>(out[i * p.lay.out.token + c]));
      fine = __all_sync(0xffffffffu, fine);
      if (fine && lane == 0) rows[r].i = -1;   // not stored
      any |= !fine;
    }
    if (!__syncthreads_or(any)) return;
  }
  // four numbers of a row of a tile to their places: lanes take 8 rows x 4 pieces, whose
  // transposed places fall on different banks but for pairs
  auto piece = [&](int e, int rows8, int& r, int& c) {
    r = e % rows8 * 8 + (lane >> 2);
    c = (e / rows8 * 4 + (lane & 3)) * 4;
  };
  for (int e = tid >> 5; e < DP / 16 * (kQT / 8); e += WARPS) {
    int r, c;
    piece(e, kQT / 8, r, c);
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (i0 + r < p.N && c < p.d) load_row<T, 4, VEC>(q + (i0 + r) * p.lay.q.token + c, p.d - c, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) Qt[(c + i) * (kQT + kPad) + r] = f[i] * p.scale;
  }
  float m[8], l[8], o[8][4 * NC];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * NC; ++c) o[r][c] = 0.f;
  }
  __syncthreads();
  // windows begin one behind another: the last query's and the first query bound them all
  const int last = min(kQT, p.N - i0) - 1;
  const int lo_last = rows[last].lo;
  WinList<kKT> w = win_list<kKT>(p, b, i0, i0 + kQT);
  WinTile t;
  while (win_next(p, w, t)) {
    // keys transposed, values as they are; rows that no query of this tile can see are
    // zero, and a value that is not finite asks for the careful sums below
    const T *ks = k, *vs = v;
    long long sk = p.lay.k.token, sv = p.lay.v.token;
    if (t.seq >= 0) {
      const long long at = ((long long)t.c.slot * p.Hk + hk) * (p.sinks + p.window) * p.d;
      ks = static_cast<const T*>(p.cache_k) + at;
      vs = static_cast<const T*>(p.cache_v) + at;
      sk = sv = p.d;
    }
    bool odd = false;
    __syncthreads();
#pragma unroll 4
    for (int e = tid >> 5; e < DP / 16 * (kKT / 8); e += WARPS) {
      int r, c;
      piece(e, kKT / 8, r, c);
      const int j = t.base + r;
      float f[4] = {0.f, 0.f, 0.f, 0.f}, g[4] = {0.f, 0.f, 0.f, 0.f};
      if (j >= 0 && j < t.end && c < p.d) {
        load_row<T, 4, VEC>(ks + j * sk + c, p.d - c, f);
        load_row<T, 4, VEC>(vs + j * sv + c, p.d - c, g);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Kt[(c + i) * (kKT + kPad) + r] = f[i];
        odd |= !isfinite(g[i]);
      }
      *reinterpret_cast<float4*>(V + r * DP + c) = make_float4(g[0], g[1], g[2], g[3]);
    }
    odd = __syncthreads_or(odd);
    if (!works) continue;
    float s[8][4] = {};
#pragma unroll 4
    for (int c = 0; c < p.d; ++c) {
      const float4 a0 = *reinterpret_cast<const float4*>(Qt + c * (kQT + kPad) + ty * 8);
      const float4 a1 = *reinterpret_cast<const float4*>(Qt + c * (kQT + kPad) + ty * 8 + 4);
      const float4 x = *reinterpret_cast<const float4*>(Kt + c * (kKT + kPad) + tx * 4);
      const float aa[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
      const float xx[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int n = 0; n < 4; ++n) s[r][n] = fmaf(aa[r], xx[n], s[r][n]);
    }
    unsigned seen = 0xffffffffu;
    if (t.seq >= 0 || t.base < lo_last || t.base + kKT - 1 > i0 || t.base + kKT > t.end) {
      seen = 0u;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const WinRow row = rows[ty * 8 + r];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int j = t.base + tx * 4 + n;
          const bool ok = t.seq < 0 ? sees_new(row, j, t.end)
                                    : sees_cache(row, t.c, j, p.sinks, p.window);
          seen |= (unsigned)ok << (r * 4 + n);
          if (!ok) s[r][n] = -INFINITY;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      float top = fmaxf(fmaxf(s[r][0], s[r][1]), fmaxf(s[r][2], s[r][3]));
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float mn = fmaxf(m[r], top);
      const float base = mn == -INFINITY ? 0.f : mn;   // nothing seen yet
      const float f = exp2f(m[r] - base);
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        s[r][n] = exp2f(s[r][n] - base);
        sum += s[r][n];
      }
      // the sum over the 16 threads of a row waits until the end
      l[r] = fmaf(l[r], f, sum);
      m[r] = mn;
#pragma unroll
      for (int c = 0; c < 4 * NC; ++c) o[r][c] *= f;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      float* to = Pt + (tx * 4 + n) * (kQT + kPad) + ty * 8;
      *reinterpret_cast<float4*>(to) = make_float4(s[0][n], s[1][n], s[2][n], s[3][n]);
      *reinterpret_cast<float4*>(to + 4) = make_float4(s[4][n], s[5][n], s[6][n], s[7][n]);
    }
    __syncwarp();   // a warp's rows are its own
    if (!odd) {
#pragma unroll 4
      for (int n = 0; n < kKT; ++n) {
        const float4 a0 = *reinterpret_cast<const float4*>(Pt + n * (kQT + kPad) + ty * 8);
        const float4 a1 = *reinterpret_cast<const float4*>(Pt + n * (kQT + kPad) + ty * 8 + 4);
        const float aa[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float4 x = *reinterpret_cast<const float4*>(V + n * DP + 64 * c + tx * 4);
          const float xx[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[r][4 * c + i] = fmaf(aa[r], xx[i], o[r][4 * c + i]);
        }
      }
    } else {
      // a value that a query does not see must not reach it, not even times 0
#pragma unroll 1
      for (int n = 0; n < kKT; ++n) {
        const unsigned bits = __shfl_sync(0xffffffffu, seen, (lane & 16) | (n >> 2)) >> (n & 3);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float a = Pt[n * (kQT + kPad) + ty * 8 + r];
          if ((bits >> (r * 4)) & 1) {
#pragma unroll
            for (int c = 0; c < 4 * NC; ++c)
              o[r][c] = fmaf(a, V[n * DP + 64 * (c / 4) + tx * 4 + c % 4], o[r][c]);
          }
        }
      }
    }
  }
  if (!works) return;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    float sum = l[r];
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    const int i = rows[ty * 8 + r].i;
    if (i < 0) continue;
    const float f = 1.f / sum;
#pragma unroll
    for (int c = 0; c < 4 * NC; ++c) {
      const int at = 64 * (c / 4) + tx * 4 + c % 4;
      if (at < p.d) out[i * p.lay.out.token + at] = from_f<T>(o[r][c] * f);
    }
  }
}

}  // namespace ttt
