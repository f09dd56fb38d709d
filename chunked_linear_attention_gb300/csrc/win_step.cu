// Window attention for one token of each of B sequences, on their caches.
//
// What a token sees lies in the first min(t + 1, sinks + window) places of its slot, in
// some order; a softmax does not mind the order.  So the step writes the token's key and
// value to their place and takes the places as one list, split over the blocks of a
// cluster: one warp reads several keys at once, DP / 8 lanes a key, 8 dimensions a lane,
// for the G query heads of a key head together, with running maxima and sums; warps and
// blocks join their sums at the end through (distributed) shared memory.  The new token's
// row is taken from its inputs, never from the place that is being written.
//
// Bound by HBM: keys and values once.
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

template <typename T, int DP, int G, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) window_step_kernel(
    const __grid_constant__ WinStepParams p) {
  constexpr int LPK = DP / 8;        // lanes per key
  constexpr int KPW = 32 / LPK;      // keys a warp reads at once
  constexpr int U = 4;               // keys of a lane on their way together
  __shared__ float acc_s[kWarps][G][DP];
  __shared__ float m_s[kWarps][G], l_s[kWarps][G];
  __shared__ float acc_b[G][DP], m_b[G], l_b[G];   // of this block
  pdl_launch_dependents();
  pdl_wait();
  const int split = blockIdx.x % p.splits;   // rank in the cluster
  const int chunk = blockIdx.x / p.splits % p.chunks;
  const int hk = blockIdx.x / p.splits / p.chunks, b = blockIdx.y;
  const int group = p.Hq / p.Hk, h0 = hk * group + chunk * G;
  const int heads = min(G, group - chunk * G);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ld = lane % LPK, lk = lane / LPK;
  T* out = static_cast<T*>(p.out) + b * p.lay.out.batch + h0 * p.lay.out.head;
  int slot = row_slot(p.slots, p.n_slots, b, p.status);
  if (slot >= 0) {
    if (p.positions[b] < 0) {
      if (tid == 0) report_status(p.status, kStatusBadArg);
      slot = -1;
    }
  }
  if (slot < 0) {   // the same for the whole cluster
    if (split == 0)
      for (int e = tid; e < heads * p.d; e += kWarps * 32)
        out[e / p.d * p.lay.out.head + e % p.d] = from_f<T>(0.f);
    return;
  }
  const int t = p.positions[b];
  const int places = p.sinks + p.window;
  const int count = t < places ? t + 1 : places;
  const int own = t < p.sinks ? t : p.sinks + (t - p.sinks) % p.window;
  const T* kn = static_cast<const T*>(p.k) + b * p.lay.k.batch + hk * p.lay.k.head;
  const T* vn = static_cast<const T*>(p.v) + b * p.lay.v.batch + hk * p.lay.v.head;
  const long long at = ((long long)slot * p.Hk + hk) * places * p.d;
  T* ck = static_cast<T*>(p.cache_k) + at;
  T* cv = static_cast<T*>(p.cache_v) + at;
  if (split == 0 && chunk == 0)
    for (int e = tid; e < p.d; e += kWarps * 32) {
      ck[(long long)own * p.d + e] = kn[e];
      cv[(long long)own * p.d + e] = vn[e];
    }
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
  const int from = (int)((long long)count * split / p.splits);
  const int to = (int)((long long)count * (split + 1) / p.splits);
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
  // the key lanes of a warp, its warps, the cluster's blocks
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
  __syncthreads();
  for (int e = tid; e < G * DP; e += kWarps * 32) {
    const int g = e / DP, x = e % DP;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w][g]);
    const float base = top == -INFINITY ? 0.f : top;
    float a = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(m_s[w][g] - base);
      a = fmaf(f, acc_s[w][g][x], a);
      sum = fmaf(f, l_s[w][g], sum);
    }
    if (p.splits == 1) {
      if (g < heads && x < p.d) out[g * p.lay.out.head + x] = from_f<T>(a / sum);
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
  // a part of the outputs each
  for (int e = split * kWarps * 32 + tid; e < heads * p.d; e += p.splits * kWarps * 32) {
    const int g = e / p.d, x = e % p.d;
    float top = -INFINITY;
    for (int r = 0; r < p.splits; ++r) top = fmaxf(top, *cl.map_shared_rank(&m_b[g], r));
    const float base = top == -INFINITY ? 0.f : top;
    float a = 0.f, sum = 0.f;
    for (int r = 0; r < p.splits; ++r) {
      const float f = ex2(*cl.map_shared_rank(&m_b[g], r) - base);
      a = fmaf(f, *cl.map_shared_rank(&acc_b[g][x], r), a);
      sum = fmaf(f, *cl.map_shared_rank(&l_b[g], r), sum);
    }
    out[g * p.lay.out.head + x] = from_f<T>(a / sum);
  }
  cl.sync();   // no block ends while another reads from it
}

template <typename T, int DP, int G>
int launch_win_step(const WindowStepArgs& a, WinStepParams p) {
  constexpr int per = 16 / sizeof(T);
  auto ok = [&](const void* x, const delta_rule_stride& s) {
    return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && s.batch % per == 0 && s.head % per == 0;
  };
  // rows of 8 numbers, 16 bytes at a time: the caches are dense and 16-byte aligned
  const bool vec = a.d % 8 == 0 && ok(a.k, a.lay.k) && ok(a.v, a.lay.v);
  p.chunks = (a.Hq / a.Hk + G - 1) / G;
  // two blocks a SM, and no block with less than 128 places
  const long long ctas = (long long)a.B * a.Hk * p.chunks, places = (long long)a.window + a.sinks;
  p.splits = 1;
  while (p.splits < 8 && ctas * p.splits * 2 <= 2 * kStepSms && places / (p.splits * 2) >= 128)
    p.splits *= 2;
  const double pairs = (double)a.B * places;
  ProfScope ps(PT_WIN_STEP, a.stream, 4.0 * pairs * a.Hq * a.d, 2.0 * pairs * a.Hk * a.d * sizeof(T));
  const dim3 grid((unsigned)(a.Hk * p.chunks * p.splits), a.B);
  const cudaError_t e =
      vec ? launch_grid(window_step_kernel<T, DP, G, true>, grid, kWarps * 32, 0, a.stream, p, p.splits)
          : launch_grid(window_step_kernel<T, DP, G, false>, grid, kWarps * 32, 0, a.stream, p, p.splits);
  return e == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
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
