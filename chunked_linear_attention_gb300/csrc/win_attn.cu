// Attention with a sliding window and sinks in fp32, for every type, size and stride, and
// the writing of new keys and values into the caches.
#include <algorithm>

#include "prof.h"
#include "win_attn.cuh"

namespace ttt {

namespace {

// ------------------------------------------------------------ prompts, fp32
// One CTA: QT queries of one head against key tiles of 64, two threads a query.  A thread
// holds 8 x 4 scores and 8 rows x DP / 16 columns of the output, with a running maximum and
// sum of the softmax per row, so that each score is made once.  Bound by the shared memory's
// words per product (12 for 32, in the scores and, at d 64, in the outputs): two thirds of
// the fp32 pipe at best.  16384 tokens, 8 heads, window 1024: heads of 64 0.99 ms (35
// TFLOP/s), of 128 1.93 ms; with 4 x 4 scores a thread (8 words for 16) and every score masked
// by itself 1.36 and 3.21.  2048 tokens with a window of 512 are 256 blocks of few warps: 126
// us, by 256 threads a block 116.
constexpr int kKT = 64, kPad = 4;

template <int DP, int QT>
constexpr int simt_smem() {
  return (DP * (QT + kPad) + DP * (kKT + kPad) + kKT * DP + kKT * (QT + kPad)) * 4 +
         QT * (int)sizeof(WinRow);
}

template <typename T, int DP, int QT, bool VEC>
__global__ void __launch_bounds__(2 * QT) window_attention_kernel(
    const __grid_constant__ WinParams p) {
  constexpr int NC = DP / 64;                  // 4 NC columns of the output a thread
  constexpr int kQT = QT, kWarps = QT / 16;
  extern __shared__ __align__(16) float sm[];
  float* Qt = sm;                              // [DP][kQT + kPad]
  float* Kt = Qt + DP * (kQT + kPad);          // [DP][kKT + kPad]
  float* V = Kt + DP * (kKT + kPad);           // [kKT][DP]
  float* Pt = V + kKT * DP;                    // [kKT][kQT + kPad]
  WinRow* rows = reinterpret_cast<WinRow*>(Pt + kKT * (kQT + kPad));
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.z, h = blockIdx.y, i0 = blockIdx.x * kQT;
  const int hk = h / (p.Hq / p.Hk);
  const int tid = threadIdx.x, lane = tid & 31, tx = tid & 15, ty = tid >> 4;
  if (blockIdx.x == 0 && h == 0 && p.starts) check_starts(p.starts, p.n_seq, p.N, p.status);
  const T* q = static_cast<const T*>(p.q) + b * p.lay.q.batch + h * p.lay.q.head;
  const T* k = static_cast<const T*>(p.k) + b * p.lay.k.batch + hk * p.lay.k.head;
  const T* v = static_cast<const T*>(p.v) + b * p.lay.v.batch + hk * p.lay.v.head;
  // four numbers of a row of a tile to their places: lanes take 8 rows x 4 pieces, whose
  // transposed places fall on different banks but for pairs
  auto piece = [&](int e, int rows8, int& r, int& c) {
    r = e % rows8 * 8 + (lane >> 2);
    c = (e / rows8 * 4 + (lane & 3)) * 4;
  };
  for (int e = tid >> 5; e < DP / 16 * (kQT / 8); e += kWarps) {
    int r, c;
    piece(e, kQT / 8, r, c);
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (i0 + r < p.N && c < p.d) load_row<T, 4, VEC>(q + (i0 + r) * p.lay.q.token + c, p.d - c, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) Qt[(c + i) * (kQT + kPad) + r] = f[i] * p.scale;
  }
  if (tid < kQT) rows[tid] = win_row(p, b, i0 + tid);
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
    for (int e = tid >> 5; e < DP / 16 * (kKT / 8); e += kWarps) {
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
  T* out = static_cast<T*>(p.out) + b * p.lay.out.batch + h * p.lay.out.head;
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

template <typename T, int DP, int QT>
int launch_simt(const WindowArgs& a, const WinParams& p) {
  auto ok = [&](const void* x, const delta_rule_stride& s) {
    return (reinterpret_cast<uintptr_t>(x) & (4 * sizeof(T) - 1)) == 0 && s.batch % 4 == 0 &&
           s.head % 4 == 0 && s.token % 4 == 0;
  };
  const bool vec = a.d % 4 == 0 && ok(a.q, a.lay.q) && ok(a.k, a.lay.k) && ok(a.v, a.lay.v);
  auto kern = vec ? window_attention_kernel<T, DP, QT, true> : window_attention_kernel<T, DP, QT, false>;
  constexpr int smem = simt_smem<DP, QT>();
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TTT_ERR_CUDA;
  const double tok = (double)a.B * a.N;
  ProfScope ps(PT_WIN_SIMT, a.stream, 4.0 * tok * a.Hq * a.d * fmin(a.N, (double)a.window + a.sinks),
               tok * (a.bf16 ? 2 : 4) * 2.0 * a.d * (a.Hq + a.Hk));
  return launch_grid(kern, dim3((a.N + QT - 1) / QT, a.Hq, a.B), 2 * QT, smem, a.stream, p) ==
                 cudaSuccess
             ? TTT_OK
             : TTT_ERR_CUDA;
}

template <typename T>
int simt_t(const WindowArgs& a, const WinParams& p) {
  // Heads of more than 64 take most of the shared memory: 128 queries a block, where those
  // fill the card twice, hold eight warps there and not four (16384 tokens, heads of 128: 1.93
  // ms, 64 queries 2.50; of 64, with three blocks on an SM, 1.06 and 0.99).
  const bool wide = (long long)((a.N + 127) / 128) * a.Hq * a.B >= 2 * 152;
  if (a.d <= 64) return launch_simt<T, 64, 64>(a, p);
  if (a.d <= 128) return wide ? launch_simt<T, 128, 128>(a, p) : launch_simt<T, 128, 64>(a, p);
  return launch_simt<T, 256, 64>(a, p);
}

// ------------------------------------------------------------ the caches after a prompt
// One CTA: some of the places of one (sequence, key head).  Kept are the sinks and the
// last `window` positions; a position's row is copied to its place.
struct StoreParams {
  const void* k;
  const void* v;
  void* cache_k;
  void* cache_v;
  const int* slots;
  const int* past;
  const int* starts;
  int* status;
  int n_slots, n_seq, Hk, N, d, window, sinks, parts;
  delta_rule_stride sk, sv;
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) window_store_kernel(const __grid_constant__ StoreParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int part = blockIdx.x, hk = blockIdx.y % p.Hk, s = blockIdx.y / p.Hk;
  const bool first = part == 0 && hk == 0;
  int slot = p.slots ? p.slots[s] : s;
  bool taken = slot >= p.n_slots;
  if (p.slots && slot >= 0)
    for (int i = threadIdx.x; i < s; i += blockDim.x) taken |= p.slots[i] == slot;
  taken = __syncthreads_or(taken);
  if (taken && slot >= 0) {
    if (first && threadIdx.x == 0) report_status(p.status, kStatusBadArg);
    slot = -1;
  }
  if (slot < 0) return;
  int t0 = 0, t1 = p.N, b = s;
  if (p.starts) {
    t0 = p.starts[s];
    t1 = p.starts[s + 1];
    b = 0;
    if (t0 < 0 || t1 <= t0 || t1 > p.N) return;
  }
  int past = p.past ? p.past[s] : 0;
  if (past < 0) {
    if (first && threadIdx.x == 0) report_status(p.status, kStatusBadArg);
    past = 0;
  }
  const long long end = (long long)past + (t1 - t0);
  // positions: sinks among the new ones, then the last of the others
  const int ns = max(0, min(p.sinks, (int)min(end, (long long)p.sinks)) - past);
  const long long from = max((long long)max(past, p.sinks), end - p.window);
  const int total = ns + (int)max(0ll, end - from);
  const T* k = static_cast<const T*>(p.k) + b * p.sk.batch + hk * p.sk.head;
  const T* v = static_cast<const T*>(p.v) + b * p.sv.batch + hk * p.sv.head;
  const long long at = ((long long)slot * p.Hk + hk) * ((long long)p.sinks + p.window) * p.d;
  T* ck = static_cast<T*>(p.cache_k) + at;
  T* cv = static_cast<T*>(p.cache_v) + at;
  constexpr int E = VEC ? 16 / sizeof(T) : 1;
  const int per = p.d / E;
  for (long long e = part * 256ll + threadIdx.x; e < (long long)total * per; e += p.parts * 256ll) {
    const int n = (int)(e / per), c = (int)(e % per) * E;
    const long long pos = n < ns ? past + n : from + (n - ns);
    const long long place = pos < p.sinks ? pos : p.sinks + (pos - p.sinks) % p.window;
    const long long j = t0 + (pos - past);
    if constexpr (VEC) {
      *reinterpret_cast<uint4*>(ck + place * p.d + c) =
          *reinterpret_cast<const uint4*>(k + j * p.sk.token + c);
      *reinterpret_cast<uint4*>(cv + place * p.d + c) =
          *reinterpret_cast<const uint4*>(v + j * p.sv.token + c);
    } else {
      ck[place * p.d + c] = k[j * p.sk.token + c];
      cv[place * p.d + c] = v[j * p.sv.token + c];
    }
  }
}

bool rows_wide(const void* x, const delta_rule_stride& s, int d, int per) {
  return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && d % per == 0 && s.batch % per == 0 &&
         s.head % per == 0 && s.token % per == 0;
}

}  // namespace

WinParams win_params(const WindowArgs& a) {
  WinParams p{};
  p.q = a.q; p.k = a.k; p.v = a.v;
  p.cache_k = a.cache_k; p.cache_v = a.cache_v;
  p.slots = a.slots; p.past = a.past; p.starts = a.seq_starts;
  p.out = a.out;
  p.status = a.status;
  p.n_slots = a.n_slots; p.n_seq = a.n_seq; p.B = a.B; p.Hq = a.Hq; p.Hk = a.Hk; p.N = a.N;
  p.d = a.d; p.window = a.window; p.sinks = a.sinks;
  p.scale = a.scale * 1.44269504088896341f;
  p.lay = a.lay;
  p.wait_ns = a.wait_ns;
  return p;
}

int window_attention_simt(const WindowArgs& a) {
  const WinParams p = win_params(a);
  return a.bf16 ? simt_t<__nv_bfloat16>(a, p) : simt_t<float>(a, p);
}

int window_attention_store(const WindowArgs& a) {
  StoreParams p{};
  p.k = a.k; p.v = a.v; p.cache_k = a.cache_k; p.cache_v = a.cache_v;
  p.slots = a.slots; p.past = a.past; p.starts = a.seq_starts;
  p.status = a.status;
  p.n_slots = a.n_slots; p.n_seq = a.n_seq; p.Hk = a.Hk; p.N = a.N; p.d = a.d;
  p.window = a.window; p.sinks = a.sinks;
  p.sk = a.lay.k; p.sv = a.lay.v;
  const int per = a.bf16 ? 8 : 4;
  const bool vec = rows_wide(a.k, p.sk, a.d, per) && rows_wide(a.v, p.sv, a.d, per);
  // two pieces of 16 bytes a thread for a full cache, and some ten blocks a SM at most
  const long long most = a.N < (long long)a.window + a.sinks ? a.N : (long long)a.window + a.sinks;
  const long long parts = most * a.d / per / 512 + 1;
  const long long room = std::max(64ll, 1536ll / ((long long)a.n_seq * a.Hk));
  p.parts = (int)std::min(parts, room);
  const dim3 grid(p.parts, (unsigned)(a.n_seq * a.Hk));
  const double bytes = 4.0 * (double)a.n_seq * a.Hk * most * a.d * (a.bf16 ? 2 : 4);
  ProfScope ps(PT_WIN_STORE, a.stream, 0.0, bytes);
  cudaError_t e;
  if (a.bf16)
    e = vec ? launch_grid(window_store_kernel<__nv_bfloat16, true>, grid, 256, 0, a.stream, p)
            : launch_grid(window_store_kernel<__nv_bfloat16, false>, grid, 256, 0, a.stream, p);
  else
    e = vec ? launch_grid(window_store_kernel<float, true>, grid, 256, 0, a.stream, p)
            : launch_grid(window_store_kernel<float, false>, grid, 256, 0, a.stream, p);
  return e == cudaSuccess ? TTT_OK : TTT_ERR_CUDA;
}

}  // namespace ttt
