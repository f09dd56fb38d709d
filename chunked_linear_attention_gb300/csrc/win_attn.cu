// Attention with a sliding window and sinks in fp32, for every type, size and stride, and
// the writing of new keys and values into the caches.
#include "prof.h"
#include "win_attn.cuh"

namespace ttt {

namespace {

// ------------------------------------------------------------ prompts, fp32
// One CTA: 64 queries of one head against key tiles of 64, 256 threads.  A thread
// holds 4 x 4 scores and 4 rows x DP / 16 columns of the output; running maximum and
// sum of the softmax per row, so that each score is made once.  Bound by the fp32 pipe
// (16 products for 8 words of shared memory in the scores, 4 DP / 16 for 4 + DP / 16 in
// the outputs).
constexpr int kQT = 64, kKT = 64, kPad = 4;

template <int DP>
constexpr int simt_smem() {
  return (DP * (kQT + kPad) * 2 + kKT * DP + kKT * (kQT + kPad)) * 4;
}

template <typename T, int DP>
__global__ void __launch_bounds__(256) window_attention_kernel(const __grid_constant__ WinParams p) {
  extern __shared__ __align__(16) float sm[];
  float* Qt = sm;                              // [DP][kQT + kPad]
  float* Kt = Qt + DP * (kQT + kPad);          // [DP][kKT + kPad]
  float* V = Kt + DP * (kKT + kPad);           // [kKT][DP]
  float* Pt = V + kKT * DP;                    // [kKT][kQT + kPad]
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.z, h = blockIdx.y, i0 = blockIdx.x * kQT;
  const int hk = h / (p.Hq / p.Hk);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  if (blockIdx.x == 0 && h == 0 && p.starts) check_starts(p.starts, p.n_seq, p.N, p.status);
  const T* q = static_cast<const T*>(p.q) + b * p.lay.q.batch + h * p.lay.q.head;
  const T* k = static_cast<const T*>(p.k) + b * p.lay.k.batch + hk * p.lay.k.head;
  const T* v = static_cast<const T*>(p.v) + b * p.lay.v.batch + hk * p.lay.v.head;
  for (int e = tid; e < kQT * DP; e += 256) {
    const int r = e / DP, c = e % DP;
    const bool in = i0 + r < p.N && c < p.d;
    Qt[c * (kQT + kPad) + r] = in ? to_f<T>(q[(i0 + r) * p.lay.q.token + c]) * p.scale : 0.f;
  }
  WinRow row[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) row[r] = win_row(p, b, i0 + ty * 4 + r);
  float m[4], l[4], o[4][DP / 16];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < DP / 16; ++c) o[r][c] = 0.f;
  }
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
    for (int e = tid; e < kKT * DP; e += 256) {
      const int r = e / DP, c = e % DP, j = t.base + r;
      const bool in = j >= 0 && j < t.end && c < p.d;
      Kt[c * (kKT + kPad) + r] = in ? to_f<T>(ks[j * sk + c]) : 0.f;
      const float x = in ? to_f<T>(vs[j * sv + c]) : 0.f;
      V[r * DP + c] = x;
      odd |= !isfinite(x);
    }
    odd = __syncthreads_or(odd);
    float s[4][4] = {};
#pragma unroll 4
    for (int c = 0; c < p.d; ++c) {
      const float4 a = *reinterpret_cast<const float4*>(Qt + c * (kQT + kPad) + ty * 4);
      const float4 x = *reinterpret_cast<const float4*>(Kt + c * (kKT + kPad) + tx * 4);
      const float aa[4] = {a.x, a.y, a.z, a.w}, xx[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int n = 0; n < 4; ++n) s[r][n] = fmaf(aa[r], xx[n], s[r][n]);
    }
    unsigned seen = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int j = t.base + tx * 4 + n;
        const bool ok = t.seq < 0 ? sees_new(row[r], j, t.end)
                                  : sees_cache(row[r], t.c, j, p.sinks, p.window);
        seen |= (unsigned)ok << (r * 4 + n);
        if (!ok) s[r][n] = -INFINITY;
        top = fmaxf(top, s[r][n]);
      }
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
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[r] = fmaf(l[r], f, sum);
      m[r] = mn;
#pragma unroll
      for (int c = 0; c < DP / 16; ++c) o[r][c] *= f;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
      *reinterpret_cast<float4*>(Pt + (tx * 4 + n) * (kQT + kPad) + ty * 4) =
          make_float4(s[0][n], s[1][n], s[2][n], s[3][n]);
    __syncthreads();
    if (!odd) {
#pragma unroll 4
      for (int n = 0; n < kKT; ++n) {
        const float4 a = *reinterpret_cast<const float4*>(Pt + n * (kQT + kPad) + ty * 4);
        const float aa[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
          const float x = V[n * DP + c * 16 + tx];
#pragma unroll
          for (int r = 0; r < 4; ++r) o[r][c] = fmaf(aa[r], x, o[r][c]);
        }
      }
    } else {
      // a value that a query does not see must not reach it, not even times 0
      for (int n = 0; n < kKT; ++n) {
        const unsigned bits = __shfl_sync(0xffffffffu, seen, (tid & 16) | (n >> 2)) >> (n & 3);
        const float4 a = *reinterpret_cast<const float4*>(Pt + n * (kQT + kPad) + ty * 4);
        const float aa[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
          const float x = V[n * DP + c * 16 + tx];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if ((bits >> (r * 4)) & 1) o[r][c] = fmaf(aa[r], x, o[r][c]);
        }
      }
    }
  }
  T* out = static_cast<T*>(p.out) + b * p.lay.out.batch + h * p.lay.out.head;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (row[r].i < 0) continue;
    const float f = 1.f / l[r];
#pragma unroll
    for (int c = 0; c < DP / 16; ++c)
      if (c * 16 + tx < p.d) out[row[r].i * p.lay.out.token + c * 16 + tx] = from_f<T>(o[r][c] * f);
  }
}

template <typename T, int DP>
int launch_simt(const WindowArgs& a, const WinParams& p) {
  auto kern = window_attention_kernel<T, DP>;
  constexpr int smem = simt_smem<DP>();
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TTT_ERR_CUDA;
  const double tok = (double)a.B * a.N;
  ProfScope ps(PT_WIN_SIMT, a.stream, 4.0 * tok * a.Hq * a.d * fmin(a.N, (double)a.window + a.sinks),
               tok * (a.bf16 ? 2 : 4) * 2.0 * a.d * (a.Hq + a.Hk));
  return launch_grid(kern, dim3((a.N + kQT - 1) / kQT, a.Hq, a.B), 256, smem, a.stream, p) ==
                 cudaSuccess
             ? TTT_OK
             : TTT_ERR_CUDA;
}

template <typename T>
int simt_t(const WindowArgs& a, const WinParams& p) {
  if (a.d <= 64) return launch_simt<T, 64>(a, p);
  if (a.d <= 128) return launch_simt<T, 128>(a, p);
  return launch_simt<T, 256>(a, p);
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
  // about eight rows of 16 bytes a thread for a full cache
  const long long most = a.N < (long long)a.window + a.sinks ? a.N : (long long)a.window + a.sinks;
  long long parts = most * a.d / per / 2048 + 1;
  p.parts = (int)(parts > 64 ? 64 : parts);
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
