// Attention with a sliding window and sinks in fp32, for every type, size and stride, and
// the writing of new keys and values into the caches.
#include <algorithm>

#include "prof.h"
#include "win_rows.cuh"

namespace ttt {

namespace {

// ------------------------------------------------------------ prompts, fp32
// One CTA: QT queries of one head.
template <typename T, int DP, int QT, bool VEC>
__global__ void __launch_bounds__(2 * QT) window_attention_kernel(
    const __grid_constant__ WinParams p) {
  extern __shared__ __align__(16) float sm[];
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0 && p.starts) check_starts(p.starts, p.n_seq, p.N, p.status);
  window_rows<T, DP, QT, VEC, QT / 16, false>(p, blockIdx.z, blockIdx.y, blockIdx.x * QT, sm);
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
  int past = p.past ? p.past[s] : 0;
  if (past < 0) {
    if (first && threadIdx.x == 0) report_status(p.status, kStatusBadArg);
    past = 0;
  }
  int t0 = 0, t1 = p.N, b = s;
  if (p.starts) {
    t0 = p.starts[s];
    t1 = p.starts[s + 1];
    b = 0;
    if (t0 < 0 || t1 <= t0 || t1 > p.N) return;
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
