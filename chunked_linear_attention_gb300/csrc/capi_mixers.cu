// The extern "C" boundary of ttt_mixers.h: argument validation on the host,
// before anything is enqueued, and dispatch.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <utility>

#include "capi_util.h"
#include "mixers.h"
#include "ttt_selftest.h"

namespace {

using ttt::capi_aligned;

// Rows of `len` elements on the given axes (distance, count) that do not lie on one
// another: from the closest axis to the farthest, each begins behind the one before.
bool rows_apart(std::pair<long long, int>* ax, int n, long long len) {
  std::sort(ax, ax + n);
  long long end = len;
  for (int i = 0; i < n; ++i) {
    if (ax[i].second == 1) continue;
    if (ax[i].first < end || ax[i].first > (1LL << 61) / ax[i].second) return false;
    end += ax[i].first * (ax[i].second - 1);
  }
  return true;
}

bool not_negative(const delta_rule_stride& s) { return s.batch >= 0 && s.head >= 0 && s.token >= 0; }
bool not_negative(const mixer_stride& s) { return s.batch >= 0 && s.token >= 0; }

int io_bytes(int io) { return io == TTT_BF16 ? 2 : 4; }

// ---------------------------------------------------------------- attention
int check_window(int B, int Hq, int Hk, int N, int d, int window, int sinks, int io, bool cache) {
  if (B <= 0 || Hq <= 0 || Hk <= 0 || N <= 0 || d <= 0 || Hq % Hk != 0) return TTT_ERR_SHAPE;
  if (window <= 0 || sinks < 0) return TTT_ERR_SHAPE;
  if (io != TTT_F32 && io != TTT_BF16) return TTT_ERR_ARG;
  if (d > 256 || window > (1 << 30) || sinks > (1 << 30) ||
      (cache && (long long)window + sinks > 1 << 30))
    return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

window_attention_layout window_layout(const window_attention_layout* layout, long long Hq,
                                      long long Hk, long long N, long long d) {
  if (layout) return *layout;
  window_attention_layout L;
  L.q = L.out = {Hq * N * d, N * d, d};
  L.k = L.v = {Hk * N * d, N * d, d};
  return L;
}

int check_window_tensors(const window_attention_layout& L, int B, int Hq, int N, int d, int io,
                         const void* q, const void* k, const void* v, const void* ck,
                         const void* cv, const void* out) {
  if (!not_negative(L.q) || !not_negative(L.k) || !not_negative(L.v) || !not_negative(L.out))
    return TTT_ERR_ARG;
  std::pair<long long, int> ax[3] = {{L.out.batch, B}, {L.out.head, Hq}, {L.out.token, N}};
  if (!rows_apart(ax, 3, d)) return TTT_ERR_ARG;
  if (out == q || out == k || out == v) return TTT_ERR_ARG;
  if (ck && (ck == cv || ck == out || cv == out || ck == k || ck == v || cv == k || cv == v ||
             ck == q || cv == q))
    return TTT_ERR_ARG;
  const unsigned es = io_bytes(io);
  if (!capi_aligned(q, es) || !capi_aligned(k, es) || !capi_aligned(v, es) ||
      !capi_aligned(out, es) || !capi_aligned(ck, 16) || !capi_aligned(cv, 16))
    return TTT_ERR_ALIGN;
  return TTT_OK;
}

// ---------------------------------------------------------------- scan and convolution
int check_rows(int n_seq, int B, int N, int D, int io) {
  if (B <= 0 || N <= 0 || D <= 0 || n_seq <= 0) return TTT_ERR_SHAPE;
  if (B != 1 && n_seq != B) return TTT_ERR_SHAPE;
  if (io != TTT_F32 && io != TTT_BF16) return TTT_ERR_ARG;
  if (B > 65535 || D > 32768 || n_seq > (1 << 20) || N > (1 << 30) ||
      (long long)B * N > (1LL << 31) - 1)
    return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

int check_scan(int n_seq, int B, int N, int D, int S, int G, int io) {
  if (S <= 0 || G <= 0) return TTT_ERR_SHAPE;
  const int rc = check_rows(n_seq, B, N, D, io);
  if (rc != TTT_OK) return rc;
  if (D % G != 0) return TTT_ERR_SHAPE;
  return S > 128 ? TTT_ERR_UNSUPPORTED : TTT_OK;
}

selective_scan_layout scan_layout(const selective_scan_layout* layout, long long N, long long D,
                                  long long GS) {
  if (layout) return *layout;
  selective_scan_layout L;
  L.x = L.dt = L.z = L.out = {N * D, D};
  L.B = L.C = {N * GS, GS};
  return L;
}

bool out_rows(const mixer_stride& s, int B, int N, int D) {
  std::pair<long long, int> ax[2] = {{s.batch, B}, {s.token, N}};
  return rows_apart(ax, 2, D);
}

bool scan_strides(const selective_scan_layout& L, int B, int N, int D) {
  return not_negative(L.x) && not_negative(L.dt) && not_negative(L.z) && not_negative(L.B) &&
         not_negative(L.C) && not_negative(L.out) && out_rows(L.out, B, N, D);
}

}  // namespace

extern "C" {

int window_attention_forward(const void* q, const void* k, const void* v, void* cache_k,
                             void* cache_v, const int* slots, int n_slots, const int* past,
                             const int* seq_starts, int n_seq, int B, int Hq, int Hk, int N, int d,
                             int window, int sinks, int io_dtype, float scale,
                             const window_attention_layout* layout, void* out,
                             ttt_stream_t stream) {
  if (!q || !k || !v || !out) return TTT_ERR_NULL;
  if ((cache_k != nullptr) != (cache_v != nullptr)) return TTT_ERR_NULL;
  if (!cache_k && (past || slots)) return TTT_ERR_NULL;
  int rc = check_window(B, Hq, Hk, N, d, window, sinks, io_dtype, cache_k != nullptr);
  if (rc != TTT_OK) return rc;
  if (n_seq <= 0 || (seq_starts ? B != 1 : n_seq != B)) return TTT_ERR_SHAPE;
  if (cache_k && (n_slots <= 0 || (!slots && n_slots < n_seq))) return TTT_ERR_SHAPE;
  if ((long long)Hq * B > 65535 || (long long)Hq * n_seq > 65535 ||
      (long long)B * N > (1LL << 31) - 1 || N > (1 << 30))
    return TTT_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return TTT_ERR_ARG;
  const window_attention_layout L = window_layout(layout, Hq, Hk, N, d);
  rc = check_window_tensors(L, B, Hq, N, d, io_dtype, q, k, v, cache_k, cache_v, out);
  if (rc != TTT_OK) return rc;
  if (!capi_aligned(slots, 4) || !capi_aligned(past, 4) || !capi_aligned(seq_starts, 4))
    return TTT_ERR_ALIGN;
  int* st = ttt::capi_status_ptr();
  if (!st) return TTT_ERR_CUDA;
  ttt::WindowArgs a;
  a.q = q; a.k = k; a.v = v; a.cache_k = cache_k; a.cache_v = cache_v;
  a.slots = slots; a.past = past; a.seq_starts = seq_starts;
  a.n_slots = n_slots; a.n_seq = n_seq; a.B = B; a.Hq = Hq; a.Hk = Hk; a.N = N; a.d = d;
  a.window = window; a.sinks = sinks;
  a.bf16 = io_dtype == TTT_BF16;
  a.scale = scale;
  a.lay = L;
  a.out = out;
  a.status = st;
  a.wait_ns = ttt::capi_wait_limit_ns();
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  rc = ttt::window_attention_tc(a);
  if (rc == 1) rc = ttt::window_attention_simt(a);
  if (rc == TTT_OK && cache_k) rc = ttt::window_attention_store(a);
  return rc;
}

int window_attention_step(const void* q, const void* k, const void* v, void* cache_k,
                          void* cache_v, const int* positions, const int* slots, int n_slots,
                          int B, int Hq, int Hk, int d, int window, int sinks, int io_dtype,
                          float scale, const window_attention_layout* layout, void* out,
                          ttt_stream_t stream) {
  if (!q || !k || !v || !cache_k || !cache_v || !positions || !out) return TTT_ERR_NULL;
  int rc = check_window(B, Hq, Hk, 1, d, window, sinks, io_dtype, true);
  if (rc != TTT_OK) return rc;
  if (n_slots <= 0 || (!slots && n_slots < B)) return TTT_ERR_SHAPE;
  if ((long long)Hq * B > (1 << 20) || B > 65535) return TTT_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return TTT_ERR_ARG;
  const window_attention_layout L = window_layout(layout, Hq, Hk, 1, d);
  rc = check_window_tensors(L, B, Hq, 1, d, io_dtype, q, k, v, cache_k, cache_v, out);
  if (rc != TTT_OK) return rc;
  if (!capi_aligned(slots, 4) || !capi_aligned(positions, 4)) return TTT_ERR_ALIGN;
  int* st = ttt::capi_status_ptr();
  if (!st) return TTT_ERR_CUDA;
  ttt::WindowStepArgs a;
  a.q = q; a.k = k; a.v = v; a.cache_k = cache_k; a.cache_v = cache_v;
  a.positions = positions;
  a.slots = slots;
  a.n_slots = n_slots; a.B = B; a.Hq = Hq; a.Hk = Hk; a.d = d; a.window = window; a.sinks = sinks;
  a.bf16 = io_dtype == TTT_BF16;
  a.scale = scale;
  a.lay = L;
  a.out = out;
  a.status = st;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return ttt::window_attention_step_launch(a);
}

size_t selective_scan_workspace_size(int B, int N, int D, int S, int G, int n_seq, int io_dtype) {
  if (check_scan(n_seq, B, N, D, S, G, io_dtype) != TTT_OK) return 0;
  const size_t need = ttt::selective_scan_workspace(B, N, D, S, G, n_seq, io_dtype == TTT_BF16);
  return need < 256 ? 256 : need;
}

int selective_scan_forward(const void* x, const void* dt, const float* A, const void* Bm,
                           const void* Cm, const float* Dx, const float* dt_bias, const void* z,
                           const float* state_in, const int* seq_starts, int n_seq, int B, int N,
                           int D, int S, int G, int io_dtype, int dt_softplus,
                           const selective_scan_layout* layout, void* out, float* state_out,
                           void* workspace, size_t workspace_bytes, ttt_stream_t stream) {
  if (!x || !dt || !A || !Bm || !Cm || !out) return TTT_ERR_NULL;
  int rc = check_scan(n_seq, B, N, D, S, G, io_dtype);
  if (rc != TTT_OK) return rc;
  if (seq_starts ? B != 1 : n_seq != B) return TTT_ERR_SHAPE;
  if (dt_softplus != 0 && dt_softplus != 1) return TTT_ERR_ARG;
  const selective_scan_layout L = scan_layout(layout, N, D, (long long)G * S);
  if (!scan_strides(L, B, N, D)) return TTT_ERR_ARG;
  if (out == x || out == dt || out == z || out == Bm || out == Cm ||
      (state_out && (state_out == state_in || (void*)state_out == out)))
    return TTT_ERR_ARG;
  const unsigned es = io_bytes(io_dtype);
  if (!capi_aligned(x, es) || !capi_aligned(dt, es) || !capi_aligned(z, es) ||
      !capi_aligned(Bm, es) || !capi_aligned(Cm, es) || !capi_aligned(out, es) ||
      !capi_aligned(A, 4) || !capi_aligned(Dx, 4) || !capi_aligned(dt_bias, 4) ||
      !capi_aligned(state_in, 4) || !capi_aligned(state_out, 4) || !capi_aligned(seq_starts, 4))
    return TTT_ERR_ALIGN;
  if (!workspace ||
      workspace_bytes < selective_scan_workspace_size(B, N, D, S, G, n_seq, io_dtype))
    return TTT_ERR_WORKSPACE;
  if (!capi_aligned(workspace, 256)) return TTT_ERR_ALIGN;
  int* st = ttt::capi_status_ptr();
  if (!st) return TTT_ERR_CUDA;
  ttt::ScanArgs a;
  a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dx = Dx; a.dt_bias = dt_bias; a.z = z;
  a.state_in = state_in;
  a.seq_starts = seq_starts;
  a.n_seq = n_seq; a.B = B; a.N = N; a.D = D; a.S = S; a.G = G;
  a.bf16 = io_dtype == TTT_BF16;
  a.softplus = dt_softplus;
  a.lay = L;
  a.out = out;
  a.state_out = state_out;
  a.workspace = workspace;
  a.status = st;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return ttt::selective_scan_launch(a);
}

int selective_scan_step(const void* x, const void* dt, const float* A, const void* Bm,
                        const void* Cm, const float* Dx, const float* dt_bias, const void* z,
                        float* state, const int* slots, int n_slots, int B, int D, int S, int G,
                        int io_dtype, int dt_softplus, const selective_scan_layout* layout,
                        void* out, ttt_stream_t stream) {
  if (!x || !dt || !A || !Bm || !Cm || !state || !out) return TTT_ERR_NULL;
  int rc = check_scan(B, B, 1, D, S, G, io_dtype);
  if (rc != TTT_OK) return rc;
  if (n_slots <= 0 || (!slots && n_slots < B)) return TTT_ERR_SHAPE;
  if (dt_softplus != 0 && dt_softplus != 1) return TTT_ERR_ARG;
  const selective_scan_layout L = scan_layout(layout, 1, D, (long long)G * S);
  if (!scan_strides(L, B, 1, D)) return TTT_ERR_ARG;
  if (out == x || out == dt || out == z || out == Bm || out == Cm || out == (void*)state)
    return TTT_ERR_ARG;
  const unsigned es = io_bytes(io_dtype);
  if (!capi_aligned(x, es) || !capi_aligned(dt, es) || !capi_aligned(z, es) ||
      !capi_aligned(Bm, es) || !capi_aligned(Cm, es) || !capi_aligned(out, es) ||
      !capi_aligned(A, 4) || !capi_aligned(Dx, 4) || !capi_aligned(dt_bias, 4) ||
      !capi_aligned(state, 4) || !capi_aligned(slots, 4))
    return TTT_ERR_ALIGN;
  int* st = ttt::capi_status_ptr();
  if (!st) return TTT_ERR_CUDA;
  ttt::ScanStepArgs a;
  a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.Dx = Dx; a.dt_bias = dt_bias; a.z = z;
  a.state = state;
  a.slots = slots;
  a.n_slots = n_slots; a.B = B; a.D = D; a.S = S; a.G = G;
  a.bf16 = io_dtype == TTT_BF16;
  a.softplus = dt_softplus;
  a.lay = L;
  a.out = out;
  a.status = st;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return ttt::selective_scan_step_launch(a);
}

int short_conv_forward(const void* x, const float* w, const float* bias, const void* state_in,
                       const int* seq_starts, int n_seq, int B, int N, int D, int W, int io_dtype,
                       int silu, const short_conv_layout* layout, void* out, void* state_out,
                       ttt_stream_t stream) {
  if (!x || !w || !out) return TTT_ERR_NULL;
  int rc = check_rows(n_seq, B, N, D, io_dtype);
  if (rc != TTT_OK) return rc;
  if (seq_starts ? B != 1 : n_seq != B) return TTT_ERR_SHAPE;
  if (W < 2) return TTT_ERR_SHAPE;
  if (W > 8) return TTT_ERR_UNSUPPORTED;
  if (silu != 0 && silu != 1) return TTT_ERR_ARG;
  short_conv_layout L;
  if (layout) L = *layout;
  else L.x = L.out = {(long long)N * D, D};
  if (!not_negative(L.x) || !not_negative(L.out) || !out_rows(L.out, B, N, D)) return TTT_ERR_ARG;
  if (out == x || out == state_in || (state_out && (state_out == state_in || state_out == out ||
                                                    state_out == x)))
    return TTT_ERR_ARG;
  const unsigned es = io_bytes(io_dtype);
  if (!capi_aligned(x, es) || !capi_aligned(out, es) || !capi_aligned(state_in, es) ||
      !capi_aligned(state_out, es) || !capi_aligned(w, 4) || !capi_aligned(bias, 4) ||
      !capi_aligned(seq_starts, 4))
    return TTT_ERR_ALIGN;
  int* st = ttt::capi_status_ptr();
  if (!st) return TTT_ERR_CUDA;
  ttt::ConvArgs a;
  a.x = x; a.w = w; a.bias = bias; a.state_in = state_in;
  a.seq_starts = seq_starts;
  a.n_seq = n_seq; a.B = B; a.N = N; a.D = D; a.W = W;
  a.bf16 = io_dtype == TTT_BF16;
  a.silu = silu;
  a.lay = L;
  a.out = out;
  a.state_out = state_out;
  a.status = st;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return ttt::short_conv_launch(a);
}

int short_conv_step(const void* x, const float* w, const float* bias, void* state,
                    const int* slots, int n_slots, int B, int D, int W, int io_dtype, int silu,
                    const short_conv_layout* layout, void* out, ttt_stream_t stream) {
  if (!x || !w || !state || !out) return TTT_ERR_NULL;
  int rc = check_rows(B, B, 1, D, io_dtype);
  if (rc != TTT_OK) return rc;
  if (W < 2) return TTT_ERR_SHAPE;
  if (W > 8) return TTT_ERR_UNSUPPORTED;
  if (n_slots <= 0 || (!slots && n_slots < B)) return TTT_ERR_SHAPE;
  if (silu != 0 && silu != 1) return TTT_ERR_ARG;
  short_conv_layout L;
  if (layout) L = *layout;
  else L.x = L.out = {D, D};
  if (!not_negative(L.x) || !not_negative(L.out) || !out_rows(L.out, B, 1, D)) return TTT_ERR_ARG;
  if (out == x || out == state || x == state) return TTT_ERR_ARG;
  const unsigned es = io_bytes(io_dtype);
  if (!capi_aligned(x, es) || !capi_aligned(out, es) || !capi_aligned(state, es) ||
      !capi_aligned(w, 4) || !capi_aligned(bias, 4) || !capi_aligned(slots, 4))
    return TTT_ERR_ALIGN;
  int* st = ttt::capi_status_ptr();
  if (!st) return TTT_ERR_CUDA;
  ttt::ConvStepArgs a;
  a.x = x; a.w = w; a.bias = bias; a.state = state;
  a.slots = slots;
  a.n_slots = n_slots; a.B = B; a.D = D; a.W = W;
  a.bf16 = io_dtype == TTT_BF16;
  a.silu = silu;
  a.lay = L;
  a.out = out;
  a.status = st;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return ttt::short_conv_step_launch(a);
}

void ttt_selftest_withhold_window(int what) { ttt::window_attention_withhold(what); }

// The Python binding's forms of the calls: their arguments in one record each (a call with
// 24 arguments through ctypes takes 7 us of the host's time, one with a record 1.5).  The
// records' fields lie as struct.pack puts them; the binding compares their sizes when it loads
// the library (ttt_binding_record_bytes).
struct WindowRecord {
  const void *q, *k, *v;
  void *cache_k, *cache_v;
  const int *slots, *past, *seq_starts;
  void* out;
  ttt_stream_t stream;
  window_attention_layout lay;
  int n_slots, n_seq, B, Hq, Hk, N, d, window, sinks, io;
  float scale;
};

int ttt_binding_window_forward(const WindowRecord* r) {
  return window_attention_forward(r->q, r->k, r->v, r->cache_k, r->cache_v, r->slots, r->n_slots,
                                  r->past, r->seq_starts, r->n_seq, r->B, r->Hq, r->Hk, r->N, r->d,
                                  r->window, r->sinks, r->io, r->scale, &r->lay, r->out, r->stream);
}

// past: the positions; n_seq and N are not used.
int ttt_binding_window_step(const WindowRecord* r) {
  return window_attention_step(r->q, r->k, r->v, r->cache_k, r->cache_v, r->past, r->slots,
                               r->n_slots, r->B, r->Hq, r->Hk, r->d, r->window, r->sinks, r->io,
                               r->scale, &r->lay, r->out, r->stream);
}

struct ScanRecord {
  const void *x, *dt;
  const float* A;
  const void *B, *C;
  const float *D, *dt_bias;
  const void* z;
  const float* state;
  const int* index;   // seq_starts or slots
  void* out;
  float* state_out;   // or the pool
  void* workspace;
  size_t workspace_bytes;
  ttt_stream_t stream;
  selective_scan_layout lay;
  int n, batch, N, channels, S, G, io, softplus;   // n: sequences or slots
};

int ttt_binding_scan_forward(const ScanRecord* r) {
  return selective_scan_forward(r->x, r->dt, r->A, r->B, r->C, r->D, r->dt_bias, r->z, r->state,
                                r->index, r->n, r->batch, r->N, r->channels, r->S, r->G, r->io,
                                r->softplus, &r->lay, r->out, r->state_out, r->workspace,
                                r->workspace_bytes, r->stream);
}

int ttt_binding_scan_step(const ScanRecord* r) {
  return selective_scan_step(r->x, r->dt, r->A, r->B, r->C, r->D, r->dt_bias, r->z, r->state_out,
                             r->index, r->n, r->batch, r->channels, r->S, r->G, r->io, r->softplus,
                             &r->lay, r->out, r->stream);
}

struct ConvRecord {
  const void* x;
  const float *w, *bias;
  const void* state;
  const int* index;
  void *out, *state_out;
  ttt_stream_t stream;
  short_conv_layout lay;
  int n, B, N, D, W, io, silu;
};

int ttt_binding_conv_forward(const ConvRecord* r) {
  return short_conv_forward(r->x, r->w, r->bias, r->state, r->index, r->n, r->B, r->N, r->D, r->W,
                            r->io, r->silu, &r->lay, r->out, r->state_out, r->stream);
}

int ttt_binding_conv_step(const ConvRecord* r) {
  return short_conv_step(r->x, r->w, r->bias, r->state_out, r->index, r->n, r->B, r->D, r->W, r->io,
                         r->silu, &r->lay, r->out, r->stream);
}

// Up to the end of the last field, as struct.pack makes them, of the window attention's (0), the
// scan's (1) and the convolution's record (2).
size_t ttt_binding_record_bytes(int which) {
  if (which == 0) return offsetof(WindowRecord, scale) + sizeof(float);
  if (which == 1) return offsetof(ScanRecord, softplus) + sizeof(int);
  return offsetof(ConvRecord, silu) + sizeof(int);
}

}  // extern "C"
