// The extern "C" boundary of ttt_delta.h: argument validation on the host,
// before anything is enqueued, and dispatch.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <utility>

#include "capi_util.h"
#include "delta_rule.h"
#include "ttt_selftest.h"

namespace {

using ttt::capi_aligned;

int check_rule(int B, int Hk, int Hv, int N, int dk, int dv, int n_seq, int io) {
  if (B <= 0 || Hk <= 0 || Hv <= 0 || N <= 0 || dk <= 0 || dv <= 0 || n_seq <= 0)
    return TTT_ERR_SHAPE;
  if (Hv % Hk != 0) return TTT_ERR_SHAPE;
  if (B != 1 && n_seq != B) return TTT_ERR_SHAPE;
  if (io != TTT_F32 && io != TTT_BF16) return TTT_ERR_ARG;
  if (dk > 512 || dv > 1024) return TTT_ERR_UNSUPPORTED;
  if ((long long)n_seq * Hv > (1 << 20) || (long long)B * Hv * N > (1LL << 31) - 1)
    return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

delta_rule_layout dense_layout(long long Hk, long long Hv, long long N, long long dk,
                               long long dv) {
  delta_rule_layout L;
  L.q = L.k = {Hk * N * dk, N * dk, dk};
  L.v = L.out = {Hv * N * dv, N * dv, dv};
  L.g = L.beta = {Hv * N, N, 1};
  return L;
}

// Strides a call may have: none negative, and no two rows of the output on one
// another (from the closest axis to the farthest, each begins behind the one before).
bool layout_ok(const delta_rule_layout& L, int B, int Hv, int N, int dv) {
  const delta_rule_stride* s[] = {&L.q, &L.k, &L.v, &L.g, &L.beta, &L.out};
  for (const delta_rule_stride* x : s)
    if (x->batch < 0 || x->head < 0 || x->token < 0) return false;
  std::pair<long long, int> ax[3] = {{L.out.batch, B}, {L.out.head, Hv}, {L.out.token, N}};
  std::sort(ax, ax + 3);
  long long end = dv;
  for (const auto& a : ax) {
    if (a.second == 1) continue;
    if (a.first < end || a.first > (1LL << 61) / a.second) return false;
    end += a.first * (a.second - 1);
  }
  return true;
}

// A tensor written over another one row by row: the same rows, or another tensor.
bool rows_match(const void* to, long long sto, const void* from, long long sfrom, bool same_type,
                long long rows) {
  return to != from || (same_type && (rows == 1 || sto == sfrom));
}

}  // namespace

extern "C" {

size_t delta_rule_workspace_size(int B, int Hk, int Hv, int N, int d_k, int d_v, int n_seq,
                                 int io_dtype) {
  if (check_rule(B, Hk, Hv, N, d_k, d_v, n_seq, io_dtype) != TTT_OK) return 0;
  const size_t need =
      io_dtype == TTT_BF16 ? ttt::delta_rule_chunk_workspace(B, Hv, N, d_k, d_v, n_seq) : 0;
  return need < 256 ? 256 : need;
}

int delta_rule_chunked_forward(const void* q, const void* k, const void* v, const float* g,
                               const float* beta, const float* S0, const int* seq_starts,
                               int n_seq, int B, int Hk, int Hv, int N, int d_k, int d_v,
                               int io_dtype, float scale, const delta_rule_layout* layout,
                               void* out, float* S_final, void* workspace,
                               size_t workspace_bytes, ttt_stream_t stream) {
  if (!q || !k || !v || !g || !beta || !out) return TTT_ERR_NULL;
  int rc = check_rule(B, Hk, Hv, N, d_k, d_v, n_seq, io_dtype);
  if (rc != TTT_OK) return rc;
  if (!seq_starts && n_seq != B) return TTT_ERR_SHAPE;
  if (seq_starts && B != 1) return TTT_ERR_SHAPE;
  if (!std::isfinite(scale)) return TTT_ERR_ARG;
  const delta_rule_layout L = layout ? *layout : dense_layout(Hk, Hv, N, d_k, d_v);
  if (!layout_ok(L, B, Hv, N, d_v)) return TTT_ERR_ARG;
  if (out == q || out == k || out == v) return TTT_ERR_ARG;
  const unsigned es = io_dtype == TTT_BF16 ? 2 : 4;
  if (!capi_aligned(q, es) || !capi_aligned(k, es) || !capi_aligned(v, es) ||
      !capi_aligned(out, es) || !capi_aligned(g, 4) || !capi_aligned(beta, 4) ||
      !capi_aligned(seq_starts, 4) || !capi_aligned(S0, 16) || !capi_aligned(S_final, 16))
    return TTT_ERR_ALIGN;
  if (!workspace ||
      workspace_bytes < delta_rule_workspace_size(B, Hk, Hv, N, d_k, d_v, n_seq, io_dtype))
    return TTT_ERR_WORKSPACE;
  if (!capi_aligned(workspace, 256)) return TTT_ERR_ALIGN;
  int* st = ttt::capi_status_ptr();
  if (!st) return TTT_ERR_CUDA;
  ttt::DeltaArgs a;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.S0 = S0;
  a.seq_starts = seq_starts;
  a.n_seq = n_seq; a.B = B; a.Hk = Hk; a.Hv = Hv; a.N = N; a.dk = d_k; a.dv = d_v;
  a.bf16 = io_dtype == TTT_BF16;
  a.scale = scale;
  a.lay = L;
  a.out = out;
  a.S_final = S_final;
  a.workspace = workspace;
  a.status = st;
  a.wait_ns = ttt::capi_wait_limit_ns();
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  rc = ttt::delta_rule_chunk_launch(a);
  return rc == 1 ? ttt::delta_rule_recurrent(a) : rc;
}

int delta_rule_step(const void* q, const void* k, const void* v, const float* g,
                    const float* beta, float* state, const int* slots, int n_slots, int B, int Hk,
                    int Hv, int d_k, int d_v, int io_dtype, float scale,
                    const delta_rule_layout* layout, void* out, ttt_stream_t stream) {
  if (!q || !k || !v || !g || !beta || !state || !out) return TTT_ERR_NULL;
  int rc = check_rule(B, Hk, Hv, 1, d_k, d_v, B, io_dtype);
  if (rc != TTT_OK) return rc;
  if (n_slots <= 0 || (!slots && n_slots < B)) return TTT_ERR_SHAPE;
  if (!std::isfinite(scale)) return TTT_ERR_ARG;
  const delta_rule_layout L = layout ? *layout : dense_layout(Hk, Hv, 1, d_k, d_v);
  if (!layout_ok(L, B, Hv, 1, d_v)) return TTT_ERR_ARG;
  if (out == q || out == k || out == v || out == state) return TTT_ERR_ARG;
  const unsigned es = io_dtype == TTT_BF16 ? 2 : 4;
  if (!capi_aligned(q, es) || !capi_aligned(k, es) || !capi_aligned(v, es) ||
      !capi_aligned(out, es) || !capi_aligned(g, 4) || !capi_aligned(beta, 4) ||
      !capi_aligned(slots, 4) || !capi_aligned(state, 16))
    return TTT_ERR_ALIGN;
  int* st = ttt::capi_status_ptr();
  if (!st) return TTT_ERR_CUDA;
  ttt::DeltaStepArgs a;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
  a.state = state;
  a.slots = slots;
  a.n_slots = n_slots; a.B = B; a.Hk = Hk; a.Hv = Hv; a.dk = d_k; a.dv = d_v;
  a.bf16 = io_dtype == TTT_BF16;
  a.scale = scale;
  a.lay = L;
  a.out = out;
  a.status = st;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return ttt::delta_rule_step_launch(a);
}

void ttt_selftest_withhold_delta(int kernel) { ttt::delta_rule_withhold(kernel); }

int block_norm_forward(const void* y, const float* w, const void* gate, const void* residual,
                       const float* scale, const float* w_next, long long rows, int D, int group,
                       int io_dtype, int stream_dtype, int gate_act, float eps,
                       const block_norm_strides* strides, void* out, void* h,
                       ttt_stream_t stream) {
  if (!y || !out) return TTT_ERR_NULL;
  if (gate_act < BLOCK_GATE_NONE || gate_act > BLOCK_GATE_SIGMOID) return TTT_ERR_ARG;
  if ((gate_act != BLOCK_GATE_NONE) != (gate != nullptr)) return TTT_ERR_NULL;
  if ((w_next != nullptr) != (h != nullptr)) return TTT_ERR_NULL;
  if (rows <= 0 || D <= 0 || group <= 0 || D % group != 0) return TTT_ERR_SHAPE;
  if (io_dtype != TTT_F32 && io_dtype != TTT_BF16) return TTT_ERR_ARG;
  if (stream_dtype != TTT_F32 && stream_dtype != TTT_BF16) return TTT_ERR_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return TTT_ERR_ARG;
  if (D > 16384 || rows > (1LL << 31) - 1) return TTT_ERR_UNSUPPORTED;
  ttt::BlockNormArgs a;
  a.st = strides ? *strides : block_norm_strides{D, D, D, D, D};
  // rows of a tensor may not overlap (inputs may repeat one row: stride 0)
  if (a.st.y < 0 || a.st.gate < 0 || a.st.residual < 0 || (rows > 1 && a.st.out < D) ||
      (h && rows > 1 && a.st.h < D))
    return TTT_ERR_ARG;
  const bool one_type = io_dtype == stream_dtype;
  if (!rows_match(out, a.st.out, y, a.st.y, one_type, rows) ||
      !rows_match(out, a.st.out, residual, a.st.residual, true, rows) ||
      !rows_match(out, a.st.out, gate, a.st.gate, one_type, rows) || out == h ||
      (h && (h == y || h == residual || h == gate)))
    return TTT_ERR_ARG;
  const unsigned es = io_dtype == TTT_BF16 ? 2 : 4, ss = stream_dtype == TTT_BF16 ? 2 : 4;
  if (!capi_aligned(y, es) || !capi_aligned(gate, es) || !capi_aligned(h, es) ||
      !capi_aligned(residual, ss) || !capi_aligned(out, ss) || !capi_aligned(w, 4) ||
      !capi_aligned(scale, 4) || !capi_aligned(w_next, 4))
    return TTT_ERR_ALIGN;
  a.y = y; a.w = w; a.gate = gate; a.residual = residual; a.scale = scale; a.w_next = w_next;
  a.rows = rows; a.D = D; a.group = group;
  a.io_bf16 = io_dtype == TTT_BF16;
  a.stream_bf16 = stream_dtype == TTT_BF16;
  a.act = gate_act;
  a.eps = eps;
  a.out = out;
  a.h = h;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return ttt::block_norm_launch(a);
}

}  // extern "C"
