/*
 * ttt_delta.h - C ABI of the gated delta rule (whole sequences and single
 * tokens) and of the norms around a block.
 *
 * The layer of ttt.h with a linear fast weight f_S(x) = S x and the squared
 * loss 1/2 |S k - v|^2 in place of the dot product takes one gradient step per
 * token, S <- S + beta (v - S k) k^T: the delta rule.  With a forget gate the
 * state first decays by a = exp(g).  Per sequence and value head, tokens in
 * order:
 *     S   <- a_t S                         a_t = exp(g_t)
 *     u   =  beta_t (v_t - S k_t)
 *     S   <- S + u k_t^T
 *     o_t =  scale * S q_t
 *
 * Conventions are those of ttt.h (device pointers unless an argument says
 * "host", asynchronous on `stream`, host-side argument checks before anything
 * is enqueued, no allocation on the call path).  After a bounded wait that ran out
 * (TTT_ERR_TIMEOUT in the device status word) the results of the call are
 * undefined; nothing but its outputs is touched.  The states are fp32
 * throughout.  Tensors need not be dense: see delta_rule_layout.
 *
 * Heads: q and k have Hk heads, v, g, beta, out and the state Hv heads; Hv is
 * a multiple of Hk, and value head h reads key head h / (Hv / Hk).
 */
#ifndef TTT_GB300_TTT_DELTA_H
#define TTT_GB300_TTT_DELTA_H

#include "ttt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Distances in elements between neighbouring sequences, heads and tokens of a
 * tensor (the last dimension is always contiguous).  Not negative; a stride
 * of 0 repeats the data (inputs only). */
typedef struct {
  long long batch, head, token;
} delta_rule_stride;

/* Strides of a call's tensors (HOST struct; NULL where a call takes one means
 * dense row-major in the shapes given there). */
typedef struct {
  delta_rule_stride q, k, v, g, beta, out;
} delta_rule_layout;

/* Bytes of device workspace delta_rule_chunked_forward needs (0 if the
 * arguments are invalid; otherwise at least 256).  For the chunk form (below)
 * these are 33296 bytes per 64 tokens and value head (32 KB of matrices: 2.2 GB
 * for 131072 tokens of 32 heads) and, where sequences are cut into segments, per
 * segment and value head 64 KB and another 128 KB per 128 of d_v. */
size_t delta_rule_workspace_size(int B, int Hk, int Hv, int N, int d_k, int d_v, int n_seq,
                                 int io_dtype);

/* The gated delta rule over whole sequences.
 *
 *   q, k        [B, Hk, N, d_k] in io_dtype; v [B, Hv, N, d_v] in io_dtype.
 *   g, beta     fp32 [B, Hv, N]: log decay (usually <= 0) and write strength.
 *               The rule is stable for keys of unit length (or shorter) and
 *               0 <= beta <= 2; the caller normalises the keys.
 *   S0          fp32 [n_seq, Hv, d_v, d_k] initial states, or NULL (zeros).
 *   seq_starts  NULL: n_seq = B sequences of N tokens.  Otherwise B = 1 and
 *               int32 [n_seq + 1] on the device: sequence s is the tokens
 *               seq_starts[s] .. seq_starts[s+1] - 1 of the token axis.  Lengths
 *               may be 0.  Tokens of no sequence are not read and their rows
 *               of out are not written.  Entries that are not ascending or not
 *               within 0..N make their sequence empty and set TTT_ERR_ARG in
 *               the device status word (ttt_device_status).  Other sequences may
 *               overlap around such entries: the rows of out that several
 *               share are undefined, and from the sequence on with which their
 *               lengths add up to more than N all may be taken for empty
 *               (nothing outside the tensors is touched).
 *               They are read on the device: a captured call may be replayed
 *               with other bounds.
 *   scale       factor of the outputs (d_k^-1/2 is usual).
 *   layout      HOST pointer or NULL.
 *   out         [B, Hv, N, d_v] in io_dtype.  May not overlap an input, nor
 *               its rows one another.
 *   S_final     fp32 [n_seq, Hv, d_v, d_k], the states after each sequence's
 *               last token (S0, or zeros, for an empty one), or NULL.  May be
 *               S0 itself.
 *   workspace   at least delta_rule_workspace_size() bytes, 256-byte aligned,
 *               not shared with a concurrent call.
 *
 * io_dtype TTT_BF16 with d_k <= 128, d_k and d_v multiples of 8, and q, k, v
 * 16-byte aligned with strides that are multiples of 8 elements (and not 0)
 * runs chunks of 64 tokens on the tensor cores, every intermediate held as a
 * pair of bf16 numbers (16 bits of significand) with fp32 sums and state; there
 * a NaN or infinity in a token's k, v, g or beta may also reach the outputs of
 * the up to 63 tokens before it in its chunk.  All other calls, and ones of a few tokens,
 * run token by token in fp32.
 * Decays below exp(-104) count as exp(-104); in the chunk form a decay below
 * 2^-126, of one token or of several together, is zero.
 * Supported: d_k <= 512, d_v <= 1024, n_seq * Hv at most 2^20, and
 * B * Hv * N below 2^31.
 * S0 and S_final must be 16-byte aligned. */
int delta_rule_chunked_forward(const void* q, const void* k, const void* v, const float* g,
                               const float* beta, const float* S0, const int* seq_starts,
                               int n_seq, int B, int Hk, int Hv, int N, int d_k, int d_v,
                               int io_dtype, float scale, const delta_rule_layout* layout,
                               void* out, float* S_final, void* workspace,
                               size_t workspace_bytes, ttt_stream_t stream);

/* One token of each of B sequences, on a pool of states updated in place.
 *
 *   q, k        [B, Hk, d_k] in io_dtype; v, out [B, Hv, d_v] in io_dtype.
 *   g, beta     fp32 [B, Hv].
 *   state       fp32 [n_slots, Hv, d_v, d_k].
 *   slots       int32 [B] on the device: the state of each row, or NULL (row
 *               b uses state b; n_slots >= B).  A negative slot marks an idle
 *               row: its inputs are not read, no state is touched, and its row
 *               of out is set to zero.  A slot >= n_slots, or one that an
 *               earlier row of the call already uses, is treated as idle and
 *               sets TTT_ERR_ARG in the device status word.
 *   layout      HOST pointer or NULL; the token strides are not used.
 *   out         overlaps no other tensor.
 *
 * Computed in fp32 for both I/O types.  Supported: d_k <= 512, d_v <= 1024,
 * B * Hv <= 2^20.  state must be 16-byte aligned. */
int delta_rule_step(const void* q, const void* k, const void* v, const float* g,
                    const float* beta, float* state, const int* slots, int n_slots, int B, int Hk,
                    int Hv, int d_k, int d_v, int io_dtype, float scale,
                    const delta_rule_layout* layout, void* out, ttt_stream_t stream);

/* Activation of the gate of block_norm_forward. */
typedef enum {
  BLOCK_GATE_NONE = 0,
  BLOCK_GATE_SILU = 1,   /* z * sigmoid(z) */
  BLOCK_GATE_SIGMOID = 2 /* sigmoid(z) */
} block_gate;

/* Row strides in elements of block_norm_forward's tensors (HOST struct; NULL =
 * dense, D each). */
typedef struct {
  long long y, gate, residual, out, h;
} block_norm_strides;

/* The norms around a block, with its gate, residual scale and residual sum,
 * in one pass over each row of D elements:
 *     n   = y / sqrt(mean(y^2) + eps) * w          (mean over each group)
 *     r   = residual + scale o n o act(gate)
 *     h   = r / sqrt(mean(r^2) + eps) * w_next     (mean over the row)
 * out = r; h is computed from r before it is rounded to the stream's type.
 *
 *   y           [rows, D] in io_dtype, the block's output.
 *   group       elements per norm (D % group == 0): D for one norm of the row,
 *               d_v for a norm of each head's output.
 *   w           fp32 [group] weight of the norm after the block, or NULL (1).
 *   gate        [rows, D] in io_dtype; NULL only with BLOCK_GATE_NONE.
 *   residual    [rows, D] in stream_dtype, or NULL (0).
 *   scale       fp32 [D] residual scale, or NULL (1).
 *   out         [rows, D] in stream_dtype; may be `residual`, and may be y
 *               or gate where the two types are the same (with the same row
 *               stride).
 *   w_next      fp32 [D] weight of the norm before the next block, or NULL.
 *   h           [rows, D] in io_dtype; given exactly when w_next is.  Overlaps
 *               no other tensor.
 *
 * Computed in fp32.  Any D up to 16384; rows from 1.  Tensors whose pointers
 * are 16-byte aligned, with D, group and the row strides multiples of 8, are
 * moved with wide accesses. */
int block_norm_forward(const void* y, const float* w, const void* gate, const void* residual,
                       const float* scale, const float* w_next, long long rows, int D, int group,
                       int io_dtype, int stream_dtype, int gate_act, float eps,
                       const block_norm_strides* strides, void* out, void* h,
                       ttt_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TTT_GB300_TTT_DELTA_H */
