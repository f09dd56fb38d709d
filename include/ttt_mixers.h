/*
 * ttt_mixers.h - C ABI of sequence mixers whose state per sequence has a fixed
 * size: attention with a sliding window and a few first tokens that stay
 * visible, the selective state space scan, and the short causal convolution in
 * front of such a recurrence.  Each takes whole or packed prompts with its
 * state carried in and out, and one token of each of B sequences on a pool.
 *
 * Conventions are those of ttt.h and ttt_delta.h (device pointers unless an
 * argument says "host", asynchronous on `stream`, host-side argument checks
 * before anything is enqueued, no allocation on the call path).
 *
 * seq_starts (where a call takes it): NULL for n_seq = B sequences of N tokens.
 * Otherwise B = 1 and int32 [n_seq + 1] on the device: sequence s is the tokens
 * seq_starts[s] .. seq_starts[s+1] - 1 of the token axis.  Lengths may be 0.
 * Tokens of no sequence reach nothing and their rows of the outputs are not
 * written.  Where entries do not ascend or leave 0..N, the call sets
 * TTT_ERR_ARG in the device status word (ttt_device_status) and its results are
 * undefined (nothing outside its outputs is touched).  They are read on the
 * device: a captured call may be replayed with other bounds.
 *
 * slots of a single-token call: int32 [B] on the device, the place in the pool
 * of each row, or NULL (row b uses place b; n_slots >= B).  A negative slot
 * marks an idle row: its inputs are not read, no state is touched, and its row
 * of out is set to zero.  A slot >= n_slots, or one that an earlier row of the
 * call already uses, is treated as idle and sets TTT_ERR_ARG in the device
 * status word.
 */
#ifndef TTT_GB300_TTT_MIXERS_H
#define TTT_GB300_TTT_MIXERS_H

#include "ttt_delta.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- attention
 * Strides of window_attention_*'s tensors (HOST struct; NULL = dense row-major
 * in the shapes given there; see delta_rule_stride). */
typedef struct {
  delta_rule_stride q, k, v, out;
} window_attention_layout;

/* Attention with a sliding window over whole sequences.  With P the tokens of
 * the sequence that came before the call (its `past`), token i has position
 * t = P + i and sees position j exactly if
 *     j <= t  and  (j < sinks  or  t - j < window),
 *     out_i = sum_j softmax_j(scale q_i . k_j) v_j.
 * Query head h reads key head h / (Hq / Hk).
 *
 *   q, out      [B, Hq, N, d] in io_dtype; k, v [B, Hk, N, d] in io_dtype.
 *   window      at least 1 (the token itself counts).
 *   sinks       0 or more.
 *   cache_k,    [n_slots, Hk, sinks + window, d] in io_dtype, dense, or both
 *   cache_v     NULL.  Position p of a sequence has its key and value at place p
 *               (p < sinks) or sinks + (p - sinks) % window of its slot: the
 *               first min(P, sinks + window) places are the ones that hold
 *               something, and exactly what the next token sees together with
 *               itself, but for the oldest of a full window.  The call
 *               reads the places of the past, and when it is done they hold those
 *               of P + N tokens.  Other places stay as they were.
 *   slots       int32 [n_seq] on the device: the slot of each sequence, or NULL
 *               (sequence s uses slot s; n_slots >= n_seq).  A sequence with a
 *               negative slot has no past and leaves none.  A slot >= n_slots is
 *               treated so too and sets TTT_ERR_ARG in the device status word; a
 *               slot that several sequences share is written for the first of
 *               them, and sets TTT_ERR_ARG.
 *   past        int32 [n_seq] on the device, tokens before the call, or NULL (0).
 *               Needs the caches.  A negative number counts as 0 and sets
 *               TTT_ERR_ARG.  past + N may not pass 2^31 - 1.
 *   seq_starts  see above.
 *   scale       factor of the scores (d^-1/2 is usual).
 *   layout      HOST pointer or NULL.
 *   out         overlaps no other tensor, nor its rows one another.
 *
 * io_dtype TTT_BF16 with scale > 0, d <= 128 and a multiple of 8, and q, k, v 16-byte
 * aligned with strides that are multiples of 8 elements (and not 0), runs on the
 * tensor cores: scores, their softmax and the sums are fp32, the weights are
 * rounded to bf16 for the product with v.  All other calls run in fp32
 * throughout.  What a token does not see does not reach it, NaN and infinity
 * included; on the tensor cores at the price that rows which share a key tile with
 * NaN or infinite values are made again in fp32, some forty times as long (places
 * of a cache that hold nothing are best zero).
 * Supported: d <= 256, Hq * B and Hq * n_seq at most 65535, N at most 2^30, B * N
 * below 2^31, window and sinks at most 2^30, with caches together.  The caches must
 * be 16-byte aligned. */
int window_attention_forward(const void* q, const void* k, const void* v, void* cache_k,
                             void* cache_v, const int* slots, int n_slots, const int* past,
                             const int* seq_starts, int n_seq, int B, int Hq, int Hk, int N, int d,
                             int window, int sinks, int io_dtype, float scale,
                             const window_attention_layout* layout, void* out,
                             ttt_stream_t stream);

/* One token of each of B sequences: its key and value are put into the cache
 * and it attends to what the cache then holds.
 *
 *   q, out      [B, Hq, d]; k, v [B, Hk, d] in io_dtype (token strides unused).
 *   positions   int32 [B] on the device: the token's position, the number of
 *               tokens before it.  A negative one makes the row idle and sets
 *               TTT_ERR_ARG in the device status word.
 *   slots       see above.
 *   out         overlaps no other tensor.
 *
 * Scores, their softmax and the sums are fp32.  TTT_BF16 with d <= 128 and a
 * multiple of 8, and k and v 16-byte aligned with strides that are multiples of
 * 8 elements, takes the products through the tensor cores, with each weight as
 * two bf16 numbers (off by 2^-17); where a value that the token sees is
 * infinite, its column is NaN or infinite there.
 * Supported: d <= 256, B <= 65535, Hq * B at most 2^20, window + sinks at most
 * 2^30.  The caches must be 16-byte aligned. */
int window_attention_step(const void* q, const void* k, const void* v, void* cache_k,
                          void* cache_v, const int* positions, const int* slots, int n_slots,
                          int B, int Hq, int Hk, int d, int window, int sinks, int io_dtype,
                          float scale, const window_attention_layout* layout, void* out,
                          ttt_stream_t stream);

/* ---------------------------------------------------------------- scan
 * Distances in elements between neighbouring sequences and tokens (channels are
 * contiguous).  Not negative; a stride of 0 repeats the data (inputs only). */
typedef struct {
  long long batch, token;
} mixer_stride;

/* Strides of selective_scan_*'s tensors (HOST struct; NULL = dense). */
typedef struct {
  mixer_stride x, dt, z, B, C, out;
} selective_scan_layout;

/* Bytes of device workspace selective_scan_forward needs (0 if the arguments
 * are invalid; otherwise at least 256). */
size_t selective_scan_workspace_size(int B, int N, int D, int S, int G, int n_seq, int io_dtype);

/* The selective state space scan over whole sequences.  Per sequence and channel
 * c (of group c / (D / G)), tokens in order, with a state h of S numbers:
 *     r    = softplus(dt_t + dt_bias)      (dt_softplus 0: dt_t + dt_bias)
 *     h    = exp(r A) h + r x_t B_t
 *     y_t  = C_t . h + Dx x_t
 *     out_t = y_t z_t sigmoid(z_t)         (without z: y_t)
 *
 *   x, dt, z, out  [B, N, D] in io_dtype; z may be NULL.
 *   A           fp32 [D, S], usually negative.
 *   Bm, Cm      [B, N, G, S] in io_dtype (a token's G S numbers contiguous);
 *               D is a multiple of G.
 *   Dx, dt_bias fp32 [D], or NULL (0).
 *   state_in    fp32 [n_seq, D, S] initial states, or NULL (zeros).
 *   seq_starts  see above.
 *   layout      HOST pointer or NULL.
 *   out         overlaps no other tensor, nor its rows one another.
 *   state_out   fp32 [n_seq, D, S], the states after each sequence's last token
 *               (state_in, or zeros, for an empty one), or NULL.  Overlaps no
 *               other tensor.
 *   workspace   at least selective_scan_workspace_size() bytes, 256-byte aligned,
 *               not shared with a concurrent call.
 *
 * Computed in fp32 for both I/O types.  A state that is NaN or infinite stays so
 * until its sequence ends.  The factor exp(r A) of one token is an fp32 number:
 * positive r A above 88 makes it infinite, and a state of 0 NaN; over many
 * tokens states may grow and shrink by more, as far as they are fp32 numbers.
 * Supported: S <= 128, D <= 32768, B <= 65535, N at most 2^30, B * N below 2^31,
 * n_seq at most 2^20. */
int selective_scan_forward(const void* x, const void* dt, const float* A, const void* Bm,
                           const void* Cm, const float* Dx, const float* dt_bias, const void* z,
                           const float* state_in, const int* seq_starts, int n_seq, int B, int N,
                           int D, int S, int G, int io_dtype, int dt_softplus,
                           const selective_scan_layout* layout, void* out, float* state_out,
                           void* workspace, size_t workspace_bytes, ttt_stream_t stream);

/* One token of each of B sequences, on a pool of states updated in place.
 *
 *   x, dt, z, out  [B, D]; Bm, Cm [B, G, S] in io_dtype (token strides unused).
 *   state       fp32 [n_slots, D, S].
 *   slots       see above.
 *   out         overlaps no other tensor.
 *
 * Computed in fp32.  Supported: S <= 128, D <= 32768, B <= 65535. */
int selective_scan_step(const void* x, const void* dt, const float* A, const void* Bm,
                        const void* Cm, const float* Dx, const float* dt_bias, const void* z,
                        float* state, const int* slots, int n_slots, int B, int D, int S, int G,
                        int io_dtype, int dt_softplus, const selective_scan_layout* layout,
                        void* out, ttt_stream_t stream);

/* ---------------------------------------------------------------- convolution
 * Strides of short_conv_*'s tensors (HOST struct; NULL = dense). */
typedef struct {
  mixer_stride x, out;
} short_conv_layout;

/* The short causal convolution over whole sequences, one filter of W taps per
 * channel:
 *     y_t = bias + sum_{j < W} w_j x_{t - (W - 1) + j},   out_t = act(y_t),
 * where the W - 1 tokens before a sequence come from its state.
 *
 *   x, out      [B, N, D] in io_dtype.
 *   w           fp32 [D, W]; w[:, W - 1] meets the token itself.
 *   bias        fp32 [D], or NULL (0).
 *   silu        1: act(y) = y sigmoid(y); 0: act(y) = y.
 *   state_in    [n_seq, W - 1, D] in io_dtype, the last inputs before each
 *               sequence, oldest first, or NULL (zeros).
 *   seq_starts  see above.
 *   layout      HOST pointer or NULL.
 *   out         overlaps no other tensor, nor its rows one another.
 *   state_out   [n_seq, W - 1, D] in io_dtype, the last inputs of each sequence
 *               with its state in front, or NULL.  Overlaps no other tensor.
 *
 * Computed in fp32.  Supported: 2 <= W <= 8, D <= 32768, B <= 65535, N at most
 * 2^30, B * N below 2^31, n_seq at most 2^20. */
int short_conv_forward(const void* x, const float* w, const float* bias, const void* state_in,
                       const int* seq_starts, int n_seq, int B, int N, int D, int W, int io_dtype,
                       int silu, const short_conv_layout* layout, void* out, void* state_out,
                       ttt_stream_t stream);

/* One token of each of B sequences, on a pool of states updated in place.
 *
 *   x, out      [B, D] in io_dtype (token strides unused).
 *   state       [n_slots, W - 1, D] in io_dtype.
 *   slots       see above.
 *   out         overlaps no other tensor.
 *
 * Computed in fp32.  Supported: 2 <= W <= 8, D <= 32768, B <= 65535. */
int short_conv_step(const void* x, const float* w, const float* bias, void* state,
                    const int* slots, int n_slots, int B, int D, int W, int io_dtype, int silu,
                    const short_conv_layout* layout, void* out, ttt_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TTT_GB300_TTT_MIXERS_H */
