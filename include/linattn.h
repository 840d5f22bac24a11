/*
 * linattn.h -- C ABI of libwkv's causal linear attention on NVIDIA B200
 * (sm_100a tensor cores).  Same shared library as wkv.h.
 *
 * The operator (linear attention post, "Transformers are RNNs: 선형 어텐션으로
 * 만드는 빠른 자기회귀 트랜스포머", section "인과 마스킹과 누적합"; 0-based
 * positions), for every head h independently:
 *
 *   S_i = sum_{j<=i} phi(K_j) V_j^T        (D x M)
 *   Z_i = sum_{j<=i} phi(K_j)              (D)
 *   V'_i = phi(Q_i)^T S_i / (phi(Q_i)^T Z_i)
 *
 * with the feature map of section "특징 맵 선택과 계산 비용",
 * phi(x) = elu(x) + 1 (x + 1 for x > 0, e^x otherwise; always positive, so
 * the denominator is positive and no epsilon is added).  The backward gives
 * the gradients of a scalar loss L with respect to Q, K and V from
 * dL/dV' (section "상수 메모리 기울기 계산": a forward cumulative sum for
 * phi(Q), reverse cumulative sums for phi(K) and V, then the chain rule
 * through the normalisation and phi).
 *
 * How it is computed: positions are cut into chunks of 128.  Per chunk the
 * causal part is the masked product tril(phi(Q) phi(K)^T) V and the earlier
 * chunks enter through phi(Q) S_prev, every product a dense tcgen05 MMA with
 * bfloat16 operands and float32 accumulation in tensor memory; the chunk
 * states are summed in a fixed order, so results are bit-reproducible.
 *
 * Conventions (those of wkv.h where not stated here)
 * ----------------------------------------------------
 * - Device pointers owned by the caller; every call is asynchronous on
 *   `stream` (a cudaStream_t as void*).  The library allocates nothing.
 * - Layout: q, k, grad_q, grad_k are [BH, N, D]; v, out, grad_out, grad_v
 *   are [BH, N, M]; all row-major (the feature index fastest), bfloat16.
 *   BH counts independent problems (batch x heads).  Results are rounded to
 *   nearest even into bfloat16.
 * - Supported head sizes: D = M = 32 (the pages' experiments: 8 heads of 32
 *   dimensions).  Other sizes return WKV_ERR_UNSUPPORTED.
 * - Sizes: BH >= 1, N >= 0, BH * N < 2^31.  N = 0 writes nothing but the
 *   (zero) state; the tensor pointers may then be null.
 * - Alignment: every tensor pointer 16-byte aligned (WKV_ERR_UNSUPPORTED
 *   otherwise); the workspace 256-byte aligned.
 * - Workspace: linattn_workspace_size() bytes, zero-filled once before its
 *   first use (the first 256 bytes are a header like the one of wkv.h's
 *   workspaces; wkv_get_status() reads it).  Calls that share a workspace
 *   must be ordered on one stream.
 * - Return codes are those of wkv.h (WKV_OK, WKV_ERR_*).  A call that
 *   returns an error other than WKV_ERR_CUDA has launched nothing.
 *   Conditions detected on the device (a bounded wait that gave up) are
 *   read with wkv_get_status(ws, stream).
 * - NaN or Inf in the inputs propagate; they are not checked.
 */
#ifndef LIBWKV_LINATTN_H
#define LIBWKV_LINATTN_H

#include <stddef.h>
#include <stdint.h>

#include "wkv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LINATTN_OP_FORWARD 0
#define LINATTN_OP_BACKWARD 1

/* Bytes of workspace for `op` at these sizes (0 if the sizes are invalid or
 * unsupported). */
size_t linattn_workspace_size(int op, int64_t BH, int64_t N, int D, int M);

/*
 * Causal linear attention forward (section "인과 마스킹과 누적합").
 *   q, k      [BH, N, D] bf16, read
 *   v         [BH, N, M] bf16, read
 *   out       [BH, N, M] bf16, written: V'
 *   state_out nullable; float32, written: S_{N-1} as [BH][D][M] followed by
 *             Z_{N-1} as [BH][D] (BH*(D*M + D) floats; zeros when N = 0)
 *   ws        workspace of linattn_workspace_size(LINATTN_OP_FORWARD, ...)
 * Returns WKV_OK, WKV_ERR_INVALID_ARG (null or overlapping-by-identity
 * pointers, negative sizes), WKV_ERR_UNSUPPORTED (head size, alignment),
 * WKV_ERR_WORKSPACE (too small) or WKV_ERR_CUDA (launch failed).
 */
int linattn_forward(int64_t BH, int64_t N, int D, int M, const void *q, const void *k, const void *v, void *out,
                    float *state_out, void *ws, size_t ws_bytes, void *stream);

/*
 * Gradients of L given grad_out = dL/dV' (section "상수 메모리 기울기 계산").
 *   q, k, v   as in linattn_forward, read
 *   grad_out  [BH, N, M] bf16, read
 *   grad_q, grad_k [BH, N, D] bf16, written; grad_v [BH, N, M] bf16, written
 *   ws        workspace of linattn_workspace_size(LINATTN_OP_BACKWARD, ...)
 * The forward is recomputed from q, k, v (nothing from linattn_forward is
 * needed).  Return codes as linattn_forward.
 */
int linattn_backward(int64_t BH, int64_t N, int D, int M, const void *q, const void *k, const void *v,
                     const void *grad_out, void *grad_q, void *grad_k, void *grad_v, void *ws, size_t ws_bytes,
                     void *stream);

/*
 * The same gradients from the forward's saved state (the saved-statistics
 * form of the backward): `ws` must be the workspace that the linattn_forward
 * call computing `out` from these q, k, v used, sized
 * linattn_workspace_size(LINATTN_OP_BACKWARD, ...) (a backward-sized
 * workspace serves the forward too), with no other call on it since.  That
 * call left in it each chunk's prefix state and its denominators; this call
 * reads them instead of recomputing the forward, and needs the forward's
 * output:
 *   out       [BH, N, M] bf16, read: linattn_forward's output
 * Other arguments and return codes as linattn_backward.  Results differ from
 * linattn_backward's by rounding only (dL/d den uses the bf16 output).
 */
int linattn_backward_saved(int64_t BH, int64_t N, int D, int M, const void *q, const void *k, const void *v,
                           const void *out, const void *grad_out, void *grad_q, void *grad_k, void *grad_v, void *ws,
                           size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Linear attention with a decay for each head, and the rotary positions of
 * its queries and keys.
 *
 * Per batch row b and head h, with lam = e^{log_decay[h]} and a float32
 * state S of D x M (0-based positions, S_{-1} = state_in or 0):
 *
 *   S_t   = lam S_{t-1} + k_t v_t^T
 *   out_t = scale * q_t^T S_t
 *         = scale * ( sum_{j<=t} lam^{t-j} (q_t . k_j) v_j + lam^{t+1} q_t^T S_{-1} )
 *
 * the cumulative state of the causal form above (section "인과 마스킹과
 * 누적합") with the time decay that WKV gives each channel, one for each head
 * here, and neither feature map nor denominator.  Three calls, as for WKV: a
 * whole sequence at once, its gradients, and one token per sequence.
 *
 * Conventions (those above where not stated here)
 * - Element type `dtype` of q, k, v, out and their gradients: WKV_F32 or
 *   WKV_BF16 (float32 arithmetic, one rounding to nearest even at the end;
 *   bfloat16 products run on the tensor cores, where the masked scores and
 *   the copy of the state that q meets are rounded to bfloat16.  The state
 *   itself is always float32; there its decayed keys enter as sums of two
 *   bfloat16 terms, 16 bits: about 4e-6 of a state that is handed out).
 * - Tensors [B, T, H, D] (q, k) and [B, T, H, M] (v, out) are given as
 *   linattn_view: a device pointer and the strides, in elements, of batch,
 *   time and head; the feature index is contiguous.  Strides are >= 0; those
 *   of an output must not make it overlap itself.  So [B, H, T, D] tensors
 *   and slices of a fused projection need no copy.  An output shares no element
 *   with an input or another output (checked is that no two start at the same
 *   address).
 * - Head sizes: 1 <= D, M <= 128.  The tensor-core kernels run when dtype is
 *   WKV_BF16, D and M are multiples of 8, pointers are 16-byte aligned,
 *   strides are multiples of 8 elements, > 0 and below 2^39, and T is above
 *   32; other calls run the recurrence on the CUDA cores.  So keys or values
 *   that heads share through a stride of 0 run the recurrence: over more than a
 *   few positions a copy for each head is faster (8 x 1024 x 12 heads of 64,
 *   forward 270 us against 48 with the copies, gradients 940 against 63).
 * - A caller that wants float32 products of bfloat16 tensors converts them:
 *   WKV_F32 runs the recurrence (states to 3e-7 instead of 4e-6; 8 x 1024 x 12
 *   heads of 64, 86 us instead of 22).
 * - Sizes: B, H >= 1, B * H < 2^24 (N * H < 2^31 for the step), 0 <= T < 2^31.
 * - The recurrence holds up to 2^16 times its state and products, so values
 *   whose sums stay below 2^111 are safe from overflow.
 * - log_decay [H] float32, at most 0 (minus infinity allowed: lam = 0).  It is
 *   a constant: no call returns a gradient for it.
 * - lengths [B] int32 on the device, or NULL (every row has T positions): row
 *   b has n = min(max(lengths[b], 0), T) positions.  What lies behind them is
 *   not used, whatever it holds; out and the gradients are zero there, and
 *   state_out is the state after n positions (state_in, or zeros, if n = 0).
 * - States and their gradients: [B, H, D, M] float32, contiguous, 16-byte
 *   aligned.
 * - NaN or Inf at a position p < n reach what depends on p; in the
 *   tensor-core kernels they may reach every position of p's chunk (128
 *   positions of the same row and head) as well.
 * - Workspace: linattn_decay_workspace_size() bytes, 256-byte aligned,
 *   uninitialised; nothing in it outlives the call.  Its size may be 0 (ws is
 *   then ignored).  Calls that may run at the same time need one each.
 * - status: a device int32 (or NULL), zeroed by its owner; a bounded wait
 *   that gave up (about one second, or the options' spin_limit) stores
 *   WKV_ERR_TIMEOUT there (that call's results are then invalid).  Any number
 *   of calls may share it.
 * - The _ex forms take wkv_options (wkv.h; NULL: the defaults).  kernel has to
 *   be WKV_KERNEL_AUTO; spin_limit bounds the waits of the tensor-core
 *   kernels, in microseconds (in steps of about 4); test_hold_first_chunk
 *   holds an arrival back in the first block of each of their launches, so
 *   that its waits run out.  The recurrence waits for nothing.
 * - Results are bit-reproducible.
 */
typedef struct {
  void *ptr;
  int64_t stride_b, stride_t, stride_h;
} linattn_view;

/* Bytes of workspace of linattn_decay_forward (op LINATTN_OP_FORWARD) or
 * linattn_decay_backward (LINATTN_OP_BACKWARD) at these sizes; 0 if none is
 * needed or the sizes are invalid. */
size_t linattn_decay_workspace_size(int op, int64_t B, int64_t T, int64_t H, int D, int M, int dtype);

/*
 * A status word of the current device for `status`: one int32, zero at first,
 * that lives as long as the library.  It may be asked for while a stream
 * captures, and captured calls may be given it.  Returns WKV_OK,
 * WKV_ERR_INVALID_ARG (null) or WKV_ERR_CUDA.
 */
int linattn_decay_status_word(int32_t **word);

/*
 * Forward over whole sequences.
 *   q, k, v    views, read
 *   state_in   nullable: the state before position 0
 *   out        view, written
 *   state_out  nullable: the state after each row's last position; may equal
 *              state_in
 * Returns WKV_OK, WKV_ERR_INVALID_ARG (null pointers, bad sizes, strides or
 * dtype, an output given as an input), WKV_ERR_UNSUPPORTED (head size,
 * misaligned pointer, partly overlapping states), WKV_ERR_WORKSPACE (missing,
 * misaligned or too small) or WKV_ERR_CUDA.
 */
int linattn_decay_forward(int64_t B, int64_t T, int64_t H, int D, int M, int dtype, const linattn_view *q,
                          const linattn_view *k, const linattn_view *v, const float *log_decay, float scale,
                          const int32_t *lengths, const float *state_in, const linattn_view *out, float *state_out,
                          void *ws, size_t ws_bytes, int32_t *status, void *stream);
int linattn_decay_forward_ex(int64_t B, int64_t T, int64_t H, int D, int M, int dtype, const linattn_view *q,
                             const linattn_view *k, const linattn_view *v, const float *log_decay, float scale,
                             const int32_t *lengths, const float *state_in, const linattn_view *out, float *state_out,
                             void *ws, size_t ws_bytes, int32_t *status, void *stream, const wkv_options *opt);

/*
 * Gradients of a scalar loss L given grad_out = dL/dout and, optionally,
 * grad_state_out = dL/dstate_out.  With W_t = scale q_t grad_out_t^T +
 * lam W_{t+1} in reverse time, W_{n-1} = scale q grad_out^T + grad_state_out:
 *   grad_q_t = scale S_t grad_out_t,  grad_k_t = W_t v_t,
 *   grad_v_t = W_t^T k_t,             grad_state_in = lam W_0
 * (cumulative sums in both directions, section "상수 메모리 기울기 계산").
 * Nothing from linattn_decay_forward is needed.
 *   state_in        the forward's, or NULL
 *   grad_state_out  nullable, read;  grad_state_in nullable, written
 * Return codes as linattn_decay_forward.
 */
int linattn_decay_backward(int64_t B, int64_t T, int64_t H, int D, int M, int dtype, const linattn_view *q,
                           const linattn_view *k, const linattn_view *v, const float *log_decay, float scale,
                           const int32_t *lengths, const float *state_in, const linattn_view *grad_out,
                           const float *grad_state_out, const linattn_view *grad_q, const linattn_view *grad_k,
                           const linattn_view *grad_v, float *grad_state_in, void *ws, size_t ws_bytes,
                           int32_t *status, void *stream);
int linattn_decay_backward_ex(int64_t B, int64_t T, int64_t H, int D, int M, int dtype, const linattn_view *q,
                              const linattn_view *k, const linattn_view *v, const float *log_decay, float scale,
                              const int32_t *lengths, const float *state_in, const linattn_view *grad_out,
                              const float *grad_state_out, const linattn_view *grad_q, const linattn_view *grad_k,
                              const linattn_view *grad_v, float *grad_state_in, void *ws, size_t ws_bytes,
                              int32_t *status, void *stream, const wkv_options *opt);

/*
 * One token for each of N sequences: state_out = lam state_in + k v^T,
 * out = scale q^T state_out.  Views of [N, H, D] and [N, H, M] (stride_b is
 * the sequences'; stride_t is not read).  state_out may equal state_in.  Needs
 * no workspace.  Return codes as linattn_decay_forward.
 */
int linattn_decay_step(int64_t N, int64_t H, int D, int M, int dtype, const linattn_view *q, const linattn_view *k,
                       const linattn_view *v, const float *log_decay, float scale, const float *state_in,
                       const linattn_view *out, float *state_out, void *stream);

/*
 * Rotary positions.  The first R elements of every head of q [B, T, Hq, D]
 * and k [B, T, Hk, D] are R / 2 pairs, (x_i, x_{i + R/2}) or, if
 * `interleaved`, (x_{2i}, x_{2i+1}); pair i at position p becomes
 *   mscale * (a cos - b sin, a sin + b cos),  angle = p * inv_freq[i]
 * (angles as pairs of float64, reduced before they are rounded to float32, so
 * that far positions lose nothing; products in float32, one rounding at the
 * end).  Elements from R on are copied.
 *   inverse    nonzero: rotates back (sin negated), which is also the
 *              gradient of the call with inverse = 0
 *   positions  [B, T] integers of pos_bytes = 4 or 8 bytes, contiguous in T,
 *              rows pos_stride_b elements apart (0: one row for every b); any
 *              value of magnitude up to 2^53
 *   inv_freq   [R / 2] float64 on the device
 *   k, out_k   NULL with Hk = 0: q alone
 *   out_q, out_k  may equal q, k (pointer and strides); no other overlap
 * 1 <= D <= 1024, R even, 2 <= R <= D.
 * Returns WKV_OK, WKV_ERR_INVALID_ARG, WKV_ERR_UNSUPPORTED (misaligned
 * pointer) or WKV_ERR_CUDA.
 */
int linattn_rotary(int64_t B, int64_t T, int D, int R, int dtype, int64_t Hq, const linattn_view *q, int64_t Hk,
                   const linattn_view *k, const void *positions, int pos_bytes, int64_t pos_stride_b,
                   const double *inv_freq, float mscale, int interleaved, int inverse, const linattn_view *out_q,
                   const linattn_view *out_k, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBWKV_LINATTN_H */
