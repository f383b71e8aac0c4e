/*
 * wkv_ssm.h — the state space operators of libwkv.so: the short causal
 * convolution, the selective scan, and an 8-bit store for carried states.
 *
 * They stand next to the WKV recurrences of wkv.h and follow its conventions
 * (device pointers owned by the caller, status codes, WKV_DEV_* bits, work
 * enqueued on `stream`, no allocation, bitwise repeatable results), with these
 * additions:
 *   - A token array has a row stride: element (token row r, column c) sits at
 *     base[r * stride + c], where row r is b*T + t of a dense call or the
 *     packed row of a varlen call.  A stride is in elements and at least the
 *     row's width, so the halves of one projection's output are passed as they
 *     are.  Token arrays need only be aligned to their element; y and the
 *     gradients are contiguous.  No output may overlap an input.
 *   - Sequences: a dense call has B rows of T tokens; a varlen call has
 *     num_slots slots of lengths[s] packed tokens (0: no work, the state row
 *     untouched, or copied when state_out != state_in) and updates their state
 *     rows, with the rules and data errors of wkv6_forward_varlen.
 *   - States are fp32: the convolution's [rows, W-1, D] (its last W-1 inputs,
 *     oldest first), the scan's [rows, D, N].
 */
#ifndef WKV_SSM_H
#define WKV_SSM_H

#include <stddef.h>

#include "wkv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t wkv_activation;
#define WKV_ACT_NONE 0
#define WKV_ACT_SILU 1          /* v * sigmoid(v)                                  */

typedef int32_t wkv_store_format;
#define WKV_STORE_INT8 0        /* scale = max|v| / 127                            */
#define WKV_STORE_E4M3 1        /* scale = max|v| / 448, OCP e4m3 codes            */

/*
 * Short causal convolution over each channel of x, W = 2, 3 or 4 taps:
 *   pre_t[d] = bias[d] + sum_j weight[d][j] x_(t-W+1+j)[d]
 *   y_t[d]   = pre_t[d]  or  pre_t[d] sigmoid(pre_t[d])
 * Inputs before the first token are the initial state's.  (RWKV's token shift,
 * x_t + mu (x_(t-1) - x_t), is W = 2 with the taps mu, 1 - mu.)
 *   x          [B,T,D] in_dtype, row stride x_stride
 *   weight     [D,W] fp32;  bias [D] fp32 or NULL
 *   y          [B,T,D] out_dtype (WKV_F32, or WKV_BF16: the fp32 result rounded)
 *   state_in   [n_state,W-1,D] fp32 or NULL (zeros); state_map, n_state as
 *              wkv6_forward
 *   state_out  [B,W-1,D] fp32 or NULL; may equal state_in only when state_map
 *              is NULL and n_state == B
 */
WKV_API wkv_status wkv_ssm_conv_forward(int B, int T, int D, int W,
                        const void *x, int64_t x_stride, wkv_dtype in_dtype,
                        const float *weight, const float *bias, wkv_activation act,
                        void *y, wkv_dtype out_dtype,
                        const float *state_in, const int32_t *state_map, int n_state,
                        float *state_out, int32_t *dev_status, void *stream);

/* The same for slots: x [total_tokens, D], y [total_tokens, D]; slot s reads
 * and writes state row state_map[s] (NULL: s) of [n_state,W-1,D]. */
WKV_API wkv_status wkv_ssm_conv_forward_varlen(int num_slots, int D, int W,
                        const int32_t *lengths, int max_len, int total_tokens,
                        const void *x, int64_t x_stride, wkv_dtype in_dtype,
                        const float *weight, const float *bias, wkv_activation act,
                        void *y, wkv_dtype out_dtype,
                        const float *state_in, float *state_out, const int32_t *state_map,
                        int n_state, int32_t *dev_status, void *stream);

/* Bytes of workspace of wkv_ssm_conv_backward.  Pure host function. */
WKV_API size_t wkv_ssm_conv_backward_workspace(int B, int T, int D, int W);

/*
 * Gradients of wkv_ssm_conv_forward (the same inputs; T >= 1) for the loss
 * L = sum(dy * y) + sum(d_state_out * final state):
 *   dy         [B,T,D] dy_dtype, row stride dy_stride
 *   d_state_out [B,W-1,D] fp32 or NULL (zero)
 *   dx         [B,T,D] grad_dtype
 *   d_weight [D,W], d_bias [D] (NULL: not wanted) fp32, summed over the batch
 *   d_state_in [B,W-1,D] fp32 or NULL: gradient of the initial state row b
 *              started from (rows that share one are not summed)
 *   workspace  16-byte aligned, at least wkv_ssm_conv_backward_workspace(...)
 *              bytes, as in wkv_ssm_scan_backward
 * A row whose state_map entry is outside the table sets WKV_DEV_BAD_STATE_MAP
 * and has no share in the summed gradients; its own rows are not written.
 */
WKV_API wkv_status wkv_ssm_conv_backward(int B, int T, int D, int W,
                        const void *x, int64_t x_stride, wkv_dtype in_dtype,
                        const float *weight, const float *bias, wkv_activation act,
                        const void *dy, int64_t dy_stride, wkv_dtype dy_dtype,
                        const float *state_in, const int32_t *state_map, int n_state,
                        const float *d_state_out, void *dx, wkv_dtype grad_dtype,
                        float *d_weight, float *d_bias, float *d_state_in,
                        void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Bytes of workspace with which a scan of `rows` sequences (batch rows or
 * slots) of up to T tokens, total_tokens in all, is cut into segments that run
 * side by side: 0 where the rows alone fill the chip, and for T <= 64.  Pure
 * host function. */
WKV_API size_t wkv_ssm_scan_workspace(int rows, int T, int64_t total_tokens, int D, int N, int G);

/*
 * Selective scan.  D channels in G equal groups that share B and C; state
 * h[d][n] of N = 1 .. 64 values per channel:
 *   delta_t[d] = softplus(dt_t[d] + dt_bias[d])  or  dt_t[d] + dt_bias[d]
 *   h[d][n]   <- exp(delta_t[d] A[d][n]) h[d][n] + delta_t[d] B_t[g][n] x_t[d]
 *   y_t[d]     = sum_n C_t[g][n] h[d][n] + skip[d] x_t[d]     (the updated state)
 *   y_t[d]    <- y_t[d] z_t[d] sigmoid(z_t[d])                (z given)
 *   x, dt, z   [B,T,D] in_dtype (z NULL: no gate), each with its row stride
 *   Bm, Cm     [B,T,G*N] in_dtype, each with its row stride
 *   A          [D,N] fp32, as it enters the exponent (usually negative)
 *   skip, dt_bias [D] fp32, each or NULL (zero)
 *   y          [B,T,D] out_dtype
 *   state_in   [n_state,D,N] fp32 or NULL (zeros); state_map, n_state, state_out
 *              ([B,D,N]), dev_status as wkv_ssm_conv_forward
 *   workspace  16-byte aligned device memory of at least
 *              wkv_ssm_scan_workspace(B, T, B*T, D, N, G) bytes, whose content does not
 *              matter and which no other call may use until this one is done; NULL:
 *              the sequences are not cut (slower where they are few and long)
 * A token whose delta is 0 (dt = -inf under the softplus) leaves the state as
 * it is, also where A is an infinity, so rows may be padded on either side that
 * way (with any finite x and B).
 */
WKV_API wkv_status wkv_ssm_scan_forward(int B, int T, int D, int N, int G,
                        const void *x, int64_t x_stride, const void *dt, int64_t dt_stride,
                        const float *A, const void *Bm, int64_t b_stride,
                        const void *Cm, int64_t c_stride, wkv_dtype in_dtype,
                        const float *skip, const void *z, int64_t z_stride,
                        const float *dt_bias, int dt_softplus, void *y, wkv_dtype out_dtype,
                        const float *state_in, const int32_t *state_map, int n_state,
                        float *state_out, void *workspace, size_t workspace_bytes,
                        int32_t *dev_status, void *stream);

/* wkv_ssm_scan_forward that also saves the state at every 16-token boundary for
 * wkv_ssm_scan_backward (y and state_out are bitwise those of that call):
 *   chunk_states [B,ceil(T/16)-1,D,N] fp32, 16-byte aligned (may be NULL when
 *              T <= 16): entry c-1 is the state after token 16c-1 */
WKV_API wkv_status wkv_ssm_scan_forward_train(int B, int T, int D, int N, int G,
                        const void *x, int64_t x_stride, const void *dt, int64_t dt_stride,
                        const float *A, const void *Bm, int64_t b_stride,
                        const void *Cm, int64_t c_stride, wkv_dtype in_dtype,
                        const float *skip, const void *z, int64_t z_stride,
                        const float *dt_bias, int dt_softplus, void *y, wkv_dtype out_dtype,
                        const float *state_in, const int32_t *state_map, int n_state,
                        float *state_out, float *chunk_states, void *workspace, size_t workspace_bytes,
                        int32_t *dev_status, void *stream);

/* Bytes of workspace of wkv_ssm_scan_backward, with the forward call's chunk
 * states at hand or without.  Pure host function. */
WKV_API size_t wkv_ssm_scan_backward_workspace(int B, int T, int D, int N, int G, int with_chunk_states);

/*
 * Gradients of wkv_ssm_scan_forward (the same inputs; T >= 1) for the loss
 * L = sum(dy * y) + sum(d_state_out * final state):
 *   dy         [B,T,D] dy_dtype, row stride dy_stride
 *   chunk_states  what wkv_ssm_scan_forward_train saved for these inputs, or
 *              NULL: they are computed first
 *   d_state_out [B,D,N] fp32 or NULL (zero)
 *   dx, ddt, dz  [B,T,D] grad_dtype, 16-byte aligned (dz: NULL exactly when z is)
 *   dB, dC     [B,T,G*N] grad_dtype, summed over the channels of a group
 *   dA [D,N], d_skip [D] (NULL: not wanted), d_dt_bias [D] (NULL: not wanted)
 *              fp32, summed over the batch
 *   d_state_in [B,D,N] fp32 or NULL: gradient of the initial state row b
 *              started from (rows that share one are not summed)
 *   workspace  16-byte aligned, at least wkv_ssm_scan_backward_workspace(...)
 *              bytes; its content does not matter, and no other call may use it
 *              until this one is done
 * Sums run in fp32 and in one order.  A row whose state_map entry is outside
 * the table sets WKV_DEV_BAD_STATE_MAP and has no share in the summed
 * gradients; its own rows are not written.
 */
WKV_API wkv_status wkv_ssm_scan_backward(int B, int T, int D, int N, int G,
                        const void *x, int64_t x_stride, const void *dt, int64_t dt_stride,
                        const float *A, const void *Bm, int64_t b_stride,
                        const void *Cm, int64_t c_stride, wkv_dtype in_dtype,
                        const float *skip, const void *z, int64_t z_stride,
                        const float *dt_bias, int dt_softplus,
                        const void *dy, int64_t dy_stride, wkv_dtype dy_dtype,
                        const float *state_in, const int32_t *state_map, int n_state,
                        const float *chunk_states, const float *d_state_out,
                        void *dx, void *ddt, void *dB, void *dC, void *dz, wkv_dtype grad_dtype,
                        float *dA, float *d_skip, float *d_dt_bias, float *d_state_in,
                        void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream);

/* wkv_ssm_scan_forward for slots: token arrays are packed [total_tokens, ..];
 * slot s reads and writes state row state_map[s] (NULL: s) of [n_state,D,N]. */
WKV_API wkv_status wkv_ssm_scan_forward_varlen(int num_slots, int D, int N, int G,
                        const int32_t *lengths, int max_len, int total_tokens,
                        const void *x, int64_t x_stride, const void *dt, int64_t dt_stride,
                        const float *A, const void *Bm, int64_t b_stride,
                        const void *Cm, int64_t c_stride, wkv_dtype in_dtype,
                        const float *skip, const void *z, int64_t z_stride,
                        const float *dt_bias, int dt_softplus, void *y, wkv_dtype out_dtype,
                        const float *state_in, float *state_out, const int32_t *state_map,
                        int n_state, void *workspace, size_t workspace_bytes,
                        int32_t *dev_status, void *stream);

/*
 * 8-bit store of carried states (snapshots of a prefix, parked slots): rows of
 * `row` fp32 values, of any state of this library, in groups of 64 with one
 * fp32 scale each (the last group may be short).
 *   code = nearest to v / scale, ties to even, both quotients in fp32; a group
 *   of zeros has scale 0; a group with an infinity or NaN has scale NaN and
 *   reads back as NaN.
 *   data       [n_store, row] one byte per value
 *   scale      [n_store, ceil(row/64)] fp32
 *   states     [n_state, row] fp32
 *   store_rows, state_rows  [count] int32 DEVICE or NULL (0 .. count-1): item i
 *              moves between states[state_rows[i]] and data[store_rows[i]]
 * Rows that two items would write set WKV_DEV_DUPLICATE_ROW and rows outside
 * their table WKV_DEV_BAD_STATE_MAP; such an item moves nothing.  (One stored
 * row may be read into many state rows, and one state written to many rows.)
 */
WKV_API wkv_status wkv_state_store_write(void *data, float *scale, int n_store, wkv_store_format format,
                        const float *states, int n_state, int64_t row,
                        const int32_t *store_rows, const int32_t *state_rows, int count,
                        int32_t *dev_status, void *stream);
WKV_API wkv_status wkv_state_store_read(const void *data, const float *scale, int n_store, wkv_store_format format,
                        float *states, int n_state, int64_t row,
                        const int32_t *store_rows, const int32_t *state_rows, int count,
                        int32_t *dev_status, void *stream);

/*
 * One of the calls above with its arguments in order as `count` words: integers,
 * and pointers as their addresses (host memory, read before the call returns).
 * For callers to whom passing each argument by itself is dear, such as
 * interpreters.  WKV_ERR_INVALID_ARG for an unknown op, another count, or an
 * integer that its parameter cannot hold.
 */
typedef int32_t wkv_ssm_op;
#define WKV_OP_CONV_FORWARD 0
#define WKV_OP_CONV_FORWARD_VARLEN 1
#define WKV_OP_CONV_BACKWARD 2
#define WKV_OP_SCAN_FORWARD 3
#define WKV_OP_SCAN_FORWARD_TRAIN 4
#define WKV_OP_SCAN_FORWARD_VARLEN 5
#define WKV_OP_SCAN_BACKWARD 6
#define WKV_OP_STORE_WRITE 7
#define WKV_OP_STORE_READ 8
WKV_API wkv_status wkv_ssm_call(wkv_ssm_op op, const int64_t *args, int count);

#ifdef __cplusplus
}
#endif

#endif /* WKV_SSM_H */
