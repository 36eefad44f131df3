/*
 * dgemm_experts.h -- C ABI of the routed-expert and 8-bit integer operators.
 *
 * Beside the dense products of dgemm.h the library computes what a
 * mixture-of-experts feed-forward block and an 8-bit integer linear layer need:
 *
 *   dgemm_route            router logits -> top-k experts, weights, grouping
 *   dgemm_combine          weighted sum of each token's expert rows
 *   dgemm_grouped_*        products grouped by expert, ragged group sizes that
 *                          only the device knows; BF16, FP8 E4M3, INT8
 *   dgemm_int8_quantize    activations -> int8 codes + one scale per row
 *   dgemm_int8_scaled      int8 product with per-token and per-channel scales
 *
 * The conventions of dgemm.h hold: row-major contiguous matrices; every pointer
 * argument except `stream` is a DEVICE pointer; the caller owns all memory; calls
 * are asynchronous on `stream`, never allocate and never synchronise; argument
 * errors return before any launch; every device-side wait is bounded and one
 * that gives up is recorded in the first DGEMM_WS_STATUS_BYTES bytes of the
 * call's workspace (or, without one, in the per-device word) for
 * dgemm_query_device_status. Of the planner overrides of dgemm.h, cta_pair,
 * wait_limit_ns and stall_after_loads apply to the products. Base pointers of matrices must be 16-byte aligned
 * (DGEMM_ERR_MISALIGNED otherwise); int32 and float tables need only their
 * natural alignment.
 */
#ifndef DGEMM_EXPERTS_H
#define DGEMM_EXPERTS_H

#include "dgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most experts of one call, and most experts of one token. */
#define DGEMM_MAX_EXPERTS 1024
#define DGEMM_MAX_TOPK 32

/* Gated activation of the grouped products, beside dgemm_act_t: B has 2 x (N/2)
 * output channels, the gate's first, and D [rows, N/2] is
 * silu(y[:, :N/2]) * y[:, N/2:]. N must be even. */
#define DGEMM_ACT_SWIGLU 4

typedef enum {
    DGEMM_GROUPED_BF16 = 0,
    DGEMM_GROUPED_FP8 = 1, /* E4M3 codes with scales */
    DGEMM_GROUPED_INT8 = 2
} dgemm_grouped_type_t;

/* Routes T tokens to k of E experts each and groups the (token, slot) pairs by
 * expert.
 *   logits     [T,E] F32 or BF16, read as FP32. -inf and NaN entries are masked
 *              (never chosen, probability 0); +inf counts as the largest finite
 *              number.
 *   ids        [T,k] int32 out: the k largest logits' experts, largest first,
 *              equal logits lowest expert first; -1 where fewer than k entries
 *              are unmasked (a fully masked row routes nowhere).
 *   weights    [T,k] F32 out: softmax over the row's unmasked entries at ids, or
 *              with renormalize != 0 over the chosen ones (they sum to 1); 0 for id -1.
 *   offsets    [E+1] int32 out: rows of expert e are [offsets[e], offsets[e+1]);
 *              offsets[E] is the number of routed pairs.
 *   row_token  [T*k] int32 out: the token of each row. Rows of one expert are in
 *              token order, so the result does not depend on timing. -1 at and
 *              beyond offsets[E].
 *   slot_row   [T,k] int32 out: the row of each pair, -1 for id -1.
 *   ws         dgemm_route_workspace_size(T, E, k) bytes, contents arbitrary
 *              (DGEMM_ERR_WORKSPACE_TOO_SMALL with less; 0 bytes may be needed). Its first
 *              DGEMM_WS_STATUS_BYTES bytes stay as they are: a status word that a product
 *              given the same workspace has left there is kept until it is queried.
 * 1 <= k <= min(E, DGEMM_MAX_TOPK), E <= DGEMM_MAX_EXPERTS, T*k < 2^30. T == 0
 * writes zero offsets. */
dgemm_status_t dgemm_route(const void* logits, dgemm_dtype_t logits_dtype, int64_t T, int64_t E, int k,
                           int renormalize, int32_t* ids, float* weights, int32_t* offsets, int32_t* row_token,
                           int32_t* slot_row, void* ws, size_t ws_bytes, dgemm_stream_t stream);
size_t dgemm_route_workspace_size(int64_t T, int64_t E, int k);

/* out[t,:] = add[t,:] + sum_j weights[t,j] * Y[slot_row[t,j],:], summed in FP32
 * with j ascending and rounded once.
 *   Y        [R,H] BF16.   slot_row [T,k] int32: a row outside [0,R) adds nothing.
 *   weights  [T,k] F32.    add [T,H] BF16 or NULL.
 *   out      [T,H] F32 or BF16; must not overlap Y; may equal add when BF16.
 * 1 <= k <= DGEMM_MAX_TOPK; H any. */
dgemm_status_t dgemm_combine(const void* Y, int64_t R, const int32_t* slot_row, const float* weights, const void* add,
                             void* out, dgemm_dtype_t out_dtype, int64_t T, int64_t H, int k, dgemm_stream_t stream);

/* Products grouped by expert: for every expert e and row r in
 * [offsets[e], offsets[e+1]),
 *   D[r,:] = act(alpha * A[a,:] . op(B_e) + bias[e,:]),   a = a_rows ? a_rows[r] : r,
 * with FP32 accumulation and one rounding to D's type.
 *   A        [a_count,K] BF16.   a_rows [R] int32 or NULL (then a_count == R); a
 *            row index outside [0,a_count) reads as a row of zeros.
 *   B        [E,N,K] (DGEMM_B_NK) or [E,K,N] (DGEMM_B_KN) BF16.
 *   offsets  [E+1] int32, ascending, on the device: the group sizes are not known
 *            to the host. Values are clamped into [0,R]; rows of D outside
 *            every group are not written.
 *   bias     [E,N] F32 or NULL.   act dgemm_act_t or DGEMM_ACT_SWIGLU. NaN stays NaN
 *            under every activation (ReLU included).
 *   D        [R,N] (SWIGLU: [R,N/2]) F32 or BF16.
 *   ws       optional: DGEMM_WS_STATUS_BYTES for the call's status word.
 * K * element size must be a multiple of 16 bytes; for K x N weights N * element size too,
 * and N/2 * element size with SWIGLU (N a multiple of 16), DGEMM_ERR_MISALIGNED otherwise;
 * N x K weights take any N.
 * E <= DGEMM_MAX_EXPERTS. */
dgemm_status_t dgemm_grouped_bf16(const void* A, int64_t a_count, const int32_t* a_rows, const void* B,
                                  dgemm_b_layout_t b_layout, const int32_t* offsets, int64_t E, void* D,
                                  dgemm_dtype_t d_dtype, int64_t R, int64_t N, int64_t K, float alpha,
                                  const float* bias, int act, void* ws, size_t ws_bytes, dgemm_stream_t stream);

/* The same with E4M3 codes: A [a_count,K], B [E,N,K], a_scale [a_count] (one per
 * row of A), b_scale [E,N] (one per expert and channel); the scaled product is
 * alpha * a_scale[a] * b_scale[e,n] * acc. */
dgemm_status_t dgemm_grouped_fp8_scaled(const void* Aq, int64_t a_count, const int32_t* a_rows, const void* Bq,
                                        const float* a_scale, const float* b_scale, const int32_t* offsets, int64_t E,
                                        void* D, dgemm_dtype_t d_dtype, int64_t R, int64_t N, int64_t K, float alpha,
                                        const float* bias, int act, void* ws, size_t ws_bytes, dgemm_stream_t stream);

/* The same with int8 codes (see dgemm_int8_scaled for the arithmetic). */
dgemm_status_t dgemm_grouped_int8_scaled(const void* Aq, int64_t a_count, const int32_t* a_rows, const void* Bq,
                                         const float* a_scale, const float* b_scale, const int32_t* offsets, int64_t E,
                                         void* D, dgemm_dtype_t d_dtype, int64_t R, int64_t N, int64_t K, float alpha,
                                         const float* bias, int act, void* ws, size_t ws_bytes, dgemm_stream_t stream);

/* Workspace bytes a grouped call with these sizes can use; 0 for invalid ones. */
size_t dgemm_grouped_workspace_size(dgemm_grouped_type_t type, int64_t R, int64_t E, int64_t N, int64_t K, int act);

/* Per-token quantisation: scale[m] = max_k |X[m,k]| * (1 / 127), with 1 / 127 rounded
 * to FP32 (1 for a row of zeros), and q[m,k] = X[m,k] / scale[m], the FP32 quotient
 * rounded to the nearest integer, ties to even.
 * The maximum is taken over finite values; infinities saturate to +-127 and NaN
 * becomes 0. X [M,K] BF16 or F32; q [M,K] int8; scale [M] F32. K any. */
dgemm_status_t dgemm_int8_quantize(const void* X, dgemm_dtype_t x_dtype, int8_t* q, float* scale, int64_t M, int64_t K,
                                   dgemm_stream_t stream);

/* D = act(alpha * diag(a_scale) (Aq . Bq^T) diag(b_scale) + beta * C + bias), int8 codes.
 *   Aq [M,K], Bq [N,K] int8 (all 256 codes); a_scale [M], b_scale [N] F32;
 *   C, D [M,N] F32 or BF16 (C read only when beta != 0; may equal D); bias [N]
 *   F32 or NULL; act dgemm_act_t (NaN stays NaN).
 * Arithmetic: int8 codes are exact in FP16 and products run on the FP16 tensor cores with
 * FP32 sums: the sum is the exact integer while partial sums stay below 2^24 in
 * magnitude, and rounded toward zero to 24 bits, once for each instruction of 16 terms,
 * beyond that. One set of weights (this call, or a grouped one with E == 1) with one or
 * two rows of at most 74 KB of codes in all (M * K <= 75776) runs on integer dot products:
 * exact 32-bit sums (K <= 131071) rounded once to FP32. So the bits of a row whose sums
 * pass 2^24 can depend on how many rows the call has; below 2^24 they do not.
 *   ws       optional: DGEMM_WS_STATUS_BYTES for the call's status word.
 * K must be a multiple of 16; N any. */
dgemm_status_t dgemm_int8_scaled(const void* Aq, const void* Bq, const float* a_scale, const float* b_scale,
                                 const void* C, dgemm_dtype_t c_dtype, void* D, dgemm_dtype_t d_dtype, int64_t M,
                                 int64_t N, int64_t K, float alpha, float beta, const float* bias, int act, void* ws,
                                 size_t ws_bytes, dgemm_stream_t stream);

/* Workspace bytes dgemm_int8_scaled can use; 0 for invalid sizes. */
size_t dgemm_int8_workspace_size(int64_t M, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* DGEMM_EXPERTS_H */
