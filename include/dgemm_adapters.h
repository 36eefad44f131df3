/*
 * dgemm_adapters.h -- C ABI of the low-rank adapters of many requests.
 *
 * The rows of a batch belong to requests, and each request may bring a low-rank
 * adapter of the layer: two matrices A_a [r,K] and B_a [N,r] whose product is added
 * to the weights that all requests share.
 *
 *   dgemm_adapter_bf16   the shared projection and every row's adapter in one call:
 *                        D[t] = act(X[t] . W^T + s_a (X[t] . A_a^T) . B_a^T + bias)
 *   dgemm_adapter_add    the adapters beside a product C of another entry point (E4M3,
 *                        int8): D[t] = act(C[t] + s_a (X[t] . A_a^T) . B_a^T + bias)
 *
 * with a = ids[t]. The conventions of dgemm.h and dgemm_experts.h hold: row-major
 * contiguous matrices on 16-byte addresses (int32 and float tables: natural alignment),
 * DEVICE pointers, memory of the caller, asynchronous calls that never allocate,
 * argument errors before any launch, bounded waits that are recorded in the first
 * DGEMM_WS_STATUS_BYTES bytes of the workspace. Of the planner overrides of dgemm.h,
 * wait_limit_ns, stall_after_loads and cta_pair apply (0: the form for few rows, 1: the
 * one for prompts; sums are in another order, so bits may differ). A workspace serves
 * one call at a time: calls that may overlap on the GPU (two streams, two graphs) need
 * one each.
 */
#ifndef DGEMM_ADAPTERS_H
#define DGEMM_ADAPTERS_H

#include "dgemm_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most adapters of one call, and the largest rank. */
#define DGEMM_MAX_ADAPTERS 4096
#define DGEMM_MAX_ADAPTER_RANK 128

/* D[t,:] = act(X[t,:] . W^T + scale[a] * (X[t,:] . A[a]^T) . B[a]^T + bias), a = ids[t].
 *   X      [T,K] BF16.     W [N,K] BF16: the weights that all rows share.
 *   A      [L,r,K] BF16.   B [L,N,r] BF16.
 *   ids    [T] int32: the adapter of each row; a value outside [0,L) (-1): none, the row
 *          is the shared projection alone. Any order; rows of one adapter next to
 *          each other cost least.
 *   scale  [L] F32 or NULL (all 1).
 *   bias   [N] F32 or NULL.
 *   act    dgemm_act_t or DGEMM_ACT_SWIGLU (gate channels first in W, B and bias; N even).
 *   D      [T,N] (SWIGLU: [T,N/2]) F32 or BF16; overlaps no operand.
 *   ws     dgemm_adapter_workspace_size(T, N, K, r, L) bytes, contents arbitrary
 *          (DGEMM_ERR_WORKSPACE_TOO_SMALL with less).
 * FP32 accumulation, one rounding to D's type. V = scale[a] * (X . A_a^T) is summed and scaled
 * in FP32. The form for few rows keeps it so; the one for prompts keeps two BF16 numbers
 * whose sum is V up to 2^-17 of it (a magnitude of 3.39e38 or more, that BF16 cannot hold,
 * counts as infinite there). A row depends on its own adapter alone:
 * NaN and infinities in another one do not reach it. NaN stays NaN under every activation.
 * r and K are multiples of 8 (DGEMM_ERR_MISALIGNED otherwise), 8 <= r <= DGEMM_MAX_ADAPTER_RANK,
 * 0 <= L <= DGEMM_MAX_ADAPTERS, T <= 2^24, N and K below 2^30 (DGEMM_ERR_NOT_SUPPORTED
 * beyond). K == 0: every product is zero. */
dgemm_status_t dgemm_adapter_bf16(const void* X, const void* W, const void* A, const void* B, const int32_t* ids,
                                  const float* scale, int64_t L, int64_t r, void* D, dgemm_dtype_t d_dtype, int64_t T,
                                  int64_t N, int64_t K, const float* bias, int act, void* ws, size_t ws_bytes,
                                  dgemm_stream_t stream);

/* D[t,:] = act(C[t,:] + scale[a] * (X[t,:] . A[a]^T) . B[a]^T + bias).
 *   C      [T,N] F32 or BF16, or NULL (zero); may equal D when the types are the same.
 *   act    dgemm_act_t (not SWIGLU).
 * The rest as above. With C == NULL the result can be the C operand (beta = 1) of a shared
 * product with a fused epilogue. */
dgemm_status_t dgemm_adapter_add(const void* X, const void* A, const void* B, const int32_t* ids, const float* scale,
                                 int64_t L, int64_t r, const void* C, dgemm_dtype_t c_dtype, void* D,
                                 dgemm_dtype_t d_dtype, int64_t T, int64_t N, int64_t K, const float* bias, int act,
                                 void* ws, size_t ws_bytes, dgemm_stream_t stream);

/* Workspace bytes either call needs with these sizes; 0 for invalid ones. */
size_t dgemm_adapter_workspace_size(int64_t T, int64_t N, int64_t K, int64_t r, int64_t L);

#ifdef __cplusplus
}
#endif

#endif /* DGEMM_ADAPTERS_H */
