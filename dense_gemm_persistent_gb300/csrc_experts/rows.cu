// rows.cu -- the row operators around the products: dgemm_combine (weighted sum
// of a token's expert rows) and dgemm_int8_quantize (per-token int8 codes).
// Both read their input once and are bound by HBM.
#include <cuda_bf16.h>

#include "dgemm_experts.h"
#include "host.h"
#include "ptx.cuh"

namespace {

__device__ __forceinline__ float load1(const void* x, int f32, int64_t i) {
    return f32 ? static_cast<const float*>(x)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(x)[i]);
}

// ---------------------------------------------------------------- combine

// out[t,h] = add[t,h] + sum_j w[t,j] Y[slot_row[t,j],h], j ascending, in FP32.
__global__ void __launch_bounds__(256)
    combine_rows(const __nv_bfloat16* Y, int64_t R, const int* slot_row, const float* weights,
                 const __nv_bfloat16* add, void* out, int out_f32, int64_t H, int k) {
    dg::grid_dependency_wait();
    if (threadIdx.x == 0) dg::grid_launch_dependents();
    const int64_t t = blockIdx.x;
    for (int64_t h = blockIdx.y * 256 + threadIdx.x; h < H; h += gridDim.y * 256) {
        float acc = 0.0f;
        for (int j = 0; j < k; ++j) {
            const int r = slot_row[t * k + j];
            if (r >= 0 && r < R) acc = fmaf(weights[t * k + j], __bfloat162float(Y[r * H + h]), acc);
        }
        if (add) acc += __bfloat162float(add[t * H + h]);
        if (out_f32)
            static_cast<float*>(out)[t * H + h] = acc;
        else
            static_cast<__nv_bfloat16*>(out)[t * H + h] = __float2bfloat16_rn(acc);
    }
}

// ---------------------------------------------------------------- int8 codes

// The code of x for scale s: x / s to the nearest integer, ties to even; NaN 0.
__device__ __forceinline__ int8_t int8_code(float x, float s) {
    const float q = rintf(__fdiv_rn(x, s));
    return x != x ? 0 : static_cast<int8_t>(fminf(fmaxf(q, -127.0f), 127.0f));
}

// One CTA per row: maximum of the finite magnitudes, then the codes.
__global__ void __launch_bounds__(512) quantize_rows(const void* X, int f32, int8_t* q, float* scale, int64_t K) {
    __shared__ unsigned part[16];
    dg::grid_dependency_wait();
    if (threadIdx.x == 0) dg::grid_launch_dependents();
    const int64_t at = static_cast<int64_t>(blockIdx.x) * K;
    unsigned m = 0;                       // magnitudes order as their bits
    for (int64_t i = threadIdx.x; i < K; i += blockDim.x) {
        const unsigned u = __float_as_uint(load1(X, f32, at + i)) & 0x7FFFFFFFu;
        if (u < 0x7F800000u) m = max(m, u);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int w = 0; w < 16; ++w) m = max(m, part[w]);
    float s = __fdiv_rn(__uint_as_float(m), 127.0f);
    if (s == 0.0f) s = 1.0f;              // a row of zeros (or one whose scale underflows)
    if (threadIdx.x == 0) scale[blockIdx.x] = s;
    for (int64_t i = threadIdx.x; i < K; i += blockDim.x) q[at + i] = int8_code(load1(X, f32, at + i), s);
}

}  // namespace

extern "C" dgemm_status_t dgemm_combine(const void* Y, int64_t R, const int32_t* slot_row, const float* weights,
                                        const void* add, void* out, dgemm_dtype_t out_dtype, int64_t T, int64_t H,
                                        int k, dgemm_stream_t stream) {
    if (T < 0 || H < 0 || R < 0 || k < 1) return DGEMM_ERR_INVALID_VALUE;
    if (out_dtype != DGEMM_F32 && out_dtype != DGEMM_BF16) return DGEMM_ERR_INVALID_VALUE;
    if (k > DGEMM_MAX_TOPK || T > INT32_MAX / 2 || H > INT32_MAX / 2 || R > INT32_MAX / 2) return DGEMM_ERR_NOT_SUPPORTED;
    if (T == 0 || H == 0) return DGEMM_OK;
    if ((R > 0 && !Y) || !slot_row || !weights || !out) return DGEMM_ERR_INVALID_VALUE;
    const uintptr_t natural = reinterpret_cast<uintptr_t>(slot_row) | reinterpret_cast<uintptr_t>(weights);
    if (!dg::host::aligned16(Y) || !dg::host::aligned16(add) || !dg::host::aligned16(out) || (natural & 3u))
        return DGEMM_ERR_MISALIGNED;
    dg::host::Device dev;
    const dgemm_status_t ds = dg::host::current_device(&dev);
    if (ds != DGEMM_OK) return ds;
    dg::host::Launch l(static_cast<unsigned>(T), 1, 256, 0, reinterpret_cast<cudaStream_t>(stream));
    const cudaError_t e =
        cudaLaunchKernelEx(&l.cfg, combine_rows, static_cast<const __nv_bfloat16*>(Y), R, static_cast<const int*>(slot_row),
                           weights, static_cast<const __nv_bfloat16*>(add), out, out_dtype == DGEMM_F32 ? 1 : 0, H, k);
    return e == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
}

extern "C" dgemm_status_t dgemm_int8_quantize(const void* X, dgemm_dtype_t x_dtype, int8_t* q, float* scale, int64_t M,
                                              int64_t K, dgemm_stream_t stream) {
    if (M < 0 || K < 0) return DGEMM_ERR_INVALID_VALUE;
    if (x_dtype != DGEMM_F32 && x_dtype != DGEMM_BF16) return DGEMM_ERR_INVALID_VALUE;
    if (M > INT32_MAX / 2 || K > INT32_MAX / 2) return DGEMM_ERR_NOT_SUPPORTED;
    if (M == 0) return DGEMM_OK;
    if ((K > 0 && (!X || !q)) || !scale) return DGEMM_ERR_INVALID_VALUE;
    if (!dg::host::aligned16(X) || !dg::host::aligned16(q) || (reinterpret_cast<uintptr_t>(scale) & 3u))
        return DGEMM_ERR_MISALIGNED;
    dg::host::Device dev;
    const dgemm_status_t ds = dg::host::current_device(&dev);
    if (ds != DGEMM_OK) return ds;
    dg::host::Launch l(static_cast<unsigned>(M), 1, 512, 0, reinterpret_cast<cudaStream_t>(stream));
    const cudaError_t e = cudaLaunchKernelEx(&l.cfg, quantize_rows, X, x_dtype == DGEMM_F32 ? 1 : 0, q, scale, K);
    return e == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
}
