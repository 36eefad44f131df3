// rows.cu -- the row operators around the products: dgemm_combine (weighted sum
// of a token's expert rows) and dgemm_int8_quantize (per-token int8 codes).
//
// Combining 8192 x 7168, top 8, takes 165 us: HBM at 6.4 TB/s. Quantising 4096 x 4096 BF16 takes
// 11.9 us (4.2 TB/s, 7.5 us for its bytes; 4096 x 8192 21.9 us): a CTA has one row and nothing of
// another in flight while it finds the maximum. Rows of more than 8192 values, or of a
// number that is no multiple of 8, are read twice, a value at a time.
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
//
// VEC: a thread sums 8 columns (16 bytes of each row), eight rows in flight. One pass
// over the rows is all there is: the bytes of T x k rows bound it.
struct CombineParams {
    const __nv_bfloat16* Y;
    const int* slot_row;
    const float* weights;
    const __nv_bfloat16* add;
    void* out;
    int64_t R, H;
    int out_f32, k;
    unsigned blocks;        // CTAs per token
};

template <bool VEC>
__global__ void __launch_bounds__(256) combine_rows(const CombineParams p) {
    constexpr int W = VEC ? 8 : 1, BATCH = 8;
    dg::grid_dependency_wait();
    if (threadIdx.x == 0) dg::grid_launch_dependents();
    const int64_t t = blockIdx.x / p.blocks;
    const int64_t h = (static_cast<int64_t>(blockIdx.x % p.blocks) * 256 + threadIdx.x) * W;
    if (h >= p.H) return;
    const int* slots = p.slot_row + t * p.k;
    const float* weights = p.weights + t * p.k;
    float acc[W];
    uint4 a = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < W; ++i) acc[i] = 0.0f;
    if constexpr (VEC)
        if (p.add) a = *reinterpret_cast<const uint4*>(p.add + t * p.H + h);
    for (int j0 = 0; j0 < p.k; j0 += BATCH) {
        int row[BATCH];
        float w[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            row[j] = j0 + j < p.k ? __ldg(slots + j0 + j) : -1;
            w[j] = j0 + j < p.k ? __ldg(weights + j0 + j) : 0.0f;
        }
        uint4 y[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            y[j] = make_uint4(0, 0, 0, 0);
            if (row[j] >= 0 && row[j] < p.R) {
                const __nv_bfloat16* src = p.Y + row[j] * p.H + h;
                if constexpr (VEC) y[j] = __ldcs(reinterpret_cast<const uint4*>(src));
                else y[j].x = __bfloat16_as_ushort(*src);
            }
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            if (row[j] < 0 || row[j] >= p.R) continue;       // adds nothing, whatever its weight
            const uint32_t u[4] = {y[j].x, y[j].y, y[j].z, y[j].w};
#pragma unroll
            for (int i = 0; i < W; ++i) acc[i] = fmaf(w[j], (i & 1) ? dg::bf16_hi(u[i / 2]) : dg::bf16_lo(u[i / 2]), acc[i]);
        }
    }
    const int64_t at = t * p.H + h;
    if constexpr (VEC) {
        if (p.add) {
            const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < W; ++i) acc[i] += (i & 1) ? dg::bf16_hi(u[i / 2]) : dg::bf16_lo(u[i / 2]);
        }
        if (p.out_f32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
            o[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            o[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at) =
                make_uint4(dg::pack_bf16x2(acc[0], acc[1]), dg::pack_bf16x2(acc[2], acc[3]),
                           dg::pack_bf16x2(acc[4], acc[5]), dg::pack_bf16x2(acc[6], acc[7]));
        }
    } else {
        if (p.add) acc[0] += __bfloat162float(p.add[at]);
        if (p.out_f32) static_cast<float*>(p.out)[at] = acc[0];
        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(acc[0]);
    }
}

// ---------------------------------------------------------------- int8 codes

// The code of x for scale s: x / s to the nearest integer, ties to even; NaN 0. The
// product with 1 / s is within 2^-15 of the quotient (|quotient| <= 127), so only
// quotients that near a half are divided.
__device__ __forceinline__ int int8_code(float x, float s, float inv) {
    const float t = x * inv;
    float q = rintf(t);
    if (!(fabsf(t - q) < 0.4999f)) q = rintf(__fdiv_rn(x, s));   // (and what is not finite)
    return x != x ? 0 : static_cast<int>(fminf(fmaxf(q, -127.0f), 127.0f));
}

__device__ __forceinline__ unsigned finite_magnitude(float x) {   // magnitudes order as their bits
    const unsigned u = __float_as_uint(x) & 0x7FFFFFFFu;
    return u < 0x7F800000u ? u : 0u;
}

// The largest of every thread's value; all threads of the CTA take part.
__device__ __forceinline__ unsigned row_max(unsigned m) {
    __shared__ unsigned part[32];
    m = __reduce_max_sync(0xffffffffu, m);
    __syncthreads();                      // (an earlier call's values have been read)
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    for (unsigned w = 0; w < blockDim.x / 32; ++w) m = max(m, part[w]);
    return m;
}

// The row's scale from the bits of its largest finite magnitude.
__device__ __forceinline__ float row_scale(unsigned m, float* scale) {
    float s = __fmul_rn(__uint_as_float(m), 1.0f / 127.0f);
    if (s == 0.0f) s = 1.0f;              // a row of zeros (or one whose scale underflows)
    if (threadIdx.x == 0) *scale = s;
    return s;
}

// Four codes in a word, without conversions: x / s + 1.5 x 2^23 holds the rounded quotient in its
// low byte (two's complement), and the rest of the product says how near a half it was.
// Quotients near a half, and values that are not finite, take int8_code.
__device__ __forceinline__ uint32_t int8_codes4(const float* x, float s, float inv) {
    constexpr float MAGIC = 12582912.0f;
    uint32_t b[4];
    bool far = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float m = fmaf(x[i], inv, MAGIC), r = m - MAGIC;
        far = far && fabsf(fmaf(x[i], inv, -r)) < 0.4999f;
        b[i] = __float_as_uint(m);
    }
    if (!far) {
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = static_cast<uint32_t>(int8_code(x[i], s, inv));
    }
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

// One CTA per row of up to 8 x CHUNKS x blockDim values, held in registers between the
// maximum and the codes: the row is read once.
template <bool F32, int CHUNKS>
__global__ void __launch_bounds__(256) quantize_held(const void* X, int8_t* q, float* scale, int K) {
    dg::grid_dependency_wait();
    if (threadIdx.x == 0) dg::grid_launch_dependents();
    const int64_t at = static_cast<int64_t>(blockIdx.x) * K;
    constexpr int WORDS = F32 ? 8 : 4;    // of 8 values
    uint32_t v[CHUNKS][WORDS];
    unsigned m = 0;                       // F32: the largest magnitude; BF16: two of them
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const int k = (c * blockDim.x + threadIdx.x) * 8;
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (k < K) w = *reinterpret_cast<const uint4*>(static_cast<const char*>(X) + (at + k) * (F32 ? 4 : 2) + i * 4);
            v[c][i] = w.x, v[c][i + 1] = w.y, v[c][i + 2] = w.z, v[c][i + 3] = w.w;
        }
#pragma unroll
        for (int i = 0; i < WORDS; ++i) m = F32 ? max(m, v[c][i] & 0x7FFFFFFFu) : __vmaxu2(m, v[c][i] & 0x7FFF7FFFu);
    }
    auto value = [&](int c, int i) {
        return F32 ? __uint_as_float(v[c][i % WORDS]) : (i & 1) ? dg::bf16_hi(v[c][i / 2]) : dg::bf16_lo(v[c][i / 2]);
    };
    m = row_max(F32 ? m : max(m << 16, m & 0xFFFF0000u));
    if (m >= 0x7F800000u) {               // infinities or NaN in the row: its finite values only
        m = 0;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, finite_magnitude(value(c, i)));
        m = row_max(m);
    }
    const float s = row_scale(m, scale + blockIdx.x), inv = __frcp_rn(s);
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const int k = (c * blockDim.x + threadIdx.x) * 8;
        if (k >= K) continue;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = value(c, i);
        *reinterpret_cast<uint2*>(q + at + k) = make_uint2(int8_codes4(x, s, inv), int8_codes4(x + 4, s, inv));
    }
}

// Rows of any length and alignment, read twice.
__global__ void __launch_bounds__(512) quantize_rows(const void* X, int f32, int8_t* q, float* scale, int64_t K) {
    dg::grid_dependency_wait();
    if (threadIdx.x == 0) dg::grid_launch_dependents();
    const int64_t at = static_cast<int64_t>(blockIdx.x) * K;
    unsigned m = 0;
    for (int64_t i = threadIdx.x; i < K; i += blockDim.x) m = max(m, finite_magnitude(load1(X, f32, at + i)));
    const float s = row_scale(row_max(m), scale + blockIdx.x), inv = __frcp_rn(s);
    for (int64_t i = threadIdx.x; i < K; i += blockDim.x) q[at + i] = static_cast<int8_t>(int8_code(load1(X, f32, at + i), s, inv));
}

template <bool F32>
cudaError_t launch_held(const void* X, int8_t* q, float* scale, int64_t M, int K, cudaStream_t s) {
    dg::host::Launch l(static_cast<unsigned>(M), 1, 256, 0, s);
    if (K <= 2048) return cudaLaunchKernelEx(&l.cfg, quantize_held<F32, 1>, X, q, scale, K);
    if (K <= 4096) return cudaLaunchKernelEx(&l.cfg, quantize_held<F32, 2>, X, q, scale, K);
    return cudaLaunchKernelEx(&l.cfg, quantize_held<F32, 4>, X, q, scale, K);
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
    CombineParams p{static_cast<const __nv_bfloat16*>(Y), slot_row, weights, static_cast<const __nv_bfloat16*>(add), out,
                    R, H, out_dtype == DGEMM_F32 ? 1 : 0, k, 0};
    const bool vec = H % 8 == 0;       // rows on 16 bytes
    p.blocks = static_cast<unsigned>((H / (vec ? 8 : 1) + 255) / 256);
    if (T * p.blocks > INT32_MAX) return DGEMM_ERR_NOT_SUPPORTED;
    dg::host::Launch l(static_cast<unsigned>(T * p.blocks), 1, 256, 0, reinterpret_cast<cudaStream_t>(stream));
    const cudaError_t e =
        vec ? cudaLaunchKernelEx(&l.cfg, combine_rows<true>, p) : cudaLaunchKernelEx(&l.cfg, combine_rows<false>, p);
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
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (K % 8 == 0 && K > 0 && K <= 8192) {
        e = x_dtype == DGEMM_F32 ? launch_held<true>(X, q, scale, M, static_cast<int>(K), st)
                                 : launch_held<false>(X, q, scale, M, static_cast<int>(K), st);
    } else {
        dg::host::Launch l(static_cast<unsigned>(M), 1, 512, 0, st);
        e = cudaLaunchKernelEx(&l.cfg, quantize_rows, X, x_dtype == DGEMM_F32 ? 1 : 0, q, scale, K);
    }
    return e == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
}
