// adapter_shrink.cuh -- V[t] = s_a X[t] . A_a^T for every row with an adapter.
#pragma once

#include "adapter_common.cuh"

namespace dg {
namespace adapters {

// A CTA computes RB numbers of one row: its threads share K, partial sums meet in shared memory.
constexpr int SHRINK_THREADS = 128;

template <int RB>
__global__ void __launch_bounds__(SHRINK_THREADS) adapter_shrink_few(const __grid_constant__ Params p) {
    __shared__ float part[SHRINK_THREADS / 32][RB];
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    const int blocks = p.r / RB, t = static_cast<int>(blockIdx.x) / blocks, j0 = (static_cast<int>(blockIdx.x) % blocks) * RB;
    const int a = adapter_of(p, t);
    if (a < 0) return;
    const uint4* x = reinterpret_cast<const uint4*>(p.X + static_cast<int64_t>(t) * p.K);
    const uint4* w = reinterpret_cast<const uint4*>(p.low + (static_cast<int64_t>(a) * p.r + j0) * p.K);
    const int vecs = p.K / 8;
    float s0[RB], s1[RB];
#pragma unroll
    for (int j = 0; j < RB; ++j) s0[j] = s1[j] = 0.0f;
#pragma unroll 4
    for (int i = threadIdx.x; i < vecs; i += SHRINK_THREADS) {
        const uint4 xv = x[i];
        const float4 x0 = make_float4(bf16_lo(xv.x), bf16_hi(xv.x), bf16_lo(xv.y), bf16_hi(xv.y));
        const float4 x1 = make_float4(bf16_lo(xv.z), bf16_hi(xv.z), bf16_lo(xv.w), bf16_hi(xv.w));
#pragma unroll
        for (int j = 0; j < RB; ++j) fma8(s0[j], s1[j], __ldg(w + static_cast<int64_t>(j) * vecs + i), x0, x1);
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j < RB; ++j) {
        float s = s0[j] + s1[j];
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAllLanes, s, o);
        if (lane == 0) part[warp][j] = s;
    }
    __syncthreads();
    if (threadIdx.x < RB) {
        float s = 0.0f;
        for (int i = 0; i < SHRINK_THREADS / 32; ++i) s += part[i][threadIdx.x];
        p.V[static_cast<int64_t>(t) * p.r + j0 + threadIdx.x] = p.scale ? s * p.scale[a] : s;
    }
}

}  // namespace adapters
}  // namespace dg
