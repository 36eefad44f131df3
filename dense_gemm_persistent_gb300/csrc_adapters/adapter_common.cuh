// adapter_common.cuh -- what the kernels of the low-rank adapters share.
//
//     D[t] = act(Y[t] + V[t] . B_a^T + bias),  V[t] = s_a X[t] . A_a^T,  a = ids[t]
//
// with Y = X . W^T (dgemm_adapter_bf16) or C (dgemm_adapter_add). One launch computes V for all
// rows (adapter_shrink.cuh), a second one the rest.
#pragma once

#include <cuda_bf16.h>

#include "dgemm_adapters.h"
#include "experts_common.cuh"
#include "experts_ptx.cuh"

namespace dg {
namespace adapters {

using experts::kAllLanes;

struct Params : experts::Params {      // (of those: C, D, bias, N, K, wide, gated, act, types, kstages, k_whole, status)
    const int* ids;                    // [T]
    const float* scale;                // [L], or null
    const __nv_bfloat16* X;            // [T][K]
    const __nv_bfloat16* low;          // A [L][r][K]
    const __nv_bfloat16* high;         // B [L][N][r]
    float* V;                          // [T][r]
    int T, L, r;
    int tiles, width;                  // token tiles and their rows
    int split;                         // CTAs of a cluster that share a tile's K
    int stages;                        // of the ring
    int wait_first;                    // no launch of this call precedes: wait for the stream before reading anything
};

// The adapter of row t, -1 for none.
__device__ __forceinline__ int adapter_of(const Params& p, int t) {
    const int a = p.ids[t];
    return static_cast<unsigned>(a) < static_cast<unsigned>(p.L) ? a : -1;
}

__device__ __forceinline__ void fma8(float& s0, float& s1, const uint4& b, const float4& v0, const float4& v1) {
    s0 = fmaf(v0.x, bf16_lo(b.x), s0);
    s1 = fmaf(v0.y, bf16_hi(b.x), s1);
    s0 = fmaf(v0.z, bf16_lo(b.y), s0);
    s1 = fmaf(v0.w, bf16_hi(b.y), s1);
    s0 = fmaf(v1.x, bf16_lo(b.z), s0);
    s1 = fmaf(v1.y, bf16_hi(b.z), s1);
    s0 = fmaf(v1.z, bf16_lo(b.w), s0);
    s1 = fmaf(v1.w, bf16_hi(b.w), s1);
}

}  // namespace adapters
}  // namespace dg
