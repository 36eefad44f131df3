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
    float* V;                          // [T][r] FP32, or for the prompt form [T][2][r] BF16: V = first + second
    int* lists;                        // prompt form: [tiles][kListPitch], the adapters of a token tile: how many, which
    unsigned long long* bad;           // prompt form: [L], this call's epoch where B_a has a number that is not finite
    int T, L, r;
    int tiles, width;                  // token tiles and their rows
    int prompt;                        // the prompt form follows
    int shrink_tiles, shrink_cols;     // token tiles of the launch that computes V, its columns of a pass
    int split;                         // CTAs of a cluster that share a tile's K
    int stages;                        // of the ring
    int ahead;                         // few-row form: items of B that a warp copies ahead
    int wait_first;                    // no launch of this call precedes: wait for the stream before reading anything
};

constexpr int kMostWidth = 256;               // rows of a token tile of the prompt form
constexpr int kListPitch = 4 + kMostWidth;    // [0] the count, from [4] on the adapters in order

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

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

__device__ __forceinline__ __nv_bfloat16* v_split(const Params& p, int t) {
    return reinterpret_cast<__nv_bfloat16*>(p.V) + static_cast<int64_t>(t) * 2 * p.r;
}

// Bits of the adapters in use among n rows, by `threads` threads that all pass; words: [128].
__device__ __forceinline__ void mark_adapters(const Params& p, int first, int n, unsigned* words, int tid, int threads) {
    // (loads of a batch before its marks; most are marked already, and a look spares the atomic)
    for (int i0 = tid; i0 < n; i0 += 16 * threads) {
        int a[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) a[k] = i0 + k * threads < n ? adapter_of(p, first + i0 + k * threads) : -1;
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (a[k] >= 0 && !((*reinterpret_cast<volatile unsigned*>(words + (a[k] >> 5)) >> (a[k] & 31)) & 1))
                atomicOr(&words[a[k] >> 5], 1u << (a[k] & 31));
    }
}
// The place of adapter a among the marked ones, and how many there are.
__device__ __forceinline__ int place_of(const Params& p, const unsigned* words, int a) {
    int before = 0;
    for (int w = 0; w < (a >> 5); ++w) before += __popc(words[w]);
    return before + __popc(words[a >> 5] & ((1u << (a & 31)) - 1));
}
__device__ __forceinline__ int marked(const Params& p, const unsigned* words) {
    int all = 0;
    for (int w = 0; w < (p.L + 31) / 32; ++w) all += __popc(words[w]);
    return all;
}

}  // namespace adapters
}  // namespace dg
