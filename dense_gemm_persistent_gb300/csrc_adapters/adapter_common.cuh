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
    void* V;                           // prompt form: BF16 [T][2][r], V = first + second; else float [T][r]
    int* lists;                        // prompt form: [tiles][kListPitch], the adapters of a token tile: how many, which
    int T, L, r;
    int tiles, width;                  // token tiles and their rows
    int prompt;                        // the prompt form follows
    int shrink_tiles, shrink_cols;     // token tiles of the launch that computes V, its columns of a pass
    int split;                         // CTAs of a cluster that share a tile's K
    int stages;                        // of the ring
    int channels;                      // few-row form: of D in a tile, a multiple of 8
    int ahead;                         // few-row form: items of B that a warp copies ahead
    int wait_first;                    // no launch of this call precedes: wait for the stream before reading anything
};

constexpr int kMostWidth = 256;               // rows of a token tile of the prompt form
constexpr int kListPitch = 4 + kMostWidth;    // [0] the count and kUniform, from [1] on the adapters in order
constexpr int kUniform = 1 << 16;             // every row of the tile has the same adapter
constexpr int kAdapterWords = DGEMM_MAX_ADAPTERS / 32, kWords = kAdapterWords + 4;    // a bit for every adapter; rows without one

// y / (1 + e^-y) by the special function unit, 2^-21 relative; below -87 the quotient is zero (at most 2e-36 off).
__device__ __forceinline__ float silu(float y) {
    float e, q;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.0f + e));
    return y * q;
}

// (r0, r1) = (a0 + b0, a1 + b1) as one instruction.
__device__ __forceinline__ void add2(float& r0, float& r1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r0), "=f"(r1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
// Two of silu's values, the products and sums as pairs.
__device__ __forceinline__ void silu2(float& y0, float& y1) {
    float e0, e1, q0, q1;
    fmul2(e0, e1, y0, y1, -1.4426950408889634f, -1.4426950408889634f);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(e0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(e1));
    add2(e0, e1, e0, e1, 1.0f, 1.0f);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q0) : "f"(e0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q1) : "f"(e1));
    fmul2(y0, y1, y0, y1, q0, q1);
}

// The activation of N values: the switch is taken once for all of them.
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
    switch (act) {
        case DGEMM_ACT_RELU:
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = experts::relu(v[j]);
            break;
        case DGEMM_ACT_GELU:
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = experts::gelu(v[j]);
            break;
        case DGEMM_ACT_SILU:
#pragma unroll
            for (int j = 0; j < N; j += 2) silu2(v[j], v[j + 1]);
            break;
        default:
            break;
    }
}

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

// Row t of V: of the prompt form, and of the few-row form.
__device__ __forceinline__ __nv_bfloat16* v_row(const Params& p, int t) {
    return static_cast<__nv_bfloat16*>(p.V) + static_cast<int64_t>(t) * 2 * p.r;
}
__device__ __forceinline__ float* v_row_f32(const Params& p, int t) { return static_cast<float*>(p.V) + static_cast<int64_t>(t) * p.r; }

// Bits of the adapters in use among n rows, by `threads` threads that all pass.
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

// Writes the list of a token tile of the prompt form; words: [kWords] in shared memory; sync() for all of the threads.
template <class Sync>
__device__ __forceinline__ void list_tile(const Params& p, int tile, unsigned* words, int tid, int threads, Sync sync) {
    const int row0 = tile * p.width, rows = min(p.width, p.T - row0);
    for (int w = tid; w < kWords; w += threads) words[w] = 0;
    sync();
    mark_adapters(p, row0, rows, words, tid, threads);
    sync();
    int* list = p.lists + static_cast<int64_t>(tile) * kListPitch;
    for (int i = tid; i < rows; i += threads) {
        const int a = adapter_of(p, row0 + i);
        if (a >= 0) list[1 + place_of(p, words, a)] = a;          // (rows of one adapter write the same)
        else words[kAdapterWords] = 1;
    }
    sync();
    if (tid == 0) {
        const int count = marked(p, words);
        list[0] = count | (count == 1 && words[kAdapterWords] == 0 ? kUniform : 0);
    }
    sync();
}

// The few-row form multiplies V by B on FP32 units and has it in FP32. To the tensor core it goes as two BF16 numbers, in
// the same bytes: a BF16 number has 8 significant bits, so that the first leaves up to 2^-8 of V and the second up to
// 2^-9 of that, V up to 2^-17 in all (an infinity has no second). One alone would cost half of the
// adapter's precision, FP32 has no exact way through.
// Eight numbers of a row, from `at` on.
__device__ __forceinline__ void store_v(const Params& p, int t, int at, const float (&v)[8]) {
    if (!p.prompt) {
        float4* out = reinterpret_cast<float4*>(v_row_f32(p, t) + at);
        out[0] = make_float4(v[0], v[1], v[2], v[3]);
        out[1] = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        hi[c] = pack_bf16x2(v[2 * c], v[2 * c + 1]);
        const float dx = v[2 * c] - bf16_lo(hi[c]), dy = v[2 * c + 1] - bf16_hi(hi[c]);
        lo[c] = pack_bf16x2(fabsf(dx) < INFINITY ? dx : 0.0f, fabsf(dy) < INFINITY ? dy : 0.0f);
    }
    __nv_bfloat16* out = v_row(p, t) + at;
    *reinterpret_cast<uint4*>(out) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(out + p.r) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}
// One of them.
__device__ __forceinline__ void store_one(const Params& p, int t, int at, float v) {
    if (!p.prompt) {
        v_row_f32(p, t)[at] = v;
        return;
    }
    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
    const float rest = v - __bfloat162float(hi);
    v_row(p, t)[at] = hi;
    v_row(p, t)[p.r + at] = __float2bfloat16_rn(fabsf(rest) < INFINITY ? rest : 0.0f);
}

}  // namespace adapters
}  // namespace dg
