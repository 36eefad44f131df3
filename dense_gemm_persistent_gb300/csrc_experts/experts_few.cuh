// experts_few.cuh -- int8 products of few token rows (up to 4 a group), on the integer
// dot-product units: every weight code is read once, multiplied with the ROWS codes of its
// K in registers, and dropped. No conversion, no tensor core, sums exact in 32 bits
// (up to K = 131071: 128 x 128 x K < 2^31).
//
// A warp holds 4 output channels (a gated call: 2 of the gate, 2 of the up half) x ROWS
// token rows as 32-bit sums; its lanes split K in chunks of 16 codes, so a warp's load of
// one channel is 512 contiguous bytes. The token rows lie in shared memory and a chunk
// read from there serves 4 channels. At the end the lanes' sums are folded so that each
// lane ends up with its own outputs (halving exchange: as many shuffles as sums).
// What bounds it: HBM for one or two rows, then the dot products (4 x ROWS per 16 bytes of
// weights). 18432 x 7168 with 1 / 2 / 4 rows takes 25.5 / 25.9 / 32.0 us (5.2 TB/s for one) where the
// tensor-core kernel takes 34.2; tiles of 8 rows took 50 and are left to that one.
#pragma once

#include "experts_common.cuh"

namespace dg {
namespace experts {

template <int ROWS_>
struct FewCfg {
    static constexpr int ROWS = ROWS_;
    static constexpr int CH = 4;                  // channels of a warp
    static constexpr int WARPS = 8, THREADS = 32 * WARPS;
    static constexpr int TILE = CH * WARPS;       // weight rows of a CTA's tile
    static constexpr int CTAS_PER_SM = 3;
};

__device__ __forceinline__ uint4 load_stream(const void* p) {
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ int dot16(uint4 a, uint4 b, int sum) {
    sum = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), sum);
    sum = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), sum);
    sum = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), sum);
    return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), sum);
}

template <class CF>
__global__ void __launch_bounds__(CF::THREADS, CF::CTAS_PER_SM) expert_few(const void* B, const Params p) {
    extern __shared__ uint4 xs[];                 // [ROWS][K / 16], then the schedule
    constexpr int ROWS = CF::ROWS, CH = CF::CH, V = ROWS * CH;
    const int chunks = p.K / 16;
    const Schedule sched(xs + static_cast<size_t>(ROWS) * chunks, p.E);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    if (warp == 0) build_schedule<ROWS>(p, sched);
    __syncthreads();
    const int tile_channels = p.gated ? CF::TILE / 2 : CF::TILE;
    // Every CTA has a run of consecutive tiles, channels first, so that the token rows in
    // shared memory serve many of them.
    const int64_t tiles = static_cast<int64_t>(sched.head[1]) * p.ctiles;
    const int first_item = static_cast<int>(tiles * blockIdx.x / gridDim.x), last_item = static_cast<int>(tiles * (blockIdx.x + 1) / gridDim.x);
    int group = 0, held = -1;                     // held: first token row of those in shared memory
    Tile t;
    for (int item = first_item; item < last_item; ++item) {
        while (item >= static_cast<int64_t>(sched.cum[group + 1]) * p.ctiles) ++group;
        const int in = item - sched.cum[group] * p.ctiles;
        t.expert = sched.id[group];
        t.row0 = sched.lo[group] + in / p.ctiles * ROWS;
        t.rows = min(ROWS, sched.hi[group] - t.row0);
        t.chan0 = in % p.ctiles * tile_channels;
        // this warp's weight rows (a channel beyond the last reads the last one's and is not stored)
        const char* w[CH];
        const int first = t.chan0 + warp * (p.gated ? CH / 2 : CH);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = min(first + (p.gated ? c % (CH / 2) : c), p.wide - 1);
            const int n = p.gated && c >= CH / 2 ? p.N / 2 + ch : ch;
            w[c] = static_cast<const char*>(B) + (static_cast<int64_t>(t.expert) * p.N + n) * p.K;
        }
        uint4 next[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) next[c] = lane < chunks ? load_stream(w[c] + lane * 16) : make_uint4(0, 0, 0, 0);
        if (t.row0 != held) {
        held = t.row0;
        __syncthreads();                          // the rows before have been read
        for (int i = threadIdx.x; i < ROWS * chunks; i += CF::THREADS) {
            const int r = i / chunks;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < t.rows) {
                const int a = p.a_rows ? __ldg(p.a_rows + t.row0 + r) : t.row0 + r;
                if (a >= 0 && a < p.a_count)
                    v = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(p.A) + static_cast<int64_t>(a) * p.K) + (i - r * chunks));
            }
            xs[i] = v;
        }
        __syncthreads();
        }
        int sum[V];
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = 0;
        for (int k = lane; k < chunks; k += 32) {
            uint4 now[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                now[c] = next[c];
                next[c] = k + 32 < chunks ? load_stream(w[c] + (k + 32) * 16) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const uint4 x = xs[r * chunks + k];
#pragma unroll
                for (int c = 0; c < CH; ++c) sum[r * CH + c] = dot16(now[c], x, sum[r * CH + c]);
            }
        }
        __syncwarp();
        // halving exchange: lanes with the bit keep the upper half of the sums
        int left = V, bit = 16;
#pragma unroll
        for (int step = 0; step < 5; ++step, bit >>= 1) {
            if (left > 1) {
                left /= 2;
                const bool upper = lane & bit;
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    if (i >= left) break;
                    const int send = upper ? sum[i] : sum[i + left];
                    sum[i] = (upper ? sum[i + left] : sum[i]) + __shfl_xor_sync(kAllLanes, send, bit);
                }
            } else {
                sum[0] += __shfl_xor_sync(kAllLanes, sum[0], bit);
            }
        }
        // sums of this lane: V >= 32: V / 32 of them from index lane * (V / 32); V < 32: one, index lane / (32 / V)
        constexpr int MINE = V >= 32 ? V / 32 : 1;
        const int base = V >= 32 ? lane * MINE : lane / (32 / V);
        float y[MINE];
        bool stored[MINE];
        int64_t at[MINE];
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
            const int r = (base + i) / CH, c = (base + i) % CH;
            const int ch = first + (p.gated ? c % (CH / 2) : c);
            stored[i] = r < t.rows && ch < p.wide && (V >= 32 || lane % (32 / (V < 32 ? V : 32)) == 0);
            const int n = min(ch, p.wide - 1) + (p.gated && c >= CH / 2 ? p.N / 2 : 0);
            const int64_t en = static_cast<int64_t>(t.expert) * p.N + n;
            const int row = t.row0 + min(r, t.rows - 1);
            const int a = p.a_rows ? __ldg(p.a_rows + row) : row;
            const float as = a >= 0 && a < p.a_count ? __ldg(p.a_scale + a) : 0.0f;
            y[i] = fmaf(static_cast<float>(sum[i]), p.alpha * __ldg(p.b_scale + en) * as, p.bias ? __ldg(p.bias + en) : 0.0f);
            at[i] = static_cast<int64_t>(row) * p.wide + ch;
            if (p.C && stored[i]) {
                const float x = p.c_f32 ? static_cast<const float*>(p.C)[at[i]]
                                        : __bfloat162float(static_cast<const __nv_bfloat16*>(p.C)[at[i]]);
                y[i] = fmaf(p.beta, x, y[i]);
            }
        }
        if (p.gated) {
            // channels 0, 1 are the gate's, 2, 3 the up half's of the same row
            if constexpr (MINE == 1) {
                const float up = __shfl_xor_sync(kAllLanes, y[0], V >= 32 ? 2 : 2 * (32 / V));
                stored[0] = stored[0] && base % CH < CH / 2;
                y[0] = silu(y[0]) * up;
            } else {
                // a lane has channels 0, 1 or 2, 3 of one row
                const float up0 = __shfl_xor_sync(kAllLanes, y[0], 1), up1 = __shfl_xor_sync(kAllLanes, y[1], 1);
                y[0] = silu(y[0]) * up0;
                y[1] = silu(y[1]) * up1;
                stored[0] = stored[0] && base % CH == 0;
                stored[1] = stored[1] && base % CH == 0;
            }
        }
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
            if (!stored[i]) continue;
            float v = y[i];
            if (p.act == DGEMM_ACT_RELU) v = fmaxf(v, 0.0f);
            else if (p.act == DGEMM_ACT_GELU) v = 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
            else if (p.act == DGEMM_ACT_SILU) v = silu(v);
            if (p.d_f32) static_cast<float*>(p.D)[at[i]] = v;
            else static_cast<__nv_bfloat16*>(p.D)[at[i]] = __float2bfloat16_rn(v);
        }
    }
}

}  // namespace experts
}  // namespace dg
