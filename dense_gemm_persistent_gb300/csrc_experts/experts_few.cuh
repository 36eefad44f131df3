// experts_few.cuh -- int8 products of one or two token rows and one set of weights, on the
// integer dot-product units: every weight code is read once, multiplied with the ROWS codes of its
// K in registers, and dropped. No conversion, no tensor core, sums exact in 32 bits
// (up to K = 131071: 128 x 128 x K < 2^31).
//
// A warp holds 4 output channels (a gated call: 2 of the gate, 2 of the up half) x ROWS
// token rows as 32-bit sums; its lanes split K in chunks of 16 codes, so a warp's load of
// one channel is 512 contiguous bytes. The token rows lie in shared memory and a chunk
// read from there serves 4 channels. At the end the lanes' sums are folded so that each
// lane ends up with its own output (halving exchange: as many shuffles as sums).
// What bounds it: HBM. On the device, one row and two, against the tensor-core kernel, whose
// tiles of 128 channels leave SMs idle where channels are few:
//   18432 x 7168   24.7, 27.3 us (5.4, 4.8 TB/s)  27.4, 27.5
//   11008 x 4096    9.5, 10.5                     17.3
//    4096 x 4096    5.8,  7.0                     16.2
//    4096 x 14336  14.0, 18.1                     44.6
// The dot products (4 x ROWS per 16 bytes of weights) of tiles of four rows took 1.13 times the
// tensor-core kernel's time for 18432 x 7168; three rows and more of fewer channels were not compared.
// Groups of several experts are left to that kernel too: 64 experts of 2048 x 4096 with one
// row each on average took 1.14 times its time, since many have two.
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
    extern __shared__ uint4 xs[];                 // [ROWS][K / 16]
    constexpr int ROWS = CF::ROWS, CH = CF::CH, V = ROWS * CH;
    static_assert(V <= 32, "an output a lane");
    const int chunks = p.K / 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    // the group's rows: at most R, which is at most ROWS
    const int row0 = p.offsets ? min(max(__ldg(p.offsets), 0), p.R) : 0;
    const int rows = p.offsets ? min(max(__ldg(p.offsets + 1), row0), p.R) - row0 : p.R;
    if (rows == 0) return;
    const int tile_channels = p.gated ? CF::TILE / 2 : CF::TILE;
    // Every CTA has a run of consecutive tiles of channels.
    const int first_item = static_cast<int>(static_cast<int64_t>(p.ctiles) * blockIdx.x / gridDim.x);
    const int last_item = static_cast<int>(static_cast<int64_t>(p.ctiles) * (blockIdx.x + 1) / gridDim.x);
    for (int item = first_item; item < last_item; ++item) {
        // this warp's weight rows (a channel beyond the last reads the last one's and is not stored)
        const char* w[CH];
        const int first = item * tile_channels + warp * (p.gated ? CH / 2 : CH);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int ch = min(first + (p.gated ? c % (CH / 2) : c), p.wide - 1);
            const int n = p.gated && c >= CH / 2 ? p.N / 2 + ch : ch;
            w[c] = static_cast<const char*>(B) + static_cast<int64_t>(n) * p.K;
        }
        uint4 next[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) next[c] = lane < chunks ? load_stream(w[c] + lane * 16) : make_uint4(0, 0, 0, 0);
        if (item == first_item) {                 // the token rows, behind the first loads of weights
            for (int i = threadIdx.x; i < ROWS * chunks; i += CF::THREADS) {
                const int r = i / chunks;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < rows) {
                    const int a = p.a_rows ? __ldg(p.a_rows + row0 + r) : row0 + r;
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
        // this lane's sum is number lane / (32 / V)
        const int mine = lane / (32 / V), r = mine / CH, c = mine % CH;
        const int ch = first + (p.gated ? c % (CH / 2) : c);
        bool stored = r < rows && ch < p.wide && lane % (32 / V) == 0;
        const int n = min(ch, p.wide - 1) + (p.gated && c >= CH / 2 ? p.N / 2 : 0);
        const int row = row0 + min(r, rows - 1);
        const int a = p.a_rows ? __ldg(p.a_rows + row) : row;
        const float as = a >= 0 && a < p.a_count ? __ldg(p.a_scale + a) : 0.0f;
        float y = fmaf(static_cast<float>(sum[0]), p.alpha * __ldg(p.b_scale + n) * as, p.bias ? __ldg(p.bias + n) : 0.0f);
        const int64_t at = static_cast<int64_t>(row) * p.wide + ch;
        if (p.C && stored) {
            const float x = p.c_f32 ? static_cast<const float*>(p.C)[at]
                                    : __bfloat162float(static_cast<const __nv_bfloat16*>(p.C)[at]);
            y = fmaf(p.beta, x, y);
        }
        if (p.gated) {                            // channels 0, 1 are the gate's, 2, 3 the up half's of the same row
            const float up = __shfl_xor_sync(kAllLanes, y, CH / 2 * (32 / V));
            stored = stored && c < CH / 2;
            y = silu(y) * up;
        }
        if (!stored) continue;
        if (p.act == DGEMM_ACT_RELU) y = relu(y);
        else if (p.act == DGEMM_ACT_GELU) y = gelu(y);
        else if (p.act == DGEMM_ACT_SILU) y = silu(y);
        if (p.d_f32) static_cast<float*>(p.D)[at] = y;
        else static_cast<__nv_bfloat16*>(p.D)[at] = __float2bfloat16_rn(y);
    }
}

}  // namespace experts
}  // namespace dg
