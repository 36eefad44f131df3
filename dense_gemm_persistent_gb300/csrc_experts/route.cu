// route.cu -- dgemm_route: top-k experts of each token, their weights, and the
// (token, slot) pairs grouped by expert.
//
// Per token: p = exp(x - max x), the k largest x (equal ones lowest index
// first), w = p / sum. Grouping is a counting sort that keeps token order: the
// row of pair (t, j) with expert e is
//     offsets[e] + #{pairs with expert e and a smaller token},
// since a token has an expert at most once. Tokens are cut into chunks of
// CHUNK; a chunk's pairs with expert e are the bits of a mask (bit = token),
// so the count inside the chunk is a popcount -- no atomics whose order shows.
// One launch for up to a chunk of tokens, two beyond.
//
// What bounds it: T x E logits in, 16 bytes per pair out; a long prompt is bound by
// HBM and by the two passes over the chunk counts, a decoding call by its launch.
#include <cuda_bf16.h>

#include "dgemm_experts.h"
#include "host.h"
#include "ptx.cuh"

namespace {

constexpr int CHUNK = 64;       // tokens per chunk: one 64-bit mask per expert
constexpr int WARPS = 16;       // warps per CTA

struct RouteParams {
    const void* logits;
    int bf16, T, E, k, renorm;
    int* ids;
    float* weights;
    int* offsets;
    int* row_token;
    int* slot_row;
    uint8_t* counts;            // [chunks][E rounded up to 4]: at most CHUNK each
    int chunks, pitch;
};

// Order-preserving map of a finite float to unsigned (0 is below every one).
__device__ __forceinline__ unsigned ordered(float x) {
    const unsigned u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(unsigned o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// One token by one warp: lane l holds entries l, l + 32, ... as ordered keys; 0 marks a
// masked or chosen one.
template <int VPL>
__device__ __forceinline__ void route_token(const RouteParams& p, int t, int lane, int* sid) {
    unsigned key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        key[i] = 0;
        if (e < p.E) {
            const int64_t at = static_cast<int64_t>(t) * p.E + e;
            float x = p.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[at])
                             : static_cast<const float*>(p.logits)[at];
            // masked: NaN and -inf; +inf counts as the largest finite number; -0 equals 0
            if (x > -INFINITY) key[i] = ordered(fminf(x, 3.402823466e38f) + 0.0f);
        }
    }
    unsigned best = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
    const unsigned top = __reduce_max_sync(0xffffffffu, best);
    const float xmax = unordered(top);
    float total = 0.0f;
    if (!p.renorm) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i]) total += expf(unordered(key[i]) - xmax);
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    int my_id = -1;             // lane j keeps the j-th choice
    float my_p = 0.0f;
    for (int j = 0; j < p.k; ++j) {
        const unsigned m = __reduce_max_sync(0xffffffffu, best);
        if (m == 0) break;      // nothing unmasked is left
        unsigned at = 0xffffffffu;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
            if (key[i] == m) at = static_cast<unsigned>(lane + 32 * i);
        const unsigned e = __reduce_min_sync(0xffffffffu, at);
        if (lane == j) {
            my_id = static_cast<int>(e);
            my_p = expf(unordered(m) - xmax);
        }
        if (at == e) {
            best = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                if (lane + 32 * i == static_cast<int>(e)) key[i] = 0;
                best = max(best, key[i]);
            }
        }
    }
    if (p.renorm) {
        total = my_p;
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (lane < p.k) {
        const int64_t at = static_cast<int64_t>(t) * p.k + lane;
        p.ids[at] = my_id;
        p.weights[at] = my_id >= 0 ? my_p / total : 0.0f;
        sid[lane] = my_id;
    }
}

// Exclusive scan of total[0 .. E) over the experts in place, by all threads of the CTA
// (each one or two experts of a run); returns the sum.
__device__ __forceinline__ int scan_experts(int* total, int E) {
    __shared__ int warp_sum[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int per = (E + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    const int first = threadIdx.x * per, last = min(first + per, E);
    int mine = 0;
    for (int e = first; e < last; ++e) mine += total[e];
    int inc = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int before = inc - mine, all = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) before += warp_sum[w];
        all += warp_sum[w];
    }
    for (int e = first; e < last; ++e) {
        const int v = total[e];
        total[e] = before;
        before += v;
    }
    __syncthreads();
    return all;
}

// Places the pairs of one chunk: base[e] is the first row of expert e, before[e] (null: none)
// the pairs with e in earlier chunks, mask[e] the chunk's tokens with e.
__device__ __forceinline__ void place_chunk(const RouteParams& p, int t0, int n, const unsigned long long* mask,
                                            const int* base, const int* before, int all) {
    for (int i = threadIdx.x; i < n * p.k; i += blockDim.x) {
        const int64_t at = static_cast<int64_t>(t0) * p.k + i;
        const int e = p.ids[at], tok = i / p.k;
        int row = -1;
        if (e >= 0) {
            row = base[e] + (before ? before[e] : 0) + __popcll(mask[e] & ((1ull << tok) - 1));
            p.row_token[row] = t0 + tok;
        }
        p.slot_row[at] = row;
        if (at >= all) p.row_token[at] = -1;
    }
}

// Selects the experts of one chunk of tokens and counts them. A call of one chunk is
// placed here as well: one launch.
template <int VPL>
__global__ void __launch_bounds__(32 * WARPS) route_select(const RouteParams p) {
    extern __shared__ unsigned long long mask[];            // [E]
    int* total = reinterpret_cast<int*>(mask + p.E);        // [E] (one chunk)
    int* sid = total + p.E;                                 // [CHUNK][k]
    dg::grid_dependency_wait();
    if (threadIdx.x == 0) dg::grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = blockIdx.x * CHUNK, n = min(CHUNK, p.T - t0);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) mask[e] = 0;
    __syncthreads();
    for (int i = warp; i < n; i += WARPS) {
        route_token<VPL>(p, t0 + i, lane, sid + i * p.k);
        __syncwarp();
        if (lane < p.k && sid[i * p.k + lane] >= 0) atomicOr(&mask[sid[i * p.k + lane]], 1ull << i);
    }
    __syncthreads();
    if (p.chunks > 1) {
        for (int e = threadIdx.x; e < p.pitch; e += blockDim.x)
            p.counts[static_cast<int64_t>(blockIdx.x) * p.pitch + e] =
                e < p.E ? static_cast<uint8_t>(__popcll(mask[e])) : 0;
        return;
    }
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) total[e] = __popcll(mask[e]);
    __syncthreads();
    const int all = scan_experts(total, p.E);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.offsets[e] = total[e];
    if (threadIdx.x == 0) p.offsets[p.E] = all;
    place_chunk(p, t0, n, mask, total, nullptr, all);
}

// Rows of one chunk's pairs: every CTA sums the counts of the chunks before its own
// and of all chunks (four experts a load, all loads of a thread in flight together),
// scans the totals over the experts, and places its pairs.
__global__ void __launch_bounds__(1024) route_place(const RouteParams p) {
    extern __shared__ unsigned long long mask[];            // [E]
    int* before = reinterpret_cast<int*>(mask + p.E);       // [pitch] pairs of e in earlier chunks
    int* base = before + p.pitch;                           // [pitch] first row of e
    dg::grid_dependency_wait();
    if (threadIdx.x == 0) dg::grid_launch_dependents();
    for (int e = threadIdx.x; e < p.pitch; e += blockDim.x) {
        if (e < p.E) mask[e] = 0;
        before[e] = 0;
        base[e] = 0;
    }
    __syncthreads();
    const int quads = p.pitch / 4, parts = max(1, static_cast<int>(blockDim.x) / quads);
    const int quad = threadIdx.x % quads, part = threadIdx.x / quads;
    const int mine = static_cast<int>(blockIdx.x);
    if (part < parts) {
        int sum[4] = {0, 0, 0, 0}, pre[4] = {0, 0, 0, 0};
#pragma unroll 8
        for (int c = part; c < p.chunks; c += parts) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(p.counts + static_cast<int64_t>(c) * p.pitch + quad * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int x = (v >> (8 * i)) & 0xFF;
                sum[i] += x;
                if (c < mine) pre[i] += x;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (sum[i]) atomicAdd(&base[quad * 4 + i], sum[i]);     // integers: any order
            if (pre[i]) atomicAdd(&before[quad * 4 + i], pre[i]);
        }
    }
    const int t0 = blockIdx.x * CHUNK, n = min(CHUNK, p.T - t0);
    for (int i = threadIdx.x; i < n * p.k; i += blockDim.x) {
        const int e = p.ids[static_cast<int64_t>(t0) * p.k + i];
        if (e >= 0) atomicOr(&mask[e], 1ull << (i / p.k));
    }
    __syncthreads();
    const int all = scan_experts(base, p.E);
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.offsets[e] = base[e];
        if (threadIdx.x == 0) p.offsets[p.E] = all;
    }
    place_chunk(p, t0, n, mask, base, before, all);
}

dgemm_status_t route_sizes(int64_t T, int64_t E, int k) {
    if (T < 0 || E < 1 || k < 1 || k > E) return DGEMM_ERR_INVALID_VALUE;
    if (E > DGEMM_MAX_EXPERTS || k > DGEMM_MAX_TOPK || T * k >= (int64_t(1) << 30) || T > (int64_t(1) << 30))
        return DGEMM_ERR_NOT_SUPPORTED;
    return DGEMM_OK;
}

template <int VPL>
cudaError_t launch_select(const RouteParams& p, cudaStream_t s) {
    dg::host::Launch l(static_cast<unsigned>(p.chunks), 1, 32 * WARPS, static_cast<size_t>(p.E) * 12 + CHUNK * p.k * 4, s);
    return cudaLaunchKernelEx(&l.cfg, route_select<VPL>, p);
}

}  // namespace

extern "C" size_t dgemm_route_workspace_size(int64_t T, int64_t E, int k) {
    if (route_sizes(T, E, k) != DGEMM_OK) return 0;
    const size_t chunks = static_cast<size_t>((T + CHUNK - 1) / CHUNK);
    return chunks > 1 ? chunks * ((static_cast<size_t>(E) + 3) / 4 * 4) : 0;
}

extern "C" dgemm_status_t dgemm_route(const void* logits, dgemm_dtype_t logits_dtype, int64_t T, int64_t E, int k,
                                      int renormalize, int32_t* ids, float* weights, int32_t* offsets,
                                      int32_t* row_token, int32_t* slot_row, void* ws, size_t ws_bytes,
                                      dgemm_stream_t stream) {
    const dgemm_status_t st = route_sizes(T, E, k);
    if (st != DGEMM_OK) return st;
    if (logits_dtype != DGEMM_F32 && logits_dtype != DGEMM_BF16) return DGEMM_ERR_INVALID_VALUE;
    if (!offsets || (T > 0 && (!logits || !ids || !weights || !row_token || !slot_row))) return DGEMM_ERR_INVALID_VALUE;
    const uintptr_t natural = reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(weights) |
                              reinterpret_cast<uintptr_t>(offsets) | reinterpret_cast<uintptr_t>(row_token) |
                              reinterpret_cast<uintptr_t>(slot_row);
    if ((natural & 3u) || !dg::host::aligned16(logits) || !dg::host::aligned16(ws)) return DGEMM_ERR_MISALIGNED;
    const size_t need = dgemm_route_workspace_size(T, E, k);
    if (need > 0 && (!ws || ws_bytes < need)) return DGEMM_ERR_WORKSPACE_TOO_SMALL;
    dg::host::Device dev;
    const dgemm_status_t ds = dg::host::current_device(&dev);
    if (ds != DGEMM_OK) return ds;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0)
        return cudaMemsetAsync(offsets, 0, static_cast<size_t>(E + 1) * 4, s) == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
    RouteParams p{};
    p.logits = logits;
    p.bf16 = logits_dtype == DGEMM_BF16;
    p.T = static_cast<int>(T);
    p.E = static_cast<int>(E);
    p.k = k;
    p.renorm = renormalize != 0;
    p.ids = ids;
    p.weights = weights;
    p.offsets = offsets;
    p.row_token = row_token;
    p.slot_row = slot_row;
    p.counts = static_cast<uint8_t*>(ws);
    p.pitch = (p.E + 3) / 4 * 4;
    p.chunks = static_cast<int>((T + CHUNK - 1) / CHUNK);
    cudaError_t e;
    if (E <= 64) e = launch_select<2>(p, s);
    else if (E <= 128) e = launch_select<4>(p, s);
    else if (E <= 256) e = launch_select<8>(p, s);
    else if (E <= 512) e = launch_select<16>(p, s);
    else e = launch_select<32>(p, s);
    if (e != cudaSuccess) return DGEMM_ERR_CUDA;
    if (p.chunks == 1) return DGEMM_OK;
    dg::host::Launch l(static_cast<unsigned>(p.chunks), 1, 1024, static_cast<size_t>(p.pitch) * 16, s);
    return cudaLaunchKernelEx(&l.cfg, route_place, p) == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
}
