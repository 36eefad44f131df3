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
// What bounds it: a decoding call its launch (one token of 64 experts 3.3 us on the device). A long
// prompt is far from its bytes (T x E logits in, 16 bytes per pair out; 16001 x 256 BF16, top 8,
// 22.5 us against 1.5): the k selection rounds of a token each wait for a reduction over the
// warp (55 % of issue slots), and every CTA that places reads the counts of all chunks, which
// grows with the square of T (131072 x 256 262 us).
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

#include "dgemm_experts.h"
#include "host.h"
#include "ptx.cuh"
#include "route_layout.h"

namespace {

constexpr int CHUNK = 64;       // most tokens of a chunk: one 64-bit mask per expert

constexpr int kMoreChunks = 64;  // chunks beyond the fewest that a call may be cut into (workspace)

struct RouteParams {
    const void* logits;
    int bf16, T, E, k, renorm;
    int* ids;
    float* weights;
    int* offsets;
    int* row_token;
    int* slot_row;
    uint8_t* counts;            // [chunks][E rounded up to 4]: at most CHUNK each
    int chunks, pitch, chunk;   // tokens of a chunk
};

// Order-preserving map of a finite float to unsigned (0 is below every one).
__device__ __forceinline__ unsigned ordered(float x) {
    const unsigned u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(unsigned o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// One token by one warp: lane l holds entries l, l + 32, ... as order-preserving keys; 0
// marks a masked or chosen one. Each round takes the warp's largest key. BF16: a
// key is the value's 16 bits over the complement of the index, so keys differ, one
// reduction names the winner, and up to 8 keys a lane are sorted first, so that a round
// looks at the first and moves the winner's up. FP32: the value's 32 bits; a ballot
// names the winner, and where several lanes hold that value the lowest index wins.
template <int VPL, bool BF16>
__device__ __forceinline__ void load_keys(const RouteParams& p, int t, int lane, unsigned (&key)[VPL]) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        key[i] = 0;
        if (e < p.E) {
            const int64_t at = static_cast<int64_t>(t) * p.E + e;
            const float x = BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[at])
                                 : static_cast<const float*>(p.logits)[at];
            // masked: NaN and -inf; +inf counts as the largest finite number; -0 equals 0
            if (x > -INFINITY) {
                const unsigned o = ordered((BF16 ? x : fminf(x, FLT_MAX)) + 0.0f);
                key[i] = BF16 ? (o & 0xFFFF0000u) | (0xFFFFu - static_cast<unsigned>(e)) : o;
            }
        }
    }
}

template <bool BF16>
__device__ __forceinline__ float key_value(unsigned key) {
    // (a negative BF16's ordered bits are complemented, so its low half reads back as ones)
    const unsigned o = BF16 ? (key & 0x80000000u ? key & 0xFFFF0000u : key | 0x0000FFFFu) : key;
    return fminf(unordered(o), FLT_MAX);
}

template <int VPL, bool BF16>
__device__ __forceinline__ void route_token(const RouteParams& p, int t, int lane, unsigned (&key)[VPL], int* sid) {
    constexpr bool SORTED = BF16 && VPL <= 8;
    if constexpr (SORTED) {     // odd-even merge sort, largest first
#pragma unroll
        for (int p2 = 1; p2 < VPL; p2 *= 2)
#pragma unroll
            for (int d = p2; d >= 1; d /= 2)
#pragma unroll
                for (int j = d % p2; j + d < VPL; j += 2 * d)
#pragma unroll
                    for (int i = 0; i < d; ++i)
                        if (i + j + d < VPL && (i + j) / (2 * p2) == (i + j + d) / (2 * p2)) {
                            const unsigned hi = max(key[i + j], key[i + j + d]), lo = min(key[i + j], key[i + j + d]);
                            key[i + j] = hi;
                            key[i + j + d] = lo;
                        }
    }
    // this lane's largest key and, for FP32, its slot (the first of equals); no branches, so
    // that a round costs little more than its reduction
    unsigned best;
    int best_i = 0;
    auto scan = [&]() {
        best = key[0];
        best_i = 0;
        if (SORTED) return;
#pragma unroll
        for (int i = 1; i < VPL; ++i) {
            if (!BF16) best_i = key[i] > best ? i : best_i;
            best = max(best, key[i]);
        }
    };
    scan();
    const unsigned top = __reduce_max_sync(0xffffffffu, best);
    const float xmax = key_value<BF16>(top);
    float total = 0.0f;
    if (!p.renorm) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i]) total += expf(key_value<BF16>(key[i]) - xmax);
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    int my_id = -1;             // lane j keeps the j-th choice
    unsigned my_key = 0;
    for (int j = 0; j < p.k; ++j) {
        const unsigned m = j == 0 ? top : __reduce_max_sync(0xffffffffu, best);
        if (m == 0) break;      // nothing unmasked is left
        int e;
        if constexpr (BF16) {
            e = static_cast<int>(0xFFFFu - (m & 0xFFFFu));
        } else {
            const unsigned who = __ballot_sync(0xffffffffu, best == m);
            const int mine = lane + 32 * best_i;
            e = (who & (who - 1)) == 0
                    ? __shfl_sync(0xffffffffu, mine, __ffs(who) - 1)
                    : static_cast<int>(__reduce_min_sync(0xffffffffu, best == m ? static_cast<unsigned>(mine) : 0xffffffffu));
        }
        my_id = lane == j ? e : my_id;
        my_key = lane == j ? m : my_key;
        if constexpr (SORTED) {
            const bool won = key[0] == m;
#pragma unroll
            for (int i = 0; i < VPL; ++i) key[i] = won ? (i + 1 < VPL ? key[i + 1] : 0) : key[i];
        } else {
#pragma unroll
            for (int i = 0; i < VPL; ++i) key[i] = (BF16 ? key[i] == m : lane + 32 * i == e) ? 0 : key[i];
        }
        scan();
    }
    float my_p = my_id >= 0 ? expf(key_value<BF16>(my_key) - xmax) : 0.0f;
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

// Selects the experts of one chunk of tokens and counts them. A call of one chunk is
// placed here as well: one launch.
template <int VPL, bool BF16>
__global__ void __launch_bounds__(VPL <= 8 ? 1024 : 512, VPL <= 8 ? 2 : 1) route_select(const RouteParams p) {
    extern __shared__ __align__(16) unsigned long long mask[];            // [E]
    int* total = reinterpret_cast<int*>(mask + p.E);        // [E] (one chunk)
    int* sid = total + p.E;                                 // [CHUNK][k]
    dg::grid_dependency_wait();
    if (threadIdx.x == 0) dg::grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int t0 = blockIdx.x * p.chunk, n = min(p.chunk, p.T - t0);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) mask[e] = 0;
    __syncthreads();
    for (int i = warp; i < n; i += warps) {
        unsigned key[VPL];
        load_keys<VPL, BF16>(p, t0 + i, lane, key);
        route_token<VPL, BF16>(p, t0 + i, lane, key, sid + i * p.k);
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
    for (int i = threadIdx.x; i < n * p.k; i += blockDim.x) {
        const int e = sid[i], tok = i / p.k;
        int row = -1;
        if (e >= 0) {
            row = total[e] + __popcll(mask[e] & ((1ull << tok) - 1));
            p.row_token[row] = tok;
        }
        p.slot_row[i] = row;
        if (i >= all) p.row_token[i] = -1;
    }
}

// Rows of one chunk's pairs: every CTA sums the counts of the chunks before its own
// and of all chunks (four experts a load, a thread's loads in flight together), scans
// the totals over the experts, and places its pairs.
constexpr int PLACE_THREADS = dg::route::kPlaceThreads;
constexpr int PLACE_PAIRS = CHUNK * DGEMM_MAX_TOPK / PLACE_THREADS;   // pairs of one thread, at most

__global__ void __launch_bounds__(PLACE_THREADS, 2) route_place(const RouteParams p) {
    extern __shared__ __align__(16) unsigned long long mask[];            // [pitch]
    const dg::route::PlaceLayout layout(p.E);
    char* const smem = reinterpret_cast<char*>(mask);
    int* before = reinterpret_cast<int*>(smem + layout.before);   // [parts][pitch] pairs of e in earlier chunks
    int* base = reinterpret_cast<int*>(smem + layout.base);       // [parts][pitch] pairs of e; then first row of e
    const int quads = p.pitch / 4, parts = layout.parts;
    dg::grid_dependency_wait();
    if (threadIdx.x == 0) dg::grid_launch_dependents();
    const int mine = static_cast<int>(blockIdx.x);
    const int t0 = mine * p.chunk, pairs = min(p.chunk, p.T - t0) * p.k;
    int id[PLACE_PAIRS];
#pragma unroll
    for (int i = 0; i < PLACE_PAIRS; ++i) {
        const int at = threadIdx.x + i * PLACE_THREADS;
        id[i] = at < pairs ? p.ids[static_cast<int64_t>(t0) * p.k + at] : -1;
    }
    for (int e = threadIdx.x; e < p.E; e += PLACE_THREADS) mask[e] = 0;
    const int quad = threadIdx.x % quads, part = threadIdx.x / quads;
    if (part < parts) {
        // two 16-bit sums in a word: at most 512 counts of up to CHUNK each between foldings
        int sum[4] = {0, 0, 0, 0}, pre[4] = {0, 0, 0, 0};
        for (int c0 = part; c0 < p.chunks; c0 += 512 * parts) {
            const int c1 = static_cast<int>(min(static_cast<int64_t>(p.chunks), c0 + static_cast<int64_t>(512) * parts));
            uint32_t s02 = 0, s13 = 0, p02 = 0, p13 = 0;
            const uint8_t* at = p.counts + static_cast<int64_t>(c0) * p.pitch + quad * 4;
            const int64_t step = static_cast<int64_t>(parts) * p.pitch;
#pragma unroll 8
            for (int c = c0; c < c1; c += parts, at += step) {
                const uint32_t v = *reinterpret_cast<const uint32_t*>(at);
                const uint32_t a = v & 0x00FF00FFu, b = (v >> 8) & 0x00FF00FFu;
                s02 += a;
                s13 += b;
                p02 += c < mine ? a : 0;
                p13 += c < mine ? b : 0;
            }
            sum[0] += s02 & 0xFFFF, sum[2] += s02 >> 16, sum[1] += s13 & 0xFFFF, sum[3] += s13 >> 16;
            pre[0] += p02 & 0xFFFF, pre[2] += p02 >> 16, pre[1] += p13 & 0xFFFF, pre[3] += p13 >> 16;
        }
        *reinterpret_cast<int4*>(base + part * p.pitch + quad * 4) = make_int4(sum[0], sum[1], sum[2], sum[3]);
        *reinterpret_cast<int4*>(before + part * p.pitch + quad * 4) = make_int4(pre[0], pre[1], pre[2], pre[3]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PLACE_PAIRS; ++i)
        if (id[i] >= 0) atomicOr(&mask[id[i]], 1ull << ((threadIdx.x + i * PLACE_THREADS) / p.k));
    for (int e = threadIdx.x; e < p.E; e += PLACE_THREADS) {
        int s = base[e], b = before[e];
        for (int q = 1; q < parts; ++q) {
            s += base[q * p.pitch + e];
            b += before[q * p.pitch + e];
        }
        base[e] = s;
        before[e] = b;
    }
    __syncthreads();
    const int all = scan_experts(base, p.E);
    if (mine == 0) {
        for (int e = threadIdx.x; e < p.E; e += PLACE_THREADS) p.offsets[e] = base[e];
        if (threadIdx.x == 0) p.offsets[p.E] = all;
    }
#pragma unroll
    for (int i = 0; i < PLACE_PAIRS; ++i) {
        const int pair = threadIdx.x + i * PLACE_THREADS;
        if (pair >= pairs) continue;
        const int64_t at = static_cast<int64_t>(t0) * p.k + pair;
        const int e = id[i], tok = pair / p.k;
        int row = -1;
        if (e >= 0) {
            row = base[e] + before[e] + __popcll(mask[e] & ((1ull << tok) - 1));
            p.row_token[row] = t0 + tok;
        }
        p.slot_row[at] = row;
        if (at >= all) p.row_token[at] = -1;
    }
}

dgemm_status_t route_sizes(int64_t T, int64_t E, int k) {
    if (T < 0 || E < 1 || k < 1 || k > E) return DGEMM_ERR_INVALID_VALUE;
    if (E > DGEMM_MAX_EXPERTS || k > DGEMM_MAX_TOPK || T * k >= (int64_t(1) << 30) || T > (int64_t(1) << 30))
        return DGEMM_ERR_NOT_SUPPORTED;
    return DGEMM_OK;
}

template <int VPL>
cudaError_t launch_select(const RouteParams& p, cudaStream_t s) {
    // a warp per token as far as registers allow (two CTAs an SM up to 256 experts), and
    // threads enough for the per-expert steps
    const int most = VPL <= 8 ? 32 : 16, warps = std::max(std::min(most, p.chunk), std::min(most, (p.E + 31) / 32));
    dg::host::Launch l(static_cast<unsigned>(p.chunks), 1, 32u * warps, static_cast<size_t>(p.E) * 12 + CHUNK * p.k * 4, s);
    return p.bf16 ? cudaLaunchKernelEx(&l.cfg, route_select<VPL, true>, p)
                  : cudaLaunchKernelEx(&l.cfg, route_select<VPL, false>, p);
}

}  // namespace

extern "C" size_t dgemm_route_workspace_size(int64_t T, int64_t E, int k) {
    if (route_sizes(T, E, k) != DGEMM_OK) return 0;
    const size_t chunks = static_cast<size_t>((T + CHUNK - 1) / CHUNK) + kMoreChunks;
    return T > CHUNK ? DGEMM_WS_STATUS_BYTES + chunks * static_cast<size_t>(dg::route::pitch_of(static_cast<int>(E))) : 0;
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
    // behind the status word, where a call given the same workspace may have left a record
    p.counts = need > 0 ? static_cast<uint8_t*>(ws) + DGEMM_WS_STATUS_BYTES : nullptr;
    p.pitch = dg::route::pitch_of(p.E);
    // As many chunks as fill the last wave of two CTAs an SM, at most kMoreChunks more.
    const int64_t fewest = (T + CHUNK - 1) / CHUNK, wave = 2 * dev.num_sms;
    const int64_t want = T <= CHUNK ? 1 : std::min((fewest + wave - 1) / wave * wave, fewest + kMoreChunks);
    p.chunk = static_cast<int>((T + want - 1) / want);
    p.chunks = static_cast<int>((T + p.chunk - 1) / p.chunk);
    cudaError_t e;
    if (E <= 64) e = launch_select<2>(p, s);
    else if (E <= 128) e = launch_select<4>(p, s);
    else if (E <= 256) e = launch_select<8>(p, s);
    else if (E <= 512) e = launch_select<16>(p, s);
    else e = launch_select<32>(p, s);
    if (e != cudaSuccess) return DGEMM_ERR_CUDA;
    if (p.chunks == 1) return DGEMM_OK;
    dg::host::Launch l(static_cast<unsigned>(p.chunks), 1, PLACE_THREADS, dg::route::PlaceLayout(p.E).bytes, s);
    return cudaLaunchKernelEx(&l.cfg, route_place, p) == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
}
