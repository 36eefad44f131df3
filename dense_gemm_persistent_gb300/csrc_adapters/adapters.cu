// adapters.cu -- low-rank adapters of many requests, host side: checks, the choice of
// a form, tensor maps and launches.
#include <algorithm>
#include <atomic>
#include <cstring>

#include "adapter_beside.cuh"
#include "adapter_few.cuh"
#include "adapter_forms.h"
#include "adapter_mma.cuh"
#include "adapter_shrink.cuh"
#include "host.h"

namespace {

using dg::adapters::Few;
using dg::adapters::Mma;
using dg::adapters::Params;
using dg::adapters::Shrink;

constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
constexpr int kShared = 232448;                   // a CTA's dynamic shared memory, at most

// Behind the workspace's status word.
struct Workspace {
    size_t lists, bytes;
    Workspace(int64_t T, int64_t r) {
        lists = DGEMM_WS_STATUS_BYTES + static_cast<size_t>(T) * static_cast<size_t>(r) * 4;
        bytes = lists + static_cast<size_t>((T + Mma::LEAST_WIDTH - 1) / Mma::LEAST_WIDTH) * dg::adapters::kListPitch * 4;
    }
};

struct Call {
    const void *X, *W, *A, *B;
    const int32_t* ids;
    const float* scale;
    int64_t L, r;
    const void* C;
    dgemm_dtype_t c_dtype;
    void* D;
    dgemm_dtype_t d_dtype;
    int64_t T, N, K;
    const float* bias;
    int act;
    void* ws;
    size_t ws_bytes;
    cudaStream_t stream;
};

// V by FP32 units, every row on its own, or by the tensor core, whose launch has a longer way to its first number. FP32 / tensor
// core in us a call of 4096 channels, every row another adapter of 32 (and one request after another): K = 4096, 256
// rows of rank 64 43 / 74 (40 / 50); 512 of rank 16 49 / 57 (43 / 40), of rank 64 78 / 92 (70 / 57); 1024 of rank 16
// 64 / 64 (58 / 47); K = 1024, 1024 rows of rank 16 37 / 42 (29 / 29), of rank 64 61 / 69 (50 / 39). Beside 11008
// channels, 4096 rows of K = 256 and rank 32: 94 / 61 (a CTA for every 8 numbers is too many).
bool few_for_v(int64_t T, int64_t r, int64_t K) { return T <= 256 || (T <= 1024 && T * r * K <= (int64_t(1) << 25)); }

dgemm_status_t check_sizes(int64_t T, int64_t N, int64_t K, int64_t r, int64_t L) {
    if (T < 0 || N < 0 || K < 0 || L < 0 || r < 1) return DGEMM_ERR_INVALID_VALUE;
    if (L > DGEMM_MAX_ADAPTERS || r > DGEMM_MAX_ADAPTER_RANK) return DGEMM_ERR_NOT_SUPPORTED;
    if (T > (int64_t(1) << 24) || N > INT32_MAX / 2 || K > INT32_MAX / 2) return DGEMM_ERR_NOT_SUPPORTED;
    if (r % 8 != 0 || K % 8 != 0) return DGEMM_ERR_MISALIGNED;
    return DGEMM_OK;
}

// A kernel's limit of dynamic shared memory, set once per device.
bool allow_shared(std::atomic<unsigned char>* ready, int device, const void* func, int bytes) {
    if (ready[device].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
        cudaFuncSetAttribute(func, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) != cudaSuccess)
        return false;
    ready[device].store(1, std::memory_order_release);
    return true;
}

// V of few rows: a CTA for some of a row's numbers.
template <int RB, int U, int THREADS>
cudaError_t shrink_few(const Params& p, const dg::host::Device& dev, cudaStream_t s) {
    // The same split of an SM's memory as the kernel behind it: one of another split does not start on an SM
    // before this one has left it.
    static std::atomic<unsigned char> ready[dg::host::kMaxDevices];
    const auto kernel = dg::adapters::adapter_shrink_few<RB, U, THREADS>;
    if (!allow_shared(ready, dev.id, reinterpret_cast<const void*>(kernel), 0)) return cudaErrorUnknown;
    const unsigned blocks = static_cast<unsigned>(p.T) * (p.r / RB) + (p.prompt ? p.tiles : 0);
    dg::host::Launch l(blocks, 1, THREADS, 0, s);
    return cudaLaunchKernelEx(&l.cfg, kernel, p);
}
// As many CTAs as the SMs hold at once, about 4 each: more numbers a CTA beyond. 256 threads share K, 128 where one batch of
// theirs (two loads of 8 numbers) is all of it, up to 2048: more threads would leave half of a batch empty. 128 / 256 threads in
// us a call: K = 512, 1024, 2048, 2560, 4096; 64 rows of rank 64, 4096 channels 29.9 / 31.0, 25.2 / 26.5, 21.9 / 22.6, 25.2 /
// 24.6, 27.7 / 26.7; 512 rows of rank 32, 2048 channels 19.6 / 24.5, 21.2 / 25.9, 22.4 / 28.4, 26.6 / 26.6, 33.6 / 33.4.
// (997 rows of rank 8, in long runs, would take 128 beyond too: 4096 33.0 / 37.7.)
template <int THREADS>
cudaError_t shrink_few(const Params& p, const dg::host::Device& dev, cudaStream_t s) {
    const int64_t numbers = static_cast<int64_t>(p.T) * p.r, at_once = 4 * dev.num_sms;
    return numbers <= 2 * at_once   ? shrink_few<2, 4, THREADS>(p, dev, s)
           : numbers <= 4 * at_once ? shrink_few<4, 2, THREADS>(p, dev, s)
                                    : shrink_few<8, 2, THREADS>(p, dev, s);
}
dgemm_status_t launch_shrink_few(const Params& p, const dg::host::Device& dev, cudaStream_t s) {
    const cudaError_t e = p.K <= 2048 ? shrink_few<128>(p, dev, s) : shrink_few<256>(p, dev, s);
    return e == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
}

dgemm_status_t launch_shrink_many(const Call& c, Params p, const dg::host::Device& dev) {
    p.shrink_tiles = (p.T + Shrink::ROWS - 1) / Shrink::ROWS;
    p.kstages = (p.K + Shrink::KS * Shrink::SL - 1) / (Shrink::KS * Shrink::SL);
    p.shrink_cols = std::min(Shrink::MOST_COLS / p.r, std::min(p.L, Shrink::ROWS)) * p.r;
    p.split = 1;
    while (p.split < Shrink::MOST_SPLIT && p.shrink_tiles * p.split * 2 <= dev.num_sms && p.kstages >= 4 * p.split) p.split *= 2;
    // (two stages always fit: a tile's 256 columns or less, and 128 numbers of its rows, 193 + 64 KB with rank 128, do not)
    while (Shrink::smem_bytes(p.shrink_cols, 2, p.r) > kShared) p.shrink_cols -= p.r;
    p.stages = 2;
    while (p.stages < Shrink::MOST_STAGES && Shrink::smem_bytes(p.shrink_cols, p.stages + 1, p.r) <= kShared) ++p.stages;
    const int smem = Shrink::smem_bytes(p.shrink_cols, p.stages, p.r);
    alignas(64) CUtensorMap x, a;
    const uint64_t K = p.K, r = p.r, T = p.T, sl = Shrink::SL;
    const uint64_t da[3] = {K, r, static_cast<uint64_t>(p.L)}, sa[2] = {K * 2, r * K * 2};
    const uint32_t ba[3] = {Shrink::SL, static_cast<uint32_t>(p.r), 1};
    bool ok;
    if (p.k_whole) {                              // a stage's slices in one copy
        const uint64_t d[3] = {sl, T, K / sl}, st[2] = {K * 2, 128};
        const uint32_t b[3] = {Shrink::SL, Shrink::ROWS, Shrink::KS};
        ok = dg::host::encode_map(&x, kBf16, c.X, 3, d, st, b);
    } else {
        const uint64_t d[2] = {K, T}, st[1] = {K * 2};
        const uint32_t b[2] = {Shrink::SL, Shrink::ROWS};
        ok = dg::host::encode_map(&x, kBf16, c.X, 2, d, st, b);
    }
    if (!ok || !dg::host::encode_map(&a, kBf16, c.A, 3, da, sa, ba)) return DGEMM_ERR_CUDA;
    static std::atomic<unsigned char> ready[dg::host::kMaxDevices];
    if (!allow_shared(ready, dev.id, reinterpret_cast<const void*>(&dg::adapters::adapter_shrink_many), kShared))
        return DGEMM_ERR_CUDA;
    dg::host::Launch l(static_cast<unsigned>(p.shrink_tiles * p.split), 1, Shrink::THREADS, smem, c.stream, p.split);
    return cudaLaunchKernelEx(&l.cfg, dg::adapters::adapter_shrink_many, x, a, p) == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
}

// The maps of X (boxes of `rows` token rows) and W (boxes of `chan` channels of D): with whole slices of K both slices
// of a stage (and the gate and up channels of a gated tile) come in one copy.
bool product_maps(const Call& c, const Params& p, CUtensorMap* w, CUtensorMap* x, int rows, int chan) {
    const uint64_t N = p.N, K = p.K, T = p.T, sl = Few::SL, halves = p.gated ? 2 : 1, H = N / halves;
    const uint32_t s = Few::SL, channels = chan, hv = static_cast<uint32_t>(halves), cols = rows, ks = Few::KS;
    if (p.k_whole) {
        const uint64_t dw[4] = {sl, H, halves, K / sl}, sw[3] = {K * 2, H * K * 2, 128};
        const uint32_t bw[4] = {s, channels, hv, ks};
        const uint64_t dx[3] = {sl, T, K / sl}, sx[2] = {K * 2, 128};
        const uint32_t bx[3] = {s, cols, ks};
        return dg::host::encode_map(w, kBf16, c.W, 4, dw, sw, bw) && dg::host::encode_map(x, kBf16, c.X, 3, dx, sx, bx);
    }
    const uint64_t dw[3] = {K, H, halves}, sw[2] = {K * 2, H * K * 2};
    const uint32_t bw[3] = {s, channels, hv};
    const uint64_t dx[2] = {K, T}, sx[1] = {K * 2};
    const uint32_t bx[2] = {s, cols};
    return dg::host::encode_map(w, kBf16, c.W, 3, dw, sw, bw) && dg::host::encode_map(x, kBf16, c.X, 2, dx, sx, bx);
}

// Clusters of `split` CTAs of the few-row form that the device holds at once (a cluster lies within one part of it).
int most_clusters(const dg::host::Device& dev, int split) {
    static std::atomic<int> known[dg::host::kMaxDevices][Few::MOST_SPLIT + 1];
    std::atomic<int>& n = known[dev.id][split];
    int v = n.load(std::memory_order_acquire);
    if (v == 0) {
        dg::host::Launch l(static_cast<unsigned>(dev.num_sms / split * split), 1, Few::THREADS, kShared, nullptr, split);
        l.cfg.attrs = l.attr + 1;                 // (the cluster's size alone)
        l.cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&v, reinterpret_cast<const void*>(&dg::adapters::adapter_few), &l.cfg) != cudaSuccess || v < 1) {
            cudaGetLastError();
            v = -1;
        }
        n.store(v, std::memory_order_release);
    }
    return v;
}

dgemm_status_t launch_few(const Call& c, Params& p, const dg::host::Device& dev) {
    static std::atomic<unsigned char> ready[dg::host::kMaxDevices];
    if (!allow_shared(ready, dev.id, reinterpret_cast<const void*>(&dg::adapters::adapter_few), kShared)) return DGEMM_ERR_CUDA;
    const int full = p.gated ? 64 : 128, ctiles = (p.wide + full - 1) / full;
    // Rows of a tile: beside a product up to 64, which share the weights; else as many as leave a CTA for every SM.
    int most = Few::MOST_COLS;
    if (p.kstages == 0)
        for (most = 16; most < Few::MOST_COLS && static_cast<int64_t>((p.T + most - 1) / most) * ctiles > dev.num_sms;) most += 16;
    const int fewest = (p.T + most - 1) / most;
    p.width = ((p.T + fewest - 1) / fewest + 15) / 16 * 16;
    p.tiles = (p.T + p.width - 1) / p.width;
    if (static_cast<int64_t>(p.tiles) * ctiles > INT32_MAX / Few::MOST_SPLIT / 2) return DGEMM_ERR_NOT_SUPPORTED;
    // CTAs of a cluster that share K, and channels of a tile: the least time by a model of what a CTA reads (rows of W
    // and X times its stages, in waves of the clusters that fit at once), a wave's ends as 1000 such units of about 4 ns, the
    // exchange of parts as 150.
    // (K = 4096: 11008 channels 138 CTAs of 80, not 86 of 128; 4096 channels 35 clusters of 4 CTAs, 120 channels and a quarter of K.)
    int64_t least = INT64_MAX;
    for (int split = 1; split <= Few::MOST_SPLIT && (split == 1 || p.kstages >= 4 * split); split *= 2) {
        const int slots = split == 1 ? dev.num_sms : most_clusters(dev, split);
        if (slots < 1) break;
        const int waves = (p.tiles * ctiles + slots - 1) / slots;
        const int channels = std::min(full, (p.wide / std::max(1, waves * slots / p.tiles) + 8) / 8 * 8);
        const int64_t stages = (p.kstages + split - 1) / split;
        const int64_t cost = waves * ((channels * (p.gated ? 2 : 1) + p.width) * stages + 1000 + (split > 1 ? 150 : 0));
        if (cost < least) {
            least = cost;
            p.split = split;
            p.channels = channels;
        }
    }
    p.ctiles = (p.wide + p.channels - 1) / p.channels;
    const int64_t tiles = static_cast<int64_t>(p.tiles) * p.ctiles;
    p.ahead = p.L > 0 ? Few::items_ahead(p.r, p.kstages > 0) : 0;
    auto shared = [&](int stages) { return Few::smem_bytes(p.width, stages, p.split, p.r, p.ahead); };
    p.stages = p.kstages > 0 ? 2 : 0;
    while (p.stages > 0 && p.stages < Few::MOST_STAGES && shared(p.stages + 1) <= kShared) ++p.stages;
    const int smem = shared(p.stages);            // (two stages always fit: Few::most_bytes)
    alignas(64) CUtensorMap w, x;
    std::memset(&w, 0, sizeof w);
    std::memset(&x, 0, sizeof x);
    if (p.kstages > 0 && !product_maps(c, p, &w, &x, p.width, p.channels)) return DGEMM_ERR_CUDA;
    dg::host::Launch l(static_cast<unsigned>(tiles * p.split), 1, Few::THREADS, smem, c.stream, p.split);
    return cudaLaunchKernelEx(&l.cfg, dg::adapters::adapter_few, w, x, p) == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
}

// The token tiles of the prompt form: their width is the one with the least time by a model of waves of tiles, a tile's
// time as its rows, at least 96 (then the weights' way to the SM is longer), and 16 more for its ends.
void prompt_tiles(Params& p, const dg::host::Device& dev) {
    p.ctiles = (p.wide + (p.gated ? 128 : 256) - 1) / (p.gated ? 128 : 256);
    int64_t least = INT64_MAX;
    for (int width = Mma::LEAST_WIDTH; width <= Mma::BN; width += Mma::Q) {
        const int64_t tiles = (p.T + width - 1) / width, units = dev.num_sms / 2;
        const int64_t cost = (tiles * p.ctiles + units - 1) / units * (std::max(width, 96) + 16);
        if (cost <= least) {
            least = cost;
            p.width = width;
            p.tiles = static_cast<int>(tiles);
        }
    }
}

dgemm_status_t launch_prompt(const Call& c, const Params& p, const dg::host::Device& dev) {
    const int64_t items = static_cast<int64_t>(p.tiles) * p.ctiles;
    if (items > INT32_MAX / 2) return DGEMM_ERR_NOT_SUPPORTED;
    alignas(64) CUtensorMap w, x, b;
    std::memset(&w, 0, sizeof w);
    std::memset(&x, 0, sizeof x);
    std::memset(&b, 0, sizeof b);
    if (p.kstages > 0 && !product_maps(c, p, &w, &x, p.width / 2, p.gated ? 64 : 128)) return DGEMM_ERR_CUDA;
    if (p.L > 0) {
        const uint64_t r = p.r, N = p.N, halves = p.gated ? 2 : 1, H = N / halves, L = p.L;
        const uint64_t d[4] = {r, H, halves, L}, st[3] = {r * 2, H * r * 2, N * r * 2};
        const uint32_t box[4] = {Mma::SL, p.gated ? 64u : 128u, static_cast<uint32_t>(halves), 1};
        if (!dg::host::encode_map(&b, kBf16, c.B, 4, d, st, box)) return DGEMM_ERR_CUDA;
    }
    static std::atomic<unsigned char> ready[dg::host::kMaxDevices];
    const void* func = reinterpret_cast<const void*>(&dg::adapters::adapter_mma);
    if (ready[dev.id].load(std::memory_order_acquire) == 0) {
        // a register split that adds up to more than the launch holds would wait forever
        cudaFuncAttributes fa{};
        if (cudaFuncGetAttributes(&fa, func) != cudaSuccess || fa.numRegs < Mma::LAUNCH_REGS) return DGEMM_ERR_CUDA;
    }
    if (!allow_shared(ready, dev.id, func, kShared)) return DGEMM_ERR_CUDA;
    const int units = static_cast<int>(std::min<int64_t>(dev.num_sms / 2, items));
    dg::host::Launch l(static_cast<unsigned>(units * 2), 1, Mma::THREADS, Mma::SMEM, c.stream, 2);
    return cudaLaunchKernelEx(&l.cfg, dg::adapters::adapter_mma, w, x, b, p) == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
}

// Beside a product, BF16 in and out, rows on 16 bytes.
template <bool NARROW>
dgemm_status_t launch_beside(const Call& c, const Params& p, const dg::host::Device& dev) {
    using dg::adapters::Beside;
    if (p.gated) return DGEMM_ERR_NOT_SUPPORTED;          // (D's map has rows of N channels)
    const int64_t items = static_cast<int64_t>(p.tiles) * p.ctiles;
    if (items > INT32_MAX / 2) return DGEMM_ERR_NOT_SUPPORTED;
    const uint64_t N = p.N, T = p.T, r = p.r, L = p.L, d[2] = {N, T}, st[1] = {N * 2};
    const uint32_t box[2] = {Beside::SL, Beside::ROWS};
    alignas(64) CUtensorMap cm, dm, b, v;
    std::memset(&cm, 0, sizeof cm);
    std::memset(&b, 0, sizeof b);
    std::memset(&v, 0, sizeof v);
    bool ok = dg::host::encode_map(&dm, kBf16, c.D, 2, d, st, box) && (!c.C || dg::host::encode_map(&cm, kBf16, c.C, 2, d, st, box));
    if (ok && p.L > 0) {
        const uint64_t db[4] = {r, N, 1, L}, sb[3] = {r * 2, N * r * 2, N * r * 2};
        const uint32_t bb[4] = {Beside::SL, Beside::COLS, 1, 1};
        ok = dg::host::encode_map(&b, kBf16, c.B, 4, db, sb, bb);
        if (NARROW) {                             // a row's numbers of V in one slice
            const uint64_t dv[2] = {2 * r, T}, sv[1] = {r * 4};
            const uint32_t bv[2] = {Beside::SL, Beside::ROWS};
            ok = ok && dg::host::encode_map(&v, kBf16, p.V, 2, dv, sv, bv);
        } else {                                  // [part][row]: both slices of a step in one copy
            const uint64_t dv[3] = {r, T, 2}, sv[2] = {r * 4, r * 2};
            const uint32_t bv[3] = {Beside::SL, Beside::ROWS, 2};
            ok = ok && dg::host::encode_map(&v, kBf16, p.V, 3, dv, sv, bv);
        }
    }
    if (!ok) return DGEMM_ERR_CUDA;
    static std::atomic<unsigned char> ready[dg::host::kMaxDevices];
    if (!allow_shared(ready, dev.id, reinterpret_cast<const void*>(&dg::adapters::adapter_beside<NARROW>), kShared)) return DGEMM_ERR_CUDA;
    const int ctas = static_cast<int>(std::min<int64_t>(dev.num_sms, items));
    dg::host::Launch l(static_cast<unsigned>(ctas), 1, Beside::THREADS, Beside::SMEM, c.stream);
    return cudaLaunchKernelEx(&l.cfg, dg::adapters::adapter_beside<NARROW>, cm, dm, b, v, p) == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
}

dgemm_status_t run_adapters(const Call& c) {
    const dgemm_status_t st = check_sizes(c.T, c.N, c.K, c.r, c.L);
    if (st != DGEMM_OK) return st;
    if (c.act < DGEMM_ACT_NONE || c.act > DGEMM_ACT_SWIGLU) return DGEMM_ERR_INVALID_VALUE;
    if (c.act == DGEMM_ACT_SWIGLU && c.N % 2 != 0) return DGEMM_ERR_INVALID_VALUE;
    if (c.d_dtype != DGEMM_F32 && c.d_dtype != DGEMM_BF16) return DGEMM_ERR_INVALID_VALUE;
    if (c.C && c.c_dtype != DGEMM_F32 && c.c_dtype != DGEMM_BF16) return DGEMM_ERR_INVALID_VALUE;
    if (c.C && c.C == c.D && c.c_dtype != c.d_dtype) return DGEMM_ERR_INVALID_VALUE;
    if (c.T == 0 || c.N == 0) return DGEMM_OK;
    if (!c.D || !c.ids || (c.K > 0 && !c.X) || (c.K > 0 && c.L > 0 && (!c.A || !c.B))) return DGEMM_ERR_INVALID_VALUE;
    if (!dg::host::aligned16(c.X) || !dg::host::aligned16(c.W) || !dg::host::aligned16(c.A) || !dg::host::aligned16(c.B) ||
        !dg::host::aligned16(c.C) || !dg::host::aligned16(c.D) || !dg::host::aligned16(c.ws))
        return DGEMM_ERR_MISALIGNED;
    const uintptr_t natural = reinterpret_cast<uintptr_t>(c.ids) | reinterpret_cast<uintptr_t>(c.scale) |
                              reinterpret_cast<uintptr_t>(c.bias);
    if (natural & 3u) return DGEMM_ERR_MISALIGNED;
    if (!c.ws || c.ws_bytes < dgemm_adapter_workspace_size(c.T, c.N, c.K, c.r, c.L)) return DGEMM_ERR_WORKSPACE_TOO_SMALL;
    dg::host::Device dev;
    const dgemm_status_t ds = dg::host::current_device(&dev);
    if (ds != DGEMM_OK) return ds;

    Params p{};
    p.X = static_cast<const __nv_bfloat16*>(c.X);
    p.low = static_cast<const __nv_bfloat16*>(c.A);
    p.high = static_cast<const __nv_bfloat16*>(c.B);
    p.ids = c.ids;
    p.scale = c.scale;
    const Workspace ws(c.T, c.r);
    p.V = static_cast<char*>(c.ws) + DGEMM_WS_STATUS_BYTES;
    p.lists = reinterpret_cast<int*>(static_cast<char*>(c.ws) + ws.lists);
    p.T = static_cast<int>(c.T);
    p.N = static_cast<int>(c.N);
    p.K = static_cast<int>(c.K);
    p.r = static_cast<int>(c.r);
    p.L = c.K > 0 ? static_cast<int>(c.L) : 0;      // (without K, V is zero)
    p.C = c.C;
    p.c_f32 = c.c_dtype == DGEMM_F32;
    p.D = c.D;
    p.d_f32 = c.d_dtype == DGEMM_F32;
    p.bias = c.bias;
    p.act = c.act;
    p.gated = c.act == DGEMM_ACT_SWIGLU;
    p.wide = p.gated ? p.N / 2 : p.N;
    p.status = dev.status;
    p.epoch = dg::host::next_launch_epoch();
    p.ws_status = static_cast<unsigned long long*>(c.ws);
    dg::host::wait_settings(&p.wait_ns, &p.stall_after);
    p.wait_first = p.L == 0;
    p.k_whole = p.K % Few::SL == 0;
    p.kstages = c.W ? (p.K + Few::KS * Few::SL - 1) / (Few::KS * Few::SL) : 0;
    const int forced = dg::host::pair_override();
    // One wave of the few-row form's tiles, or the prompt form: on the device 128 rows of 4096 channels, every row another
    // adapter of rank 64, 33 against 55 us, 256 rows 47 against 63 (one request: 28, 29), 384 115 against 99; of 11008
    // channels 64 rows 37 against 49, 128 65 against 61 (one request: 48, 31). Beside a product of 11008 channels, rank 32, 200
    // rows of one request after another 49 against 21, every row another of 48 60 against 62; 600 rows 90 and 28, 132 and 114.
    const int full = p.gated ? 64 : 128;
    const int64_t few_tiles = static_cast<int64_t>((p.T + Few::MOST_COLS - 1) / Few::MOST_COLS) * ((p.wide + full - 1) / full);
    p.prompt = forced >= 0 ? forced : few_tiles > dev.num_sms;
    // Beside a product in BF16 whose rows TMA can copy: a form of its own (4096 x 11008 with SiLU, rank 32, 8
    // requests in runs 66 us, in the general one 114; every row another of 48 547 and 407: the mix is not known here).
    const bool beside = dg::adapters::beside_form(p.prompt, c.W != nullptr, p.gated, p.d_f32, c.C && p.c_f32, p.N);
    if (beside) {
        p.width = dg::adapters::Beside::ROWS;
        p.tiles = (p.T + p.width - 1) / p.width;
        p.ctiles = (p.N + dg::adapters::Beside::COLS - 1) / dg::adapters::Beside::COLS;
    } else if (p.prompt) {
        prompt_tiles(p, dev);
    }
    if (p.L > 0) {
        const dgemm_status_t s = few_for_v(p.T, p.r, p.K) ? launch_shrink_few(p, dev, c.stream) : launch_shrink_many(c, p, dev);
        if (s != DGEMM_OK) return s;
    }
    // (three steps on their way or two: see Beside::Steps)
    if (beside) return p.r == 16 || p.r == 32 ? launch_beside<true>(c, p, dev) : launch_beside<false>(c, p, dev);
    return p.prompt ? launch_prompt(c, p, dev) : launch_few(c, p, dev);
}

}  // namespace

extern "C" {

size_t dgemm_adapter_workspace_size(int64_t T, int64_t N, int64_t K, int64_t r, int64_t L) {
    if (check_sizes(T, N, K, r, L) != DGEMM_OK) return 0;
    return Workspace(T, r).bytes;
}

dgemm_status_t dgemm_adapter_bf16(const void* X, const void* W, const void* A, const void* B, const int32_t* ids,
                                  const float* scale, int64_t L, int64_t r, void* D, dgemm_dtype_t d_dtype, int64_t T,
                                  int64_t N, int64_t K, const float* bias, int act, void* ws, size_t ws_bytes,
                                  dgemm_stream_t stream) {
    if (!W && T > 0 && N > 0 && K > 0) return DGEMM_ERR_INVALID_VALUE;
    return run_adapters(Call{X, K > 0 ? W : nullptr, A, B, ids, scale, L, r, nullptr, DGEMM_F32, D, d_dtype, T, N, K, bias, act, ws,
                             ws_bytes, reinterpret_cast<cudaStream_t>(stream)});
}

dgemm_status_t dgemm_adapter_add(const void* X, const void* A, const void* B, const int32_t* ids, const float* scale,
                                 int64_t L, int64_t r, const void* C, dgemm_dtype_t c_dtype, void* D,
                                 dgemm_dtype_t d_dtype, int64_t T, int64_t N, int64_t K, const float* bias, int act,
                                 void* ws, size_t ws_bytes, dgemm_stream_t stream) {
    if (act == DGEMM_ACT_SWIGLU) return DGEMM_ERR_INVALID_VALUE;
    return run_adapters(Call{X, nullptr, A, B, ids, scale, L, r, C, c_dtype, D, d_dtype, T, N, K, bias, act, ws, ws_bytes,
                             reinterpret_cast<cudaStream_t>(stream)});
}

}  // extern "C"
