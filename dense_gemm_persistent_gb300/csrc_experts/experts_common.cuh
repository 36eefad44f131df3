// experts_common.cuh -- what the expert products' kernels share: parameters, the
// tile schedule built from device-side group offsets, and the epilogue.
//
// The kernels compute D^T: the output channels run over the 128 rows of the MMA
// (256 for a CTA pair) and a group's token rows over its columns. The MMA's
// column count is an operand of each instruction, so a ragged group of c rows
// costs ceil(c / 16) x 16 columns (x 32 for a pair) instead of whole tiles of 128 rows.
#pragma once

#include <cuda_bf16.h>

#include "dgemm_experts.h"
#include "gemm_kernel.cuh"

namespace dg {
namespace experts {

struct Params {
    const int* offsets;          // [E+1], or null: one group of R rows
    const int* a_rows;           // [R], or null
    const void* A;               // gathered or converted rows: [a_count][K]
    const float* a_scale;        // [a_count], or null
    const float* b_scale;        // [E][N], or null
    const float* bias;           // [E][N], or null
    const void* C;               // [R][wide], or null
    void* D;                     // [R][wide]
    int E, R, N, K, a_count;
    int wide;                    // columns of D: N, or N / 2 when gated
    int gated, act, d_f32, c_f32;
    int ctiles;                  // channel tiles of an expert
    int kstages;                 // pipeline stages of one tile
    int k_whole;                 // 1: K is whole 128-byte slices (two of them in one copy)
    float alpha, beta;
    unsigned* status;
    unsigned long long* ws_status;
    unsigned long long epoch;
    uint64_t wait_ns;
    long long stall_after;       // testing the bounded waits (< 0: off)
};

constexpr unsigned kAllLanes = 0xffffffffu;

// Error bits in the workspace's status word (tagged with the launch epoch), else in the per-device
// word: the format that record_error of gemm_kernel.cuh writes and the query reads.
__device__ __forceinline__ void record(const Params& p, unsigned bit) {
    if (p.ws_status != nullptr) {
        unsigned long long old = *reinterpret_cast<volatile unsigned long long*>(p.ws_status);
        for (int tries = 0; tries < 4096; ++tries) {
            const bool mine = (old >> 8) == p.epoch;
            if (mine && (old & bit) == bit) return;
            const unsigned long long next = mine ? (old | bit) : ((p.epoch << 8) | bit);
            const unsigned long long seen = atomicCAS(p.ws_status, old, next);
            if (seen == old) return;
            old = seen;
        }
    }
    atomicOr(p.status, bit);
}

__device__ __forceinline__ void fail(const Params& p, unsigned bit, volatile int* abort) {
    record(p, bit);
    *abort = 1;
}

// ---------------------------------------------------------------- schedule

// The groups that have rows, in order, with the running count of their token
// tiles: [E] first row, [E] end, [E] expert, [E+1] tiles before.
struct Schedule {
    int* lo;
    int* hi;
    int* id;
    int* cum;
    int* head;   // [0] groups with rows, [1] token tiles in all
    static __host__ __device__ constexpr size_t bytes(int E) { return (4 * static_cast<size_t>(E) + 4) * 4; }
    __device__ Schedule(void* mem, int E) {
        int* m = static_cast<int*>(mem);
        head = m;
        lo = m + 2;
        hi = lo + E;
        id = hi + E;
        cum = id + E;
    }
};

// Run by one whole warp. Offsets are clamped into [0, R].
template <int BN>
__device__ __forceinline__ void build_schedule(const Params& p, const Schedule& s) {
    const int lane = threadIdx.x & 31;
    int groups = 0, tiles = 0;
#pragma unroll 4
    for (int base = 0; base < p.E; base += 32) {
        const int e = base + lane;
        int lo = 0, hi = 0;
        if (e < p.E) {
            lo = p.offsets ? min(max(p.offsets[e], 0), p.R) : 0;
            hi = p.offsets ? min(max(p.offsets[e + 1], lo), p.R) : p.R;
        }
        const int mine = (hi - lo + BN - 1) / BN;
        const unsigned live = __ballot_sync(kAllLanes, mine > 0);
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAllLanes, inc, o);
            if (lane >= o) inc += v;
        }
        if (mine > 0) {
            const int at = groups + __popc(live & ((1u << lane) - 1));
            s.lo[at] = lo;
            s.hi[at] = hi;
            s.id[at] = e;
            s.cum[at] = tiles + inc - mine;
        }
        groups += __popc(live);
        tiles += __shfl_sync(kAllLanes, inc, 31);
    }
    if (lane == 0) {
        s.cum[groups] = tiles;
        s.head[0] = groups;
        s.head[1] = tiles;
    }
}

struct Tile {
    int expert;
    int row0, rows;     // token rows
    int chan0;          // first output channel (of D) of the tile
    int n;              // MMA columns: rows rounded up
};

// Walks one role through its unit's tiles (item = unit, unit + units, ...).
// Inside an expert, bands of 8 token tiles: token tiles first, then channels, so
// that units running side by side share weights and token rows in L2.
struct Cursor {
    int group = 0;
    template <int BN, int CTAS>
    __device__ __forceinline__ bool at(const Params& p, const Schedule& s, int item, int tile_channels, Tile& t) {
        constexpr int BAND = 8, Q = 16 * CTAS;
        if (static_cast<int64_t>(item) >= static_cast<int64_t>(s.head[1]) * p.ctiles) return false;
        while (item >= static_cast<int64_t>(s.cum[group + 1]) * p.ctiles) ++group;
        int r = item - s.cum[group] * p.ctiles;
        const int nt = s.cum[group + 1] - s.cum[group];
        const int band = r / (BAND * p.ctiles);
        r -= band * BAND * p.ctiles;
        const int deep = min(BAND, nt - band * BAND);
        const int tt = band * BAND + r % deep;
        const int lo = s.lo[group], hi = s.hi[group];
        // equal tiles: ceil(rows / tiles) rounded up to the MMA's column step
        const int w = ((hi - lo + nt - 1) / nt + Q - 1) / Q * Q;
        t.expert = s.id[group];
        t.row0 = lo + tt * w;
        t.rows = min(w, hi - t.row0);
        t.n = (t.rows + Q - 1) / Q * Q;
        t.chan0 = (r / deep) * tile_channels;
        return true;
    }
};

// ---------------------------------------------------------------- epilogue

__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.0f + __expf(-v)); }
__device__ __forceinline__ float gelu(float v) { return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f)); }
// max(v, 0), NaN kept (fmaxf would answer 0).
__device__ __forceinline__ float relu(float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(0.0f));
    return r;
}

// The switch is taken once for 32 values, so that the per-element code is straight-line.
__device__ __forceinline__ void activate32(float (&v)[32], int act) {
    switch (act) {
        case DGEMM_ACT_RELU:
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = relu(v[j]);
            break;
        case DGEMM_ACT_GELU:
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = gelu(v[j]);
            break;
        case DGEMM_ACT_SILU:
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = silu(v[j]);
            break;
        default:
            break;
    }
}

// Stores one channel's COLS values, one row of D each (lanes: consecutive channels; `at`: this
// lane's first). BF16 rows of even length: neighbouring lanes swap their packed pairs of rows,
// so that a lane stores two channels of one row and the warp two rows at once. The values are
// ready before any store, and the swap is a permute by a constant of the lane: choosing
// between packings cost a divergent branch per pair, 45 % more time for 16384 x 4096 x 256 (50 us).
template <int COLS>
__device__ __forceinline__ void store_columns(const Params& p, int64_t at, const float (&v)[COLS], bool live, int valid) {
    const int64_t wide = p.wide;
    if (p.d_f32) {
        if (!live) return;
        float* d = static_cast<float*>(p.D) + at;
#pragma unroll
        for (int j = 0; j < COLS; ++j, d += wide)
            if (j < valid) *d = v[j];
    } else if ((p.wide & 1) == 0) {
        const int odd = threadIdx.x & 1;
        const uint32_t pick = odd ? 0x3276u : 0x5410u;    // (partner's row j + 1, own), or (own row j, partner's)
        uint32_t w[COLS / 2];
#pragma unroll
        for (int j = 0; j < COLS / 2; ++j) {
            const uint32_t own = pack_bf16x2(v[2 * j], v[2 * j + 1]);
            w[j] = __byte_perm(own, __shfl_xor_sync(kAllLanes, own, 1), pick);
        }
        if (!live) return;                                // (an even row length: both lanes of a pair are live or neither)
        uint32_t* d = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.D) + at - odd + odd * wide);
        if (valid >= COLS) {
#pragma unroll
            for (int j = 0; j < COLS / 2; ++j, d += wide) *d = w[j];
        } else {
#pragma unroll
            for (int j = 0; j < COLS / 2; ++j, d += wide)
                if (2 * j + odd < valid) *d = w[j];
        }
    } else {
        if (!live) return;
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.D) + at;
#pragma unroll
        for (int j = 0; j < COLS; ++j, d += wide)
            if (j < valid) *d = __float2bfloat16_rn(v[j]);
    }
}

// Named barrier of the two warps that exchange gate and up halves; every thread
// learns whether all 64 passed `ok`.
__device__ __forceinline__ bool pair_all(int id, bool ok) {
    unsigned r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<unsigned>(ok)), "r"(id)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }

// Bytes of the gate / up exchange: 16 columns x 32 lanes FP32 each way for each
// pair of epilogue warps.
template <int EPI_WARPS>
__host__ __device__ constexpr int exchange_bytes() { return EPI_WARPS / 2 * 2 * 16 * 32 * 4; }

// The epilogue of one tile by one of EPI_WARPS warps (ew = 0 ..): warp quarter
// ew % 4 reads its 32 accumulator lanes (channels), the warps of a quarter share
// the columns (token rows) in chunks of 32. A gated tile has 64 gate channels
// in lanes 0-63 and their up channels in lanes 64-127: the two warps of a
// channel swap 16 columns each through shared memory, so both do half of the products.
//   acc      TMEM address of the accumulator (lane 0)
//   ready()  waits for it; released() hands it back after the last read
template <int EPI_WARPS, class Ready, class Released>
__device__ __forceinline__ bool tile_epilogue(const Params& p, const Tile& t, uint32_t acc, int ew, int cta_chan0,
                                              float* exchange, Ready ready, Released released) {
    constexpr int COLS = EPI_WARPS / 4;                      // warps that share a lane quarter
    const int lane = threadIdx.x & 31, q = ew & 3, part = ew >> 2;
    const int i = q * 32 + lane;                             // accumulator lane
    const int ch = cta_chan0 + (p.gated ? (i & 63) : i);     // channel of D
    const bool live = ch < p.wide;
    const int n = p.gated && i >= 64 ? p.N / 2 + ch : ch;    // channel of B
    const int64_t en = static_cast<int64_t>(t.expert) * p.N + n;
    float bs = p.alpha, bias = 0.0f;
    if (live) {
        if (p.b_scale) bs *= __ldg(p.b_scale + en);
        if (p.bias) bias = __ldg(p.bias + en);
    }
    // lane j: the scale of column j of a chunk
    auto column_scale = [&](int c) {
        const int col = (c * COLS + part) * 32 + lane;
        if (!p.a_scale || col >= t.rows) return 0.0f;
        const int a = p.a_rows ? __ldg(p.a_rows + t.row0 + col) : t.row0 + col;
        return a >= 0 && a < p.a_count ? __ldg(p.a_scale + a) : 0.0f;
    };
    float as_next = column_scale(0);
    bool ok = ready();
    const int swap_id = 1 + part * 2 + (q & 1);              // barrier of warps q and q ^ 2
    if (p.gated) ok = pair_all(swap_id, ok);
    if (!ok) return false;
    tc_fence_after();
    float* mine = exchange + ((part * 2 + (q & 1)) * 2 + (q >> 1)) * 512;
    const float* theirs = exchange + ((part * 2 + (q & 1)) * 2 + ((q >> 1) ^ 1)) * 512;
    const int chunks = (t.rows + 31) / 32;
    // The accumulator goes back once its last columns are in registers (a relaxed
    // arrive: its reads have completed, and the stores to come need no ordering).
    auto hand_back = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) released();
    };
    if (part >= chunks) hand_back();
    // (one copy of the loop's code: unrolled, it pushed the other warps' loops out of the
    // instruction cache)
#pragma unroll 1
    for (int c = 0; c * COLS + part < chunks; ++c) {
        const int col0 = (c * COLS + part) * 32;
        const float as = as_next;
        as_next = column_scale(c + 1);
        uint32_t r[32];
        tmem_ld32(acc + (static_cast<uint32_t>(q * 32) << 16) + col0, r);
        tmem_ld_wait();
        if ((c + 1) * COLS + part >= chunks) hand_back();
        float v[32];
        if (p.kstages == 0) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = bias;
        } else if (p.a_scale) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                v[j] = fmaf(__uint_as_float(r[j]), bs * __shfl_sync(kAllLanes, as, j), bias);
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = fmaf(__uint_as_float(r[j]), bs, bias);
        }
        const int64_t at = static_cast<int64_t>(t.row0 + col0) * p.wide + ch;
        const int valid = t.rows - col0;
        if (p.gated) {
            // gate warps keep columns 0-15 and get up's; up warps keep 16-31 and get the gate's
            const bool up = q >= 2;
            if (c > 0) pair_sync(swap_id);                   // the other warp has read the last chunk
#pragma unroll
            for (int j = 0; j < 16; ++j) mine[j * 32 + lane] = up ? v[j] : v[16 + j];
            pair_sync(swap_id);
            float y[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float x = theirs[j * 32 + lane];
                y[j] = up ? silu(x) * v[16 + j] : silu(v[j]) * x;
            }
            const int skip = up ? 16 : 0;
            store_columns<16>(p, at + static_cast<int64_t>(skip) * p.wide, y, live, valid - skip);
        } else {
            if (p.C && live) {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (j >= valid) continue;
                    const int64_t o = at + static_cast<int64_t>(j) * p.wide;
                    const float x = p.c_f32 ? static_cast<const float*>(p.C)[o]
                                            : __bfloat162float(static_cast<const __nv_bfloat16*>(p.C)[o]);
                    v[j] = fmaf(p.beta, x, v[j]);
                }
            }
            activate32(v, p.act);
            store_columns<32>(p, at, v, live, valid);
        }
    }
    if (p.gated && part < chunks) pair_sync(swap_id);        // before the next tile's first write
    return true;
}

}  // namespace experts
}  // namespace dg
