// adapter_mma.cuh -- the projection with adapters for prompts.
//
// One persistent pair of CTAs per two SMs walks tiles of 256 output channels (the MMA's rows) by
// up to 256 token rows (its columns). The adapters are more K: behind the slices of X and W, the
// sum of a tile goes on, for every adapter a that its rows have, with B_a against the rows'
// V, rows of other requests as zeros. So nothing but V (r numbers a row) is written and read in
// between, and D is rounded once. V = first + second BF16 number (adapter_shrink.cuh): two
// slices against the same slice of B_a.
// Warps of a CTA: 0 TMA producer, 1 MMA issuer and owner of the Tensor Memory, 2-3 idle,
// 4-11 epilogue, 12-19 write the masked rows of V and look at B.
// A zero does not hide a number that is not finite: B_a goes through products with the zeros of other
// requests' rows. So the last warps look at a slice of B_a before it is used, put finite numbers in the
// place of what is not, and the epilogue adds those terms to the rows that they belong to, by FP32
// units: slow, and of these rows only.
#pragma once

#include "adapter_common.cuh"

namespace dg {
namespace adapters {

struct Mma {
    static constexpr int BN = kMostWidth, BN_CTA = BN / 2, LEAST_WIDTH = 64, KS = 2, SL = 64, Q = 32;
    static constexpr int SLICE_W = 128 * 128;
    static constexpr int W_BYTES = KS * SLICE_W, STAGE = W_BYTES + KS * BN_CTA * 128, STAGES = 3;
    static constexpr int EPI_WARP0 = 4, EPI_WARPS = 8, V_WARP0 = 12, V_WARPS = 8, THREADS = 32 * (V_WARP0 + V_WARPS);
    // Registers: the epilogue holds a chunk, the next chunk of C and what it writes; with the launch's 96 a thread it spilled
    // (4096 x 11008 beside another product 155 us, not 109), so the other warpgroups hand some over.
    static constexpr int LAUNCH_REGS = 96, REGS_FIRST = 64, REGS_EPI = 128, REGS_V = 80;
    static_assert(REGS_FIRST + 2 * REGS_EPI + 2 * REGS_V <= 5 * LAUNCH_REGS, "register split exceeds the launch allocation");
    static constexpr int TMEM_COLS = 512, BAR_BYTES = 1024;
    static constexpr int SMEM = 1024 + STAGES * STAGE + experts::exchange_bytes<EPI_WARPS>() + BAR_BYTES;
    static constexpr uint32_t IDESC0 = make_idesc(1u, false, false, 256, 0);
    static_assert(SMEM <= 232448, "shared memory");
    static constexpr int MARKS = 8;      // tiles with adapters that may be between their V and their epilogue: STAGES + 2 at most
    static_assert((4 * STAGES + 5 + MARKS) * 8 + 8 + MARKS * V_WARPS * 4 <= BAR_BYTES, "barriers fit");
};

struct MmaTile {
    int tt, row0, rows, n, chan0;
};

// The item-th tile: bands of 8 token tiles, inside them token tiles first, then channels, so that
// units running side by side share weights and token rows in L2.
__device__ __forceinline__ bool mma_tile(const Params& p, int item, MmaTile& t) {
    constexpr int BAND = 8;
    if (item >= p.tiles * p.ctiles) return false;
    const int band = item / (BAND * p.ctiles), r = item - band * BAND * p.ctiles, deep = min(BAND, p.tiles - band * BAND);
    t.tt = band * BAND + r % deep;
    t.row0 = t.tt * p.width;
    t.rows = min(p.width, p.T - t.row0);
    t.n = (t.rows + Mma::Q - 1) / Mma::Q * Mma::Q;
    t.chan0 = (r / deep) * (p.gated ? 128 : 256);
    return true;
}

// The adapters of a token tile, looked up by a whole warp: one load brings the count and the first 31, and may be
// made a tile ahead.
struct TileAdapters {
    const int* list;
    int count, at, mine, ahead;
    bool uniform;                                // one adapter, which every row has
    __device__ __forceinline__ void look_ahead(const Params& p, int tt) {
        ahead = p.L > 0 ? __ldcg(p.lists + static_cast<int64_t>(tt) * kListPitch + (threadIdx.x & 31)) : 0;
    }
    __device__ __forceinline__ void open(const Params& p, int tt) {          // (after look_ahead of the same tile)
        list = p.lists + static_cast<int64_t>(tt) * kListPitch;
        mine = ahead;
        count = __shfl_sync(kAllLanes, mine, 0);
        uniform = (count & kUniform) != 0;
        count &= kUniform - 1;
        at = 0;
    }
    // the next one, -1 when there is none left
    __device__ __forceinline__ int next() {
        if (at >= count) return -1;
        const int place = ++at;
        if ((place & 31) == 0) mine = place + static_cast<int>(threadIdx.x & 31) <= count ? __ldcg(list + place + (threadIdx.x & 31)) : -1;
        return __shfl_sync(kAllLanes, mine, place & 31);
    }
};

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }

// Replaces the numbers that are not finite in the 16-byte vectors [first, last), four at most, of a swizzled row; whether
// there were any. Such a number times zero is NaN, and a sum keeps it: one operation for two numbers. In its place comes the
// smallest normal number of its sign, not zero: where the row's own V is infinite and B too, the product is then the
// infinity that it has to be (with a zero it would be NaN, which nothing added later takes back). Of a finite V it
// leaves 2^-126 of it, 4 at most, in a sum that not_finite_terms makes infinite or NaN.
__device__ __forceinline__ bool make_finite(uint8_t* row, int swizzle, int first, int last) {
    const __nv_bfloat162 zero = __float2bfloat162_rn(0.0f);
    __nv_bfloat162 nan[2] = {zero, zero};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = first + k;
        if (c >= last) break;
        const uint4 b = *reinterpret_cast<const uint4*>(row + ((c ^ swizzle) << 4));
        nan[0] = __hfma2(as_bf162(b.x), zero, nan[0]);
        nan[1] = __hfma2(as_bf162(b.y), zero, nan[1]);
        nan[0] = __hfma2(as_bf162(b.z), zero, nan[0]);
        nan[1] = __hfma2(as_bf162(b.w), zero, nan[1]);
    }
    const __nv_bfloat162 any = __hadd2(nan[0], nan[1]);
    if (!__hisnan(any.x) && !__hisnan(any.y)) return false;
    for (int c = first; c < last; ++c) {
        uint32_t* word = reinterpret_cast<uint32_t*>(row + ((c ^ swizzle) << 4));
        for (int k = 0; k < 4; ++k) {
            const uint32_t v = word[k];             // (the sign and the exponent's last bit)
            word[k] = ((v & 0x7F80u) == 0x7F80u ? v & 0x8080u : v & 0xFFFFu) |
                      ((v & 0x7F800000u) == 0x7F800000u ? v & 0x80800000u : v & 0xFFFF0000u);
        }
    }
    return true;
}

// The terms of V[t] . B_a[n] whose factor of B is not finite.
__device__ __forceinline__ float not_finite_terms(const Params& p, int t, int a, int n) {
    const __nv_bfloat16* b = p.high + (static_cast<int64_t>(a) * p.N + n) * p.r;
    const __nv_bfloat16* v = v_row(p, t);
    float s = 0.0f;
    for (int i = 0; i < p.r; ++i) {
        const float w = __bfloat162float(b[i]);
        if (!(fabsf(w) < INFINITY)) s = fmaf(__bfloat162float(v[i]) + __bfloat162float(v[p.r + i]), w, s);
    }
    return s;
}

template <class Ready, class Released>
__device__ __forceinline__ bool mma_epilogue(const Params& p, const MmaTile& t, uint32_t acc, bool product, int ew,
                                             int cta_chan0, float* exchange, Ready ready, Released released) {
    const int lane = threadIdx.x & 31, q = ew & 3, part = ew >> 2;
    const int i = q * 32 + lane;                             // accumulator lane
    const int ch = cta_chan0 + (p.gated ? (i & 63) : i);     // channel of D
    const bool live = ch < p.wide;
    const int n = p.gated && i >= 64 ? p.N / 2 + ch : ch;    // channel of W and B
    const float bias = live && p.bias ? __ldg(p.bias + n) : 0.0f;
    bool dirty = false;                                      // B of the tile had numbers that are not finite
    bool ok = ready(&dirty);
    const int swap_id = 1 + part * 2 + (q & 1);              // barrier of warps q and q ^ 2
    if (p.gated) ok = experts::pair_all(swap_id, ok);
    if (!ok) return false;
    tc_fence_after();
    float* mine = exchange + ((part * 2 + (q & 1)) * 2 + (q >> 1)) * 512;
    const float* theirs = exchange + ((part * 2 + (q & 1)) * 2 + ((q >> 1) ^ 1)) * 512;
    const int chunks = (t.rows + 31) / 32;
    auto hand_back = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) released();
    };
    if (part >= chunks) hand_back();
    // C in BF16 with rows of even length is read as it is stored, two channels of one row a lane (store_columns), a
    // chunk ahead
    const bool c_pairs = p.C && !p.c_f32 && (p.wide & 1) == 0;
    const int odd = lane & 1;
    uint32_t c_next[16];
    auto load_c = [&](int c) {
        const int col0 = (c * 2 + part) * 32, valid = t.rows - col0;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.C) + static_cast<int64_t>(t.row0 + col0 + odd) * p.wide + ch - odd;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            c_next[j] = live && 2 * j + odd < valid ? *reinterpret_cast<const uint32_t*>(src + static_cast<int64_t>(2 * j) * p.wide) : 0;
    };
    if (c_pairs && part < chunks) load_c(0);
#pragma unroll 1
    for (int c = 0; c * 2 + part < chunks; ++c) {
        const int col0 = (c * 2 + part) * 32;
        float v[32];
        {
            uint32_t r[32];
            tmem_ld32(acc + (static_cast<uint32_t>(q * 32) << 16) + col0, r);
            tmem_ld_wait();
            if ((c + 1) * 2 + part >= chunks) hand_back();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = (product ? __uint_as_float(r[j]) : 0.0f) + bias;
        }
        if (dirty) {
#pragma unroll 1
            for (int j = 0; j < 32; ++j) {
                float more = 0.0f;
                const int a = col0 + j < t.rows ? adapter_of(p, t.row0 + col0 + j) : -1;
                if (a >= 0 && live) more = not_finite_terms(p, t.row0 + col0 + j, a, n);
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] += k == j ? more : 0.0f;
            }
        }
        const int64_t at = static_cast<int64_t>(t.row0 + col0) * p.wide + ch;
        const int valid = t.rows - col0;
        if (p.gated) {
            // gate warps keep columns 0-15 and get up's; up warps keep 16-31 and get the gate's
            const bool up = q >= 2;
            if (c > 0) experts::pair_sync(swap_id);          // the other warp has read the last chunk
#pragma unroll
            for (int j = 0; j < 16; ++j) mine[j * 32 + lane] = up ? v[j] : v[16 + j];
            experts::pair_sync(swap_id);
            float y[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float x = theirs[j * 32 + lane];
                y[j] = up ? silu(x) * v[16 + j] : silu(v[j]) * x;
            }
            const int skip = up ? 16 : 0;
            experts::store_columns<16>(p, at + static_cast<int64_t>(skip) * p.wide, y, live, valid - skip);
        } else {
            if (c_pairs) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint32_t other = __shfl_xor_sync(kAllLanes, c_next[j], 1);
                    const uint32_t both = odd ? __byte_perm(other, c_next[j], 0x7632u) : __byte_perm(c_next[j], other, 0x5410u);
                    v[2 * j] += bf16_lo(both);
                    v[2 * j + 1] += bf16_hi(both);
                }
                if ((c + 1) * 2 + part < chunks) load_c(c + 1);
            } else if (p.C) {
                float more[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int64_t o = at + static_cast<int64_t>(j) * p.wide;
                    const bool there = live && j < valid;
                    if (p.c_f32) more[j] = there ? static_cast<const float*>(p.C)[o] : 0.0f;
                    else more[j] = there ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.C)[o]) : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] += more[j];
            }
            activate(v, p.act);
            experts::store_columns<32>(p, at, v, live, valid);
        }
    }
    if (p.gated && part < chunks) experts::pair_sync(swap_id);        // before the next tile's first write
    return true;
}

__global__ void __launch_bounds__(Mma::THREADS, 1)
    adapter_mma(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const __grid_constant__ CUtensorMap tmB, const __grid_constant__ Params p) {
    constexpr int S = Mma::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* exchange = reinterpret_cast<float*>(ring + S * Mma::STAGE);
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + S * Mma::STAGE + experts::exchange_bytes<Mma::EPI_WARPS>());
    uint64_t* empty = full + S;
    uint64_t* b_full = empty + S;                // a slice of B has landed here, and the stage's token rows are free for V
    uint64_t* v_full = b_full + S;               // masked rows of V are written and B is finite (both CTAs)
    uint64_t* acc_full = v_full + S;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint64_t* looked = drain + 1;                // [MARKS] the n-th tile with adapters: its slices of B have been looked at
    int* dirty = reinterpret_cast<int*>(looked + Mma::MARKS);        // [MARKS][V_WARPS]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dirty + Mma::MARKS * Mma::V_WARPS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int unit = static_cast<int>(blockIdx.x) / 2, units = static_cast<int>(gridDim.x) / 2;
    const int chunks_r = (p.r + Mma::SL - 1) / Mma::SL;          // stages of one adapter
    const int slice_x = p.width / 2 * 128;                       // bytes of a slice of this CTA's token rows

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&b_full[s], 1);
            mbar_init(&v_full[s], 2 * Mma::V_WARPS);
        }
        for (int m = 0; m < Mma::MARKS; ++m) mbar_init(&looked[m], Mma::V_WARPS);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], Mma::EPI_WARPS * 2);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        if (p.kstages > 0) {
            tma_prefetch_desc(&tmW);
            tma_prefetch_desc(&tmX);
        }
        if (p.L > 0) tma_prefetch_desc(&tmB);
    }
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, Mma::TMEM_COLS);
        tmem_relinquish_pair();
    }
    if (p.wait_first) grid_dependency_wait();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (threadIdx.x == 0) grid_launch_dependents();
    const uint32_t tmem = *tmem_slot;

    // Every role looks a tile's adapters up for itself. The slices of X and W of a role's first tile
    // need none of them: the launch that computes them may still run.
    if (warp < Mma::EPI_WARP0) {
    regs_dec<Mma::REGS_FIRST>();
    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        const uint64_t pol = policy_evict_last();
        uint32_t stage = 0, phase = 0;
        uint32_t x_phase = 0, b_phase = 0, last_b = 0;   // bit s: parity of the next use of full[s], b_full[s]; the last was b_full's
        int64_t issued = 0;
        bool ok = true, stalled = false, waited = p.wait_first;
        MmaTile t;
        TileAdapters ta;
        auto wait_v = [&]() {
            if (!waited) grid_dependency_wait();
            waited = true;
        };
        auto advance = [&](bool is_b) {
            if (is_b) b_phase ^= 1u << stage, last_b |= 1u << stage;
            else x_phase ^= 1u << stage, last_b &= ~(1u << stage);
            ++issued;
            if (++stage == S) {
                stage = 0;
                phase ^= 1;
            }
        };
        for (int item = unit; ok && !stalled && mma_tile(p, item, t); item += units) {
            const int chan = t.chan0 + static_cast<int>(rank) * (p.gated ? 64 : 128);
            const int x0 = t.row0 + static_cast<int>(rank) * (t.n / 2);
            if (waited || p.kstages == 0) {
                wait_v();
                ta.look_ahead(p, t.tt);
                ta.open(p, t.tt);
            }
            for (int kb = 0; kb < p.kstages; ++kb) {
                stalled = issued == p.stall_after;
                if (stalled) break;
                ok = mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag, p.wait_ns);
                if (!ok) break;
                if (elect_one()) {
                    uint8_t* w = ring + stage * Mma::STAGE;
                    uint8_t* x = w + Mma::W_BYTES;
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (Mma::W_BYTES + Mma::KS * slice_x));
                    const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
                    const int k0 = kb * Mma::KS * Mma::SL;
                    if (p.k_whole) {
                        tma_load_nd<true>(w, &tmW, fb, 0, chan, 0, kb * Mma::KS, pol);
                        tma_load_nd<true>(x, &tmX, fb, 0, x0, kb * Mma::KS, pol);
                    } else {
                        for (int s = 0; s < Mma::KS; ++s) {
                            tma_load_nd<true>(w + s * Mma::SLICE_W, &tmW, fb, k0 + s * Mma::SL, chan, 0, pol);
                            tma_load_nd<true>(x + s * slice_x, &tmX, fb, k0 + s * Mma::SL, x0, pol);
                        }
                    }
                }
                __syncwarp();
                advance(false);
            }
            if (!ok || stalled) break;
            if (!waited) {
                wait_v();
                ta.look_ahead(p, t.tt);
                ta.open(p, t.tt);
            }
            for (int a = ta.next(); ok && !stalled && a >= 0; a = ta.next()) {
                for (int i = 0; i < chunks_r; ++i) {
                    stalled = issued == p.stall_after;
                    if (stalled) break;
                    ok = mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag, p.wait_ns);
                    if (!ok) break;
                    if (elect_one()) {
                        // (each CTA's own barrier: its own warps look at the slice first)
                        mbar_arrive_expect_tx(&b_full[stage], Mma::SLICE_W);
                        tma_load_nd<true>(ring + stage * Mma::STAGE, &tmB, smem_u32(&b_full[stage]), i * Mma::SL, chan, 0, a, pol);
                    }
                    __syncwarp();
                    advance(true);
                }
            }
        }
        wait_v();
        if (!ok && lane == 0) experts::fail(p, ERR_TIMEOUT_PRODUCER, abort_flag);
        // every copy issued has landed before the CTA leaves: its stage was released by the MMAs that read it, or, where
        // they gave up, the barrier that it counts on says so (of the pair's peer that is the leader's)
        for (int s = 0; s < S; ++s) {
            const int64_t cnt = issued > s ? (issued - s + S - 1) / S : 0;
            if (cnt == 0 || mbar_wait_warp(&empty[s], static_cast<uint32_t>((cnt - 1) & 1), nullptr, p.wait_ns)) continue;
            if (lane == 0) experts::fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
            if ((last_b >> s) & 1) mbar_wait_warp(&b_full[s], ((b_phase >> s) & 1) ^ 1, nullptr, p.wait_ns);
            else if (rank == 0) mbar_wait_warp(&full[s], ((x_phase >> s) & 1) ^ 1, nullptr, p.wait_ns);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (rank == 0) {
            const uint32_t s0 = smem_u32(ring), tmem_u = __shfl_sync(kAllLanes, tmem, 0);
            const uint64_t wd0 = smem_desc_sw128(s0, 16, 1024), xd0 = smem_desc_sw128(s0 + Mma::W_BYTES, 16, 1024);
            uint32_t stage = 0, x_phase = 0, v_phase = 0;    // bit s: the next parity of full[s], v_full[s]
            int local = 0;
            bool ok = true, waited = p.wait_first;
            MmaTile t;
            TileAdapters ta;
            auto wait_v = [&]() {
                if (!waited) grid_dependency_wait();
                waited = true;
            };
            auto release = [&]() {
                if (elect_one()) mma_commit_pair(&empty[stage], 3);
                __syncwarp();
                if (++stage == S) stage = 0;
            };
            for (int item = unit; ok && mma_tile(p, item, t); item += units, ++local) {
                const int buf = local & 1;
                ok = mbar_wait_warp(&acc_empty[buf], ((local >> 1) & 1) ^ 1, abort_flag, p.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem_u + static_cast<uint32_t>(buf * Mma::BN);
                const uint32_t idesc = Mma::IDESC0 | (static_cast<uint32_t>(__shfl_sync(kAllLanes, t.n, 0) >> 3) << 17);
                if (waited || p.kstages == 0) {
                    wait_v();
                    ta.look_ahead(p, t.tt);
                    ta.open(p, t.tt);
                }
                for (int kb = 0; kb < p.kstages; ++kb) {
                    ok = mbar_wait_warp(&full[stage], (x_phase >> stage) & 1, abort_flag, p.wait_ns);
                    if (!ok) break;
                    x_phase ^= 1u << stage;
                    tc_fence_after();
                    const uint64_t wd = wd0 + stage * (Mma::STAGE >> 4), xd = xd0 + stage * (Mma::STAGE >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < Mma::KS * 4; ++k)
                            mma_bf16_pair(acc, wd + (k / 4) * (Mma::SLICE_W >> 4) + (k % 4) * 2,
                                          xd + (k / 4) * (slice_x >> 4) + (k % 4) * 2, idesc, kb > 0 || k > 0 ? 1u : 0u);
                    }
                    release();
                }
                if (!ok) break;
                if (!waited) {
                    wait_v();
                    ta.look_ahead(p, t.tt);
                    ta.open(p, t.tt);
                }
                uint32_t more = p.kstages > 0;
                for (int a = ta.next(); ok && a >= 0; a = ta.next()) {
                    for (int i = 0; i < chunks_r; ++i) {
                        ok = mbar_wait_warp_at<true>(&v_full[stage], (v_phase >> stage) & 1, abort_flag, p.wait_ns);
                        if (!ok) break;
                        v_phase ^= 1u << stage;
                        tc_fence_after();
                        const uint64_t wd = wd0 + stage * (Mma::STAGE >> 4), xd = xd0 + stage * (Mma::STAGE >> 4);
                        const int steps = (min(Mma::SL, p.r - i * Mma::SL) + 15) / 16;
                        if (elect_one()) {
                            for (int part = 0; part < 2; ++part)
                                for (int k = 0; k < steps; ++k) {
                                    mma_bf16_pair(acc, wd + k * 2, xd + part * (slice_x >> 4) + k * 2, idesc, more);
                                    more = 1;
                                }
                        }
                        more = 1;
                        release();
                    }
                }
                if (!ok) break;
                if (elect_one()) mma_commit_pair(&acc_full[buf], 3);
                __syncwarp();
            }
            wait_v();
            if (elect_one()) {
                if (!ok) experts::fail(p, ERR_TIMEOUT_MMA, abort_flag);
                mma_commit_pair(drain, 1);
                if (!mbar_wait(drain, 0, nullptr, p.wait_ns)) experts::fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
            }
        }
        __syncwarp();
    }
    } else if (warp < Mma::EPI_WARP0 + Mma::EPI_WARPS) {
        // ---------------------------------------------------------------- epilogue
        regs_inc<Mma::REGS_EPI>();
        const int ew = warp - Mma::EPI_WARP0;
        int local = 0, marks = 0;                // tiles; tiles with adapters
        bool ok = true;
        MmaTile t;
        grid_dependency_wait();
        for (int item = unit; ok && mma_tile(p, item, t); item += units, ++local) {
            const int buf = local & 1;
            MmaTile ahead;
            if (p.C && mma_tile(p, item + units, ahead)) {       // the next tile's C into L2: 32 channels of this warp's rows
                const int part = ew >> 2, ch = ahead.chan0 + static_cast<int>(rank) * 128 + (ew & 3) * 32, esz = p.c_f32 ? 4 : 2;
                for (int c = part * 32 + lane; c < ahead.rows; c += 64) {
                    const char* at = static_cast<const char*>(p.C) + (static_cast<int64_t>(ahead.row0 + c) * p.wide + ch) * esz;
                    if (ch < p.wide) asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
                    if (ch + 31 < p.wide) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + 31 * esz));
                }
            }
            const bool some = p.L > 0 && __ldcg(p.lists + static_cast<int64_t>(t.tt) * kListPitch) > 0;      // rows with adapters
            ok = mma_epilogue(
                p, t, tmem + static_cast<uint32_t>(buf * Mma::BN), p.kstages > 0 || some, ew,
                t.chan0 + static_cast<int>(rank) * (p.gated ? 64 : 128), exchange,
                [&](bool* any) {
                    if (!mbar_wait_warp(&acc_full[buf], (local >> 1) & 1, abort_flag, p.wait_ns)) return false;
                    if (!some) return true;
                    const int mark = marks % Mma::MARKS;
                    if (!mbar_wait_warp(&looked[mark], (marks / Mma::MARKS) & 1, abort_flag, p.wait_ns)) return false;
                    for (int w = 0; w < Mma::V_WARPS; ++w) *any = *any || dirty[mark * Mma::V_WARPS + w] != 0;
                    return true;
                },
                [&]() {
                    if (rank != 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&acc_empty[buf]), 0));
                    else mbar_arrive_relaxed(&acc_empty[buf]);
                });
            marks += some;
        }
        if (!ok) experts::fail(p, ERR_TIMEOUT_EPILOGUE, abort_flag);
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- masked rows of V, a look at B
        regs_dec<Mma::REGS_V>();
        // Two threads share a token row of this CTA, one has its first numbers and one its second, and a channel of B, half of
        // its slice each. A row's V is loaded ahead (a row has one adapter: up to rank 64 once for the tile).
        const int row = (threadIdx.x - 32 * Mma::V_WARP0) & 127, part = (threadIdx.x - 32 * Mma::V_WARP0) >> 7, swizzle = row & 7;
        uint32_t b_phase = 0;                    // bit s: the next parity of b_full[s]
        int stage = 0, marks = 0;
        bool ok = true;
        MmaTile t;
        TileAdapters ta;
        grid_dependency_wait();
        for (int item = unit; ok && mma_tile(p, item, t); item += units) {
            const int half = t.n / 2, at = static_cast<int>(rank) * half + row;
            const int own = row < half && at < t.rows && p.L > 0 ? adapter_of(p, t.row0 + at) : -1;
            const uint4* src = reinterpret_cast<const uint4*>(v_row(p, t.row0 + at)) + part * (p.r / 8);
            uint4 v[8];
            auto load = [&](int i, int vecs) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    v[c] = make_uint4(0, 0, 0, 0);
                    if (own >= 0 && c < vecs) v[c] = __ldcg(src + i * 8 + c);
                }
            };
            if (chunks_r == 1) load(0, p.r / 8);
            ta.look_ahead(p, t.tt);
            ta.open(p, t.tt);
            stage = (stage + p.kstages) % S;
            bool found = false;
            for (int a = ta.next(); ok && a >= 0; a = ta.next()) {
                for (int i = 0; i < chunks_r; ++i) {
                    const int vecs = min(Mma::SL, p.r - i * Mma::SL) / 8, steps = (vecs + 1) / 2;
                    if (chunks_r > 1) load(i, vecs);
                    ok = mbar_wait_warp(&b_full[stage], (b_phase >> stage) & 1, abort_flag, p.wait_ns);
                    if (!ok) break;
                    b_phase ^= 1u << stage;
                    uint8_t* w = ring + stage * Mma::STAGE + row * 128;
                    uint8_t* x = w + Mma::W_BYTES + part * slice_x;
                    const bool hit = own == a;
                    if (row < half) {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            if (c < 2 * steps) *reinterpret_cast<uint4*>(x + ((c ^ swizzle) << 4)) = hit ? v[c] : make_uint4(0, 0, 0, 0);
                    }
                    found = make_finite(w, swizzle, 4 * part, min(vecs, 4 * part + 4)) || found;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank != 0) mbar_arrive_peer(mapa_shared(smem_u32(&v_full[stage]), 0));
                        else mbar_arrive(&v_full[stage]);
                    }
                    __syncwarp();
                    if (++stage == S) stage = 0;
                }
            }
            if (ok && ta.count > 0) {
                const int any = __any_sync(kAllLanes, found);
                if (lane == 0) {
                    dirty[marks % Mma::MARKS * Mma::V_WARPS + warp - Mma::V_WARP0] = any;
                    mbar_arrive(&looked[marks % Mma::MARKS]);
                }
                __syncwarp();
                ++marks;
            }
        }
        if (!ok && lane == 0) experts::fail(p, ERR_TIMEOUT_PRODUCER, abort_flag);
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, Mma::TMEM_COLS);
    }
}

}  // namespace adapters
}  // namespace dg
