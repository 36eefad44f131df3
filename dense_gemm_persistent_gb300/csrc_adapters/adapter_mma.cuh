// adapter_mma.cuh -- the projection with adapters for prompts.
//
// One persistent pair of CTAs per two SMs walks tiles of 256 output channels (the MMA's rows) by
// up to 256 token rows (its columns). The adapters are more K: behind the slices of X and W, the
// sum of a tile goes on, for every adapter a that its rows have, with B_a against the rows'
// V, rows of other requests as zeros. So nothing but V (r numbers a row) is written and read in
// between, and D is rounded once. V = first + second BF16 number (adapter_shrink.cuh): two
// slices against the same slice of B_a.
// Warps of a CTA: 0 TMA producer, 1 MMA issuer and owner of the Tensor Memory, 2-3 idle,
// 4-11 epilogue, 12-15 write the masked rows of V.
// A zero does not hide a number that is not finite. An adapter whose B holds one (p.bad) is left
// out of the products, and the epilogue adds its rows' V . B_a^T by FP32 units: slow, and of its own
// rows only.
#pragma once

#include "adapter_common.cuh"

namespace dg {
namespace adapters {

struct Mma {
    static constexpr int BN = kMostWidth, BN_CTA = BN / 2, LEAST_WIDTH = 64, KS = 2, SL = 64, Q = 32;
    static constexpr int SLICE_W = 128 * 128;
    static constexpr int W_BYTES = KS * SLICE_W, STAGE = W_BYTES + KS * BN_CTA * 128, STAGES = 3;
    static constexpr int EPI_WARP0 = 4, EPI_WARPS = 8, V_WARP0 = 12, V_WARPS = 4, THREADS = 32 * (V_WARP0 + V_WARPS);
    static constexpr int TMEM_COLS = 512, BAR_BYTES = 256;
    static constexpr int SMEM = 1024 + STAGES * STAGE + experts::exchange_bytes<EPI_WARPS>() + BAR_BYTES;
    static constexpr uint32_t IDESC0 = make_idesc(1u, false, false, 256, 0);
    static_assert(SMEM <= 232448, "shared memory");
    static_assert((4 * STAGES + 5) * 8 + 8 <= BAR_BYTES, "barriers fit");
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

// The adapters of a token tile that go through the tensor core, looked up by a whole warp 32 at a time.
struct TileAdapters {
    const int* list;
    int count, base, mine;
    unsigned good;
    __device__ __forceinline__ void look(const Params& p) {
        const int lane = threadIdx.x & 31;
        mine = base + lane < count ? __ldcg(list + 4 + base + lane) : -1;
        good = __ballot_sync(kAllLanes, mine >= 0 && __ldcg(p.bad + mine) != p.epoch);
    }
    __device__ __forceinline__ void open(const Params& p, int tt) {
        list = p.lists + static_cast<int64_t>(tt) * kListPitch;
        count = p.L > 0 ? __ldcg(list) : 0;
        base = 0;
        good = 0;
        if (count > 0) look(p);
    }
    // the next one, -1 when there is none left
    __device__ __forceinline__ int next(const Params& p) {
        while (good == 0) {
            base += 32;
            if (base >= count) return -1;
            look(p);
        }
        const int a = __shfl_sync(kAllLanes, mine, __ffs(good) - 1);
        good &= good - 1;
        return a;
    }
};

// V[t] . B_a[n] from the two BF16 numbers of V.
__device__ __forceinline__ float high_dot_split(const Params& p, int t, int a, int n) {
    const __nv_bfloat16* b = p.high + (static_cast<int64_t>(a) * p.N + n) * p.r;
    const __nv_bfloat16* v = v_split(p, t);
    float s = 0.0f;
    for (int i = 0; i < p.r; ++i) s = fmaf(__bfloat162float(v[i]) + __bfloat162float(v[p.r + i]), __bfloat162float(b[i]), s);
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
    // any adapter of the tile that was left out
    bool left_out = false;
    const int count = p.L > 0 ? __ldcg(p.lists + static_cast<int64_t>(t.tt) * kListPitch) : 0;
    for (int j = lane; j < count; j += 32)
        left_out = left_out || __ldcg(p.bad + __ldcg(p.lists + static_cast<int64_t>(t.tt) * kListPitch + 4 + j)) == p.epoch;
    left_out = __any_sync(kAllLanes, left_out);
    bool ok = ready();
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
        if (left_out) {
#pragma unroll 1
            for (int j = 0; j < 32; ++j) {
                float more = 0.0f;
                const int a = col0 + j < t.rows ? adapter_of(p, t.row0 + col0 + j) : -1;
                if (a >= 0 && live && __ldcg(p.bad + a) == p.epoch) more = high_dot_split(p, t.row0 + col0 + j, a, n);
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
                y[j] = up ? experts::silu(x) * v[16 + j] : experts::silu(v[j]) * x;
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
            experts::activate32(v, p.act);
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
    uint64_t* v_go = empty + S;                  // a stage's token rows are free for masked rows of V (this CTA)
    uint64_t* v_full = v_go + S;                 // they are written (both CTAs)
    uint64_t* acc_full = v_full + S;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
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
            mbar_init(&v_go[s], 1);
            mbar_init(&v_full[s], 2 * Mma::V_WARPS);
        }
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
    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        const uint64_t pol = policy_evict_last();
        uint32_t stage = 0, phase = 0;
        int64_t issued = 0;
        bool ok = true, stalled = false, waited = p.wait_first;
        MmaTile t;
        TileAdapters ta;
        auto wait_v = [&]() {
            if (!waited) grid_dependency_wait();
            waited = true;
        };
        auto advance = [&]() {
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
                advance();
            }
            if (!ok || stalled) break;
            if (!waited) {
                wait_v();
                ta.open(p, t.tt);
            }
            for (int a = ta.next(p); ok && !stalled && a >= 0; a = ta.next(p)) {
                for (int i = 0; i < chunks_r; ++i) {
                    stalled = issued == p.stall_after;
                    if (stalled) break;
                    ok = mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag, p.wait_ns);
                    if (!ok) break;
                    if (elect_one()) {
                        uint8_t* w = ring + stage * Mma::STAGE;
                        if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * Mma::SLICE_W);
                        const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
                        tma_load_nd<true>(w, &tmB, fb, i * Mma::SL, chan, 0, a, pol);
                        mbar_arrive(&v_go[stage]);
                    }
                    __syncwarp();
                    advance();
                }
            }
        }
        wait_v();
        if (!ok && lane == 0) experts::fail(p, ERR_TIMEOUT_PRODUCER, abort_flag);
        // every copy issued has landed before the CTA leaves (the peer of the pair signals the leader's
        // barriers, so it waits for the MMA's release)
        for (int s = 0; s < S; ++s) {
            const int64_t cnt = issued > s ? (issued - s + S - 1) / S : 0;
            uint64_t* bar = rank != 0 ? &empty[s] : &full[s];
            if (cnt > 0 && !mbar_wait_warp(bar, static_cast<uint32_t>((cnt - 1) & 1), nullptr, p.wait_ns) && lane == 0)
                experts::fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (rank == 0) {
            const uint32_t s0 = smem_u32(ring), tmem_u = __shfl_sync(kAllLanes, tmem, 0);
            const uint64_t wd0 = smem_desc_sw128(s0, 16, 1024), xd0 = smem_desc_sw128(s0 + Mma::W_BYTES, 16, 1024);
            uint32_t stage = 0, phase = 0, v_phase = 0;      // bit s of v_phase: the next parity of v_full[s]
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
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
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
                    ta.open(p, t.tt);
                }
                for (int kb = 0; kb < p.kstages; ++kb) {
                    ok = mbar_wait_warp(&full[stage], phase, abort_flag, p.wait_ns);
                    if (!ok) break;
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
                    ta.open(p, t.tt);
                }
                uint32_t more = p.kstages > 0;
                for (int a = ta.next(p); ok && a >= 0; a = ta.next(p)) {
                    for (int i = 0; i < chunks_r; ++i) {
                        ok = mbar_wait_warp(&full[stage], phase, abort_flag, p.wait_ns) &&
                             mbar_wait_warp_at<true>(&v_full[stage], (v_phase >> stage) & 1, abort_flag, p.wait_ns);
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
    } else if (warp >= Mma::EPI_WARP0 && warp < Mma::EPI_WARP0 + Mma::EPI_WARPS) {
        // ---------------------------------------------------------------- epilogue
        const int ew = warp - Mma::EPI_WARP0;
        int local = 0;
        bool ok = true;
        MmaTile t;
        grid_dependency_wait();
        for (int item = unit; ok && mma_tile(p, item, t); item += units, ++local) {
            const int buf = local & 1;
            bool product = p.kstages > 0;
            if (!product) {                      // the tile's rows may have no adapter, or only bad ones: nothing is summed
                TileAdapters ta;
                ta.open(p, t.tt);
                product = ta.next(p) >= 0;
            }
            ok = mma_epilogue(
                p, t, tmem + static_cast<uint32_t>(buf * Mma::BN), product, ew, t.chan0 + static_cast<int>(rank) * (p.gated ? 64 : 128),
                exchange, [&]() { return mbar_wait_warp(&acc_full[buf], (local >> 1) & 1, abort_flag, p.wait_ns); },
                [&]() {
                    if (rank != 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&acc_empty[buf]), 0));
                    else mbar_arrive_relaxed(&acc_empty[buf]);
                });
        }
        if (!ok) experts::fail(p, ERR_TIMEOUT_EPILOGUE, abort_flag);
        __syncwarp();
    } else if (warp >= Mma::V_WARP0) {
        // ---------------------------------------------------------------- masked rows of V
        // A thread has one token row of this CTA, whose numbers it loads ahead (a row has one adapter: up to
        // rank 64 once for the tile).
        const int row = threadIdx.x - 32 * Mma::V_WARP0;
        uint32_t stage = 0, v_phase = 0;
        int64_t done = 0;                        // stages before the tile
        bool ok = true;
        MmaTile t;
        TileAdapters ta;
        grid_dependency_wait();
        for (int item = unit; ok && mma_tile(p, item, t); item += units) {
            const int half = t.n / 2, at = static_cast<int>(rank) * half + row;
            const int own = row < half && at < t.rows && p.L > 0 ? adapter_of(p, t.row0 + at) : -1;
            const uint4* src = reinterpret_cast<const uint4*>(v_split(p, t.row0 + at));
            uint4 v[2][8];
            auto load = [&](int i, int vecs) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    v[0][c] = v[1][c] = make_uint4(0, 0, 0, 0);
                    if (own >= 0 && c < vecs) {
                        v[0][c] = __ldcg(src + i * 8 + c);
                        v[1][c] = __ldcg(src + p.r / 8 + i * 8 + c);
                    }
                }
            };
            if (chunks_r == 1) load(0, p.r / 8);
            ta.open(p, t.tt);
            done += p.kstages;
            for (int a = ta.next(p); ok && a >= 0; a = ta.next(p)) {
                for (int i = 0; i < chunks_r; ++i, ++done) {
                    const int vecs = min(Mma::SL, p.r - i * Mma::SL) / 8, steps = (vecs + 1) / 2;
                    stage = static_cast<uint32_t>(done % S);
                    if (chunks_r > 1) load(i, vecs);
                    ok = mbar_wait_warp(&v_go[stage], (v_phase >> stage) & 1, abort_flag, p.wait_ns);
                    if (!ok) break;
                    v_phase ^= 1u << stage;
                    uint8_t* x = ring + stage * Mma::STAGE + Mma::W_BYTES + row * 128;
                    if (row < half) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            if (c < 2 * steps) {
                                const uint4 none = make_uint4(0, 0, 0, 0);
                                *reinterpret_cast<uint4*>(x + ((c ^ (row & 7)) << 4)) = own == a ? v[0][c] : none;
                                *reinterpret_cast<uint4*>(x + slice_x + ((c ^ (row & 7)) << 4)) = own == a ? v[1][c] : none;
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank != 0) mbar_arrive_peer(mapa_shared(smem_u32(&v_full[stage]), 0));
                        else mbar_arrive(&v_full[stage]);
                    }
                    __syncwarp();
                }
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
