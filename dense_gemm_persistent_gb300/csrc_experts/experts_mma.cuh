// experts_mma.cuh -- products grouped by expert, BF16 and E4M3.
//
// One persistent CTA per SM (or CTA pair per two SMs) walks the tiles of the
// schedule. Warps of a CTA:
//   0       TMA producer: weights, and token rows that are already in order
//   1       MMA issuer, owner of the Tensor Memory
//   2       gathering variants: announces gathered stages to the MMA issuer
//   3       idle (completes the first warpgroup)
//   4-11    epilogue
//   12-..   gathering variants (4 warps, 8 of a pair's CTA): cp.async of token rows by index into the swizzled
//           slices that the MMA reads
// A stage of the ring holds two 128-byte slices of K of both operands; TMA brings
// each operand's in one copy.
//
// What bounds it: long groups the tensor pipe and the operands' way to it, short ones HBM. Gated BF16,
// 16384 rows of 4096 x 4096 over 16 experts, takes 342-351 us with rows in order and 369-388
// gathered (1.4-1.5 PFLOP/s); E4M3 over 32 experts 204 and 217-237; 64 gathered rows over 64 experts of
// 4096 x 4096 BF16 158.
// What the gather's choices were worth when they were made, as the other side's time over its own:
//   cp.async, not TMA copies by index (four rows each, one per ~17 ns, 64 a stage)     1.73
//   copies that arrive by themselves and a warp of its own that announces them, not
//     copying warps that wait for them and announce them                                1.16
//   waits by converged warps, not by one lane                                           1.10
//   stages of two slices, not one                                                       1.04
//   eight copying warps in each CTA of a pair, not four (single CTAs: four, not eight)  1.02 (1.03)
//   row indexes loaded a tile ahead                                                     1.02
// The output channels are the MMA's rows, the token rows its columns, as many as
// the tile has.
#pragma once

#include "experts_common.cuh"
#include "experts_ptx.cuh"

namespace dg {
namespace experts {

template <bool FP8_, bool KN_, bool PAIR_, bool GATHER_>
struct MmaCfg {
    static constexpr bool FP8 = FP8_, KN = KN_, PAIR = PAIR_, GATHER = GATHER_;
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int BN = PAIR ? 256 : 64;           // most token rows of a tile
    static constexpr int BN_CTA = BN / CTAS;
    static constexpr int ESZ = FP8 ? 1 : 2;
    static constexpr int SL = 128 / ESZ;                 // K elements of a slice
    static constexpr int KS = 2;                          // slices per stage
    static constexpr int UK = 32 / ESZ;                  // K elements of one MMA
    static constexpr int SLICE_W = 128 * 128, SLICE_X = BN_CTA * 128;
    static constexpr int W_BYTES = KS * SLICE_W, X_BYTES = KS * SLICE_X, STAGE = W_BYTES + X_BYTES;
    static constexpr int ATOM = KS * SL * 128;           // KN weights: 64 channels of a stage's K rows
    static constexpr int STAGES = (PAIR ? 6 : 8) / KS;
    static constexpr int SMALL_ROWS = 16;                // rows of a small copy of token rows
    static constexpr int EPI_WARPS = 8, EPI_WARP0 = 4, GATHER_WARP0 = 12, GATHER_WARPS = PAIR ? 8 : 4;
    static constexpr int THREADS = 32 * (GATHER ? GATHER_WARP0 + GATHER_WARPS : EPI_WARP0 + EPI_WARPS);
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int BAR_BYTES = 256;
    static constexpr int FIXED = 1024 + STAGES * STAGE + exchange_bytes<EPI_WARPS>() + BAR_BYTES;
    static constexpr uint32_t IDESC0 = make_idesc(FP8 ? 0u : 1u, KN, false, 128 * CTAS, 0);
    static_assert(!(FP8 && KN), "E4M3 weights are stored N x K");
    static_assert(FIXED + Schedule::bytes(DGEMM_MAX_EXPERTS) <= 232448, "shared memory");
    static_assert((3 * STAGES + 5) * 8 + 8 <= BAR_BYTES, "barriers fit");
};

template <class CF>
__global__ void __launch_bounds__(CF::THREADS, 1)
    expert_mma(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
               const __grid_constant__ CUtensorMap tmXs, const Params p) {
    constexpr int S = CF::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* exchange = reinterpret_cast<float*>(ring + S * CF::STAGE);
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + S * CF::STAGE + exchange_bytes<CF::EPI_WARPS>());
    uint64_t* empty = full + S;
    uint64_t* landed = empty + S;                // gathered rows of a stage
    uint64_t* acc_full = landed + S;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const Schedule sched(reinterpret_cast<uint8_t*>(full) + CF::BAR_BYTES, p.E);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CF::PAIR ? cluster_ctarank() : 0u;
    const int unit = static_cast<int>(blockIdx.x) / CF::CTAS, units = static_cast<int>(gridDim.x) / CF::CTAS;
    const int tile_channels = (p.gated ? 64 : 128) * CF::CTAS;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1 + (CF::GATHER ? CF::CTAS : 0));
            mbar_init(&landed[s], 32 * CF::GATHER_WARPS);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], CF::EPI_WARPS * CF::CTAS);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        if (p.kstages > 0) {
            tma_prefetch_desc(&tmW);
            if (!CF::GATHER) {
                tma_prefetch_desc(&tmX);
                tma_prefetch_desc(&tmXs);
            }
        }
    }
    if constexpr (CF::PAIR) {
        __syncthreads();
        cluster_sync();
        if (warp == 1) {
            tmem_alloc_pair(tmem_slot, CF::TMEM_COLS);
            tmem_relinquish_pair();
        }
    } else if (warp == 1) {
        tmem_alloc(tmem_slot, CF::TMEM_COLS);
        tmem_relinquish();
    }
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    if (warp == 0) build_schedule<CF::BN>(p, sched);
    tc_fence_before();
    __syncthreads();
    if constexpr (CF::PAIR) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        const uint64_t pol = policy_evict_last();
        uint32_t stage = 0, phase = 0;
        int64_t issued = 0;
        bool ok = true, stalled = false;
        Cursor cur;
        Tile t;
        for (int item = unit; ok && !stalled && __all_sync(kAllLanes, cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t));
             item += units) {
            const int chan = t.chan0 + static_cast<int>(rank) * (p.gated ? 64 : 128);
            const int xrows = __shfl_sync(kAllLanes, t.n, 0) / CF::CTAS;   // token rows of this CTA
            const int x0 = t.row0 + static_cast<int>(rank) * xrows;
            // few rows: copies of 16; else one copy of the whole box (rows beyond the tile are not used)
            const int small = xrows <= 2 * CF::SMALL_ROWS ? (xrows + CF::SMALL_ROWS - 1) / CF::SMALL_ROWS : 0;
            const uint32_t xbytes = CF::GATHER ? 0 : small ? small * CF::SMALL_ROWS * 128 * CF::KS : CF::X_BYTES;
            for (int kb = 0; kb < p.kstages; ++kb) {
                stalled = issued == p.stall_after;
                if (stalled) break;
                ok = mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag, p.wait_ns);
                if (!ok) break;
                if (elect_one()) {
                    uint8_t* w = ring + stage * CF::STAGE;
                    uint8_t* x = w + CF::W_BYTES;
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], CF::CTAS * (CF::W_BYTES + xbytes));
                    const uint32_t fb = CF::PAIR ? mapa_shared(smem_u32(&full[stage]), 0) : smem_u32(&full[stage]);
                    const int k0 = kb * CF::KS * CF::SL;
                    if constexpr (CF::KN) {
                        // atoms of 64 channels, a stage's K rows each
                        const int second = p.gated ? p.N / 2 + chan : chan + 64;
                        tma_load_nd<CF::PAIR>(w, &tmW, fb, chan, k0, t.expert, pol);
                        tma_load_nd<CF::PAIR>(w + CF::ATOM, &tmW, fb, second, k0, t.expert, pol);
                    } else if (p.k_whole) {
                        tma_load_nd<CF::PAIR>(w, &tmW, fb, 0, chan, 0, kb * CF::KS, t.expert, pol);
                    } else {
                        for (int s = 0; s < CF::KS; ++s)
                            tma_load_nd<CF::PAIR>(w + s * CF::SLICE_W, &tmW, fb, k0 + s * CF::SL, chan, 0, t.expert, pol);
                    }
                    if constexpr (!CF::GATHER) {
                        const CUtensorMap* m = small ? &tmXs : &tmX;
                        const int copies = small ? small : 1;
                        for (int c = 0; c < copies; ++c) {
                            const int y = x0 + c * CF::SMALL_ROWS;
                            // slices one copy apart: a small copy's two slices land in place only one by one
                            if (p.k_whole && !small) {
                                tma_load_nd<CF::PAIR>(x, m, fb, 0, y, kb * CF::KS, pol);
                            } else {
                                for (int s = 0; s < CF::KS; ++s) {
                                    uint8_t* d = x + s * CF::SLICE_X + c * CF::SMALL_ROWS * 128;
                                    if (p.k_whole)
                                        tma_load_nd<CF::PAIR>(d, m, fb, 0, y, kb * CF::KS + s, pol);
                                    else
                                        tma_load_nd<CF::PAIR>(d, m, fb, k0 + s * CF::SL, y, pol);
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                ++issued;
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok && lane == 0) fail(p, ERR_TIMEOUT_PRODUCER, abort_flag);
        // Drain: every copy issued has landed before the CTA may exit (the peer of a pair
        // signals the leader's barriers, so it waits for the MMA's release).
        for (int s = 0; s < S; ++s) {
            const int64_t cnt = issued > s ? (issued - s + S - 1) / S : 0;
            uint64_t* bar = (CF::PAIR && rank != 0) ? &empty[s] : &full[s];
            if (cnt > 0 && !mbar_wait_warp(bar, static_cast<uint32_t>((cnt - 1) & 1), nullptr, p.wait_ns) && lane == 0)
                fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (rank == 0) {
            // (values and branches that the compiler knows to be the warp's stay in uniform registers)
            const uint32_t s0 = smem_u32(ring), tmem_u = __shfl_sync(kAllLanes, tmem, 0);
            const uint64_t wd0 = smem_desc_sw128(s0, CF::KN ? CF::ATOM : 16, 1024);
            const uint64_t xd0 = smem_desc_sw128(s0 + CF::W_BYTES, 16, 1024);
            constexpr int NK = CF::SL / CF::UK;                  // MMAs per slice
            constexpr uint32_t W_STEP = (CF::KN ? CF::UK * 128 : 32) >> 4;
            uint32_t stage = 0, phase = 0;
            int local = 0;
            bool ok = true;
            Cursor cur;
            Tile t;
            for (int item = unit; ok && __all_sync(kAllLanes, cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t));
                 item += units, ++local) {
                const int buf = local & 1;
                ok = mbar_wait_warp(&acc_empty[buf], ((local >> 1) & 1) ^ 1, abort_flag, p.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem_u + static_cast<uint32_t>(buf * CF::BN);
                const uint32_t idesc = CF::IDESC0 | (static_cast<uint32_t>(__shfl_sync(kAllLanes, t.n, 0) >> 3) << 17);
                for (int kb = 0; kb < p.kstages; ++kb) {
                    ok = mbar_wait_warp_at<CF::PAIR && CF::GATHER>(&full[stage], phase, abort_flag, p.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t wd = wd0 + stage * (CF::STAGE >> 4), xd = xd0 + stage * (CF::STAGE >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < CF::KS * NK; ++k) {
                            const uint32_t more = (kb > 0 || k > 0) ? 1u : 0u;
                            const uint64_t a = wd + (CF::KN ? k * W_STEP : (k / NK) * (CF::SLICE_W >> 4) + (k % NK) * W_STEP);
                            const uint64_t b = xd + (k / NK) * (CF::SLICE_X >> 4) + (k % NK) * 2;
                            if constexpr (CF::PAIR) {
                                if constexpr (CF::FP8) mma_f8_pair(acc, a, b, idesc, more);
                                else mma_bf16_pair(acc, a, b, idesc, more);
                            } else {
                                if constexpr (CF::FP8) mma_f8(acc, a, b, idesc, more);
                                else mma_bf16(acc, a, b, idesc, more);
                            }
                        }
                        if constexpr (CF::PAIR) mma_commit_pair(&empty[stage], 3);
                        else mma_commit(&empty[stage]);
                    }
                    __syncwarp();
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                if (elect_one()) {
                    if constexpr (CF::PAIR) mma_commit_pair(&acc_full[buf], 3);
                    else mma_commit(&acc_full[buf]);
                }
                __syncwarp();
            }
            if (elect_one()) {
                if (!ok) fail(p, ERR_TIMEOUT_MMA, abort_flag);
                if constexpr (CF::PAIR) mma_commit_pair(drain, 1);
                else mma_commit(drain);
                if (!mbar_wait(drain, 0, nullptr, p.wait_ns)) fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
            }
        }
        __syncwarp();
    } else if (warp >= CF::EPI_WARP0 && warp < CF::EPI_WARP0 + CF::EPI_WARPS) {
        // ---------------------------------------------------------------- epilogue
        const int ew = warp - CF::EPI_WARP0;
        int local = 0;
        bool ok = true;
        Cursor cur;
        Tile t;
        for (int item = unit; ok && cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t); item += units, ++local) {
            const int buf = local & 1;
            ok = tile_epilogue<CF::EPI_WARPS>(
                p, t, tmem + static_cast<uint32_t>(buf * CF::BN), ew,
                t.chan0 + static_cast<int>(rank) * (p.gated ? 64 : 128), exchange,
                [&]() { return mbar_wait_warp(&acc_full[buf], (local >> 1) & 1, abort_flag, p.wait_ns); },
                [&]() {
                    if (CF::PAIR && rank != 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&acc_empty[buf]), 0));
                    else mbar_arrive_relaxed(&acc_empty[buf]);
                });
        }
        if (!ok) fail(p, ERR_TIMEOUT_EPILOGUE, abort_flag);
        __syncwarp();
    } else if (CF::GATHER && warp == 2) {
        // ---------------------------------------------------------------- announcer
        // A stage whose copies have landed becomes visible to the tensor core's
        // (asynchronous) reads by a proxy fence, then counts on its full barrier.
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        Cursor cur;
        Tile t;
        for (int item = unit; ok && cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t); item += units) {
            for (int kb = 0; kb < p.kstages; ++kb) {
                ok = mbar_wait_warp(&landed[stage], phase, abort_flag, p.wait_ns);
                if (!ok) break;
                fence_proxy_async_smem();
                if (elect_one()) {
                    if (CF::PAIR && rank != 0) mbar_arrive_peer(mapa_shared(smem_u32(&full[stage]), 0));
                    else mbar_arrive(&full[stage]);
                }
                __syncwarp();
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok && lane == 0) fail(p, ERR_TIMEOUT_PRODUCER, abort_flag);
    } else if (CF::GATHER && warp >= CF::GATHER_WARP0) {
        // ---------------------------------------------------------------- gather
        // Eight lanes copy the 16-byte chunks of one row's slice, four rows a warp at a time; every
        // thread's copies arrive on the stage's landed barrier by themselves.
        constexpr int STEP = 4 * CF::GATHER_WARPS, ROUNDS = CF::BN_CTA / STEP;
        const int sub = (warp - CF::GATHER_WARP0) * 4 + (lane >> 3), chunk = lane & 7;
        const int64_t pitch = static_cast<int64_t>(p.K) * CF::ESZ;
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        Cursor cur;
        Tile t;
        int item = unit, next[ROUNDS];                       // next: row indexes of tile t, loaded a tile ahead
        bool live = cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t);
        auto look = [&]() {
            const int xrows = t.n / CF::CTAS, first = static_cast<int>(rank) * xrows;
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int r = first + i * STEP + sub;
                next[i] = i * STEP + sub < xrows && r < t.rows ? __ldg(p.a_rows + t.row0 + r) : -1;
            }
        };
        if (live) look();
        while (ok && live) {
            const char* src[ROUNDS];
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i)
                src[i] = next[i] >= 0 && next[i] < p.a_count ? static_cast<const char*>(p.A) + next[i] * pitch : nullptr;
            const int rounds = (t.n / CF::CTAS + STEP - 1) / STEP;
            item += units;
            live = cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t);
            if (live) look();
            for (int kb = 0; kb < p.kstages; ++kb) {
                if (!mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag, p.wait_ns)) {
                    ok = false;
                    break;
                }
                uint8_t* x = ring + stage * CF::STAGE + CF::W_BYTES;
#pragma unroll
                for (int s = 0; s < CF::KS; ++s) {
                    const int64_t kbyte = (static_cast<int64_t>(kb) * CF::KS + s) * 128 + chunk * 16;
#pragma unroll
                    for (int i = 0; i < ROUNDS; ++i) {
                        if (i >= rounds) break;
                        const int row = i * STEP + sub;
                        const bool read = kbyte < pitch && src[i] != nullptr;
                        cp_async_16(x + s * CF::SLICE_X + row * 128 + ((chunk ^ (row & 7)) << 4),
                                    read ? src[i] + kbyte : static_cast<const char*>(p.A), read ? 16u : 0u);
                    }
                }
                cp_async_mbar_arrive(&landed[stage]);
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        cp_async_commit();
        cp_async_wait<0>();      // nothing of this thread's is in flight when it leaves
        if (!ok) fail(p, ERR_TIMEOUT_PRODUCER, abort_flag);
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (CF::PAIR) {
        cluster_sync();
        if (warp == 1) {
            tc_fence_after();
            tmem_dealloc_pair(tmem, CF::TMEM_COLS);
        }
    } else if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, CF::TMEM_COLS);
    }
}

}  // namespace experts
}  // namespace dg
