// experts_int8.cuh -- int8 products, dense (one group) or grouped by expert.
//
// GB300's integer tensor rate is far below its FP16 one, so the codes are
// converted on the way: every int8 is exact in FP16 and every product of two in
// the FP32 sum. A byte b becomes FP16 with one byte permute and one subtraction:
// with u = b + 128 (a flipped sign bit), the bits 0x6400 | u are 1024 + u, less 1152.
//
// The weights are the MMA's A operand and go from shared memory through
// registers into Tensor Memory; the token rows are its B operand and go from global
// memory through registers to shared memory. What bounds a prompt is shared memory's 128
// bytes a clock: a stage of 128 K and 192 rows moves 80 KB through it (weights in and out,
// rows in, the MMA's reads) in the 768 clocks that the tensor core needs; with the weights
// converted back into shared memory it would be 112 KB, with raw rows staged there 104 KB.
// Warps of a CTA:
//   0       TMA producer of weight codes: 128 channels x 128 K, 128B swizzle
//   1       MMA issuer (one thread), owner of the Tensor Memory
//   2-3     idle (they complete the first warpgroup)
//   4-7     epilogue
//   8-15    weight converters, two teams: one channel a thread, 128 codes a stage
//   16-23   token converters, two teams: rows by index or in order
// The teams take alternate stages: a stage passes through a chain of waits and
// conversions that is longer than the tensor core takes for it.
#pragma once

#include "experts_common.cuh"
#include "experts_ptx.cuh"

namespace dg {
namespace experts {

template <bool PAIR_>
struct Int8Cfg {
    static constexpr bool PAIR = PAIR_;
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int BN = PAIR ? 192 : 64;           // most token rows of a tile
    static constexpr int BN_CTA = BN / CTAS;
    static constexpr int KB = 128;                       // codes of K per stage
    static constexpr int W_RAW = 128 * KB, W_STAGES = PAIR ? 5 : 8;
    static constexpr int SLICE_X = BN_CTA * 128;         // 64 FP16 of K
    static constexpr int X_CONV = 2 * SLICE_X;
    static constexpr int A_STAGES = 2, C_STAGES = 3;     // converted weights (Tensor Memory), converted rows
    // Converted stage g counts on barriers g % STAGE_BARS, whatever slots it lies in: full by both
    // converters, done by the MMAs (one commit: a second one cost ~250 clocks a stage).
    // The weights' slot is free when stage g - A_STAGES is done, the rows' when g - C_STAGES
    // is; each barrier's next completion needs stage g, so no phase can be missed.
    static constexpr int STAGE_BARS = 4;
    static_assert(A_STAGES < STAGE_BARS && C_STAGES < STAGE_BARS, "stage barriers");
    static constexpr int A_COLS = KB / 2;                // TMEM columns of a converted weight stage
    static constexpr int EPI_WARPS = 4, EPI_WARP0 = 4, W_WARP0 = 8, X_WARP0 = 16, TEAMS = 2;
    static constexpr int THREADS = 768;
    // registers per thread: at launch, and of the warpgroups after the split
    static constexpr int LAUNCH_REGS = 80, REGS_CONTROL = 48, REGS_EPILOGUE = 128, REGS_WEIGHTS = 72, REGS_TOKENS = 80;
    static_assert(REGS_CONTROL + REGS_EPILOGUE + TEAMS * (REGS_WEIGHTS + REGS_TOKENS) <= THREADS / 128 * LAUNCH_REGS,
                  "register split exceeds the launch allocation");
    static constexpr int ACC_COLS = 2 * BN;
    static constexpr int TMEM_COLS = ACC_COLS + A_STAGES * A_COLS <= 256 ? 256 : 512;
    static constexpr int BAR_BYTES = 384;
    static constexpr int BUFFERS = W_STAGES * W_RAW + C_STAGES * X_CONV;
    static constexpr int FIXED = 1024 + BUFFERS + exchange_bytes<EPI_WARPS>() + BAR_BYTES;
    static constexpr uint32_t IDESC0 = make_idesc(0u, false, false, 128 * CTAS, 0);   // FP16 operands
    static_assert(ACC_COLS + A_STAGES * A_COLS <= 512, "Tensor Memory");
    static_assert(FIXED + Schedule::bytes(DGEMM_MAX_EXPERTS) <= 232448, "shared memory");
    static_assert((2 * W_STAGES + 2 * STAGE_BARS + 5) * 8 + 8 <= BAR_BYTES, "barriers fit");
};

// Four int8 codes to four FP16 numbers.
__device__ __forceinline__ void int8x4_to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = codes ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

template <class CF>
__global__ void __launch_bounds__(CF::THREADS, 1) expert_int8(const __grid_constant__ CUtensorMap tmW, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* wraw = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* xconv = wraw + CF::W_STAGES * CF::W_RAW;
    float* exchange = reinterpret_cast<float*>(wraw + CF::BUFFERS);
    uint64_t* w_full = reinterpret_cast<uint64_t*>(wraw + CF::BUFFERS + exchange_bytes<CF::EPI_WARPS>());
    uint64_t* w_empty = w_full + CF::W_STAGES;
    uint64_t* full = w_empty + CF::W_STAGES;             // converted stages
    uint64_t* done = full + CF::STAGE_BARS;
    uint64_t* acc_full = done + CF::STAGE_BARS;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const Schedule sched(reinterpret_cast<uint8_t*>(w_full) + CF::BAR_BYTES, p.E);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CF::PAIR ? cluster_ctarank() : 0u;
    const int unit = static_cast<int>(blockIdx.x) / CF::CTAS, units = static_cast<int>(gridDim.x) / CF::CTAS;
    const int tile_channels = (p.gated ? 64 : 128) * CF::CTAS;

    if (threadIdx.x == 0) {
        for (int s = 0; s < CF::W_STAGES; ++s) {
            mbar_init(&w_full[s], 1);
            mbar_init(&w_empty[s], 4);                   // every weight converter warp
        }
        for (int s = 0; s < CF::STAGE_BARS; ++s) {
            mbar_init(&full[s], 8 * CF::CTAS);           // a team's warps of both converters, of both CTAs
            mbar_init(&done[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], CF::EPI_WARPS * CF::CTAS);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        if (p.kstages > 0) tma_prefetch_desc(&tmW);
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
    // converter warps: counts a converted stage in at the pair's leader
    auto converted = [&](uint32_t g) {
        uint64_t* bar = &full[g % CF::STAGE_BARS];
        if (CF::PAIR && rank != 0) mbar_arrive_peer(mapa_shared(smem_u32(bar), 0));
        else mbar_arrive(bar);
    };
    // ... and wait until the slot of stage g is free in a ring of `slots`
    auto slot_free = [&](uint32_t g, uint32_t slots) {
        if (g < slots) return true;
        const uint32_t last = g - slots;
        return mbar_wait_warp(&done[last % CF::STAGE_BARS], (last / CF::STAGE_BARS) & 1, abort_flag, p.wait_ns);
    };

    Cursor cur;
    Tile t;
    bool ok = true;
    if (warp < CF::EPI_WARP0) {
    regs_dec<CF::REGS_CONTROL>();
    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        if (lane == 0) {
            const uint64_t pol = policy_evict_last();
            uint32_t stage = 0, phase = 0;
            int64_t issued = 0;
            bool stalled = false;
            for (int item = unit; ok && !stalled && cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t); item += units) {
                const int chan = t.chan0 + static_cast<int>(rank) * (p.gated ? 64 : 128);
                for (int kb = 0; kb < p.kstages; ++kb) {
                    if (issued == p.stall_after) {
                        stalled = true;
                        break;
                    }
                    if (!mbar_poll(&w_empty[stage], phase ^ 1, abort_flag, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&w_full[stage], CF::W_RAW);
                    tma_load_nd<false>(wraw + stage * CF::W_RAW, &tmW, smem_u32(&w_full[stage]), kb * CF::KB, chan, 0,
                                       t.expert, pol);
                    ++issued;
                    if (++stage == CF::W_STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) fail(p, ERR_TIMEOUT_PRODUCER, abort_flag);
            for (int s = 0; s < CF::W_STAGES; ++s) {     // every copy issued lands before the CTA may exit
                const int64_t cnt = issued > s ? (issued - s + CF::W_STAGES - 1) / CF::W_STAGES : 0;
                if (cnt > 0 && !mbar_wait(&w_full[s], static_cast<uint32_t>((cnt - 1) & 1), nullptr, p.wait_ns))
                    fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (lane == 0 && rank == 0) {
            const uint64_t xd0 = smem_desc_sw128(smem_u32(xconv), 16, 1024);
            uint32_t g = 0, cs = 0;                      // stages so far; the rows' slot
            int local = 0;
            for (int item = unit; ok && cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t); item += units, ++local) {
                const int buf = local & 1;
                if (!mbar_wait(&acc_empty[buf], ((local >> 1) & 1) ^ 1, abort_flag, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t acc = tmem + static_cast<uint32_t>(buf * CF::BN);
                const uint32_t idesc = CF::IDESC0 | (static_cast<uint32_t>(t.n >> 3) << 17);
                for (int kb = 0; kb < p.kstages; ++kb) {
                    const uint32_t bar = g % CF::STAGE_BARS, phase = (g / CF::STAGE_BARS) & 1;
                    const bool got = CF::PAIR ? mbar_wait_cluster(&full[bar], phase, abort_flag, p.wait_ns)
                                              : mbar_wait(&full[bar], phase, abort_flag, p.wait_ns);
                    if (!got) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = tmem + CF::ACC_COLS + g % CF::A_STAGES * CF::A_COLS;
                    const uint64_t xd = xd0 + cs * (CF::X_CONV >> 4);
#pragma unroll
                    for (int k = 0; k < CF::KB / 16; ++k)
                        mma_f16_tmem_a<CF::PAIR>(acc, a + k * 8, xd + (k / 4) * (CF::SLICE_X >> 4) + (k % 4) * 2, idesc,
                                                 (kb > 0 || k > 0) ? 1u : 0u);
                    if constexpr (CF::PAIR) mma_commit_pair(&done[bar], 3);
                    else mma_commit(&done[bar]);
                    ++g;
                    if (++cs == CF::C_STAGES) cs = 0;
                }
                if (!ok) break;
                if constexpr (CF::PAIR) mma_commit_pair(&acc_full[buf], 3);
                else mma_commit(&acc_full[buf]);
            }
            if (!ok) fail(p, ERR_TIMEOUT_MMA, abort_flag);
            if constexpr (CF::PAIR) mma_commit_pair(drain, 1);
            else mma_commit(drain);
            if (!mbar_wait(drain, 0, nullptr, p.wait_ns)) fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
        }
        __syncwarp();
    }
    } else if (warp < CF::W_WARP0) {
        // ---------------------------------------------------------------- epilogue
        regs_inc<CF::REGS_EPILOGUE>();
        int local = 0;
        for (int item = unit; ok && cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t); item += units, ++local) {
            const int buf = local & 1;
            ok = tile_epilogue<CF::EPI_WARPS, CF::BN>(
                p, t, tmem + static_cast<uint32_t>(buf * CF::BN), warp - CF::EPI_WARP0,
                t.chan0 + static_cast<int>(rank) * (p.gated ? 64 : 128), exchange,
                [&]() { return mbar_wait_warp(&acc_full[buf], (local >> 1) & 1, abort_flag, p.wait_ns); },
                [&]() {
                    if (CF::PAIR && rank != 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&acc_empty[buf]), 0));
                    else mbar_arrive_relaxed(&acc_empty[buf]);
                });
        }
        if (!ok) fail(p, ERR_TIMEOUT_EPILOGUE, abort_flag);
        __syncwarp();
    } else if (warp < CF::X_WARP0) {
        // ---------------------------------------------------------------- weight converters
        regs_dec<CF::REGS_WEIGHTS>();
        const int team = (warp - CF::W_WARP0) >> 2;
        const int row = (warp & 3) * 32 + lane;              // TMEM lane: the warp's own quarter
        const uint32_t a_base = tmem + CF::ACC_COLS + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        uint32_t raw = 0, raw_phase = 0, g = 0;
        for (int item = unit; ok && cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t); item += units) {
            for (int kb = 0; kb < p.kstages; ++kb, ++g) {
                if (static_cast<int>(g % CF::TEAMS) == team) {
                    if (!mbar_wait_warp(&w_full[raw], raw_phase, abort_flag, p.wait_ns)) {
                        ok = false;
                        break;
                    }
                    const uint8_t* src = wraw + raw * CF::W_RAW + row * 128;
                    uint4 codes[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) codes[c] = *reinterpret_cast<const uint4*>(src + ((c ^ (row & 7)) << 4));
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&w_empty[raw]);   // the codes are in registers
                    uint32_t h[32];
                    auto convert = [&](int half) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t* d = h + c * 8;
                            int8x4_to_f16(codes[half * 4 + c].x, d[0], d[1]);
                            int8x4_to_f16(codes[half * 4 + c].y, d[2], d[3]);
                            int8x4_to_f16(codes[half * 4 + c].z, d[4], d[5]);
                            int8x4_to_f16(codes[half * 4 + c].w, d[6], d[7]);
                        }
                    };
                    convert(0);
                    if (!slot_free(g, CF::A_STAGES)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = a_base + g % CF::A_STAGES * CF::A_COLS;
                    tmem_st32(a, h);
                    convert(1);
                    tmem_st32(a + 32, h);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) converted(g);
                }
                if (++raw == CF::W_STAGES) {
                    raw = 0;
                    raw_phase ^= 1;
                }
            }
        }
        if (!ok) fail(p, ERR_TIMEOUT_PRODUCER, abort_flag);
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- token converters
        // Eight threads load and convert one row's 128 codes, 16 each; a team's next stage is
        // being loaded while it converts this one.
        regs_dec<CF::REGS_TOKENS>();
        constexpr int ROUNDS = CF::BN_CTA / 16;
        const int team = (warp - CF::X_WARP0) >> 2;
        const int tid = threadIdx.x & 127, sub = tid >> 3, chunk = tid & 7;
        // a thread's 32 bytes of FP16 are two 16-byte chunks of one slice; threads of the second
        // slice write theirs in the other order, so that the eight of a row meet different banks
        const int j = (chunk & 3) * 2, flip = chunk >> 2;
        const int at0 = (((j + flip) ^ (sub & 7)) << 4), at1 = (((j + 1 - flip) ^ (sub & 7)) << 4);
        int item = unit, kb = team, rounds = 0, src[ROUNDS];
        bool live = p.kstages > 0 && cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t);
        auto point = [&]() {                                 // the rows of tile t
            const int xrows = t.n / CF::CTAS, first = static_cast<int>(rank) * xrows;
            rounds = xrows / 16;
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int r = first + i * 16 + sub;
                src[i] = -1;
                if (i < rounds && r < t.rows) {
                    const int a = p.a_rows ? __ldg(p.a_rows + t.row0 + r) : t.row0 + r;
                    if (a >= 0 && a < p.a_count) src[i] = a;
                }
            }
        };
        auto settle = [&]() {                                // kb into its tile
            bool moved = false;
            while (live && kb >= p.kstages) {
                kb -= p.kstages;
                item += units;
                live = cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t);
                moved = true;
            }
            if (live && moved) point();
        };
        uint4 next[ROUNDS];
        auto load = [&]() {
            const int k = kb * CF::KB + chunk * 16;
            const char* base = static_cast<const char*>(p.A) + k;
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                next[i] = make_uint4(0, 0, 0, 0);
                if (live && src[i] >= 0 && k < p.K)
                    next[i] = __ldg(reinterpret_cast<const uint4*>(base + static_cast<int64_t>(src[i]) * p.K));
            }
        };
        if (live) point();
        settle();
        load();
        uint32_t g = team, cs = team;
        while (live) {
            uint4 codes[ROUNDS];
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) codes[i] = next[i];
            const int now = rounds;
            kb += CF::TEAMS;
            settle();
            load();
            if (!slot_free(g, CF::C_STAGES)) {
                ok = false;
                break;
            }
            uint8_t* slice = xconv + cs * CF::X_CONV + (chunk >> 2) * CF::SLICE_X + sub * 128;
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                if (i >= now) break;
                uint4 lo, hi;
                int8x4_to_f16(codes[i].x, lo.x, lo.y);
                int8x4_to_f16(codes[i].y, lo.z, lo.w);
                int8x4_to_f16(codes[i].z, hi.x, hi.y);
                int8x4_to_f16(codes[i].w, hi.z, hi.w);
                *reinterpret_cast<uint4*>(slice + i * 2048 + at0) = flip ? hi : lo;
                *reinterpret_cast<uint4*>(slice + i * 2048 + at1) = flip ? lo : hi;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) converted(g);
            g += CF::TEAMS;
            cs += CF::TEAMS;
            if (cs >= CF::C_STAGES) cs -= CF::C_STAGES;
        }
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
