// experts_int8.cuh -- int8 products, dense (one group) or grouped by expert.
//
// GB300's integer tensor rate is far below its FP16 one, so the codes are
// converted on the way: every int8 is exact in FP16 and every product of two in
// the FP32 sum. A byte b becomes FP16 with one byte permute and one subtraction:
// with u = b + 128 (a flipped sign bit), the bits 0x6400 | u are 1024 + u, less 1152.
//
// Weights come by TMA as codes and go through registers into Tensor Memory, where the
// MMA takes its A operand from; token rows go from global memory through registers to
// shared memory, its B operand. 128 K of a 256 x 192 tile of a CTA pair move 80 KB through
// each SM's shared memory; with the converted weights there too (256 x 256 tiles) it
// would be 160 KB, 78 % of what shared memory can move in the time taken.
// Warps of a CTA:
//   0       TMA producer of weight codes: 128 channels x 128 K, 128B swizzle
//   1       MMA issuer, owner of the Tensor Memory
//   2-3     idle (they complete the first warpgroup)
//   4-7     epilogue
//   8-..    weight converters, one channel a thread; three teams of four warps (pairs: two)
//   then    token converters, rows by index or in order; four teams of two warps
// A converted stage is 64 K; the teams take them in turn, since a stage passes through a
// chain of waits and conversions (1200-1500 clocks) longer than its MMAs (~400 for a whole
// tile). Four teams of two warps convert tokens faster than two of four: a stage's fixed
// part, its waits and arrivals, is spread over twice as long. The MMA warp shares its scheduler
// with five others, so it takes two stages per wait. A third team of weight converters helps
// single CTAs, whose tokens need few registers; a fourth has too few. For pairs the registers
// that a third takes from the token teams cost more than it gives.
//
// Measured: 4096 x 11008 x 4096 with SiLU and bias 287 us (1.29 PFLOP/s), 16384 rows of 4096 x 4096 over
// 16 experts 416, 768 gathered rows over 64 experts of 2048 x 4096 (single CTAs) 101 (5.3 TB/s).
// What each choice was worth when it was made, as the other side's time over its own:
//   weights in Tensor Memory, not shared memory   1.10 (prompt), 1.08 (768 rows)
//   four token teams of two warps, not 2 of 4     1.13 (16384 rows), 1.06 (768 rows)
//   two stages per MMA wait, not one              1.04 (768 rows)
//   single CTAs: three weight teams, not 2 or 4   1.15, 1.08 (768 rows)
//   pairs: two weight teams, not 3                1.11 (prompt)
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
    static constexpr int KB = 128, KC = 64;              // K of a raw and of a converted stage
    static constexpr int W_RAW = 128 * KB, W_STAGES = 7 + PAIR;
    static constexpr int AHEAD = 2;                      // single CTAs: stages that a token team has copies of
    static constexpr int X_CONV = BN_CTA * KC * 2;       // a converted stage: rows here, weights in Tensor Memory
    static constexpr int A_COLS = KC / 2, C_STAGES = 4;
    static constexpr int ACC_COLS = 2 * BN;
    static constexpr int EPI_WARPS = 4, EPI_WARP0 = 4, W_WARP0 = 8, W_TEAMS = PAIR ? 2 : 3, X_WARP0 = W_WARP0 + 4 * W_TEAMS, X_TEAMS = 4;
    static constexpr int STAGE_ARRIVALS = 4 + 2;         // warps of a weight and of a token team
    static constexpr int THREADS = 32 * (X_WARP0 + 2 * X_TEAMS);
    // registers per thread: at launch, and of the warpgroups after the split
    static constexpr int LAUNCH_REGS = PAIR ? 80 : 72, REGS_CONTROL = 48, REGS_EPILOGUE = 128, REGS_WEIGHTS = 72, REGS_TOKENS = PAIR ? 80 : 56;
    static_assert(REGS_CONTROL + REGS_EPILOGUE + W_TEAMS * REGS_WEIGHTS + X_TEAMS / 2 * REGS_TOKENS <= THREADS / 128 * LAUNCH_REGS,
                  "register split exceeds the launch allocation");
    static constexpr int TMEM_COLS = ACC_COLS + C_STAGES * A_COLS;
    static_assert(TMEM_COLS == 256 || TMEM_COLS == 512, "Tensor Memory");
    static constexpr int BAR_BYTES = 384;
    static constexpr int X_RAW = PAIR ? 0 : BN_CTA * KC;   // copies of codes
    static constexpr int BUFFERS = W_STAGES * W_RAW + C_STAGES * X_CONV + X_TEAMS * AHEAD * X_RAW;
    static constexpr int FIXED = 1024 + BUFFERS + exchange_bytes<EPI_WARPS>() + BAR_BYTES;
    static constexpr uint32_t IDESC0 = make_idesc(0u, false, false, 128 * CTAS, 0);   // FP16 operands
    static_assert(FIXED + Schedule::bytes(DGEMM_MAX_EXPERTS) <= 232448, "shared memory");
    static_assert((2 * W_STAGES + 3 * C_STAGES / 2 + 5) * 8 + 8 <= BAR_BYTES, "barriers fit");
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
    uint8_t* conv = wraw + CF::W_STAGES * CF::W_RAW;     // converted rows
    float* exchange = reinterpret_cast<float*>(wraw + CF::BUFFERS);
    uint64_t* w_full = reinterpret_cast<uint64_t*>(wraw + CF::BUFFERS + exchange_bytes<CF::EPI_WARPS>());
    uint64_t* w_empty = w_full + CF::W_STAGES;
    uint64_t* full = w_empty + CF::W_STAGES;             // two converted stages, of one raw stage
    uint64_t* done = full + CF::C_STAGES / 2;            // one of them
    uint64_t* acc_full = done + CF::C_STAGES;
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
            mbar_init(&w_empty[s], 8);                   // the teams that convert its two halves
        }
        for (int s = 0; s < CF::C_STAGES / 2; ++s) mbar_init(&full[s], 2 * CF::STAGE_ARRIVALS * CF::CTAS);
        for (int s = 0; s < CF::C_STAGES; ++s) mbar_init(&done[s], 1);
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
    // converter warps: their part of converted stage g is in place ...
    auto converted = [&](uint32_t g) {
        __syncwarp();
        uint64_t* bar = &full[(g >> 1) % (CF::C_STAGES / 2)];
        if (lane == 0) {
            if (CF::PAIR && rank != 0) mbar_arrive_peer(mapa_shared(smem_u32(bar), 0));
            else mbar_arrive(bar);
        }
    };
    // ... and a wait until the MMAs have read the stage before it in the same slot
    auto slot_free = [&](uint32_t g) {
        return mbar_wait_warp(&done[g % CF::C_STAGES], ((g / CF::C_STAGES) & 1) ^ 1, abort_flag, p.wait_ns);
    };

    Cursor cur;
    Tile t;
    bool ok = true;
    if (warp < CF::EPI_WARP0) {
    regs_dec<CF::REGS_CONTROL>();
    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        const uint64_t pol = policy_evict_last();
        uint32_t stage = 0, phase = 0;
        int64_t issued = 0;
        bool stalled = false;
        for (int item = unit; ok && !stalled && __all_sync(kAllLanes, cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t));
             item += units) {
            const int chan = t.chan0 + static_cast<int>(rank) * (p.gated ? 64 : 128);
            for (int kb = 0; kb < p.kstages; ++kb) {
                stalled = issued == p.stall_after;
                if (stalled) break;
                ok = mbar_wait_warp(&w_empty[stage], phase ^ 1, abort_flag, p.wait_ns);
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&w_full[stage], CF::W_RAW);
                    tma_load_nd<false>(wraw + stage * CF::W_RAW, &tmW, smem_u32(&w_full[stage]), kb * CF::KB, chan, 0,
                                       t.expert, pol);
                }
                __syncwarp();
                ++issued;
                if (++stage == CF::W_STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok && lane == 0) fail(p, ERR_TIMEOUT_PRODUCER, abort_flag);
        for (int s = 0; s < CF::W_STAGES; ++s) {         // every copy issued lands before the CTA may exit
            const int64_t cnt = issued > s ? (issued - s + CF::W_STAGES - 1) / CF::W_STAGES : 0;
            if (cnt > 0 && !mbar_wait_warp(&w_full[s], static_cast<uint32_t>((cnt - 1) & 1), nullptr, p.wait_ns) && lane == 0)
                fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (rank == 0) {
            const uint64_t xd0 = smem_desc_sw128(smem_u32(conv), 16, 1024);
            uint32_t g = 0;                              // raw stages so far
            int local = 0;
            const uint32_t tmem_u = __shfl_sync(kAllLanes, tmem, 0);   // (values and branches that the compiler knows to
                                                                       // be the warp's stay in uniform registers)
            for (int item = unit; ok && __all_sync(kAllLanes, cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t));
                 item += units, ++local) {
                const int buf = local & 1;
                ok = mbar_wait_warp(&acc_empty[buf], ((local >> 1) & 1) ^ 1, abort_flag, p.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem_u + static_cast<uint32_t>(buf * CF::BN);
                const uint32_t idesc = CF::IDESC0 | (static_cast<uint32_t>(__shfl_sync(kAllLanes, t.n, 0) >> 3) << 17);
                for (int kb = 0; kb < p.kstages; ++kb, ++g) {
                    const uint32_t two = g % (CF::C_STAGES / 2), phase = (g / (CF::C_STAGES / 2)) & 1;
                    ok = mbar_wait_warp_at<CF::PAIR>(&full[two], phase, abort_flag, p.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = tmem_u + CF::ACC_COLS + two * (2 * CF::A_COLS);
                    const uint64_t xd = xd0 + two * (2 * CF::X_CONV >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 2 * CF::KC / 16; ++k) {
                            const uint32_t more = (kb > 0 || k > 0) ? 1u : 0u;
                            mma_16_tmem_a<CF::PAIR>(acc, a + k * 8, xd + (k / 4) * (CF::X_CONV >> 4) + (k % 4) * 2, idesc, more);
                            if (k % 4 == 3) {
                                if constexpr (CF::PAIR) mma_commit_pair(&done[2 * two + k / 4], 3);
                                else mma_commit(&done[2 * two + k / 4]);
                            }
                        }
                    }
                    __syncwarp();
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
    }
    } else if (warp < CF::W_WARP0) {
        // ---------------------------------------------------------------- epilogue
        regs_inc<CF::REGS_EPILOGUE>();
        int local = 0;
        for (int item = unit; ok && cur.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, t); item += units, ++local) {
            const int buf = local & 1;
            ok = tile_epilogue<CF::EPI_WARPS>(
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
        const int row = threadIdx.x & 127;                   // TMEM lane: the warp's own quarter
        const uint32_t a_base = tmem + CF::ACC_COLS + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        // Stages are counted over all of the CTA's tiles (operands that fit in memory keep the count
        // below 2^31). The next codes are fetched before the wait for this stage's slot, or behind
        // its store where a pair's MMAs are what takes longest (either is 1 to 3 % better in its place).
        const int64_t tiles = static_cast<int64_t>(sched.head[1]) * p.ctiles;
        const uint32_t total = tiles > unit ? static_cast<uint32_t>((tiles - unit + units - 1) / units * 2 * p.kstages) : 0u;
        const uint8_t* src = wraw + row * 128;
        const int low = row & 3;
        uint4 codes[4];
        auto fetch = [&](uint32_t g) {                       // a stage's codes into registers
            const uint32_t n = g >> 1, raw = n % CF::W_STAGES;
            if (!mbar_wait_warp(&w_full[raw], (n / CF::W_STAGES) & 1, abort_flag, p.wait_ns)) return false;
            const uint8_t* from = src + raw * CF::W_RAW;
            const int at = (static_cast<int>(g & 1) * 4) ^ (row & 4);
#pragma unroll
            for (int c = 0; c < 4; ++c) codes[c] = *reinterpret_cast<const uint4*>(from + ((at + (c ^ low)) << 4));
            __syncwarp();
            if (lane == 0) mbar_arrive(&w_empty[raw]);
            return true;
        };
        if (static_cast<uint32_t>(team) < total) ok = fetch(team);
        for (uint32_t g = team; ok && g < total; g += CF::W_TEAMS) {
            uint32_t h[32];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                int8x4_to_f16(codes[c].x, h[8 * c], h[8 * c + 1]);
                int8x4_to_f16(codes[c].y, h[8 * c + 2], h[8 * c + 3]);
                int8x4_to_f16(codes[c].z, h[8 * c + 4], h[8 * c + 5]);
                int8x4_to_f16(codes[c].w, h[8 * c + 6], h[8 * c + 7]);
            }
            const bool again = g + CF::W_TEAMS < total;
            if (!CF::PAIR && again) ok = fetch(g + CF::W_TEAMS);
            ok = ok && slot_free(g);
            if (!ok) break;
            tc_fence_after();
            tmem_st32(a_base + g % CF::C_STAGES * CF::A_COLS, h);
            tmem_st_wait();
            tc_fence_before();
            converted(g);
            if (CF::PAIR && again) ok = fetch(g + CF::W_TEAMS);
        }
        if (!ok) fail(p, ERR_TIMEOUT_PRODUCER, abort_flag);
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- token converters
        // Four threads load and convert a row's 64 codes, 16 each, 16 rows a round; the team's next
        // stage is on its way before one is converted.
        regs_dec<CF::REGS_TOKENS>();
        constexpr int ROUNDS = CF::BN_CTA / 16;
        const int team = (warp - CF::X_WARP0) >> 1;
        const int tid = threadIdx.x & 63, sub = tid >> 2, chunk = tid & 3;
        const int at0 = ((2 * chunk) ^ (sub & 7)) << 4, at1 = ((2 * chunk + 1) ^ (sub & 7)) << 4;
        int item = unit, kb = team >> 1, rounds = 0, src[ROUNDS], next[ROUNDS];
        Cursor ahead;
        Tile ta;                                             // the tile after the one that is loaded from
        bool more = p.kstages > 0 && ahead.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, ta), live = false;
        auto look = [&]() {                                  // its row indexes, a tile before they are needed
            const int xrows = ta.n / CF::CTAS, first = static_cast<int>(rank) * xrows;
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int row = i * 16 + sub, r = first + row;
                next[i] = -1;
                if (row < xrows && r < ta.rows) next[i] = p.a_rows ? __ldg(p.a_rows + ta.row0 + r) : ta.row0 + r;
            }
        };
        auto advance = [&]() {                               // on to that tile
            live = more;
            if (!more) return;
            rounds = ta.n / (16 * CF::CTAS);
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) src[i] = next[i] < p.a_count ? next[i] : -1;
            item += units;
            more = ahead.at<CF::BN, CF::CTAS>(p, sched, item, tile_channels, ta);
            if (more) look();
        };
        auto settle = [&]() {                                // kb past a tile's last stage is a stage of a later tile
            while (live && kb >= p.kstages) {
                kb -= p.kstages;
                advance();
            }
        };
        if (more) look();
        advance();
        settle();
        const int half = (team & 1) * CF::KC + chunk * 16;
        if constexpr (CF::PAIR) {
            // A stage's codes in registers; as one is converted its registers take the next.
            uint4 codes[ROUNDS];
            auto load = [&](int i) {
                const int k = kb * CF::KB + half;
                codes[i] = make_uint4(0, 0, 0, 0);
                if (live && src[i] >= 0 && k < p.K)
                    codes[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(p.A) + k + static_cast<int64_t>(src[i]) * p.K));
            };
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) load(i);
            for (uint32_t g = team; live; g += CF::X_TEAMS) {
                const int now = rounds;
                kb += CF::X_TEAMS / 2;
                settle();
                ok = slot_free(g);
                if (!ok) break;
                uint8_t* dst = conv + g % CF::C_STAGES * CF::X_CONV + sub * 128;
#pragma unroll
                for (int i = 0; i < ROUNDS; ++i) {
                    if (i < now) {
                        uint4 lo, hi;
                        int8x4_to_f16(codes[i].x, lo.x, lo.y);
                        int8x4_to_f16(codes[i].y, lo.z, lo.w);
                        int8x4_to_f16(codes[i].z, hi.x, hi.y);
                        int8x4_to_f16(codes[i].w, hi.z, hi.w);
                        *reinterpret_cast<uint4*>(dst + i * 2048 + at0) = lo;
                        *reinterpret_cast<uint4*>(dst + i * 2048 + at1) = hi;
                    }
                    load(i);
                }
                fence_proxy_async_smem();
                converted(g);
            }
        } else {
            // A thread's own places in shared memory, AHEAD stages of ROUNDS x 16 bytes: copies
            // are waited for stage by stage, where registers in flight all wait for the last.
            // (Registers took 14 % longer for 768 rows over 64 experts of 2048 x 4096. For pairs the
            // extra traffic and the fence behind the copies cost more: copies 14 % longer for 4096 x 11008 x 4096.)
            uint8_t* place = conv + CF::C_STAGES * CF::X_CONV + team * CF::AHEAD * CF::X_RAW + tid * 16;
            int slot_in = 0, slot_out = 0;
            auto load = [&]() {                                  // the team's next stage (an empty group past the last)
                if (live) {
                    const int k = kb * CF::KB + half;
                    const char* base = static_cast<const char*>(p.A) + k;
#pragma unroll
                    for (int i = 0; i < ROUNDS; ++i) {
                        if (i >= rounds) break;
                        const bool read = src[i] >= 0 && k < p.K;
                        cp_async_16(place + slot_in * CF::X_RAW + i * 1024,
                                    read ? base + static_cast<int64_t>(src[i]) * p.K : static_cast<const char*>(p.A), read ? 16u : 0u);
                    }
                    kb += CF::X_TEAMS / 2;
                    settle();
                }
                cp_async_commit();
                if (++slot_in == CF::AHEAD) slot_in = 0;
            };
#pragma unroll 1
            for (int i = 0; i < CF::AHEAD - 1; ++i) load();
            uint32_t g = team;
            int n = team >> 1;
            for (int at = unit; ok && cur.at<CF::BN, CF::CTAS>(p, sched, at, tile_channels, t); at += units) {
                const int now = t.n / (16 * CF::CTAS);
                for (; n < p.kstages; n += CF::X_TEAMS / 2, g += CF::X_TEAMS) {
                    load();
                    cp_async_wait<CF::AHEAD - 1>();              // this stage's copies (this thread's own) have landed
                    ok = slot_free(g);
                    if (!ok) break;
                    uint8_t* dst = conv + g % CF::C_STAGES * CF::X_CONV + sub * 128;
#pragma unroll
                    for (int i = 0; i < ROUNDS; ++i) {
                        if (i >= now) break;
                        const uint4 c = *reinterpret_cast<const uint4*>(place + slot_out * CF::X_RAW + i * 1024);
                        uint4 lo, hi;
                        int8x4_to_f16(c.x, lo.x, lo.y);
                        int8x4_to_f16(c.y, lo.z, lo.w);
                        int8x4_to_f16(c.z, hi.x, hi.y);
                        int8x4_to_f16(c.w, hi.z, hi.w);
                        *reinterpret_cast<uint4*>(dst + i * 2048 + at0) = lo;
                        *reinterpret_cast<uint4*>(dst + i * 2048 + at1) = hi;
                    }
                    fence_proxy_async_smem();
                    converted(g);
                    if (++slot_out == CF::AHEAD) slot_out = 0;
                }
                n -= p.kstages;
            }
            cp_async_wait<0>();                                  // nothing of this thread's is in flight when it leaves
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
