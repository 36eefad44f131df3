// adapter_beside.cuh -- many rows' adapters beside a product C, BF16 in and out: D = act(C + V . B_a^T + bias).
//
// Its bytes are C and D, so everything else is arranged around them: one persistent CTA an SM walks tiles of 128
// token rows (the MMA's rows) by 128 channels (its columns); C comes by TMA, four tiles ahead, is replaced in
// shared memory by the result and leaves by TMA. A step is one adapter of a tile: a slice of B_a, and beside it
// the tile's rows of V with zeros for other requests' rows; two or three steps are on their way. A CTA has
// an equal share of the tiles in an order that goes round the token tiles, so that token tiles of many
// adapters are shared out too.
// As in adapter_mma.cuh, B_a is looked at before it is used: a zero does not hide a number that is not finite, and the two
// numbers of V may have opposite signs. The masked rows and the look are the work of warps of their own, 2.3 us a
// tile. Where all rows of a token tile have the same adapter V needs no zeros and comes by TMA as it is.
// 4096 x 11008, 8 adapters of rank 32 in runs of rows, SiLU and bias: 64-67 us with the launch that computes V (10-12 of
// them); the bytes take 33. The epilogue computes for 26 of a CTA's 40 us (two operations of the special function unit a
// value; 17 without an activation); the rest are waits for C and for sums of token tiles of several adapters.
// (Tried and measured when this form was made: that case by the prompt form of adapter_mma.cuh, which has C and D by
// registers, 116 us; every token tile's channels in one run, the tile of many adapters last, 222; V of every tile by
// the warps 80; sums read from Tensor Memory a part ahead, with more registers for it, 80 against 67.)
// Warps: 0 TMA producer, 1 MMA issuer and owner of the Tensor Memory, 2 TMA stores, 3 idle, 4-11 and 12-19 epilogue
// (every second tile each: one tile's chain of waits beside the other's),
// 20-27 masked rows of V and the look at B.
#pragma once

#include "adapter_mma.cuh"

namespace dg {
namespace adapters {

struct Beside {
    static constexpr int ROWS = 128, COLS = 128, SL = 64, BOX = ROWS * 128;       // a box: 64 columns of 128 rows
    static constexpr int B_BYTES = COLS * 128, C_STAGES = 4, C_BYTES = 2 * BOX, ACCS = 4, MOST_B_STAGES = 3;
    static constexpr int EPI_WARP0 = 4, EPI_WARPS = 8, EPI_TEAMS = 2, V_WARP0 = EPI_WARP0 + EPI_TEAMS * EPI_WARPS, V_WARPS = 8, THREADS = 32 * (V_WARP0 + V_WARPS);
    static constexpr int MARKS = 8;      // tiles that may be between their V or their sum and their epilogue: ACCS + B_STAGES at most
    static constexpr int BAR_BYTES = 768;
    // Steps on their way. With rank 16 or 32 both numbers of V fit into one slice as they stand in memory (the second ones on a
    // step of the MMA), and a third step into the memory of two: rank 32, 4096 x 11008, 8 requests in runs 71 -> 66 us, every
    // row another of 48 747 -> 547.
    template <bool NARROW>
    struct Steps {
        static constexpr int B_STAGES = NARROW ? 3 : 2, V_BYTES = NARROW ? BOX : 2 * BOX;
        static constexpr int BYTES = B_STAGES * (V_BYTES + B_BYTES);
    };
    static constexpr int SMEM = 1024 + Steps<true>::BYTES + C_STAGES * C_BYTES + BAR_BYTES;
    static_assert(Steps<true>::BYTES == Steps<false>::BYTES, "the same shared memory");
    static constexpr uint32_t IDESC = make_idesc(1u, false, false, 128, 128);
    static_assert((3 * MOST_B_STAGES + 3 * C_STAGES + 2 * ACCS + MARKS + 1) * 8 + 8 + MARKS * (V_WARPS + 4) <= BAR_BYTES, "barriers fit");
    static_assert(SMEM <= 232448 && V_WARPS == 8, "shared memory; a tile's marks are one 64-bit word");
};

// A CTA's tiles, in order: token tiles first, then channels. (Steps, not divisions: sixteen warps take them for every tile.)
struct BesideTiles {
    int left, next_tt, next_ch, tt, ch;
    __device__ __forceinline__ explicit BesideTiles(const Params& p) {
        const int64_t all = static_cast<int64_t>(p.tiles) * p.ctiles;
        const int at = static_cast<int>(all * blockIdx.x / gridDim.x), column = at / p.tiles;
        left = static_cast<int>(all * (blockIdx.x + 1) / gridDim.x) - at;
        next_tt = at - column * p.tiles;
        next_ch = column * Beside::COLS;
        tt = ch = 0;
    }
    __device__ __forceinline__ bool next(const Params& p) {
        if (left == 0) return false;
        --left;
        tt = next_tt;
        ch = next_ch;
        if (++next_tt == p.tiles) {
            next_tt = 0;
            next_ch += Beside::COLS;
        }
        return true;
    }
};

template <bool NARROW>
__global__ void __launch_bounds__(Beside::THREADS, 1)
    adapter_beside(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmD,
                   const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ Params p) {
    using Steps = Beside::Steps<NARROW>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* v_rows = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* b_ring = v_rows + Steps::B_STAGES * Steps::V_BYTES;
    uint8_t* c_ring = b_ring + Steps::B_STAGES * Beside::B_BYTES;
    uint64_t* b_full = reinterpret_cast<uint64_t*>(c_ring + Beside::C_STAGES * Beside::C_BYTES);
    uint64_t* ready = b_full + Steps::B_STAGES;          // B has been looked at, V is there
    uint64_t* b_empty = ready + Steps::B_STAGES;         // and both have been used
    uint64_t* c_full = b_empty + Steps::B_STAGES;
    uint64_t* c_done = c_full + Beside::C_STAGES;         // the result stands in C's place
    uint64_t* c_empty = c_done + Beside::C_STAGES;        // and has left
    uint64_t* acc_full = c_empty + Beside::C_STAGES;
    uint64_t* acc_empty = acc_full + Beside::ACCS;
    uint64_t* looked = acc_empty + Beside::ACCS;          // [MARKS] the n-th tile with adapters: its slices of B have been looked at
    uint64_t* drain = looked + Beside::MARKS;
    uint64_t* dirty = drain + 1;                          // [MARKS] a byte for every warp that looked
    int* mark_of = reinterpret_cast<int*>(dirty + Beside::MARKS);   // [MARKS] which of the tiles with adapters a tile is, -1: none
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mark_of + Beside::MARKS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunks_r = NARROW ? 1 : (p.r + Beside::SL - 1) / Beside::SL;       // steps of one adapter
    const int second = NARROW ? p.r * 2 : Beside::BOX;               // bytes from a row's first numbers of V to its second
    BesideTiles tile(p);
    if (threadIdx.x == 0) {
        for (int s = 0; s < Steps::B_STAGES; ++s) {
            mbar_init(&b_full[s], 1);
            mbar_init(&ready[s], Beside::V_WARPS);
            mbar_init(&b_empty[s], 1);
        }
        for (int s = 0; s < Beside::C_STAGES; ++s) {
            mbar_init(&c_full[s], 1);
            mbar_init(&c_done[s], Beside::EPI_WARPS);
            mbar_init(&c_empty[s], 1);
        }
        for (int s = 0; s < Beside::ACCS; ++s) {
            mbar_init(&acc_full[s], 2);             // the MMAs, and the word on the tile's adapters
            mbar_init(&acc_empty[s], Beside::EPI_WARPS);
        }
        for (int s = 0; s < Beside::MARKS; ++s) mbar_init(&looked[s], Beside::V_WARPS);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        if (p.C) tma_prefetch_desc(&tmC);
        tma_prefetch_desc(&tmD);
        if (p.L > 0) {
            tma_prefetch_desc(&tmB);
            tma_prefetch_desc(&tmV);
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    grid_dependency_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0) grid_launch_dependents();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        const uint64_t pol = policy_evict_last(), pol_c = policy_evict_first();
        int64_t c_count = 0, b_count = 0;
        bool ok = true, stalled = false;
        TileAdapters ta;
        bool live = tile.next(p);
        if (live) ta.look_ahead(p, tile.tt);
        while (ok && !stalled && live) {
            const int tt = tile.tt, ch = tile.ch;
            ta.open(p, tt);
            live = tile.next(p);
            if (live) ta.look_ahead(p, tile.tt);
            if (p.C) {
                stalled = c_count + b_count == p.stall_after;
                if (stalled) break;
                const int s = static_cast<int>(c_count % Beside::C_STAGES);
                ok = mbar_wait_warp(&c_empty[s], static_cast<uint32_t>((c_count / Beside::C_STAGES) & 1) ^ 1, abort_flag, p.wait_ns);
                if (!ok) break;
                if (elect_one()) {
                    uint8_t* to = c_ring + s * Beside::C_BYTES;
                    const bool two = ch + Beside::SL < p.N;
                    mbar_arrive_expect_tx(&c_full[s], two ? 2 * Beside::BOX : Beside::BOX);
                    const uint32_t bar = smem_u32(&c_full[s]);
                    tma_load_nd<false>(to, &tmC, bar, ch, tt * Beside::ROWS, pol_c);
                    if (two) tma_load_nd<false>(to + Beside::BOX, &tmC, bar, ch + Beside::SL, tt * Beside::ROWS, pol_c);
                }
                __syncwarp();
                ++c_count;
            }
            for (int a = ta.next(); ok && !stalled && a >= 0; a = ta.next()) {
                for (int i = 0; i < chunks_r; ++i) {
                    stalled = c_count + b_count == p.stall_after;
                    if (stalled) break;
                    const int s = static_cast<int>(b_count % Steps::B_STAGES);
                    ok = mbar_wait_warp(&b_empty[s], static_cast<uint32_t>((b_count / Steps::B_STAGES) & 1) ^ 1, abort_flag, p.wait_ns);
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t bar = smem_u32(&b_full[s]);
                        mbar_arrive_expect_tx(&b_full[s], Beside::B_BYTES + (ta.uniform ? Steps::V_BYTES : 0));
                        tma_load_nd<false>(b_ring + s * Beside::B_BYTES, &tmB, bar, i * Beside::SL, ch, 0, a, pol);
                        if (ta.uniform) {
                            uint8_t* to = v_rows + s * Steps::V_BYTES;
                            if constexpr (NARROW) tma_load_nd<false>(to, &tmV, bar, 0, tt * Beside::ROWS, pol);
                            else tma_load_nd<false>(to, &tmV, bar, i * Beside::SL, tt * Beside::ROWS, 0, pol);
                        }
                    }
                    __syncwarp();
                    ++b_count;
                }
            }
        }
        if (!ok && lane == 0) experts::fail(p, ERR_TIMEOUT_PRODUCER, abort_flag);
        // every copy issued has landed before the CTA leaves
        for (int s = 0; s < Beside::C_STAGES; ++s) {
            const int64_t cnt = c_count > s ? (c_count - s + Beside::C_STAGES - 1) / Beside::C_STAGES : 0;
            if (cnt > 0 && !mbar_wait_warp(&c_full[s], static_cast<uint32_t>((cnt - 1) & 1), nullptr, p.wait_ns) && lane == 0)
                experts::fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
        }
        for (int s = 0; s < Steps::B_STAGES; ++s) {
            const int64_t cnt = b_count > s ? (b_count - s + Steps::B_STAGES - 1) / Steps::B_STAGES : 0;
            if (cnt > 0 && !mbar_wait_warp(&b_full[s], static_cast<uint32_t>((cnt - 1) & 1), nullptr, p.wait_ns) && lane == 0)
                experts::fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        const uint32_t acc0 = __shfl_sync(kAllLanes, tmem, 0);
        const uint64_t vd0 = smem_desc_sw128(smem_u32(v_rows), 16, 1024), bd0 = smem_desc_sw128(smem_u32(b_ring), 16, 1024);
        int64_t steps_done = 0;
        int local = 0, marks = 0;
        bool ok = true;
        TileAdapters ta;
        bool live = tile.next(p);
        if (live) ta.look_ahead(p, tile.tt);
        for (; ok && live; ++local) {
            ta.open(p, tile.tt);
            live = tile.next(p);
            if (live) ta.look_ahead(p, tile.tt);
            const int buf = local % Beside::ACCS;
            ok = mbar_wait_warp(&acc_empty[buf], ((local / Beside::ACCS) & 1) ^ 1, abort_flag, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = acc0 + static_cast<uint32_t>(buf * Beside::COLS);
            uint32_t more = 0;
            for (int a = ta.next(); ok && a >= 0; a = ta.next()) {
                for (int i = 0; i < chunks_r; ++i) {
                    const int s = static_cast<int>(steps_done % Steps::B_STAGES);
                    ok = mbar_wait_warp(&ready[s], static_cast<uint32_t>((steps_done / Steps::B_STAGES) & 1), abort_flag, p.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vd = vd0 + s * (Steps::V_BYTES >> 4), bd = bd0 + s * (Beside::B_BYTES >> 4);
                    const int steps = (min(Beside::SL, p.r - i * Beside::SL) + 15) / 16;
                    if (elect_one()) {
                        for (int part = 0; part < 2; ++part)
                            for (int k = 0; k < steps; ++k) {
                                mma_bf16(acc, vd + part * (second >> 4) + k * 2, bd + k * 2, Beside::IDESC, more);
                                more = 1;
                            }
                        mma_commit(&b_empty[s]);
                    }
                    __syncwarp();
                    more = 1;
                    ++steps_done;
                }
            }
            if (!ok) break;
            if (elect_one()) {
                mma_commit(&acc_full[buf]);
                mark_of[local % Beside::MARKS] = more ? marks : -1;
                mbar_arrive(&acc_full[buf]);
            }
            marks += more;
            __syncwarp();
        }
        if (elect_one()) {
            if (!ok) experts::fail(p, ERR_TIMEOUT_MMA, abort_flag);
            mma_commit(drain);
            if (!mbar_wait(drain, 0, nullptr, p.wait_ns)) experts::fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---------------------------------------------------------------- stores of finished tiles
        // A place in the ring is free again when its store has read it.
        int local = 0;
        bool ok = true;
        for (; ok && tile.next(p); ++local) {
            const int s = local % Beside::C_STAGES, tt = tile.tt, ch = tile.ch;
            ok = mbar_wait_warp(&c_done[s], (local / Beside::C_STAGES) & 1, abort_flag, p.wait_ns);
            if (!ok) break;
            if (lane == 0) {
                const uint8_t* from = c_ring + s * Beside::C_BYTES;
                tma_store_2d(&tmD, from, ch, tt * Beside::ROWS);
                if (ch + Beside::SL < p.N) tma_store_2d(&tmD, from + Beside::BOX, ch + Beside::SL, tt * Beside::ROWS);
                bulk_commit();
                bulk_wait_read<0>();
                mbar_arrive(&c_empty[s]);
            }
            __syncwarp();
        }
        if (!ok && lane == 0) experts::fail(p, ERR_TIMEOUT_EPILOGUE, abort_flag);
        if (lane == 0) bulk_wait_all();         // the results have been written when the CTA leaves
        __syncwarp();
    } else if (warp >= Beside::EPI_WARP0 && warp < Beside::V_WARP0) {
        // ---------------------------------------------------------------- epilogue
        // A thread has one token row and 64 of its channels, 16 at a time.
        const int ew = (warp - Beside::EPI_WARP0) % Beside::EPI_WARPS, team = (warp - Beside::EPI_WARP0) / Beside::EPI_WARPS;
        const int quarter = warp & 3, part = ew >> 2, row = quarter * 32 + lane, swizzle = row & 7;
        const bool bias_vec = p.bias && (reinterpret_cast<uintptr_t>(p.bias) & 15) == 0;
        int local = 0;
        bool ok = true;
        for (; ok && tile.next(p); ++local) {
            if (p.bias && lane < 2 && tile.ch + part * 64 + lane * 32 < p.N)        // (of the other team's tile too: a line may serve both)
                asm volatile("prefetch.global.L1 [%0];" ::"l"(p.bias + tile.ch + part * 64 + lane * 32));
            if (local % Beside::EPI_TEAMS != team) continue;
            const int s = local % Beside::C_STAGES, buf = local % Beside::ACCS;
            const int ch = tile.ch + part * 64, t = tile.tt * Beside::ROWS + row;
            if (p.C) ok = mbar_wait_warp(&c_full[s], (local / Beside::C_STAGES) & 1, abort_flag, p.wait_ns);
            else ok = mbar_wait_warp(&c_empty[s], ((local / Beside::C_STAGES) & 1) ^ 1, abort_flag, p.wait_ns);
            if (!ok) break;
            ok = mbar_wait_warp(&acc_full[buf], (local / Beside::ACCS) & 1, abort_flag, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const int mark = mark_of[local % Beside::MARKS];
            const bool some = mark >= 0;
            bool found = false;
            if (some) {
                ok = mbar_wait_warp(&looked[mark % Beside::MARKS], (mark / Beside::MARKS) & 1, abort_flag, p.wait_ns);
                if (!ok) break;
                found = dirty[mark % Beside::MARKS] != 0;
            }
            uint8_t* at = c_ring + s * Beside::C_BYTES + part * Beside::BOX + row * 128;
            const int a = found && t < p.T ? adapter_of(p, t) : -1;
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
                uint32_t r[16];
                if (!some) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) r[j] = 0;
                } else {
                    tmem_ld16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * Beside::COLS + part * 64 + h * 16, r);
                    tmem_ld_wait();
                }
                if (h == 3) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_relaxed(&acc_empty[buf]);
                }
                uint4* place[2];
                uint32_t c[8];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    place[k] = reinterpret_cast<uint4*>(at + (((h * 2 + k) ^ swizzle) << 4));
                    const uint4 x = p.C ? *place[k] : make_uint4(0, 0, 0, 0);
                    c[4 * k] = x.x, c[4 * k + 1] = x.y, c[4 * k + 2] = x.z, c[4 * k + 3] = x.w;
                }
                float v[16];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    add2(v[2 * j], v[2 * j + 1], bf16_lo(c[j]), bf16_hi(c[j]), __uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                if (bias_vec && ch + h * 16 + 16 <= p.N) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 b = __ldg(reinterpret_cast<const float4*>(p.bias + ch + h * 16) + j);
                        add2(v[4 * j], v[4 * j + 1], v[4 * j], v[4 * j + 1], b.x, b.y);
                        add2(v[4 * j + 2], v[4 * j + 3], v[4 * j + 2], v[4 * j + 3], b.z, b.w);
                    }
                } else if (p.bias) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] += ch + h * 16 + j < p.N ? __ldg(p.bias + ch + h * 16 + j) : 0.0f;
                }
                if (found) {
#pragma unroll 1
                    for (int j = 0; j < 16; ++j) {
                        const int n = ch + h * 16 + j;
                        const float more = a >= 0 && n < p.N ? not_finite_terms(p, t, a, n) : 0.0f;
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] += k == j ? more : 0.0f;
                    }
                }
                activate(v, p.act);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    *place[k] = make_uint4(pack_bf16x2(v[8 * k], v[8 * k + 1]), pack_bf16x2(v[8 * k + 2], v[8 * k + 3]),
                                           pack_bf16x2(v[8 * k + 4], v[8 * k + 5]), pack_bf16x2(v[8 * k + 6], v[8 * k + 7]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_done[s]);
        }
        if (!ok && lane == 0) experts::fail(p, ERR_TIMEOUT_EPILOGUE, abort_flag);
        __syncwarp();
    } else if (warp >= Beside::V_WARP0) {
        // ---------------------------------------------------------------- masked rows of V, a look at B
        // Two threads share a token row, one has its first numbers and one its second, and a channel of B, half of its
        // slice each. A row's V is loaded ahead (up to rank 64).
        const int row = (threadIdx.x - 32 * Beside::V_WARP0) & 127, part = (threadIdx.x - 32 * Beside::V_WARP0) >> 7, swizzle = row & 7;
        int64_t step = 0;
        int marks = 0, had = -1, own = -1;           // had: the token tile whose V is loaded
        bool ok = true;
        constexpr int VECS = NARROW ? 4 : 8;
        uint4 v[VECS];
        TileAdapters ta;
        bool live = tile.next(p);
        if (live) ta.look_ahead(p, tile.tt);
        while (ok && live) {
            const int tt = tile.tt, t = tt * Beside::ROWS + row;
            const uint4* src = reinterpret_cast<const uint4*>(v_row(p, t)) + part * (p.r / 8);
            auto load = [&](int i, int vecs) {
#pragma unroll
                for (int c = 0; c < VECS; ++c) {
                    v[c] = make_uint4(0, 0, 0, 0);
                    if (own >= 0 && c < vecs) v[c] = __ldcg(src + i * 8 + c);
                }
            };
            ta.open(p, tt);
            live = tile.next(p);
            if (live) ta.look_ahead(p, tile.tt);
            if (tt != had && !ta.uniform) {              // (uniform: V comes with B)
                own = t < p.T && p.L > 0 ? adapter_of(p, t) : -1;
                if (chunks_r == 1) load(0, p.r / 8);
                had = tt;
            }
            bool found = false;
            for (int a = ta.next(); ok && a >= 0; a = ta.next()) {
                for (int i = 0; i < chunks_r; ++i) {
                    const int s = static_cast<int>(step % Steps::B_STAGES);
                    const int vecs = min(Beside::SL, p.r - i * Beside::SL) / 8, steps = (vecs + 1) / 2;
                    if (chunks_r > 1 && !ta.uniform) load(i, vecs);
                    ok = mbar_wait_warp(&b_full[s], static_cast<uint32_t>((step / Steps::B_STAGES) & 1), abort_flag, p.wait_ns);
                    if (!ok) break;
                    if (!ta.uniform) {
                        // (B was copied after the stage's last step had been used: its rows of V are free too)
                        uint8_t* to = v_rows + s * Steps::V_BYTES + (NARROW ? 0 : part * second) + row * 128;
                        const int c0 = NARROW ? part * (second / 16) : 0;
                        const bool hit = own == a;
#pragma unroll
                        for (int c = 0; c < VECS; ++c)
                            if (c < 2 * steps) *reinterpret_cast<uint4*>(to + (((c0 + c) ^ swizzle) << 4)) = hit ? v[c] : make_uint4(0, 0, 0, 0);
                    }
                    found = make_finite(b_ring + s * Beside::B_BYTES + row * 128, swizzle, 4 * part, min(vecs, 4 * part + 4)) || found;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ready[s]);
                    __syncwarp();
                    ++step;
                }
            }
            if (ok && ta.count > 0) {
                const int any = __any_sync(kAllLanes, found);
                if (lane == 0) {
                    reinterpret_cast<uint8_t*>(dirty + marks % Beside::MARKS)[warp - Beside::V_WARP0] = static_cast<uint8_t>(any);
                    mbar_arrive(&looked[marks % Beside::MARKS]);
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
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace adapters
}  // namespace dg
