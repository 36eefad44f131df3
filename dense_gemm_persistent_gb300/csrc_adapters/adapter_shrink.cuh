// adapter_shrink.cuh -- V[t] = s_a X[t] . A_a^T for every row with an adapter.
#pragma once

#include <climits>

#include "adapter_common.cuh"

namespace dg {
namespace adapters {

// Few rows, by FP32 units: a CTA computes RB numbers of one row; its threads share K, partial sums meet in shared
// memory. Its loads go out in batches of U steps, whether there are as many or not: with a remainder loop
// most calls waited for every step. CTAs behind the rows' write the lists of the prompt form's token tiles.
template <int RB, int U, int SHRINK_THREADS>
__global__ void __launch_bounds__(SHRINK_THREADS) adapter_shrink_few(const __grid_constant__ Params p) {
    __shared__ float part[SHRINK_THREADS / 32][RB];
    __shared__ unsigned words[kWords];
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    const int blocks = p.r / RB;
    if (static_cast<int>(blockIdx.x) >= p.T * blocks) {
        list_tile(p, static_cast<int>(blockIdx.x) - p.T * blocks, words, threadIdx.x, SHRINK_THREADS, []() { __syncthreads(); });
        return;
    }
    const int t = static_cast<int>(blockIdx.x) / blocks, j0 = (static_cast<int>(blockIdx.x) - t * blocks) * RB;
    const int a = adapter_of(p, t);
    if (a < 0) return;
    const uint4* x = reinterpret_cast<const uint4*>(p.X + static_cast<int64_t>(t) * p.K);
    const uint4* w = reinterpret_cast<const uint4*>(p.low + (static_cast<int64_t>(a) * p.r + j0) * p.K);
    const int vecs = p.K / 8;
    float s0[RB], s1[RB];
#pragma unroll
    for (int j = 0; j < RB; ++j) s0[j] = s1[j] = 0.0f;
    for (int i0 = threadIdx.x; i0 < vecs; i0 += U * SHRINK_THREADS) {
        uint4 xv[U], wv[U][RB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * SHRINK_THREADS;
            const bool there = i < vecs;
            xv[u] = there ? __ldg(x + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < RB; ++j) wv[u][j] = there ? __ldg(w + static_cast<int64_t>(j) * vecs + i) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float4 x0 = make_float4(bf16_lo(xv[u].x), bf16_hi(xv[u].x), bf16_lo(xv[u].y), bf16_hi(xv[u].y));
            const float4 x1 = make_float4(bf16_lo(xv[u].z), bf16_hi(xv[u].z), bf16_lo(xv[u].w), bf16_hi(xv[u].w));
#pragma unroll
            for (int j = 0; j < RB; ++j) fma8(s0[j], s1[j], wv[u][j], x0, x1);
        }
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j < RB; ++j) {
        float s = s0[j] + s1[j];
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAllLanes, s, o);
        if (lane == 0) part[warp][j] = s;
    }
    __syncthreads();
    if (threadIdx.x < RB) {
        float s = 0.0f;
        for (int i = 0; i < SHRINK_THREADS / 32; ++i) s += part[i][threadIdx.x];
        if (p.scale) s *= p.scale[a];
        const int j = j0 + threadIdx.x;
        store_one(p, t, j, s);
    }
}

// Many rows, on the tensor core. A tile is 128 rows of X (the MMA's rows); its columns are the
// rows of A of every adapter that the tile's rows have, stacked, up to 256 a pass: X is read
// once whatever the mix, and a row takes the columns of its own adapter from its accumulator. A
// cluster of `split` CTAs shares K; the parts meet in shared memory and are added in
// their order.
// Rows whose adapter has less than 4 rows among their 32 neighbours (sequences that decode, next to prompts) are left
// out where a tile has up to 32 of them: each would bring its whole A through one cluster, and 24 of
// them held up a prompt of 4096 for 18 us (rank 64). They are FP32 sums, shared out over the launch.
// Warps: 0 TMA producer, 1 MMA issuer, 2-5 accumulator to V, 6-9 single rows and, for the prompt form, the
// adapters of its token tiles.
struct Shrink {
    static constexpr int ROWS = 128, SL = 64, KS = 2, SLICE_X = ROWS * 128, X_BYTES = KS * SLICE_X;
    static constexpr int MOST_COLS = 256, MOST_STAGES = 6, MOST_SPLIT = 8;
    static constexpr int EPI_WARP0 = 2, HELP_WARP0 = 6, THREADS = 320, HELPERS = 128;
    static constexpr int TMEM_COLS = 256, WORDS = kWords;
    static constexpr int FEW = 4, MOST_SINGLE = 32, SINGLE_N = 4, BATCH = 32, WINDOW = 512;      // single rows: see above; tiles looked at together, shared
    static constexpr int TABLES = 2 * WORDS * 4 + 2 * ROWS * 4 + BATCH * 16, BAR_BYTES = 256;
    static constexpr uint32_t IDESC0 = make_idesc(1u, false, false, 128, 0);
    static constexpr int stage_bytes(int cols) { return X_BYTES + KS * cols * 128; }
    static constexpr int smem_bytes(int cols, int stages, int rank) {
        return 1024 + stages * stage_bytes(cols) + rank * ROWS * 4 + TABLES + BAR_BYTES;
    }
    static_assert((2 * MOST_STAGES + 3) * 8 + 12 <= BAR_BYTES, "barriers fit");
};

// Bits of the rows of a warp's 32 (a: their adapters) that are single.
__device__ __forceinline__ unsigned single_rows(int a) {
    const unsigned same = __match_any_sync(kAllLanes, a);
    return __ballot_sync(kAllLanes, a >= 0 && __popc(same) < Shrink::FEW);
}

// Four numbers of V of one row by a warp. (Eight took twice the time: half the loads of X and A on their way.)
__device__ __forceinline__ void single_row(const Params& p, int t, int at) {
    constexpr int N = Shrink::SINGLE_N, U = 4;
    const int lane = threadIdx.x & 31, a = adapter_of(p, t), vecs = p.K / 8;
    const uint4* x = reinterpret_cast<const uint4*>(p.X + static_cast<int64_t>(t) * p.K);
    const uint4* w = reinterpret_cast<const uint4*>(p.low + (static_cast<int64_t>(a) * p.r + at) * p.K);
    float s0[N], s1[N];
#pragma unroll
    for (int j = 0; j < N; ++j) s0[j] = s1[j] = 0.0f;
    for (int i0 = lane; i0 < vecs; i0 += 32 * U) {
        uint4 xv[U], wv[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + 32 * u;
            const bool there = i < vecs;
            xv[u] = there ? __ldg(x + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < N; ++j) wv[u][j] = there ? __ldg(w + static_cast<int64_t>(j) * vecs + i) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float4 x0 = make_float4(bf16_lo(xv[u].x), bf16_hi(xv[u].x), bf16_lo(xv[u].y), bf16_hi(xv[u].y));
            const float4 x1 = make_float4(bf16_lo(xv[u].z), bf16_hi(xv[u].z), bf16_lo(xv[u].w), bf16_hi(xv[u].w));
#pragma unroll
            for (int j = 0; j < N; ++j) fma8(s0[j], s1[j], wv[u][j], x0, x1);
        }
    }
    const float scale = p.scale ? p.scale[a] : 1.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        float v = s0[j] + s1[j];
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAllLanes, v, o);
        if (lane == 0) store_one(p, t, at + j, v * scale);
    }
}

// The single rows of a window of tiles: an item is a row's four numbers, the items of a tile go round the warps of the
// window's CTAs. (Each of them looks at the window's rows: over the whole of a long launch that would grow with the
// square of the rows.) masks: [BATCH][4], the single rows of a tile.
template <class Sync>
__device__ __forceinline__ void share_single_rows(const Params& p, uint4* masks, int warp, Sync sync) {
    const int lane = threadIdx.x & 31, groups = p.r / Shrink::SINGLE_N;
    const int begin = static_cast<int>(blockIdx.x) / p.split / Shrink::WINDOW * Shrink::WINDOW, end = min(begin + Shrink::WINDOW, p.shrink_tiles);
    const int all = (end - begin) * p.split * 4, me = (static_cast<int>(blockIdx.x) - begin * p.split) * 4 + warp;
    for (int base = begin; base < end; base += Shrink::BATCH) {
        // (four tiles' rows are loaded together)
        for (int k0 = warp; k0 < Shrink::BATCH && base + k0 < end; k0 += 16) {
            int a[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int t = (base + k0 + 4 * k) * Shrink::ROWS + b * 32 + lane;
                    a[k][b] = t < p.T ? adapter_of(p, t) : -1;
                }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                unsigned m[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) m[b] = single_rows(a[k][b]);
                if (lane == 0) masks[k0 + 4 * k] = make_uint4(m[0], m[1], m[2], m[3]);
            }
        }
        sync();
        const bool there = base + lane < end;
        const uint4 m = there ? masks[lane] : make_uint4(0, 0, 0, 0);
        int rows = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
        if (rows > Shrink::MOST_SINGLE) rows = 0;
        const int first = ((me - (base + lane) * 61) % all + all) % all;      // (another warp begins at each tile)
        for (unsigned todo = __ballot_sync(kAllLanes, first < rows * groups); todo; todo &= todo - 1) {
            const int l = __ffs(todo) - 1, n = __shfl_sync(kAllLanes, rows, l) * groups;
            unsigned mk[4] = {__shfl_sync(kAllLanes, m.x, l), __shfl_sync(kAllLanes, m.y, l), __shfl_sync(kAllLanes, m.z, l),
                              __shfl_sync(kAllLanes, m.w, l)};
            for (int item = __shfl_sync(kAllLanes, first, l); item < n; item += all) {
                int j = item / groups, row = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {           // the j-th bit
                    const int c = __popc(mk[b]);
                    if (j >= 0 && j < c) row = 32 * b + static_cast<int>(__fns(mk[b], 0, j + 1));
                    j = j < c ? -1 : j - c;
                    if (j < 0) j = INT_MIN / 2;
                }
                single_row(p, (base + l) * Shrink::ROWS + row, item % groups * Shrink::SINGLE_N);
            }
        }
        sync();
    }
}

__global__ void __launch_bounds__(Shrink::THREADS, 1)
    adapter_shrink_many(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = p.stages, split = p.split, slice_a = p.shrink_cols * 128, stage_bytes = Shrink::X_BYTES + Shrink::KS * slice_a;
    float* park = reinterpret_cast<float*>(ring + S * stage_bytes);                    // [r][128]
    unsigned* words = reinterpret_cast<unsigned*>(park + p.r * Shrink::ROWS);
    unsigned* help_words = words + Shrink::WORDS;
    int* list = reinterpret_cast<int*>(help_words + Shrink::WORDS);                    // [128] adapters of this tile
    int* slot_of = list + Shrink::ROWS;                                                // [128] of a row's adapter there, -1
    uint4* masks = reinterpret_cast<uint4*>(slot_of + Shrink::ROWS);
    uint64_t* full = reinterpret_cast<uint64_t*>(masks + Shrink::BATCH);
    uint64_t* empty = full + S;
    uint64_t* acc_full = empty + S;
    uint64_t* acc_empty = acc_full + 1;
    uint64_t* drain = acc_empty + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* singles = reinterpret_cast<int*>(tmem_slot + 2);                              // single rows of this tile

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x) % split, row0 = static_cast<int>(blockIdx.x) / split * Shrink::ROWS;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.kstages) * rank / split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.kstages) * (rank + 1) / split);

    for (int w = threadIdx.x; w < Shrink::WORDS; w += Shrink::THREADS) words[w] = 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 4);
        mbar_init(drain, 1);
        *abort_flag = 0;
        *singles = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmA);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Shrink::TMEM_COLS);
        tmem_relinquish();
    }
    __syncthreads();
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    // the adapters of this tile's rows, in order; a thread of the accumulator's warps has the row that
    // its lane of the accumulator is (a warp reads the quarter that its number says)
    const int at = (warp & 3) * 32 + lane;
    int mine = -1, slot = -1;
    bool single = false;
    if (warp >= Shrink::EPI_WARP0 && warp < Shrink::HELP_WARP0) {
        if (row0 + at < p.T) mine = adapter_of(p, row0 + at);
        const unsigned who = single_rows(mine);
        single = (who >> lane) & 1;
        if (lane == 0 && who) atomicAdd(singles, __popc(who));
    }
    __syncthreads();
    if (single && *singles <= Shrink::MOST_SINGLE) mine = -1;
    if (mine >= 0) atomicOr(&words[mine >> 5], 1u << (mine & 31));
    __syncthreads();
    if (warp >= Shrink::EPI_WARP0 && warp < Shrink::HELP_WARP0) {
        if (mine >= 0) {
            slot = place_of(p, words, mine);
            list[slot] = mine;
        }
        slot_of[at] = slot;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int count = marked(p, words), per_pass = p.shrink_cols / p.r, passes = (count + per_pass - 1) / per_pass;

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        const uint64_t pol = policy_evict_last();
        uint32_t stage = 0, phase = 0;
        int64_t issued = 0;
        bool ok = true, stalled = false;
        for (int pass = 0; ok && !stalled && pass < passes; ++pass) {
            const int first = pass * per_pass, n = min(per_pass, count - first);
            for (int kb = kb0; kb < kb1; ++kb) {
                stalled = issued == p.stall_after;
                if (stalled) break;
                ok = mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag, p.wait_ns);
                if (!ok) break;
                if (elect_one()) {
                    uint8_t* x = ring + stage * stage_bytes;
                    const uint32_t bar = smem_u32(&full[stage]);
                    mbar_arrive_expect_tx(&full[stage], Shrink::X_BYTES + Shrink::KS * n * p.r * 128);
                    const int k0 = kb * Shrink::KS * Shrink::SL;
                    if (p.k_whole) {
                        tma_load_nd<false>(x, &tmX, bar, 0, row0, kb * Shrink::KS, pol);
                    } else {
                        for (int s = 0; s < Shrink::KS; ++s)
                            tma_load_nd<false>(x + s * Shrink::SLICE_X, &tmX, bar, k0 + s * Shrink::SL, row0, pol);
                    }
                    for (int i = 0; i < n; ++i)
                        for (int s = 0; s < Shrink::KS; ++s)
                            tma_load_nd<false>(x + Shrink::X_BYTES + s * slice_a + i * p.r * 128, &tmA, bar, k0 + s * Shrink::SL, 0,
                                               list[first + i], pol);
                }
                __syncwarp();
                ++issued;
                if (++stage == static_cast<uint32_t>(S)) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok && lane == 0) experts::fail(p, ERR_TIMEOUT_PRODUCER, abort_flag);
        for (int s = 0; s < S; ++s) {
            const int64_t cnt = issued > s ? (issued - s + S - 1) / S : 0;
            if (cnt > 0 && !mbar_wait_warp(&full[s], static_cast<uint32_t>((cnt - 1) & 1), nullptr, p.wait_ns) && lane == 0)
                experts::fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        const uint32_t s0 = smem_u32(ring), acc = __shfl_sync(kAllLanes, tmem, 0);
        const uint64_t xd0 = smem_desc_sw128(s0, 16, 1024), ad0 = smem_desc_sw128(s0 + Shrink::X_BYTES, 16, 1024);
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        for (int pass = 0; ok && pass < passes; ++pass) {
            // (a rank of 8 may end inside a step of 16 columns: what lies there is in columns that no row takes)
            const int n = (min(per_pass, count - pass * per_pass) * p.r + 15) / 16 * 16;
            const uint32_t idesc = Shrink::IDESC0 | (static_cast<uint32_t>(n >> 3) << 17);
            ok = mbar_wait_warp(acc_empty, (pass & 1) ^ 1, abort_flag, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = mbar_wait_warp(&full[stage], phase, abort_flag, p.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const uint64_t xd = xd0 + stage * (stage_bytes >> 4), ad = ad0 + stage * (stage_bytes >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < Shrink::KS * 4; ++k)
                        mma_bf16(acc, xd + (k / 4) * (Shrink::SLICE_X >> 4) + (k % 4) * 2, ad + (k / 4) * (slice_a >> 4) + (k % 4) * 2, idesc,
                                 kb > kb0 || k > 0 ? 1u : 0u);
                    mma_commit(&empty[stage]);
                }
                __syncwarp();
                if (++stage == static_cast<uint32_t>(S)) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (ok && elect_one()) mma_commit(acc_full);
            __syncwarp();
        }
        if (elect_one()) {
            if (!ok) experts::fail(p, ERR_TIMEOUT_MMA, abort_flag);
            mma_commit(drain);
            if (!mbar_wait(drain, 0, nullptr, p.wait_ns)) experts::fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
        }
        __syncwarp();
    } else if (warp < Shrink::HELP_WARP0) {
        // ---------------------------------------------------------------- each row's own columns
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        bool ok = true;
        for (int pass = 0; pass < passes; ++pass) {
            ok = mbar_wait_warp(acc_full, pass & 1, abort_flag, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const int first = pass * per_pass, n = min(per_pass, count - first);
            for (int i = 0; i < n; ++i) {
                const bool take = slot == first + i;
                if (!__any_sync(kAllLanes, take)) continue;
                for (int j = 0; j < p.r; j += 8) {
                    uint32_t v[8];
                    tmem_ld8(lanes + i * p.r + j, v);
                    tmem_ld_wait();
                    if (take) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) park[(j + c) * Shrink::ROWS + at] = __uint_as_float(v[c]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty);
        }
        if (!ok && lane == 0) experts::fail(p, ERR_TIMEOUT_EPILOGUE, abort_flag);
    } else {
        auto sync = []() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(Shrink::HELPERS) : "memory"); };
        if (p.prompt)
            for (int tile = static_cast<int>(blockIdx.x); tile < p.tiles; tile += static_cast<int>(gridDim.x))
                list_tile(p, tile, help_words, threadIdx.x - 32 * Shrink::HELP_WARP0, Shrink::HELPERS, sync);
        share_single_rows(p, masks, warp - Shrink::HELP_WARP0, sync);
    }
    __syncwarp();
    if (split > 1) cluster_sync();
    else __syncthreads();
    // ---------------------------------------------------------------- the parts of a row together
    if (!*abort_flag) {
        const uint32_t parked = smem_u32(park);
        const int groups = p.r / 8;
        for (int i = threadIdx.x; i < (groups + split - 1) / split * Shrink::ROWS; i += Shrink::THREADS) {
            const int r128 = i % Shrink::ROWS, g = i / Shrink::ROWS * split + rank;
            if (g >= groups || slot_of[r128] < 0) continue;
            const float scale = p.scale ? p.scale[list[slot_of[r128]]] : 1.0f;
            // (all parts on their way before the first sum)
            float part[Shrink::MOST_SPLIT][8], v[8];
#pragma unroll
            for (int s = 0; s < Shrink::MOST_SPLIT; ++s) {
                if (s >= split) break;
                const uint32_t from = (split > 1 ? mapa_shared(parked, s) : parked) + (g * 8 * Shrink::ROWS + r128) * 4;
#pragma unroll
                for (int c = 0; c < 8; ++c) part[s][c] = ld_shared_cluster_f32(from + c * Shrink::ROWS * 4);
            }
#pragma unroll
            for (int s = 0; s < Shrink::MOST_SPLIT; ++s) {
                if (s >= split) break;
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] = s == 0 ? part[0][c] : v[c] + part[s][c];
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] *= scale;
            store_v(p, row0 + r128, g * 8, v);
        }
    }
    tc_fence_before();
    if (split > 1) cluster_sync();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, Shrink::TMEM_COLS);
    }
}

}  // namespace adapters
}  // namespace dg
