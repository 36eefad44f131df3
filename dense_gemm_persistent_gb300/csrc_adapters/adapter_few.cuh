// adapter_few.cuh -- the projection with adapters for tiles of up to 64 rows.
//
// The output channels are the MMA's rows, up to 128 (fewer where that spreads the weights over more SMs), the token
// rows its columns. A cluster of
// `split` CTAs shares a tile's K: each sums its part in Tensor Memory and writes every split-th row of it
// to the shared memory of the CTA that finishes those rows, from all parts in their order.
// V . B_a^T runs on the FP32 units of the epilogue's warps meanwhile: rows may be of as many requests as there are,
// and no row's product holds another's numbers. The rows that a CTA finishes are put in the order of
// their adapters; an item is some channels of one adapter, a run of B_a that a bulk copy brings
// to shared memory, for all of its rows. Every warp copies its own items, some ahead. It needs V, the rest
// does not: only these warps wait for the launch that computes it. (Warp-wide matrix
// instructions, m16n8k16 with V as two of the columns, were slower here: 64 rows of 11008 channels, rank
// 64, took 104 us with them and 42 on the FP32 units, otherwise the same.)
// Warps: 0 TMA producer, 1 MMA issuer and owner of the Tensor Memory, 2-9 epilogue.
#pragma once

#include <type_traits>

#include "adapter_common.cuh"

namespace dg {
namespace adapters {

struct Few {
    static constexpr int KS = 2, SL = 64;                 // 128-byte slices of K per stage, elements of a slice
    static constexpr int MOST_COLS = 64, MOST_STAGES = 8, MOST_SPLIT = 8;
    static constexpr int SLICE_W = 128 * 128, W_BYTES = KS * SLICE_W;
    static constexpr int EPI_WARP0 = 2, EPI_WARPS = 8, EPI_THREADS = 32 * EPI_WARPS, THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
    static constexpr int MOST_AHEAD = 4, TMEM_COLS = 64, BAR_BYTES = 512, GROUP_BYTES = 768;
    // channels of an item: at most 4 KB of B
    static __host__ __device__ constexpr int item_channels(int r) { return r <= 32 ? 64 : r <= 64 ? 32 : 16; }
    static constexpr uint32_t IDESC0 = make_idesc(1u, false, false, 128, 0);
    static constexpr int stage_bytes(int cols) { return W_BYTES + KS * cols * 128; }
    // the ring; rows that a CTA finishes: 128 results and V; items ahead
    static constexpr int smem_bytes(int cols, int stages, int split, int r, int ahead) {
        return 1024 + stages * stage_bytes(cols) + (cols + split - 1) / split * (512 + r * 4) +
               EPI_WARPS * ahead * item_channels(r) * r * 2 + GROUP_BYTES + BAR_BYTES;
    }
    // Items of B that a warp copies ahead: up to 128 KB of them in a CTA, 64 beside a product; the ring has what is left.
    static __host__ __device__ constexpr int items_ahead(int r, bool product) {
        const int n = (product ? 64 : 128) * 1024 / (EPI_WARPS * item_channels(r) * r * 2);
        return n < MOST_AHEAD ? n : MOST_AHEAD;
    }
    // the most that two stages need, or none
    static __host__ __device__ constexpr int most_bytes() {
        int most = 0;
        for (int r = 8; r <= DGEMM_MAX_ADAPTER_RANK; r += 8) {
            const int with = smem_bytes(MOST_COLS, 2, 1, r, items_ahead(r, true)), without = smem_bytes(MOST_COLS, 0, 1, r, items_ahead(r, false));
            most = with > most ? with : most;
            most = without > most ? without : most;
        }
        return most;
    }
    static_assert((2 * MOST_STAGES + EPI_WARPS * MOST_AHEAD + 2) * 8 + 8 <= BAR_BYTES, "barriers fit");
    // (a split divides the columns, a multiple of 16: all parts of a CTA's rows are MOST_COLS rows of 128 floats)
    static_assert(MOST_COLS * 512 <= 2 * (W_BYTES + KS * 16 * 128), "two stages hold the parts of a CTA's rows");
};
static_assert(Few::most_bytes() <= 232448, "two stages always fit");

template <int ACT>
__device__ __forceinline__ float activate_one(float v) {
    if constexpr (ACT == DGEMM_ACT_RELU) return experts::relu(v);
    else if constexpr (ACT == DGEMM_ACT_GELU) return experts::gelu(v);
    else if constexpr (ACT == DGEMM_ACT_SILU) return silu(v);
    else return v;
}

// The rows of a tile that a CTA finishes, one channel of D a thread: parts of the product in their order, C and
// adapter, bias, activation, one rounding. (A copy for every activation: with the choice inside, every
// one of them was computed for every value, 0.4 us a row.)
template <int ACT>
__device__ __forceinline__ void finish_rows(const Params& p, const float* parts, const float* beside, int own, int rank, int row0,
                                            int rows, int chan0, int tid) {
    constexpr bool GATED = ACT == DGEMM_ACT_SWIGLU;
    constexpr int OUT = GATED ? 64 : 128, STEP = Few::EPI_THREADS / OUT;
    const int oc = tid % OUT, ch = chan0 + oc, mine = (rows - rank + p.split - 1) / p.split;
    if (oc >= p.channels || ch >= p.wide) return;
    const float bias = p.bias ? __ldg(p.bias + ch) : 0.0f, bias_up = GATED && p.bias ? __ldg(p.bias + p.N / 2 + ch) : 0.0f;
    const int split = p.kstages > 0 ? p.split : 0;
    auto row = [&](int q, int splits) {
        const int c = rank + p.split * q;
        float v = beside[q * 128 + oc] + bias, u = 0.0f;
        if (GATED) u = beside[q * 128 + 64 + oc] + bias_up;
        const float* from = parts + q * 128 + oc;
        float product = 0.0f, product_up = 0.0f;
        for (int s = 0; s < splits; ++s, from += own * 128) {
            product += from[0];
            if (GATED) product_up += from[p.channels];
        }
        v += product;
        v = GATED ? silu(v) * (u + product_up) : activate_one<ACT>(v);
        const int64_t o = static_cast<int64_t>(row0 + c) * p.wide + ch;
        if (p.d_f32) static_cast<float*>(p.D)[o] = v;
        else static_cast<__nv_bfloat16*>(p.D)[o] = __float2bfloat16_rn(v);
    };
    // (the ends of the inner loop known where there is one part or none: rows then overlap)
    if (split == 0) {
#pragma unroll 4
        for (int q = tid / OUT; q < mine; q += STEP) row(q, 0);
    } else if (split == 1) {
#pragma unroll 4
        for (int q = tid / OUT; q < mine; q += STEP) row(q, 1);
    } else {
        for (int q = tid / OUT; q < mine; q += STEP) row(q, split);
    }
}

// V . B_a^T for CHANNELS channels and the `rows` rows of one adapter, by one warp. L = 2^LG lanes share a channel (r / 8,
// rounded up to a power of two); the sums over them are taken for several loads at a time, each lane ending
// with one channel's (L - 1 shuffles for L channels, not L LG).
// b, v: the item's B [CHANNELS][r] and V [own][r] in shared memory; order: the rows; results are added to out [own][128].
template <int LG>
__device__ __forceinline__ void high_item(const __nv_bfloat16* b, const float* v, int r,
                                          const uint8_t* order, int rows, float* out) {
    constexpr int L = 1 << LG, STEP = 32 >> LG, CHANNELS = LG <= 2 ? 64 : LG == 3 ? 32 : 16;
    constexpr int LOADS = CHANNELS / STEP, G = LOADS < L ? LOADS : L;       // of the item, of a group of sums
    const int lane = threadIdx.x & 31, part = lane & (L - 1);
    const bool has = part < r / 8;
    const uint4* from = reinterpret_cast<const uint4*>(b + (lane >> LG) * r) + (has ? part : 0);
    const int pitch = STEP * (r / 8);
    uint4 w[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k) w[k] = from[k * pitch];
    out += lane >> LG;
#pragma unroll 1
    for (int n = 0; n < rows; ++n) {
        const int q = order[n];
        const float4* vq = reinterpret_cast<const float4*>(v + q * r) + (has ? 2 * part : 0);
        const float4 v0 = vq[0], v1 = vq[1];
        float s[LOADS];
#pragma unroll
        for (int k = 0; k < LOADS; ++k) {
            float a0 = v0.x * bf16_lo(w[k].x), a1 = v0.y * bf16_hi(w[k].x);
            ffma2(a0, a1, bf16_lo(w[k].y), bf16_hi(w[k].y), v0.z, v0.w);
            ffma2(a0, a1, bf16_lo(w[k].z), bf16_hi(w[k].z), v1.x, v1.y);
            ffma2(a0, a1, bf16_lo(w[k].w), bf16_hi(w[k].w), v1.z, v1.w);
            s[k] = has ? a0 + a1 : 0.0f;            // (a lane without a part reads another's)
        }
#pragma unroll
        for (int g = 0; g < LOADS; g += G) {
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
                for (int k = 0; k < o; ++k) {
                    const bool upper = part & o;
                    const float keep = upper ? s[g + k + o] : s[g + k], send = upper ? s[g + k] : s[g + k + o];
                    s[g + k] = keep + __shfl_xor_sync(kAllLanes, send, o);
                }
#pragma unroll
            for (int o = G; o < L; o <<= 1) s[g] += __shfl_xor_sync(kAllLanes, s[g], o);
            if (part < G) out[q * 128 + (g + part) * STEP] += s[g];
        }
    }
}

// The rows that a CTA finishes in the order of their adapters.
struct Grouped {
    alignas(16) int count;              // adapters
    alignas(16) int of[Few::MOST_COLS];             // [rows] their adapters, -1 for none
    int adapter[Few::MOST_COLS];        // [count]
    uint8_t first[Few::MOST_COLS + 4];  // [count + 1] places in order
    uint8_t order[Few::MOST_COLS];      // rows
};
// By one warp: a row's place is the number of rows before it, a group starts where the adapter changes.
__device__ __forceinline__ void group_rows(Grouped& g, const int (&of)[2], int mine) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < 2; ++k) g.of[lane + 32 * k] = of[k];
    __syncwarp();
    int place[2] = {0, 0}, all = 0;
    const int4* rows = reinterpret_cast<const int4*>(g.of);
#pragma unroll 4
    for (int j = 0; j < mine; j += 4) {
        const int4 a4 = rows[j >> 2];
        const int a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            all += a[i] >= 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) place[k] += a[i] >= 0 && (a[i] < of[k] || (a[i] == of[k] && j + i < lane + 32 * k));
        }
    }
    int* sorted = g.adapter;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (of[k] >= 0) {
            g.order[place[k]] = static_cast<uint8_t>(lane + 32 * k);
            sorted[place[k]] = of[k];           // (of every place first)
        }
    __syncwarp();
    int a[2], before[2], groups = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = lane + 32 * k;
        a[k] = i < all ? sorted[i] : -1;
        const bool starts = i < all && (i == 0 || sorted[i - 1] != a[k]);
        const unsigned who = __ballot_sync(kAllLanes, starts);
        before[k] = starts ? groups + __popc(who & ((1u << lane) - 1)) : -1;
        groups += __popc(who);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (before[k] >= 0) {
            g.adapter[before[k]] = a[k];
            g.first[before[k]] = static_cast<uint8_t>(lane + 32 * k);
        }
    if (lane == 0) {
        g.first[groups] = static_cast<uint8_t>(all);
        g.count = groups;
    }
}

__device__ __forceinline__ void st_shared_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// (At most 128 registers a thread: beside CTAs of the launch before, it starts earlier than with the 168 it would take: 48 rows of
// 18432 channels, rank 32, beside a product 21.8 us, not 22.2.)
__global__ void __launch_bounds__(65536 / 128, 1)
    adapter_few(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = p.stages, cols = p.width, split = p.split, lg_split = 31 - __clz(split);
    const int slice_x = cols * 128, stage_bytes = Few::W_BYTES + Few::KS * slice_x;
    const int own = (cols + split - 1) / split;                 // rows of the tile that a CTA finishes, at most
    float* parts = reinterpret_cast<float*>(ring);              // [split][own][128], once the cluster's rings have been read
    float* beside = reinterpret_cast<float*>(ring + S * stage_bytes);          // [own][128]: C, then C + V . B_a^T
    float* v_rows = beside + own * 128;                                        // [own][r]
    const int channels = Few::item_channels(p.r);
    __nv_bfloat16* slots = reinterpret_cast<__nv_bfloat16*>(v_rows + own * p.r);   // [warps][ahead][channels][r]
    Grouped& grouped = *reinterpret_cast<Grouped*>(slots + Few::EPI_WARPS * p.ahead * channels * p.r);
    uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(&grouped) + Few::GROUP_BYTES);
    uint64_t* empty = full + S;
    uint64_t* b_full = empty + S;
    uint64_t* acc_full = b_full + Few::EPI_WARPS * p.ahead;
    uint64_t* drain = acc_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x) % split, tile = static_cast<int>(blockIdx.x) / split;
    const int row0 = (tile % p.tiles) * p.width, rows = min(p.width, p.T - row0);
    const int chan0 = (tile / p.tiles) * p.channels;
    // bytes of a slice of W: the MMA reads 128 rows, and what lies behind the slice goes to lanes that nobody reads
    const int slice_w = p.channels * (p.gated ? 2 : 1) * 128;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.kstages) * rank / split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.kstages) * (rank + 1) / split);

    // (a thread for each barrier: one after another they took 0.4 us)
    const int bars = 2 * S + Few::EPI_WARPS * p.ahead + 2;
    for (int b = threadIdx.x; b < bars; b += Few::THREADS) mbar_init(full + b, 1);
    if (threadIdx.x < static_cast<unsigned>(bars)) fence_mbarrier_init();
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        if (p.kstages > 0) {
            tma_prefetch_desc(&tmW);
            tma_prefetch_desc(&tmX);
        }
    }
    if (warp == 1 && p.kstages > 0) {
        tmem_alloc(tmem_slot, Few::TMEM_COLS);
        tmem_relinquish();
    }
    if (p.wait_first) grid_dependency_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0) grid_launch_dependents();
    const uint32_t tmem = p.kstages > 0 ? *tmem_slot : 0;
    bool summed = false;                                        // an epilogue warp: the accumulator is there
    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        const uint64_t pol = policy_evict_first(), pol_x = policy_evict_last();
        uint32_t stage = 0, phase = 0;
        int64_t issued = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (issued == p.stall_after) break;
            ok = mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag, p.wait_ns);
            if (!ok) break;
            if (elect_one()) {
                uint8_t* w = ring + stage * stage_bytes;
                uint8_t* x = w + Few::W_BYTES;
                const uint32_t bar = smem_u32(&full[stage]);
                const int k0 = kb * Few::KS * Few::SL;
                mbar_arrive_expect_tx(&full[stage], Few::KS * (slice_w + slice_x));
                if (p.k_whole) {
                    tma_load_nd<false>(w, &tmW, bar, 0, chan0, 0, kb * Few::KS, pol);
                    tma_load_nd<false>(x, &tmX, bar, 0, row0, kb * Few::KS, pol_x);
                } else {
                    for (int s = 0; s < Few::KS; ++s) {
                        tma_load_nd<false>(w + s * slice_w, &tmW, bar, k0 + s * Few::SL, chan0, 0, pol);
                        tma_load_nd<false>(x + s * slice_x, &tmX, bar, k0 + s * Few::SL, row0, pol_x);
                    }
                }
            }
            __syncwarp();
            ++issued;
            if (++stage == static_cast<uint32_t>(S)) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (!ok && lane == 0) experts::fail(p, ERR_TIMEOUT_PRODUCER, abort_flag);
        // every copy issued has landed before the ring is parked in, or the CTA leaves
        for (int s = 0; s < S; ++s) {
            const int64_t cnt = issued > s ? (issued - s + S - 1) / S : 0;
            if (cnt > 0 && !mbar_wait_warp(&full[s], static_cast<uint32_t>((cnt - 1) & 1), nullptr, p.wait_ns) && lane == 0)
                experts::fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (p.kstages > 0) {
            const uint32_t s0 = smem_u32(ring), acc = __shfl_sync(kAllLanes, tmem, 0);
            const uint64_t wd0 = smem_desc_sw128(s0, 16, 1024), xd0 = smem_desc_sw128(s0 + Few::W_BYTES, 16, 1024);
            const uint32_t idesc = Few::IDESC0 | (static_cast<uint32_t>(cols >> 3) << 17);
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = mbar_wait_warp(&full[stage], phase, abort_flag, p.wait_ns);
                if (!ok) break;
                tc_fence_after();
                const uint64_t wd = wd0 + stage * (stage_bytes >> 4), xd = xd0 + stage * (stage_bytes >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < Few::KS * 4; ++k)
                        mma_bf16(acc, wd + (k / 4) * (slice_w >> 4) + (k % 4) * 2, xd + (k / 4) * (slice_x >> 4) + (k % 4) * 2,
                                 idesc, kb > kb0 || k > 0 ? 1u : 0u);
                    mma_commit(&empty[stage]);
                }
                __syncwarp();
                if (++stage == static_cast<uint32_t>(S)) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (elect_one()) {
                if (ok) mma_commit(acc_full);
                else experts::fail(p, ERR_TIMEOUT_MMA, abort_flag);
                mma_commit(drain);
                if (!mbar_wait(drain, 0, nullptr, p.wait_ns)) experts::fail(p, ERR_TIMEOUT_DRAIN, abort_flag);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- adapters, then this CTA's part of the sum
        const int ew = warp - Few::EPI_WARP0;
        const int mine = p.L > 0 && rows > rank ? (rows - rank + split - 1) / split : 0;    // rows that this CTA finishes
        const int lg_items = channels == 64 ? 1 : channels == 32 ? 2 : 3;
        // This warp's rows of C, on their way while the rows are put in order (afterwards, four rows at a time, they took 2 us more).
        constexpr int MOST = Few::MOST_COLS / Few::EPI_WARPS;
        uint32_t c_rows[MOST][4];
#pragma unroll
        for (int n = 0; n < MOST; ++n) {
            const int q = ew + n * Few::EPI_WARPS, c = rank + split * q;
            const bool row = p.C && q < own && c < rows;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t o = static_cast<int64_t>(row0 + c) * p.wide + chan0 + lane + 32 * k;
                c_rows[n][k] = 0;
                if (row && lane + 32 * k < p.channels && chan0 + lane + 32 * k < p.wide)
                    c_rows[n][k] = p.c_f32 ? static_cast<const uint32_t*>(p.C)[o] : static_cast<const uint16_t*>(p.C)[o];
            }
        }
        if (mine > 0) {
            if (ew == 0) {
                int of[2] = {-1, -1};
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (lane + 32 * k < mine) of[k] = adapter_of(p, row0 + rank + split * (lane + 32 * k));
                group_rows(grouped, of, mine);
            }
            asm volatile("barrier.cta.sync 1, %0;" ::"n"(Few::EPI_THREADS) : "memory");
        }
        // Where there are fewer items than warps, parts of a group's rows are items of their own (48 rows of one adapter of rank
        // 32, 18432 channels: 21.3 -> 14.5 us).
        int lg_parts = 0;
        if (mine > 0)
            while (grouped.count << (lg_items + lg_parts) < Few::EPI_WARPS && lg_parts < 3) ++lg_parts;
        const int items = mine > 0 ? grouped.count << (lg_items + lg_parts) : 0;
        // (a part may be empty, its items then have nothing to do)
        auto group_of = [&](int item) { return item >> (lg_items + lg_parts); };
        auto part_rows = [&](int item, int& at) {
            const int g = group_of(item), k = (item >> lg_items) & ((1 << lg_parts) - 1);
            const int begin = grouped.first[g], n = grouped.first[g + 1] - begin, lo = (n * k) >> lg_parts;
            at = begin + lo;
            return ((n * (k + 1)) >> lg_parts) - lo;
        };
        // An item's copy: the channels that there are (D's channels beyond the last have none).
        __nv_bfloat16* my_slots = slots + ew * p.ahead * channels * p.r;
        uint64_t* my_full = b_full + ew * p.ahead;
        auto there = [&](int item) {
            const int i0 = (item & ((1 << lg_items) - 1)) * channels;
            return min(channels, min(p.channels, p.wide - chan0) - (p.gated ? i0 & 63 : i0));
        };
        uint32_t pending = 0;                                   // bit s: a copy to slot s is on its way
        auto copy = [&](int item, int slot) {
            if (item >= items) return;
            const int a = grouped.adapter[group_of(item)], n = there(item);
            if (n <= 0) return;
            pending |= 1u << slot;
            if (elect_one()) {
                const int i0 = (item & ((1 << lg_items) - 1)) * channels;
                const int ch = p.gated && i0 >= 64 ? p.N / 2 + chan0 + i0 - 64 : chan0 + i0;
                mbar_arrive_expect_tx(&my_full[slot], n * p.r * 2);
                bulk_load_1d(my_slots + slot * channels * p.r, p.high + (static_cast<int64_t>(a) * p.N + ch) * p.r, n * p.r * 2,
                             &my_full[slot]);
            }
            __syncwarp();
        };
        for (int k = 0; k < p.ahead; ++k) copy(ew + k * Few::EPI_WARPS, k);
        // C is the first term of the rows' sums.
#pragma unroll
        for (int n = 0; n < MOST; ++n) {
            const int q = ew + n * Few::EPI_WARPS;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (q < own) beside[q * 128 + lane + 32 * k] = __uint_as_float(p.c_f32 ? c_rows[n][k] : c_rows[n][k] << 16);
        }
        if (!p.wait_first) grid_dependency_wait();              // V, and nothing of D before the stream allows it
        if (mine > 0) {
            {
                const int q0 = ew;                          // rows of a warp: all of their loads together
                float4 v[MOST];
#pragma unroll
                for (int n = 0; n < MOST; ++n) {
                    const int q = q0 + n * Few::EPI_WARPS;
                    v[n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (q < mine && lane < p.r / 4)         // (rows without an adapter have no V; theirs is not used)
                        v[n] = __ldcg(reinterpret_cast<const float4*>(v_row_f32(p, row0 + rank + split * q)) + lane);
                }
#pragma unroll
                for (int n = 0; n < MOST; ++n) {
                    const int q = q0 + n * Few::EPI_WARPS;
                    if (q < mine && lane < p.r / 4) reinterpret_cast<float4*>(v_rows + q * p.r)[lane] = v[n];
                }
            }
            asm volatile("barrier.cta.sync 1, %0;" ::"n"(Few::EPI_THREADS) : "memory");
            int slot = 0;
            uint32_t phases = 0;            // bit s: the next parity of my_full[s]
            bool ok = true;
            for (int item = ew; item < items; item += Few::EPI_WARPS) {
                if (there(item) > 0) {
                    int first;
                    const int n = part_rows(item, first);
                    ok = mbar_wait_warp(&my_full[slot], (phases >> slot) & 1, abort_flag, p.wait_ns);
                    if (!ok) break;
                    pending &= ~(1u << slot);
                    phases ^= 1u << slot;
                    const __nv_bfloat16* b = my_slots + slot * channels * p.r;
                    const uint8_t* order = grouped.order + first;
                    float* out = beside + (item & ((1 << lg_items) - 1)) * channels;
                    if (p.r <= 8) high_item<0>(b, v_rows, p.r, order, n, out);
                    else if (p.r <= 16) high_item<1>(b, v_rows, p.r, order, n, out);
                    else if (p.r <= 32) high_item<2>(b, v_rows, p.r, order, n, out);
                    else if (p.r <= 64) high_item<3>(b, v_rows, p.r, order, n, out);
                    else high_item<4>(b, v_rows, p.r, order, n, out);
                    __syncwarp();
                }
                copy(item + p.ahead * Few::EPI_WARPS, slot);
                slot = slot + 1 == p.ahead ? 0 : slot + 1;
            }
            if (!ok) {
                if (lane == 0) experts::fail(p, ERR_TIMEOUT_EPILOGUE, abort_flag);
                for (int s = 0; s < p.ahead; ++s)               // no copy is in flight when the CTA leaves
                    if ((pending >> s) & 1) mbar_wait_warp(&my_full[s], (phases >> s) & 1, nullptr, p.wait_ns);
            }
        }
        if (p.kstages > 0) {
            summed = mbar_wait_warp(acc_full, 0, abort_flag, p.wait_ns);
            if (!summed && lane == 0) experts::fail(p, ERR_TIMEOUT_EPILOGUE, abort_flag);
        }
    }
    __syncwarp();
    if (split > 1) cluster_sync();               // nobody reads a ring any more
    if (summed) {
        tc_fence_after();
        const int quarter = warp & 3, i = quarter * 32 + lane;
        const uint32_t mine = smem_u32(parts) + (rank * own * 128 + i) * 4;
        for (int c = ((warp - Few::EPI_WARP0) >> 2) * 16; c < cols; c += 32) {
            uint32_t v[16];
            tmem_ld16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {       // (a split divides 16)
                const uint32_t to = (split > 1 ? mapa_shared(mine, j & (split - 1)) : mine) + ((c + j) >> lg_split) * 512;
                st_shared_cluster_f32(to, __uint_as_float(v[j]));
            }
        }
        tc_fence_before();
    }
    if (split > 1) cluster_sync();
    else __syncthreads();
    if (warp >= Few::EPI_WARP0 && !*abort_flag) {
        // ---------------------------------------------------------------- the rows that this CTA finishes
        const int tid = threadIdx.x - 32 * Few::EPI_WARP0;
        auto finish = [&](auto act) { finish_rows<decltype(act)::value>(p, parts, beside, own, rank, row0, rows, chan0, tid); };
        if (p.act == DGEMM_ACT_NONE) finish(std::integral_constant<int, DGEMM_ACT_NONE>());
        else if (p.act == DGEMM_ACT_RELU) finish(std::integral_constant<int, DGEMM_ACT_RELU>());
        else if (p.act == DGEMM_ACT_GELU) finish(std::integral_constant<int, DGEMM_ACT_GELU>());
        else if (p.act == DGEMM_ACT_SILU) finish(std::integral_constant<int, DGEMM_ACT_SILU>());
        else finish(std::integral_constant<int, DGEMM_ACT_SWIGLU>());
    }
    if (warp == 1 && p.kstages > 0) {
        tc_fence_after();
        tmem_dealloc(tmem, Few::TMEM_COLS);
    }
}

}  // namespace adapters
}  // namespace dg
