// adapter_few.cuh -- the projection with adapters for tiles of up to 64 rows.
//
// The output channels are the MMA's 128 rows, the token rows its columns. A cluster of
// `split` CTAs shares a tile's K: each sums its part in Tensor Memory, parks it in its shared
// memory, and finishes every split-th row of the tile from all parts in their order.
// V . B_a^T runs on the FP32 units meanwhile, row by row: every row reads the adapter of its own, and
// rows may be of as many requests as there are. It needs V, the rest does not: only these
// warps wait for the launch that computes it.
// Warps: 0 TMA producer, 1 MMA issuer and owner of the Tensor Memory, 2-9 epilogue.
#pragma once

#include "adapter_common.cuh"

namespace dg {
namespace adapters {

struct Few {
    static constexpr int KS = 2, SL = 64;                 // 128-byte slices of K per stage, elements of a slice
    static constexpr int MOST_COLS = 64, MOST_STAGES = 8, MOST_SPLIT = 8;
    static constexpr int SLICE_W = 128 * 128, W_BYTES = KS * SLICE_W;
    static constexpr int EPI_WARP0 = 2, EPI_WARPS = 8, EPI_THREADS = 32 * EPI_WARPS, THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
    static constexpr int TMEM_COLS = 64, BAR_BYTES = 256;
    static constexpr uint32_t IDESC0 = make_idesc(1u, false, false, 128, 0);
    static constexpr int stage_bytes(int cols) { return W_BYTES + KS * cols * 128; }
    static constexpr int smem_bytes(int cols, int stages, int split) {
        return 1024 + stages * stage_bytes(cols) + (cols + split - 1) / split * 512 + BAR_BYTES;
    }
    static_assert((2 * MOST_STAGES + 2) * 8 + 8 <= BAR_BYTES, "barriers fit");
    // (a parked tile, 64 columns of 128 floats, is never larger than two stages)
};

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case DGEMM_ACT_RELU: return experts::relu(v);
        case DGEMM_ACT_GELU: return experts::gelu(v);
        case DGEMM_ACT_SILU: return experts::silu(v);
        default: return v;
    }
}

// V[t] . B_a^T for one row t of the tile and some of its 128 channels, by one warp: r / 8 lanes (rounded up to
// a power of two) share a channel, so that a load of the warp is one run of memory, eight loads in
// flight. `out`: the row's [128] results.
struct HighItems {
    int lanes, channels, per_row;       // lanes of a channel, channels of an item, items of a row
    __device__ __forceinline__ explicit HighItems(int r) {
        lanes = r <= 8 ? 1 : 1 << (32 - __clz(r / 8 - 1));
        channels = min(128, 256 / lanes);
        per_row = 128 / channels;
    }
};
__device__ __forceinline__ void high_item(const Params& p, const HighItems& h, int t, int a, int chan0, int item, float* out) {
    const int lane = threadIdx.x & 31, part = lane & (h.lanes - 1), first = item * h.channels + lane / h.lanes;
    const int step = 32 / h.lanes;
    const bool has = part < p.r / 8;
    float4 v0 = make_float4(0, 0, 0, 0), v1 = v0;
    if (has) {
        const float4* v = reinterpret_cast<const float4*>(p.V + static_cast<int64_t>(t) * p.r + part * 8);
        v0 = v[0];
        v1 = v[1];
    }
    const __nv_bfloat16* b = p.high + static_cast<int64_t>(a) * p.N * p.r + part * 8;
    uint4 w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int i = first + k * step, ch = chan0 + (p.gated ? i & 63 : i), n = p.gated && i >= 64 ? p.N / 2 + ch : ch;
        w[k] = has && k * step < h.channels && ch < p.wide ? __ldg(reinterpret_cast<const uint4*>(b + static_cast<int64_t>(n) * p.r))
                                                           : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (k * step >= h.channels) break;
        float s0 = 0.0f, s1 = 0.0f;
        fma8(s0, s1, w[k], v0, v1);
        float s = s0 + s1;
        for (int o = 1; o < h.lanes; o <<= 1) s += __shfl_xor_sync(kAllLanes, s, o);
        if (part == 0) out[first + k * step] = s;
    }
}

// The sum of a parked tile's value over the CTAs of its cluster, in their order, for COLS rows of the tile
// (cols[i] < 0: none): every load is on its way before the first sum.
template <int COLS>
__device__ __forceinline__ void gather_parts(uint32_t parked, int split, const int (&cols)[COLS], int i, float (&y)[COLS]) {
    float v[COLS][Few::MOST_SPLIT];
#pragma unroll
    for (int s = 0; s < Few::MOST_SPLIT; ++s) {
        if (s >= split) break;
        const uint32_t from = split > 1 ? mapa_shared(parked, s) : parked;
#pragma unroll
        for (int c = 0; c < COLS; ++c) v[c][s] = cols[c] >= 0 ? ld_shared_cluster_f32(from + (cols[c] * 128 + i) * 4) : 0.0f;
    }
#pragma unroll
    for (int s = 0; s < Few::MOST_SPLIT; ++s) {
        if (s >= split) break;
#pragma unroll
        for (int c = 0; c < COLS; ++c) y[c] = s == 0 ? v[c][0] : y[c] + v[c][s];
    }
}

__global__ void __launch_bounds__(Few::THREADS, 1)
    adapter_few(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = p.stages, cols = p.width, split = p.split;
    const int slice_x = cols * 128, stage_bytes = Few::W_BYTES + Few::KS * slice_x;
    const int own = (cols + split - 1) / split;                 // rows of the tile that a CTA finishes, at most
    float* park = reinterpret_cast<float*>(ring);               // [cols][128], once the ring has been read
    float* delta = reinterpret_cast<float*>(ring + S * stage_bytes);           // [own][128]
    uint64_t* full = reinterpret_cast<uint64_t*>(delta + own * 128);
    uint64_t* empty = full + S;
    uint64_t* acc_full = empty + S;
    uint64_t* drain = acc_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x) % split, tile = static_cast<int>(blockIdx.x) / split;
    const int row0 = (tile % p.tiles) * p.width, rows = min(p.width, p.T - row0);
    const int chan0 = (tile / p.tiles) * (p.gated ? 64 : 128);
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.kstages) * rank / split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.kstages) * (rank + 1) / split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
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
                mbar_arrive_expect_tx(&full[stage], stage_bytes);
                if (p.k_whole) {
                    tma_load_nd<false>(w, &tmW, bar, 0, chan0, 0, kb * Few::KS, pol);
                    tma_load_nd<false>(x, &tmX, bar, 0, row0, kb * Few::KS, pol_x);
                } else {
                    for (int s = 0; s < Few::KS; ++s) {
                        tma_load_nd<false>(w + s * Few::SLICE_W, &tmW, bar, k0 + s * Few::SL, chan0, 0, pol);
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
                        mma_bf16(acc, wd + (k / 4) * (Few::SLICE_W >> 4) + (k % 4) * 2, xd + (k / 4) * (slice_x >> 4) + (k % 4) * 2,
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
        if (!p.wait_first) grid_dependency_wait();              // V, and nothing of D before the stream allows it
        if (p.L > 0) {
            const HighItems h(p.r);
            for (int item = warp - Few::EPI_WARP0; item < own * h.per_row; item += Few::EPI_WARPS) {
                const int q = item / h.per_row, c = rank + split * q;
                if (c >= rows) break;
                const int a = adapter_of(p, row0 + c), part = item % h.per_row;
                if (a >= 0) high_item(p, h, row0 + c, a, chan0, part, delta + q * 128);
                else for (int i = lane; i < h.channels; i += 32) delta[q * 128 + part * h.channels + i] = 0.0f;
            }
        }
        if (p.kstages > 0) {
            const bool ok = mbar_wait_warp(acc_full, 0, abort_flag, p.wait_ns);
            if (ok) {
                tc_fence_after();
                const int quarter = warp & 3, part = (warp - Few::EPI_WARP0) >> 2;
                for (int c = part * 16; c < cols; c += 32) {
                    uint32_t v[16];
                    tmem_ld16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) park[(c + j) * 128 + quarter * 32 + lane] = __uint_as_float(v[j]);
                }
                tc_fence_before();
            } else if (lane == 0) {
                experts::fail(p, ERR_TIMEOUT_EPILOGUE, abort_flag);
            }
        }
    }
    if (split > 1) cluster_sync();
    else __syncthreads();
    if (warp >= Few::EPI_WARP0 && !*abort_flag) {
        // ---------------------------------------------------------------- the rows that this CTA finishes
        const int tid = threadIdx.x - 32 * Few::EPI_WARP0;
        const int out = p.gated ? 64 : 128, oc = tid & (out - 1), step = Few::EPI_THREADS / out;
        const int ch = chan0 + oc;
        if (ch < p.wide) {
            constexpr int COLS = 2;
            const float bias = p.bias ? __ldg(p.bias + ch) : 0.0f, bias_up = p.bias && p.gated ? __ldg(p.bias + p.N / 2 + ch) : 0.0f;
            const uint32_t parked = smem_u32(park);
            for (int q0 = tid / out; q0 < own; q0 += COLS * step) {
                int cols[COLS];
                float y[COLS], up[COLS], c_in[COLS];
#pragma unroll
                for (int k = 0; k < COLS; ++k) {
                    const int q = q0 + k * step, c = rank + split * q;
                    cols[k] = q < own && c < rows ? c : -1;
                    y[k] = up[k] = c_in[k] = 0.0f;
                    if (p.C && cols[k] >= 0) {
                        const int64_t o = static_cast<int64_t>(row0 + c) * p.wide + ch;
                        c_in[k] = p.c_f32 ? static_cast<const float*>(p.C)[o] : __bfloat162float(static_cast<const __nv_bfloat16*>(p.C)[o]);
                    }
                }
                if (p.kstages > 0) {
                    gather_parts(parked, split, cols, oc, y);
                    if (p.gated) gather_parts(parked, split, cols, 64 + oc, up);
                }
#pragma unroll
                for (int k = 0; k < COLS; ++k) {
                    if (cols[k] < 0) continue;
                    const int q = q0 + k * step;
                    float v = y[k] + c_in[k] + bias;
                    if (p.L > 0) v += delta[q * 128 + oc];
                    if (p.gated) {
                        float u = up[k] + bias_up;
                        if (p.L > 0) u += delta[q * 128 + 64 + oc];
                        v = experts::silu(v) * u;
                    } else {
                        v = activate(v, p.act);
                    }
                    const int64_t o = static_cast<int64_t>(row0 + cols[k]) * p.wide + ch;
                    if (p.d_f32) static_cast<float*>(p.D)[o] = v;
                    else static_cast<__nv_bfloat16*>(p.D)[o] = __float2bfloat16_rn(v);
                }
            }
        }
    }
    tc_fence_before();
    if (split > 1) cluster_sync();
    else __syncthreads();
    if (warp == 1 && p.kstages > 0) {
        tc_fence_after();
        tmem_dealloc(tmem, Few::TMEM_COLS);
    }
}

}  // namespace adapters
}  // namespace dg
