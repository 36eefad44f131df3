// experts.cu -- products grouped by expert and the int8 product (one group):
//
//     D[r,n] = act(alpha * as[a] * bs[e,n] * sum_k A[a,k] B_e[n,k] + beta * C[r,n] + bias[e,n])
//
// for the rows r of expert e, a = a_rows[r] or r. The output channels n run over the
// 128 rows of the MMA and the token rows over its columns, so a group's few rows
// cost few columns. The simplest form: every thread loads operands, converts them to
// BF16 (exact for E4M3 and int8) and stores them swizzled; one thread multiplies.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "dgemm_experts.h"
#include "experts_kernels.h"
#include "host.h"

namespace {

struct ExpertParams {
    const void* A;
    const int* a_rows;
    const void* B;
    const float* a_scale;
    const float* b_scale;
    const int* offsets;          // null: one group of R rows
    const float* bias;
    const void* C;
    void* D;
    int type, kn, E, R, N, K, a_count, act, d_f32, c_f32;
    int wide;                    // columns of D: N, or N / 2 when gated
    float alpha, beta;
    unsigned* status;
    unsigned long long* ws_status;
    unsigned long long epoch;
    uint64_t wait_ns;
};

constexpr int ACT_SWIGLU = DGEMM_ACT_SWIGLU;
constexpr int TM = 128, TN = 64;

__device__ __forceinline__ float load_value(const void* x, int type, int64_t i) {
    if (type == DGEMM_GROUPED_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(x)[i]);
    if (type == DGEMM_GROUPED_INT8) return static_cast<float>(static_cast<const int8_t*>(x)[i]);
    return static_cast<float>(static_cast<const __nv_fp8_e4m3*>(x)[i]);
}

__device__ __forceinline__ void expert_error(const ExpertParams& p, unsigned bit) {
    if (p.ws_status) atomicExch(p.ws_status, (p.epoch << 8) | bit);
    else atomicOr(p.status, bit);
}

__device__ __forceinline__ float silu1(float v) { return __fdividef(v, 1.0f + __expf(-v)); }

__device__ __forceinline__ float activation1(float v, int act) {
    if (act == DGEMM_ACT_RELU) return fmaxf(v, 0.0f);
    if (act == DGEMM_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    if (act == DGEMM_ACT_SILU) return silu1(v);
    return v;
}

__global__ void __launch_bounds__(256, 1) expert_product(const ExpertParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sa = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sb = sa + TM * 128;
    float* sy = reinterpret_cast<float*>(sb + TN * 128);    // [TN][TM + 1]
    __shared__ uint64_t done;
    __shared__ uint32_t tmem_slot;
    __shared__ int s_e, s_r0, s_r1, s_ok;
    dg::grid_dependency_wait();
    if (threadIdx.x == 0) dg::grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        // which group's tile of token rows this CTA has
        int left = blockIdx.y;
        s_e = -1;
        for (int e = 0; e < p.E; ++e) {
            const int lo = p.offsets ? min(max(p.offsets[e], 0), p.R) : 0;
            const int hi = p.offsets ? min(max(p.offsets[e + 1], lo), p.R) : p.R;
            const int tiles = (hi - lo + TN - 1) / TN;
            if (left < tiles) {
                s_e = e;
                s_r0 = lo + left * TN;
                s_r1 = min(hi, s_r0 + TN);
                break;
            }
            left -= tiles;
        }
        dg::mbar_init(&done, 1);
        dg::fence_mbarrier_init();
        s_ok = 1;
    }
    __syncthreads();
    if (s_e < 0) return;
    if (warp == 0) {
        dg::tmem_alloc(&tmem_slot, 64);
        dg::tmem_relinquish();
    }
    dg::tc_fence_before();
    __syncthreads();
    dg::tc_fence_after();
    const int e = s_e, r0 = s_r0, rows = s_r1 - s_r0;
    const bool gated = p.act == ACT_SWIGLU;
    const int half = p.N / 2;
    const int n0 = blockIdx.x * (gated ? TM / 2 : TM);
    // MMA row i is this output channel (-1: none); gated: 64 of the gate, 64 of the up half
    auto channel = [&](int i) {
        const int n = gated ? n0 + (i & 63) : n0 + i;
        if (n >= p.wide) return -1;
        return gated && i >= 64 ? half + n : n;
    };
    const int64_t eb = static_cast<int64_t>(e) * p.N * p.K;
    bool ok = true;
    for (int k0 = 0; ok && k0 < p.K; k0 += 64) {
        for (int c = threadIdx.x; c < (TM + TN) * 8; c += 256) {
            const bool is_a = c < TM * 8;
            const int i = is_a ? c % TM : (c - TM * 8) % TN, chunk = is_a ? c / TM : (c - TM * 8) / TN;
            const int k = k0 + chunk * 8;
            float v[8];
            int64_t row = -1;
            if (is_a) {
                row = channel(i);
            } else if (i < rows) {
                row = p.a_rows ? p.a_rows[r0 + i] : r0 + i;
                if (row < 0 || row >= p.a_count) row = -1;
            }
            for (int j = 0; j < 8; ++j) {
                v[j] = 0.0f;
                if (row >= 0 && k + j < p.K)
                    v[j] = !is_a ? load_value(p.A, p.type, row * p.K + k + j)
                           : p.kn ? load_value(p.B, p.type, eb + static_cast<int64_t>(k + j) * p.N + row)
                                  : load_value(p.B, p.type, eb + row * p.K + k + j);
            }
            const uint4 w = make_uint4(dg::pack_bf16x2(v[0], v[1]), dg::pack_bf16x2(v[2], v[3]),
                                       dg::pack_bf16x2(v[4], v[5]), dg::pack_bf16x2(v[6], v[7]));
            *reinterpret_cast<uint4*>((is_a ? sa : sb) + i * 128 + ((chunk ^ (i & 7)) << 4)) = w;
        }
        dg::fence_proxy_async_smem();
        __syncthreads();
        if (threadIdx.x == 0) {
            dg::tc_fence_after();
            const uint64_t ad = dg::smem_desc_sw128(dg::smem_u32(sa), 16, 1024);
            const uint64_t bd = dg::smem_desc_sw128(dg::smem_u32(sb), 16, 1024);
            const uint32_t idesc = dg::make_idesc(1u, false, false, TM, TN);
            for (int s = 0; s < 4; ++s)
                dg::mma_bf16(tmem_slot, ad + s * 2, bd + s * 2, idesc, (k0 > 0 || s > 0) ? 1u : 0u);
            dg::mma_commit(&done);
        }
        ok = dg::mbar_wait(&done, (k0 / 64) & 1, nullptr, p.wait_ns);
        if (!ok) s_ok = 0;
        __syncthreads();
        ok = s_ok != 0;
    }
    if (!ok && threadIdx.x == 0) expert_error(p, dg::ERR_TIMEOUT_MMA);
    dg::tc_fence_after();
    if (ok && warp < 4) {
        const int i = warp * 32 + lane, ch = channel(i);
        const float bs = p.alpha * (p.b_scale && ch >= 0 ? p.b_scale[static_cast<int64_t>(e) * p.N + ch] : 1.0f);
        const float bias = p.bias && ch >= 0 ? p.bias[static_cast<int64_t>(e) * p.N + ch] : 0.0f;
        for (int c0 = 0; c0 < TN; c0 += 32) {
            uint32_t acc[32];
            dg::tmem_ld32(tmem_slot + (static_cast<uint32_t>(warp * 32) << 16) + c0, acc);
            dg::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const int c = c0 + j;
                float v = 0.0f;
                if (c < rows) {
                    const int a = p.a_rows ? p.a_rows[r0 + c] : r0 + c;
                    const float as = p.a_scale && a >= 0 && a < p.a_count ? p.a_scale[a] : p.a_scale ? 0.0f : 1.0f;
                    v = (p.K > 0 ? __uint_as_float(acc[j]) : 0.0f) * as * bs + bias;
                }
                sy[c * (TM + 1) + i] = v;
            }
        }
    }
    dg::tc_fence_before();
    __syncthreads();
    if (ok) {
        const int width = gated ? 64 : 128;
        for (int c = threadIdx.x; c < rows * width; c += 256) {
            const int r = c / width, i = c % width, n = n0 + i;
            if (n >= p.wide) continue;
            const int64_t at = static_cast<int64_t>(r0 + r) * p.wide + n;
            float v = sy[r * (TM + 1) + i];
            if (p.C) {
                const float x = p.c_f32 ? static_cast<const float*>(p.C)[at]
                                        : __bfloat162float(static_cast<const __nv_bfloat16*>(p.C)[at]);
                v = fmaf(p.beta, x, v);
            }
            v = gated ? silu1(v) * sy[r * (TM + 1) + 64 + i] : activation1(v, p.act);
            if (p.d_f32) static_cast<float*>(p.D)[at] = v;
            else static_cast<__nv_bfloat16*>(p.D)[at] = __float2bfloat16_rn(v);
        }
    }
    if (warp == 0) {
        dg::tc_fence_after();
        dg::tmem_dealloc(tmem_slot, 64);
    }
}

constexpr size_t SMEM = 1024 + TM * 128 + TN * 128 + TN * (TM + 1) * 4;

using dg::experts::Variant;

const Variant* find_variant(int fp8, int kn, int pair, int gather) {
    int n = 0;
    const Variant* v = fp8 ? dg::experts::variants_fp8(&n) : kn ? dg::experts::variants_bf16_kn(&n) : dg::experts::variants_bf16(&n);
    for (int i = 0; i < n; ++i)
        if (v[i].pair == pair && v[i].gather == gather) return v + i;
    return nullptr;
}

struct Call {
    int type;
    const void* A;
    int64_t a_count;
    const int32_t* a_rows;
    const void* B;
    dgemm_b_layout_t layout;
    const float *a_scale, *b_scale;
    const int32_t* offsets;
    int64_t E;
    const void* C;
    dgemm_dtype_t c_dtype;
    float beta;
    void* D;
    dgemm_dtype_t d_dtype;
    int64_t R, N, K;
    float alpha;
    const float* bias;
    int act;
    void* ws;
    size_t ws_bytes;
    cudaStream_t stream;
};

// The sizes and enums of a call: no device needed.
dgemm_status_t check_sizes(int type, int64_t R, int64_t E, int64_t N, int64_t K, dgemm_b_layout_t layout, int act) {
    if (R < 0 || E < 0 || N < 0 || K < 0) return DGEMM_ERR_INVALID_VALUE;
    if (type < DGEMM_GROUPED_BF16 || type > DGEMM_GROUPED_INT8) return DGEMM_ERR_INVALID_VALUE;
    if (layout != DGEMM_B_KN && layout != DGEMM_B_NK) return DGEMM_ERR_INVALID_VALUE;
    if (act < DGEMM_ACT_NONE || act > DGEMM_ACT_SWIGLU) return DGEMM_ERR_INVALID_VALUE;
    if (act == DGEMM_ACT_SWIGLU && N % 2 != 0) return DGEMM_ERR_INVALID_VALUE;
    if (E > DGEMM_MAX_EXPERTS) return DGEMM_ERR_NOT_SUPPORTED;
    if (R > INT32_MAX / 2 || N > INT32_MAX / 2 || K > INT32_MAX / 2) return DGEMM_ERR_NOT_SUPPORTED;
    const int64_t esz = type == DGEMM_GROUPED_BF16 ? 2 : 1;
    if (K * esz % 16 != 0) return DGEMM_ERR_MISALIGNED;
    if (layout == DGEMM_B_KN && N * esz % 16 != 0) return DGEMM_ERR_MISALIGNED;
    return DGEMM_OK;
}

// Launches the tensor-core variant for BF16 or E4M3 operands.
dgemm_status_t run_mma(const Call& c, const dg::host::Device& dev) {
    const int fp8 = c.type == DGEMM_GROUPED_FP8, kn = c.layout == DGEMM_B_KN, gated = c.act == DGEMM_ACT_SWIGLU;
    const uint64_t esz = fp8 ? 1 : 2, sl = 128 / esz;
    const uint64_t N = static_cast<uint64_t>(c.N), K = static_cast<uint64_t>(c.K), E = static_cast<uint64_t>(c.E);
    // KN: both halves of a gated product start on 16 bytes
    if (kn && gated && (N / 2) * esz % 16 != 0) return DGEMM_ERR_MISALIGNED;
    // CTA pairs (256 channels, up to 256 rows a tile) where groups are long enough to
    // share weights between two SMs; single CTAs (128 channels, up to 64 rows) where
    // the calls read weights for few rows each.
    const int pair = c.R > 48 * c.E;
    const Variant* v = find_variant(fp8, kn, pair, c.a_rows != nullptr);
    if (!v) return DGEMM_ERR_NOT_SUPPORTED;

    dg::experts::Params p{};
    p.offsets = c.offsets;
    p.a_rows = c.a_rows;
    p.A = c.A;
    p.a_scale = c.a_scale;
    p.b_scale = c.b_scale;
    p.bias = c.bias;
    p.D = c.D;
    p.E = static_cast<int>(c.E);
    p.R = static_cast<int>(c.R);
    p.N = static_cast<int>(c.N);
    p.K = static_cast<int>(c.K);
    p.a_count = static_cast<int>(c.a_count);
    p.gated = gated;
    p.wide = gated ? p.N / 2 : p.N;
    p.act = c.act;
    p.d_f32 = c.d_dtype == DGEMM_F32;
    const int tile_channels = (gated ? 64 : 128) * v->ctas;
    p.ctiles = (p.wide + tile_channels - 1) / tile_channels;
    const uint64_t ks = static_cast<uint64_t>(v->slices);
    p.kstages = static_cast<int>((K + ks * sl - 1) / (ks * sl));
    p.k_whole = K % sl == 0;
    p.alpha = c.alpha;
    p.status = dev.status;
    p.epoch = dg::host::next_launch_epoch();
    p.ws_status = c.ws && c.ws_bytes >= DGEMM_WS_STATUS_BYTES ? static_cast<unsigned long long*>(c.ws) : nullptr;
    dg::host::wait_settings(&p.wait_ns, &p.stall_after);

    // at most one partial tile per group
    const int64_t most_tiles = ((c.R + v->bn - 1) / v->bn + std::min(c.E, c.R)) * p.ctiles;
    if (most_tiles > INT32_MAX / 2) return DGEMM_ERR_NOT_SUPPORTED;
    const int units = static_cast<int>(std::min<int64_t>(dev.num_sms / v->ctas, most_tiles));

    alignas(64) CUtensorMap w, x, xs;
    std::memset(&w, 0, sizeof w);
    std::memset(&x, 0, sizeof x);
    std::memset(&xs, 0, sizeof xs);
    if (K > 0) {
        const CUtensorMapDataType dt = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        const uint32_t s = static_cast<uint32_t>(sl);
        const uint64_t halves = gated ? 2 : 1, H = N / halves;
        const uint32_t box_rows = gated ? 64 : 128, box_halves = static_cast<uint32_t>(halves);
        bool ok;
        if (kn) {
            const uint64_t d[3] = {N, K, E}, st[2] = {N * esz, K * N * esz};
            const uint32_t b[3] = {s, static_cast<uint32_t>(ks) * s, 1};
            ok = dg::host::encode_map(&w, dt, c.B, 3, d, st, b);
        } else if (p.k_whole) {
            // a stage's K slices, and the gate and up channels of a gated tile, in one copy
            const uint64_t d[5] = {sl, H, halves, K / sl, E}, st[4] = {K * esz, H * K * esz, 128, N * K * esz};
            const uint32_t b[5] = {s, box_rows, box_halves, static_cast<uint32_t>(ks), 1};
            ok = dg::host::encode_map(&w, dt, c.B, 5, d, st, b);
        } else {
            const uint64_t d[4] = {K, H, halves, E}, st[3] = {K * esz, H * K * esz, N * K * esz};
            const uint32_t b[4] = {s, box_rows, box_halves, 1};
            ok = dg::host::encode_map(&w, dt, c.B, 4, d, st, b);
        }
        if (ok && !c.a_rows) {
            const uint64_t rows = static_cast<uint64_t>(c.a_count);
            const uint32_t big = static_cast<uint32_t>(v->bn_cta), few = static_cast<uint32_t>(v->small_rows);
            if (p.k_whole) {
                const uint64_t d[3] = {sl, rows, K / sl}, st[2] = {K * esz, 128};
                const uint32_t b[3] = {s, big, 2}, bs[3] = {s, few, 1};
                ok = dg::host::encode_map(&x, dt, c.A, 3, d, st, b) && dg::host::encode_map(&xs, dt, c.A, 3, d, st, bs);
            } else {
                const uint64_t d[2] = {K, rows}, st[1] = {K * esz};
                const uint32_t b[2] = {s, big}, bs[2] = {s, few};
                ok = dg::host::encode_map(&x, dt, c.A, 2, d, st, b) && dg::host::encode_map(&xs, dt, c.A, 2, d, st, bs);
            }
        }
        if (!ok) return DGEMM_ERR_CUDA;
    }
    const size_t smem = v->smem_fixed + dg::experts::Schedule::bytes(p.E);
    static std::atomic<unsigned char> ready[12][dg::host::kMaxDevices];
    std::atomic<unsigned char>& flag = ready[(fp8 ? 8 : kn ? 4 : 0) + pair * 2 + (c.a_rows ? 1 : 0)][dev.id];
    if (!flag.load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(v->func, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(v->smem_fixed + dg::experts::Schedule::bytes(DGEMM_MAX_EXPERTS))) != cudaSuccess)
            return DGEMM_ERR_CUDA;
        flag.store(1, std::memory_order_release);
    }
    return v->launch(w, x, xs, p, units * v->ctas, smem, c.stream) == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
}

dgemm_status_t run_experts(const Call& c) {
    const dgemm_status_t st = check_sizes(c.type, c.R, c.E, c.N, c.K, c.layout, c.act);
    if (st != DGEMM_OK) return st;
    if (c.d_dtype != DGEMM_F32 && c.d_dtype != DGEMM_BF16) return DGEMM_ERR_INVALID_VALUE;
    if (c.a_count < 0 || (!c.a_rows && c.a_count != c.R)) return DGEMM_ERR_INVALID_VALUE;
    if (c.a_count > INT32_MAX / 2) return DGEMM_ERR_NOT_SUPPORTED;
    if (c.R == 0 || c.N == 0 || c.E == 0) return DGEMM_OK;
    if (!c.D || (c.K > 0 && (!c.B || (c.a_count > 0 && !c.A)))) return DGEMM_ERR_INVALID_VALUE;
    if (c.type != DGEMM_GROUPED_BF16 && (!c.a_scale || !c.b_scale)) return DGEMM_ERR_INVALID_VALUE;
    if (c.beta != 0.0f && (!c.C || (c.c_dtype != DGEMM_F32 && c.c_dtype != DGEMM_BF16))) return DGEMM_ERR_INVALID_VALUE;
    if (!dg::host::aligned16(c.A) || !dg::host::aligned16(c.B) || !dg::host::aligned16(c.D) || !dg::host::aligned16(c.ws) ||
        (c.beta != 0.0f && !dg::host::aligned16(c.C)))
        return DGEMM_ERR_MISALIGNED;
    const uintptr_t natural = reinterpret_cast<uintptr_t>(c.a_scale) | reinterpret_cast<uintptr_t>(c.b_scale) |
                              reinterpret_cast<uintptr_t>(c.bias) | reinterpret_cast<uintptr_t>(c.offsets) |
                              reinterpret_cast<uintptr_t>(c.a_rows);
    if (natural & 3u) return DGEMM_ERR_MISALIGNED;
    dg::host::Device dev;
    const dgemm_status_t ds = dg::host::current_device(&dev);
    if (ds != DGEMM_OK) return ds;

    if (c.type != DGEMM_GROUPED_INT8) return run_mma(c, dev);
    ExpertParams p{};
    p.A = c.A;
    p.a_rows = c.a_rows;
    p.B = c.B;
    p.a_scale = c.a_scale;
    p.b_scale = c.b_scale;
    p.offsets = c.offsets;
    p.bias = c.bias;
    p.C = c.beta != 0.0f ? c.C : nullptr;
    p.c_f32 = c.c_dtype == DGEMM_F32;
    p.D = c.D;
    p.type = c.type;
    p.kn = c.layout == DGEMM_B_KN;
    p.E = static_cast<int>(c.E);
    p.R = static_cast<int>(c.R);
    p.N = static_cast<int>(c.N);
    p.K = static_cast<int>(c.K);
    p.a_count = static_cast<int>(c.a_count);
    p.act = c.act;
    p.d_f32 = c.d_dtype == DGEMM_F32;
    p.wide = c.act == DGEMM_ACT_SWIGLU ? p.N / 2 : p.N;
    p.alpha = c.alpha;
    p.beta = c.beta;
    p.status = dev.status;
    p.epoch = dg::host::next_launch_epoch();
    p.ws_status = c.ws && c.ws_bytes >= DGEMM_WS_STATUS_BYTES ? static_cast<unsigned long long*>(c.ws) : nullptr;
    long long stall;
    dg::host::wait_settings(&p.wait_ns, &stall);
    static std::atomic<unsigned char> ready[dg::host::kMaxDevices];
    if (!ready[dev.id].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(expert_product, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess)
            return DGEMM_ERR_CUDA;
        ready[dev.id].store(1, std::memory_order_release);
    }
    const int step = c.act == DGEMM_ACT_SWIGLU ? TM / 2 : TM;
    const int64_t tiles = (c.R + TN - 1) / TN + c.E - 1;     // at most: one partial tile per group
    if (tiles > 65535) return DGEMM_ERR_NOT_SUPPORTED;
    dg::host::Launch l(static_cast<unsigned>((p.wide + step - 1) / step), static_cast<unsigned>(tiles), 256, SMEM, c.stream);
    return cudaLaunchKernelEx(&l.cfg, expert_product, p) == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
}

}  // namespace

extern "C" {

dgemm_status_t dgemm_grouped_bf16(const void* A, int64_t a_count, const int32_t* a_rows, const void* B,
                                  dgemm_b_layout_t b_layout, const int32_t* offsets, int64_t E, void* D,
                                  dgemm_dtype_t d_dtype, int64_t R, int64_t N, int64_t K, float alpha,
                                  const float* bias, int act, void* ws, size_t ws_bytes, dgemm_stream_t stream) {
    if (!offsets && R > 0 && N > 0 && E > 0) return DGEMM_ERR_INVALID_VALUE;
    return run_experts(Call{DGEMM_GROUPED_BF16, A, a_count, a_rows, B, b_layout, nullptr, nullptr, offsets, E, nullptr,
                            DGEMM_F32, 0.0f, D, d_dtype, R, N, K, alpha, bias, act, ws, ws_bytes,
                            reinterpret_cast<cudaStream_t>(stream)});
}

dgemm_status_t dgemm_grouped_fp8_scaled(const void* Aq, int64_t a_count, const int32_t* a_rows, const void* Bq,
                                        const float* a_scale, const float* b_scale, const int32_t* offsets, int64_t E,
                                        void* D, dgemm_dtype_t d_dtype, int64_t R, int64_t N, int64_t K, float alpha,
                                        const float* bias, int act, void* ws, size_t ws_bytes, dgemm_stream_t stream) {
    if (!offsets && R > 0 && N > 0 && E > 0) return DGEMM_ERR_INVALID_VALUE;
    return run_experts(Call{DGEMM_GROUPED_FP8, Aq, a_count, a_rows, Bq, DGEMM_B_NK, a_scale, b_scale, offsets, E,
                            nullptr, DGEMM_F32, 0.0f, D, d_dtype, R, N, K, alpha, bias, act, ws, ws_bytes,
                            reinterpret_cast<cudaStream_t>(stream)});
}

dgemm_status_t dgemm_grouped_int8_scaled(const void* Aq, int64_t a_count, const int32_t* a_rows, const void* Bq,
                                         const float* a_scale, const float* b_scale, const int32_t* offsets, int64_t E,
                                         void* D, dgemm_dtype_t d_dtype, int64_t R, int64_t N, int64_t K, float alpha,
                                         const float* bias, int act, void* ws, size_t ws_bytes, dgemm_stream_t stream) {
    if (!offsets && R > 0 && N > 0 && E > 0) return DGEMM_ERR_INVALID_VALUE;
    return run_experts(Call{DGEMM_GROUPED_INT8, Aq, a_count, a_rows, Bq, DGEMM_B_NK, a_scale, b_scale, offsets, E,
                            nullptr, DGEMM_F32, 0.0f, D, d_dtype, R, N, K, alpha, bias, act, ws, ws_bytes,
                            reinterpret_cast<cudaStream_t>(stream)});
}

size_t dgemm_grouped_workspace_size(dgemm_grouped_type_t type, int64_t R, int64_t E, int64_t N, int64_t K, int act) {
    return check_sizes(type, R, E, N, K, DGEMM_B_NK, act) == DGEMM_OK ? DGEMM_WS_STATUS_BYTES : 0;
}

dgemm_status_t dgemm_int8_scaled(const void* Aq, const void* Bq, const float* a_scale, const float* b_scale,
                                 const void* C, dgemm_dtype_t c_dtype, void* D, dgemm_dtype_t d_dtype, int64_t M,
                                 int64_t N, int64_t K, float alpha, float beta, const float* bias, int act, void* ws,
                                 size_t ws_bytes, dgemm_stream_t stream) {
    if (act == DGEMM_ACT_SWIGLU) return DGEMM_ERR_INVALID_VALUE;
    return run_experts(Call{DGEMM_GROUPED_INT8, Aq, M, nullptr, Bq, DGEMM_B_NK, a_scale, b_scale, nullptr, 1, C, c_dtype,
                            beta, D, d_dtype, M, N, K, alpha, bias, act, ws, ws_bytes,
                            reinterpret_cast<cudaStream_t>(stream)});
}

size_t dgemm_int8_workspace_size(int64_t M, int64_t N, int64_t K) {
    return check_sizes(DGEMM_GROUPED_INT8, M, 1, N, K, DGEMM_B_NK, DGEMM_ACT_NONE) == DGEMM_OK ? DGEMM_WS_STATUS_BYTES : 0;
}

}  // extern "C"
