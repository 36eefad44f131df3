// experts.cu -- products grouped by expert and the int8 product (one group):
//
//     D[r,n] = act(alpha * as[a] * bs[e,n] * sum_k A[a,k] B_e[n,k] + beta * C[r,n] + bias[e,n])
//
// for the rows r of expert e, a = a_rows[r] or r. Host side: checks, the choice of a
// variant, tensor maps and the launch. The kernels are in experts_mma.cuh and experts_int8.cuh.

#include <algorithm>
#include <atomic>
#include <cstring>

#include "dgemm_experts.h"
#include "experts_kernels.h"
#include "experts_plan.h"
#include "host.h"

namespace {

using dg::experts::Variant;

const Variant* find_variant(int type, int kn, int pair, int gather) {
    int n = 0;
    const Variant* v = type == DGEMM_GROUPED_INT8  ? dg::experts::variants_int8(&n)
                       : type == DGEMM_GROUPED_FP8 ? dg::experts::variants_fp8(&n)
                       : kn                        ? dg::experts::variants_bf16_kn(&n)
                                                   : dg::experts::variants_bf16(&n);
    for (int i = 0; i < n; ++i)
        if (v[i].pair == pair && (v[i].gather == gather || v[i].gather < 0)) return v + i;
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
    // K x N rows on 16 bytes, and the up half of a gated one too: tiled copies start there
    const int64_t row = act == DGEMM_ACT_SWIGLU ? N / 2 : N;
    if (layout == DGEMM_B_KN && row * esz % 16 != 0) return DGEMM_ERR_MISALIGNED;
    return DGEMM_OK;
}

// What every kernel of a call is given.
dg::experts::Params make_params(const Call& c, const dg::host::Device& dev) {
    dg::experts::Params p{};
    p.offsets = c.offsets;
    p.a_rows = c.a_rows;
    p.A = c.A;
    p.a_scale = c.a_scale;
    p.b_scale = c.b_scale;
    p.bias = c.bias;
    p.C = c.beta != 0.0f ? c.C : nullptr;
    p.c_f32 = c.c_dtype == DGEMM_F32;
    p.beta = c.beta;
    p.D = c.D;
    p.E = static_cast<int>(c.E);
    p.R = static_cast<int>(c.R);
    p.N = static_cast<int>(c.N);
    p.K = static_cast<int>(c.K);
    p.a_count = static_cast<int>(c.a_count);
    p.gated = c.act == DGEMM_ACT_SWIGLU;
    p.wide = p.gated ? p.N / 2 : p.N;
    p.act = c.act;
    p.d_f32 = c.d_dtype == DGEMM_F32;
    p.alpha = c.alpha;
    p.status = dev.status;
    p.epoch = dg::host::next_launch_epoch();
    p.ws_status = c.ws && c.ws_bytes >= DGEMM_WS_STATUS_BYTES ? static_cast<unsigned long long*>(c.ws) : nullptr;
    dg::host::wait_settings(&p.wait_ns, &p.stall_after);
    return p;
}

// Shared memory of the kernels of few rows.
constexpr size_t kFewSharedBytes = 74 * 1024;     // three CTAs an SM

// Most rows (1 or 2) of the few-rows kernel for an int8 call that it takes, 0 where the
// tensor-core kernel does: one set of weights and at most two rows whose codes fit (one row, two
// rows, tensor-core kernel: 18432 x 7168 24.7, 27.3, 27.5 us; 4096 x 4096 5.8, 7.0, 16.2; experts_few.cuh has more).
int few_rows(const Call& c) {
    if (c.type != DGEMM_GROUPED_INT8 || c.E != 1 || c.R > 2 || c.K == 0 || c.K > 131071) return 0;
    return static_cast<size_t>(c.R) * static_cast<size_t>(c.K) <= kFewSharedBytes ? static_cast<int>(c.R) : 0;
}

dgemm_status_t launch_few(const Call& c, const dg::host::Device& dev, int rows) {
    int n = 0, at = 0;
    const dg::experts::FewVariant* v = dg::experts::variants_few(&n);
    while (at < n && v[at].rows != rows) ++at;
    if (at == n) return DGEMM_ERR_NOT_SUPPORTED;
    v += at;
    dg::experts::Params p = make_params(c, dev);
    const int tile_channels = p.gated ? v->tile / 2 : v->tile;
    p.ctiles = (p.wide + tile_channels - 1) / tile_channels;
    const int grid = std::min(dev.num_sms * v->ctas_per_sm, p.ctiles);
    static std::atomic<unsigned char> ready[2][dg::host::kMaxDevices];
    std::atomic<unsigned char>& flag = ready[at][dev.id];
    if (!flag.load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(v->func, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kFewSharedBytes)) != cudaSuccess)
            return DGEMM_ERR_CUDA;
        flag.store(1, std::memory_order_release);
    }
    const size_t smem = rows * static_cast<size_t>(c.K);
    return v->launch(c.B, p, grid, smem, c.stream) == cudaSuccess ? DGEMM_OK : DGEMM_ERR_CUDA;
}

// Picks the variant, encodes the tensor maps and launches.
dgemm_status_t launch(const Call& c, const dg::host::Device& dev) {
    const int kn = c.layout == DGEMM_B_KN, gated = c.act == DGEMM_ACT_SWIGLU;
    const int int8 = c.type == DGEMM_GROUPED_INT8;   // (its token rows need no map: converted on the way)
    const uint64_t esz = c.type == DGEMM_GROUPED_BF16 ? 2 : 1, sl = 128 / esz;
    const uint64_t N = static_cast<uint64_t>(c.N), K = static_cast<uint64_t>(c.K), E = static_cast<uint64_t>(c.E);
    const int forced = dg::host::pair_override();
    const int pair = forced >= 0 ? forced
                                 : dg::experts::takes_pairs(c.R, c.E, gated ? c.N / 2 : c.N, gated ? 64 : 128, dev.num_sms);
    const Variant* v = find_variant(c.type, kn, pair, c.a_rows != nullptr);
    if (!v) return DGEMM_ERR_NOT_SUPPORTED;

    dg::experts::Params p = make_params(c, dev);
    const int tile_channels = (gated ? 64 : 128) * v->ctas;
    p.ctiles = (p.wide + tile_channels - 1) / tile_channels;
    const uint64_t ks = static_cast<uint64_t>(v->slices);
    p.kstages = static_cast<int>((K + ks * sl - 1) / (ks * sl));
    p.k_whole = K % sl == 0 && !int8;

    // at most one partial tile per group
    const int64_t most_tiles = ((c.R + v->bn - 1) / v->bn + std::min(c.E, c.R)) * p.ctiles;
    if (most_tiles > INT32_MAX / 2) return DGEMM_ERR_NOT_SUPPORTED;
    const int units = static_cast<int>(std::min<int64_t>(dev.num_sms / v->ctas, most_tiles));

    alignas(64) CUtensorMap w, x, xs;
    std::memset(&w, 0, sizeof w);
    std::memset(&x, 0, sizeof x);
    std::memset(&xs, 0, sizeof xs);
    if (K > 0) {
        const CUtensorMapDataType dt = esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
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
        if (ok && !c.a_rows && !int8) {
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
    static std::atomic<unsigned char> ready[16][dg::host::kMaxDevices];
    std::atomic<unsigned char>& flag = ready[c.type * 4 + (kn ? 12 : 0) + pair * 2 + (c.a_rows ? 1 : 0)][dev.id];
    if (!flag.load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(v->func, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(v->smem_fixed + dg::experts::Schedule::bytes(DGEMM_MAX_EXPERTS))) != cudaSuccess)
            return DGEMM_ERR_CUDA;
        // a register split that adds up to more than the launch holds would wait forever
        cudaFuncAttributes fa{};
        if (v->launch_regs > 0 && (cudaFuncGetAttributes(&fa, v->func) != cudaSuccess || fa.numRegs < v->launch_regs))
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

    const int rows = few_rows(c);
    return rows ? launch_few(c, dev, rows) : launch(c, dev);
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
