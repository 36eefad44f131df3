// experts_kernels.h -- the compiled variants of the expert products, for the host side.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "experts_common.cuh"

namespace dg {
namespace experts {

struct Variant {
    int type, kn, pair;          // dgemm_grouped_type_t; weights K x N; CTA pairs
    int gather;                  // 1: rows by index, 0: rows in order, -1: either
    int bn, bn_cta, ctas, slices, small_rows, threads;   // slices: 128-byte slices of K per stage
    int launch_regs;             // registers per thread that the kernel's register split assumes (0: none)
    size_t smem_fixed;           // dynamic shared memory without the schedule
    const void* func;
    cudaError_t (*launch)(const CUtensorMap& w, const CUtensorMap& x, const CUtensorMap& xs, const Params& p, int grid,
                          size_t smem, cudaStream_t s);
};

const Variant* variants_bf16(int* count);
const Variant* variants_bf16_kn(int* count);
const Variant* variants_fp8(int* count);
const Variant* variants_int8(int* count);

// One or two rows in all (int8).
struct FewVariant {
    int rows, tile, ctas_per_sm;   // most rows; weight rows of a tile
    const void* func;
    cudaError_t (*launch)(const void* B, const Params& p, int grid, size_t smem, cudaStream_t s);
};
const FewVariant* variants_few(int* count);

}  // namespace experts
}  // namespace dg
