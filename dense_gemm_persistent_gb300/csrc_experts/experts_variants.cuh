// experts_variants.cuh -- builds the table entry of one variant.
#pragma once

#include "experts_kernels.h"
#include "experts_mma.cuh"
#include "host.h"

namespace dg {
namespace experts {

template <class CF>
cudaError_t launch_mma(const CUtensorMap& w, const CUtensorMap& x, const CUtensorMap& xs, const Params& p, int grid,
                       size_t smem, cudaStream_t s) {
    host::Launch l(static_cast<unsigned>(grid), 1, CF::THREADS, smem, s, CF::CTAS);
    return cudaLaunchKernelEx(&l.cfg, expert_mma<CF>, w, x, xs, p);
}

template <class CF>
Variant make_variant() {
    return Variant{CF::FP8 ? DGEMM_GROUPED_FP8 : DGEMM_GROUPED_BF16, CF::KN, CF::PAIR, CF::GATHER, CF::BN, CF::BN_CTA, CF::CTAS, CF::KS, CF::SMALL_ROWS, CF::THREADS, 0,
                   CF::FIXED, reinterpret_cast<const void*>(&expert_mma<CF>), &launch_mma<CF>};
}

}  // namespace experts
}  // namespace dg
