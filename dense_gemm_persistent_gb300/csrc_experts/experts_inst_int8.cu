// experts_inst_int8.cu -- variants of the int8 products: with and without CTA pairs.
#include "experts_int8.cuh"
#include "experts_kernels.h"
#include "host.h"

namespace dg {
namespace experts {

namespace {

template <class CF>
cudaError_t launch_int8(const CUtensorMap& w, const CUtensorMap&, const CUtensorMap&, const Params& p, int grid,
                        size_t smem, cudaStream_t s) {
    host::Launch l(static_cast<unsigned>(grid), 1, CF::THREADS, smem, s, CF::CTAS);
    return cudaLaunchKernelEx(&l.cfg, expert_int8<CF>, w, p);
}

template <class CF>
Variant make_int8() {
    return Variant{DGEMM_GROUPED_INT8, 0, CF::PAIR, -1, CF::BN, CF::BN_CTA, CF::CTAS, 1, 0, CF::THREADS, CF::LAUNCH_REGS, CF::FIXED,
                   reinterpret_cast<const void*>(&expert_int8<CF>), &launch_int8<CF>};
}

}  // namespace

const Variant* variants_int8(int* count) {
    static const Variant t[] = {make_int8<Int8Cfg<false>>(), make_int8<Int8Cfg<true>>()};
    *count = 2;
    return t;
}

}  // namespace experts
}  // namespace dg
