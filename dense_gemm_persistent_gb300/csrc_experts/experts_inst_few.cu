// experts_inst_few.cu -- variants of the int8 products of one or two rows.
#include "experts_few.cuh"
#include "experts_kernels.h"
#include "host.h"

namespace dg {
namespace experts {

namespace {

template <class CF>
cudaError_t launch_few(const void* B, const Params& p, int grid, size_t smem, cudaStream_t s) {
    host::Launch l(static_cast<unsigned>(grid), 1, CF::THREADS, smem, s);
    return cudaLaunchKernelEx(&l.cfg, expert_few<CF>, B, p);
}

template <class CF>
FewVariant make_few() {
    return FewVariant{CF::ROWS, CF::TILE, CF::CTAS_PER_SM, reinterpret_cast<const void*>(&expert_few<CF>), &launch_few<CF>};
}

}  // namespace

const FewVariant* variants_few(int* count) {
    static const FewVariant t[] = {make_few<FewCfg<1>>(), make_few<FewCfg<2>>()};
    *count = 2;
    return t;
}

}  // namespace experts
}  // namespace dg
