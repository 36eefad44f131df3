// experts_inst_fp8.cu -- variants of the grouped products: with and without CTA pairs, rows in order or gathered.
#include "experts_variants.cuh"

namespace dg {
namespace experts {

const Variant* variants_fp8(int* count) {
    static const Variant t[] = {
        make_variant<MmaCfg<true, false, false, false>>(), make_variant<MmaCfg<true, false, false, true>>(),
        make_variant<MmaCfg<true, false, true, false>>(),  make_variant<MmaCfg<true, false, true, true>>(),
    };
    *count = 4;
    return t;
}

}  // namespace experts
}  // namespace dg
