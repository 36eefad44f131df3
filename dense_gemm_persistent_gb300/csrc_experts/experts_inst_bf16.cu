// experts_inst_bf16.cu -- variants of the grouped products: with and without CTA pairs, rows in order or gathered.
#include "experts_variants.cuh"

namespace dg {
namespace experts {

const Variant* variants_bf16(int* count) {
    static const Variant t[] = {
        make_variant<MmaCfg<false, false, false, false>>(), make_variant<MmaCfg<false, false, false, true>>(),
        make_variant<MmaCfg<false, false, true, false>>(),  make_variant<MmaCfg<false, false, true, true>>(),
    };
    *count = 4;
    return t;
}

}  // namespace experts
}  // namespace dg
