// experts_inst_bf16_kn.cu -- variants of the grouped products: with and without CTA pairs, rows in order or gathered.
#include "experts_variants.cuh"

namespace dg {
namespace experts {

const Variant* variants_bf16_kn(int* count) {
    static const Variant t[] = {
        make_variant<MmaCfg<false, true, false, false>>(), make_variant<MmaCfg<false, true, false, true>>(),
        make_variant<MmaCfg<false, true, true, false>>(),  make_variant<MmaCfg<false, true, true, true>>(),
    };
    *count = 4;
    return t;
}

}  // namespace experts
}  // namespace dg
