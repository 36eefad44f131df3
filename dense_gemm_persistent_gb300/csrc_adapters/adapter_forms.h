// adapter_forms.h -- which calls the kernel of adapter_beside.cuh serves. Plain C++: the host
// tests compile it.
#pragma once

#include <cstdint>

namespace dg {
namespace adapters {

// Many rows (prompt) without a product X . W^T in the same call, D and C (where there is one) in BF16, rows of D on 16
// bytes for TMA. That kernel writes the N channels of B: a gated D has half of them, and comes here without a product
// where K is 0.
inline bool beside_form(bool prompt, bool product, bool gated, bool d_f32, bool c_f32, int64_t N) {
    return prompt && !product && !gated && !d_f32 && !c_f32 && N % 8 == 0;
}

}  // namespace adapters
}  // namespace dg
