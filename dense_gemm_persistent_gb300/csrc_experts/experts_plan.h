// experts_plan.h -- the choice between single CTAs and CTA pairs of the expert and int8
// products. Plain C++: the host tests compile it.
#pragma once

#include <algorithm>
#include <cstdint>

namespace dg {
namespace experts {

// Whether R rows in E groups, `wide` channels in tiles of `step` (of a single CTA), take CTA
// pairs: 256 channels and up to 256 rows (INT8 192) a tile, where groups are long enough to
// share weights between two SMs. Single CTAs, 128 channels and up to 64 rows a tile, read
// weights for few rows each; they are also taken where their tiles, for groups of the mean
// size, are at most one wave.
//
// Single / pairs in us, groups of random sizes:
//   mean of        40       48       56       64       80 rows
//   BF16       162/171  162/171  165/172  174/173  199/175   32 experts of 4096 x 4096, gathered, gated
//   E4M3         85/91    85/92    87/92    91/93   106/94   the same
//   INT8       114/132  120/133  135/134  167/135  202/139   64 experts of 2048 x 4096
//   INT8       185/212  192/213  225/215  267/218  354/223   32 experts of 4096 x 7168
// One wave: BF16 512 rows of 1024 x 2048 9.9/15.8, just above it 512 rows of 4096 x 2048
// 15.6/16.4; INT8 64 rows of 18432 x 7168 34/41, 256 of 4096 x 4096 21/25, above it 96 rows of
// 18432 x 7168 54/43, 512 of 4096 x 4096 37/29.
// The sizes of the groups are not known to the host. Where one of 64 experts has 80 % of the
// rows and the mean is 32, the single CTAs that the mean asks for take 362 us against 347 (BF16
// 4096 x 4096), 187 against 177 (E4M3) and 144 against 146 (INT8 2048 x 4096).
inline bool takes_pairs(int64_t R, int64_t E, int64_t wide, int64_t step, int num_sms) {
    const int64_t mean = (R + E - 1) / E;
    const bool one_wave = (mean + 63) / 64 * std::min(E, R) * ((wide + step - 1) / step) <= num_sms;
    return R > 48 * E && !one_wave;
}

}  // namespace experts
}  // namespace dg
