// Which kernel an integer product takes (product_i8.hip), by its tokens and weight
// rows: plain C++, so that the tests can ask the same question.
#pragma once

#include <stdint.h>

namespace dq {

// few_R_T: workgroups of four waves, 16 R weight rows by 16 T tokens; split_T: of
// eight waves that split K, 32 rows by 16 T tokens; tiles: tokens x weight rows.
enum class I8Kernel {
    few_1_1, few_2_1, few_4_1, few_7_1,
    few_1_2, few_2_2, few_4_2, few_7_2,
    few_2_4, few_4_4, few_7_4,
    split_2, split_4,
    tiles_256x256, tiles_128x128, tiles_64x128_deep, tiles_64x128,
    kCount
};

inline I8Kernel i8_kernel(int64_t M, int64_t N)
{
    const auto tiles = [&](int64_t m, int64_t n) { return ((M + m - 1) / m) * ((N + n - 1) / n); };
    // Too few tiles for the CUs: 32 weight rows by 32 or 64 tokens per workgroup, whose
    // eight waves split K, in one round of workgroups.  100 x 2000 x 4096 at b = 4 / 7:
    // 32 tokens 9.2 / 11.4 us, 64 tokens 13.2 / 15.4, 64 x 128 tiles 14.6 / 22.7; 200 x
    // 1500 x 4096: 15.4 / 20.8, 13.6 / 15.7, 14.9 / 22.9; 128 x 6000 x 4096 (more than
    // a round): 21.8 / 29.9, 25.2 / 29.9, 14.8 / 22.8
    if (M > 32) {
        if (tiles(32, 32) <= 256) return I8Kernel::split_2;
        if (tiles(64, 32) <= 256) return I8Kernel::split_4;
    }
    if (M <= 64) {
        // the most rows per workgroup that leave 224 workgroups or more for the 256 CUs
        constexpr int64_t kFill = 224;
        const int r = N >= 16 * 7 * kFill ? 3 : (N >= 16 * 4 * kFill ? 2 : (N >= 16 * 2 * kFill ? 1 : 0));
        // (33 to 64 tokens by fewer than 2 rows of 16 went to split_4)
        const I8Kernel first = M <= 16 ? I8Kernel::few_1_1 : (M <= 32 ? I8Kernel::few_1_2 : I8Kernel::few_2_4);
        return (I8Kernel)((int)first + (M <= 32 ? r : r - 1));
    }
    // 256 x 256 tiles, eight waves, when they fill the 256 CUs in whole rounds (at
    // least 80 % of the last round busy): 2048 x 8192 x 8192 at b = 8 122 us (2.25 POP/s)
    // against 139 us for 128 x 128 tiles of four waves, two or three to a CU
    const int64_t wide = tiles(256, 256);
    if (M >= 256 && wide >= 256 && wide * 5 >= (wide + 255) / 256 * 256 * 4) return I8Kernel::tiles_256x256;
    // 128 x 128 tiles: 333 x 17408 x 5120 at b = 5 51 us (64 x 128 67 us, 192 x 128 59 us,
    // 128 x 256 55 us, 256 x 256 82 us); half as high while they leave CUs without one
    if (tiles(128, 128) >= 256) return I8Kernel::tiles_128x128;
    // and with four stages while a CU has one workgroup at most, whose copies nothing
    // else hides: 300 x 3000 x 8192 at b = 4 / 7 / 8 23.2 / 39.7 / 24.6 us, two stages
    // 28.2 / 44.9 / 37.8 (the same within 2 % where the caches hold the operands)
    return tiles(64, 128) <= 256 ? I8Kernel::tiles_64x128_deep : I8Kernel::tiles_64x128;
}

}  // namespace dq
