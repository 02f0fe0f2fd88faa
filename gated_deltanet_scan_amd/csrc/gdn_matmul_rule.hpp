// The rule by which gdn_matmul_fp8 chooses its kernel: plain C++, so that a host test can
// ask it which kernels a set of sizes reaches.
#pragma once

#include <algorithm>
#include <cstdint>

namespace gdnmatmul {

// Which kernel, in tenths of a microsecond at K = 2048 (and in proportion at others).
// Few tokens: what a workgroup takes, and more as a compute unit gets several.  100
// tokens, N = 512: 4.5 us with 16 tokens to a workgroup, 5.9 with 32, 8.8 in tiles; 100 and
// N = 1000: 6.8, 6.0, 9.1; 64 and N = 2048: 6.8, 6.0, 9.0; 64 and N = 6144: 15.8, 13.1,
// 8.9; 200 and N = 1000: 10.8, 9.6, 9.2 (K = 8192: 36, 31, 25).
// Tiles: the fewest rounds of the card times what a round takes: 128 x 64 two a unit
// 14 us, one a unit 9.6; 128 x 128 13.2; 256 x 128 20; 256 x 256 32.  So 880 x 2048 takes
// 10.0 us in the first where the others take 12.5, 16.7 and 26; 880 x 6144 18.8 in the
// third (21.4, 22.5, -, 27.9); 7040 x 2048 32 in the last (42, 42, 35).
enum Kind : int { kFew16, kFew32, k128x64, k128x128, k256x128, k256x256 };
inline Kind choose(int64_t M, int N, int cus) {
    if (M <= 16) return kFew16;
    auto share = [&](int m) { return std::max(1.0, (double)((N + 15) / 16) * ((M + m - 1) / m) / cus); };
    const double few16 = 23 + 23 * share(16), few32 = 18 + 41 * share(32);
    if (std::min(few16, few32) < 85) return few16 < few32 ? kFew16 : kFew32;
    auto tiles = [&](int n, int m) { return ((N + n - 1) / n) * ((M + m - 1) / m); };
    auto rounds = [&](int64_t t, int at_once) { return (t + at_once - 1) / at_once; };
    const int64_t t = tiles(128, 64);
    const int64_t cost[] = {t <= cus ? 96 : 140 * rounds(t, 2 * cus), 132 * rounds(tiles(128, 128), cus),
                            200 * rounds(tiles(256, 128), cus), 320 * rounds(tiles(256, 256), cus)};
    int best = 0;
    for (int i = 1; i < 4; ++i)
        if (cost[i] < cost[best]) best = i;
    return (Kind)(k128x64 + best);
}

}  // namespace gdnmatmul
