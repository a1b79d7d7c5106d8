// How a product of microscaled 4-bit operands is cut: which kernel, tiles, pieces of K.
// Host code without HIP, so that tests can ask it which kernel sizes reach.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace biloco {
namespace mx {

constexpr int kGroup = 8;      // stages of 128 k whose scales come together
// Rows of A up to which W is streamed.  32 rows of 5120 to 13824 20.0 us, in tiles 22.2; 8192
// to 8192 16.8 and 19.6; 17 rows of 5120 to 5120 9.5 and 14.2; 48 are past the kernels' operands.
constexpr int kRows = 32;
// Workgroups that the pieces of K are to make, one a CU: 200 rows of 13824 to 5120 in 3
// pieces (240 workgroups) 31.4 us, in 2 36.7, in 6 34.0, in 9 44.
constexpr int kWant = 256;

constexpr int kCUs = 256;

struct MxPlan {
    bool rows;
    int bm, bn, pieces;
    size_t part_bytes;
};
inline MxPlan plan_of(int M, int N, int K) {
    MxPlan p{M <= kRows, 0, 0, 1, 0};
    if (p.rows) return p;
    const auto tiles = [&](int b) { return (int64_t)((M + b - 1) / b) * ((N + b - 1) / b); };
    // Large tiles where they fill at least four fifths of their rounds over the CUs: 2048 x
    // 8192 x 8192 (256 of them) 87 us, in small ones 109; 4096 x 4096 x 4096 54 and 60; but
    // 4096 x 5120 x 5120 (320) 110 and 84, 1500 x 13824 x 5120 (324) 114 and 95.
    const int64_t large = tiles(256), rounds = (large + kCUs - 1) / kCUs;
    p.bm = p.bn = 5 * large >= 4 * kCUs * rounds ? 256 : 128;
    const int64_t n = tiles(p.bm);
    int64_t pieces = n >= kWant ? 1 : (kWant + n / 2) / n;
    const int64_t most = ((int64_t)K + 128 * kGroup - 1) / (128 * kGroup);      // groups of stages
    if (pieces > most) pieces = most;
    p.pieces = pieces < 1 ? 1 : (int)pieces;
    if (p.pieces > 1) p.part_bytes = (size_t)p.pieces * M * N * 4;
    return p;
}

}  // namespace mx
}  // namespace biloco
