// fp4q_gated8_plan.h -- which of fp4q_gated8's kernels a gated product runs on, and in how many
// runs K is cut (host only; fp4q_gated8.hip and the tests' view of it).
#pragma once

#include "fp4q_f8.h"

namespace fp4q_gated_plan {

using fp4q_f8::ceil_div;
using fp4q_f8::kGroup;

constexpr int kCus = 256;
constexpr int kStripOut = 16;  // outputs that a workgroup of gated_strip_kernel makes at a time
enum class Way { kStrip, kLow32, kLow64, kMedium, kTall, kLarge };
struct Plan {
    Way way;
    int tile_m, tile_n, parts;  // rows of a and outputs of a tile, runs of K
    int64_t part_size;          // floats of one of a run's two sums
    size_t workspace;
};

// Strips for up to 16 rows of a, and for up to 64 where every unit has a workgroup and K is
// short (us, weights from HBM; the tiles' time in brackets: 17 x 2752, K = 4096 9.3 (13.1), 48
// x 2752, K = 4096 13.0 (16.0), 48 x 1024, K = 1024 5.9 (8.6); with more units a's rows are read
// too often: 48 x 11008, K = 4096 31.7 (26.1); with long K too: 48 x 2752, K = 11008 28.7
// (24.3)).
// Else the least of an estimate as for fp4q_gemm8: a tile's block of K costs block_us with one,
// two or three workgroups on a CU and its beginning and end, the activation and three outputs
// among them, cost start_us; fitted to the times of every tile with 1 to 6 runs over 13 products
// (48 x 11008 to 8192 x 11008, K = 4096 and 11008) and to the tiles' alone with every CU full.
// Over those products the choice takes 3 % longer than the best way on average, 11 % at most
// (128 x 2752, K = 11008).  At K = 4096, in the series of the fit (the first one takes 53 us now, the
// second 740, the third 24): 2047 x 2752 57.8 us in 192-row tiles (256 rows 67.4, 128
// x 64 71.4, 64 x 64 81.0), 8192 x 11008 756 in 256-row tiles (827, 900, 1097), 48 x 11008 26.5 in
// 64 x 64 tiles and two or four runs (32 x 64 29.2, whole 32.3).  Runs of K are added by a second
// launch.
inline Plan plan_of(int64_t M, int64_t N, int64_t K) {
    Plan plan = {Way::kStrip, 64, kStripOut, 1, 0, 0};
    const bool few = M <= 16 || (M <= 64 && N <= (int64_t)kStripOut * kCus && K <= 4096);
    if (few && K > 0) return plan;  // (a strip loads a first block of K, the tiles none where there is none)
    struct Kind {
        Way way;
        int m, n, per_cu;
        double start_us, block_us[3];
    };
    static const Kind kinds[] = {{Way::kLow32, 32, 64, 3, 1.3, {0.62, 0.75, 0.96}},
                                 {Way::kLow64, 64, 64, 3, 2.9, {0.69, 0.77, 1.18}},
                                 {Way::kMedium, 128, 64, 2, 3.1, {0.79, 1.04}},
                                 {Way::kTall, 192, 128, 1, 4.0, {1.47}},
                                 {Way::kLarge, 256, 128, 1, 6.8, {1.80}}};
    constexpr double kLaunchUs = 4.7, kJoinUs = 1.5, kJoinUsPerPart = 0.4, kJoinUsPerSum = 1.03e-6;
    const int64_t blocks = ceil_div(K, kGroup);
    double best = 1e300;
    for (const Kind &k : kinds) {
        const int64_t tiles = ceil_div(M, k.m) * ceil_div(N, k.n);
        for (int parts = 1; parts <= 16 && (parts == 1 || parts * 2 <= blocks); ++parts) {
            const int64_t all = tiles * parts, full = all / (kCus * k.per_cu), rest = all % (kCus * k.per_cu);
            const double run = (double)ceil_div(blocks, parts);
            double us = kLaunchUs + full * (k.start_us + run * k.block_us[k.per_cu - 1]);
            if (rest) us += k.start_us + run * k.block_us[ceil_div(rest, kCus) - 1];
            if (parts > 1) us += kJoinUs + (kJoinUsPerPart + kJoinUsPerSum * 2 * M * N) * parts;
            if (us < best) {
                best = us;
                plan = {k.way, k.m, k.n, parts, 0, 0};
            }
        }
    }
    if (plan.parts > 1) {
        plan.part_size = ceil_div(M * N, 4) * 4;
        plan.workspace = (size_t)(2 * plan.part_size * plan.parts) * 4;
    }
    return plan;
}

}  // namespace fp4q_gated_plan
