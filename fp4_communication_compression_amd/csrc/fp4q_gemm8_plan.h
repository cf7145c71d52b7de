// fp4q_gemm8_plan.h -- which of fp4q_gemm8's kernels a product runs on, and in how many runs
// K is cut (host only; fp4q_gemm8.hip and the tests' view of it).
#pragma once

#include "fp4q_f8.h"

namespace fp4q_plan {

using fp4q_f8::ceil_div;
using fp4q_f8::kGroup;

constexpr int kStrip = 16;  // rows of a and of b that a workgroup of strip_kernel takes
enum class Way { kStrip, kLow32, kLow64, kMedium, kLarge };
struct Plan {
    Way way;
    int tile_m, tile_n, parts;
    int64_t part_size;
    size_t workspace;
};

// The tile and the number of runs that K is cut into: the least of an estimate made of
// what the kernels take on this card.  A tile's block costs block_us with one, two or
// three workgroups on a CU and its beginning and end cost start_us besides: fitted to the
// times of every tile with 1 to 16 runs over 44 products (17 x 4096 to 8192 x 4096, K from
// 1000 to 16384, both output types; over these the choice takes 1.6 % longer than the best
// way on average, 20 % at most; over 24 others, drawn at random, 2.0 % and 14 %).  So large
// tiles serve large outputs (the GPU's own time on one card for 8192 x 11008, K = 4096:
// 359 us in 256 x 256 tiles, 415 in 128 x 128) and small ones fill the card when the output
// is small (1000 x 4096, K = 4096: 25 us in 64 x 128 tiles, 54 in 256 x 256).  Cutting K
// fills it further, for a second launch and one write and read of every run's sums
// (17 x 4096, K = 4096: 10.1 us in 6 runs, 12.4 in 16, 19.1 in one).
constexpr int kCus = 256;
inline Plan plan_of(int64_t M, int64_t N, int64_t K, bool precise) {
    Plan plan = {Way::kStrip, kStrip, kStrip, 1, 0, 0};
    if (M <= kStrip) return plan;
    struct Kind {
        Way way;
        int m, n, per_cu;
        double start_us, block_us[3];
    };
    static const Kind fast[] = {{Way::kLow32, 32, 128, 3, 0.6, {0.45, 0.53, 0.69}},
                                {Way::kLow64, 64, 128, 3, 1.5, {0.48, 0.62, 0.93}},
                                {Way::kMedium, 128, 128, 2, 2.6, {0.62, 0.98}},
                                {Way::kLarge, 256, 256, 1, 5.7, {1.54}}};
    static const Kind exact[] = {{Way::kLow32, 32, 128, 3, 0.6, {0.52, 0.73, 0.94}},
                                 {Way::kLow64, 64, 128, 2, 0.5, {0.75, 1.05}},
                                 {Way::kMedium, 128, 128, 2, 1.9, {1.16, 1.75}},
                                 {Way::kLarge, 128, 256, 1, 4.4, {1.68}}};
    constexpr double kLaunchUs = 4.7, kJoinUs = 1.5, kJoinUsPerPart = 0.25, kJoinUsPerSum = 1.1e-6;
    const int64_t blocks = ceil_div(K, kGroup);
    double best = 1e300;
    for (const Kind &k : precise ? exact : fast) {
        const int64_t tiles = ceil_div(M, k.m) * ceil_div(N, k.n);
        for (int parts = 1; parts <= 16 && (parts == 1 || parts * 2 <= blocks); ++parts) {
            const int64_t all = tiles * parts, full = all / (kCus * k.per_cu), rest = all % (kCus * k.per_cu);
            const double run = (double)ceil_div(blocks, parts);
            double us = kLaunchUs + full * (k.start_us + run * k.block_us[k.per_cu - 1]);
            if (rest) us += k.start_us + run * k.block_us[ceil_div(rest, kCus) - 1];
            if (parts > 1) us += kJoinUs + (kJoinUsPerPart + kJoinUsPerSum * M * N) * parts;
            if (us < best) {
                best = us;
                plan.way = k.way;
                plan.tile_m = k.m;
                plan.tile_n = k.n;
                plan.parts = parts;
            }
        }
    }
    if (plan.parts > 1) {
        plan.part_size = ceil_div(M * N, 4) * 4;
        plan.workspace = (size_t)(plan.part_size * plan.parts) * 4;
    }
    return plan;
}

}  // namespace fp4q_plan
