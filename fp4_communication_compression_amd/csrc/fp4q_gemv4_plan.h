// fp4q_gemv4_plan.h -- which of fp4q_gemv4's and fp4q_gated4's kernels a product runs on (host
// only; fp4q_gemv4.hip and the tests' view of it).
#pragma once

#include "fp4q_f8.h"

namespace fp4q_few_plan {

using fp4q_f8::ceil_div;

constexpr int kBlock = FP4Q_BLOCK, kStrip = 16, kCus = 256;
constexpr int kTurnBytes = 16 * 128 + 64 * 4 + 16 * 4;  // LDS in which a wavefront turns a block of 16 rows
constexpr int64_t kLds = 160 * 1024;

// Transformed bf16 x takes one part where out is bf16: 11 bits of values that come from 8.
inline int parts_of(int dtype, int out_dtype, uint32_t flags) {
    return dtype == FP4Q_OUT_F32 || (!(flags & FP4Q_FLAG_NO_FWHT) && out_dtype == FP4Q_OUT_F32) ? 2 : 1;
}

// Whether every workgroup makes x ready itself, which saves a launch, for as many blocks of 256
// of x as its wavefronts do while the weight's first loads are on their way (one that has to be
// transformed counts twice).  us, payloads from HBM, the other way in brackets, in one series when
// the rule was made (the first takes 9.1 now): one row of 11008 10.1 (13.3), two 11.7 (13.9); 8
// rows of 4096 with two payloads of 11008 rows 20.0 (20.8), with one of 4096 rows 10.5 (10.0); 4
// transformed rows of 4096 10.6 (10.5), 5 12.9 (11.7).
constexpr int kStageBlocks = 128;
inline int64_t staged_bytes(int64_t cols, int64_t K) { return cols * (2 * (K + 8) + 4 * (K / kBlock)); }
inline bool staged(int64_t M, int64_t K, int parts, uint32_t flags) {
    const int64_t cols = M * parts, rest = 16 * (2 * 2 * cols * 64 + kTurnBytes);  // of the widest kernel
    const int64_t work = M * (K / kBlock) * (flags & FP4Q_FLAG_NO_FWHT ? 1 : 2);
    return cols <= 16 && work <= kStageBlocks && staged_bytes(cols, K) + rest <= kLds;
}
inline size_t workspace_of(int64_t M, int64_t K, int parts, uint32_t flags) {
    return staged(M, K, parts, flags) ? 0 : (size_t)(M * parts * (2 * K + 4 * (K / kBlock)));
}

// What a product runs on: where x comes from (kStaged: made ready by each workgroup, in LDS;
// kHeld: made ready in memory, a wavefront's one block of K in registers; kLoaded, kWide: made
// ready in memory, loaded with each block, for one and for two column tiles), wavefronts and
// column tiles of 16, rows of x of a chunk and chunks, outputs of a unit, workgroups of a chunk
// and bytes of LDS.
enum class Way { kStaged, kHeld, kLoaded, kWide };
struct Plan {
    Way way;
    int waves, tiles, each;
    int64_t chunks, unit, groups, lds;
};
// One or two workgroups a CU.  Measured (us, payloads from HBM; the other way in brackets), in the
// series of the rule above:
//   x made ready in the kernel: 16 wavefronts for one row of long K, 4096 x 11008 10.1 (8 of them:
//   12.3), and for more than 32 blocks of x; else 8, two workgroups a CU: 1024 x 1024 3.7 (4.6),
//   11008 x 4096 gated 13.7 (15.5)
//   x in registers where 16 wavefronts have a block each: 16 x 32768 x 4096 22.5 (24.9 without
//   the second block's loads ahead); gated, where two strips leave no registers for those (and
//   spill 9 of 128 as it is, 40 bytes of scratch a lane), with more than one unit a workgroup:
//   16 x 11008 x 4096 22.6 (27.5), but 16 x 2752 14.3 (13.5)
//   two strips, which share x, for two column tiles: 64 x 4096 x 4096 19.0 (30.8 with one); one
//   strip, and more workgroups, for one: 16 x 4096 x 11008 21.8 (24.1)
inline Plan plan_of(int64_t M, int64_t N, int64_t K, int parts, uint32_t flags, bool gated) {
    const int64_t cols = M * parts, blocks = K / kBlock;
    const bool stage = staged(M, K, parts, flags);
    Way way = Way::kWide;
    int waves = 8, most = kCus;
    if (stage) {
        way = Way::kStaged;
        if ((!gated && blocks > 16) || M * blocks > 32)
            waves = 16;
        else
            most = 2 * kCus;
    } else if (cols <= 16 && blocks <= 16 && (!gated || N > kStrip * kCus)) {
        way = Way::kHeld;
        waves = 16;
    } else if (cols <= 16) {
        way = Way::kLoaded;
    }
    const int tiles = way == Way::kWide ? 2 : 1, strips = gated || tiles == 2 ? 2 : 1, each = 16 * tiles / parts;
    const int64_t unit = gated ? kStrip : kStrip * strips, units = ceil_div(N, unit), here = M < each ? M : each;
    return {way, waves, tiles, each, ceil_div(M, each), unit, units < most ? units : most,
            waves * (2 * strips * here * parts * 64 + kTurnBytes) + (stage ? staged_bytes(cols, K) : 0)};
}

}  // namespace fp4q_few_plan
