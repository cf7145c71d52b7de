// fp4q_gemm8.hip -- the product of two 8-bit operands with a scale for each block
// of 128 (declared in include/fp4q_linear.h):
//
//   out[m][n] = sum over blocks kb of sa[kb][m] sb[kb][n or n / 128]
//               sum over k in kb of a[m][k] b[n][k]
//
// b is the matrix core's first operand: a lane then holds four neighbouring n of
// one m, a's scale is one value per lane, and the output leaves in pieces of four
// neighbours.  A block's sum over its 128 k is multiplied by b's scale, then by a's,
// and added to the fp32 accumulators.  The product of the two scales is never taken
// by itself: it can leave fp32's range where the scaled sum does not (a sum of 0
// under two scales of 2^70 is 0, not 0 infinity).  A scale of a row of b is a
// multiplication after the matrix core.  The scale of a tile of b, one for all of a
// wavefront's columns, is split: its power of two goes into the matrix core's
// products, its rest to a's scales, with no work on the sums: against the product of
// the scales it takes 2.5 to 4 % longer (8192 x 11008, K = 4096: 361 for 352 us on one
// card; 2047 x 4096, K = 11008: 92.5 for 89), a multiplication of the sums 16 to 18 %
// (408 and 106).  Two forms of a step, the plain one for blocks whose scales allow it,
// spill hundreds of registers.
//
// Two ways to the block's sum:
//   8-bit matrix core  (bf16 output) one v_mfma_f32_16x16x128_f8f6f4 covers the
//     block of a 16 x 16 tile.  It adds the products of 8 neighbouring k at the
//     largest one's exponent and drops what lies below 2^-13 of it (seen with
//     powers of two; groups of 8 are added in fp32): at most 7 2^-13 of each
//     group's largest product (2.1 2^-13 seen on groups of two large products that
//     cancel and six small ones, there two thirds of the result).  Over normal
//     values it is about 2e-5 of the result, a hundredth of the output's own
//     rounding: that is why bf16 output takes it, and fp32 output does not.
//   16-bit matrix core (fp32 output) the codes become bf16, which holds every
//     E4M3 and E5M2 value, and four v_mfma_f32_16x16x32_bf16 add their exact
//     products in fp32: half the rate, 1e-8 per block.
#include "fp4q_f8.h"
#include "fp4q_gemm8_plan.h"
#include "fp4q_gemm8_tile.h"

namespace {

using namespace fp4q_f8;
using namespace fp4q_plan;
using namespace fp4q_tile;

// Two blocks in LDS: one is multiplied while the next one's loads are under way.
// Over cards, 8192 x 11008, K = 4096, E4M3 to bf16 takes 361 to 378 us (2046 to 1954
// TFLOP/s), 8192 x 8192 x 8192 480 to 507 (2290 to 2169), 2047 x 4096, K = 11008 92 to 97
// (2007 to 1903) and 11008 x 4096, K = 4001, rows of 128, fp32 output 375 to 400 (962 to
// 902).  The matrix cores are busy for 42 to 44 % of the cycles.  Of the first one's 371 us
// on one card a copy of the loop takes 280 without its loads, 321 without its LDS reads, 321
// without the scaled additions and 242 without loads and reads; of the last one's 400 us
// 290, 342, 330 and 273.  So no one part sets the time: they overlap in part, loads least
// of all, with one block under way.  256 x 256 tiles with rows of b's scales spill one
// register.
template <typename S, int kFmtA, int kFmtB, bool kTiles, bool kPrecise>
__global__ __launch_bounds__(S::kThreads, 2) void gemm_kernel(GemmArgs p) {
    __shared__ Stage<S> even;
    __shared__ Stage<S> odd;
    const Place at = place_of(p);
    Tile<S, kFmtA, kFmtB, kTiles, kPrecise> t(p, at.tm, at.tn);
    t.multiply(even, odd, at.part);
    if (p.parts > 1)
        t.store(even, p.partial + at.part * p.part_size, false);
    else if constexpr (kPrecise)
        t.store(even, static_cast<float *>(p.out), p.accumulate);
    else
        t.store(even, static_cast<bf16 *>(p.out), false);
}

// Adds the runs' sums in their order, four neighbours a thread: 48 x 11008 in 4 runs 4 us
// (8.5 MB read), 4096 x 4096 in 2 runs 29 us with fp32 and 25 with bf16 output (134 MB read,
// 67 or 34 written: 6.9 and 6.8 TB/s, out of the last-level cache in part).
constexpr int kJoinThreads = 256;
template <typename Out>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const float *partial, int64_t part_size, int parts,
                                                            int64_t count, Out *out, int accumulate) {
    const int64_t at = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x) * 4;
    if (at >= count) return;
    f32x4 sum = *reinterpret_cast<const f32x4 *>(partial + at);
    for (int s = 1; s < parts; ++s) sum += *reinterpret_cast<const f32x4 *>(partial + s * part_size + at);
    if (at + 4 <= count) {
        if constexpr (std::is_same_v<Out, float>) {
            f32x4 *to = reinterpret_cast<f32x4 *>(out + at);
            *to = accumulate ? *to + sum : sum;
        } else {
            u32x2 w;
            w[0] = fp4q_num::bf16_rne_pair(sum[0], sum[1]);
            w[1] = fp4q_num::bf16_rne_pair(sum[2], sum[3]);
            *reinterpret_cast<u32x2 *>(out + at) = w;
        }
    } else {
        for (int e = 0; at + e < count; ++e) {
            if constexpr (std::is_same_v<Out, float>)
                out[at + e] = accumulate ? out[at + e] + sum[e] : sum[e];
            else
                out[at + e] = from_float<bf16>(sum[e]);
        }
    }
}
// Up to 16 rows of a: the time is that of reading b once.  A workgroup takes 16 rows of
// b; its wavefronts share K, each taking every kStripWaves-th block, whole fragments straight
// from memory into registers, kAhead blocks' loads at a time.  A load takes 64 neighbouring
// bytes of each of 16 rows (with a lane's 32 bytes side by side, 16 bytes at every 32, it
// took a tenth longer).  The parts of the sum are joined through LDS in the wavefronts'
// order.  4096 x 11008 codes that come from HBM take 12.2 us with one row of a (3.7 TB/s; 9.5
// out of the last-level cache), 14.5 with 16 rows; 32768 x 4096 33 us (4.1 TB/s, with two
// workgroups on a CU: at most 64 registers; 37 us with one).
constexpr int kStripWaves = 16, kAhead = 4, kStripThreads = kStripWaves * kWave;
template <int kFmtA, int kFmtB, bool kTiles, bool kPrecise>
__global__ __launch_bounds__(kStripThreads, kTiles && !kPrecise ? 8 : 4) void strip_kernel(GemmArgs p) {
    __shared__ f32x4 part[kStripWaves][kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int row16 = lane & 15, quarter = lane >> 4;
    const int n0 = (int)blockIdx.x * kStrip;  // within one of b's tiles of scales
    const int blocks = (p.K + kGroup - 1) / kGroup, whole = p.K / kGroup;
    const int cols = kTiles ? (p.N + kGroup - 1) / kGroup : p.N;
    // rows past the end repeat the last one
    const int m = min(row16, p.M - 1);
    const uint8_t *a = p.a, *b = p.b + n0 * p.b_pitch;
    const unsigned row_a = m * (unsigned)p.a_pitch, row_b = (min(n0 + row16, p.N - 1) - n0) * (unsigned)p.b_pitch;
    f32x4 acc = {0, 0, 0, 0};

    // kCount blocks from kb0, kStripWaves apart; kWhole: all their codes lie before K
    auto run = [&](int kb0, auto count_of, auto whole_of) FP4Q_INLINE {
        constexpr int kCount = count_of.value;
        constexpr bool kWhole = whole_of.value;
        Raw ra[kCount], rb[kCount];
        float sa[kCount];
        f32x4 sb[kCount];
#pragma unroll
        for (int u = 0; u < kCount; ++u) {
            const int kb = kb0 + u * kStripWaves, low = kb * kGroup + 16 * quarter;
            if constexpr (kWhole) {
                rb[u] = {*reinterpret_cast<const u32x4 *>(b + (row_b + low)),
                         *reinterpret_cast<const u32x4 *>(b + (row_b + low) + 64)};
                ra[u] = {*reinterpret_cast<const u32x4 *>(a + (row_a + low)),
                         *reinterpret_cast<const u32x4 *>(a + (row_a + low) + 64)};
            } else {
                rb[u] = {load_chunk(b + row_b, low, p.K), load_chunk(b + row_b, low + 64, p.K)};
                ra[u] = {load_chunk(a + row_a, low, p.K), load_chunk(a + row_a, low + 64, p.K)};
            }
            sa[u] = p.sa[(int64_t)kb * p.M + m];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sb[u][e] = p.sb[(int64_t)kb * cols + (kTiles ? n0 / kGroup : min(n0 + 4 * quarter + e, p.N - 1))];
        }
#pragma unroll
        for (int u = 0; u < kCount; ++u) {
            Frag<kFmtB, kPrecise> first;
            Frag<kFmtA, kPrecise> second;
            first.set(rb[u]);
            second.set(ra[u]);
            const f32x4 d = block_product<false>(first, second, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = fmaf(d[e] * sb[u][e], sa[u], acc[e]);
        }
    };
    int kb = wave;
    for (; kb + (kAhead - 1) * kStripWaves < whole; kb += kAhead * kStripWaves)
        run(kb, std::integral_constant<int, kAhead>{}, std::true_type{});
    // what is left in a second and a third batch at most
    for (; kb + kStripWaves < whole; kb += 2 * kStripWaves) run(kb, std::integral_constant<int, 2>{}, std::true_type{});
    for (; kb < whole; kb += kStripWaves) run(kb, std::integral_constant<int, 1>{}, std::true_type{});
    for (; kb < blocks; kb += kStripWaves) run(kb, std::integral_constant<int, 1>{}, std::false_type{});

    part[wave][lane] = acc;
    __syncthreads();
    if (wave > 0 || row16 >= p.M) return;
#pragma unroll 5
    for (int w = 1; w < kStripWaves; ++w) acc += part[w][lane];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int n = n0 + 4 * quarter + e;
        if (n >= p.N) break;
        const int64_t at = (int64_t)row16 * p.N + n;
        if constexpr (kPrecise) {
            float *to = static_cast<float *>(p.out) + at;
            *to = p.accumulate ? *to + acc[e] : acc[e];
        } else {
            static_cast<bf16 *>(p.out)[at] = from_float<bf16>(acc[e]);
        }
    }
}

using Large = Shape<2, 4, 8, 4>;         // 256 x 256, a workgroup a CU
using LargePrecise = Shape<2, 4, 4, 4>;  // 128 x 256
using Medium = Shape<2, 2, 4, 4>;        // 128 x 128, two workgroups a CU
using Low64 = Shape<2, 2, 2, 4>;         // 64 x 128
using Low32 = Shape<1, 4, 2, 2>;         // 32 x 128
struct Strip {
    static constexpr int kThreads = kStripThreads;
};

template <typename S, int kFmtA, int kFmtB, bool kTiles, bool kPrecise>
struct Kernel {
    static const void *get() { return (const void *)&gemm_kernel<S, kFmtA, kFmtB, kTiles, kPrecise>; }
};
template <int kFmtA, int kFmtB, bool kTiles, bool kPrecise>
struct Kernel<Strip, kFmtA, kFmtB, kTiles, kPrecise> {
    static const void *get() { return (const void *)&strip_kernel<kFmtA, kFmtB, kTiles, kPrecise>; }
};
template <typename S, bool kPrecise, int kFmtA, int kFmtB>
const void *pick(bool tiles) {
    return tiles ? Kernel<S, kFmtA, kFmtB, true, kPrecise>::get() : Kernel<S, kFmtA, kFmtB, false, kPrecise>::get();
}
template <typename S, bool kPrecise>
const void *pick(int fa, int fb, bool tiles) {
    if (fa == FP4Q_E4M3)
        return fb == FP4Q_E4M3 ? pick<S, kPrecise, FP4Q_E4M3, FP4Q_E4M3>(tiles)
                               : pick<S, kPrecise, FP4Q_E4M3, FP4Q_E5M2>(tiles);
    return fb == FP4Q_E4M3 ? pick<S, kPrecise, FP4Q_E5M2, FP4Q_E4M3>(tiles)
                           : pick<S, kPrecise, FP4Q_E5M2, FP4Q_E5M2>(tiles);
}

bool bad_gemm(int64_t M, int64_t N, int64_t K) {
    return M < 0 || N < 0 || K < 0 || M >= kDimLimit || N >= kDimLimit || K >= kDimLimit ||
           ceil_div(M, 32) * ceil_div(N, 128) > (int64_t)0x7FFFFFFF / 16;
}

// What a product's sizes, output type and flags are refused for.
int check_gemm(int64_t M, int64_t N, int64_t K, int out_dtype, uint32_t flags) {
    if (bad_gemm(M, N, K)) return FP4Q_ERR_SHAPE;
    if (flags & ~(uint32_t)(FP4Q_FLAG_TILES | FP4Q_FLAG_ACCUMULATE)) return FP4Q_ERR_ARG;
    if (out_dtype == FP4Q_OUT_F32) return FP4Q_OK;
    return out_dtype == FP4Q_OUT_BF16 && !(flags & FP4Q_FLAG_ACCUMULATE) ? FP4Q_OK : FP4Q_ERR_ARG;
}

}  // namespace

extern "C" {

int fp4q_gemm8_workspace(int64_t M, int64_t N, int64_t K, int out_dtype, uint32_t flags, size_t *bytes) {
    const int st = check_gemm(M, N, K, out_dtype, flags);
    if (st != FP4Q_OK) return st;
    if (!bytes) return FP4Q_ERR_NULL;
    *bytes = M && N ? plan_of(M, N, K, out_dtype == FP4Q_OUT_F32).workspace : 0;
    return FP4Q_OK;
}

int fp4q_gemm8(const uint8_t *a, int64_t a_pitch, int a_format, const float *a_scales,
               const uint8_t *b, int64_t b_pitch, int b_format, const float *b_scales, int64_t M,
               int64_t N, int64_t K, void *out, int out_dtype, uint32_t flags, void *workspace,
               size_t workspace_bytes, void *stream) {
    if (!bad_gemm(M, N, K) && K > 0 &&
        (a_pitch < K || b_pitch < K || a_pitch >= (1 << 23) || b_pitch >= (1 << 23)))
        return FP4Q_ERR_SHAPE;
    const int st = check_gemm(M, N, K, out_dtype, flags);
    if (st != FP4Q_OK) return st;
    const bool add = flags & FP4Q_FLAG_ACCUMULATE, tiles = flags & FP4Q_FLAG_TILES;
    if ((a_format != FP4Q_E4M3 && a_format != FP4Q_E5M2) || (b_format != FP4Q_E4M3 && b_format != FP4Q_E5M2))
        return FP4Q_ERR_ARG;
    if (M == 0 || N == 0) return FP4Q_OK;
    const bool precise = out_dtype == FP4Q_OUT_F32;
    const Plan plan = plan_of(M, N, K, precise);
    const size_t need = plan.workspace;
    if (!out || (K > 0 && (!a || !a_scales || !b || !b_scales)) || (need && !workspace)) return FP4Q_ERR_NULL;
    if (!aligned(out, 16) || !aligned(workspace, 16)) return FP4Q_ERR_ALIGN;
    if (K > 0 && (!aligned(a, 16) || !aligned(b, 16) || a_pitch % 16 || b_pitch % 16)) return FP4Q_ERR_ALIGN;
    if (!aligned(a_scales, 4) || !aligned(b_scales, 4)) return FP4Q_ERR_ALIGN;
    if (workspace_bytes < need) return FP4Q_ERR_SHAPE;
    const int64_t groups = ceil_div(K, kGroup);
    const Range outs[] = {rng(out, M * N * esize(out_dtype)), rng(workspace, (int64_t)need)};
    const Range ins[] = {rng(a, pitched(M, K, a_pitch)), rng(b, pitched(N, K, b_pitch)),
                         rng(a_scales, 4 * groups * M),
                         rng(b_scales, 4 * groups * (tiles ? ceil_div(N, kGroup) : N))};
    if (clash(outs, 2, ins, K > 0 ? 4 : 0)) return FP4Q_ERR_ARG;
    GemmArgs p = {a, b, a_scales, b_scales, out, a_pitch, b_pitch, (int)M, (int)N, (int)K,
                  (int)ceil_div(M, plan.tile_m), (int)ceil_div(N, plan.tile_n), add,
                  plan.parts, plan.part_size, static_cast<float *>(workspace)};
    void *args[] = {&p};
    const void *fn = nullptr;
    int threads = 0;
    auto use = [&](auto fast, auto exact) {
        using Fast = decltype(fast);
        using Exact = decltype(exact);
        static_assert(Fast::kThreads == Exact::kThreads, "one launch for both");
        fn = precise ? pick<Exact, true>(a_format, b_format, tiles) : pick<Fast, false>(a_format, b_format, tiles);
        threads = Fast::kThreads;
    };
    switch (plan.way) {
        case Way::kStrip: use(Strip{}, Strip{}); break;
        case Way::kLow32: use(Low32{}, Low32{}); break;
        case Way::kLow64: use(Low64{}, Low64{}); break;
        case Way::kMedium: use(Medium{}, Medium{}); break;
        case Way::kLarge: use(Large{}, LargePrecise{}); break;
    }
    const int done = launch(fn, dim3((unsigned)(p.tiles_m * p.tiles_n * p.parts)), threads, args, stream);
    if (plan.parts == 1 || done != FP4Q_OK) return done;
    int64_t count = M * N;
    void *join_args[] = {&p.partial, &p.part_size, &p.parts, &count, &out, &p.accumulate};
    return launch(precise ? (const void *)&join_kernel<float> : (const void *)&join_kernel<bf16>,
                  dim3((unsigned)ceil_div(count, 4 * kJoinThreads)), kJoinThreads, join_args, stream);
}

}  // extern "C"
