// fp4q_gated8.hip -- the gated product of 8-bit operands (declared in include/fp4q_gated.h):
//
//   y[m][n] = act(g) u,  g = sum over k of a[m][k] w[n][k],  u = the same of row P + n of w
//
// One pass of the product's tiles (fp4q_gemm8_tile.h) over the joined weight.  Half of a
// tile's rows of w come from the gate, half from the up projection, dealt out so that a lane
// ends with both sums of an output in registers: the activation and the product are a few
// operations on them, and neither g nor u need be written and read again.
#include "fp4q_act.h"
#include "fp4q_gemm8_plan.h"
#include "fp4q_gemm8_tile.h"

namespace {

using namespace fp4q_f8;
using namespace fp4q_plan;
using namespace fp4q_tile;
using namespace fp4q_act;

template <typename S, int kFmtA, int kFmtW>
__global__ __launch_bounds__(S::kThreads, 2) void gated_kernel(GatedArgs p) {
    __shared__ Stage<S> even;
    __shared__ Stage<S> odd;
    const Place at = place_of(p);
    Tile<S, kFmtA, kFmtW, true, false, true> t(p, at.tm, at.tn);
    t.multiply(even, odd, at.part);
    constexpr int kHalf = S::kTilesN / 2;
    if (p.parts > 1) {
        // a run's sums: all of the gate's, then the up projection's
        float *to = p.partial + 2 * at.part * p.part_size;
        t.template store<0>(even, to, false);
        t.template store<kHalf>(even, to + p.part_size, false);
        return;
    }
    if (p.gate) {
        t.template store<0>(even, static_cast<bf16 *>(p.gate), false);
        t.template store<kHalf>(even, static_cast<bf16 *>(p.up), false);
    }
    with_act(p.act, [&](auto act) FP4Q_INLINE {
#pragma unroll
        for (int i = 0; i < S::kTilesM; ++i)
#pragma unroll
            for (int j = 0; j < kHalf; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    t.acc[i][j][e] = activate<act.value>(t.acc[i][j][e]).act * t.acc[i][j + kHalf][e];
    });
    t.template store<0>(even, static_cast<bf16 *>(p.out), false);
}

// Up to four bf16 of v at `to`.
__device__ __forceinline__ void store4(bf16 *to, const f32x4 &v, int left) {
    if (left >= 4) {
        u32x2 w;
        w[0] = fp4q_num::bf16_rne_pair(v[0], v[1]);
        w[1] = fp4q_num::bf16_rne_pair(v[2], v[3]);
        *reinterpret_cast<u32x2 *>(to) = w;
    } else {
        for (int e = 0; e < left; ++e) to[e] = from_float<bf16>(v[e]);
    }
}

// Adds the runs' sums in their order and makes the outputs, four neighbours a thread.
constexpr int kJoinThreads = 256;
__global__ __launch_bounds__(kJoinThreads) void gated_join_kernel(GatedArgs p) {
    const int64_t count = (int64_t)p.M * p.N, at = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x) * 4;
    if (at >= count) return;
    f32x4 g = {0, 0, 0, 0}, u = g;
    for (int s = 0; s < p.parts; ++s) {
        const float *from = p.partial + 2 * s * p.part_size + at;
        g += *reinterpret_cast<const f32x4 *>(from);
        u += *reinterpret_cast<const f32x4 *>(from + p.part_size);
    }
    const int left = (int)min((int64_t)4, count - at);
    if (p.gate) {
        store4(static_cast<bf16 *>(p.gate) + at, g, left);
        store4(static_cast<bf16 *>(p.up) + at, u, left);
    }
    with_act(p.act, [&](auto act) FP4Q_INLINE {
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = activate<act.value>(g[e]).act * u[e];
    });
    store4(static_cast<bf16 *>(p.out) + at, g, left);
}

// Up to 16 rows of a: the time is that of reading w once.  A workgroup takes 8 rows of the
// gate and the same 8 of the up projection as the matrix core's 16; its wavefronts share K,
// each taking every kWaves-th block, whole fragments straight from memory into registers,
// kAhead blocks' loads at a time.  The parts of the sum are joined through LDS in the
// wavefronts' order; lanes l and l + 32 hold an output's g and u.
constexpr int kStripWaves = 16, kAhead = 4, kStripThreads = kStripWaves * kWave, kStripOut = 8;
template <int kFmtA, int kFmtW>
__global__ __launch_bounds__(kStripThreads, 4) void gated_strip_kernel(GatedArgs p) {
    __shared__ f32x4 part[kStripWaves][kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int row16 = lane & 15, quarter = lane >> 4;
    const int n0 = (int)blockIdx.x * kStripOut;  // within one tile of scales of either half
    const int blocks = (p.K + kGroup - 1) / kGroup, whole = p.K / kGroup;
    const int tiles = 2 * (p.second / kGroup);
    // rows past the end repeat the last one
    const int m = min(row16, p.M - 1), n = min(n0 + (row16 & 7), p.N - 1);
    const uint8_t *a = p.a, *w = p.b + (int64_t)(n + (row16 < 8 ? 0 : p.second)) * p.b_pitch + 16 * quarter;
    const unsigned row_a = m * (unsigned)p.a_pitch + 16 * quarter;
    const int tile = n0 / kGroup + (quarter < 2 ? 0 : p.second / kGroup);
    f32x4 acc = {0, 0, 0, 0};

    // kCount blocks from kb0, kStripWaves apart; kWhole: all their codes lie before K
    auto run = [&](int kb0, auto count_of, auto whole_of) FP4Q_INLINE {
        constexpr int kCount = count_of.value;
        constexpr bool kWhole = whole_of.value;
        Raw ra[kCount], rw[kCount];
        float sa[kCount], s[kCount];
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int kb = kb0 + i * kStripWaves, low = kb * kGroup;
            if constexpr (kWhole) {
                rw[i] = {*reinterpret_cast<const u32x4 *>(w + low), *reinterpret_cast<const u32x4 *>(w + low + 64)};
                ra[i] = {*reinterpret_cast<const u32x4 *>(a + (row_a + low)),
                         *reinterpret_cast<const u32x4 *>(a + (row_a + low) + 64)};
            } else {
                const int left = p.K - 16 * quarter;
                rw[i] = {load_chunk(w, low, left), load_chunk(w, low + 64, left)};
                ra[i] = {load_chunk(a + row_a, low, left), load_chunk(a + row_a, low + 64, left)};
            }
            sa[i] = p.sa[(int64_t)kb * p.M + m];
            s[i] = p.sb[(int64_t)kb * tiles + tile];
        }
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            Frag<kFmtW, false> first;
            Frag<kFmtA, false> second;
            first.set(rw[i]);
            second.set(ra[i]);
            const f32x4 d = block_product<false>(first, second, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = fmaf(d[e] * s[i], sa[i], acc[e]);
        }
    };
    int kb = wave;
    for (; kb + (kAhead - 1) * kStripWaves < whole; kb += kAhead * kStripWaves)
        run(kb, std::integral_constant<int, kAhead>{}, std::true_type{});
    for (; kb + kStripWaves < whole; kb += 2 * kStripWaves) run(kb, std::integral_constant<int, 2>{}, std::true_type{});
    for (; kb < whole; kb += kStripWaves) run(kb, std::integral_constant<int, 1>{}, std::true_type{});
    for (; kb < blocks; kb += kStripWaves) run(kb, std::integral_constant<int, 1>{}, std::false_type{});

    part[wave][lane] = acc;
    __syncthreads();
    if (wave > 0 || lane >= 32 || row16 >= p.M) return;
    f32x4 u = part[0][lane + 32];
#pragma unroll 3
    for (int w = 1; w < kStripWaves; ++w) {
        acc += part[w][lane];
        u += part[w][lane + 32];
    }
    const int first = n0 + 4 * quarter;
    const int64_t at = (int64_t)row16 * p.N + first;
    with_act(p.act, [&](auto act) FP4Q_INLINE {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (first + e >= p.N) break;
            if (p.gate) {
                static_cast<bf16 *>(p.gate)[at + e] = from_float<bf16>(acc[e]);
                static_cast<bf16 *>(p.up)[at + e] = from_float<bf16>(u[e]);
            }
            static_cast<bf16 *>(p.out)[at + e] = from_float<bf16>(activate<act.value>(acc[e]).act * u[e]);
        }
    });
}

using Large = Shape<2, 4, 8, 4>;   // 256 rows by 128 outputs, a workgroup a CU
using Medium = Shape<2, 2, 4, 4>;  // 128 by 64, two workgroups a CU
using Low64 = Shape<2, 2, 2, 4>;   // 64 by 64
using Low32 = Shape<1, 4, 2, 2>;   // 32 by 64

template <template <int, int> class Kernel>
const void *pick(int fa, int fw) {
    if (fa == FP4Q_E4M3)
        return fw == FP4Q_E4M3 ? Kernel<FP4Q_E4M3, FP4Q_E4M3>::get() : Kernel<FP4Q_E4M3, FP4Q_E5M2>::get();
    return fw == FP4Q_E4M3 ? Kernel<FP4Q_E5M2, FP4Q_E4M3>::get() : Kernel<FP4Q_E5M2, FP4Q_E5M2>::get();
}
template <typename S>
struct Tiled {
    template <int kFmtA, int kFmtW>
    struct Kernel {
        static const void *get() { return (const void *)&gated_kernel<S, kFmtA, kFmtW>; }
    };
    static const void *get(int fa, int fw) { return pick<Kernel>(fa, fw); }
};
template <int kFmtA, int kFmtW>
struct Strip {
    static const void *get() { return (const void *)&gated_strip_kernel<kFmtA, kFmtW>; }
};

constexpr int64_t kLimit = kDimLimit / 2;
bool bad_gated(int64_t M, int64_t N, int64_t K) {
    return M < 0 || N < 0 || K < 0 || M >= kLimit || N >= kLimit || K >= kLimit ||
           ceil_div(M, 32) * ceil_div(N, 64) > (int64_t)0x7FFFFFFF / 16;
}
// The product's plan of the joined rows: tiles of both halves' columns.
Plan gated_plan(int64_t M, int64_t N, int64_t K) {
    Plan plan = plan_of(M, 2 * N, K, false);
    plan.tile_n /= 2;
    if (plan.parts > 1) {
        plan.part_size = ceil_div(M * N, 4) * 4;
        plan.workspace = (size_t)(2 * plan.part_size * plan.parts) * 4;
    }
    return plan;
}

}  // namespace

extern "C" {

int fp4q_gated8_workspace(int64_t M, int64_t N, int64_t K, size_t *bytes) {
    if (bad_gated(M, N, K)) return FP4Q_ERR_SHAPE;
    if (!bytes) return FP4Q_ERR_NULL;
    *bytes = M && N ? gated_plan(M, N, K).workspace : 0;
    return FP4Q_OK;
}

int fp4q_gated8(const uint8_t *a, int64_t a_pitch, int a_format, const float *a_scales,
                const uint8_t *w, int64_t w_pitch, int w_format, const float *w_scales, int64_t M,
                int64_t N, int64_t K, int act, void *y, void *gate, void *up, void *workspace,
                size_t workspace_bytes, void *stream) {
    if (bad_gated(M, N, K)) return FP4Q_ERR_SHAPE;
    if (K > 0 && (a_pitch < K || w_pitch < K || a_pitch >= (1 << 23) || w_pitch >= (1 << 23))) return FP4Q_ERR_SHAPE;
    if ((a_format != FP4Q_E4M3 && a_format != FP4Q_E5M2) || (w_format != FP4Q_E4M3 && w_format != FP4Q_E5M2) ||
        bad_act(act))
        return FP4Q_ERR_ARG;
    if (M == 0 || N == 0) return FP4Q_OK;
    const Plan plan = gated_plan(M, N, K);
    if (!y || (K > 0 && (!a || !a_scales || !w || !w_scales)) || (plan.workspace && !workspace)) return FP4Q_ERR_NULL;
    if (!gate != !up) return FP4Q_ERR_NULL;
    if (!aligned(y, 16) || !aligned(gate, 16) || !aligned(up, 16) || !aligned(workspace, 16)) return FP4Q_ERR_ALIGN;
    if (K > 0 && (!aligned(a, 16) || !aligned(w, 16) || a_pitch % 16 || w_pitch % 16)) return FP4Q_ERR_ALIGN;
    if (!aligned(a_scales, 4) || !aligned(w_scales, 4)) return FP4Q_ERR_ALIGN;
    if (workspace_bytes < plan.workspace) return FP4Q_ERR_SHAPE;
    const int64_t groups = ceil_div(K, kGroup), col_tiles = ceil_div(N, kGroup), second = col_tiles * kGroup;
    const Range outs[] = {rng(y, 2 * M * N), rng(gate, 2 * M * N), rng(up, 2 * M * N),
                          rng(workspace, (int64_t)plan.workspace)};
    const Range ins[] = {rng(a, pitched(M, K, a_pitch)), rng(w, pitched(second + N, K, w_pitch)),
                         rng(a_scales, 4 * groups * M), rng(w_scales, 4 * groups * 2 * col_tiles)};
    if (clash(outs, 4, ins, K > 0 ? 4 : 0)) return FP4Q_ERR_ARG;
    GatedArgs p;
    static_cast<GemmArgs &>(p) = {a, w, a_scales, w_scales, y, a_pitch, w_pitch, (int)M, (int)N, (int)K,
                                  (int)ceil_div(M, plan.tile_m), (int)ceil_div(N, plan.tile_n), 0,
                                  plan.parts, plan.part_size, static_cast<float *>(workspace)};
    p.second = (int)second;
    p.act = act;
    p.gate = gate;
    p.up = up;
    void *args[] = {&p};
    const void *fn = nullptr;
    int threads = kStripThreads;
    auto use = [&](auto shape) {
        using S = decltype(shape);
        fn = Tiled<S>::get(a_format, w_format);
        threads = S::kThreads;
    };
    switch (plan.way) {
        case Way::kStrip: fn = pick<Strip>(a_format, w_format); break;
        case Way::kLow32: use(Low32{}); break;
        case Way::kLow64: use(Low64{}); break;
        case Way::kMedium: use(Medium{}); break;
        case Way::kLarge: use(Large{}); break;
    }
    const int done = launch(fn, dim3((unsigned)(p.tiles_m * p.tiles_n * p.parts)), threads, args, stream);
    if (plan.parts == 1 || done != FP4Q_OK) return done;
    return launch((const void *)&gated_join_kernel, dim3((unsigned)ceil_div(M * N, 4 * kJoinThreads)), kJoinThreads,
                  args, stream);
}

}  // extern "C"
