// fp4q_gated8.hip -- the gated product of 8-bit operands (declared in include/fp4q_gated.h):
//
//   y[m][n] = act(g) u,  g = sum over k of a[m][k] w[n][k],  u = the same of row P + n of w
//
// One pass of the product's tiles (fp4q_gemm8_tile.h) over the joined weight.  Half of a
// tile's rows of w come from the gate, half from the up projection, dealt out so that a lane
// ends with both sums of an output in registers: the activation and the product are a few
// operations on them, and neither g nor u need be written and read again.
//
// Tiles are bound as fp4q_gemm8's, by loads, LDS reads and scaled additions beside the matrix
// cores: 8192 x 11008, K = 4096, with g and u 740 to 744 us, 1985 to 1995 TFLOP/s (of a tile's 69 us 11.5 are its
// beginning, the activation and three outputs); 2047 x 2752 53 to 54 us, 1719 to 1741 TFLOP/s.  Strips are bound
// by HBM: one row, 11008 x 4096 19.2 us, 4.7 TB/s of the weights (a large copy reaches 5.2).
#include "fp4q_act.h"
#include "fp4q_gated8_plan.h"
#include "fp4q_gemm8_tile.h"

namespace {

using namespace fp4q_f8;
using namespace fp4q_gated_plan;
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

// Few rows of a: the time is that of reading w once.  A workgroup takes units of 16 outputs in
// turn: 16 rows of the gate and the same 16 of the up projection, as two strips, for up to
// 16 kCols rows of a.  Its wavefronts share K, every kWaves-th block of 128 each; the next
// block's loads, or the next unit's, are under way while one is multiplied.  There are no
// branches around loads: what does not exist is read through an empty descriptor (behind a
// branch the compiler would wait for all loads under way).  A load takes the whole 128 bytes
// of 8 rows; they go through a part of LDS of the wavefront's own to the matrix core's rows.
// `rows` rows of `pitch` bytes at `base`, the last one to be read up to `wide` bytes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const uint8_t *base, int64_t first, int rows, int pitch, int wide) {
    const uint64_t at = (uint64_t)base + (uint64_t)(first * pitch);
    // (all of it is uniform, which the compiler does not see in a loop)
    const unsigned low = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)at);
    const unsigned high = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)(at >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void *)((uint64_t)high << 32 | low), 0,
                                             __builtin_amdgcn_readfirstlane(rows > 0 ? (rows - 1) * pitch + wide : 0),
                                             0x00020000);
}
// 16 bytes of which the first `keep` count.
__device__ __forceinline__ u32x4 keep_bytes(u32x4 w, int keep) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = keep - 4 * i;
        w[i] = k >= 4 ? w[i] : k <= 0 ? 0u : w[i] & ((1u << (8 * k)) - 1);
    }
    return w;
}

template <int kFmtA, int kFmtW, int kWaves, int kCols>
__global__ __launch_bounds__(kWaves *kWave) void gated_strip_kernel(GatedArgs p) {
    __shared__ u32x4 turn[kWaves][16 * 8];  // chunk c of row r at chunk c ^ (r / 2 & 7)
    extern __shared__ float sums_room[];    // a unit's [kWaves][2][M][16], or two units' in turn
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int row16 = lane & 15, quarter = lane >> 4;
    const int blocks = (p.K + kGroup - 1) / kGroup, turns = (blocks + kWaves - 1) / kWaves;
    const int units = (p.N + kStripOut - 1) / kStripOut, step = (int)gridDim.x;
    const int tiles = 2 * (p.second / kGroup), wide = (p.K + 15) & ~15, w_pitch = (int)p.b_pitch, a_pitch = (int)p.a_pitch;

    float *sums = sums_room;
    const int sums_each = kWaves * 2 * p.M * 16;

    const int row8 = lane >> 3, chunk = (lane & 7) ^ (row8 >> 1);
    const int w_at = row8 * w_pitch + 16 * chunk, w_at8 = (row8 + 8) * w_pitch + 16 * (chunk ^ 4);
    const auto a_rows = rows_at(p.a, 0, p.M, a_pitch, wide);
    struct Part {  // a block of a
        Raw codes[kCols];
        float scale[kCols];
    };
    auto load_a = [&](Part &to, int turn_) {
        const int kb = min(wave + turn_ * kWaves, blocks - 1);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
            const int m = min(16 * c + row16, p.M - 1), at = m * a_pitch + 16 * quarter;
            to.codes[c].low = __builtin_amdgcn_raw_buffer_load_b128(a_rows, at, kb * kGroup, 0);
            to.codes[c].high = __builtin_amdgcn_raw_buffer_load_b128(a_rows, at + 64, kb * kGroup, 0);
            to.scale[c] = p.sa[(int64_t)kb * p.M + m];
        }
    };
    struct Fetched {  // a block of a strip of w
        u32x4 codes[2];
        float scale;
    };
    auto load_w = [&](Fetched &to, int unit, int turn_, int strip) {
        const int n0 = unit * kStripOut, kb = wave + turn_ * kWaves;
        const int here = unit < units && kb < blocks ? min(kStripOut, p.N - n0) : 0;
        const auto rows = rows_at(p.b, (int64_t)n0 + (strip ? p.second : 0), here, w_pitch, wide);
        to.codes[0] = __builtin_amdgcn_raw_buffer_load_b128(rows, w_at, kb * kGroup, 0);
        to.codes[1] = __builtin_amdgcn_raw_buffer_load_b128(rows, w_at8, kb * kGroup, 0);
        // (a block or a unit that does not exist has zero codes and a zero scale)
        const int tile = min(n0, p.N - 1) / kGroup + (strip ? tiles / 2 : 0);
        to.scale = here > 0 ? p.sb[(int64_t)min(kb, blocks - 1) * tiles + tile] : 0.0f;
    };
    int load_unit = (int)blockIdx.x, load_turn = 0, unit = load_unit, turn_now = 0;
    auto advance = [&](int &of, int &at) {
        const bool last = ++at == turns;
        at = last ? 0 : at;
        of += last ? step : 0;
    };
    Part part;
    Fetched fetched[2];
    load_a(part, 0);
    load_w(fetched[0], load_unit, 0, 0);
    load_w(fetched[1], load_unit, 0, 1);
    advance(load_unit, load_turn);

    f32x4 acc[2][kCols];
    auto clear = [&]() {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int c = 0; c < kCols; ++c) acc[s][c] = f32x4{0, 0, 0, 0};
    };
    clear();
    // two units' sums in turn: one meeting a unit keeps writers and readers apart
    auto finish = [&]() {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                if (16 * c + row16 < p.M)
                    *reinterpret_cast<f32x4 *>(sums + ((wave * 2 + s) * p.M + 16 * c + row16) * 16 + 4 * quarter) = acc[s][c];
        __syncthreads();
        for (int t = threadIdx.x; t < p.M * kStripOut; t += kWaves * kWave) {
            const int m = t / kStripOut, n = unit * kStripOut + t % kStripOut;
            if (n >= p.N) continue;
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                g += sums[w * 2 * p.M * 16 + t];
                u += sums[(w * 2 + 1) * p.M * 16 + t];
            }
            const int64_t to = (int64_t)m * p.N + n;
            if (p.gate) {
                static_cast<bf16 *>(p.gate)[to] = from_float<bf16>(g);
                static_cast<bf16 *>(p.up)[to] = from_float<bf16>(u);
            }
            with_act(p.act, [&](auto act) FP4Q_INLINE { g = activate<act.value>(g).act * u; });
            static_cast<bf16 *>(p.out)[to] = from_float<bf16>(g);
        }
        sums = sums == sums_room ? sums + sums_each : sums_room;
        clear();
    };

    const int mine = (units - 1 - (int)blockIdx.x) / step + 1;
    for (int left = mine * turns; left > 0; --left) {
        const int kb = wave + turn_now * kWaves, end = p.K - kb * kGroup;  // codes from `end` on do not count
        if (end < kGroup) {
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                part.codes[c].low = keep_bytes(part.codes[c].low, end - 16 * quarter);
                part.codes[c].high = keep_bytes(part.codes[c].high, end - 16 * quarter - 64);
                // a block that does not exist: a's last one's scale was read, and 0 times an infinity is not 0
                part.scale[c] = end > 0 ? part.scale[c] : 0.0f;
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                fetched[s].codes[0] = keep_bytes(fetched[s].codes[0], end - 16 * chunk);
                fetched[s].codes[1] = keep_bytes(fetched[s].codes[1], end - 16 * (chunk ^ 4));
            }
        }
        Frag<kFmtA, false> second[kCols];
        float sa[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
            second[c].set(part.codes[c]);
            sa[c] = part.scale[c];
        }
        load_a(part, load_turn);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            u32x4 *const mine_here = turn[wave];
            mine_here[lane] = fetched[s].codes[0];
            mine_here[64 + lane] = fetched[s].codes[1];
            const float sw = fetched[s].scale;
            load_w(fetched[s], load_unit, load_turn, s);
            Frag<kFmtW, false> first;
            first.set({mine_here[row16 * 8 + (quarter ^ (row16 >> 1))], mine_here[row16 * 8 + ((quarter + 4) ^ (row16 >> 1))]});
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const f32x4 d = block_product<false>(first, second[c], 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[s][c][e] = fmaf(d[e] * sw, sa[c], acc[s][c][e]);
            }
        }
        advance(load_unit, load_turn);
        if (turn_now == turns - 1) finish();
        advance(unit, turn_now);
    }
}

using Large = Shape<2, 4, 8, 4>;   // 256 rows by 128 outputs, a workgroup a CU
using Tall = Shape<2, 4, 6, 4>;    // 192 by 128, a workgroup a CU
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
template <int kWaves, int kCols>
struct Strip {
    template <int kFmtA, int kFmtW>
    struct Kernel {
        static const void *get() { return (const void *)&gated_strip_kernel<kFmtA, kFmtW, kWaves, kCols>; }
    };
    static const void *get(int fa, int fw) { return pick<Kernel>(fa, fw); }
};

constexpr int64_t kLimit = kDimLimit / 2;
bool bad_gated(int64_t M, int64_t N, int64_t K) {
    return M < 0 || N < 0 || K < 0 || M >= kLimit || N >= kLimit || K >= kLimit ||
           ceil_div(M, 32) * ceil_div(N, 64) > (int64_t)0x7FFFFFFF / 16;
}
}  // namespace

extern "C" {

int fp4q_gated8_workspace(int64_t M, int64_t N, int64_t K, size_t *bytes) {
    if (bad_gated(M, N, K)) return FP4Q_ERR_SHAPE;
    if (!bytes) return FP4Q_ERR_NULL;
    *bytes = M && N ? plan_of(M, N, K).workspace : 0;
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
    const Plan plan = plan_of(M, N, K);
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
    if (plan.way == Way::kStrip) {
        const int waves = M <= 32 ? 16 : 8;
        const void *fn = M <= 16 ? Strip<16, 1>::get(a_format, w_format)
                         : M <= 32 ? Strip<16, 2>::get(a_format, w_format) : Strip<8, 4>::get(a_format, w_format);
        // one unit's sums where no workgroup has a second one: always with more than 16 rows (plan_of)
        const int64_t units = ceil_div(N, kStripOut), places = units > kCus ? 2 : 1;
        const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)(units < kCus ? units : kCus)), dim3(waves * kWave), args,
                                             (size_t)(places * waves * 2 * M * 16 * 4), (hipStream_t)stream);
        return e == hipSuccess ? FP4Q_OK : FP4Q_ERR_LAUNCH;
    }
    const void *fn = nullptr;
    int threads = 0;
    auto use = [&](auto shape) {
        using S = decltype(shape);
        fn = Tiled<S>::get(a_format, w_format);
        threads = S::kThreads;
    };
    switch (plan.way) {
        case Way::kStrip: break;
        case Way::kLow32: use(Low32{}); break;
        case Way::kLow64: use(Low64{}); break;
        case Way::kMedium: use(Medium{}); break;
        case Way::kTall: use(Tall{}); break;
        case Way::kLarge: use(Large{}); break;
    }
    const int done = launch(fn, dim3((unsigned)(p.tiles_m * p.tiles_n * p.parts)), threads, args, stream);
    if (plan.parts == 1 || done != FP4Q_OK) return done;
    return launch((const void *)&gated_join_kernel, dim3((unsigned)ceil_div(M * N, 4 * kJoinThreads)), kJoinThreads,
                  args, stream);
}

}  // extern "C"
