// fp4q_gemm8.hip -- the product of two 8-bit operands with a scale for each block
// of 128 (declared in include/fp4q_linear.h):
//
//   out[m][n] = sum over blocks kb of sa[kb][m] sb[kb][n or n / 128]
//               sum over k in kb of a[m][k] b[n][k]
//
// b is the matrix core's first operand: a lane then holds four neighbouring n of
// one m, a's scale is one value per lane, and the output leaves in pieces of four
// neighbours.  A block's sum over its 128 k is scaled by the block's two scales
// and added to the fp32 accumulators.
//
// Two ways to the block's sum:
//   8-bit matrix core  (bf16 output) one v_mfma_f32_16x16x128_f8f6f4 covers the
//     block of a 16 x 16 tile.  It adds the products of 8 neighbouring k at the
//     largest one's exponent and drops what lies below 2^-13 of it (seen with
//     powers of two; groups of 8 are added in fp32): about 2e-5 of the result,
//     a hundredth of the output's own rounding.
//   16-bit matrix core (fp32 output) the codes become bf16, which holds every
//     E4M3 and E5M2 value, and four v_mfma_f32_16x16x32_bf16 add their exact
//     products in fp32: half the rate, 1e-8 per block.
#include "fp4q_f8.h"

namespace {

using namespace fp4q_f8;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct GemmArgs {
    const uint8_t *a, *b;
    const float *sa, *sb;
    void *out;
    int64_t a_pitch, b_pitch;
    int M, N, K;
    int tiles_m, tiles_n;
    int out_f32, accumulate;
};

// 32 codes of one row (half a block's 64 for every 16 lanes, in the order that both
// operands share) as the matrix core takes them.
template <int kFmt, bool kPrecise>
struct Frag;
template <int kFmt>
struct Frag<kFmt, false> {
    i32x8 v;
    __device__ __forceinline__ void set(u32x4 lo, u32x4 hi) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = (int)lo[i];
            v[4 + i] = (int)hi[i];
        }
    }
};
template <int kFmt>
struct Frag<kFmt, true> {
    bf16x8 v[4];
    __device__ __forceinline__ void set(u32x4 lo, u32x4 hi) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned w = i < 4 ? lo[i] : hi[i - 4];
            bf16x2 p, q;
            if constexpr (kFmt == FP4Q_E4M3) {
                p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
                q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true);
            } else {
                p = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.0f, false);
                q = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.0f, true);
            }
            const int at = 4 * (i & 1);
            v[i >> 1][at] = p[0];
            v[i >> 1][at + 1] = p[1];
            v[i >> 1][at + 2] = q[0];
            v[i >> 1][at + 3] = q[1];
        }
    }
};

// One block's product of a 16 x 16 tile.
template <int kFirst, int kSecond>
__device__ __forceinline__ f32x4 block_product(const Frag<kFirst, false> &first, const Frag<kSecond, false> &second) {
    // with scale operands 0 this is the instruction without the matrix core's own scaling
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(first.v, second.v, f32x4{0, 0, 0, 0}, kFirst, kSecond,
                                                            0, 0, 0, 0);
}
template <int kFirst, int kSecond>
__device__ __forceinline__ f32x4 block_product(const Frag<kFirst, true> &first, const Frag<kSecond, true> &second) {
    f32x4 d = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(first.v[i], second.v[i], d, 0, 0, 0);
    return d;
}

// A workgroup's tile: kWavesM x kWavesN wavefronts of kTilesM x kTilesN tiles of
// 16 x 16 each, a block of 128 k at a time.
template <int kWavesM_, int kWavesN_, int kTilesM_, int kTilesN_>
struct Shape {
    static constexpr int kWavesM = kWavesM_, kWavesN = kWavesN_, kTilesM = kTilesM_, kTilesN = kTilesN_;
    static constexpr int kWaveM = 16 * kTilesM, kWaveN = 16 * kTilesN;
    static constexpr int kM = kWavesM * kWaveM, kN = kWavesN * kWaveN;
    static constexpr int kWaves = kWavesM * kWavesN;
    static constexpr int kThreads = kWave * kWaves;
    static constexpr int kLoads = (kM + kN) / 8 / kWaves;  // 8 rows of 128 bytes per load and wavefront
    static_assert((kM + kN) % (8 * kWaves) == 0 && kM % 8 == 0, "whole loads");
};

typedef __attribute__((address_space(3))) void lds_void;

// One block of both operands with its scales, as staged in LDS.  Rows are 128 bytes;
// chunk c (16 bytes) of row r lies at chunk c ^ (r & 7), so that 8 rows' equal
// chunks meet 8 different bank groups.
template <typename S>
struct alignas(16) Stage {
    u32x4 a[S::kM * 8], b[S::kN * 8];
    float sa[S::kM], sb[S::kN];
};

template <typename S, int kFmtA, int kFmtB, bool kTiles, bool kPrecise>
struct Tile {
    const GemmArgs &p;
    int lane, wave, m0, n0, wm, wn, row16, quarter;
    int offset[S::kLoads];  // of each load's bytes from its operand's tile
    __amdgpu_buffer_rsrc_t ra, rb;
    f32x4 acc[S::kTilesM][S::kTilesN];

    __device__ __forceinline__ Tile(const GemmArgs &args, int tm, int tn) : p(args) {
        lane = threadIdx.x & (kWave - 1);
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        m0 = tm * S::kM;
        n0 = tn * S::kN;
        wm = wave % S::kWavesM * S::kWaveM;
        wn = wave / S::kWavesM * S::kWaveN;
        row16 = lane & 15;
        quarter = lane >> 4;
        // rows past the end repeat the last one, and the descriptors end with the last
        // row's last whole 16 bytes: no load leaves an operand
        const int rows_a = min(S::kM, p.M - m0), rows_b = min(S::kN, p.N - n0);
        const int wide = (p.K + 15) & ~15;
        ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p.a) + (int64_t)m0 * p.a_pitch, 0,
                                               (rows_a - 1) * (int)p.a_pitch + wide, 0x00020000);
        rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p.b) + (int64_t)n0 * p.b_pitch, 0,
                                               (rows_b - 1) * (int)p.b_pitch + wide, 0x00020000);
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) {
            const int r = (i * S::kWaves + wave) * 8 + (lane >> 3), chunk = (lane & 7) ^ (lane >> 3);
            const bool of_a = (i * S::kWaves + wave) * 8 < S::kM;
            offset[i] = 16 * chunk + (of_a ? min(r, rows_a - 1) * (int)p.a_pitch
                                           : min(r - S::kM, rows_b - 1) * (int)p.b_pitch);
        }
#pragma unroll
        for (int i = 0; i < S::kTilesM; ++i)
#pragma unroll
            for (int j = 0; j < S::kTilesN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    }

    // Queues block kb's loads, straight into LDS.
    __device__ __forceinline__ void fetch(Stage<S> &to, int kb) {
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) {
            const int r0 = (i * S::kWaves + wave) * 8;
            if (r0 < S::kM)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(to.a + r0 * 8), 16, offset[i],
                                                         kb * kGroup, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void *)(to.b + (r0 - S::kM) * 8), 16, offset[i],
                                                         kb * kGroup, 0, 0);
        }
        // scales, 64 to a wavefront; of b's tiles one for each 128 columns
        constexpr int kScalesB = kTiles ? (S::kN + kGroup - 1) / kGroup : S::kN;
#pragma unroll
        for (int k = 0; k < S::kM; k += kWave)
            if (wave == k / kWave % S::kWaves) {
                const float *from = p.sa + (int64_t)kb * p.M + min(m0 + k + lane, p.M - 1);
                __builtin_amdgcn_global_load_lds(const_cast<float *>(from), (lds_void *)(to.sa + k), 4, 0, 0);
            }
#pragma unroll
        for (int k = 0; k < kScalesB; k += kWave)
            if (wave == S::kWaves - 1 - k / kWave % S::kWaves) {
                const int cols = kTiles ? (p.N + kGroup - 1) / kGroup : p.N, c0 = kTiles ? n0 / kGroup : n0;
                const float *from = p.sb + (int64_t)kb * cols + min(c0 + k + lane, cols - 1);
                __builtin_amdgcn_global_load_lds(const_cast<float *>(from), (lds_void *)(to.sb + k), 4, 0, 0);
            }
    }

    // Clears the codes from K on in the last block.
    __device__ __forceinline__ void clear_tail(Stage<S> &in) {
        const int left = p.K % kGroup;
        for (int r = threadIdx.x; r < S::kM + S::kN; r += S::kThreads) {
            u32x4 *row = r < S::kM ? in.a + r * 8 : in.b + (r - S::kM) * 8;
            for (int c = left / 16; c < 8; ++c) {
                u32x4 w = row[c ^ (r & 7)];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int keep = left - 16 * c - 4 * i;
                    w[i] = keep >= 4 ? w[i] : keep <= 0 ? 0u : w[i] & ((1u << (8 * keep)) - 1);
                }
                row[c ^ (r & 7)] = w;
            }
        }
    }

    // Rows row .. row + 15; row is a multiple of 8.
    template <int kFmt>
    __device__ __forceinline__ Frag<kFmt, kPrecise> frag(const u32x4 *rows, int row) {
        const u32x4 *mine = rows + row16 * 8 + row * 8;
        Frag<kFmt, kPrecise> f;
        f.set(mine[(2 * quarter) ^ (row16 & 7)], mine[(2 * quarter + 1) ^ (row16 & 7)]);
        return f;
    }

    // The products run kLag tiles ahead of their scaled addition, so that the vector
    // unit adds one tile while the matrix core works on the next ones.
    __device__ __forceinline__ void multiply(const Stage<S> &in) {
        constexpr int kLag = 3, kCount = S::kTilesM * S::kTilesN;
        Frag<kFmtB, kPrecise> fb[S::kTilesN];
        f32x4 sb[S::kTilesN], d[kLag + 1];
        float sa[2], sb_tile = 1.0f;
#pragma unroll
        for (int j = 0; j < S::kTilesN; ++j) fb[j] = frag<kFmtB>(in.b, wn + j * 16);
        Frag<kFmtA, kPrecise> fa[2];
        fa[0] = frag<kFmtA>(in.a, wm);
        sa[0] = in.sa[wm + row16];
        if constexpr (kTiles) {
            static_assert(kGroup % S::kWaveN == 0, "one tile of b's scales per wavefront");
            sb_tile = in.sb[wn / kGroup];
            sa[0] *= sb_tile;
        } else {
#pragma unroll
            for (int j = 0; j < S::kTilesN; ++j)
                sb[j] = *reinterpret_cast<const f32x4 *>(in.sb + wn + j * 16 + 4 * quarter);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < kCount + kLag; ++t) {
            const int i = t / S::kTilesN, j = t % S::kTilesN;
            if (t < kCount) {
                if (j == 0 && i + 1 < S::kTilesM) fa[(i + 1) & 1] = frag<kFmtA>(in.a, wm + (i + 1) * 16);
                if (j == S::kTilesN - 1 && i + 1 < S::kTilesM)
                    sa[(i + 1) & 1] = in.sa[wm + (i + 1) * 16 + row16] * sb_tile;
                d[t % (kLag + 1)] = block_product(fb[j], fa[i & 1]);
            }
            if (t >= kLag) {
                const int ui = (t - kLag) / S::kTilesN, uj = (t - kLag) % S::kTilesN;
                const f32x4 v = d[(t - kLag) % (kLag + 1)];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[ui][uj][e] = fmaf(v[e], kTiles ? sa[ui & 1] : sa[ui & 1] * sb[uj][e], acc[ui][uj][e]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // the sums are due here: without this the compiler moves the work above into the
        // next block's branches and keeps all fragments alive for it
#pragma unroll
        for (int i = 0; i < S::kTilesM; ++i)
#pragma unroll
            for (int j = 0; j < S::kTilesN; ++j) asm volatile("" : "+v"(acc[i][j]));
    }

    __device__ __forceinline__ void store() {
#pragma unroll
        for (int i = 0; i < S::kTilesM; ++i) {
            const int m = m0 + wm + i * 16 + row16;
            if (m >= p.M) continue;
#pragma unroll
            for (int j = 0; j < S::kTilesN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = n0 + wn + j * 16 + 4 * quarter + e;
                    if (n >= p.N) continue;
                    const int64_t at = (int64_t)m * p.N + n;
                    if (kPrecise) {
                        float *o = static_cast<float *>(p.out) + at;
                        *o = p.accumulate ? *o + acc[i][j][e] : acc[i][j][e];
                    } else {
                        static_cast<bf16 *>(p.out)[at] = from_float<bf16>(acc[i][j][e]);
                    }
                }
        }
    }
};

// Two blocks in LDS: one is multiplied while the next one's loads are under way.
template <typename S, int kFmtA, int kFmtB, bool kTiles, bool kPrecise>
__global__ __launch_bounds__(S::kThreads, 2) void gemm_kernel(GemmArgs p) {
    __shared__ Stage<S> even;
    __shared__ Stage<S> odd;
    // consecutive workgroups go to the 8 XCDs in turn: each XCD takes a run of tiles,
    // and a run walks 8 tiles of m before it steps in n, so that the tiles that an XCD
    // works on at one time share their operands in its L2
    const int count = p.tiles_m * p.tiles_n, each = count / 8, more = count % 8;
    const int xcd = (int)blockIdx.x % 8, turn = (int)blockIdx.x / 8;
    const int at = xcd * each + min(xcd, more) + turn;
    const int band = at / (8 * p.tiles_n), in_band = at - band * 8 * p.tiles_n;
    const int high = min(8, p.tiles_m - band * 8);
    const int tm = band * 8 + in_band % high, tn = in_band / high;
    Tile<S, kFmtA, kFmtB, kTiles, kPrecise> t(p, tm, tn);
    const int blocks = (p.K + kGroup - 1) / kGroup, ragged = p.K % kGroup;
    int kb = 0;
    if (blocks & 1) {  // then pairs of blocks are left
        t.fetch(odd, 0);
        __syncthreads();
        if (blocks > 1) {
            t.fetch(even, 1);
        } else if (ragged) {
            t.clear_tail(odd);
            __syncthreads();
        }
        t.multiply(odd);
        kb = 1;
    } else if (blocks) {
        t.fetch(even, 0);
    }
    for (; kb < blocks; kb += 2) {
        // the loads of block kb have landed, and nobody reads the other buffer
        __syncthreads();
        t.fetch(odd, kb + 1);
        t.multiply(even);
        __syncthreads();
        if (kb + 2 < blocks) {
            t.fetch(even, kb + 2);
        } else if (ragged) {
            t.clear_tail(odd);
            __syncthreads();
        }
        t.multiply(odd);
    }
    t.store();
}

using Large = Shape<2, 4, 8, 4>;
using LargePrecise = Shape<2, 4, 4, 4>;
using Small = Shape<2, 2, 4, 4>;

template <typename S, bool kPrecise, int kFmtA, int kFmtB>
const void *pick(bool tiles) {
    return tiles ? (const void *)&gemm_kernel<S, kFmtA, kFmtB, true, kPrecise>
                 : (const void *)&gemm_kernel<S, kFmtA, kFmtB, false, kPrecise>;
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
           ceil_div(M, Small::kM) * ceil_div(N, Small::kN) > (int64_t)0x7FFFFFFF;
}

}  // namespace

extern "C" {

int fp4q_gemm8_workspace(int64_t M, int64_t N, int64_t K, uint32_t flags, size_t *bytes) {
    if (bad_gemm(M, N, K)) return FP4Q_ERR_SHAPE;
    if (flags & ~(uint32_t)(FP4Q_FLAG_TILES | FP4Q_FLAG_ACCUMULATE)) return FP4Q_ERR_ARG;
    if (!bytes) return FP4Q_ERR_NULL;
    *bytes = 0;
    return FP4Q_OK;
}

int fp4q_gemm8(const uint8_t *a, int64_t a_pitch, int a_format, const float *a_scales,
               const uint8_t *b, int64_t b_pitch, int b_format, const float *b_scales, int64_t M,
               int64_t N, int64_t K, void *out, int out_dtype, uint32_t flags, void *workspace,
               size_t workspace_bytes, void *stream) {
    size_t need = 0;
    if (bad_gemm(M, N, K)) return FP4Q_ERR_SHAPE;
    if (K > 0 && (a_pitch < K || b_pitch < K || a_pitch >= (1 << 23) || b_pitch >= (1 << 23))) return FP4Q_ERR_SHAPE;
    const int st = fp4q_gemm8_workspace(M, N, K, flags, &need);
    if (st != FP4Q_OK) return st;
    const bool add = flags & FP4Q_FLAG_ACCUMULATE, tiles = flags & FP4Q_FLAG_TILES;
    if (out_dtype != FP4Q_OUT_F32 && (out_dtype != FP4Q_OUT_BF16 || add)) return FP4Q_ERR_ARG;
    if ((a_format != FP4Q_E4M3 && a_format != FP4Q_E5M2) || (b_format != FP4Q_E4M3 && b_format != FP4Q_E5M2))
        return FP4Q_ERR_ARG;
    if (M == 0 || N == 0) return FP4Q_OK;
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
                  0, 0, out_dtype == FP4Q_OUT_F32, add};
    void *args[] = {&p};
    const bool precise = p.out_f32;
    const int lm = precise ? LargePrecise::kM : Large::kM, ln = precise ? LargePrecise::kN : Large::kN;
    const bool large = ceil_div(M, lm) * ceil_div(N, ln) >= 200;
    p.tiles_m = (int)ceil_div(M, large ? lm : Small::kM);
    p.tiles_n = (int)ceil_div(N, large ? ln : Small::kN);
    const void *fn = large ? precise ? pick<LargePrecise, true>(a_format, b_format, tiles)
                                     : pick<Large, false>(a_format, b_format, tiles)
                   : precise ? pick<Small, true>(a_format, b_format, tiles)
                             : pick<Small, false>(a_format, b_format, tiles);
    return launch(fn, dim3((unsigned)(p.tiles_m * p.tiles_n)), large ? 512 : 256, args, stream);
}

}  // extern "C"
