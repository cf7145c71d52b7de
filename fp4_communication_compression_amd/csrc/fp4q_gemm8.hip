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
    // scale operands 127 = 2^0: the matrix core's own scaling is not used
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(first.v, second.v, f32x4{0, 0, 0, 0}, kFirst, kSecond,
                                                            0, 127, 0, 127);
}
template <int kFirst, int kSecond>
__device__ __forceinline__ f32x4 block_product(const Frag<kFirst, true> &first, const Frag<kSecond, true> &second) {
    f32x4 d = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(first.v[i], second.v[i], d, 0, 0, 0);
    return d;
}

// 16 bytes of a row at byte k of K: zero from K on.
__device__ __forceinline__ u32x4 load_chunk(const uint8_t *row, int k, int K) {
    if (k >= K) return u32x4{0, 0, 0, 0};
    u32x4 w = *reinterpret_cast<const u32x4 *>(row + k);
    const int left = K - k;
    if (left < 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int keep = left - 4 * i;
            w[i] = keep >= 4 ? w[i] : keep <= 0 ? 0u : w[i] & ((1u << (8 * keep)) - 1);
        }
    }
    return w;
}

constexpr int kBM = 128, kBN = 128, kThreads = 256;

// kTiles: b's scales are tiles.  LDS rows are 128 bytes, chunk c of row r at
// chunk c ^ (r & 7).
template <int kFmtA, int kFmtB, bool kTiles, bool kPrecise>
__global__ __launch_bounds__(kThreads) void gemm_kernel(GemmArgs p) {
    __shared__ u32x4 lds_a[kBM * 8], lds_b[kBN * 8];
    const int t = threadIdx.x, lane = t & 63, wave = t / 64;
    const int tm = (int)(blockIdx.x % (unsigned)p.tiles_m), tn = (int)(blockIdx.x / (unsigned)p.tiles_m);
    const int m0 = tm * kBM, n0 = tn * kBN;
    const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
    const int row16 = lane & 15, quarter = lane >> 4;
    const int blocks = (p.K + kGroup - 1) / kGroup;
    const int sb_pitch = kTiles ? (p.N + kGroup - 1) / kGroup : p.N;

    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    for (int kb = 0; kb < blocks; ++kb) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kBM * 8 / kThreads; ++i) {
            const int q = i * kThreads + t, r = q >> 3, c = q & 7;
            const int m = min(m0 + r, p.M - 1), n = min(n0 + r, p.N - 1);
            lds_a[r * 8 + (c ^ (r & 7))] = load_chunk(p.a + m * p.a_pitch, kb * kGroup + 16 * c, p.K);
            lds_b[r * 8 + (c ^ (r & 7))] = load_chunk(p.b + n * p.b_pitch, kb * kGroup + 16 * c, p.K);
        }
        __syncthreads();
        Frag<kFmtB, kPrecise> fb[4];
        f32x4 sb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = wn + j * 16 + row16;
            fb[j].set(lds_b[r * 8 + ((2 * quarter) ^ (r & 7))], lds_b[r * 8 + ((2 * quarter + 1) ^ (r & 7))]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = min(n0 + wn + j * 16 + 4 * quarter + e, p.N - 1);
                sb[j][e] = p.sb[(int64_t)kb * sb_pitch + (kTiles ? n / kGroup : n)];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = wm + i * 16 + row16;
            Frag<kFmtA, kPrecise> fa;
            fa.set(lds_a[r * 8 + ((2 * quarter) ^ (r & 7))], lds_a[r * 8 + ((2 * quarter + 1) ^ (r & 7))]);
            const float sa = p.sa[(int64_t)kb * p.M + min(m0 + r, p.M - 1)];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4 d = block_product(fb[j], fa);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[e], sa * sb[j][e], acc[i][j][e]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + wm + i * 16 + row16;
        if (m >= p.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = n0 + wn + j * 16 + 4 * quarter + e;
                if (n >= p.N) continue;
                const int64_t at = (int64_t)m * p.N + n;
                if (p.out_f32) {
                    float *o = static_cast<float *>(p.out) + at;
                    *o = p.accumulate ? *o + acc[i][j][e] : acc[i][j][e];
                } else {
                    static_cast<bf16 *>(p.out)[at] = from_float<bf16>(acc[i][j][e]);
                }
            }
    }
}

template <int kFmtA, int kFmtB>
const void *pick(bool tiles, bool precise) {
    if (precise)
        return tiles ? (const void *)&gemm_kernel<kFmtA, kFmtB, true, true>
                     : (const void *)&gemm_kernel<kFmtA, kFmtB, false, true>;
    return tiles ? (const void *)&gemm_kernel<kFmtA, kFmtB, true, false>
                 : (const void *)&gemm_kernel<kFmtA, kFmtB, false, false>;
}
const void *pick(int fa, int fb, bool tiles, bool precise) {
    if (fa == FP4Q_E4M3)
        return fb == FP4Q_E4M3 ? pick<FP4Q_E4M3, FP4Q_E4M3>(tiles, precise)
                               : pick<FP4Q_E4M3, FP4Q_E5M2>(tiles, precise);
    return fb == FP4Q_E4M3 ? pick<FP4Q_E5M2, FP4Q_E4M3>(tiles, precise)
                           : pick<FP4Q_E5M2, FP4Q_E5M2>(tiles, precise);
}

bool bad_gemm(int64_t M, int64_t N, int64_t K) {
    return M < 0 || N < 0 || K < 0 || M >= kDimLimit || N >= kDimLimit || K >= kDimLimit ||
           ceil_div(M, kBM) * ceil_div(N, kBN) > (int64_t)0x7FFFFFFF;
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
                  (int)ceil_div(M, kBM), (int)ceil_div(N, kBN), out_dtype == FP4Q_OUT_F32, add};
    void *args[] = {&p};
    return launch(pick(a_format, b_format, tiles, p.out_f32), dim3((unsigned)(p.tiles_m * p.tiles_n)), kThreads, args, stream);
}

}  // extern "C"
