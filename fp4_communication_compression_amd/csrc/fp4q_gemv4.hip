// fp4q_gemv4.hip -- a few rows times a weight held as an FP4 payload, and the gated form of
// two such products (declared in include/fp4q_gated.h):
//
//   out[m][n] = sum over blocks b of 256 of s[n][b] sum over k in b of x[m][k] e[n][k] u[n][k / 16]
//
// with E2M1 codes e, E4M3 micro-scales u and fp32 block scales s.  e u has at most 6
// significant bits, so it is exact in bf16, and so are its products with a bf16 x in the
// 16-bit matrix core, which adds them in fp32.  An fp32 x (given, or x transformed instead of
// a transformed weight) is cut into three bf16 parts that sum to it; the parts are rows of
// their own, three to a row of x, and their sums are added at the end: the matrix core has 16
// columns anyway, and the time is that of reading the payload.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "fp4q_act.h"
#include "fp4q_f8.h"

namespace {

using namespace fp4q_f8;
using namespace fp4q_act;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kBlock = FP4Q_BLOCK, kStrip = 16, kParts = 3;

struct Payload {
    const uint8_t *codes, *micro;
    const float *block;
};
struct Gemv4Args {
    const uint16_t *x;  // [M parts x K] bf16
    Payload w, up;      // up: the gated form's second weight
    void *out;
    int M, N, K, parts, act, out_f32;
};

// ------------------------------------------------------------------ x in parts
// A wavefront takes a block of 256 of a row, four neighbours a lane: the Walsh-Hadamard
// transform in fp32 (strides 1 and 2 in a lane, 4 to 128 over the lanes), then three parts of
// 8 bits each, cut off and not rounded, so that a part never leaves bf16's range.
template <typename T, bool kTransform>
__global__ __launch_bounds__(kWave) void parts_kernel(const T *x, uint16_t *parts, int K) {
    const int lane = threadIdx.x, blocks = K / kBlock;
    const int64_t row = (int64_t)(blockIdx.x / (unsigned)blocks);
    const int k = (int)(blockIdx.x % (unsigned)blocks) * kBlock + 4 * lane;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = to_float(x[row * K + k + i]);
    if constexpr (kTransform) {
        const float a = v[0] + v[1], b = v[0] - v[1], c = v[2] + v[3], d = v[2] - v[3];
        v[0] = a + c;
        v[1] = b + d;
        v[2] = a - c;
        v[3] = b - d;
#pragma unroll
        for (int far = 1; far < kWave; far *= 2) {
            const bool second = lane & far;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float other = __shfl_xor(v[i], far);
                v[i] = second ? other - v[i] : v[i] + other;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= 0.0625f;
    }
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
        u32x2 w = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned high = __float_as_uint(v[i]) & 0xFFFF0000u;
            w[i >> 1] |= i & 1 ? high : high >> 16;
            // what is not finite is all in the first part
            v[i] = mag(v[i]) < 0x7F800000u ? v[i] - __uint_as_float(high) : 0.0f;
        }
        *reinterpret_cast<u32x2 *>(parts + (row * kParts + p) * K + k) = w;
    }
}

// -------------------------------------------------------------------- product
// What a lane holds of a block of a weight's row: its codes 32 q .. 32 q + 31 and 128 + 32 q
// .. (a load takes 64 neighbouring bytes of each of 16 rows), their micro-scales and the
// block scales of the four rows whose sums it gets.
struct Piece {
    u32x4 codes[2];
    unsigned micro[2];
    float scale[4];
};

// Eight codes times their micro-scale and 2^-11 in bf16: at most 1.32, so that a block's sum
// with |x| < 2^118 stays finite; the block scale takes the 2^11 back (a finite weight's block
// scale is below 2^117).
constexpr float kDown = 0x1p-11f, kUp = 0x1p11f;
__device__ __forceinline__ bf16x8 weights_of(unsigned codes, float micro) {
    u32x4 w;
    auto pair = [&](auto v) {
        // exact: the low halves are zero
        return __builtin_amdgcn_perm(__float_as_uint(v[1] * micro), __float_as_uint(v[0] * micro), 0x07060302u);
    };
    w[0] = pair(fp4q_num::e2m1_values<0>(codes, kDown));
    w[1] = pair(fp4q_num::e2m1_values<1>(codes, kDown));
    w[2] = pair(fp4q_num::e2m1_values<2>(codes, kDown));
    w[3] = pair(fp4q_num::e2m1_values<3>(codes, kDown));
    return __builtin_bit_cast(bf16x8, w);
}

// A workgroup takes 16 rows of the weight (gated: 8 of each) and up to 16 kCols rows of x
// or of its parts; its wavefronts share K, a block each in turn.
template <int kWaves, int kCols, bool kGated>
__global__ __launch_bounds__(kWaves *kWave) void gemv4_kernel(Gemv4Args p) {
    __shared__ f32x4 part[kWaves][kCols][kWave];
    __shared__ float sums[16 * kCols][kStrip + 1];
    constexpr int kOut = kGated ? kStrip / 2 : kStrip;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int row16 = lane & 15, quarter = lane >> 4;
    const int n0 = (int)blockIdx.x * kOut, blocks = p.K / kBlock;
    const int each = 16 * kCols / p.parts, m0 = (int)blockIdx.y * each;  // rows of x here
    const int cols = min(each, p.M - m0) * p.parts;
    // the weight and row behind row r of 16; rows past the end repeat the last one
    auto row_of = [&](int r) { return (int64_t)min(n0 + r % kOut, p.N - 1); };
    auto weight_of = [&](int r) -> const Payload & { return kGated && r >= kOut ? p.up : p.w; };
    const uint8_t *codes = weight_of(row16).codes + row_of(row16) * (p.K / 2) + 16 * quarter;
    const uint8_t *micro = weight_of(row16).micro + row_of(row16) * (p.K / 16) + 2 * quarter;
    const float *block = weight_of(4 * quarter).block;
    const uint16_t *x = p.x + (int64_t)m0 * p.parts * p.K + 32 * quarter;

    f32x4 acc[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[c] = f32x4{0, 0, 0, 0};
    auto load = [&](Piece &w, int kb) {
        w.codes[0] = *reinterpret_cast<const u32x4 *>(codes + kb * (kBlock / 2));
        w.codes[1] = *reinterpret_cast<const u32x4 *>(codes + kb * (kBlock / 2) + 64);
        w.micro[0] = *reinterpret_cast<const uint16_t *>(micro + kb * 16);
        w.micro[1] = *reinterpret_cast<const uint16_t *>(micro + kb * 16 + 8);
#pragma unroll
        for (int e = 0; e < 4; ++e) w.scale[e] = kUp * block[row_of(4 * quarter + e) * blocks + kb];
    };
    auto multiply = [&](const Piece &w, int kb) {
        f32x4 d[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) d[c] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = i < 2 ? __builtin_amdgcn_cvt_f32_fp8(w.micro[h], 0) : __builtin_amdgcn_cvt_f32_fp8(w.micro[h], 1);
                const bf16x8 a = weights_of(w.codes[h][i], u);
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    u32x4 b = {0, 0, 0, 0};
                    const int col = 16 * c + row16;
                    if (col < cols)
                        b = *reinterpret_cast<const u32x4 *>(x + (int64_t)col * p.K + kb * kBlock + 128 * h + 8 * i);
                    d[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, b), d[c], 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][e] = fmaf(d[c][e], w.scale[e], acc[c][e]);
    };
    for (int kb = wave; kb < blocks; kb += kWaves) {
        Piece w;
        load(w, kb);
        multiply(w, kb);
    }
#pragma unroll
    for (int c = 0; c < kCols; ++c) part[wave][c][lane] = acc[c];
    __syncthreads();
    for (int t = threadIdx.x; t < kCols * kWave; t += kWaves * kWave) {
        const int c = t / kWave, l = t % kWave;
        f32x4 sum = part[0][c][l];
#pragma unroll 5
        for (int w = 1; w < kWaves; ++w) sum += part[w][c][l];
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[16 * c + (l & 15)][4 * (l >> 4) + e] = sum[e];
    }
    __syncthreads();
    const int rows = min(each, p.M - m0);
    for (int t = threadIdx.x; t < rows * kOut; t += kWaves * kWave) {
        const int m = t / kOut, n = t % kOut;
        if (n0 + n >= p.N) continue;
        float v = 0.0f, u = 0.0f;
        for (int i = p.parts - 1; i >= 0; --i) {  // the smallest part first
            v += sums[m * p.parts + i][n];
            if (kGated) u += sums[m * p.parts + i][n + kOut];
        }
        if constexpr (kGated) v = with_act(p.act, [&](auto act) { return activate<act.value>(v).act * u; });
        const int64_t at = (int64_t)(m0 + m) * p.N + n0 + n;
        if (p.out_f32)
            static_cast<float *>(p.out)[at] = v;
        else
            static_cast<bf16 *>(p.out)[at] = from_float<bf16>(v);
    }
}

// ------------------------------------------------------------------------ host
constexpr int64_t kLimit = kDimLimit / 2;

bool cut(int dtype, uint32_t flags) { return dtype == FP4Q_OUT_F32 || !(flags & FP4Q_FLAG_NO_FWHT); }

int check_sizes(int64_t M, int64_t K, int dtype, uint32_t flags) {
    if (M < 0 || K <= 0 || M >= kLimit || K >= kLimit || K % kBlock) return FP4Q_ERR_SHAPE;
    if (flags & ~(uint32_t)FP4Q_FLAG_NO_FWHT) return FP4Q_ERR_ARG;
    return dtype == FP4Q_OUT_F32 || dtype == FP4Q_OUT_BF16 ? FP4Q_OK : FP4Q_ERR_ARG;
}
size_t workspace_of(int64_t M, int64_t K, int dtype, uint32_t flags) {
    return cut(dtype, flags) ? (size_t)(2 * kParts * M * K) : 0;
}

template <int kWaves, int kCols, bool kGated>
int run_kernel(Gemv4Args &p, void *stream) {
    const int each = 16 * kCols / p.parts;
    void *args[] = {&p};
    const dim3 grid((unsigned)ceil_div(p.N, kGated ? kStrip / 2 : kStrip), (unsigned)ceil_div(p.M, each));
    if (grid.y > 65535u) return FP4Q_ERR_SHAPE;
    return launch((const void *)&gemv4_kernel<kWaves, kCols, kGated>, grid, kWaves * kWave, args, stream);
}
template <bool kGated>
int run_product(Gemv4Args &p, void *stream) {
    const int64_t cols = (int64_t)p.M * p.parts;
    if (p.parts == kParts) return cols <= 15 ? run_kernel<16, 1, kGated>(p, stream) : run_kernel<16, 3, kGated>(p, stream);
    if (cols <= 16) return run_kernel<16, 1, kGated>(p, stream);
    return cols <= 32 ? run_kernel<16, 2, kGated>(p, stream) : run_kernel<16, 4, kGated>(p, stream);
}

int run(const void *x, int dtype, int64_t M, const Payload &w, const Payload *up, int64_t N, int64_t K, int act,
        void *out, int out_dtype, uint32_t flags, void *workspace, size_t workspace_bytes, void *stream) {
    if (N < 0 || N >= kLimit) return FP4Q_ERR_SHAPE;
    const int st = check_sizes(M, K, dtype, flags);
    if (st != FP4Q_OK) return st;
    if ((out_dtype != FP4Q_OUT_F32 && out_dtype != FP4Q_OUT_BF16) || bad_act(act)) return FP4Q_ERR_ARG;
    if (M == 0 || N == 0) return FP4Q_OK;
    const size_t need = workspace_of(M, K, dtype, flags);
    const Payload weights[] = {w, up ? *up : w};
    if (!x || !out || (need && !workspace)) return FP4Q_ERR_NULL;
    for (const Payload &q : weights)
        if (!q.codes || !q.micro || !q.block) return FP4Q_ERR_NULL;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(workspace, 16)) return FP4Q_ERR_ALIGN;
    for (const Payload &q : weights)
        if (!aligned(q.codes, 16) || !aligned(q.micro, 16) || !aligned(q.block, 4)) return FP4Q_ERR_ALIGN;
    if (workspace_bytes < need) return FP4Q_ERR_SHAPE;
    const Range outs[] = {rng(out, M * N * esize(out_dtype)), rng(workspace, (int64_t)need)};
    Range ins[7] = {rng(x, M * K * esize(dtype))};
    for (int i = 0; i < 2; ++i) {
        ins[1 + 3 * i] = rng(weights[i].codes, N * (K / 2));
        ins[2 + 3 * i] = rng(weights[i].micro, N * (K / 16));
        ins[3 + 3 * i] = rng(weights[i].block, 4 * N * (K / kBlock));
    }
    if (clash(outs, 2, ins, 7)) return FP4Q_ERR_ARG;
    Gemv4Args p = {static_cast<const uint16_t *>(x), weights[0], weights[1], out, (int)M, (int)N, (int)K, 1, act,
                   out_dtype == FP4Q_OUT_F32};
    if (need) {
        p.x = static_cast<const uint16_t *>(workspace);
        p.parts = kParts;
        const bool f32 = dtype == FP4Q_OUT_F32, transform = !(flags & FP4Q_FLAG_NO_FWHT);
        const void *fn = f32 ? (transform ? (const void *)&parts_kernel<float, true> : (const void *)&parts_kernel<float, false>)
                             : (const void *)&parts_kernel<bf16, true>;
        void *args[] = {&x, &workspace, &p.K};
        if (M * (K / kBlock) > (int64_t)0x7FFFFFFF) return FP4Q_ERR_SHAPE;
        const int done = launch(fn, dim3((unsigned)(M * (K / kBlock))), kWave, args, stream);
        if (done != FP4Q_OK) return done;
    }
    return up ? run_product<true>(p, stream) : run_product<false>(p, stream);
}

}  // namespace

extern "C" {

int fp4q_gemv4_workspace(int64_t M, int64_t K, int dtype, uint32_t flags, size_t *bytes) {
    const int st = check_sizes(M, K, dtype, flags);
    if (st != FP4Q_OK) return st;
    if (!bytes) return FP4Q_ERR_NULL;
    *bytes = workspace_of(M, K, dtype, flags);
    return FP4Q_OK;
}

int fp4q_gemv4(const void *x, int dtype, int64_t M, const uint8_t *codes, const uint8_t *micro_scales,
               const float *block_scales, int64_t N, int64_t K, void *out, int out_dtype, uint32_t flags,
               void *workspace, size_t workspace_bytes, void *stream) {
    const Payload w = {codes, micro_scales, block_scales};
    return run(x, dtype, M, w, nullptr, N, K, FP4Q_ACT_SILU, out, out_dtype, flags, workspace, workspace_bytes, stream);
}

int fp4q_gated4(const void *x, int dtype, int64_t M, const uint8_t *gate_codes, const uint8_t *gate_micro,
                const float *gate_block, const uint8_t *up_codes, const uint8_t *up_micro, const float *up_block,
                int64_t N, int64_t K, int act, void *out, int out_dtype, uint32_t flags, void *workspace,
                size_t workspace_bytes, void *stream) {
    const Payload gate = {gate_codes, gate_micro, gate_block}, up = {up_codes, up_micro, up_block};
    return run(x, dtype, M, gate, &up, N, K, act, out, out_dtype, flags, workspace, workspace_bytes, stream);
}

}  // extern "C"
