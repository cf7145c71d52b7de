// fp4q_quant8.hip -- 8-bit codes with a scale per 128 values (declared in
// include/fp4q_linear.h): along rows, along columns (written transposed), or
// per 128 x 128 tile in both orders.
//
// One pass over the tensor: a workgroup holds a 128 x 128 tile in registers,
// 8 x 8 elements a thread, finds the maxima it needs and writes both orders of
// codes.  Bound by HBM: 2 bytes read and 1 or 2 written per bf16 element.
// 8192 x 4096 bf16: both orders 25.0 us (5.4 TB/s), rows alone 17.3 us (5.9 TB/s);
// fp32: 41.7 us (4.8 TB/s) and 31.1 us (5.4 TB/s), tiles in both orders 38.7 us (5.2 TB/s).
// 11008 x 4096 bf16, tiles in both orders: 32.3 us (5.6 TB/s).
#include "fp4q_f8.h"

namespace {

using namespace fp4q_f8;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

struct QuantArgs {
    const void *x;
    uint8_t *codes, *codes_t;
    float *scales, *scales_t;
    int64_t pitch, pitch_t;
    int rows, cols, row_tiles, col_tiles;
};

// Thread t holds rows 8 (t / 16) + i and columns 8 (t % 16) + j of the tile: a
// row's 128 columns are one DPP row of 16 lanes.
template <typename T, int kFmt, bool kTiles, bool kWhole>
__global__ __launch_bounds__(kThreads) void quant_kernel(QuantArgs a) {
    __shared__ unsigned top_lds[kWaves][kGroup];
    __shared__ u32x4 turn[kGroup * kGroup / 16];
    const int t = threadIdx.x, lane = t & (kWave - 1), wave = t / kWave;
    const int across = t & 15, down = t >> 4;
    const int tc = (int)(blockIdx.x % (unsigned)a.col_tiles), tr = (int)(blockIdx.x / (unsigned)a.col_tiles);
    const int r0 = tr * kGroup + 8 * down, c0 = tc * kGroup + 8 * across;
    const T *x = static_cast<const T *>(a.x) + (int64_t)r0 * a.cols + c0;

    Eight<T> in[8];
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        in[i].template load<kWhole>(x + (int64_t)i * a.cols, r0 + i < a.rows ? a.cols - c0 : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) in[i].get(v[i]);

    Scale tile;
    if (kTiles) {
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) top = umax(top, mag(v[i][j]));
        top = max64(top);
        if (lane == 0) top_lds[wave][0] = top;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kWaves; ++k) top = umax(top, top_lds[k][0]);
        tile = scale_of<kFmt>(top);
        if (t == 0) {
            if (a.codes) a.scales[(int64_t)tc * a.row_tiles + tr] = tile.s;
            if (a.codes_t) a.scales_t[(int64_t)tr * a.col_tiles + tc] = tile.s;
        }
    }

    if (a.codes) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            Scale sc = tile;
            if (!kTiles) {
                unsigned top = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = umax(top, mag(v[i][j]));
                sc = scale_of<kFmt>(max16(top));
                if (across == 0 && r0 + i < a.rows) a.scales[(int64_t)tc * a.rows + r0 + i] = sc.s;
            }
            u32x2 w;
            w[0] = code_quad<kFmt>(v[i][0], v[i][1], v[i][2], v[i][3], sc);
            w[1] = code_quad<kFmt>(v[i][4], v[i][5], v[i][6], v[i][7], sc);
            if (r0 + i < a.rows) store_bytes8(a.codes + (int64_t)(r0 + i) * a.pitch + c0, a.cols - c0, w);
        }
    }

    if (a.codes_t) {
        Scale sc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) sc[j] = tile;
        if (!kTiles) {
            unsigned top[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                top[j] = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) top[j] = umax(top[j], mag(v[i][j]));
                top[j] = umax(top[j], (unsigned)__shfl_xor((int)top[j], 16));
                top[j] = umax(top[j], (unsigned)__shfl_xor((int)top[j], 32));
                if (lane < 16) top_lds[wave][8 * across + j] = top[j];
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int k = 0; k < kWaves; ++k) top[j] = umax(top[j], top_lds[k][8 * across + j]);
                sc[j] = scale_of<kFmt>(top[j]);
                if (down == 0 && c0 + j < a.cols) a.scales_t[(int64_t)tr * a.cols + c0 + j] = sc[j].s;
            }
        }
        // column c of the tile: 16 slots of 8 bytes (rows 8 s .. 8 s + 7) at slot
        // s ^ (c / 8), so that the 16 lanes of a store meet 16 different slots
        u32x2 *slots = reinterpret_cast<u32x2 *>(turn);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u32x2 w;
            w[0] = code_quad<kFmt>(v[0][j], v[1][j], v[2][j], v[3][j], sc[j]);
            w[1] = code_quad<kFmt>(v[4][j], v[5][j], v[6][j], v[7][j], sc[j]);
            slots[(8 * across + j) * 16 + (down ^ across)] = w;
        }
        __syncthreads();
        // 8 threads write the 128 bytes of a column
        const int pair = t & 7;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int c = n * 32 + t / 8, key = c / 8;
            const u32x4 q = turn[c * 8 + (pair ^ (key >> 1))];
            const u32x4 w = key & 1 ? u32x4{q[2], q[3], q[0], q[1]} : q;
            const int col = tc * kGroup + c, row = tr * kGroup + 16 * pair;
            if (col < a.cols && row < a.rows) {
                uint8_t *p = a.codes_t + (int64_t)col * a.pitch_t + row;
                if (a.rows - row >= 16) {
                    __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(p));
                } else {
                    store_bytes8(p, a.rows - row, u32x2{w[0], w[1]});
                    if (a.rows - row > 8) store_bytes8(p + 8, a.rows - row - 8, u32x2{w[2], w[3]});
                }
            }
        }
    }
}

template <typename T, int kFmt, bool kTiles>
const void *pick(bool whole) {
    return whole ? (const void *)&quant_kernel<T, kFmt, kTiles, true>
               : (const void *)&quant_kernel<T, kFmt, kTiles, false>;
}
template <typename T>
const void *pick(int fmt, bool tiles, bool whole) {
    if (fmt == FP4Q_E4M3) return tiles ? pick<T, FP4Q_E4M3, true>(whole) : pick<T, FP4Q_E4M3, false>(whole);
    return tiles ? pick<T, FP4Q_E5M2, true>(whole) : pick<T, FP4Q_E5M2, false>(whole);
}

}  // namespace

extern "C" int fp4q_quantize8(const void *x, int64_t rows, int64_t cols, int dtype, int format,
                              uint8_t *codes, int64_t code_pitch, float *scales, uint8_t *codes_t,
                              int64_t code_t_pitch, float *scales_t, uint32_t flags, void *stream) {
    if (bad_dims(rows, cols)) return FP4Q_ERR_SHAPE;
    const int64_t row_tiles = ceil_div(rows, kGroup), col_tiles = ceil_div(cols, kGroup);
    if (row_tiles * col_tiles > (int64_t)0x7FFFFFFF) return FP4Q_ERR_SHAPE;
    if (codes && (code_pitch < cols || code_pitch >= 2 * kDimLimit)) return FP4Q_ERR_SHAPE;
    if (codes_t && (code_t_pitch < rows || code_t_pitch >= 2 * kDimLimit)) return FP4Q_ERR_SHAPE;
    if (flags & ~(uint32_t)FP4Q_FLAG_TILES) return FP4Q_ERR_ARG;
    if (dtype != FP4Q_OUT_F32 && dtype != FP4Q_OUT_BF16) return FP4Q_ERR_ARG;
    if (format != FP4Q_E4M3 && format != FP4Q_E5M2) return FP4Q_ERR_ARG;
    if (rows == 0) return FP4Q_OK;
    if (!x || (!codes && !codes_t) || (codes && !scales) || (codes_t && !scales_t)) return FP4Q_ERR_NULL;
    if ((!codes && scales) || (!codes_t && scales_t)) return FP4Q_ERR_ARG;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(codes_t, 16)) return FP4Q_ERR_ALIGN;
    if ((codes && code_pitch % 16) || (codes_t && code_t_pitch % 16)) return FP4Q_ERR_ALIGN;
    if (!aligned(scales, 4) || !aligned(scales_t, 4)) return FP4Q_ERR_ALIGN;
    const bool tiles = flags & FP4Q_FLAG_TILES;
    const Range outs[] = {rng(codes, pitched(rows, cols, code_pitch)),
                          rng(scales, 4 * col_tiles * (tiles ? row_tiles : rows)),
                          rng(codes_t, pitched(cols, rows, code_t_pitch)),
                          rng(scales_t, 4 * row_tiles * (tiles ? col_tiles : cols))};
    const Range in = rng(x, rows * cols * esize(dtype));
    if (clash(outs, 4, &in, 1)) return FP4Q_ERR_ARG;
    QuantArgs a = {x, codes, codes_t, scales, scales_t, code_pitch, code_t_pitch,
                   (int)rows, (int)cols, (int)row_tiles, (int)col_tiles};
    void *args[] = {&a};
    const bool whole = cols % 8 == 0;
    const void *fn = dtype == FP4Q_OUT_F32 ? pick<float>(format, tiles, whole) : pick<bf16>(format, tiles, whole);
    return launch(fn, dim3((unsigned)(row_tiles * col_tiles)), kThreads, args, stream);
}
