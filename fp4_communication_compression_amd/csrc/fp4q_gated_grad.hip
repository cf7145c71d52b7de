// fp4q_gated_grad.hip -- the gradients of the gated product as 8-bit codes (declared in
// include/fp4q_gated.h):
//
//   dgate = dy up act'(gate),  dup = dy act(gate),  and y = act(gate) up again
//
// One pass over the three tensors: a workgroup holds a 128 x 128 tile of each result in
// registers, 8 x 8 elements a thread, and writes dgate and dup along rows and along columns
// and y along columns.  Bound by HBM: 6 bytes read and 5 written per bf16 element.
#include "fp4q_act.h"
#include "fp4q_f8.h"

namespace {

using namespace fp4q_f8;
using namespace fp4q_act;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// One order of codes: rows are the rows of the joined tensor, or its columns.
struct Codes {
    uint8_t *codes;
    float *scales;
    int64_t pitch;
};
struct GradArgs {
    const void *dy, *gate, *up;
    Codes along, across, y;
    int rows, cols, row_tiles, col_tiles;
};

struct Room {
    unsigned top[kWaves][kGroup];
    u32x4 turn[kGroup * kGroup / 16];
};

// Codes along the rows of a tile: row r0 + i of `rows`, group `group` of `out`, columns
// c0 .. c0 + 7 of the tensor of which `left` exist.
template <int kFmt>
__device__ __forceinline__ void write_rows(const float (&v)[8][8], const Codes &out, int rows, int r0, int c0, int left,
                                           int group, int across) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        unsigned top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = umax(top, mag(v[i][j]));
        const Scale sc = scale_of<kFmt>(max16(top));
        u32x2 w;
        w[0] = code_quad<kFmt>(v[i][0], v[i][1], v[i][2], v[i][3], sc);
        w[1] = code_quad<kFmt>(v[i][4], v[i][5], v[i][6], v[i][7], sc);
        if (r0 + i >= rows) continue;
        if (across == 0) out.scales[(int64_t)group * rows + r0 + i] = sc.s;
        store_bytes8(out.codes + (int64_t)(r0 + i) * out.pitch + c0, left, w);
    }
}

// Codes along the columns of a tile, turned in LDS: column c of `room` is column first + c of
// the tensor, of `cols` that exist here, its rows those from row on of `rows`, group `group`.
template <int kFmt>
__device__ __forceinline__ void write_cols(const float (&v)[8][8], Room &room, const Codes &out, int64_t all, int first,
                                           int cols, int row, int rows, int group) {
    const int t = threadIdx.x, lane = t & (kWave - 1), wave = t / kWave;
    const int across = t & 15, down = t >> 4;
    Scale sc[8];
    unsigned top[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        top[j] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top[j] = umax(top[j], mag(v[i][j]));
        top[j] = umax(top[j], (unsigned)__shfl_xor((int)top[j], 16));
        top[j] = umax(top[j], (unsigned)__shfl_xor((int)top[j], 32));
        if (lane < 16) room.top[wave][8 * across + j] = top[j];
    }
    __syncthreads();  // (also: the last tile's reads of `turn` are done)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int k = 0; k < kWaves; ++k) top[j] = umax(top[j], room.top[k][8 * across + j]);
        sc[j] = scale_of<kFmt>(top[j]);
        if (down == 0 && 8 * across + j < cols) out.scales[(int64_t)group * all + first + 8 * across + j] = sc[j].s;
    }
    // column c: 16 slots of 8 bytes (rows 8 s .. 8 s + 7) at slot s ^ (c / 8), so that the 16
    // lanes of a store meet 16 different slots
    u32x2 *slots = reinterpret_cast<u32x2 *>(room.turn);
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
        const int c = n * 32 + t / 8, key = c / 8, at = row + 16 * pair;
        const u32x4 q = room.turn[c * 8 + (pair ^ (key >> 1))];
        const u32x4 w = key & 1 ? u32x4{q[2], q[3], q[0], q[1]} : q;
        if (c < cols && at < rows) {
            uint8_t *p = out.codes + (int64_t)(first + c) * out.pitch + at;
            if (rows - at >= 16) {
                __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(p));
            } else {
                store_bytes8(p, rows - at, u32x2{w[0], w[1]});
                if (rows - at > 8) store_bytes8(p + 8, rows - at - 8, u32x2{w[2], w[3]});
            }
        }
    }
}

// Thread t holds rows 8 (t / 16) + i and columns 8 (t % 16) + j of the tile.
template <typename T, int kAct, int kFmt, bool kWhole>
__global__ __launch_bounds__(kThreads) void gated_grad_kernel(GradArgs a) {
    __shared__ Room room;
    const int t = threadIdx.x, across = t & 15, down = t >> 4;
    const int tc = (int)(blockIdx.x % (unsigned)a.col_tiles), tr = (int)(blockIdx.x / (unsigned)a.col_tiles);
    const int row = tr * kGroup, col = tc * kGroup, r0 = row + 8 * down, c0 = col + 8 * across;
    const int64_t from = (int64_t)r0 * a.cols + c0;

    float dgate[8][8], dup[8][8], y[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int left = r0 + i < a.rows ? a.cols - c0 : 0;
        const int64_t at = from + (int64_t)i * a.cols;
        Eight<T> dy, gate, up;
        dy.template load<kWhole>(static_cast<const T *>(a.dy) + at, left);
        gate.template load<kWhole>(static_cast<const T *>(a.gate) + at, left);
        up.template load<kWhole>(static_cast<const T *>(a.up) + at, left);
        float d[8], g[8], u[8];
        dy.get(d);
        gate.get(g);
        up.get(u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const Value v = activate<kAct>(g[j]);
            dgate[i][j] = d[j] * u[j] * v.slope;
            dup[i][j] = d[j] * v.act;
            y[i][j] = v.act * u[j];
        }
    }
    // the joined tensor: columns N .. P of its first half are zeros, as those of the tile are
    const int second = a.col_tiles * kGroup, cols = min(kGroup, a.cols - col);
    const int64_t joined = (int64_t)second + a.cols;
    if (a.along.codes) {
        write_rows<kFmt>(dgate, a.along, a.rows, r0, c0, 8, tc, across);
        write_rows<kFmt>(dup, a.along, a.rows, r0, second + c0, a.cols - c0, a.col_tiles + tc, across);
    }
    if (a.across.codes) {
        write_cols<kFmt>(dgate, room, a.across, joined, col, kGroup, row, a.rows, tr);
        write_cols<kFmt>(dup, room, a.across, joined, second + col, cols, row, a.rows, tr);
    }
    if (a.y.codes) write_cols<FP4Q_E4M3>(y, room, a.y, a.cols, col, cols, row, a.rows, tr);
}

template <typename T, int kAct>
const void *pick(int fmt, bool whole) {
    if (fmt == FP4Q_E4M3)
        return whole ? (const void *)&gated_grad_kernel<T, kAct, FP4Q_E4M3, true>
                     : (const void *)&gated_grad_kernel<T, kAct, FP4Q_E4M3, false>;
    return whole ? (const void *)&gated_grad_kernel<T, kAct, FP4Q_E5M2, true>
                 : (const void *)&gated_grad_kernel<T, kAct, FP4Q_E5M2, false>;
}

}  // namespace

extern "C" int fp4q_gated8_backward(const void *dy, const void *gate, const void *up, int64_t rows, int64_t cols,
                                    int dtype, int act, int format, uint8_t *codes, int64_t code_pitch,
                                    float *scales, uint8_t *codes_t, int64_t code_t_pitch, float *scales_t,
                                    uint8_t *y_codes_t, int64_t y_t_pitch, float *y_scales_t, void *stream) {
    if (bad_dims(rows, cols) || rows >= kDimLimit / 2 || cols >= kDimLimit / 2) return FP4Q_ERR_SHAPE;
    const int64_t row_tiles = ceil_div(rows, kGroup), col_tiles = ceil_div(cols, kGroup);
    const int64_t joined = col_tiles * kGroup + cols;
    if (row_tiles * col_tiles > (int64_t)0x7FFFFFFF) return FP4Q_ERR_SHAPE;
    if (codes && (code_pitch < joined || code_pitch >= 2 * kDimLimit)) return FP4Q_ERR_SHAPE;
    if (codes_t && (code_t_pitch < rows || code_t_pitch >= 2 * kDimLimit)) return FP4Q_ERR_SHAPE;
    if (y_codes_t && (y_t_pitch < rows || y_t_pitch >= 2 * kDimLimit)) return FP4Q_ERR_SHAPE;
    if ((dtype != FP4Q_OUT_F32 && dtype != FP4Q_OUT_BF16) || bad_act(act) ||
        (format != FP4Q_E4M3 && format != FP4Q_E5M2))
        return FP4Q_ERR_ARG;
    if (rows == 0) return FP4Q_OK;
    if (!dy || !gate || !up || (!codes && !codes_t && !y_codes_t) || (codes && !scales) || (codes_t && !scales_t) ||
        (y_codes_t && !y_scales_t))
        return FP4Q_ERR_NULL;
    if ((!codes && scales) || (!codes_t && scales_t) || (!y_codes_t && y_scales_t)) return FP4Q_ERR_ARG;
    if (!aligned(dy, 16) || !aligned(gate, 16) || !aligned(up, 16)) return FP4Q_ERR_ALIGN;
    if (!aligned(codes, 16) || !aligned(codes_t, 16) || !aligned(y_codes_t, 16)) return FP4Q_ERR_ALIGN;
    if ((codes && code_pitch % 16) || (codes_t && code_t_pitch % 16) || (y_codes_t && y_t_pitch % 16)) return FP4Q_ERR_ALIGN;
    if (!aligned(scales, 4) || !aligned(scales_t, 4) || !aligned(y_scales_t, 4)) return FP4Q_ERR_ALIGN;
    const Range outs[] = {rng(codes, pitched(rows, joined, code_pitch)),     rng(scales, 4 * 2 * col_tiles * rows),
                          rng(codes_t, pitched(joined, rows, code_t_pitch)), rng(scales_t, 4 * row_tiles * joined),
                          rng(y_codes_t, pitched(cols, rows, y_t_pitch)),    rng(y_scales_t, 4 * row_tiles * cols)};
    const int64_t bytes = rows * cols * esize(dtype);
    const Range ins[] = {rng(dy, bytes), rng(gate, bytes), rng(up, bytes)};
    if (clash(outs, 6, ins, 3)) return FP4Q_ERR_ARG;
    GradArgs a = {dy, gate, up, {codes, scales, code_pitch}, {codes_t, scales_t, code_t_pitch},
                  {y_codes_t, y_scales_t, y_t_pitch}, (int)rows, (int)cols, (int)row_tiles, (int)col_tiles};
    void *args[] = {&a};
    const bool whole = cols % 8 == 0;
    const void *fn = with_act(act, [&](auto kind) {
        return dtype == FP4Q_OUT_F32 ? pick<float, kind.value>(format, whole) : pick<bf16, kind.value>(format, whole);
    });
    return launch(fn, dim3((unsigned)(row_tiles * col_tiles)), kThreads, args, stream);
}
