// fp4q_gated_grad.hip -- the gradients of the gated product as 8-bit codes (declared in
// include/fp4q_gated.h):
//
//   dgate = dy up act'(gate),  dup = dy act(gate),  and y = act(gate) up again
//
// One pass over the three tensors: a workgroup of 512 threads holds a 128 x 128 tile of each
// result, 4 x 8 elements a thread, and writes dgate and dup along rows and along columns and y
// along columns.  A scale needs its 128 elements before their first code, and the tile is what
// gives both orders theirs with the tensors read once.  Bound by HBM: 6 bytes read and 5 written
// per bf16 element.  8192 x 11008 bf16, all three orders: silu 214 us, 4.6 TB/s of these bytes
// (a large copy reaches 5.2), over cards gelu_tanh 221 to 231, gelu 225 to 236; 2047 x 2752
// gelu_tanh 23 us.
//
// 512 threads, not 256 of 8 x 8: 96 results a thread leave room for four wavefronts a SIMD, that
// is for one workgroup to load while the other computes.  (Not so fp32 relu: 129 or 130 registers,
// one workgroup a CU; 2048 x 4096 28.8 us, silu 27.5.)
#include "fp4q_act.h"
#include "fp4q_f8.h"

namespace {

using namespace fp4q_f8;
using namespace fp4q_act;

constexpr int kRows = 4, kThreads = kGroup / kRows * 16;  // rows of a thread; 8 columns
constexpr int kWaves = kThreads / kWave;
// Rows of the inputs under way at once: with all four the registers do not last, and fewer than
// two leave the loads' latency open (2 against 4: 2048 x 4096 fp32 28.9 us and 30.5, 8192 x 11003
// bf16 274 and 288; 3: 8192 x 11008 251 us against 241).
constexpr int kAhead = 2;
// Quads of y that a thread keeps in LDS, not registers, until the scales are there: 4 wavefronts a
// SIMD leave a thread 128 registers, and what does not fit would go through memory (8192 x 11008:
// 212 us against 241 with none aside, and 575 MB written where the codes are 460).
constexpr int kAside = 3;
enum { kGate, kUp, kY, kTensors };

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

// The largest magnitude of three, NaN if one is: one instruction.
__device__ __forceinline__ float largest(float a, float b, float c) {
    return __builtin_elementwise_maximum(__builtin_elementwise_maximum(fabsf(a), fabsf(b)), fabsf(c));
}

// Codes of eight neighbours of a tile's row, `left` of which exist, to offset `at` of the tile's
// codes, and the row's scale to its place among the tile's.
template <int kFmt>
__device__ __forceinline__ void write_row(const float (&v)[8], uint8_t *codes, float *scales, bool exists, unsigned at,
                                          int row, int left, int across) {
    const float top = largest(largest(largest(v[0], v[1], v[2]), v[3], v[4]), v[5], largest(v[6], v[7], v[7]));
    const Scale sc = scale_of<kFmt>(max16(mag(top)));
    u32x2 w;
    w[0] = code_quad<kFmt>(v[0], v[1], v[2], v[3], sc);
    w[1] = code_quad<kFmt>(v[4], v[5], v[6], v[7], sc);
    if (!exists) return;
    if (across == 0) scales[row] = sc.s;
    store_bytes8(codes + at, left, w);
}

// Thread t holds rows kRows (t / 16) + i and columns 8 (t % 16) + j of the tile.
template <typename T, int kAct, int kFmt, bool kWhole>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) void gated_grad_kernel(GradArgs a) {
    __shared__ union {
        unsigned top[kWaves][kTensors][kGroup];           // the wavefronts' largest magnitudes of each column
        unsigned turn[kTensors][kGroup * kGroup / 4];     // then the columns' codes
    } room;
    __shared__ Scale scales[kTensors][kGroup];
    __shared__ float4 aside[kAside][kThreads];
    const int t = threadIdx.x, lane = t & (kWave - 1), wave = t / kWave, across = t & 15, down = t >> 4;
    const int tc = (int)(blockIdx.x % (unsigned)a.col_tiles), tr = (int)(blockIdx.x / (unsigned)a.col_tiles);
    const int row = tr * kGroup, col = tc * kGroup, r0 = row + kRows * down, c0 = col + 8 * across;
    // places in memory: of the tile, the same for all lanes, in 64 bits; within it in 32
    const int64_t tile = (int64_t)row * a.cols + col;
    auto of_tile = [&](const void *base, unsigned bytes) {
        return reinterpret_cast<const T *>(reinterpret_cast<const char *>(static_cast<const T *>(base) + tile) + bytes);
    };
    // the joined tensor: columns N .. P of its first half are zeros, as those of the tile are
    const int second = a.col_tiles * kGroup;
    const int64_t joined = (int64_t)second + a.cols;

    float v[kTensors][kRows][8];
    Eight<T> dy[kAhead], gate[kAhead], up[kAhead];
    auto load = [&](int i) {
        const int left = r0 + i < a.rows ? a.cols - c0 : 0, to = i % kAhead;
        const unsigned at = ((unsigned)(kRows * down + i) * (unsigned)a.cols + 8 * across) * (unsigned)sizeof(T);
        dy[to].template load<kWhole>(of_tile(a.dy, at), left);
        gate[to].template load<kWhole>(of_tile(a.gate, at), left);
        up[to].template load<kWhole>(of_tile(a.up, at), left);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i);
    const int64_t along = row * a.along.pitch + col;
    float *const gate_scales = a.along.scales + (int64_t)tc * a.rows + row;
    float *const up_scales = gate_scales + (int64_t)a.col_tiles * a.rows;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        float d[8], g[8], u[8];
        dy[i % kAhead].get(d);
        gate[i % kAhead].get(g);
        up[i % kAhead].get(u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const Value f = activate<kAct>(g[j]);
            v[kGate][i][j] = d[j] * u[j] * f.slope;
            v[kUp][i][j] = d[j] * f.act;
            v[kY][i][j] = f.act * u[j];
        }
        if (i + kAhead < kRows) load(i + kAhead);
#pragma unroll
        for (int k = 2 * i; k < 2 * i + 2; ++k) {
            const float *q = v[kY][i] + 4 * (k % 2);
            if (k < kAside) aside[k][t] = make_float4(q[0], q[1], q[2], q[3]);
        }
        if (a.along.codes) {
            const int r = kRows * down + i;
            const unsigned at = (unsigned)r * (unsigned)a.along.pitch + 8 * across;
            write_row<kFmt>(v[kGate][i], a.along.codes + along, gate_scales, r0 + i < a.rows, at, r, 8, across);
            write_row<kFmt>(v[kUp][i], a.along.codes + along + second, up_scales, r0 + i < a.rows, at, r, a.cols - c0, across);
        }
    }
    if (!a.across.codes && !a.y.codes) return;
#pragma unroll
    for (int k = 0; k < kAside; ++k) {  // a thread's own: no barrier
        const float4 q = aside[k][t];
        float *const to = v[kY][k / 2] + 4 * (k % 2);
        to[0] = q.x, to[1] = q.y, to[2] = q.z, to[3] = q.w;
    }

    // The columns' largest magnitudes: over a thread's rows, then over the four rows of 16
    // lanes: an exchange of two registers between rows leaves one's maximum over two rows in
    // one row and the other's in the other, so that 24 values end as 6 with no lane idle.
    unsigned top[kTensors * 8];
#pragma unroll
    for (int k = 0; k < kTensors * 8; ++k) {
        const auto &w = v[k / 8];
        static_assert(kRows == 4, "four rows");
        top[k] = mag(largest(largest(w[0][k % 8], w[1][k % 8], w[2][k % 8]), w[3][k % 8], w[3][k % 8]));
    }
#pragma unroll
    for (int k = 0; k < kTensors * 8; k += 4) {
        const auto p = __builtin_amdgcn_permlane16_swap(top[k], top[k + 1], false, false);
        const auto q = __builtin_amdgcn_permlane16_swap(top[k + 2], top[k + 3], false, false);
        const auto r = __builtin_amdgcn_permlane32_swap(umax(p[0], p[1]), umax(q[0], q[1]), false, false);
        room.top[wave][k / 8][8 * across + k % 8 + (lane >> 4)] = umax(r[0], r[1]);
    }
    __syncthreads();
    const int cols = min(kGroup, a.cols - col);  // that exist here; of dgate all, zeros too
    if (t < kTensors * kGroup) {
        const int which = t / kGroup, c = t % kGroup;
        unsigned most = room.top[0][which][c];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) most = umax(most, room.top[w][which][c]);
        const Scale sc = which == kY ? scale_of<FP4Q_E4M3>(most) : scale_of<kFmt>(most);
        scales[which][c] = sc;
        if (which == kY) {
            if (a.y.codes && c < cols) a.y.scales[(int64_t)tr * a.cols + col + c] = sc.s;
        } else if (a.across.codes && (which == kGate || c < cols)) {
            a.across.scales[tr * joined + (which == kGate ? 0 : second) + col + c] = sc.s;
        }
    }
    __syncthreads();
    // column c: 32 slots of 4 bytes (rows 4 s .. 4 s + 3) at slot s ^ 2 (c / 8), so that the 64
    // lanes of a store meet every second bank twice at most
#pragma unroll
    for (int k = 0; k < kTensors; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const Scale sc = scales[k][8 * across + j];
            room.turn[k][(8 * across + j) * 32 + (down ^ 2 * across)] =
                k == kY ? code_quad<FP4Q_E4M3>(v[k][0][j], v[k][1][j], v[k][2][j], v[k][3][j], sc)
                        : code_quad<kFmt>(v[k][0][j], v[k][1][j], v[k][2][j], v[k][3][j], sc);
        }
    __syncthreads();
    // 8 threads write the 128 bytes of a column
    const int pair = t & 7, at = row + 16 * pair;
#pragma unroll
    for (int k = 0; k < kTensors; ++k) {
        const Codes &out = k == kY ? a.y : a.across;
        if (!out.codes) continue;
        uint8_t *const codes = out.codes + ((k == kUp ? second : 0) + col) * out.pitch + row;
#pragma unroll
        for (int n = 0; n < kGroup / (kThreads / 8); ++n) {
            const int c = n * (kThreads / 8) + t / 8, key = c / 8;
            const u32x4 q = reinterpret_cast<const u32x4 *>(room.turn[k])[c * 8 + (pair ^ (key >> 1))];
            const u32x4 w = key & 1 ? u32x4{q[2], q[3], q[0], q[1]} : q;
            if ((k == kGate || c < cols) && at < a.rows) {
                uint8_t *p = codes + ((unsigned)c * (unsigned)out.pitch + 16 * pair);
                if (a.rows - at >= 16) {
                    __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(p));
                } else {
                    store_bytes8(p, a.rows - at, u32x2{w[0], w[1]});
                    if (a.rows - at > 8) store_bytes8(p + 8, a.rows - at - 8, u32x2{w[2], w[3]});
                }
            }
        }
    }
}

template <typename T, int kAct>
const void *pick(int fmt, bool whole) {
    if (fmt == FP4Q_E4M3)
        return whole ? (const void *)&gated_grad_kernel<T, kAct, FP4Q_E4M3, true>
                     : (const void *)&gated_grad_kernel<T, kAct, FP4Q_E4M3, false>;
    return whole ? (const void *)&gated_grad_kernel<T, kAct, FP4Q_E5M2, true>
                 : (const void *)&gated_grad_kernel<T, kAct, FP4Q_E5M2, false>;
}

// So that a tile's places in any of the arrays are offsets of 32 bits.
constexpr int64_t kLimit = (int64_t)1 << 23;
static_assert((kGroup - 1) * kLimit * 4 + kGroup * 4 < ((int64_t)1 << 32), "of 128 rows of floats");
static_assert((kGroup - 1) * 4 * kLimit + kGroup < ((int64_t)1 << 32), "of 128 pitches");

}  // namespace

extern "C" int fp4q_gated8_backward(const void *dy, const void *gate, const void *up, int64_t rows, int64_t cols,
                                    int dtype, int act, int format, uint8_t *codes, int64_t code_pitch,
                                    float *scales, uint8_t *codes_t, int64_t code_t_pitch, float *scales_t,
                                    uint8_t *y_codes_t, int64_t y_t_pitch, float *y_scales_t, void *stream) {
    if (bad_dims(rows, cols) || rows >= kLimit || cols >= kLimit) return FP4Q_ERR_SHAPE;
    const int64_t row_tiles = ceil_div(rows, kGroup), col_tiles = ceil_div(cols, kGroup);
    const int64_t joined = col_tiles * kGroup + cols;
    if (row_tiles * col_tiles > (int64_t)0x7FFFFFFF) return FP4Q_ERR_SHAPE;
    if (codes && (code_pitch < joined || code_pitch >= 4 * kLimit)) return FP4Q_ERR_SHAPE;
    if (codes_t && (code_t_pitch < rows || code_t_pitch >= 4 * kLimit)) return FP4Q_ERR_SHAPE;
    if (y_codes_t && (y_t_pitch < rows || y_t_pitch >= 4 * kLimit)) return FP4Q_ERR_SHAPE;
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
