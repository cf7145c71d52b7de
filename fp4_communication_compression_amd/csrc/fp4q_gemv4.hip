// fp4q_gemv4.hip -- a few rows times a weight held as an FP4 payload, and the gated form of
// two such products (declared in include/fp4q_gated.h):
//
//   out[m][n] = sum over blocks b of 256 of s[n][b] sum over k in b of x[m][k] e[n][k] u[n][k / 16]
//
// with E2M1 codes e, E4M3 micro-scales u and fp32 block scales s.  e u has at most 6
// significant bits and lies between 2^-10 and 2688: it is exact in fp16, at one packed
// conversion and one packed multiplication for two codes.  x becomes fp16 under a power of
// two for each row and block of 256: for bf16 x that is exact but for what lies 2^-28 below
// the block's largest value; fp32 x, and x transformed instead of a transformed weight where
// out is fp32, are cut into two fp16 parts, 22 bits below the largest (transformed x with bf16
// out takes one).  The parts are columns of the matrix core's product like the rows of x, their
// sums are added at the end: it has 16 columns anyway, and the time is that of reading the
// payload.  Products are exact and added in fp32.
//
// Bound by HBM where the payload is large: 16 x 32768 x 4096 20.2 us, 3.8 TB/s; two payloads of
// 11008 x 4096 and one row 12.3 us, 4.2 TB/s; by the launch and the first loads' latency where it
// is small: one row through 4096 x 11008 9.1 us, 2.9 TB/s.  (A large copy reaches 5.2.)
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "fp4q_act.h"
#include "fp4q_f8.h"
#include "fp4q_gemv4_plan.h"

namespace {

using namespace fp4q_f8;
using namespace fp4q_act;
using namespace fp4q_few_plan;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct Payload {
    const uint8_t *codes, *micro;
    const float *block;
};
struct Gemv4Args {
    const void *x;      // [M x K] of the given type; or, made ready, [M parts x K] fp16
    const float *down;  // made ready: what each part's block is to be multiplied by
    Payload w, up;      // up: the gated form's second weight
    void *out;
    int M, N, K, parts, act, out_f32, x_f32, transform;
};

// ------------------------------------------------------------------ x as fp16
// A lane's place of columns k .. k + 7 of a block of 256, in units of 8: the matrix core's
// step (h, j) takes the codes' dword j of a lane's 16 bytes from each half h of the block's
// 128, so quarter q needs columns 128 h + 32 q + 8 j; they lie at 16 h + 4 j + q.
__device__ __forceinline__ int place_of(int k) { return (k & 128) | (k & 24) << 2 | (k & 96) >> 2 | (k & 7); }

// The value of another lane of the same 16 (a DPP control), and a swap of a's odd rows of 16
// lanes with b's even ones (or of a's upper 32 lanes with b's lower ones).
template <int kControl>
__device__ __forceinline__ float moved(float v) {
    return __uint_as_float((unsigned)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), kControl, 0xF, 0xF, true));
}
__device__ __forceinline__ void exchange(int far, float &a, float &b) {
    const unsigned x = __float_as_uint(a), y = __float_as_uint(b);
    if (far == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
        a = __uint_as_float(r[0]);
        b = __uint_as_float(r[1]);
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
        a = __uint_as_float(r[0]);
        b = __uint_as_float(r[1]);
    }
}
__device__ __forceinline__ unsigned most64(unsigned v) {
    v = max16(v);
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = umax(r[0], r[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return umax(q[0], q[1]);
}

// A block of 256 of a row, four neighbours a lane of a wavefront.
struct Rowblock {
    float v[4];
    __device__ __forceinline__ void load(const float *x) {
        const f32x4 w = reinterpret_cast<const f32x4 *>(x)[threadIdx.x & (kWave - 1)];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = w[i];
    }
    __device__ __forceinline__ void load(const bf16 *x) {
        const u32x2 w = reinterpret_cast<const u32x2 *>(x)[threadIdx.x & (kWave - 1)];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    }
    // y = H v / 16 in fp32: strides 1 and 2 in a lane, 4 to 128 over the lanes, by exchanges
    // within rows of 16 lanes and between the rows.
    __device__ __forceinline__ void transform() {
        const int lane = threadIdx.x & (kWave - 1);
        const float a = v[0] + v[1], b = v[0] - v[1], c = v[2] + v[3], d = v[2] - v[3];
        v[0] = a + c;
        v[1] = b + d;
        v[2] = a - c;
        v[3] = b - d;
        auto within = [&](int far, auto partner) {
            const float sign = lane & far ? -1.0f : 1.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fmaf(v[i], sign, partner(v[i]));  // (exact: a sum or a difference)
        };
        within(1, [](float x) { return moved<0xB1>(x); });                 // lanes 1 0 3 2
        within(2, [](float x) { return moved<0x4E>(x); });                 // lanes 2 3 0 1
        within(4, [](float x) { return moved<0x141>(moved<0x1B>(x)); });   // lanes 3 2 1 0 of four, then 7 .. 0 of eight
        within(8, [](float x) { return moved<0x128>(x); });                // a turn by 8 of 16
#pragma unroll
        for (int far = 16; far <= 32; far *= 2)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                exchange(far, v[i], v[i + 1]);  // one register gets both first halves, the other both second ones
                const float sum = v[i] + v[i + 1], difference = v[i] - v[i + 1];
                v[i] = sum;
                v[i + 1] = difference;
                exchange(far, v[i], v[i + 1]);
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= 0.0625f;
    }
    // The parts at to, to + pitch and what brings each back at down, down + down_pitch.  The
    // largest value comes to 2^14 .. 2^15; the second part holds what the first one's rounding
    // left, times 2^11.  A block that is not finite keeps its values, which are not either.
    // (down is 2^-17 of the factor that it stands for: see the product.)
    __device__ __forceinline__ void store(_Float16 *to, int64_t pitch, float *down, int64_t down_pitch, int parts) {
        const int lane = threadIdx.x & (kWave - 1);
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = umax(top, mag(v[i]));
        top = most64(top);
        const bool finite = top < 0x7F800000u;
        const int e = finite ? max((int)(top >> 23) - 127, -84) : 14;
        const float power = __uint_as_float((unsigned)(127 + 14 - e) << 23);
        if (lane < parts) down[lane * down_pitch] = __uint_as_float((unsigned)(127 - 14 - 17 + e - 11 * lane) << 23);
        const int at = place_of(4 * lane);
        for (int p = 0; p < parts; ++p) {
            f16x2 w[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float scaled = p ? v[i] : v[i] * power;
                const _Float16 half = (_Float16)scaled;
                w[i >> 1][i & 1] = half;
                v[i] = finite ? (scaled - (float)half) * 2048.0f : 0.0f;
            }
            *reinterpret_cast<u32x2 *>(to + p * pitch + at) =
                u32x2{__builtin_bit_cast(unsigned, w[0]), __builtin_bit_cast(unsigned, w[1])};
        }
    }
};
__device__ __forceinline__ Rowblock ready(const Gemv4Args &p, int64_t row, int kb) {
    Rowblock r;
    const int64_t from = row * p.K + kb * kBlock;
    if (p.x_f32)
        r.load(static_cast<const float *>(p.x) + from);
    else
        r.load(static_cast<const bf16 *>(p.x) + from);
    return r;
}

// x made ready in memory, for calls whose x does not fit a workgroup's LDS: parts [M parts x
// K] and factors [M parts x K / 256].
constexpr int kReadyWaves = 4;
__global__ __launch_bounds__(kReadyWaves *kWave) void ready_kernel(Gemv4Args p, _Float16 *to, float *down) {
    const int blocks = p.K / kBlock, kb = (int)blockIdx.x * kReadyWaves + threadIdx.x / kWave;
    if (kb >= blocks) return;
    for (int64_t row = blockIdx.y; row < p.M; row += gridDim.y) {
        Rowblock r = ready(p, row, kb);
        if (p.transform) r.transform();
        r.store(to + row * p.parts * p.K + kb * kBlock, p.K, down + row * p.parts * blocks + kb, blocks, p.parts);
    }
}

// -------------------------------------------------------------------- product
// A range of rows of one of a payload's arrays, read through a descriptor: rows past the
// end read as zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const void *base, int first, int rows, int pitch) {
    const uint64_t at = (uint64_t)base + (uint64_t)((int64_t)first * pitch);
    // (all of it is uniform, which the compiler does not see in a loop: it would read the
    // descriptor lane by lane)
    const unsigned low = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)at);
    const unsigned high = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)(at >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void *)((uint64_t)high << 32 | low), 0,
                                             __builtin_amdgcn_readfirstlane(rows * pitch), 0x00020000);
}

// A block of 16 rows of a weight as loaded: whole 128-byte pieces of 8 rows a load (16 rows'
// 64 bytes, as the matrix core wants them, took 8.0 instead of 5.9 us for 22 MB, without any
// work on them), a dword of the micro-scales and a row's block scale ...
struct Fetched {
    u32x4 codes[2];
    unsigned micro, scale;
};
// ... and as a lane needs it: its row's codes 32 q .. 32 q + 31 and 128 + 32 q .., their
// micro-scales, and the block scales of the four rows whose sums it gets.
struct Piece {
    u32x4 codes[2];
    unsigned micro[2];
    f32x4 scale;
};
// Through a part of LDS of the wavefront's own.  Chunk c (16 bytes) of row r lies at chunk
// c ^ (r / 2 & 7), so that no two lanes of a read meet in a bank; the loads fetch it so.
struct Turn {
    u32x4 codes[16 * 8];
    unsigned micro[64];
    float scale[16];
};
static_assert(sizeof(Turn) == kTurnBytes, "what the plan counts");
// (other types' views of them, which the compiler has to keep in order with the stores)
typedef uint16_t AnyHalf __attribute__((may_alias));
typedef f32x4 AnyQuad __attribute__((may_alias));

// Eight codes times their micro-scale.
__device__ __forceinline__ f16x8 weights_of(unsigned codes, _Float16 micro) {
    f16x2 w[4] = {fp4q_num::e2m1_halves<0>(codes), fp4q_num::e2m1_halves<1>(codes), fp4q_num::e2m1_halves<2>(codes),
                  fp4q_num::e2m1_halves<3>(codes)};
    f16x8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] *= f16x2{micro, micro};
        v[2 * i] = w[i][0];
        v[2 * i + 1] = w[i][1];
    }
    return v;
}

template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F &&f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F &&f) {
    static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// Where the matrix core's second operand comes from.
enum class Source {
    kStaged,  // the workgroup makes x ready itself, in LDS
    kOne,     // made ready in memory; a wavefront has one block of K, whose x it holds for all units
    kMemory,  // made ready in memory, loaded with each block
};

// A workgroup takes units of the weight in turn, kStrips strips of 16 rows each (gated: 16 rows
// of the gate and the same of the up projection), for up to 16 kCols rows of x or of its parts.
// Its wavefronts share K, every kWaves-th block each; loads run kBlocksAhead blocks ahead, into
// the next unit too.  There are no branches around them: what does not exist is read through an
// empty descriptor (behind a branch the compiler would wait for all loads under way).
template <int kWaves, int kCols, int kStrips, int kBlocksAhead, bool kGated, Source kSource>
__global__ __launch_bounds__(kWaves *kWave) void gemv4_kernel(Gemv4Args p) {
    static_assert(!kGated || kStrips == 2, "a pair");
    constexpr int kOut = kGated ? kStrip : kStrip * kStrips, kAhead = kBlocksAhead * kStrips;
    constexpr bool kStage = kSource == Source::kStaged, kRing = kSource == Source::kMemory;
    extern __shared__ char room[];  // two units' sums; x and its factors
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int row16 = lane & 15, quarter = lane >> 4;
    const int blocks = p.K / kBlock, units = (p.N + kOut - 1) / kOut, step = (int)gridDim.x;
    const int each = 16 * kCols / p.parts, m0 = (int)blockIdx.y * each;  // rows of x here
    const int rows = min(each, p.M - m0), cols = rows * p.parts;
    float *sums = reinterpret_cast<float *>(room);  // [2][kWaves][kStrips][cols][16]
    const int sums_each = kWaves * kStrips * cols * 16;

    const int code_pitch = p.K / 2, micro_pitch = p.K / 16, block_pitch = 4 * blocks;
    const int row8 = lane >> 3, chunk = (lane & 7) ^ (row8 >> 1);
    const int code_at = row8 * code_pitch + 16 * chunk, code_at8 = (row8 + 8) * code_pitch + 16 * (chunk ^ 4);
    const int micro_at = (lane >> 2) * micro_pitch + 4 * (lane & 3), block_at = row16 * block_pitch;
    const int turns = (blocks + kWaves - 1) / kWaves;  // blocks of a wavefront, the last one perhaps missing
    Fetched fetched[kAhead];
    auto load = [&](Fetched &w, int unit, int turn, int strip) {
        const Payload &from = kGated && strip ? p.up : p.w;
        const int n0 = unit * kOut + (kGated ? 0 : strip * kStrip), kb = wave + turn * kWaves;
        const int here = unit < units && kb < blocks ? max(min(kStrip, p.N - n0), 0) : 0;
        const auto codes = rows_at(from.codes, n0, here, code_pitch), micro = rows_at(from.micro, n0, here, micro_pitch),
                   block = rows_at(from.block, n0, here, block_pitch);
        w.codes[0] = __builtin_amdgcn_raw_buffer_load_b128(codes, code_at, kb * (kBlock / 2), 0);
        w.codes[1] = __builtin_amdgcn_raw_buffer_load_b128(codes, code_at8, kb * (kBlock / 2), 0);
        w.micro = __builtin_amdgcn_raw_buffer_load_b32(micro, micro_at, kb * 16, 0);
        w.scale = __builtin_amdgcn_raw_buffer_load_b32(block, block_at, 4 * kb, 0);
    };
    Turn &room_here = reinterpret_cast<Turn *>(sums + 2 * sums_each)[wave];
    auto turned = [&](const Fetched &w) {
        room_here.codes[lane] = w.codes[0];
        room_here.codes[64 + lane] = w.codes[1];
        room_here.micro[lane] = w.micro;
        room_here.scale[row16] = __uint_as_float(w.scale);
        Piece t;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            t.codes[h] = room_here.codes[row16 * 8 + ((quarter + 4 * h) ^ (row16 >> 1))];
            t.micro[h] = reinterpret_cast<const AnyHalf *>(room_here.micro)[row16 * 8 + 4 * h + quarter];
        }
        t.scale = reinterpret_cast<const AnyQuad *>(room_here.scale)[quarter];
        return t;
    };

    // x: in LDS rows of p.K columns, 16 bytes apart in their banks, then the factors
    _Float16 *const staged = reinterpret_cast<_Float16 *>(reinterpret_cast<Turn *>(sums + 2 * sums_each) + kWaves);
    const int pitch = p.K + 8;
    float *const staged_down = reinterpret_cast<float *>(staged + cols * pitch);
    struct Part {
        u32x4 x[kCols][8];
        float down[kCols];
    };
    Part part[kRing ? kBlocksAhead : 1];
    auto load_x = [&](Part &to, int turn) {
        const int kb = min(wave + turn * kWaves, blocks - 1);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
            const int col = min(16 * c + row16, cols - 1);
            const _Float16 *from;
            if constexpr (kStage) {
                from = staged + col * pitch + kb * kBlock;
                to.down[c] = staged_down[col * blocks + kb];
            } else {
                const int64_t row = (int64_t)m0 * p.parts + col;
                from = static_cast<const _Float16 *>(p.x) + row * p.K + kb * kBlock;
                to.down[c] = p.down[row * blocks + kb];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) to.x[c][i] = reinterpret_cast<const u32x4 *>(from)[4 * i + quarter];
        }
    };
    // where the next loads and the next products are
    int load_unit = (int)blockIdx.x, load_turn = 0, unit = load_unit, turn = 0;
    auto advance = [&](int &of, int &at) {
        const bool last = ++at == turns;
        at = last ? 0 : at;
        of += last ? step : 0;
    };
    auto load_first = [&]() {
        static_for<kAhead>([&](auto i) {
            if constexpr (kRing && i.value % kStrips == 0) load_x(part[i.value / kStrips], load_turn);
            load(fetched[i.value], load_unit, load_turn, i.value % kStrips);
            if constexpr (i.value % kStrips == kStrips - 1) advance(load_unit, load_turn);
        });
    };
    if constexpr (kStage) {
        // the first loads of x before the weight's: a wavefront's loads return in order
        const int all = rows * blocks;
        Rowblock r = ready(p, m0 + min(wave, all - 1) / blocks, min(wave, all - 1) % blocks);
        load_first();
        for (int at = wave; at < all; at += kWaves) {
            const int row = at / blocks, kb = at % blocks;
            if (at != wave) r = ready(p, m0 + row, kb);
            if (p.transform) r.transform();
            r.store(staged + row * p.parts * pitch + kb * kBlock, pitch, staged_down + row * p.parts * blocks + kb, blocks,
                    p.parts);
        }
        __syncthreads();
    } else {
        if constexpr (!kRing) load_x(part[0], 0);
        load_first();
    }

    f32x4 acc[kStrips][kCols];
    auto clear = [&]() {
#pragma unroll
        for (int s = 0; s < kStrips; ++s)
#pragma unroll
            for (int c = 0; c < kCols; ++c) acc[s][c] = f32x4{0, 0, 0, 0};
    };
    clear();
    auto multiply = [&](const Piece &w, const Part &x, f32x4 (&sum)[kCols]) {
        f32x4 d[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) d[c] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f16x2 u = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.micro[h], 1.0f, false);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f16x8 a = weights_of(w.codes[h][j], u[j >> 1]);
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    d[c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, __builtin_bit_cast(f16x8, x.x[c][4 * h + j]), d[c], 0, 0, 0);
            }
        }
        // (d down) 2^17 s: with |x| and the weights below 2^118 both products are finite
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[c][e] = fmaf(d[c][e] * x.down[c], w.scale[e] * 0x1p17f, sum[c][e]);
    };
    // two units' sums in turn: one meeting a unit keeps writers and readers apart
    auto finish = [&]() {
#pragma unroll
        for (int s = 0; s < kStrips; ++s)
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                if (16 * c + row16 < cols)
                    *reinterpret_cast<f32x4 *>(sums + ((wave * kStrips + s) * cols + 16 * c + row16) * 16 + 4 * quarter) = acc[s][c];
        __syncthreads();
        for (int t = threadIdx.x; t < rows * kOut; t += kWaves * kWave) {
            const int m = t / kOut, n = t % kOut, strip = kGated ? 0 : n / kStrip;
            if (unit * kOut + n >= p.N) continue;
            float v = 0.0f, u = 0.0f;
            for (int i = 0; i < p.parts; ++i) {
                const float *from = sums + (strip * cols + m * p.parts + i) * 16 + n % kStrip;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
                    v += from[w * kStrips * cols * 16];
                    if constexpr (kGated) u += from[(w * kStrips + 1) * cols * 16];
                }
            }
            if constexpr (kGated) v = with_act(p.act, [&](auto act) { return activate<act.value>(v).act * u; });
            const int64_t to = (int64_t)(m0 + m) * p.N + unit * kOut + n;
            if (p.out_f32)
                static_cast<float *>(p.out)[to] = v;
            else
                static_cast<bf16 *>(p.out)[to] = from_float<bf16>(v);
        }
        sums = sums == reinterpret_cast<float *>(room) ? sums + sums_each : reinterpret_cast<float *>(room);
        clear();
    };

    // whole rounds of the ring: the last one may end with items that do not exist, all zeros
    const int mine = (units - 1 - (int)blockIdx.x) / step + 1;
    for (int left = mine * turns; left > 0; left -= kBlocksAhead) {
        static_for<kAhead>([&](auto i) {
            constexpr int strip = i.value % kStrips;
            Part &x = part[kRing ? i.value / kStrips : 0];
            if constexpr (kStage && strip == 0) load_x(x, turn);
            multiply(turned(fetched[i.value]), x, acc[strip]);
            if constexpr (kRing && strip == kStrips - 1) load_x(x, load_turn);
            load(fetched[i.value], load_unit, load_turn, strip);
            if constexpr (strip == kStrips - 1) {
                advance(load_unit, load_turn);
                if (turn == turns - 1 && unit < units) finish();
                advance(unit, turn);
            }
        });
    }
}

// ------------------------------------------------------------------------ host
// M: so that the chunks of 16 rows or more are a grid's second dimension
constexpr int64_t kLimit = kDimLimit / 2, kLimitM = (int64_t)1 << 19, kLimitK = (int64_t)1 << 24;

int check_sizes(int64_t M, int64_t K, int dtype, uint32_t flags) {
    if (M < 0 || K <= 0 || M >= kLimitM || K >= kLimitK || K % kBlock) return FP4Q_ERR_SHAPE;
    if (flags & ~(uint32_t)FP4Q_FLAG_NO_FWHT) return FP4Q_ERR_ARG;
    return dtype == FP4Q_OUT_F32 || dtype == FP4Q_OUT_BF16 ? FP4Q_OK : FP4Q_ERR_ARG;
}
template <int kWaves, int kCols, int kStrips, int kBlocksAhead, bool kGated, Source kSource>
int run_kernel(Gemv4Args &p, const Plan &plan, void *stream) {
    static_assert(kLimitM / 16 <= 65535, "chunks");
    void *args[] = {&p};
    const dim3 grid((unsigned)plan.groups, (unsigned)plan.chunks);
    const hipError_t e = hipLaunchKernel((const void *)&gemv4_kernel<kWaves, kCols, kStrips, kBlocksAhead, kGated, kSource>,
                                         grid, dim3(kWaves * kWave), args, (size_t)plan.lds, (hipStream_t)stream);
    return e == hipSuccess ? FP4Q_OK : FP4Q_ERR_LAUNCH;
}
template <bool kGated>
int run_product(Gemv4Args &p, const Plan &plan, void *stream) {
    constexpr int kS = kGated ? 2 : 1;
    switch (plan.way) {
        case Way::kStaged:
            if (plan.waves == 16) return run_kernel<16, 1, kS, 1, kGated, Source::kStaged>(p, plan, stream);
            return run_kernel<8, 1, kS, 1, kGated, Source::kStaged>(p, plan, stream);
        case Way::kHeld: return run_kernel<16, 1, kS, 3 - kS, kGated, Source::kOne>(p, plan, stream);
        case Way::kLoaded: return run_kernel<8, 1, kS, 1, kGated, Source::kMemory>(p, plan, stream);
        default: return run_kernel<8, 2, 2, 1, kGated, Source::kMemory>(p, plan, stream);
    }
}

int run(const void *x, int dtype, int64_t M, const Payload &w, const Payload *up, int64_t N, int64_t K, int act,
        void *out, int out_dtype, uint32_t flags, void *workspace, size_t workspace_bytes, void *stream) {
    if (N < 0 || N >= kLimit) return FP4Q_ERR_SHAPE;
    const int st = check_sizes(M, K, dtype, flags);
    if (st != FP4Q_OK) return st;
    if ((out_dtype != FP4Q_OUT_F32 && out_dtype != FP4Q_OUT_BF16) || bad_act(act)) return FP4Q_ERR_ARG;
    if (M == 0 || N == 0) return FP4Q_OK;
    const int parts = parts_of(dtype, out_dtype, flags);
    const size_t need = workspace_of(M, K, parts, flags);
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
    Gemv4Args p = {x, nullptr, weights[0], weights[1], out, (int)M, (int)N, (int)K, parts, act,
                   out_dtype == FP4Q_OUT_F32, dtype == FP4Q_OUT_F32, !(flags & FP4Q_FLAG_NO_FWHT)};
    if (need) {
        _Float16 *to = static_cast<_Float16 *>(workspace);
        float *down = reinterpret_cast<float *>(to + M * parts * K);
        void *args[] = {&p, &to, &down};
        const dim3 grid((unsigned)ceil_div(K / kBlock, kReadyWaves), (unsigned)std::min<int64_t>(M, 65535));
        const int done = launch((const void *)&ready_kernel, grid, kReadyWaves * kWave, args, stream);
        if (done != FP4Q_OK) return done;
        p.x = to;
        p.down = down;
    }
    const Plan plan = plan_of(M, N, K, parts, flags, up != nullptr);
    return up ? run_product<true>(p, plan, stream) : run_product<false>(p, plan, stream);
}

}  // namespace

extern "C" {

int fp4q_gemv4_workspace(int64_t M, int64_t K, int dtype, uint32_t flags, size_t *bytes) {
    const int st = check_sizes(M, K, dtype, flags);
    if (st != FP4Q_OK) return st;
    if (!bytes) return FP4Q_ERR_NULL;
    // enough for either type of out
    *bytes = std::max(workspace_of(M, K, parts_of(dtype, FP4Q_OUT_F32, flags), flags),
                      workspace_of(M, K, parts_of(dtype, FP4Q_OUT_BF16, flags), flags));
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
