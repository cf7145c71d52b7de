// fp4q_norm.hip -- root-mean-square norm with the residual's addition and 8-bit
// output, and its gradients (declared in include/fp4q_linear.h).
//
//   h = x + residual    r = 1 / sqrt(mean(h^2) + eps)    y = h r w
//   dx = r (g - xhat mean(g xhat)) + dh with g = dy w, xhat = h r
//   dw = sum over the rows of dy xhat
//
// About ten operations per element against 6 to 8 bytes: bound by HBM.  Every
// tensor is read once and written once: a row stays in the registers of the
// wavefronts that share it from its load to its last store.  (The widest fp32 rows
// that go this way do not fit: where, and what it costs, stands at the kernels.)
#include "fp4q_f8.h"

namespace {

using namespace fp4q_f8;

typedef float f32x4 __attribute__((ext_vector_type(4)));

// Sum of one value per lane over the kWaves wavefronts that share a row.
// `lds` holds kWaves floats per row and call.
template <int kWaves>
__device__ __forceinline__ float row_sum(float v, float *lds, int wave) {
    v = sum64(v);
    if constexpr (kWaves > 1) {
        if ((threadIdx.x & (kWave - 1)) == 0) lds[wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) v += lds[i];
    }
    return v;
}

__device__ __forceinline__ float rstd_of(float sumsq, int cols, float eps) {
    return 1.0f / sqrtf(sumsq / (float)cols + eps);
}

struct NormArgs {
    const void *x, *residual, *weight;
    void *h, *y;
    uint8_t *codes;
    float *scales, *rstd;
    int64_t code_pitch;
    float eps;
    int rows, cols;
};

// kWaves wavefronts share a row, each lane holds kChunks chunks of 8 elements; a 128-group
// is 16 neighbouring lanes, so its maximum is four DPP steps.  kWhole: rows of whole
// 16-byte chunks; otherwise chunks lie at any element and the last one may be shorter.
// 8192 x 4096 bf16 with residual, y and codes: 54.6 us, 5.5 TB/s (a copy reaches 5.2); four
// wavefronts a row there: with eight it takes 57.5 us, with one (no barrier, 8 chunks a lane)
// 60.7.  999 x 5003 fp32: 12 us; one row of 4096: 4.7 us.  With fp32 rows of 32769 to 65536
// 43 words a lane go to scratch memory and back (116 when rows are not whole): 512 x 65536
// with residual, y and codes takes 140 us (4.1 TB/s; 1024 x 32768 130 us, bf16 of 512 x 65536
// 58 us and 5.2 TB/s), 512 x 40001 111 us (3.1 TB/s).
template <typename T, int kWaves, int kChunks, bool kWhole>
__global__ __launch_bounds__(kWaves == 1 ? 256 : kWaves * kWave) void norm_kernel(NormArgs a) {
    constexpr int kRows = kWaves == 1 ? 4 : 1;
    __shared__ float lds[kWaves];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave;
    const int part = kWaves == 1 ? 0 : wave;
    const int row = (int)blockIdx.x * kRows + (kWaves == 1 ? wave : 0);
    if (row >= a.rows) return;  // whole wavefronts, and no barrier with kWaves == 1
    const int64_t base = (int64_t)row * a.cols;
    const int first = 8 * (part * kWave + lane);  // element of chunk 0; chunk c is kStep c further
    constexpr int kStep = 8 * kWaves * kWave;

    Eight<T> in[kChunks];
    float v[kChunks][8];
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
        in[c].template load<kWhole>(static_cast<const T *>(a.x) + base + first + c * kStep, a.cols - first - c * kStep);
    if (a.residual) {
        Eight<T> add[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
            add[c].template load<kWhole>(static_cast<const T *>(a.residual) + base + first + c * kStep,
                                         a.cols - first - c * kStep);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            float p[8], q[8];
            in[c].get(p);
            add[c].get(q);
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] += q[i];
            in[c].set(p);  // the norm is taken of the stored sum
            in[c].template store<kWhole>(static_cast<T *>(a.h) + base + first + c * kStep, a.cols - first - c * kStep);
        }
    }
    float sumsq = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        in[c].get(v[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sumsq = fmaf(v[c][i], v[c][i], sumsq);
    }
    const float r = rstd_of(row_sum<kWaves>(sumsq, lds, part), a.cols, a.eps);
    if (a.rstd && threadIdx.x % (kWaves * kWave) == 0) a.rstd[row] = r;

#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int at = first + c * kStep, left = a.cols - at;
        Eight<T> wk;
        wk.template load<true>(static_cast<const T *>(a.weight) + at, left >= 8 ? 8 : 0);
        if (!kWhole && left < 8) wk.template load<false>(static_cast<const T *>(a.weight) + at, left);
        float wv[8];
        wk.get(wv);
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[c][i] = v[c][i] * r * wv[i];
            top = umax(top, mag(v[c][i]));
        }
        if (a.y) {
            Eight<T> o;
            o.set(v[c]);
            o.template store<kWhole>(static_cast<T *>(a.y) + base + at, left);
        }
        if (a.codes) {
            const Scale sc = scale_of<FP4Q_E4M3>(max16(top));
            if (left > 0) {
                u32x2 q;
                q[0] = code_quad<FP4Q_E4M3>(v[c][0], v[c][1], v[c][2], v[c][3], sc);
                q[1] = code_quad<FP4Q_E4M3>(v[c][4], v[c][5], v[c][6], v[c][7], sc);
                store_bytes8(a.codes + (int64_t)row * a.code_pitch + at, left, q);
                if ((lane & 15) == 0) a.scales[(int64_t)(at / kGroup) * a.rows + row] = sc.s;
            }
        }
    }
}

// Rows too long for registers: a workgroup per row, a wavefront per 128-group, two passes
// over the row (the second reads what the same lanes have read or written before).
constexpr int kAnyWaves = 4;
template <typename T>
__global__ __launch_bounds__(kAnyWaves * kWave) void norm_any_kernel(NormArgs a) {
    __shared__ float lds[kAnyWaves];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave;
    const int row = (int)blockIdx.x;
    const int groups = (a.cols + kGroup - 1) / kGroup;
    const int64_t base = (int64_t)row * a.cols;
    const T *x = static_cast<const T *>(a.x) + base;
    const T *res = static_cast<const T *>(a.residual);
    T *h = static_cast<T *>(a.h) + base;
    float sumsq = 0.0f;
    for (int g = wave; g < groups; g += kAnyWaves)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = g * kGroup + i * kWave + lane;
            if (k < a.cols) {
                float v = to_float(x[k]);
                if (res) {
                    const T s = from_float<T>(v + to_float(res[base + k]));
                    h[k] = s;
                    v = to_float(s);
                }
                sumsq = fmaf(v, v, sumsq);
            }
        }
    const float r = rstd_of(row_sum<kAnyWaves>(sumsq, lds, wave), a.cols, a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = r;
    const T *from = res ? h : x;
    const T *w = static_cast<const T *>(a.weight);
    for (int g = wave; g < groups; g += kAnyWaves) {
        float v[2];
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = g * kGroup + i * kWave + lane;
            v[i] = 0.0f;
            if (k < a.cols) {
                v[i] = to_float(from[k]) * r * to_float(w[k]);
                if (a.y) static_cast<T *>(a.y)[base + k] = from_float<T>(v[i]);
            }
            top = umax(top, mag(v[i]));
        }
        if (a.codes) {
            const Scale sc = scale_of<FP4Q_E4M3>(max64(top));
            const unsigned q = code_pair<FP4Q_E4M3, false>(0u, v[0], v[1], sc);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k = g * kGroup + i * kWave + lane;
                if (k < a.cols) a.codes[(int64_t)row * a.code_pitch + k] = (uint8_t)(q >> (8 * i));
            }
            if (lane == 0) a.scales[(int64_t)g * a.rows + row] = sc.s;
        }
    }
}

// ---------------------------------------------------------------- gradients
struct GradArgs {
    const void *dy, *h, *weight, *dh;
    const float *rstd;
    void *dx;
    float *partial;  // [workgroups x partial_pitch]
    int rows, cols, partial_pitch;
};

// kTeams teams of kWaves wavefronts, a row each at a time; the rows of a workgroup's teams
// are kTeams blockIdx.x + team, and gridDim.x kTeams further each turn.  The next row's
// loads are queued before the present row's sum is waited for (kAhead).  Each lane keeps
// its columns' part of dw in registers over all its rows; a workgroup's teams add theirs
// through LDS at the end, and weight_grad_kernel adds the workgroups'.  8192 x 4096 bf16 with
// dh: 54.7 us with the sum of the parts, 4.9 TB/s; a workgroup for each of 1024 rows at a
// time, without the loads ahead and with four times the parts, took 72 us.  With fp32 rows of
// 8193 to 16384 23 words a lane go to scratch memory and back in every turn (13 when rows are
// not whole): 2048 x 16384 with dh takes 137 us (3.9 TB/s; bf16 56 us and 4.8 TB/s),
// 1000 x 16384 80 us (3.3 TB/s).
template <typename T, int kTeams, int kWaves, int kChunks, bool kWhole>
__global__ __launch_bounds__(kTeams * kWaves * kWave) void norm_grad_kernel(GradArgs a) {
    constexpr bool kAhead = kChunks == 1;  // where the registers allow it
    constexpr int kStep = 8 * kWaves * kWave;
    constexpr int kKept = kTeams > 1 ? (kTeams - 1) * kWaves * kWave * kChunks * 2 : 1;
    __shared__ f32x4 kept[kKept];
    __shared__ float lds[2][kTeams][kWaves];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave, team = wave / kWaves, part = wave % kWaves;
    const int first = 8 * (part * kWave + lane);
    struct Row {
        Eight<T> dy[kChunks], h[kChunks], dh[kChunks];
        float r;
    };
    auto load = [&](Row &to, int row) __attribute__((always_inline)) {
        const bool here = row < a.rows;
        const int64_t base = (int64_t)(here ? row : 0) * a.cols;
        to.r = here ? a.rstd[row] : 0.0f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int at = first + c * kStep, left = here ? a.cols - at : 0;
            to.dy[c].template load<kWhole>(static_cast<const T *>(a.dy) + base + at, left);
            to.h[c].template load<kWhole>(static_cast<const T *>(a.h) + base + at, left);
            if (a.dh) to.dh[c].template load<kWhole>(static_cast<const T *>(a.dh) + base + at, left);
        }
    };
    Eight<T> weight[kChunks];
    float dw[kChunks][8];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int at = first + c * kStep;
        weight[c].template load<kWhole>(static_cast<const T *>(a.weight) + at, a.cols - at);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
    }
    const int stride = (int)gridDim.x * kTeams;
    Row now, next;
    int row = (int)blockIdx.x * kTeams + team, turn = 0;
    load(now, row);
    // every team makes the workgroup's number of turns, for the barrier in row_sum
    for (int lead = (int)blockIdx.x * kTeams; lead < a.rows; lead += stride, row += stride, turn ^= 1) {
        if (kAhead) load(next, row + stride);
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            float p[8], q[8], w[8];
            now.dy[c].get(p);
            now.h[c].get(q);
            weight[c].get(w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xhat = q[i] * now.r;
                dot = fmaf(p[i] * w[i], xhat, dot);
                dw[c][i] = fmaf(p[i], xhat, dw[c][i]);
            }
        }
        // two buffers in turn: a row's sums are read before the next barrier, and written
        // again only after it
        const float m = row_sum<kWaves>(dot, lds[turn][team], part) / (float)a.cols;
        const int64_t base = (int64_t)row * a.cols;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            now.dy[c].forget();
            now.h[c].forget();
            weight[c].forget();
            float p[8], q[8], w[8], s[8] = {};
            now.dy[c].get(p);
            now.h[c].get(q);
            weight[c].get(w);
            if (a.dh) now.dh[c].get(s);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[i] = fmaf(now.r, fmaf(-(q[i] * now.r), m, p[i] * w[i]), s[i]);
            Eight<T> o;
            o.set(p);
            const int at = first + c * kStep;
            o.template store<kWhole, false>(static_cast<T *>(a.dx) + base + at, row < a.rows ? a.cols - at : 0);
        }
        if (kAhead) now = next; else load(now, row + stride);
    }
    if constexpr (kTeams > 1) {
        f32x4 *mine = kept + (part * kWave + lane);
        if (team > 0) {
#pragma unroll
            for (int k = 0; k < 2 * kChunks; ++k)
                mine[((team - 1) * 2 * kChunks + k) * kWaves * kWave] =
                    f32x4{dw[k / 2][4 * (k % 2)], dw[k / 2][4 * (k % 2) + 1], dw[k / 2][4 * (k % 2) + 2], dw[k / 2][4 * (k % 2) + 3]};
        }
        __syncthreads();
        if (team > 0) return;
        for (int t = 0; t < kTeams - 1; ++t)
#pragma unroll
            for (int k = 0; k < 2 * kChunks; ++k) {
                const f32x4 v = mine[(t * 2 * kChunks + k) * kWaves * kWave];
#pragma unroll
                for (int i = 0; i < 4; ++i) dw[k / 2][4 * (k % 2) + i] += v[i];
            }
    }
    float *to = a.partial + (int64_t)blockIdx.x * a.partial_pitch;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int at = first + c * kStep;
        Eight<float> o;
        o.set(dw[c]);
        o.template store<kWhole, false>(to + at, a.cols - at);  // (16-byte aligned in either case)
    }
}

// Rows too long for registers: dx a row at a time (two passes over the row) ...
template <typename T>
__global__ __launch_bounds__(kAnyWaves * kWave) void norm_grad_any_kernel(GradArgs a) {
    __shared__ float lds[kAnyWaves];
    const int row = (int)blockIdx.x;
    const int64_t base = (int64_t)row * a.cols;
    const T *dy = static_cast<const T *>(a.dy) + base;
    const T *h = static_cast<const T *>(a.h) + base;
    const T *dh = static_cast<const T *>(a.dh);
    const T *w = static_cast<const T *>(a.weight);
    const float r = a.rstd[row];
    float dot = 0.0f;
    for (int k = threadIdx.x; k < a.cols; k += kAnyWaves * kWave)
        dot = fmaf(to_float(dy[k]) * to_float(w[k]), to_float(h[k]) * r, dot);
    const float m = row_sum<kAnyWaves>(dot, lds, threadIdx.x / kWave) / (float)a.cols;
    for (int k = threadIdx.x; k < a.cols; k += kAnyWaves * kWave) {
        const float add = dh ? to_float(dh[base + k]) : 0.0f;
        const float g = to_float(dy[k]) * to_float(w[k]);
        static_cast<T *>(a.dx)[base + k] = from_float<T>(fmaf(r, fmaf(-(to_float(h[k]) * r), m, g), add));
    }
}
// ... and its part of dw: 64 columns of every gridDim.y-th row per workgroup.
template <typename T>
__global__ __launch_bounds__(kAnyWaves * kWave) void weight_grad_any_kernel(GradArgs a) {
    __shared__ float lds[kAnyWaves][kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave;
    const int k = (int)blockIdx.x * kWave + lane;
    float sum = 0.0f;
    if (k < a.cols)
        for (int row = (int)blockIdx.y * kAnyWaves + wave; row < a.rows; row += (int)gridDim.y * kAnyWaves) {
            const int64_t at = (int64_t)row * a.cols + k;
            sum = fmaf(to_float(static_cast<const T *>(a.dy)[at]),
                       to_float(static_cast<const T *>(a.h)[at]) * a.rstd[row], sum);
        }
    lds[wave][lane] = sum;
    __syncthreads();
    if (wave == 0 && k < a.cols) {
#pragma unroll
        for (int i = 1; i < kAnyWaves; ++i) sum += lds[i][lane];
        a.partial[(int64_t)blockIdx.y * a.partial_pitch + k] = sum;
    }
}

// dw = sum of the parts: kSlices slices of them (part p in slice p % kSlices), four columns
// a thread, then the slices in their order.  A thread's loads do not wait for each other.
constexpr int kSlices = 32, kSumLanes = 16, kSumCols = 4 * kSumLanes;
__global__ __launch_bounds__(kSlices * kSumLanes) void weight_grad_kernel(const float *partial, int parts, int pitch,
                                                                          int cols, float *dweight) {
    __shared__ float lds[kSlices][kSumCols];
    const int lane = threadIdx.x % kSumLanes, slice = threadIdx.x / kSumLanes;
    const int k = (int)blockIdx.x * kSumCols + 4 * lane;
    f32x4 sum = {0, 0, 0, 0};
    if (k + 4 <= cols) {
#pragma unroll 8
        for (int p = slice; p < parts; p += kSlices) {
            sum += *reinterpret_cast<const f32x4 *>(partial + (int64_t)p * pitch + k);
        }
    } else {
        for (int p = slice; p < parts; p += kSlices)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (k + i < cols) sum[i] += partial[(int64_t)p * pitch + k + i];
    }
    *reinterpret_cast<f32x4 *>(&lds[slice][4 * lane]) = sum;
    __syncthreads();
    const int at = (int)blockIdx.x * kSumCols + (int)threadIdx.x;
    if (threadIdx.x < kSumCols && at < cols) {
        float total = lds[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < kSlices; ++i) total += lds[i][threadIdx.x];
        dweight[at] = total;
    }
}

// --------------------------------------------------------------------- host
// The kernel whose lanes hold a row of `cols` elements, its workgroup's threads and rows.
struct Pick {
    const void *fn;
    int threads, rows;
};
constexpr int kWidestNorm = 65536, kWidestGrad = 16384;

template <typename T, bool kWhole>
Pick pick_norm(int64_t cols) {
    if (cols <= 512) return {(const void *)&norm_kernel<T, 1, 1, kWhole>, 256, 4};
    if (cols <= 1024) return {(const void *)&norm_kernel<T, 1, 2, kWhole>, 256, 4};
    if (cols <= 2048) return {(const void *)&norm_kernel<T, 4, 1, kWhole>, 256, 1};
    if (cols <= 4096) return {(const void *)&norm_kernel<T, 4, 2, kWhole>, 256, 1};
    if (cols <= 8192) return {(const void *)&norm_kernel<T, 4, 4, kWhole>, 256, 1};
    if (cols <= 16384) return {(const void *)&norm_kernel<T, 16, 2, kWhole>, 1024, 1};
    if (cols <= 32768) return {(const void *)&norm_kernel<T, 16, 4, kWhole>, 1024, 1};
    return {(const void *)&norm_kernel<T, 16, 8, kWhole>, 1024, 1};
}
template <typename T, bool kWhole>
Pick pick_grad(int64_t cols) {
    if (cols <= 512) return {(const void *)&norm_grad_kernel<T, 16, 1, 1, kWhole>, 1024, 16};
    if (cols <= 1024) return {(const void *)&norm_grad_kernel<T, 8, 2, 1, kWhole>, 1024, 8};
    if (cols <= 2048) return {(const void *)&norm_grad_kernel<T, 4, 4, 1, kWhole>, 1024, 4};
    if (cols <= 4096) return {(const void *)&norm_grad_kernel<T, 2, 8, 1, kWhole>, 1024, 2};
    if (cols <= 8192) return {(const void *)&norm_grad_kernel<T, 1, 16, 1, kWhole>, 1024, 1};
    return {(const void *)&norm_grad_kernel<T, 1, 16, 2, kWhole>, 1024, 1};
}
Pick pick_norm(int64_t cols, int dtype) {
    const bool whole = cols % 8 == 0;
    if (dtype == FP4Q_OUT_F32) return whole ? pick_norm<float, true>(cols) : pick_norm<float, false>(cols);
    return whole ? pick_norm<bf16, true>(cols) : pick_norm<bf16, false>(cols);
}
Pick pick_grad(int64_t cols, int dtype) {
    const bool whole = cols % 8 == 0;
    if (dtype == FP4Q_OUT_F32) return whole ? pick_grad<float, true>(cols) : pick_grad<float, false>(cols);
    return whole ? pick_grad<bf16, true>(cols) : pick_grad<bf16, false>(cols);
}

int64_t partial_pitch(int64_t cols) { return ceil_div(cols, 4) * 4; }

// Parts of dw: at most a workgroup on each CU, and no more than make the same number of
// turns (333 rows in turns of one: 167 workgroups take two turns as 256 do).
int64_t grad_parts(int64_t rows, int64_t cols) {
    const int64_t each = cols <= kWidestGrad ? pick_grad(cols, FP4Q_OUT_F32).rows : kAnyWaves;
    const int64_t need = ceil_div(rows, each), turns = ceil_div(need, 256);
    return need ? ceil_div(need, turns) : 0;
}

}  // namespace

extern "C" {

int fp4q_rmsnorm(const void *x, const void *residual, const void *weight, float eps, int64_t rows,
                 int64_t cols, int dtype, void *h, void *y, uint8_t *codes, int64_t code_pitch,
                 float *scales, float *rstd, void *stream) {
    if (bad_dims(rows, cols)) return FP4Q_ERR_SHAPE;
    if (codes && (code_pitch < cols || code_pitch >= 2 * kDimLimit)) return FP4Q_ERR_SHAPE;
    if (dtype != FP4Q_OUT_F32 && dtype != FP4Q_OUT_BF16) return FP4Q_ERR_ARG;
    if (!(eps > 0.0f) || !(eps < __builtin_inff())) return FP4Q_ERR_ARG;
    if (rows == 0) return FP4Q_OK;
    if (!x || !weight || (residual && !h) || (!y && !codes) || (codes && !scales)) return FP4Q_ERR_NULL;
    if (!residual && h) return FP4Q_ERR_ARG;
    if (!codes && scales) return FP4Q_ERR_ARG;
    for (const void *p : {x, residual, weight, (const void *)h, (const void *)y, (const void *)codes})
        if (!aligned(p, 16)) return FP4Q_ERR_ALIGN;
    if (codes && code_pitch % 16) return FP4Q_ERR_ALIGN;
    if (!aligned(scales, 4) || !aligned(rstd, 4)) return FP4Q_ERR_ALIGN;
    const int64_t bytes = rows * cols * esize(dtype);
    const Range outs[] = {rng(h, bytes), rng(y, bytes), rng(codes, pitched(rows, cols, code_pitch)),
                          rng(scales, 4 * rows * ceil_div(cols, kGroup)), rng(rstd, 4 * rows)};
    // h may be the residual itself: each element is read before it is written
    const Range ins[] = {rng(x, bytes), rng(weight, cols * esize(dtype)),
                         h == residual ? Range{0, 0} : rng(residual, bytes)};
    if (clash(outs, 5, ins, 3)) return FP4Q_ERR_ARG;
    NormArgs a = {x, residual, weight, h, y, codes, scales, rstd, code_pitch, eps, (int)rows, (int)cols};
    void *args[] = {&a};
    if (cols > kWidestNorm)
        return launch(dtype == FP4Q_OUT_F32 ? (const void *)&norm_any_kernel<float>
                                            : (const void *)&norm_any_kernel<bf16>,
                      dim3((unsigned)rows), kAnyWaves * kWave, args, stream);
    const Pick p = pick_norm(cols, dtype);
    return launch(p.fn, dim3((unsigned)ceil_div(rows, p.rows)), p.threads, args, stream);
}

int fp4q_rmsnorm_backward_workspace(int64_t rows, int64_t cols, size_t *bytes) {
    if (bad_dims(rows, cols)) return FP4Q_ERR_SHAPE;
    if (!bytes) return FP4Q_ERR_NULL;
    *bytes = (size_t)(grad_parts(rows, cols) * partial_pitch(cols) * 4);
    return FP4Q_OK;
}

int fp4q_rmsnorm_backward(const void *dy, const void *h, const void *weight, const float *rstd,
                          const void *dh, int64_t rows, int64_t cols, int dtype, void *dx,
                          float *dweight, void *workspace, size_t workspace_bytes, void *stream) {
    if (bad_dims(rows, cols)) return FP4Q_ERR_SHAPE;
    if (dtype != FP4Q_OUT_F32 && dtype != FP4Q_OUT_BF16) return FP4Q_ERR_ARG;
    if (!dweight) return FP4Q_ERR_NULL;
    if (rows > 0 && (!dy || !h || !weight || !rstd || !dx || !workspace)) return FP4Q_ERR_NULL;
    if (!aligned(dweight, 4) || !aligned(rstd, 4)) return FP4Q_ERR_ALIGN;
    for (const void *p : {dy, h, weight, dh, (const void *)dx, (const void *)workspace})
        if (!aligned(p, 16)) return FP4Q_ERR_ALIGN;
    int parts = (int)grad_parts(rows, cols);
    int pitch = (int)partial_pitch(cols);
    const int64_t need = (int64_t)parts * pitch * 4;
    if (workspace_bytes < (size_t)need) return FP4Q_ERR_SHAPE;
    const int64_t bytes = rows * cols * esize(dtype);
    const Range outs[] = {rng(dx, bytes), rng(dweight, 4 * cols), rng(workspace, need)};
    const Range ins[] = {rng(dy, bytes), rng(h, bytes), rng(dh, bytes), rng(weight, cols * esize(dtype)),
                         rng(rstd, 4 * rows)};
    if (clash(outs, 3, ins, 5)) return FP4Q_ERR_ARG;
    GradArgs a = {dy, h, weight, dh, rstd, dx, static_cast<float *>(workspace), (int)rows, (int)cols, pitch};
    void *args[] = {&a};
    const bool f32 = dtype == FP4Q_OUT_F32;
    int st = FP4Q_OK;
    if (rows > 0 && cols <= kWidestGrad) {
        const Pick p = pick_grad(cols, dtype);
        st = launch(p.fn, dim3((unsigned)parts), p.threads, args, stream);
    } else if (rows > 0) {
        st = launch(f32 ? (const void *)&norm_grad_any_kernel<float> : (const void *)&norm_grad_any_kernel<bf16>,
                    dim3((unsigned)rows), kAnyWaves * kWave, args, stream);
        if (st == FP4Q_OK)
            st = launch(f32 ? (const void *)&weight_grad_any_kernel<float>
                            : (const void *)&weight_grad_any_kernel<bf16>,
                        dim3((unsigned)ceil_div(cols, kWave), (unsigned)parts), kAnyWaves * kWave, args, stream);
    }
    if (st != FP4Q_OK) return st;
    int c = (int)cols;
    const float *partial = a.partial;
    void *sum_args[] = {&partial, &parts, &pitch, &c, &dweight};
    return launch((const void *)&weight_grad_kernel, dim3((unsigned)ceil_div(cols, kSumCols)),
                  kSlices * kSumLanes, sum_args, stream);
}

}  // extern "C"
