// fp4q_norm.hip -- root-mean-square norm with the residual's addition and 8-bit
// output, and its gradients (declared in include/fp4q_linear.h).
//
//   h = x + residual    r = 1 / sqrt(mean(h^2) + eps)    y = h r w
//   dx = r (g - xhat mean(g xhat)) + dh with g = dy w, xhat = h r
//   dw = sum over the rows of dy xhat
//
// About ten operations per element against 6 to 8 bytes: bound by HBM.  Every
// tensor is read once and written once: a row stays in the registers of the
// wavefronts that share it from its load to its last store.
#include "fp4q_f8.h"

namespace {

using namespace fp4q_f8;

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

// Rows of whole 16-byte chunks.  kWaves wavefronts share a row, each lane holds
// kChunks chunks of 8 elements; a 128-group is 16 neighbouring lanes, so its
// maximum is four DPP steps.
template <typename T, int kWaves, int kChunks>
__global__ __launch_bounds__(kWaves == 1 ? 256 : kWaves * kWave) void norm_kernel(NormArgs a) {
    constexpr int kRows = kWaves == 1 ? 4 : 1;
    __shared__ float lds[kWaves];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave;
    const int part = kWaves == 1 ? 0 : wave;
    const int row = (int)blockIdx.x * kRows + (kWaves == 1 ? wave : 0);
    if (row >= a.rows) return;  // whole wavefronts, and no barrier with kWaves == 1
    const int chunks = a.cols / 8;
    const int64_t base = (int64_t)row * a.cols;
    const T *x = static_cast<const T *>(a.x) + base;

    Eight<T> in[kChunks];
    float v[kChunks][8];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int k = (c * kWaves + part) * kWave + lane;
        if (k < chunks) in[c].load(x + 8 * k); else in[c].zero();
    }
    if (a.residual) {
        const T *res = static_cast<const T *>(a.residual) + base;
        T *h = static_cast<T *>(a.h) + base;
        Eight<T> add[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = (c * kWaves + part) * kWave + lane;
            if (k < chunks) add[c].load(res + 8 * k); else add[c].zero();
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = (c * kWaves + part) * kWave + lane;
            float p[8], q[8];
            in[c].get(p);
            add[c].get(q);
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] += q[i];
            in[c].set(p);  // the norm is taken of the stored sum
            if (k < chunks) in[c].store(h + 8 * k);
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

    const T *w = static_cast<const T *>(a.weight);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int k = (c * kWaves + part) * kWave + lane;
        const bool valid = k < chunks;
        Eight<T> wk;
        if (valid) wk.load(w + 8 * k); else wk.zero();
        float wv[8];
        wk.get(wv);
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[c][i] = v[c][i] * r * wv[i];
            top = umax(top, mag(v[c][i]));
        }
        if (a.y && valid) {
            Eight<T> o;
            o.set(v[c]);
            o.store(static_cast<T *>(a.y) + base + 8 * k);
        }
        if (a.codes) {
            const Scale sc = scale_of<FP4Q_E4M3>(max16(top));
            if (valid) {
                u32x2 q;
                q[0] = code_quad<FP4Q_E4M3>(v[c][0], v[c][1], v[c][2], v[c][3], sc);
                q[1] = code_quad<FP4Q_E4M3>(v[c][4], v[c][5], v[c][6], v[c][7], sc);
                *reinterpret_cast<u32x2 *>(a.codes + (int64_t)row * a.code_pitch + 8 * k) = q;
                if ((lane & 15) == 0) a.scales[(int64_t)(k / 16) * a.rows + row] = sc.s;
            }
        }
    }
}

// Any width: a workgroup per row, a wavefront per 128-group, two passes over the
// row (the second reads what the same lanes have read or written before).
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
    float *partial;  // [workgroups x cols]
    int rows, cols;
};

// Rows of whole chunks.  A workgroup takes rows blockIdx.x, + gridDim.x, ...,
// and keeps its part of dw in registers over all of them; the parts are added
// by weight_grad_kernel.
template <typename T, int kWaves, int kChunks>
__global__ __launch_bounds__(kWaves * kWave) void norm_grad_kernel(GradArgs a) {
    __shared__ float lds[2][kWaves];
    const int lane = threadIdx.x & (kWave - 1);
    const int part = threadIdx.x / kWave;
    const int chunks = a.cols / 8;
    float dw[kChunks][8], w[kChunks][8];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int k = (c * kWaves + part) * kWave + lane;
        Eight<T> wk;
        if (k < chunks) wk.load(static_cast<const T *>(a.weight) + 8 * k); else wk.zero();
        wk.get(w[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
    }
    int turn = 0;
    for (int row = (int)blockIdx.x; row < a.rows; row += (int)gridDim.x, turn ^= 1) {
        const int64_t base = (int64_t)row * a.cols;
        Eight<T> dy[kChunks], h[kChunks], add[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = (c * kWaves + part) * kWave + lane;
            if (k < chunks) {
                dy[c].load(static_cast<const T *>(a.dy) + base + 8 * k);
                h[c].load(static_cast<const T *>(a.h) + base + 8 * k);
                if (a.dh) add[c].load(static_cast<const T *>(a.dh) + base + 8 * k);
            } else {
                dy[c].zero();
                h[c].zero();
                add[c].zero();
            }
        }
        const float r = a.rstd[row];
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            float p[8], q[8];
            dy[c].get(p);
            h[c].get(q);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xhat = q[i] * r;
                dot = fmaf(p[i] * w[c][i], xhat, dot);
                dw[c][i] = fmaf(p[i], xhat, dw[c][i]);
            }
        }
        // two buffers in turn: a row's sums are read before the next barrier,
        // and written again only after it
        const float m = row_sum<kWaves>(dot, lds[turn], part) / (float)a.cols;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int k = (c * kWaves + part) * kWave + lane;
            float p[8], q[8], s[8] = {};
            dy[c].get(p);
            h[c].get(q);
            if (a.dh) add[c].get(s);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[i] = fmaf(r, fmaf(-(q[i] * r), m, p[i] * w[c][i]), s[i]);
            Eight<T> o;
            o.set(p);
            if (k < chunks) o.store(static_cast<T *>(a.dx) + base + 8 * k);
        }
    }
    float *to = a.partial + (int64_t)blockIdx.x * a.cols;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int k = (c * kWaves + part) * kWave + lane;
        if (k < chunks) {
            Eight<float> o;
            o.set(dw[c]);
            o.store(to + 8 * k);
        }
    }
}

// Any width: dx a row at a time (two passes over the row) ...
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
        a.partial[(int64_t)blockIdx.y * a.cols + k] = sum;
    }
}

// dw[k] = sum of the parts, in their order: 16 slices of the parts, then those.
constexpr int kSlices = 16;
constexpr int kSliceCols = 16;
__global__ __launch_bounds__(kSlices * kSliceCols) void weight_grad_kernel(const float *partial, int parts,
                                                                           int cols, float *dweight) {
    __shared__ float lds[kSlices][kSliceCols];
    const int lane = threadIdx.x % kSliceCols;
    const int slice = threadIdx.x / kSliceCols;
    const int k = (int)blockIdx.x * kSliceCols + lane;
    float sum = 0.0f;
    if (k < cols)
        for (int p = slice; p < parts; p += kSlices) sum += partial[(int64_t)p * cols + k];
    lds[slice][lane] = sum;
    __syncthreads();
    if (slice == 0 && k < cols) {
#pragma unroll
        for (int i = 1; i < kSlices; ++i) sum += lds[i][lane];
        dweight[k] = sum;
    }
}

// --------------------------------------------------------------------- host
// The kernel whose lanes hold a row of `cols` elements, and its launch.
struct Pick {
    const void *fn;
    int threads, rows_per_wg;
};
constexpr int kWidest = 16 * kWave * 8 * 4;  // 16 wavefronts of 4 chunks

template <typename T>
Pick pick_norm(int64_t cols) {
    const int64_t c = ceil_div(cols / 8, kWave);  // chunks per lane of one wavefront
    if (c <= 1) return {(const void *)&norm_kernel<T, 1, 1>, 256, 4};
    if (c <= 2) return {(const void *)&norm_kernel<T, 1, 2>, 256, 4};
    if (c <= 4) return {(const void *)&norm_kernel<T, 4, 1>, 256, 1};
    if (c <= 8) return {(const void *)&norm_kernel<T, 4, 2>, 256, 1};
    if (c <= 16) return {(const void *)&norm_kernel<T, 4, 4>, 256, 1};
    if (c <= 32) return {(const void *)&norm_kernel<T, 16, 2>, 1024, 1};
    return {(const void *)&norm_kernel<T, 16, 4>, 1024, 1};
}
template <typename T>
Pick pick_grad(int64_t cols) {
    const int64_t c = ceil_div(cols / 8, kWave);
    if (c <= 4) return {(const void *)&norm_grad_kernel<T, 4, 1>, 256, 1};
    if (c <= 8) return {(const void *)&norm_grad_kernel<T, 4, 2>, 256, 1};
    if (c <= 16) return {(const void *)&norm_grad_kernel<T, 4, 4>, 256, 1};
    if (c <= 32) return {(const void *)&norm_grad_kernel<T, 16, 2>, 1024, 1};
    return {(const void *)&norm_grad_kernel<T, 16, 4>, 1024, 1};
}
bool whole_chunks(int64_t cols) { return cols % 8 == 0 && cols <= kWidest; }

// Parts of dw: as many workgroups as the card holds at once, at most a row each.
int64_t grad_parts(int64_t rows, int64_t cols) {
    const int64_t most = whole_chunks(cols) ? 1024 : 64;
    return rows < most ? rows : most;
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
    if (!whole_chunks(cols))
        return launch(dtype == FP4Q_OUT_F32 ? (const void *)&norm_any_kernel<float>
                                            : (const void *)&norm_any_kernel<bf16>,
                      dim3((unsigned)rows), kAnyWaves * kWave, args, stream);
    const Pick p = dtype == FP4Q_OUT_F32 ? pick_norm<float>(cols) : pick_norm<bf16>(cols);
    return launch(p.fn, dim3((unsigned)ceil_div(rows, p.rows_per_wg)), p.threads, args, stream);
}

int fp4q_rmsnorm_backward_workspace(int64_t rows, int64_t cols, size_t *bytes) {
    if (bad_dims(rows, cols)) return FP4Q_ERR_SHAPE;
    if (!bytes) return FP4Q_ERR_NULL;
    *bytes = (size_t)(grad_parts(rows, cols) * cols * 4);
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
    if (workspace_bytes < (size_t)parts * cols * 4) return FP4Q_ERR_SHAPE;
    const int64_t bytes = rows * cols * esize(dtype);
    const Range outs[] = {rng(dx, bytes), rng(dweight, 4 * cols), rng(workspace, (int64_t)parts * cols * 4)};
    const Range ins[] = {rng(dy, bytes), rng(h, bytes), rng(dh, bytes), rng(weight, cols * esize(dtype)),
                         rng(rstd, 4 * rows)};
    if (clash(outs, 3, ins, 5)) return FP4Q_ERR_ARG;
    GradArgs a = {dy, h, weight, dh, rstd, dx, static_cast<float *>(workspace), (int)rows, (int)cols};
    void *args[] = {&a};
    const bool f32 = dtype == FP4Q_OUT_F32;
    int st = FP4Q_OK;
    if (rows > 0 && whole_chunks(cols)) {
        const Pick p = f32 ? pick_grad<float>(cols) : pick_grad<bf16>(cols);
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
    void *sum_args[] = {&partial, &parts, &c, &dweight};
    return launch((const void *)&weight_grad_kernel, dim3((unsigned)ceil_div(cols, kSliceCols)),
                  kSlices * kSliceCols, sum_args, stream);
}

}  // extern "C"
