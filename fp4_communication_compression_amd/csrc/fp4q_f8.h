// fp4q_f8.h -- device and host helpers shared by the 8-bit linear-layer kernels
// (fp4q_norm.hip, fp4q_quant8.hip, fp4q_gemm8.hip): element types, 8-bit scales
// and codes, reductions over lanes, argument checks.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "fp4q_linear.h"
#include "fp4q_numerics.h"

namespace fp4q_f8 {

constexpr int kWave = 64;
constexpr int kGroup = FP4Q_GROUP8;
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

struct bf16 {
    uint16_t bits;
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(bf16 v) { return __uint_as_float((unsigned)v.bits << 16); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 from_float<bf16>(float v) {
    return bf16{(uint16_t)fp4q_num::bf16_rne_pair(v, v)};
}

// Eight consecutive elements, 16-byte aligned: one load of bf16, two of fp32.
template <typename T>
struct Eight;
template <>
struct Eight<bf16> {
    u32x4 w;
    __device__ __forceinline__ void load(const bf16 *p) { w = *reinterpret_cast<const u32x4 *>(p); }
    __device__ __forceinline__ void zero() { w = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = fp4q_num::bf16_rne_pair(v[2 * i], v[2 * i + 1]);
    }
    __device__ __forceinline__ void store(bf16 *p) const { *reinterpret_cast<u32x4 *>(p) = w; }
};
template <>
struct Eight<float> {
    u32x4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const u32x4 *>(p)[0];
        b = reinterpret_cast<const u32x4 *>(p)[1];
    }
    __device__ __forceinline__ void zero() { a = b = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(a[i]);
            v[4 + i] = __uint_as_float(b[i]);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = __float_as_uint(v[i]);
            b[i] = __float_as_uint(v[4 + i]);
        }
    }
    __device__ __forceinline__ void store(float *p) const {
        reinterpret_cast<u32x4 *>(p)[0] = a;
        reinterpret_cast<u32x4 *>(p)[1] = b;
    }
};

// ---------------------------------------------------------- scales and codes
template <int kFmt>
constexpr float kF8Max = kFmt == FP4Q_E4M3 ? 448.0f : 57344.0f;
constexpr float kAmaxFloor = 0x1p-100f;

// Magnitudes are compared as bit patterns: NaN > infinity > finite, so a block's
// largest pattern also says whether all of it is finite.
__device__ __forceinline__ unsigned mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ unsigned umax(unsigned a, unsigned b) { return a > b ? a : b; }

struct Scale {
    float s;    // what is stored
    float inv;  // correctly rounded 1 / s, for div_rn
};
template <int kFmt>
__device__ __forceinline__ Scale scale_of(unsigned amax_bits) {
    const float a = fmaxf(__uint_as_float(amax_bits), kAmaxFloor);
    float s = fp4q_num::div_rn(a, kF8Max<kFmt>, 1.0f / kF8Max<kFmt>);
    if (amax_bits >= 0x7F800000u) s = __uint_as_float(0x7FC00000u);
    return Scale{s, fp4q_num::rcp_rn(s)};
}

// Codes of v0 / s, v1 / s into bytes 0, 1 (kHi = false) or 2, 3 of old.  The
// quotients are at most fmax (1 + 2^-23), which rounds to fmax: no clamp.
template <int kFmt, bool kHi>
__device__ __forceinline__ unsigned code_pair(unsigned old, float v0, float v1, Scale sc) {
    const float q0 = fp4q_num::div_rn(v0, sc.s, sc.inv), q1 = fp4q_num::div_rn(v1, sc.s, sc.inv);
    if constexpr (kFmt == FP4Q_E4M3)
        return __builtin_amdgcn_cvt_pk_fp8_f32(q0, q1, old, kHi);
    else
        return __builtin_amdgcn_cvt_pk_bf8_f32(q0, q1, old, kHi);
}
template <int kFmt>
__device__ __forceinline__ unsigned code_quad(float v0, float v1, float v2, float v3, Scale sc) {
    return code_pair<kFmt, true>(code_pair<kFmt, false>(0u, v0, v1, sc), v2, v3, sc);
}

// --------------------------------------------------------- lane reductions
// Rotations inside a row of 16 lanes (DPP row_ror): every lane of the row ends
// with the row's result, in the same order of operations on every lane pair.
template <int kRot>
__device__ __forceinline__ unsigned ror16(unsigned v) {
    return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + kRot, 0xF, 0xF, true);
}
__device__ __forceinline__ unsigned max16(unsigned v) {
    v = umax(v, ror16<8>(v));
    v = umax(v, ror16<4>(v));
    v = umax(v, ror16<2>(v));
    return umax(v, ror16<1>(v));
}
__device__ __forceinline__ float sum16(float v) {
    v += __uint_as_float(ror16<8>(__float_as_uint(v)));
    v += __uint_as_float(ror16<4>(__float_as_uint(v)));
    v += __uint_as_float(ror16<2>(__float_as_uint(v)));
    v += __uint_as_float(ror16<1>(__float_as_uint(v)));
    return v;
}
__device__ __forceinline__ float sum64(float v) {
    v = sum16(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}
__device__ __forceinline__ unsigned max64(unsigned v) {
    v = max16(v);
    v = umax(v, (unsigned)__shfl_xor((int)v, 16));
    return umax(v, (unsigned)__shfl_xor((int)v, 32));
}

// ------------------------------------------------------------------- host
inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Range {
    uintptr_t lo, hi;
};
// A NULL pointer or an empty array overlaps nothing.
inline Range rng(const void *p, int64_t bytes) {
    if (!p || bytes <= 0) return {0, 0};
    return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
// Bytes of a pitched byte matrix, without the last row's padding.
inline int64_t pitched(int64_t rows, int64_t cols, int64_t pitch) {
    return rows > 0 ? (rows - 1) * pitch + cols : 0;
}
// Whether any of outs[0 .. no) meets another of them or one of ins[0 .. ni).
inline bool clash(const Range *outs, int no, const Range *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i], outs[j])) return true;
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i], ins[j])) return true;
    }
    return false;
}

constexpr int64_t kDimLimit = (int64_t)1 << 28;
inline bool bad_dims(int64_t rows, int64_t cols) {
    return rows < 0 || cols <= 0 || rows >= kDimLimit || cols >= kDimLimit;
}
inline int esize(int dtype) { return dtype == FP4Q_OUT_F32 ? 4 : 2; }

inline int launch(const void *fn, dim3 grid, int threads, void **args, void *stream) {
    const hipError_t e = hipLaunchKernel(fn, grid, dim3((unsigned)threads), args, 0, (hipStream_t)stream);
    return e == hipSuccess ? FP4Q_OK : FP4Q_ERR_LAUNCH;
}

}  // namespace fp4q_f8
