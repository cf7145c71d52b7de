// fp4q_f8.h -- device and host helpers shared by the 8-bit linear-layer kernels
// (fp4q_norm.hip, fp4q_quant8.hip, fp4q_gemm8.hip): element types, 8-bit scales
// and codes, reductions over lanes, argument checks.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

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

// 16 bytes at an element's alignment: one load or store all the same (rows of an odd
// length begin anywhere).
template <typename T>
struct Loose;
template <>
struct Loose<bf16> {
    typedef u32x4 Vec __attribute__((aligned(2)));
};
template <>
struct Loose<float> {
    typedef u32x4 Vec __attribute__((aligned(4)));
};

// Eight consecutive elements as they lie in memory.  With kWhole, p is 16-byte aligned and
// all eight exist or none; otherwise the first `left` exist.
// Non-temporal stores leave the caches to what is read: at 8192 x 4096 bf16 the norm takes
// 54.8 us with them and 58.9 without, the quantiser 26.9 and 31.2 (both orders).  Not for
// the backward's one output against three inputs (1 us more), and not for loads: those cost
// the norm 4 us, and the backward of tensors that the caches still hold a tenth (1000 x
// 11008: 25 against 22 us).
template <typename T>
struct Eight {
    static constexpr int kWords = 2 * (int)sizeof(T);
    unsigned w[kWords];

    template <bool kWhole>
    __device__ __forceinline__ void load(const T *p, int left) {
        using Vec = std::conditional_t<kWhole, u32x4, typename Loose<T>::Vec>;
        if (left >= 8) {
#pragma unroll
            for (int k = 0; k < kWords / 4; ++k) {
                const u32x4 v = reinterpret_cast<const Vec *>(p)[k];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[4 * k + i] = v[i];
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
        if (!kWhole) {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < left) put(i, p[i]);
        }
    }
    template <bool kWhole, bool kStream = true>
    __device__ __forceinline__ void store(T *p, int left) const {
        using Vec = std::conditional_t<kWhole, u32x4, typename Loose<T>::Vec>;
        if (left >= 8) {
#pragma unroll
            for (int k = 0; k < kWords / 4; ++k) {
                const Vec v = {w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]};
                Vec *to = reinterpret_cast<Vec *>(p) + k;
                if constexpr (kStream)
                    __builtin_nontemporal_store(v, to);
                else
                    *to = v;
            }
        } else if (!kWhole) {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < left) p[i] = pick(i);
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_float(pick(i));
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = fp4q_num::bf16_rne_pair(v[2 * i], v[2 * i + 1]);
        }
    }

    // Hides the words' origin: what was computed from them before is computed again rather
    // than held in registers.
    __device__ __forceinline__ void forget() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(w[i]));
    }

   private:
    __device__ __forceinline__ void put(int i, T v) {
        if constexpr (sizeof(T) == 4)
            w[i] = __float_as_uint(v);
        else
            w[i >> 1] |= (unsigned)v.bits << (16 * (i & 1));
    }
    __device__ __forceinline__ T pick(int i) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[i]);
        else
            return bf16{(uint16_t)(w[i >> 1] >> (16 * (i & 1)))};
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

// The first min(left, 8) bytes of w; p is 8-byte aligned.
__device__ __forceinline__ void store_bytes8(uint8_t *p, int left, u32x2 w) {
    if (left >= 8) {
        __builtin_nontemporal_store(w, reinterpret_cast<u32x2 *>(p));
    } else {
        for (int j = 0; j < left; ++j) p[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
    }
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

// A launch's size is counted in threads, in 32 bits.
inline int launch(const void *fn, dim3 grid, int threads, void **args, void *stream) {
    if ((uint64_t)grid.x * (uint64_t)threads > 0xFFFFFFFFu) return FP4Q_ERR_SHAPE;
    const hipError_t e = hipLaunchKernel(fn, grid, dim3((unsigned)threads), args, 0, (hipStream_t)stream);
    return e == hipSuccess ? FP4Q_OK : FP4Q_ERR_LAUNCH;
}

}  // namespace fp4q_f8
