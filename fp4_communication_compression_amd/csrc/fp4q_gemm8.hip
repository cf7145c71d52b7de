// fp4q_gemm8.hip -- the product of two 8-bit operands with a scale for each block
// of 128 (declared in include/fp4q_linear.h):
//
//   out[m][n] = sum over blocks kb of sa[kb][m] sb[kb][n or n / 128]
//               sum over k in kb of a[m][k] b[n][k]
//
// b is the matrix core's first operand: a lane then holds four neighbouring n of
// one m, a's scale is one value per lane, and the output leaves in pieces of four
// neighbours.  A block's sum over its 128 k is multiplied by b's scale, then by a's,
// and added to the fp32 accumulators.  The product of the two scales is never taken
// by itself: it can leave fp32's range where the scaled sum does not (a sum of 0
// under two scales of 2^70 is 0, not 0 infinity).  A scale of a row of b is a
// multiplication after the matrix core.  The scale of a tile of b, one for all of a
// wavefront's columns, is split: its power of two goes into the matrix core's
// products, its rest to a's scales, with no work on the sums: against the product of
// the scales it takes 2.5 to 4 % longer (8192 x 11008, K = 4096: 361 for 352 us on one
// card; 2047 x 4096, K = 11008: 92.5 for 89), a multiplication of the sums 16 to 18 %
// (408 and 106).  Two forms of a step, the plain one for blocks whose scales allow it,
// spill hundreds of registers.
//
// Two ways to the block's sum:
//   8-bit matrix core  (bf16 output) one v_mfma_f32_16x16x128_f8f6f4 covers the
//     block of a 16 x 16 tile.  It adds the products of 8 neighbouring k at the
//     largest one's exponent and drops what lies below 2^-13 of it (seen with
//     powers of two; groups of 8 are added in fp32): at most 7 2^-13 of each
//     group's largest product (2.1 2^-13 seen on groups of two large products that
//     cancel and six small ones, there two thirds of the result).  Over normal
//     values it is about 2e-5 of the result, a hundredth of the output's own
//     rounding: that is why bf16 output takes it, and fp32 output does not.
//   16-bit matrix core (fp32 output) the codes become bf16, which holds every
//     E4M3 and E5M2 value, and four v_mfma_f32_16x16x32_bf16 add their exact
//     products in fp32: half the rate, 1e-8 per block.
#include <type_traits>
#include <utility>

#include "fp4q_f8.h"
#include "fp4q_gemm8_plan.h"

namespace {

using namespace fp4q_f8;
using namespace fp4q_plan;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

#define FP4Q_INLINE __attribute__((always_inline))
// Calls f(std::integral_constant<int, I>) for I = 0 .. N-1.
template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F &&f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F &&f) {
    static_for_impl(f, std::make_integer_sequence<int, N>{});
}

struct GemmArgs {
    const uint8_t *a, *b;
    const float *sa, *sb;
    void *out;
    int64_t a_pitch, b_pitch;
    int M, N, K;
    int tiles_m, tiles_n;
    int accumulate;
    // K in `parts` runs of blocks, a workgroup each; with more than one, run s's sums go
    // to partial + s part_size, and join_kernel adds them
    int parts;
    int64_t part_size;
    float *partial;
};

// 32 codes of a row as loaded (of a block's 128, in an order that both operands share) ...
struct Raw {
    u32x4 low, high;
};
// A scale as a power of two times the rest, 1 <= |rest| < 2: a finite value of an operand
// over its scale's rest is finite.  Scales below 2^-100 leave more to the rest (a code times
// the power is a normal bf16), and zero, infinity and NaN are all rest.
struct Split {
    int powers;  // byte 0: the power's exponent, biased as in fp32; byte 2: that of 1
    float rest;
    __device__ __forceinline__ void set(float scale) {
        const int e = max(__builtin_amdgcn_frexp_expf(scale), -99);  // scale = rest 2^(e - 1)
        powers = e + (126 | 127 << 16);
        rest = ldexpf(scale, 1 - e);
    }
    __device__ __forceinline__ float factor() const { return __uint_as_float((unsigned)powers << 23); }
};
// ... and as the matrix core takes them, times a power of two.
template <int kFmt, bool kPrecise>
struct Frag;
template <int kFmt>
struct Frag<kFmt, false> {
    i32x8 v;
    __device__ __forceinline__ void set(const Raw &raw, float = 1.0f) {  // (block_product takes the power here)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = (int)raw.low[i];
            v[4 + i] = (int)raw.high[i];
        }
    }
};
template <int kFmt>
struct Frag<kFmt, true> {
    bf16x8 v[4];
    __device__ __forceinline__ void set(const Raw &raw, float power = 1.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned w = i < 4 ? raw.low[i] : raw.high[i - 4];
            bf16x2 p, q;
            if constexpr (kFmt == FP4Q_E4M3) {
                p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, power, false);
                q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, power, true);
            } else {
                p = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, power, false);
                q = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, power, true);
            }
            const int at = 4 * (i & 1);
            v[i >> 1][at] = p[0];
            v[i >> 1][at + 1] = p[1];
            v[i >> 1][at + 2] = q[0];
            v[i >> 1][at + 3] = q[1];
        }
    }
};

// One block's product of a 16 x 16 tile.  With kScaled the 8-bit matrix core's products take
// the powers of two in bytes 0 (for `first`) and 2 (for `second`) of powers.
template <bool kScaled, int kFirst, int kSecond>
__device__ __forceinline__ f32x4 block_product(const Frag<kFirst, false> &first, const Frag<kSecond, false> &second,
                                               int powers) {
    constexpr f32x4 kZero = {0, 0, 0, 0};
    if constexpr (kScaled)
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(first.v, second.v, kZero, kFirst, kSecond, 0, powers,
                                                                2, powers);
    // with scale operands 0 this is the instruction without the matrix core's own scaling
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(first.v, second.v, kZero, kFirst, kSecond, 0, 0, 0, 0);
}
template <bool kScaled, int kFirst, int kSecond>
__device__ __forceinline__ f32x4 block_product(const Frag<kFirst, true> &first, const Frag<kSecond, true> &second, int) {
    f32x4 d = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(first.v[i], second.v[i], d, 0, 0, 0);
    return d;
}

// A workgroup's tile: kWavesM x kWavesN wavefronts of kTilesM x kTilesN tiles of
// 16 x 16 each, a block of 128 k at a time.
template <int kWavesM_, int kWavesN_, int kTilesM_, int kTilesN_>
struct Shape {
    static constexpr int kWavesM = kWavesM_, kWavesN = kWavesN_, kTilesM = kTilesM_, kTilesN = kTilesN_;
    static constexpr int kWaveM = 16 * kTilesM, kWaveN = 16 * kTilesN;
    static constexpr int kM = kWavesM * kWaveM, kN = kWavesN * kWaveN;
    static constexpr int kWaves = kWavesM * kWavesN;
    static constexpr int kThreads = kWave * kWaves;
    // loads of 8 rows of 128 bytes for a wavefront and block
    static constexpr int kLoadsA = kM / 8 / kWaves, kLoadsB = kN / 8 / kWaves;
    static_assert(kM % (8 * kWaves) == 0 && kN % (8 * kWaves) == 0, "whole loads");
};

typedef __attribute__((address_space(3))) void lds_void;

// One block of both operands with its scales, as staged in LDS.  Rows are 128 bytes;
// chunk c (16 bytes) of row r lies at chunk c ^ (r / 2 & 7).
template <typename S>
struct alignas(16) Stage {
    static constexpr int kScalesA = (S::kM + kWave - 1) / kWave * kWave;
    float scales[kScalesA + S::kN];  // a's, then b's; first: within reach of a read's 16-bit offset
    u32x4 a[S::kM * 8], b[S::kN * 8];
};

// kBytes (4 or 16) a lane from `bytes` bytes at `from` straight into LDS at `to` (uniform;
// lane l's part goes to to + kBytes l).  Lanes whose offset lies outside read nothing.  As
// instructions of its own, out of the compiler's sight: it would make LDS reads of other
// blocks wait for these loads.  meet() waits for them; they write no register.
template <int kBytes>
__device__ __forceinline__ void load_to_lds(void *to, const void *from, int bytes, int offset) {
    const uint64_t base = (uint64_t)from;
    const u32x4 descriptor = {(unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)base),
                              (unsigned)__builtin_amdgcn_readfirstlane((int)((base >> 32) & 0xFFFF)),
                              (unsigned)__builtin_amdgcn_readfirstlane(max(bytes, 0)), 0x00020000u};
    const int at = __builtin_amdgcn_readfirstlane((int)(unsigned)(uintptr_t)(lds_void *)to);
    // M0 holds the address in LDS; then the wait states between scalar writes and the load
    // that reads them.  The compiler warns that it does not keep M0 across the assembly: it
    // need not, only to know that M0 is written.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
    if constexpr (kBytes == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     : : "s"(at), "v"(offset), "s"(descriptor) : "m0", "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds"
                     : : "s"(at), "v"(offset), "s"(descriptor) : "m0", "memory");
#pragma clang diagnostic pop
}

// A meeting of the workgroup's wavefronts, each with at most kLeft of its loads into LDS
// on their way: the barrier alone waits for a wavefront's LDS reads and writes, not for
// those loads.
template <int kLeft>
__device__ __forceinline__ void meet() {
    static_assert(kLeft < 64, "six bits");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (kLeft & 15) | (kLeft >> 4) << 14);  // vmcnt(kLeft)
    __syncthreads();
}

template <typename S, int kFmtA, int kFmtB, bool kTiles, bool kPrecise>
struct Tile {
    const GemmArgs &p;
    int lane, wave, m0, n0, wm, wn, row16, quarter;
    int low_a, high_a, low_b, high_b;  // a lane's two chunks of its wavefront's first 16 rows in LDS
    int offset_a, offset_b;  // of a lane's 16 bytes from the 8 rows that its wavefront loads at once
    const uint8_t *from_a, *from_b;  // the tile's rows
    int bytes_a, bytes_b;            // to the end of their last one's last whole 16 bytes
    f32x4 acc[S::kTilesM][S::kTilesN];

    __device__ __forceinline__ Tile(const GemmArgs &args, int tm, int tn) : p(args) {
        lane = threadIdx.x & (kWave - 1);
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        m0 = tm * S::kM;
        n0 = tn * S::kN;
        wm = wave % S::kWavesM * S::kWaveM;
        wn = wave / S::kWavesM * S::kWaveN;
        row16 = lane & 15;
        quarter = lane >> 4;
        // a lane's 32 codes of a row are its chunks quarter and quarter + 4: with chunks 2 quarter
        // and 2 quarter + 1 two lanes of each 16 that a read takes at once meet in one bank
        // (8.1 instead of 4.6 cycles a read)
        const int low = row16 * kGroup + 16 * (quarter ^ (row16 >> 1));
        const int high = row16 * kGroup + 16 * ((quarter + 4) ^ (row16 >> 1));
        low_a = wm * kGroup + low;
        high_a = wm * kGroup + high;
        low_b = wn * kGroup + low;
        high_b = wn * kGroup + high;
        const int wide = (p.K + 15) & ~15;
        from_a = p.a + (int64_t)m0 * p.a_pitch;
        from_b = p.b + (int64_t)n0 * p.b_pitch;
        bytes_a = (min(S::kM, p.M - m0) - 1) * (int)p.a_pitch + wide;
        bytes_b = (min(S::kN, p.N - n0) - 1) * (int)p.b_pitch + wide;
        static_assert(S::kWaves % 2 == 0, "the rows of a wavefront's loads have one swizzle");
        const int chunk = (lane & 7) ^ ((wave * 8 + (lane >> 3)) >> 1 & 7);
        offset_a = (lane >> 3) * (int)p.a_pitch + 16 * chunk;
        offset_b = (lane >> 3) * (int)p.b_pitch + 16 * chunk;
#pragma unroll
        for (int i = 0; i < S::kTilesM; ++i)
#pragma unroll
            for (int j = 0; j < S::kTilesN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    }

    // Eight rows of one operand straight into LDS.  The descriptor begins with the first of
    // them and ends with the operand, so rows past its end are not read (what their place
    // in LDS holds only meets outputs that are not stored).
    __device__ __forceinline__ void fetch_rows(u32x4 *to, const uint8_t *from, int bytes, int at, int offset) {
        load_to_lds<16>(to, from + at, bytes - at, offset);
    }

    // Queues block kb's loads.
    __device__ __forceinline__ void fetch(Stage<S> &to, int kb) {
        const int a_pitch = (int)p.a_pitch, b_pitch = (int)p.b_pitch;
#pragma unroll
        for (int i = 0; i < S::kLoadsA; ++i) {
            const int r = (i * S::kWaves + wave) * 8;
            fetch_rows(to.a + r * 8, from_a, bytes_a, r * a_pitch + kb * kGroup, offset_a);
        }
#pragma unroll
        for (int i = 0; i < S::kLoadsB; ++i) {
            const int r = (i * S::kWaves + wave) * 8;
            fetch_rows(to.b + r * 8, from_b, bytes_b, r * b_pitch + kb * kGroup, offset_b);
        }
        // 64 scales a wavefront; of b's tiles one for each 128 columns.  A wavefront without
        // scales of its own repeats another one's: each has the same number of loads to wait for.
        constexpr int kCountA = (S::kM + kWave - 1) / kWave;
        constexpr int kCountB = kTiles ? 1 : (S::kN + kWave - 1) / kWave;
        static_assert(kCountA + kCountB <= S::kWaves && S::kM % 32 == 0 && S::kN % kGroup == 0, "one load each");
        const int cols = kTiles ? (p.N + kGroup - 1) / kGroup : p.N, c0 = kTiles ? n0 / kGroup : n0;
        const int w = min(wave, kCountA + kCountB - 1);
        const bool of_a = w < kCountA;
        const int count = of_a ? p.M : cols, at = of_a ? m0 + w * kWave : c0 + (w - kCountA) * kWave;
        load_to_lds<4>(to.scales + w * kWave, (of_a ? p.sa : p.sb) + (int64_t)kb * count + at,
                       min(count - at, kWave) * 4, 4 * lane);
    }
    static constexpr int kFetched = S::kLoadsA + S::kLoadsB + 1;  // loads of a wavefront and block

    // Clears the codes from K on in the last block.
    __device__ __forceinline__ void clear_tail(Stage<S> &in) {
        const int left = p.K % kGroup;
        for (int r = threadIdx.x; r < S::kM + S::kN; r += S::kThreads) {
            u32x4 *row = r < S::kM ? in.a + r * 8 : in.b + (r - S::kM) * 8;
            for (int c = left / 16; c < 8; ++c) {
                u32x4 w = row[c ^ (r >> 1 & 7)];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int keep = left - 16 * c - 4 * i;
                    w[i] = keep >= 4 ? w[i] : keep <= 0 ? 0u : w[i] & ((1u << (8 * keep)) - 1);
                }
                row[c ^ (r >> 1 & 7)] = w;
            }
        }
    }

    // LDS is read at one byte offset from its variable: through longer chains of addresses
    // the compiler loses sight of the variable, and then waits for every load under way.
    template <typename T>
    static __device__ __forceinline__ T at(const Stage<S> &in, int offset) {
        return *reinterpret_cast<const T *>(reinterpret_cast<const char *>(&in) + offset);
    }
    static constexpr int kA = (int)__builtin_offsetof(Stage<S>, a), kB = (int)__builtin_offsetof(Stage<S>, b);
    __device__ __forceinline__ Raw raw_a(const Stage<S> &in, int i) {
        return {at<u32x4>(in, low_a + (kA + i * 16 * kGroup)), at<u32x4>(in, high_a + (kA + i * 16 * kGroup))};
    }
    __device__ __forceinline__ Raw raw_b(const Stage<S> &in, int j) {
        return {at<u32x4>(in, low_b + (kB + j * 16 * kGroup)), at<u32x4>(in, high_b + (kB + j * 16 * kGroup))};
    }
    __device__ __forceinline__ float scale_a(const Stage<S> &in, int i) {
        return at<float>(in, 4 * (wm + row16) + 64 * i);
    }

    // What a block's multiplication begins with, read during the one before it.
    struct Head {
        Raw b[S::kTilesN], a;
        float sa, sb;
        Split tile;  // sb, with kTiles
    };
    __device__ __forceinline__ void read_head(const Stage<S> &in, Head &h, int item) {
        if (item == 0) {
            h.a = raw_a(in, 0);
            h.sa = scale_a(in, 0);
            h.sb = 1.0f;
            if constexpr (kTiles) {
                static_assert(kGroup % S::kWaveN == 0, "one tile of b's scales per wavefront");
                h.sb = at<float>(in, 4 * (in.kScalesA + wn / kGroup));
            }
        } else {
            h.b[item - 1] = raw_b(in, item - 1);
        }
    }

    // b's tiles in a head; the other ones are read at the block's beginning
    static constexpr int kHeadB = S::kTilesN - 2;
    // rows of a's tiles multiplied before the wavefronts meet, and rows read by the end of row i
    static constexpr int kMeet = S::kTilesM * 3 / 4;
    static constexpr int rows_read(int i) { return i + 3 < S::kTilesM ? i + 3 : S::kTilesM; }
    static_assert(rows_read(kMeet - 1) == S::kTilesM, "the block is in registers when the wavefronts meet");
    // items of the next block's head read by the end of row i >= kMeet
    static constexpr int head_read(int i) {
        const int before = i > kMeet ? head_read(i - 1) : 0;
        return before + (kHeadB + 1 - before) / (S::kTilesM - i);
    }

    // Multiplies the block in `cur`.  At three quarters, when all of it is in registers,
    // the wavefronts meet: the next block's loads have landed in `nxt` then, and those of
    // the one after it can go to `cur`.  The last quarter reads the next block's head, so
    // no wavefront waits for LDS at a block's beginning.  The products run kLag tiles
    // ahead of their scaled addition, so that the vector unit adds one tile while the
    // matrix core works on the next ones.
    __device__ __forceinline__ void step(Stage<S> &cur, Stage<S> &nxt, Head &h, Head &n, int kb, int end, bool ragged) {
        constexpr int kLag = 3, kTilesM = S::kTilesM, kTilesN = S::kTilesN;
        constexpr int kCount = kTilesM * kTilesN;
        Raw ra[kTilesM];
        Frag<kFmtA, kPrecise> fa[2];
        Frag<kFmtB, kPrecise> fb[kTilesN];
        float sa[kTilesM];
        f32x4 sb[kTilesN], d[kLag + 1];
        const float factor = kTiles ? h.tile.factor() : 1.0f;
        const int powers = kTiles ? h.tile.powers : 0;
        ra[0] = h.a;
        sa[0] = h.sa;
#pragma unroll
        for (int j = kHeadB; j < kTilesN; ++j) h.b[j] = raw_b(cur, j);
        if constexpr (!kTiles) {
#pragma unroll
            for (int j = 0; j < kTilesN; ++j)
                sb[j] = at<f32x4>(cur, 4 * (cur.kScalesA + wn + 4 * quarter) + 64 * j);
        }
        static_for<kCount + kLag>([&](auto step_of) FP4Q_INLINE {
            constexpr int t = step_of.value, i = t / kTilesN, j = t % kTilesN;
            if constexpr (j == 0 && i < kMeet) {
                constexpr int from = i ? rows_read(i - 1) : 1, count = rows_read(i) - from;
                static_for<count>([&](auto k) FP4Q_INLINE {
                    ra[from + k.value] = raw_a(cur, from + k.value);
                    sa[from + k.value] = scale_a(cur, from + k.value);
                });
            }
            if constexpr (t == kMeet * kTilesN) {
                static_for<kMeet * kTilesN>([&](auto x) FP4Q_INLINE { asm volatile("" : "+v"(acc[x.value / kTilesN][x.value % kTilesN])); });
                meet<0>();
                if (kb + 2 < end) {
                    fetch(cur, kb + 2);
                } else if (kb + 2 == end && ragged) {
                    clear_tail(nxt);
                    __syncthreads();
                }
            }
            if constexpr (j == 0 && i >= kMeet && i < kTilesM) {
                constexpr int from = i > kMeet ? head_read(i - 1) : 0, count = head_read(i) - from;
                static_for<count>([&](auto k) FP4Q_INLINE { read_head(nxt, n, from + k.value); });
            }
            if constexpr (t < kCount) {
                // fragments are made where their first product needs them, and the next row's
                // while the matrix core works on this one's
                if constexpr (t == 0) fa[0].set(ra[0]);
                if constexpr (i == 0) fb[j].set(h.b[j], factor);
                d[t % (kLag + 1)] = block_product<kTiles>(fb[j], fa[i & 1], powers);
            }
            __builtin_amdgcn_sched_barrier(0);  // the matrix core first
            if constexpr (kTiles && t == kCount - 1) n.tile.set(n.sb);
            if constexpr (j == kTilesN - 1 && i + 1 < kTilesM) fa[(i + 1) & 1].set(ra[i + 1]);
            if constexpr (t >= kLag) {
                constexpr int ui = (t - kLag) / kTilesN, uj = (t - kLag) % kTilesN;
                if constexpr (kTiles && uj == 0) sa[ui] *= h.tile.rest;
                const f32x4 v = d[(t - kLag) % (kLag + 1)];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[ui][uj][e] = fmaf(kTiles ? v[e] : v[e] * sb[uj][e], sa[ui], acc[ui][uj][e]);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
        // the sums are due here: without this the compiler moves the work above into later
        // branches and keeps the fragments alive for it
#pragma unroll
        for (int i = 0; i < kTilesM; ++i)
#pragma unroll
            for (int j = 0; j < kTilesN; ++j) asm volatile("" : "+v"(acc[i][j]));
    }

    // The sums leave a tile row (16 m) at a time through a part of LDS of the wavefront's
    // own, from four neighbours a lane to whole rows: 16 bytes a lane where the output's
    // rows allow it, else one element a lane.  Nobody reads LDS after the last meeting.
    template <typename Out>
    __device__ __forceinline__ void store(Stage<S> &room, Out *out, bool accumulate) {
        constexpr bool kFloat = std::is_same_v<Out, float>;
        constexpr int kPer16 = 16 / (int)sizeof(Out), kCols = S::kWaveN;
        constexpr int kPitch = kCols + kPer16;  // elements; the shift keeps rows off each other's banks
        static_assert(S::kWaves * 16 * kPitch * sizeof(Out) <= sizeof(room.a) + sizeof(room.b), "fits the stage");
        Out *mine = reinterpret_cast<Out *>(room.a) + wave * 16 * kPitch;
        const int n1 = n0 + wn;
        const bool wide = p.N % kPer16 == 0;
#pragma unroll
        for (int i = 0; i < S::kTilesM; ++i) {
            const int m1 = m0 + wm + i * 16;
            if (m1 >= p.M || n1 >= p.N) break;
#pragma unroll
            for (int j = 0; j < S::kTilesN; ++j) {
                Out *to = mine + row16 * kPitch + j * 16 + 4 * quarter;
                if constexpr (kFloat) {
                    *reinterpret_cast<f32x4 *>(to) = acc[i][j];
                } else {
                    u32x2 w;
                    w[0] = fp4q_num::bf16_rne_pair(acc[i][j][0], acc[i][j][1]);
                    w[1] = fp4q_num::bf16_rne_pair(acc[i][j][2], acc[i][j][3]);
                    *reinterpret_cast<u32x2 *>(to) = w;
                }
            }
            if (wide) {
                constexpr int kLanes = kCols / kPer16, kRows = kWave / kLanes;
#pragma unroll
                for (int k = 0; k < 16 / kRows; ++k) {
                    const int r = k * kRows + lane / kLanes, c = lane % kLanes * kPer16;
                    if (m1 + r < p.M && n1 + c < p.N) {
                        u32x4 w = *reinterpret_cast<const u32x4 *>(mine + r * kPitch + c);
                        u32x4 *to = reinterpret_cast<u32x4 *>(out + (int64_t)(m1 + r) * p.N + n1 + c);
                        if (kFloat && accumulate) {
                            const u32x4 had = *to;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = __float_as_uint(__uint_as_float(had[e]) + __uint_as_float(w[e]));
                        }
                        *to = w;
                    }
                }
            } else {
                constexpr int kRows = kWave / kCols;
                const int c = lane % kCols;
                for (int r = lane / kCols; r < 16 && m1 + r < p.M; r += kRows)
                    if (n1 + c < p.N) {
                        Out *to = out + (int64_t)(m1 + r) * p.N + n1 + c;
                        Out v = mine[r * kPitch + c];
                        if constexpr (kFloat)
                            if (accumulate) v = *to + v;
                        *to = v;
                    }
            }
        }
    }
};

// Two blocks in LDS: one is multiplied while the next one's loads are under way.
// Over cards, 8192 x 11008, K = 4096, E4M3 to bf16 takes 361 to 378 us (2046 to 1954
// TFLOP/s), 8192 x 8192 x 8192 480 to 507 (2290 to 2169), 2047 x 4096, K = 11008 92 to 97
// (2007 to 1903) and 11008 x 4096, K = 4001, rows of 128, fp32 output 375 to 400 (962 to
// 902).  The matrix cores are busy for 42 to 44 % of the cycles.  Of the first one's 371 us
// on one card a copy of the loop takes 280 without its loads, 321 without its LDS reads, 321
// without the scaled additions and 242 without loads and reads; of the last one's 400 us
// 290, 342, 330 and 273.  So no one part sets the time: they overlap in part, loads least
// of all, with one block under way.  256 x 256 tiles with rows of b's scales spill one
// register.
template <typename S, int kFmtA, int kFmtB, bool kTiles, bool kPrecise>
__global__ __launch_bounds__(S::kThreads, 2) void gemm_kernel(GemmArgs p) {
    __shared__ Stage<S> even;
    __shared__ Stage<S> odd;
    // consecutive workgroups go to the 8 XCDs in turn: each XCD takes a run of tiles,
    // and a run walks 8 tiles of m before it steps in n, so that the tiles that an XCD
    // works on at one time share their operands in its L2
    const int tiles = p.tiles_m * p.tiles_n;
    const int count = tiles * p.parts, each = count / 8, more = count % 8;
    const int xcd = (int)blockIdx.x % 8, turn = (int)blockIdx.x / 8;
    const int index = xcd * each + min(xcd, more) + turn;
    const int part = __builtin_amdgcn_readfirstlane(index / tiles), at = index - part * tiles;
    const int band = at / (8 * p.tiles_n), in_band = at - band * 8 * p.tiles_n;
    const int high = min(8, p.tiles_m - band * 8);
    // (the divisions leave uniform values in vector registers; descriptors need scalars)
    const int tm = __builtin_amdgcn_readfirstlane(band * 8 + in_band % high);
    const int tn = __builtin_amdgcn_readfirstlane(in_band / high);
    Tile<S, kFmtA, kFmtB, kTiles, kPrecise> t(p, tm, tn);
    const int blocks = (p.K + kGroup - 1) / kGroup;
    int kb = __builtin_amdgcn_readfirstlane((int)((int64_t)blocks * part / p.parts));
    const int end = __builtin_amdgcn_readfirstlane((int)((int64_t)blocks * (part + 1) / p.parts));
    const bool ragged = end == blocks && p.K % kGroup;
    if (kb < end) {
        typename decltype(t)::Head h0, h1;
        t.fetch(even, kb);
        if (kb + 1 < end) {
            t.fetch(odd, kb + 1);
            meet<t.kFetched>();
        } else {
            meet<0>();
            if (ragged) {
                t.clear_tail(even);
                __syncthreads();
            }
        }
        static_for<t.kHeadB + 1>([&](auto i) FP4Q_INLINE { t.read_head(even, h0, i.value); });
        if constexpr (kTiles) h0.tile.set(h0.sb);
        for (; kb + 1 < end; kb += 2) {
            t.step(even, odd, h0, h1, kb, end, ragged);
            t.step(odd, even, h1, h0, kb + 1, end, ragged);
        }
        if (kb < end) t.step(even, odd, h0, h1, kb, end, ragged);
    }
    if (p.parts > 1)
        t.store(even, p.partial + part * p.part_size, false);
    else if constexpr (kPrecise)
        t.store(even, static_cast<float *>(p.out), p.accumulate);
    else
        t.store(even, static_cast<bf16 *>(p.out), false);
}

// Adds the runs' sums in their order, four neighbours a thread: 48 x 11008 in 4 runs 4 us
// (8.5 MB read), 4096 x 4096 in 2 runs 29 us with fp32 and 25 with bf16 output (134 MB read,
// 67 or 34 written: 6.9 and 6.8 TB/s, out of the last-level cache in part).
constexpr int kJoinThreads = 256;
template <typename Out>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const float *partial, int64_t part_size, int parts,
                                                            int64_t count, Out *out, int accumulate) {
    const int64_t at = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x) * 4;
    if (at >= count) return;
    f32x4 sum = *reinterpret_cast<const f32x4 *>(partial + at);
    for (int s = 1; s < parts; ++s) sum += *reinterpret_cast<const f32x4 *>(partial + s * part_size + at);
    if (at + 4 <= count) {
        if constexpr (std::is_same_v<Out, float>) {
            f32x4 *to = reinterpret_cast<f32x4 *>(out + at);
            *to = accumulate ? *to + sum : sum;
        } else {
            u32x2 w;
            w[0] = fp4q_num::bf16_rne_pair(sum[0], sum[1]);
            w[1] = fp4q_num::bf16_rne_pair(sum[2], sum[3]);
            *reinterpret_cast<u32x2 *>(out + at) = w;
        }
    } else {
        for (int e = 0; at + e < count; ++e) {
            if constexpr (std::is_same_v<Out, float>)
                out[at + e] = accumulate ? out[at + e] + sum[e] : sum[e];
            else
                out[at + e] = from_float<bf16>(sum[e]);
        }
    }
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

// Up to 16 rows of a: the time is that of reading b once.  A workgroup takes 16 rows of
// b; its wavefronts share K, each taking every kStripWaves-th block, whole fragments straight
// from memory into registers, kAhead blocks' loads at a time.  A load takes 64 neighbouring
// bytes of each of 16 rows (with a lane's 32 bytes side by side, 16 bytes at every 32, it
// took a tenth longer).  The parts of the sum are joined through LDS in the wavefronts'
// order.  4096 x 11008 codes that come from HBM take 12.2 us with one row of a (3.7 TB/s; 9.5
// out of the last-level cache), 14.5 with 16 rows; 32768 x 4096 33 us (4.1 TB/s, with two
// workgroups on a CU: at most 64 registers; 37 us with one).
constexpr int kStripWaves = 16, kAhead = 4, kStripThreads = kStripWaves * kWave;
template <int kFmtA, int kFmtB, bool kTiles, bool kPrecise>
__global__ __launch_bounds__(kStripThreads, kTiles && !kPrecise ? 8 : 4) void strip_kernel(GemmArgs p) {
    __shared__ f32x4 part[kStripWaves][kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int row16 = lane & 15, quarter = lane >> 4;
    const int n0 = (int)blockIdx.x * kStrip;  // within one of b's tiles of scales
    const int blocks = (p.K + kGroup - 1) / kGroup, whole = p.K / kGroup;
    const int cols = kTiles ? (p.N + kGroup - 1) / kGroup : p.N;
    // rows past the end repeat the last one
    const int m = min(row16, p.M - 1);
    const uint8_t *a = p.a, *b = p.b + n0 * p.b_pitch;
    const unsigned row_a = m * (unsigned)p.a_pitch, row_b = (min(n0 + row16, p.N - 1) - n0) * (unsigned)p.b_pitch;
    f32x4 acc = {0, 0, 0, 0};

    // kCount blocks from kb0, kStripWaves apart; kWhole: all their codes lie before K
    auto run = [&](int kb0, auto count_of, auto whole_of) FP4Q_INLINE {
        constexpr int kCount = count_of.value;
        constexpr bool kWhole = whole_of.value;
        Raw ra[kCount], rb[kCount];
        float sa[kCount];
        f32x4 sb[kCount];
#pragma unroll
        for (int u = 0; u < kCount; ++u) {
            const int kb = kb0 + u * kStripWaves, low = kb * kGroup + 16 * quarter;
            if constexpr (kWhole) {
                rb[u] = {*reinterpret_cast<const u32x4 *>(b + (row_b + low)),
                         *reinterpret_cast<const u32x4 *>(b + (row_b + low) + 64)};
                ra[u] = {*reinterpret_cast<const u32x4 *>(a + (row_a + low)),
                         *reinterpret_cast<const u32x4 *>(a + (row_a + low) + 64)};
            } else {
                rb[u] = {load_chunk(b + row_b, low, p.K), load_chunk(b + row_b, low + 64, p.K)};
                ra[u] = {load_chunk(a + row_a, low, p.K), load_chunk(a + row_a, low + 64, p.K)};
            }
            sa[u] = p.sa[(int64_t)kb * p.M + m];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sb[u][e] = p.sb[(int64_t)kb * cols + (kTiles ? n0 / kGroup : min(n0 + 4 * quarter + e, p.N - 1))];
        }
#pragma unroll
        for (int u = 0; u < kCount; ++u) {
            Frag<kFmtB, kPrecise> first;
            Frag<kFmtA, kPrecise> second;
            first.set(rb[u]);
            second.set(ra[u]);
            const f32x4 d = block_product<false>(first, second, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = fmaf(d[e] * sb[u][e], sa[u], acc[e]);
        }
    };
    int kb = wave;
    for (; kb + (kAhead - 1) * kStripWaves < whole; kb += kAhead * kStripWaves)
        run(kb, std::integral_constant<int, kAhead>{}, std::true_type{});
    // what is left in a second and a third batch at most
    for (; kb + kStripWaves < whole; kb += 2 * kStripWaves) run(kb, std::integral_constant<int, 2>{}, std::true_type{});
    for (; kb < whole; kb += kStripWaves) run(kb, std::integral_constant<int, 1>{}, std::true_type{});
    for (; kb < blocks; kb += kStripWaves) run(kb, std::integral_constant<int, 1>{}, std::false_type{});

    part[wave][lane] = acc;
    __syncthreads();
    if (wave > 0 || row16 >= p.M) return;
#pragma unroll 5
    for (int w = 1; w < kStripWaves; ++w) acc += part[w][lane];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int n = n0 + 4 * quarter + e;
        if (n >= p.N) break;
        const int64_t at = (int64_t)row16 * p.N + n;
        if constexpr (kPrecise) {
            float *to = static_cast<float *>(p.out) + at;
            *to = p.accumulate ? *to + acc[e] : acc[e];
        } else {
            static_cast<bf16 *>(p.out)[at] = from_float<bf16>(acc[e]);
        }
    }
}

using Large = Shape<2, 4, 8, 4>;         // 256 x 256, a workgroup a CU
using LargePrecise = Shape<2, 4, 4, 4>;  // 128 x 256
using Medium = Shape<2, 2, 4, 4>;        // 128 x 128, two workgroups a CU
using Low64 = Shape<2, 2, 2, 4>;         // 64 x 128
using Low32 = Shape<1, 4, 2, 2>;         // 32 x 128
struct Strip {
    static constexpr int kThreads = kStripThreads;
};

template <typename S, int kFmtA, int kFmtB, bool kTiles, bool kPrecise>
struct Kernel {
    static const void *get() { return (const void *)&gemm_kernel<S, kFmtA, kFmtB, kTiles, kPrecise>; }
};
template <int kFmtA, int kFmtB, bool kTiles, bool kPrecise>
struct Kernel<Strip, kFmtA, kFmtB, kTiles, kPrecise> {
    static const void *get() { return (const void *)&strip_kernel<kFmtA, kFmtB, kTiles, kPrecise>; }
};
template <typename S, bool kPrecise, int kFmtA, int kFmtB>
const void *pick(bool tiles) {
    return tiles ? Kernel<S, kFmtA, kFmtB, true, kPrecise>::get() : Kernel<S, kFmtA, kFmtB, false, kPrecise>::get();
}
template <typename S, bool kPrecise>
const void *pick(int fa, int fb, bool tiles) {
    if (fa == FP4Q_E4M3)
        return fb == FP4Q_E4M3 ? pick<S, kPrecise, FP4Q_E4M3, FP4Q_E4M3>(tiles)
                               : pick<S, kPrecise, FP4Q_E4M3, FP4Q_E5M2>(tiles);
    return fb == FP4Q_E4M3 ? pick<S, kPrecise, FP4Q_E5M2, FP4Q_E4M3>(tiles)
                           : pick<S, kPrecise, FP4Q_E5M2, FP4Q_E5M2>(tiles);
}

bool bad_gemm(int64_t M, int64_t N, int64_t K) {
    return M < 0 || N < 0 || K < 0 || M >= kDimLimit || N >= kDimLimit || K >= kDimLimit ||
           ceil_div(M, 32) * ceil_div(N, 128) > (int64_t)0x7FFFFFFF / 16;
}

// What a product's sizes, output type and flags are refused for.
int check_gemm(int64_t M, int64_t N, int64_t K, int out_dtype, uint32_t flags) {
    if (bad_gemm(M, N, K)) return FP4Q_ERR_SHAPE;
    if (flags & ~(uint32_t)(FP4Q_FLAG_TILES | FP4Q_FLAG_ACCUMULATE)) return FP4Q_ERR_ARG;
    if (out_dtype == FP4Q_OUT_F32) return FP4Q_OK;
    return out_dtype == FP4Q_OUT_BF16 && !(flags & FP4Q_FLAG_ACCUMULATE) ? FP4Q_OK : FP4Q_ERR_ARG;
}

}  // namespace

extern "C" {

int fp4q_gemm8_workspace(int64_t M, int64_t N, int64_t K, int out_dtype, uint32_t flags, size_t *bytes) {
    const int st = check_gemm(M, N, K, out_dtype, flags);
    if (st != FP4Q_OK) return st;
    if (!bytes) return FP4Q_ERR_NULL;
    *bytes = M && N ? plan_of(M, N, K, out_dtype == FP4Q_OUT_F32).workspace : 0;
    return FP4Q_OK;
}

int fp4q_gemm8(const uint8_t *a, int64_t a_pitch, int a_format, const float *a_scales,
               const uint8_t *b, int64_t b_pitch, int b_format, const float *b_scales, int64_t M,
               int64_t N, int64_t K, void *out, int out_dtype, uint32_t flags, void *workspace,
               size_t workspace_bytes, void *stream) {
    if (!bad_gemm(M, N, K) && K > 0 &&
        (a_pitch < K || b_pitch < K || a_pitch >= (1 << 23) || b_pitch >= (1 << 23)))
        return FP4Q_ERR_SHAPE;
    const int st = check_gemm(M, N, K, out_dtype, flags);
    if (st != FP4Q_OK) return st;
    const bool add = flags & FP4Q_FLAG_ACCUMULATE, tiles = flags & FP4Q_FLAG_TILES;
    if ((a_format != FP4Q_E4M3 && a_format != FP4Q_E5M2) || (b_format != FP4Q_E4M3 && b_format != FP4Q_E5M2))
        return FP4Q_ERR_ARG;
    if (M == 0 || N == 0) return FP4Q_OK;
    const bool precise = out_dtype == FP4Q_OUT_F32;
    const Plan plan = plan_of(M, N, K, precise);
    const size_t need = plan.workspace;
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
                  (int)ceil_div(M, plan.tile_m), (int)ceil_div(N, plan.tile_n), add,
                  plan.parts, plan.part_size, static_cast<float *>(workspace)};
    void *args[] = {&p};
    const void *fn = nullptr;
    int threads = 0;
    auto use = [&](auto fast, auto exact) {
        using Fast = decltype(fast);
        using Exact = decltype(exact);
        static_assert(Fast::kThreads == Exact::kThreads, "one launch for both");
        fn = precise ? pick<Exact, true>(a_format, b_format, tiles) : pick<Fast, false>(a_format, b_format, tiles);
        threads = Fast::kThreads;
    };
    switch (plan.way) {
        case Way::kStrip: use(Strip{}, Strip{}); break;
        case Way::kLow32: use(Low32{}, Low32{}); break;
        case Way::kLow64: use(Low64{}, Low64{}); break;
        case Way::kMedium: use(Medium{}, Medium{}); break;
        case Way::kLarge: use(Large{}, LargePrecise{}); break;
    }
    const int done = launch(fn, dim3((unsigned)(p.tiles_m * p.tiles_n * p.parts)), threads, args, stream);
    if (plan.parts == 1 || done != FP4Q_OK) return done;
    int64_t count = M * N;
    void *join_args[] = {&p.partial, &p.part_size, &p.parts, &count, &out, &p.accumulate};
    return launch(precise ? (const void *)&join_kernel<float> : (const void *)&join_kernel<bf16>,
                  dim3((unsigned)ceil_div(count, 4 * kJoinThreads)), kJoinThreads, join_args, stream);
}

}  // extern "C"
