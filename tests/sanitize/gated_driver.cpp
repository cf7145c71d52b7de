// Calls every entry point of fp4q_gated.h with arguments that its validation rejects (or that
// ask for nothing), over many sizes, so that no kernel is launched: the host code's arithmetic
// on sizes, pitches and addresses runs under the sanitizers.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "fp4q_gated.h"

static int failures = 0;
static void expect(int got, int want, const char *what) {
    if (got != want) {
        std::printf("%s: status %d, expected %d\n", what, got, want);
        ++failures;
    }
}

int main() {
    const int64_t far = (int64_t)1 << 58, limit = (int64_t)1 << 27;
    auto at = [&](int i) { return reinterpret_cast<uint8_t *>(far * i); };
    auto fl = [&](int i) { return reinterpret_cast<float *>(far * i); };
    const int64_t dims[] = {INT64_MIN, -1, 0, 1, 7, 16, 17, 64, 65, 127, 128, 129, 1000, 4096, 16384, 65537,
                            limit - 1, limit, (int64_t)1 << 40, INT64_MAX};
    for (int64_t m : dims)
        for (int64_t n : dims) {
            const bool bad = m < 0 || n < 0 || m >= limit || n >= limit;
            size_t bytes = 0;
            for (int64_t k : {(int64_t)0, (int64_t)1, (int64_t)256, (int64_t)4096, (int64_t)8388352, limit}) {
                const int st = fp4q_gated8_workspace(m, n, k, &bytes);
                if (bad || k >= limit) expect(st, FP4Q_ERR_SHAPE, "gated8 workspace");
                const int64_t wide = (k + 15) / 16 * 16;
                if (st != FP4Q_OK || wide >= (1 << 23)) continue;
                expect(fp4q_gated8(at(1), wide, 0, fl(2), at(3), wide, 1, fl(4), m, n, k, 0, nullptr, at(6), at(7), at(8), bytes, nullptr),
                       m && n ? FP4Q_ERR_NULL : FP4Q_OK, "gated8 without output");
                if (m && n && k)
                    expect(fp4q_gated8(at(1), wide, 0, fl(2), at(3), wide, 1, fl(4), m, n, k, 3, at(3), at(6), at(7), at(8), bytes, nullptr),
                           FP4Q_ERR_ARG, "gated8 over its operand");
            }
            const bool none = n == 0, vast = !bad && (m >= (1 << 23) || n >= (1 << 23));
            const int64_t pitch = bad ? 16 : ((n + 127) / 128 * 128 + n + 15) / 16 * 16, high = bad ? 16 : (m + 15) / 16 * 16 + 16;
            expect(fp4q_gated8_backward(nullptr, at(2), at(3), m, n, 1, 1, 1, at(4), pitch, fl(5), at(6), high, fl(7), at(8), high,
                                        fl(9), nullptr),
                   bad || none || vast ? FP4Q_ERR_SHAPE : m == 0 ? FP4Q_OK : FP4Q_ERR_NULL, "backward without input");
            expect(fp4q_gated8_backward(at(1), at(2), at(3), m, n, 0, 2, 0, at(4), pitch, fl(5), at(1), high, fl(7), at(8), high,
                                        fl(9), nullptr),
                   bad || none || vast ? FP4Q_ERR_SHAPE : m == 0 ? FP4Q_OK : FP4Q_ERR_ARG, "backward over its input");
            for (int64_t k : {INT64_MIN, (int64_t)0, (int64_t)100, (int64_t)256, (int64_t)4096, ((int64_t)1 << 24) - 256, (int64_t)1 << 24})
                for (int type : {0, 1})
                    for (uint32_t flags : {0u, (uint32_t)FP4Q_FLAG_NO_FWHT}) {
                        const bool wrong = bad || m >= ((int64_t)1 << 19) || k <= 0 || k % 256 || k >= ((int64_t)1 << 24);
                        const int st = fp4q_gemv4_workspace(m, k, type, flags, &bytes);
                        if (!bad) expect(st, wrong ? FP4Q_ERR_SHAPE : FP4Q_OK, "gemv4 workspace");
                        const int empty = m == 0 || n == 0 ? FP4Q_OK : FP4Q_ERR_NULL;
                        expect(fp4q_gemv4(at(1), type, m, nullptr, at(3), fl(4), n, k, at(5), 0, flags, at(6), SIZE_MAX, nullptr),
                               wrong ? FP4Q_ERR_SHAPE : empty, "gemv4 without codes");
                        expect(fp4q_gated4(at(1), type, m, at(2), at(3), fl(4), at(7), at(8), fl(9), n, k, 1, at(7), 1, flags, at(6),
                                           SIZE_MAX, nullptr),
                               wrong ? FP4Q_ERR_SHAPE : m == 0 || n == 0 ? FP4Q_OK : FP4Q_ERR_ARG, "gated4 over its payload");
                    }
        }
    if (failures) return 1;
    std::printf("gated driver ok\n");
    return 0;
}
