// Calls every entry point of fp4q_linear.h with arguments that its validation rejects (or
// that ask for nothing), over many sizes, so that no kernel is launched: the host code's
// arithmetic on sizes, pitches and addresses runs under the sanitizers.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "fp4q_linear.h"

static int failures = 0;
static void expect(int got, int want, const char *what) {
    if (got != want) {
        std::printf("%s: status %d, expected %d\n", what, got, want);
        ++failures;
    }
}

int main() {
    const int64_t far = (int64_t)1 << 40;
    auto at = [&](int i) { return reinterpret_cast<uint8_t *>(far * i); };
    auto fl = [&](int i) { return reinterpret_cast<float *>(far * i); };
    const int64_t dims[] = {INT64_MIN, -1, 0, 1, 7, 16, 17, 64, 127, 128, 129, 1000, 4096, 16384, 65536, 65537,
                            ((int64_t)1 << 27) + 5, ((int64_t)1 << 28) - 1, (int64_t)1 << 28, (int64_t)1 << 40, INT64_MAX};
    for (int64_t rows : dims)
        for (int64_t cols : dims) {
            size_t bytes = 0;
            const bool bad = rows < 0 || cols <= 0 || rows >= ((int64_t)1 << 28) || cols >= ((int64_t)1 << 28);
            expect(fp4q_rmsnorm_backward_workspace(rows, cols, &bytes), bad ? FP4Q_ERR_SHAPE : FP4Q_OK, "workspace");
            const int64_t pitch = bad ? 16 : (cols + 15) / 16 * 16, pitch_t = bad ? 16 : (rows + 15) / 16 * 16 + 16;
            const int none = bad ? FP4Q_ERR_SHAPE : rows == 0 ? FP4Q_OK : FP4Q_ERR_NULL;
            expect(fp4q_rmsnorm(nullptr, at(2), at(3), 1e-6f, rows, cols, 0, at(4), at(5), at(6), pitch, fl(7), fl(8), nullptr),
                   none, "rmsnorm without input");
            expect(fp4q_rmsnorm(at(1), at(2), at(3), 1e-6f, rows, cols, 1, at(4), at(1), at(6), pitch, fl(7), fl(8), nullptr),
                   bad ? FP4Q_ERR_SHAPE : rows == 0 ? FP4Q_OK : FP4Q_ERR_ARG, "rmsnorm over its input");
            expect(fp4q_rmsnorm_backward(at(1), at(2), at(3), fl(4), at(5), rows, cols, 1, at(6), nullptr, at(8), bytes, nullptr),
                   bad ? FP4Q_ERR_SHAPE : FP4Q_ERR_NULL, "backward without dweight");
            if (bad || rows > 0)
                expect(fp4q_rmsnorm_backward(at(1), at(2), at(3), fl(4), at(5), rows, cols, 1, at(6), fl(7), at(8),
                                             bytes ? bytes - 1 : 0, nullptr),
                       FP4Q_ERR_SHAPE, "backward with a short workspace");
            const bool vast = !bad && ((rows + 127) / 128) * ((cols + 127) / 128) > 0x7FFFFFFF;
            expect(fp4q_quantize8(nullptr, rows, cols, 1, 1, at(2), pitch, fl(3), at(4), pitch_t, fl(5), 0, nullptr),
                   vast ? FP4Q_ERR_SHAPE : none, "quantize without input");
            expect(fp4q_quantize8(at(1), rows, cols, 0, 0, at(2), pitch, fl(3), at(1), pitch_t, fl(5), FP4Q_FLAG_TILES, nullptr),
                   bad || vast ? FP4Q_ERR_SHAPE : rows == 0 ? FP4Q_OK : FP4Q_ERR_ARG, "quantize over its input");
            for (int64_t k : {(int64_t)0, (int64_t)1, (int64_t)4096, (int64_t)8000000, (int64_t)1 << 28})
                for (int type : {0, 1}) {
                    const int st = fp4q_gemm8_workspace(rows, cols, k, type, FP4Q_FLAG_TILES, &bytes);
                    if (rows < 0 || cols < 0 || rows >= ((int64_t)1 << 28) || cols >= ((int64_t)1 << 28) || k >= ((int64_t)1 << 28))
                        expect(st, FP4Q_ERR_SHAPE, "gemm workspace");
                    if (st != FP4Q_OK) continue;
                    const int64_t wide = (k + 15) / 16 * 16;
                    if (wide >= (1 << 23)) continue;
                    expect(fp4q_gemm8(at(1), wide, 0, fl(2), at(3), wide, 1, fl(4), rows, cols, k, nullptr, type,
                                      FP4Q_FLAG_TILES, at(6), bytes, nullptr),
                           rows && cols ? FP4Q_ERR_NULL : FP4Q_OK, "gemm without output");
                    if (rows && cols && k)
                        expect(fp4q_gemm8(at(1), wide, 0, fl(2), at(3), wide, 1, fl(4), rows, cols, k, at(3), type,
                                          FP4Q_FLAG_TILES, at(6), bytes, nullptr), FP4Q_ERR_ARG, "gemm over its operand");
                }
        }
    if (failures) return 1;
    std::printf("linear driver ok\n");
    return 0;
}
