// fp4q_gemv4_plan.hip -- test library: the choice of kernel that fp4q_gemv4 and fp4q_gated4 make.
#include "fp4q_gemv4_plan.h"

// out: the way, wavefronts, rows of x of a chunk, chunks, units that a workgroup takes at most,
// bytes of LDS.
extern "C" void fp4q_gemv4_plan(int64_t M, int64_t N, int64_t K, int x_f32, int out_f32, int transformed, int gated,
                                int64_t *out) {
    const uint32_t flags = transformed ? 0 : FP4Q_FLAG_NO_FWHT;
    const int parts = fp4q_few_plan::parts_of(x_f32 ? FP4Q_OUT_F32 : FP4Q_OUT_BF16,
                                                out_f32 ? FP4Q_OUT_F32 : FP4Q_OUT_BF16, flags);
    const fp4q_few_plan::Plan plan = fp4q_few_plan::plan_of(M, N, K, parts, flags, gated != 0);
    out[0] = (int)plan.way;
    out[1] = plan.waves;
    out[2] = plan.each;
    out[3] = plan.chunks;
    out[4] = fp4q_f8::ceil_div(fp4q_f8::ceil_div(N, plan.unit), plan.groups);
    out[5] = plan.lds;
}
