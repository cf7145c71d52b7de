// fp4q_gated8_plan.hip -- test library: the choice of kernel and cuts that fp4q_gated8 makes.
#include "fp4q_gated8_plan.h"

// out: rows and outputs of the kernel's tile, runs that K is cut into.
extern "C" void fp4q_gated8_plan(int64_t M, int64_t N, int64_t K, int *out) {
    const fp4q_gated_plan::Plan plan = fp4q_gated_plan::plan_of(M, N, K);
    out[0] = plan.tile_m;
    out[1] = plan.tile_n;
    out[2] = plan.parts;
}
