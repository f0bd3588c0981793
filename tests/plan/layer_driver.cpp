// layer_driver.cpp -- prints the form of the second product of a layer whose h is held
// in two bf16 parts (csrc/qmm_internal.h, built for the host alone).  One launch per
// input line, TYPE: 0 MXFP4, 1 Q4_0, 2 Q8_0
//   CUS TYPE M F R E
// Exits 1, naming the launch, where the plan breaks a rule that the kernels rely on.
#include "../../quantized_matmul_ggml_amd/csrc/qmm_internal.h"

#include <stdio.h>

using namespace qmm;

int main()
{
    char line[256];
    while (fgets(line, sizeof line, stdin)) {
        long long cus, type, M, F, R, E;
        if (sscanf(line, "%lld %lld %lld %lld %lld %lld", &cus, &type, &M, &F, &R, &E) != 6) return 1;
        const int w = type == 0 ? W_MXFP4 : type == 1 ? W_Q4_0 : W_Q8_0;
        const GroupedForm form = grouped_form(M, F, R, E, w, false, cus, 2);
        const RowsPlan p = plan_grouped_rows(M, F, R, E, w, false, cus, 2);
        const int64_t rows = 8 * p.tiles_per_wave * 16;
        if ((p.tiles_per_wave != 1 && F > 1024) || p.m_tiles * rows < M || (p.m_tiles - 1) * rows >= M) {
            fprintf(stderr, "%s", line);
            return 1;
        }
        printf("%d%s %d %d %d\n", form.kp, form.deep ? "deep" : "", p.depth, p.tiles_per_wave, grouped_fits(M, F, R, E, w, false, cus, 2));
    }
    return 0;
}
