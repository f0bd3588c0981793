// plan_driver.cpp -- prints how the launches over row tiles split their work
// (csrc/row_plan.h, built for the host alone).  One launch per input line:
//   mx CUS PAIR K N M [M ...]         the MXFP4 GEMV, its batch, or a gate / up pair
//   moe CUS TYPE E k N F K            the experts' gate and up products
// and one line of "name=value" fields per launch.  Exits 1, naming the launch,
// where a plan breaks a rule that the kernels rely on.
#include "../../quantized_matmul_ggml_amd/csrc/row_plan.h"

#include <stdio.h>
#include <string.h>

static int g_cus = 256;

namespace qmm {
int device_cus() { return g_cus; }
}  // namespace qmm

using namespace qmm;

static int bad(const char *line, const char *rule)
{
    fprintf(stderr, "%s: %s\n", line, rule);
    return 1;
}

// What both kernels need of a plan: the image holds `pass` steps of `tokens`
// tokens, a pass is all steps or whole rounds of the waves that share a tile.
static const char *check(const RowPlan &p, int64_t units, int pass, int tokens, int lds)
{
    const int S = 1 << p.s_log2;
    if (p.waves != 4 && p.waves != 8 && p.waves != 16) return "waves";
    if (p.s_log2 < 0 || S > p.waves) return "waves of a tile";
    if (p.steps != (units + p.half) / (1 + p.half)) return "steps";
    if (pass < 1) return "a pass without steps";
    if (pass < p.steps && pass % S != 0) return "a pass that is no multiple of the waves";
    if ((int64_t)(pass < p.steps ? pass : p.steps) * p.step_bytes * tokens > p.image) return "image";
    if (lds > kLdsMost) return "LDS";
    return nullptr;
}

int main()
{
    char line[1024];
    while (fgets(line, sizeof line, stdin)) {
        line[strcspn(line, "\n")] = 0;
        int at = 0, pair;
        long long K, N, E, k, F, type;
        if (sscanf(line, "mx %d %d %lld %lld%n", &g_cus, &pair, &K, &N, &at) == 4) {
            int64_t M[QMM_GEMV_BATCH_MAX], full = 0, half = 0;
            int count = 0, more = 0;
            for (long long v; count < QMM_GEMV_BATCH_MAX && sscanf(line + at, "%lld%n", &v, &more) == 1; at += more) M[count++] = v;
            const MxPlan m = plan_mx(M, count, K, N, pair != 0);
            const RowPlan &p = m.rows;
            for (int i = 0; i < count; ++i) {
                full += (M[i] + 15) / 16;
                half += (M[i] + 7) / 8;
            }
            if (const char *rule = check(p, (K + 127) / 128, m.pass, (int)m.N, m.lds)) return bad(line, rule);
            if (m.parts * count > QMM_GEMV_BATCH_MAX || m.N * m.parts < N || m.N * (m.parts - 1) >= N) return bad(line, "parts");
            if (m.tg != (m.N > 4 ? 2 : 1) || (p.half && (m.tg > 1 || pair))) return bad(line, "token groups");
            if (m.tile_rows * m.T < 8 || m.T < 1 || m.groups < count) return bad(line, "tiles");
            const RowPlan first = plan_rows((K + 127) / 128, 4, m.parts * (pair ? half : full), pair ? 0 : m.parts * half, (int)m.N, (int)m.N);
            const bool few = 2 * (pair ? half : full) <= g_cus;
            printf("tg=%d pair=%d half=%d depth=%d passes=%d loops=%d halved=%s more=%d waves=%d S=%d\n", m.tg, pair, p.half, m.depth,
                   m.pass < p.steps ? 1 : 0, m.groups > m.cap ? 1 : 0, m.parts == 1 ? "no" : few ? "few" : "fits",
                   p.s_log2 - first.s_log2, p.waves, 1 << p.s_log2);
        } else if (sscanf(line, "moe %d %lld %lld %lld %lld %lld %lld", &g_cus, &type, &E, &k, &N, &F, &K) == 7) {
            const int mf = type == W_Q8_0 ? 2 : 4;
            const int64_t units = (K + 32 * mf - 1) / (32 * mf);
            const RowPlan p = plan_moe(E, k, N, F, units, mf);
            int passes = 0;
            for (int now = 1; now <= (N * k < 2 ? 1 : 2); ++now) {
                const int pass = pass_steps(p.image, mf * kImageBytes, now, p.s_log2, p.steps);
                if (const char *rule = check(p, units, pass, now, moe_lds(p))) return bad(line, rule);
                if (pass < p.steps) passes = 1;
            }
            if (p.half) return bad(line, "half tiles");
            printf("type=%lld depth=%d passes=%d waves=%d S=%d\n", type, moe_depth((p.steps + (1 << p.s_log2) - 1) >> p.s_log2), passes,
                   p.waves, 1 << p.s_log2);
        } else {
            return bad(line, "not a launch");
        }
    }
    return 0;
}
