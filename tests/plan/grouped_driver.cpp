// grouped_driver.cpp -- prints how grouped products and adapters split their work
// (csrc/qmm_internal.h, csrc/lora_plan.h, built for the host alone).  One launch
// per input line:
//   grouped CUS TYPE PAIR M K R E     TYPE: 0 MXFP4, 1 Q4_0, 2 Q8_0
//   lora CUS N K M RANK WIDE          WIDE: aligned rows of x
// and one line of "name=value" fields per launch.  Exits 1, naming the launch,
// where a plan breaks a rule that the kernels rely on.
#include "../../quantized_matmul_ggml_amd/csrc/lora_plan.h"

#include <stdio.h>

using namespace qmm;

static int bad(const char *line, const char *rule)
{
    fprintf(stderr, "%s: %s\n", line, rule);
    return 1;
}

static const char *check(const LoraPlan &p, int64_t N, int64_t K, int64_t M, int64_t r, bool wide)
{
    auto power = [](int64_t v, int64_t most) { return v >= 1 && v <= most && (v & (v - 1)) == 0; };
    if (!power(p.rt, 8) || 16 * p.rt < r || (p.rt > 1 && 8 * p.rt >= r)) return "rank tiles";
    if (p.single) {
        if (N > 65535) return "tokens of one launch";
        return p.mt >= 1 && (int64_t)(p.mt - 1) * 512 < M ? nullptr : "outputs of one launch";
    }
    if (p.tiled && !wide) return "tiles of unaligned rows";
    if (K == 0) {
        if (p.chunks != 0 || p.blocks1 != 0) return "parts of nothing";
    } else {
        if (p.chunks < 1 || p.chunks > kMostParts || p.chunk % 64 != 0) return "parts";
        if ((int64_t)p.chunk * p.chunks < K || (int64_t)p.chunk * (p.chunks - 1) >= K) return "parts of K";
    }
    const int64_t tile1 = p.tiled ? 32 : 16;
    if (!power(p.j1, tile1) || !power(p.j2, 32) || !power(p.mt, 8)) return "workgroups of a tile";
    if (p.blocks1 != (N + tile1 - 1) / tile1 * p.chunks * p.j1) return "workgroups of the first launch";
    if (p.m_blocks * p.mt * 128 < M || (p.m_blocks - 1) * p.mt * 128 >= M) return "outputs";
    if (p.blocks2 != (N + 31) / 32 * p.m_blocks * p.j2) return "workgroups of the second launch";
    return nullptr;
}

int main()
{
    char line[256];
    while (fgets(line, sizeof line, stdin)) {
        long long cus, type, pair, M, K, R, E, N, r, wide;
        if (sscanf(line, "grouped %lld %lld %lld %lld %lld %lld %lld", &cus, &type, &pair, &M, &K, &R, &E) == 7) {
            const int w = type == 0 ? W_MXFP4 : type == 1 ? W_Q4_0 : W_Q8_0;
            const GroupedForm form = grouped_form(M, K, R, E, w, pair, cus);
            const int kp = form.kp;
            const RowsPlan p = plan_grouped_rows(M, K, R, E, w, pair, cus);
            if (kp != 0 && kp != 1 && kp != 2 && kp != 4) return bad(line, "form");
            const int64_t tile = pair ? 8 : 16, rows = 8 * p.tiles_per_wave * tile;
            if (p.m_tiles * rows < M || (p.m_tiles - 1) * rows >= M) return bad(line, "weight rows");
            if (p.depth != 4 && p.depth != 8) return bad(line, "depth");
            // several tiles one after the other keep one image
            if (p.tiles_per_wave != 1 && K > 2048) return bad(line, "tiles over passes");
            // the most tiles that groups can need: all but one of a row, one with the rest; and even groups
            const int bn = kp ? 128 / kp : 16;
            const int64_t used = E < R ? E : R, lone = (R - (used - 1) + bn - 1) / bn + used - 1;
            if (grouped_row_tiles(R, E, bn) < lone || grouped_row_tiles(R, E, bn) < R / bn) return bad(line, "row tiles");
            const bool fits = grouped_fits(M, K, R, E, w, pair, cus);
            const int64_t bm = kp ? (pair ? 64 : 128) / kp : 0, m = kp ? (M + bm - 1) / bm : p.m_tiles;
            if (fits && (double)m * (double)grouped_row_tiles(R, E, bn) * (kp ? 256 : 512) >= 4294967296.0) return bad(line, "threads");
            printf("form=%d%s depth=%d tiles=%d passes=%d fits=%d\n", kp, form.deep ? "deep" : "", p.depth, p.tiles_per_wave, K > 2048, fits);
        } else if (sscanf(line, "lora %lld %lld %lld %lld %lld %lld", &cus, &N, &K, &M, &r, &wide) == 6) {
            const LoraPlan p = plan_lora(N, K, M, r, wide, cus);
            if (const char *rule = check(p, N, K, M, r, wide)) return bad(line, rule);
            printf("single=%d rt=%d tiled=%d chunks=%d j1=%d j2=%d mt=%d\n", p.single, p.rt, p.tiled, p.chunks, p.j1, p.j2, p.mt);
        } else {
            return bad(line, "not a launch");
        }
    }
    return 0;
}
