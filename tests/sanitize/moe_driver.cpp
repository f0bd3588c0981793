// moe_driver.cpp -- drives the host layer of the mixture-of-experts entry
// points (moe_api.cpp, with its launchers stubbed out here) under
// AddressSanitizer and UndefinedBehaviorSanitizer: a deterministic stream of
// well-formed descriptors, and of the same with one field replaced, over fake
// device addresses that are validated and never read.  Exits 0 when every
// well-formed call reached its launcher, no refused call did, and no sanitizer
// reported anything (a report aborts the process).
#include "../../include/qmm.h"
#include "../../quantized_matmul_ggml_amd/csrc/qmm_internal.h"

#include <stdio.h>

extern int g_launches;

namespace qmm {

hipError_t launch_moe_route(const float *, uint64_t, int64_t, int, int, bool, int32_t *, float *, hipStream_t)
{
    ++g_launches;
    return hipSuccess;
}
uint64_t moe_workspace(int64_t N, int64_t k, int64_t F) { return (uint64_t)(N * k) * (uint64_t)((F + 127) / 128) * 768; }
hipError_t launch_moe_swiglu(const ExpertView &, const ExpertView &, const ExpertView &, const ActView &, const int32_t *,
                             const float *, int, const OutView &, void *, hipStream_t)
{
    ++g_launches;
    return hipSuccess;
}

}  // namespace qmm

namespace {

uint64_t state = 0x2545F4914F6CDD1Dull;
uint64_t next()
{
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return state;
}
template <class T, size_t N> T pick(const T (&v)[N]) { return v[next() % N]; }

qmm_tensor dense(int64_t cols, int64_t rows, uintptr_t at)
{
    qmm_tensor t = {QMM_TYPE_F32, 2, {cols, rows, 1, 1}, {4, (uint64_t)cols * 4, 0, 0}, (void *)at};
    t.nb[2] = t.nb[3] = t.nb[1] * (uint64_t)(rows > 1 ? rows : 1);
    return t;
}
qmm_tensor experts(int32_t type, int64_t K, int64_t M, int64_t E, uintptr_t at)
{
    qmm_tensor t = {type, 3, {K, M, E, 1}, {0, qmm_row_size(type, K), 0, 0}, (void *)at};
    t.nb[2] = t.nb[1] * (uint64_t)(M > 1 ? M : 1);
    t.nb[3] = t.nb[2] * (uint64_t)E;
    return t;
}
// One field of t replaced by a value from the edges of its range.
void spoil(qmm_tensor &t)
{
    static const int64_t sizes[] = {INT64_MIN, -32, -1, 0, 1, 7, 33, 64, 1ll << 28, 1ll << 31, 1ll << 40, INT64_MAX};
    static const uint64_t strides[] = {0, 1, 4, 15, 16, 1ull << 28, 1ull << 29, 1ull << 40, 1ull << 62, UINT64_MAX};
    static const uintptr_t at[] = {0, 1, 0x100000000ull, 0x100000004ull, 0x200000010ull, UINTPTR_MAX - 15, UINTPTR_MAX};
    switch (next() % 5) {
    case 0: t.type = (int32_t)(next() % 12) - 2; break;
    case 1: t.n_dims = (int32_t)(next() % 6); break;
    case 2: t.ne[next() % 4] = pick(sizes); break;
    case 3: t.nb[next() % 4] = pick(strides); break;
    default: t.data = (void *)pick(at); break;
    }
}

struct Call {
    qmm_tensor gate, up, down, x, y, logits;
    int32_t *ids, *route_ids;
    float *weights, *route_weights;
    void *ws;
    uint64_t ws_bytes;
    int32_t k, rule;
    qmm_tensor *null;             // passed as NULL instead, or none
    qmm_tensor *arg(qmm_tensor &t) { return &t == null ? nullptr : &t; }
    int swiglu()
    {
        return qmm_moe_swiglu(arg(gate), arg(up), arg(down), arg(x), ids, weights, k, arg(y), ws, ws_bytes, nullptr);
    }
    int route() { return qmm_moe_route(arg(logits), k, rule, route_ids, route_weights, nullptr); }
};

Call good()
{
    static const int32_t types[] = {QMM_TYPE_Q8_0, QMM_TYPE_Q4_0, QMM_TYPE_Q8_B64, QMM_TYPE_Q4_B64, QMM_TYPE_MXFP4};
    static const int64_t dims[] = {64, 128, 320, 2048};
    Call c;
    const int32_t type = pick(types);
    const int64_t K = pick(dims), F = pick(dims), M = 1 + (int64_t)(next() % 70), E = 1 + (int64_t)(next() % 20),
                  N = 1 + (int64_t)(next() % 8);
    c.k = 1 + (int32_t)(next() % (uint64_t)(E < 16 ? E : 16));
    c.rule = (int32_t)(next() % 2);
    c.gate = experts(type, K, F, E, 0x100000000ull);
    c.up = experts(type, K, F, E, 0x200000000ull);
    c.down = experts(type, F, M, E, 0x300000000ull);
    c.x = dense(K, N, 0x400000000ull);
    c.y = dense(M, N, 0x500000000ull);
    c.logits = dense(E, N, 0x600000000ull);
    c.ids = (int32_t *)0x700000000ull;
    c.weights = (float *)0x800000000ull;
    c.route_ids = (int32_t *)0x900000000ull;
    c.route_weights = (float *)0xA00000000ull;
    c.ws = (void *)0xB00000000ull;
    c.ws_bytes = qmm_moe_workspace_size(&c.gate, &c.x, c.k);
    c.null = nullptr;
    return c;
}

}  // namespace

int main()
{
    long refused = 0, passed = 0;
    for (int i = 0; i < 20000; ++i) {
        Call c = good();
        const int before = g_launches;
        if (c.swiglu() != QMM_OK || c.route() != QMM_OK || g_launches != before + 2) {
            fprintf(stderr, "call %d: a well-formed call was refused\n", i);
            return 1;
        }
        qmm_tensor *all[] = {&c.gate, &c.up, &c.down, &c.x, &c.y, &c.logits};
        static const uintptr_t at[] = {0, 1, 2, 0x100000000ull, 0x400000000ull, 0x500000000ull, UINTPTR_MAX - 3, UINTPTR_MAX};
        switch (next() % 8) {
        case 0: c.null = all[next() % 6]; break;
        case 1: c.ids = c.route_ids = (int32_t *)pick(at); break;
        case 2: c.weights = c.route_weights = (float *)pick(at); break;
        case 3: c.ws = (void *)pick(at); break;
        case 4: c.ws_bytes = next() % 3 ? c.ws_bytes - 1 : 0; break;
        case 5: c.k = (int32_t)(next() % 40) - 2; break;
        case 6: c.rule = (int32_t)(next() % 5) - 1; break;
        default: spoil(*all[next() % 6]); break;
        }
        qmm_moe_workspace_size(c.arg(c.gate), c.arg(c.x), c.k);
        for (int which = 0; which < 2; ++which) {
            const int had = g_launches, rc = which ? c.route() : c.swiglu();
            if (rc > 0 || (rc < 0 && g_launches != had)) {
                fprintf(stderr, "call %d: status %d, %d launches\n", i, rc, g_launches - had);
                return 1;
            }
            ++(rc < 0 ? refused : passed);
        }
    }
    printf("%ld refused, %ld passed\n", refused, passed);
    return refused > 5000 && passed > 5000 ? 0 : 1;
}
