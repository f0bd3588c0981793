// grouped_driver.cpp -- drives the host layer of the grouped products, the layer of
// many tokens and the adapters (grouped_api.cpp, with its launchers stubbed out
// here) under AddressSanitizer and UndefinedBehaviorSanitizer: a deterministic
// stream of well-formed calls, and of the same with one argument replaced, over
// fake device addresses that are validated and never read.  Exits 0 when every
// well-formed call reached its launchers, no refused call did, and no sanitizer
// reported anything (a report aborts the process).
#include "../../include/qmm.h"
#include "../../quantized_matmul_ggml_amd/csrc/qmm_internal.h"

#include <stdio.h>

extern int g_launches;

namespace qmm {

int device_cus() { return 256; }
hipError_t launch_moe_group(const int32_t *, int64_t, int64_t, int32_t *, int32_t *, int32_t *, void *, hipStream_t)
{
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_gemm_grouped(const ExpertView &, const ExpertView *, const ActView &, const int32_t *, const int32_t *, int,
                               const GroupedOut &, hipStream_t)
{
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_moe_combine(const float *, uint64_t, const int32_t *, const float *, int, int64_t, int64_t, const GroupedOut &,
                              hipStream_t)
{
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_lora(const LoraTask &, hipStream_t)
{
    ++g_launches;
    return hipSuccess;
}

}  // namespace qmm

namespace {

uint64_t state = 0x9E3779B97F4A7C15ull;
uint64_t next()
{
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return state;
}
template <class T, size_t N> T pick(const T (&v)[N]) { return v[next() % N]; }

qmm_tensor dense(int32_t type, int64_t cols, int64_t rows, uintptr_t at)
{
    const uint64_t size = type == QMM_TYPE_F32 ? 4 : 2;
    qmm_tensor t = {type, 2, {cols, rows, 1, 1}, {size, (uint64_t)cols * size, 0, 0}, (void *)at};
    t.nb[2] = t.nb[3] = t.nb[1] * (uint64_t)(rows > 1 ? rows : 1);
    return t;
}
qmm_tensor matrices(int32_t type, int64_t K, int64_t M, int64_t E, uintptr_t at)
{
    qmm_tensor t = {type, 3, {K, M, E, 1}, {type == QMM_TYPE_BF16 ? 2ull : 0ull, qmm_row_size(type, K), 0, 0}, (void *)at};
    t.nb[2] = t.nb[1] * (uint64_t)(M > 1 ? M : 1);
    t.nb[3] = t.nb[2] * (uint64_t)E;
    return t;
}
void spoil(qmm_tensor &t)
{
    static const int64_t sizes[] = {INT64_MIN, -32, -1, 0, 1, 7, 33, 64, 1ll << 24, 1ll << 28, 1ll << 31, 1ll << 40, INT64_MAX};
    static const uint64_t strides[] = {0, 1, 4, 15, 16, 1ull << 24, 1ull << 28, 1ull << 40, 1ull << 62, UINT64_MAX};
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
    qmm_tensor gate, up, down, x, h, y, a, b, xl, base, yl;
    int64_t slots;
    int32_t experts, k;
    int32_t *ids, *offsets, *order, *place;
    float *weights;
    void *ws;
    uint64_t ws_bytes;
    bool picked;
    qmm_tensor *null;             // passed as NULL instead, or none
    qmm_tensor *arg(qmm_tensor &t) { return &t == null ? nullptr : &t; }
    int run(int which)
    {
        switch (which) {
        case 0: return qmm_moe_group(ids, slots, experts, offsets, order, place, ws, ws_bytes, nullptr);
        case 1: return qmm_gemm_grouped(arg(gate), arg(x), offsets, picked ? order : nullptr, k, arg(h), nullptr);
        case 2: return qmm_gemm_grouped_swiglu(arg(gate), arg(up), arg(x), offsets, picked ? order : nullptr, k, arg(h), nullptr);
        case 3: return qmm_moe_gemm_swiglu(arg(gate), arg(up), arg(down), arg(x), ids, weights, k, arg(y), ws, ws_bytes, nullptr);
        default: return qmm_lora(arg(a), arg(b), arg(xl), ids, weights, base.data ? arg(base) : nullptr, arg(yl), ws, ws_bytes, nullptr);
        }
    }
};
constexpr int kCalls = 5;
constexpr int kLaunches[kCalls] = {1, 1, 1, 4, 1};

Call good()
{
    static const int32_t types[] = {QMM_TYPE_Q8_0, QMM_TYPE_Q4_0, QMM_TYPE_Q8_B64, QMM_TYPE_Q4_B64, QMM_TYPE_MXFP4};
    static const int64_t dims[] = {64, 128, 320, 2048};
    static const int64_t counts[] = {1, 2, 63, 700, 9000};
    Call c;
    const int32_t type = pick(types), xt = next() % 2 ? QMM_TYPE_F32 : QMM_TYPE_BF16, yt = next() % 2 ? QMM_TYPE_F32 : QMM_TYPE_BF16;
    const int64_t K = pick(dims), F = pick(dims), M = 1 + (int64_t)(next() % 700), E = 1 + (int64_t)(next() % 200), N = pick(counts),
                  r = 8 * (1 + (int64_t)(next() % 16)), L = 1 + (int64_t)(next() % 30);
    c.k = 1 + (int32_t)(next() % 16);
    c.picked = next() % 2;
    const int64_t R = c.picked ? N * c.k : N;
    c.gate = matrices(type, K, F, E, 0x100000000ull);
    c.up = matrices(type, K, F, E, 0x200000000ull);
    c.down = matrices(type, F, M, E, 0x300000000ull);
    c.x = dense(QMM_TYPE_BF16, K, N, 0x400000000ull);
    c.h = dense(yt, F, R, 0x500000000ull);
    c.y = dense(yt, M, N, 0x600000000ull);
    c.a = matrices(QMM_TYPE_BF16, K, r, L, 0x700000000ull);
    c.b = matrices(QMM_TYPE_BF16, r, M, L, 0x800000000ull);
    c.xl = dense(xt, K, N, 0x900000000ull);
    c.yl = dense(QMM_TYPE_F32, M, N, 0xA00000000ull);
    c.base = dense(QMM_TYPE_F32, M, N, next() % 3 == 0 ? 0 : next() % 2 ? 0xA00000000ull : 0xB00000000ull);
    c.slots = N * 16;
    c.experts = (int32_t)E;
    c.ids = (int32_t *)0xC00000000ull;
    c.offsets = (int32_t *)0xD00000000ull;
    c.order = (int32_t *)0xE00000000ull;
    c.place = (int32_t *)0xF00000000ull;
    c.weights = (float *)0x1000000000ull;
    c.ws = (void *)0x1100000000ull;
    const uint64_t layer = qmm_moe_gemm_workspace_size(&c.gate, &c.down, &c.x, c.k), lora = qmm_lora_workspace_size(&c.a, &c.b, &c.xl),
                   group = qmm_moe_group_workspace_size(c.slots, c.experts);
    c.ws_bytes = layer > lora ? layer : lora;
    if (group > c.ws_bytes) c.ws_bytes = group;
    c.null = nullptr;
    return c;
}

}  // namespace

int main()
{
    long refused = 0, passed = 0;
    for (int i = 0; i < 20000; ++i) {
        Call c = good();
        for (int which = 0; which < kCalls; ++which) {
            const int had = g_launches, rc = c.run(which);
            if (rc != QMM_OK || g_launches != had + kLaunches[which]) {
                fprintf(stderr, "call %d.%d: a well-formed call was refused (%d)\n", i, which, rc);
                return 1;
            }
        }
        qmm_tensor *all[] = {&c.gate, &c.up, &c.down, &c.x, &c.h, &c.y, &c.a, &c.b, &c.xl, &c.base, &c.yl};
        static const uintptr_t at[] = {0, 1, 2, 0x100000000ull, 0x400000000ull, 0x500000000ull, 0xA00000000ull, UINTPTR_MAX - 3, UINTPTR_MAX};
        static const int64_t counts[] = {INT64_MIN, -1, 0, 65536, 65537, (1ll << 31) - 1, 1ll << 31, INT64_MAX};
        switch (next() % 12) {
        case 0: c.null = all[next() % 11]; break;
        case 1: c.ids = (int32_t *)pick(at); break;
        case 2: c.weights = (float *)pick(at); break;
        case 3: c.ws = (void *)pick(at); break;
        case 4: c.ws_bytes = next() % 3 ? c.ws_bytes - 1 : 0; break;
        case 5: c.k = next() % 3 ? (int32_t)(next() % 40) - 2 : INT32_MAX; break;
        case 6: c.slots = pick(counts); break;
        case 7: c.experts = next() % 2 ? (int32_t)(next() % 2000) - 400 : INT32_MIN; break;
        case 8: (next() % 2 ? c.offsets : next() % 2 ? c.order : c.place) = (int32_t *)pick(at); break;
        default: spoil(*all[next() % 11]); break;
        }
        qmm_moe_gemm_workspace_size(c.arg(c.gate), c.arg(c.down), c.arg(c.x), c.k);
        qmm_lora_workspace_size(c.arg(c.a), c.arg(c.b), c.arg(c.xl));
        qmm_moe_group_workspace_size(c.slots, c.experts);
        for (int which = 0; which < kCalls; ++which) {
            const int had = g_launches, rc = c.run(which);
            if (rc > 0 || (rc < 0 && g_launches != had)) {
                fprintf(stderr, "call %d.%d: status %d, %d launches\n", i, which, rc, g_launches - had);
                return 1;
            }
            ++(rc < 0 ? refused : passed);
        }
    }
    printf("%ld refused, %ld passed\n", refused, passed);
    return refused > 5000 && passed > 5000 ? 0 : 1;
}
