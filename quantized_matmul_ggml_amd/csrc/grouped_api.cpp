// grouped_api.cpp -- the C entry points of the products whose weights each
// token picks: slots grouped by expert, products grouped by expert, the
// mixture-of-experts layer for many tokens, and low-rank adapters.  Argument
// checks and dispatch, with the rules of qmm_api.cpp (host only; a call
// enqueues its kernels or returns a negative qmm_status with nothing enqueued).
#include "api_checks.h"
#include "lora_plan.h"

using namespace qmm::api;

namespace {

constexpr int64_t kMaxRows = (1ll << 31) - 1;        // grouped rows, tokens: 32-bit numbers
constexpr int64_t kMaxDim = 1ll << 28;               // K and M
constexpr uint64_t kMaxPitch = 1ull << 24;           // of weight rows (bytes: 128 below 2^31), base and y (floats: 32)

uint64_t align256(uint64_t n) { return (n + 255) / 256 * 256; }

// A group's operands apart from the output: the weights' shape as checked
// by check_experts, x BF16 of the same K.
int check_products(const qmm_tensor *w, const qmm_tensor *up, const qmm_tensor *x)
{
    if (!w || !up || !x) return QMM_ERR_NULL;
    int rc = check_experts(w);
    if (rc) return rc;
    rc = check_experts(up);
    if (rc) return rc;
    rc = check_tensor(x, 16);
    if (rc) return rc;
    if (x->type != QMM_TYPE_BF16 || up->type != w->type) return QMM_ERR_TYPE;
    for (int i = 0; i < 3; ++i)
        if (up->ne[i] != w->ne[i]) return QMM_ERR_SHAPE;
    if (x->ne[0] != w->ne[0]) return QMM_ERR_SHAPE;
    if (w->ne[2] > QMM_MOE_MAX_ROUTED || w->ne[0] > kMaxDim || w->ne[1] > kMaxDim || x->ne[1] > kMaxRows) return QMM_ERR_UNSUPPORTED;
    // offsets within a tile of 128 weight rows are 32-bit
    if (weight_view(w).pitch >= kMaxPitch || weight_view(up).pitch >= kMaxPitch) return QMM_ERR_UNSUPPORTED;
    return QMM_OK;
}

// Whether the kernel reaches x's rows with 32-bit offsets: all of x from its
// start when rows are picked, else a tile of 128 from the tile's first.
bool x_reach(const qmm_tensor *x, bool picked)
{
    const uint64_t rows = picked ? (uint64_t)x->ne[1] : 128;
    uint64_t bytes;
    return !__builtin_mul_overflow(rows, 2 * pitch_elems(x), &bytes) && bytes < 1ull << 31;
}

int check_out(const qmm_tensor *y)
{
    if (!y) return QMM_ERR_NULL;
    const int rc = check_tensor(y, y->type == QMM_TYPE_BF16 ? 2 : 4);
    if (rc) return rc;
    return y->type == QMM_TYPE_F32 || y->type == QMM_TYPE_BF16 ? QMM_OK : QMM_ERR_TYPE;
}

qmm::GroupedOut grouped_out(const qmm_tensor *y)
{
    return qmm::GroupedOut{y->data, pitch_elems(y), y->ne[1], y->type == QMM_TYPE_BF16};
}

// Whether R rows times w's experts make a launch that one grid takes.
bool fits(const qmm_tensor *w, int64_t R, bool swiglu)
{
    return qmm::grouped_fits(w->ne[1], w->ne[0], R, w->ne[2], weight_view(w).type, swiglu, qmm::device_cus());
}

// The products of one launch; up is w again without SwiGLU.
int grouped(const qmm_tensor *w, const qmm_tensor *up, bool swiglu, const qmm_tensor *x, const int32_t *offsets,
            const int32_t *order, int32_t top_k, qmm_tensor *y, void *stream)
{
    int rc = check_products(w, up, x);
    if (rc) return rc;
    rc = check_out(y);
    if (rc) return rc;
    const int64_t R = y->ne[1], E = w->ne[2];
    if (y->ne[0] != w->ne[1] || top_k < 1 || (!order && x->ne[1] != R)) return QMM_ERR_SHAPE;
    if (R > kMaxRows || !x_reach(x, order != nullptr) || !fits(w, R, swiglu)) return QMM_ERR_UNSUPPORTED;
    if (R == 0 || w->ne[1] == 0) return QMM_OK;
    if (!offsets) return QMM_ERR_NULL;
    if ((uintptr_t)offsets % 4 != 0 || (uintptr_t)order % 4 != 0) return QMM_ERR_LAYOUT;
    const uint64_t ob = 4 * ((uint64_t)E + 1), rb = order ? 4 * (uint64_t)R : 0;
    if (!spans(offsets, ob) || !spans(order, rb)) return QMM_ERR_UNSUPPORTED;
    const Range out = range_of(y), in[] = {range_of(w), range_of(up), range_of(x), range_of(offsets, ob), range_of(order, rb)};
    for (const Range &r : in)
        if (meet(out, r)) return QMM_ERR_ALIAS;
    const qmm::ExpertView uv = expert_view(up);
    return status_of(qmm::launch_gemm_grouped(expert_view(w), swiglu ? &uv : nullptr,
                                              qmm::ActView{x->data, pitch_elems(x), x->ne[1]}, offsets, order, top_k,
                                              grouped_out(y), static_cast<hipStream_t>(stream)));
}

// The parts of a layer's workspace, each a multiple of 256 bytes.
struct LayerSpace {
    uint64_t offsets, order, place, counts, h, d, bytes;
    int64_t d_pitch;             // floats between d's rows
};
bool layer_space(int64_t N, int64_t k, int64_t E, int64_t F, int64_t M, bool split, LayerSpace *s)
{
    const uint64_t R = (uint64_t)(N * k);            // below 2^31, F and M at most 2^28
    s->d_pitch = (M + 3) / 4 * 4;
    s->offsets = 0;
    s->order = s->offsets + align256(4 * ((uint64_t)E + 1));
    s->place = s->order + align256(4 * R);
    s->counts = s->place + align256(4 * R);
    s->h = s->counts + align256(qmm::moe_group_workspace((int64_t)R, E));
    s->d = s->h + align256((split ? 4 : 2) * R * (uint64_t)F);
    s->bytes = s->d + align256(4 * R * (uint64_t)s->d_pitch);
    return s->bytes <= kMaxSpan;
}

// The shape rules of a layer.
int check_layer(const qmm_tensor *gate, const qmm_tensor *up, const qmm_tensor *down, const qmm_tensor *x, int32_t top_k,
                LayerSpace *s)
{
    if (!down) return QMM_ERR_NULL;
    int rc = check_products(gate, up, x);
    if (rc) return rc;
    rc = check_experts(down);
    if (rc) return rc;
    if (down->type != gate->type) return QMM_ERR_TYPE;
    if (down->ne[0] != gate->ne[1] || down->ne[2] != gate->ne[2]) return QMM_ERR_SHAPE;
    if (top_k < 1 || top_k > QMM_MOE_MAX_TOP_K) return QMM_ERR_SHAPE;
    const int64_t N = x->ne[1], E = gate->ne[2];
    if (down->ne[1] > kMaxDim || weight_view(down).pitch >= kMaxPitch || N > kMaxRows / top_k) return QMM_ERR_UNSUPPORTED;
    const int64_t R = N * top_k;
    // the rows of h are F apart; a tile has 128 of them
    if (!x_reach(x, true) || 256 * (uint64_t)gate->ne[1] >= 1ull << 31 ||
        !fits(gate, R, true) || !fits(down, R, false)) return QMM_ERR_UNSUPPORTED;
    return layer_space(N, top_k, E, gate->ne[1], down->ne[1], false, s) ? QMM_OK : QMM_ERR_UNSUPPORTED;
}

// An adapter tensor: BF16, ne = [cols, rows, L].
int check_adapters(const qmm_tensor *t)
{
    if (!t) return QMM_ERR_NULL;
    if (t->type != QMM_TYPE_BF16) return QMM_ERR_TYPE;
    return check_matrices(t);
}

// The shape rules of the adapters and x.
int check_lora(const qmm_tensor *a, const qmm_tensor *b, const qmm_tensor *x)
{
    if (!a || !b || !x) return QMM_ERR_NULL;
    int rc = check_adapters(a);
    if (rc) return rc;
    rc = check_adapters(b);
    if (rc) return rc;
    rc = check_tensor(x, x->type == QMM_TYPE_BF16 ? 16 : 4);
    if (rc) return rc;
    if (x->type != QMM_TYPE_F32 && x->type != QMM_TYPE_BF16) return QMM_ERR_TYPE;
    const int64_t K = a->ne[0], r = a->ne[1];
    if (x->ne[0] != K || K % 32 != 0 || r < 8 || r % 8 != 0 || r > QMM_LORA_MAX_RANK) return QMM_ERR_SHAPE;
    if (b->ne[0] != r || b->ne[2] != a->ne[2]) return QMM_ERR_SHAPE;
    // 32 rows of x and 128 rows of A and B are reached with 32-bit offsets
    if (x->ne[1] > QMM_LORA_MAX_TOKENS || pitch_elems(x) >= kMaxPitch || pitch_elems(a) >= kMaxPitch / 2 ||
        pitch_elems(b) >= kMaxPitch / 2 || b->ne[1] >= (int64_t)kMaxPitch)
        return QMM_ERR_UNSUPPORTED;
    return QMM_OK;
}

// What the call needs wherever x lies.
uint64_t lora_workspace(int64_t N, int64_t K, int64_t M, int64_t r)
{
    uint64_t most = 0;
    for (const bool wide : {false, true}) {
        const qmm::LoraPlan p = qmm::plan_lora(N, K, M, r, wide, qmm::device_cus());
        const uint64_t bytes = p.single ? 0 : (uint64_t)p.chunks * (uint64_t)N * 16 * (uint64_t)p.rt * 4;
        most = bytes > most ? bytes : most;
    }
    return most;
}

}  // namespace

extern "C" {

size_t qmm_moe_group_workspace_size(int64_t n_slots, int32_t n_experts)
{
    if (n_slots < 1 || n_slots > kMaxRows || n_experts < 1 || n_experts > QMM_MOE_MAX_ROUTED) return 0;
    return (size_t)qmm::moe_group_workspace(n_slots, n_experts);
}

int qmm_moe_group(const int32_t *ids, int64_t n_slots, int32_t n_experts, int32_t *offsets, int32_t *order, int32_t *place,
                  void *workspace, size_t workspace_bytes, void *stream)
{
    if (n_slots < 0 || n_experts < 1) return QMM_ERR_SHAPE;
    if (n_slots > kMaxRows || n_experts > QMM_MOE_MAX_ROUTED) return QMM_ERR_UNSUPPORTED;
    const uint64_t need = qmm_moe_group_workspace_size(n_slots, n_experts);
    if (!offsets || (n_slots > 0 && (!ids || !order || !place)) || (need && !workspace)) return QMM_ERR_NULL;
    if (((uintptr_t)ids | (uintptr_t)offsets | (uintptr_t)order | (uintptr_t)place) % 4 != 0 || (need && (uintptr_t)workspace % 16 != 0))
        return QMM_ERR_LAYOUT;
    if (workspace_bytes < need) return QMM_ERR_SCRATCH;
    const uint64_t slots = 4 * (uint64_t)n_slots, ends = 4 * ((uint64_t)n_experts + 1);
    if (!spans(ids, slots) || !spans(offsets, ends) || !spans(order, slots) || !spans(place, slots) || !spans(workspace, need))
        return QMM_ERR_UNSUPPORTED;
    const Range all[] = {range_of(ids, slots), range_of(offsets, ends), range_of(order, slots), range_of(place, slots),
                         range_of(workspace, need)};
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (meet(all[i], all[j])) return QMM_ERR_ALIAS;
    return status_of(qmm::launch_moe_group(ids, n_slots, n_experts, offsets, order, place, workspace,
                                           static_cast<hipStream_t>(stream)));
}

int qmm_gemm_grouped(const qmm_tensor *w, const qmm_tensor *x, const int32_t *offsets, const int32_t *order, int32_t top_k,
                     qmm_tensor *y, void *stream)
{
    return grouped(w, w, false, x, offsets, order, top_k, y, stream);
}

int qmm_gemm_grouped_swiglu(const qmm_tensor *w_gate, const qmm_tensor *w_up, const qmm_tensor *x, const int32_t *offsets,
                            const int32_t *order, int32_t top_k, qmm_tensor *h, void *stream)
{
    return grouped(w_gate, w_up, true, x, offsets, order, top_k, h, stream);
}

size_t qmm_moe_gemm_workspace_size(const qmm_tensor *w_gate, const qmm_tensor *w_down, const qmm_tensor *x, int32_t top_k)
{
    LayerSpace s;
    if (check_layer(w_gate, w_gate, w_down, x, top_k, &s) || x->ne[1] == 0 || w_down->ne[1] == 0) return 0;
    return (size_t)s.bytes;
}

int qmm_moe_gemm_swiglu(const qmm_tensor *w_gate, const qmm_tensor *w_up, const qmm_tensor *w_down, const qmm_tensor *x,
                        const int32_t *ids, const float *weights, int32_t top_k, qmm_tensor *y, void *workspace,
                        size_t workspace_bytes, void *stream)
{
    LayerSpace s;
    int rc = check_layer(w_gate, w_up, w_down, x, top_k, &s);
    if (rc) return rc;
    rc = check_out(y);
    if (rc) return rc;
    const int64_t N = x->ne[1], E = w_gate->ne[2], F = w_gate->ne[1], M = w_down->ne[1], R = N * top_k;
    if (y->ne[0] != M || y->ne[1] != N) return QMM_ERR_SHAPE;
    if (N == 0 || M == 0) return QMM_OK;
    if (!ids || !weights || !workspace) return QMM_ERR_NULL;
    if (((uintptr_t)ids | (uintptr_t)weights) % 4 != 0 || (uintptr_t)workspace % 16 != 0) return QMM_ERR_LAYOUT;
    if (workspace_bytes < s.bytes) return QMM_ERR_SCRATCH;
    // h between the products.  In one bf16 part it is the activation of every product of
    // many tokens, and takes 2 R F bytes, but is off by up to 2^-8 of a value, which a
    // BF16 y shows beside its own rounding (4096 tokens over 8 experts, 2048 x 5632 Q4_0:
    // 2.35e-3 of y's norm, 1.66e-3 with h exact, and 1.66e-3 with an F32 y too).  Two
    // parts are off by 2^-16 (1.66e-3, and 2.4e-6), take another 2 R F bytes and a second
    // matrix instruction in the second product (722 -> 858 us; 64 tokens over 64 experts,
    // 2048 x 1024 MXFP4 78 -> 81): taken where the caller gives the room, and where its
    // rows' tiles are reached with 32-bit offsets.
    LayerSpace both;
    const bool split = layer_space(N, top_k, E, F, M, true, &both) && workspace_bytes >= both.bytes && 512 * (uint64_t)F < 1ull << 31 &&
                       qmm::grouped_fits(M, F, R, E, weight_view(w_down).type, false, qmm::device_cus(), 2);
    if (split) s = both;
    const uint64_t pairs = 4 * (uint64_t)R;
    if (!spans(ids, pairs) || !spans(weights, pairs) || !spans(workspace, s.bytes)) return QMM_ERR_UNSUPPORTED;
    const Range in[] = {range_of(w_gate), range_of(w_up), range_of(w_down), range_of(x), range_of(ids, pairs),
                        range_of(weights, pairs)};
    const Range out = range_of(y), ws = range_of(workspace, s.bytes);
    if (meet(out, ws)) return QMM_ERR_ALIAS;
    for (const Range &r : in)
        if (meet(out, r) || meet(ws, r)) return QMM_ERR_ALIAS;
    uint8_t *const base = static_cast<uint8_t *>(workspace);
    int32_t *const offsets = reinterpret_cast<int32_t *>(base + s.offsets), *const order = reinterpret_cast<int32_t *>(base + s.order);
    int32_t *const place = reinterpret_cast<int32_t *>(base + s.place);
    float *const d = reinterpret_cast<float *>(base + s.d);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = qmm::launch_moe_group(ids, R, E, offsets, order, place, base + s.counts, st);
    if (e == hipSuccess && F > 0) {
        const qmm::ExpertView up = expert_view(w_up);
        e = qmm::launch_gemm_grouped(expert_view(w_gate), &up, qmm::ActView{x->data, pitch_elems(x), N}, offsets, order, top_k,
                                     qmm::GroupedOut{base + s.h, (uint64_t)(split ? 2 * F : F), R, true, split}, st);
    }
    if (e == hipSuccess)
        e = qmm::launch_gemm_grouped(expert_view(w_down), nullptr,
                                     qmm::ActView{base + s.h, (uint64_t)(split ? 2 * F : F), R, qmm::W_BF16, split}, offsets, nullptr, 1,
                                     qmm::GroupedOut{d, (uint64_t)s.d_pitch, R, false}, st);
    if (e == hipSuccess) e = qmm::launch_moe_combine(d, (uint64_t)s.d_pitch, place, weights, top_k, N, M, grouped_out(y), st);
    return status_of(e);
}

size_t qmm_lora_workspace_size(const qmm_tensor *a, const qmm_tensor *b, const qmm_tensor *x)
{
    if (check_lora(a, b, x) || x->ne[1] == 0 || b->ne[1] == 0) return 0;
    return (size_t)lora_workspace(x->ne[1], a->ne[0], b->ne[1], a->ne[1]);
}

int qmm_lora(const qmm_tensor *a, const qmm_tensor *b, const qmm_tensor *x, const int32_t *ids, const float *scales,
             const qmm_tensor *base, qmm_tensor *y, void *workspace, size_t workspace_bytes, void *stream)
{
    int rc = check_lora(a, b, x);
    if (rc) return rc;
    rc = check_tensor(y, 4);
    if (rc) return rc;
    if (y->type != QMM_TYPE_F32) return QMM_ERR_TYPE;
    const int64_t K = a->ne[0], r = a->ne[1], L = a->ne[2], M = b->ne[1], N = x->ne[1];
    if (y->ne[0] != M || y->ne[1] != N) return QMM_ERR_SHAPE;
    if (base) {
        rc = check_tensor(base, 4);
        if (rc) return rc;
        if (base->type != QMM_TYPE_F32) return QMM_ERR_TYPE;
        if (base->ne[0] != M || base->ne[1] != N) return QMM_ERR_SHAPE;
    }
    if (pitch_elems(y) >= kMaxPitch || (base && pitch_elems(base) >= kMaxPitch)) return QMM_ERR_UNSUPPORTED;
    if (N == 0 || M == 0) return QMM_OK;
    const bool f32x = x->type == QMM_TYPE_F32;
    const qmm::LoraPlan p = qmm::plan_lora(N, K, M, r, qmm::lora_wide(x->data, pitch_elems(x), f32x), qmm::device_cus());
    const int64_t most = (int64_t)(qmm::kMaxGridThreads / 256) - 1;
    if (2 * p.blocks1 > most || p.blocks2 > most) return QMM_ERR_UNSUPPORTED;
    const uint64_t need = lora_workspace(N, K, M, r);
    if (!ids || (need && !workspace)) return QMM_ERR_NULL;
    if (((uintptr_t)ids | (uintptr_t)scales) % 4 != 0 || (need && (uintptr_t)workspace % 16 != 0)) return QMM_ERR_LAYOUT;
    if (workspace_bytes < need) return QMM_ERR_SCRATCH;
    const uint64_t ib = 4 * (uint64_t)N, sb = scales ? 4 * (uint64_t)L : 0;
    if (!spans(ids, ib) || !spans(scales, sb) || !spans(workspace, need)) return QMM_ERR_UNSUPPORTED;
    const Range in[] = {range_of(a), range_of(b), range_of(x), range_of(ids, ib), range_of(scales, sb)};
    const Range out = range_of(y), ws = range_of(workspace, need);
    if (meet(out, ws)) return QMM_ERR_ALIAS;
    for (const Range &v : in)
        if (meet(out, v) || meet(ws, v)) return QMM_ERR_ALIAS;
    if (base) {
        // y may be base itself: each output is read and written by one thread
        const bool same = base->data == y->data && (N == 1 || base->nb[1] == y->nb[1]);
        if (meet(ws, range_of(base)) || (!same && meet(out, range_of(base)))) return QMM_ERR_ALIAS;
    }
    qmm::LoraTask t = {};
    t.a = static_cast<const uint16_t *>(a->data);
    t.b = static_cast<const uint16_t *>(b->data);
    t.a_pitch = pitch_elems(a);
    t.b_pitch = pitch_elems(b);
    t.a_adapter = L > 1 ? a->nb[2] / 2 : 0;
    t.b_adapter = L > 1 ? b->nb[2] / 2 : 0;
    t.x = x->data;
    t.x_pitch = pitch_elems(x);
    t.f32x = f32x;
    t.ids = ids;
    t.scales = scales;
    t.base = base ? static_cast<const float *>(base->data) : nullptr;
    t.base_pitch = base ? pitch_elems(base) : 0;
    t.y = static_cast<float *>(y->data);
    t.y_pitch = pitch_elems(y);
    t.ws = workspace;
    t.N = N;
    t.K = K;
    t.M = M;
    t.r = r;
    t.L = L;
    return status_of(qmm::launch_lora(t, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
