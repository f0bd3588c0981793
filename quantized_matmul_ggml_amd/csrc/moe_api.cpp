// moe_api.cpp -- the C entry points of the mixture-of-experts layer: argument
// checks and dispatch, with the rules of qmm_api.cpp (host only; a call
// enqueues its kernels or returns a negative qmm_status with nothing
// enqueued).
#include "api_checks.h"

using namespace qmm::api;

namespace {

// The shape rules of a layer; on success *ws_bytes is its workspace.
int check_layer(const qmm_tensor *gate, const qmm_tensor *up, const qmm_tensor *down, const qmm_tensor *x, int32_t top_k,
                uint64_t *ws_bytes)
{
    if (!gate || !up || !down || !x) return QMM_ERR_NULL;
    int rc = check_experts(gate);
    if (rc) return rc;
    rc = check_experts(up);
    if (rc) return rc;
    rc = check_experts(down);
    if (rc) return rc;
    rc = check_tensor(x, 4);
    if (rc) return rc;
    if (x->type != QMM_TYPE_F32 || up->type != gate->type || down->type != gate->type) return QMM_ERR_TYPE;
    for (int i = 0; i < 3; ++i)
        if (up->ne[i] != gate->ne[i]) return QMM_ERR_SHAPE;
    if (down->ne[0] != gate->ne[1] || down->ne[2] != gate->ne[2] || x->ne[0] != gate->ne[0]) return QMM_ERR_SHAPE;
    if (top_k < 1 || top_k > QMM_MOE_MAX_TOP_K || x->ne[1] > QMM_MOE_MAX_TOKENS) return QMM_ERR_SHAPE;
    // row counts, blocks and the workspace are indexed with 32 bits
    const int64_t lim = 1ll << 28;
    if (gate->ne[0] > lim || gate->ne[1] > lim || down->ne[1] > qmm::kMoeMostRows) return QMM_ERR_UNSUPPORTED;
    *ws_bytes = x->ne[1] > 0 ? qmm::moe_workspace(x->ne[1], top_k, gate->ne[1]) : 0;
    if (*ws_bytes >= (1ull << 31)) return QMM_ERR_UNSUPPORTED;
    return QMM_OK;
}

}  // namespace

extern "C" {

int qmm_moe_route(const qmm_tensor *logits, int32_t top_k, int32_t rule, int32_t *ids, float *weights, void *stream)
{
    if (rule != QMM_ROUTE_ALL && rule != QMM_ROUTE_CHOSEN) return QMM_ERR_UNSUPPORTED;
    int rc = check_tensor(logits, 4);
    if (rc) return rc;
    if (logits->type != QMM_TYPE_F32) return QMM_ERR_TYPE;
    const int64_t E = logits->ne[0], N = logits->ne[1];
    if (top_k < 1 || top_k > QMM_MOE_MAX_TOP_K || top_k > E) return QMM_ERR_SHAPE;
    if (E > QMM_MOE_MAX_ROUTED || N >= (1ll << 31)) return QMM_ERR_UNSUPPORTED;
    if (N == 0) return QMM_OK;
    if (!ids || !weights) return QMM_ERR_NULL;
    if ((uintptr_t)ids % 4 != 0 || (uintptr_t)weights % 4 != 0) return QMM_ERR_LAYOUT;
    const uint64_t bytes = 4 * (uint64_t)N * (uint64_t)top_k;
    if (!spans(ids, bytes) || !spans(weights, bytes)) return QMM_ERR_UNSUPPORTED;
    const Range i = range_of(ids, bytes), w = range_of(weights, bytes), l = range_of(logits);
    if (meet(i, w) || meet(i, l) || meet(w, l)) return QMM_ERR_ALIAS;
    return status_of(qmm::launch_moe_route(static_cast<const float *>(logits->data), pitch_elems(logits), N, (int)E,
                                           top_k, rule == QMM_ROUTE_ALL, ids, weights,
                                           static_cast<hipStream_t>(stream)));
}

size_t qmm_moe_workspace_size(const qmm_tensor *w_gate, const qmm_tensor *x_f32, int32_t top_k)
{
    if (!w_gate || !x_f32 || check_experts(w_gate) || check_tensor(x_f32, 4)) return 0;
    if (top_k < 1 || top_k > QMM_MOE_MAX_TOP_K || x_f32->ne[1] > QMM_MOE_MAX_TOKENS) return 0;
    if (w_gate->ne[1] > (1ll << 28)) return 0;
    return x_f32->ne[1] > 0 ? (size_t)qmm::moe_workspace(x_f32->ne[1], top_k, w_gate->ne[1]) : 0;
}

int qmm_moe_swiglu(const qmm_tensor *w_gate, const qmm_tensor *w_up, const qmm_tensor *w_down, const qmm_tensor *x,
                   const int32_t *ids, const float *weights, int32_t top_k, qmm_tensor *y, void *workspace,
                   size_t workspace_bytes, void *stream)
{
    uint64_t need = 0;
    int rc = check_layer(w_gate, w_up, w_down, x, top_k, &need);
    if (rc) return rc;
    rc = check_tensor(y, 4);
    if (rc) return rc;
    if (y->type != QMM_TYPE_F32) return QMM_ERR_TYPE;
    if (y->ne[0] != w_down->ne[1] || y->ne[1] != x->ne[1]) return QMM_ERR_SHAPE;
    const int64_t N = x->ne[1];
    if (N == 0 || y->ne[0] == 0) return QMM_OK;
    if (!ids || !weights || (need && !workspace)) return QMM_ERR_NULL;
    if ((uintptr_t)ids % 4 != 0 || (uintptr_t)weights % 4 != 0 || (uintptr_t)workspace % 16 != 0) return QMM_ERR_LAYOUT;
    if (workspace_bytes < need) return QMM_ERR_SCRATCH;
    const uint64_t pairs = 4 * (uint64_t)N * (uint64_t)top_k;
    if (!spans(ids, pairs) || !spans(weights, pairs) || !spans(workspace, need)) return QMM_ERR_UNSUPPORTED;
    const Range in[] = {range_of(w_gate), range_of(w_up), range_of(w_down), range_of(x), range_of(ids, pairs),
                        range_of(weights, pairs)};
    const Range out = range_of(y), ws = range_of(workspace, need);
    if (meet(out, ws)) return QMM_ERR_ALIAS;
    for (const Range &r : in)
        if (meet(out, r) || meet(ws, r)) return QMM_ERR_ALIAS;
    qmm::ActView xv{x->data, pitch_elems(x), N};
    qmm::OutView yv{static_cast<float *>(y->data), pitch_elems(y)};
    return status_of(qmm::launch_moe_swiglu(expert_view(w_gate), expert_view(w_up), expert_view(w_down), xv, ids,
                                            weights, top_k, yv, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
