// api_checks.h -- descriptor rules shared by the entry points (qmm_api.cpp,
// moe_api.cpp).  Host only; nothing here touches device memory.
#pragma once

#include "../../include/qmm.h"
#include "qmm_internal.h"

namespace qmm {
namespace api {

// The types whose scales are fp16 and whose codes are integers.
inline bool is_int_quant(int t)
{
    return t == QMM_TYPE_Q8_0 || t == QMM_TYPE_Q4_0 || t == QMM_TYPE_Q8_B64 || t == QMM_TYPE_Q4_B64;
}
inline bool is_quant(int t) { return is_int_quant(t) || t == QMM_TYPE_MXFP4; }
inline bool is_b64(int t) { return t == QMM_TYPE_Q8_B64 || t == QMM_TYPE_Q4_B64; }
// Weights per scale of a quantized type.
inline int64_t block_len(int t) { return is_b64(t) ? 64 : 32; }

inline int64_t elem_size(int t)
{
    switch (t) {
    case QMM_TYPE_F32: return 4;
    case QMM_TYPE_F16: return 2;
    case QMM_TYPE_BF16: return 2;
    default: return 0;
    }
}

// Largest element count per dimension and byte span of one tensor the
// library accepts (far beyond any device memory, and small enough that
// every size computed from them fits 64 bits).
constexpr int64_t kMaxElems = (int64_t)1 << 48;
constexpr uint64_t kMaxSpan = 1ull << 62;

// Shape / layout rules shared by every operand.  `align` is the byte
// alignment required of data and nb[1].
inline int check_tensor(const qmm_tensor *t, uint64_t align)
{
    if (!t) return QMM_ERR_NULL;
    if (t->type < QMM_TYPE_F32 || t->type > QMM_TYPE_MXFP4) return QMM_ERR_TYPE;
    if (t->n_dims < 1 || t->n_dims > 4) return QMM_ERR_UNSUPPORTED;
    if (t->n_dims > 2 || t->ne[2] != 1 || t->ne[3] != 1) return QMM_ERR_UNSUPPORTED;
    if (t->ne[0] < 0 || t->ne[1] < 0) return QMM_ERR_SHAPE;
    if (t->ne[0] > kMaxElems || t->ne[1] > kMaxElems) return QMM_ERR_UNSUPPORTED;
    if (t->n_dims == 1 && t->ne[1] != 1) return QMM_ERR_SHAPE;
    if (is_quant(t->type)) {
        if (t->ne[0] % block_len(t->type) != 0) return QMM_ERR_SHAPE;
        if (t->nb[0] != 0) return QMM_ERR_LAYOUT;
    } else if ((int64_t)t->nb[0] != elem_size(t->type)) {
        return QMM_ERR_LAYOUT;
    }
    const uint64_t rs = qmm_row_size(t->type, t->ne[0]);
    if (t->ne[1] > 1 && t->nb[1] < rs) return QMM_ERR_LAYOUT;
    if (t->ne[1] > 1 && t->nb[1] % align != 0) return QMM_ERR_LAYOUT;
    // the bytes the tensor spans must be a range of the address space
    uint64_t span = rs;
    if (t->ne[1] > 1) {
        uint64_t rows;
        if (__builtin_mul_overflow((uint64_t)(t->ne[1] - 1), t->nb[1], &rows) || rows > kMaxSpan)
            return QMM_ERR_UNSUPPORTED;
        span = rows + rs;
    }
    if (span > kMaxSpan || (uintptr_t)t->data > UINTPTR_MAX - span) return QMM_ERR_UNSUPPORTED;
    const bool empty = t->ne[0] == 0 || t->ne[1] == 0;
    if (!t->data && !empty) return QMM_ERR_NULL;
    if ((uintptr_t)t->data % align != 0) return QMM_ERR_LAYOUT;
    return QMM_OK;
}

// Byte range [lo, hi) a 2-D tensor touches.
inline void extent(const qmm_tensor *t, uintptr_t *lo, uintptr_t *hi)
{
    const uint64_t rs = qmm_row_size(t->type, t->ne[0]);
    *lo = (uintptr_t)t->data;
    *hi = *lo + (t->ne[1] > 0 ? (uint64_t)(t->ne[1] - 1) * t->nb[1] + rs : 0);
}

inline bool overlaps(const qmm_tensor *a, const qmm_tensor *b)
{
    uintptr_t alo, ahi, blo, bhi;
    extent(a, &alo, &ahi);
    extent(b, &blo, &bhi);
    if (alo == ahi || blo == bhi) return false;
    return alo < bhi && blo < ahi;
}

inline WeightView weight_view(const qmm_tensor *w)
{
    WeightView v;
    v.base = static_cast<const uint8_t *>(w->data);
    v.pitch = w->ne[1] > 1 ? w->nb[1] : qmm_row_size(w->type, w->ne[0]);
    v.K = w->ne[0];
    v.M = w->ne[1];
    // the 64-block types are their code format with one scale per two runs;
    // an MXFP4 row's one-byte scales take as many bytes as two runs sharing
    // an fp16 scale, so its codes start at the same offset
    v.type = w->type == QMM_TYPE_Q8_B64 ? W_Q8_0 : w->type == QMM_TYPE_Q4_B64 ? W_Q4_0 : w->type;
    v.scale_shift = is_b64(w->type) || w->type == QMM_TYPE_MXFP4 ? 1 : 0;
    return v;
}

inline uint64_t pitch_elems(const qmm_tensor *t)
{
    const int64_t es = elem_size(t->type);
    return t->ne[1] > 1 ? t->nb[1] / (uint64_t)es : (uint64_t)t->ne[0];
}

// The activations of a GEMM: bf16 rows, or MXFP4 rows with a pitch in bytes.
inline ActView gemm_act(const qmm_tensor *x)
{
    if (x->type == QMM_TYPE_MXFP4) return ActView{x->data, weight_view(x).pitch, x->ne[1], W_MXFP4};
    return ActView{x->data, pitch_elems(x), x->ne[1]};
}

inline int status_of(hipError_t e) { return e == hipSuccess ? QMM_OK : QMM_ERR_DEVICE; }

}  // namespace api
}  // namespace qmm
