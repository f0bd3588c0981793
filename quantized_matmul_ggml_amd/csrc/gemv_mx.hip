// gemv_mx.hip -- decode GEMV for MXFP4 weights and 1 to 8 fp32 tokens on the
// bf16 matrix cores, alone, batched, or as the gate/up pair fused with SwiGLU.
//
// y[n][m] = sum_k W'[m][k] x[n][k] (A Complete Guide to llama.cpp and
// Customization with C++, §2.1: at one token per step every projection is a
// GEMV, bound by the weight stream), with the arithmetic of row_tiles.h: every
// product is exact and only the binary32 accumulation rounds.
//
// Work split: a workgroup of sixteen waves covers 16 / S tiles of 16 weight
// rows, S waves sharing a tile's K in interleaved quanta of QU units (128 QU
// values of k, 64 QU code bytes of each row).  Few tiles take more waves per
// tile so that the chip still fills; the first quantum of every wave is in
// flight while the workgroup splits its tokens into the LDS image.  Each
// wave's next quantum (of this tile or, at its end, of the workgroup's next
// one) is loaded before the current one is multiplied.  The S partial sums
// meet in LDS and are added in wave order.
#include "row_tiles.h"

namespace qmm {
namespace {

constexpr int kWaves = 16;
constexpr int kThreads = 64 * kWaves;
constexpr int kImageMax = 96 * 1024;       // LDS bytes of the activation image

struct alignas(64) MxItem {
    const uint8_t *w;
    const uint8_t *w2;        // fused SwiGLU: the up projection (w is the gate)
    const float *x;
    float *y;
    uint32_t pitch;           // bytes between weight rows
    uint32_t pitch2;
    uint32_t x_pitch;         // elements between token rows of x
    uint32_t y_pitch;
    int32_t M;
    int32_t n_groups;         // tile groups (16 / S tiles each)
    int32_t wgs;              // workgroups of this item (grid x)
    int32_t pad;
};
static_assert(sizeof(MxItem) == 64, "one 64-byte record per item");

struct MxArgs {
    int32_t N;
    int32_t nb;               // 32-blocks per row
    int32_t qoff;
    int32_t nq;               // quanta per row
    int32_t s_log2;           // waves per tile
    int32_t pass_q;           // quanta per K pass (a multiple of S)
    int32_t pad[10];
    MxItem item[QMM_GEMV_BATCH_MAX];
};

template <int QU, int TG, bool SW>
__global__ __launch_bounds__(kThreads) void gemv_mx_kernel(const MxArgs a)
{
    constexpr int WT = W_MXFP4, SS = 0;
    using F = RowFmt<WT, SS>;
    constexpr int QB = QU * F::MF;                 // blocks (and instructions) per quantum
    constexpr int ROWS = SW ? 8 : 16;              // row indices per tile
    extern __shared__ __attribute__((aligned(16))) uint8_t img[];
    __shared__ float red[2][kWaves][TG][64];

    const MxItem &it = a.item[blockIdx.y];
    const uint8_t *const W = it.w, *const W2 = it.w2;
    const float *const X = it.x;
    float *const Y = it.y;
    const uint32_t pitch = it.pitch, pitch2 = it.pitch2, x_pitch = it.x_pitch, y_pitch = it.y_pitch;
    const int M = it.M, n_groups = it.n_groups, wgs = it.wgs;
    const int N = a.N, nb = a.nb, qoff = a.qoff, nq = a.nq, s_log2 = a.s_log2, pass_q = a.pass_q;
    if ((int)blockIdx.x >= wgs) return;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, g = lane >> 4;
    const int S = 1 << s_log2, T = kWaves >> s_log2;
    const int split = wave & (S - 1), tile_in = wave >> s_log2;

    // ---- the lane's row of a tile: a column of the gate or up matrix; rows
    // past M repeat the last one and are not stored ----
    const bool second = SW && j >= 8;
    const uint8_t *const Wl = second ? W2 : W;
    const uint32_t pl = second ? pitch2 : pitch;
    auto load = [&](Quantum<WT, SS, QU> &z, int grp, int qi) {
        const int64_t r = (int64_t)(grp * T + tile_in) * ROWS + (SW ? j & 7 : j);
        load_quantum<WT, SS, QU>(z, Wl + (uint64_t)(r < M ? r : M - 1) * pl, qoff, 16 * nb, qi, g);
    };
    // ---- activation fragments: matrix row 4 t + p is part p of token t ----
    uint32_t frag_off[TG];
#pragma unroll
    for (int tg = 0; tg < TG; ++tg) {
        const int tok = 4 * tg + (j >> 2), part = (j & 3) < 2 ? (j & 3) : 2;
        frag_off[tg] = (uint32_t)((tok < N ? tok : N - 1) * kImageBytes + 64 * part + 16 * g);
    }
    const uint32_t step_bytes = (uint32_t)N * kImageBytes;

    int grp = blockIdx.x;
    Quantum<WT, SS, QU> cur, nxt;
    if (split < nq) load(cur, grp, split);
    int parity = 0;
    bool built = false;
    for (; grp < n_groups; grp += wgs, parity ^= 1) {
        RowAcc<WT> acc[TG];
        for (int q0 = 0; q0 < nq; q0 += pass_q) {
            const int q1 = q0 + pass_q < nq ? q0 + pass_q : nq;
            if (!built || pass_q < nq) {
                if (built) __syncthreads();        // the last pass's image is no longer read
                build_image<WT>(img, N, q0 * QB, (q1 - q0) * QB, nb, kThreads,
                                [&](int t) { return X + (uint64_t)t * x_pitch; });
                built = true;
                __syncthreads();
            }
            for (int q = q0 + split; q < q1; q += S) {
                const bool more = q + S < nq;
                const int ngrp = more ? grp : grp + wgs;
                if (ngrp < n_groups) load(nxt, ngrp, more ? q + S : split);
                const uint8_t *base = img + (uint32_t)((q - q0) * QB) * step_bytes;
                multiply_quantum<WT, SS, QU, TG>(cur, q, nb, g, TG, acc, [&](int tg, int step) {
                    return *reinterpret_cast<const rt_bf16x8 *>(base + (uint32_t)step * step_bytes + frag_off[tg]);
                });
                cur = nxt;
            }
        }
#pragma unroll
        for (int tg = 0; tg < TG; ++tg) red[parity][wave][tg][lane] = row_total(acc[tg]);
        __syncthreads();
        // the other parity's buffer is free again once every wave is here
        for (int i = threadIdx.x; i < T * TG * 64; i += kThreads) {
            const int l = i & 63, tg = (i >> 6) % TG, t = (i >> 6) / TG;
            const int col = l & 15, tok = 4 * tg + (l >> 4);
            const int64_t m = (int64_t)(grp * T + t) * ROWS + (SW ? col & 7 : col);
            if (m >= M || tok >= N || (SW && col >= 8)) continue;
            float s = 0.0f, u = 0.0f;
            for (int k = 0; k < S; ++k) {
                s += red[parity][t * S + k][tg][l];
                if constexpr (SW) u += red[parity][t * S + k][tg][l + 8];
            }
            Y[(uint64_t)tok * y_pitch + m] = SW ? rt_swish(s) * u : s;
        }
    }
}

typedef void (*Kernel)(MxArgs);
template <bool SW>
Kernel pick(int qu, int tg)
{
    if (tg == 1) return qu == 4 ? gemv_mx_kernel<4, 1, SW> : qu == 2 ? gemv_mx_kernel<2, 1, SW> : gemv_mx_kernel<1, 1, SW>;
    return qu == 4 ? gemv_mx_kernel<4, 2, SW> : qu == 2 ? gemv_mx_kernel<2, 2, SW> : gemv_mx_kernel<1, 2, SW>;
}

hipError_t launch(const GemvTask *tasks, const WeightView *up, int count, hipStream_t stream)
{
    const int64_t K = tasks[0].w.K, N = tasks[0].x.N;
    const bool sw = up != nullptr;
    const int rows = sw ? 8 : 16;
    int64_t tiles = 0;
    for (int i = 0; i < count; ++i) tiles += (tasks[i].w.M + rows - 1) / rows;
    if (tiles == 0 || N == 0) return hipSuccess;
    const int64_t units = (K + 127) / 128;
    // Large quanta (one scale load per four units) unless the tiles are too
    // few to give every CU a workgroup with K in fewer pieces.
    int qu = 4, s_log2 = 0;
    auto quanta = [&](int q) { return (units + q - 1) / q; };
    auto grow = [&] {
        s_log2 = 0;
        while (s_log2 < 4 && (2 << s_log2) <= quanta(qu)) {
            ++s_log2;
        }
    };
    grow();
    while (qu > 1 && tiles * (1 << s_log2) < 256 * kWaves && s_log2 < 4) {
        qu /= 2;
        grow();
    }
    // a pass over K holds at least one quantum of every wave of a tile
    while (((int64_t)qu << s_log2) * 4 * kImageBytes * N > kImageMax) {
        if (qu > 1) qu /= 2;
        else --s_log2;
    }
    MxArgs a = {};
    a.N = (int32_t)N;
    a.nb = (int32_t)(K / 32);
    a.qoff = (int32_t)quant_offset(K, 1);
    a.nq = (int32_t)quanta(qu);
    a.s_log2 = s_log2;
    const int S = 1 << s_log2, T = kWaves >> s_log2;
    const int64_t q_bytes = (int64_t)qu * 4 * kImageBytes * N;
    int64_t pass = kImageMax / q_bytes / S * S;
    a.pass_q = (int32_t)(pass < a.nq ? pass : (a.nq > 0 ? a.nq : 1));
    const int lds = (int)(a.pass_q * q_bytes);
    const int64_t cap = 2 * (int64_t)device_cus();
    int64_t total = 0, widest = 0;
    for (int i = 0; i < count; ++i) total += ((tasks[i].w.M + rows - 1) / rows + T - 1) / T;
    int n = 0;
    for (int i = 0; i < count; ++i) {
        if (tasks[i].w.M == 0) continue;
        MxItem &it = a.item[n++];
        it.w = tasks[i].w.base;
        it.pitch = (uint32_t)tasks[i].w.pitch;
        it.w2 = sw ? up->base : it.w;
        it.pitch2 = sw ? (uint32_t)up->pitch : it.pitch;
        it.x = static_cast<const float *>(tasks[i].x.data);
        it.x_pitch = (uint32_t)tasks[i].x.pitch_elems;
        it.y = tasks[i].y.data;
        it.y_pitch = (uint32_t)tasks[i].y.pitch_elems;
        it.M = (int32_t)tasks[i].w.M;
        it.n_groups = (int32_t)(((tasks[i].w.M + rows - 1) / rows + T - 1) / T);
        int64_t wgs = it.n_groups;
        if (total > cap) {
            wgs = wgs * cap / total;
            if (wgs < 1) wgs = 1;
        }
        it.wgs = (int32_t)wgs;
        if (wgs > widest) widest = wgs;
    }
    const Kernel k = sw ? pick<true>(qu, N > 4 ? 2 : 1) : pick<false>(qu, N > 4 ? 2 : 1);
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(k), kImageMax + 32 * 1024);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k, dim3((unsigned)widest, (unsigned)n), dim3(kThreads), (unsigned)lds, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemv_mx(const GemvTask *tasks, int count, hipStream_t stream)
{
    if (count < 1 || count > QMM_GEMV_BATCH_MAX) return hipErrorInvalidValue;
    return launch(tasks, nullptr, count, stream);
}

hipError_t launch_gemv_mx_swiglu(const WeightView &wg, const WeightView &wu, const ActView &x, const OutView &h,
                                 hipStream_t stream)
{
    const GemvTask t{wg, x, h};
    return launch(&t, &wu, 1, stream);
}

}  // namespace qmm
