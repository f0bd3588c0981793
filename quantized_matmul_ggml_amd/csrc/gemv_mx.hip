// gemv_mx.hip -- decode GEMV for MXFP4 weights and 1 to 8 fp32 tokens on the
// bf16 matrix cores, alone, batched, or as the gate/up pair fused with SwiGLU.
//
// y[n][m] = sum_k W'[m][k] x[n][k] (A Complete Guide to llama.cpp and
// Customization with C++, §2.1: at one token per step every projection is a
// GEMV, bound by the weight stream), with the arithmetic of row_tiles.h: every
// product is exact and only the binary32 accumulation rounds.
//
// Work split: a workgroup of W waves covers W / S tiles of 16 weight rows, S
// waves sharing a tile's K in interleaved quanta of QU units (128 QU values of
// k, 64 QU code bytes of each row); where that leaves the chip idle a tile has
// eight rows and a wave takes two quanta of each at once (HALF, row_tiles.h).
// The first quanta of every wave are in flight while the workgroup splits its
// tokens into the LDS image, and those of its next tile while the S partial
// sums of this one meet in LDS, where they are added in wave order.
#include "row_tiles.h"

namespace qmm {
namespace {

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
    int32_t steps;            // quanta (HALF: pairs of quanta) per row
    int32_t s_log2;           // waves per tile
    int32_t pass;             // steps per pass over K (a multiple of S, or all)
    int32_t pad[10];
    MxItem item[QMM_GEMV_BATCH_MAX];
};

template <int QU, int TG, bool SW, bool HALF, int D>
__global__ __launch_bounds__(1024) void gemv_mx_kernel(const MxArgs a)
{
    constexpr int WT = W_MXFP4, SS = 0;
    constexpr int QB = QU * RowFmt<WT, SS>::MF;            // blocks (and instructions) per quantum
    constexpr int SB = QB * (HALF ? 2 : 1);                // per step
    constexpr int ROWS = SW || HALF ? 8 : 16;              // row indices per tile
    static_assert(!(SW && HALF), "a fused tile has its two matrices in the halves");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

    const MxItem &it = a.item[blockIdx.y];
    const uint8_t *const W = it.w, *const W2 = it.w2;
    const float *const X = it.x;
    float *const Y = it.y;
    const uint32_t pitch = it.pitch, pitch2 = it.pitch2, x_pitch = it.x_pitch, y_pitch = it.y_pitch;
    const int M = it.M, n_groups = it.n_groups, wgs = it.wgs;
    const int N = a.N, nb = a.nb, qoff = a.qoff, steps = a.steps, s_log2 = a.s_log2, pass = a.pass;
    if ((int)blockIdx.x >= wgs) return;

    const int threads = blockDim.x, waves = threads >> 6;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, g = lane >> 4;
    const bool upper = j >= 8;
    const int S = 1 << s_log2, T = waves >> s_log2;
    const int split = wave & (S - 1), tile_in = wave >> s_log2;
    float *const red = reinterpret_cast<float *>(lds);     // [2][waves][TG][64]
    uint8_t *const img = lds + 2 * waves * TG * 64 * 4;

    // ---- the rows of a tile: columns of the gate or up matrix; rows past M
    // repeat the last one and are not stored ----
    const int last_q = (nb - 1) / QB;
    auto quantum = [&](int p) { return HALF ? 2 * p + (upper ? 1 : 0) : p; };
    auto whole = [&](int p) { return (p + 1) * SB <= nb; };
    Quantum<WT, SS, QU> z[D];
    // the wave's k-th quantum from step p0 of tile group grp on
    auto load = [&](int grp, int p0) {
        return [&, grp, p0](auto d, int k) {
            // load_quantum's two rows: with one unit the lane's own (HALF:
            // the row its half is of), with two rows j % 8 of both halves
            auto at = [&](const uint8_t *base, uint32_t step, int64_t r) { return base + (uint64_t)(r < M ? r : M - 1) * step; };
            const int64_t r = (int64_t)(grp * T + tile_in) * ROWS + (j & 7);
            const bool own = QU == 1 && !HALF && upper;
            const uint8_t *row0 = SW && own ? at(W2, pitch2, r) : at(W, pitch, !SW && own ? r + 8 : r);
            const uint8_t *row1 = QU == 1 ? row0 : SW ? at(W2, pitch2, r) : at(W, pitch, r + 8);
            load_quantum<WT, SS, QU>(z[d.value], row0, row1, qoff, 16 * nb, quantum(p0 + split + k * S), last_q, g, upper);
        };
    };
    // its quanta in [p0, p1)
    auto share = [&](int p0, int p1) { return p0 + split < p1 ? (p1 - p0 - split + S - 1) >> s_log2 : 0; };
    // ---- activation fragments: matrix row 4 t + p is part p of token t ----
    uint32_t frag_off[TG];
#pragma unroll
    for (int tg = 0; tg < TG; ++tg) {
        const int tok = 4 * tg + (j >> 2), part = (j & 3) < 2 ? (j & 3) : 2;
        frag_off[tg] = (uint32_t)((tok < N ? tok : N - 1) * kImageBytes + 64 * part + 16 * g);
    }
    const uint32_t block_bytes = (uint32_t)N * kImageBytes;

    // ---- the first pass's activations, then the first weights ----
    auto row = [&](int t) { return X + (uint64_t)t * x_pitch; };
    int grp = blockIdx.x;
    ImageAhead ahead;
    const int p_end = pass < steps ? pass : steps;
    if (steps > 0) {
        image_ahead<WT>(ahead, N, 0, p_end * SB, nb, threads, row);
        stream_begin<0, 1>(share(0, p_end), load(grp, 0));
    }
    int parity = 0;
    bool built = false;
    for (; grp < n_groups; grp += wgs, parity ^= 1) {
        RowAcc<WT, HALF> acc[TG];
        for (int p0 = 0; p0 < steps; p0 += pass) {
            const int p1 = p0 + pass < steps ? p0 + pass : steps;
            if (!built || pass < steps) {
                if (built) {
                    __syncthreads();               // the last pass's image is no longer read
                    build_image<WT, false>(img, N, p0 * SB, (p1 - p0) * SB, nb, threads, row, ahead);
                } else {
                    build_image<WT, true>(img, N, p0 * SB, (p1 - p0) * SB, nb, threads, row, ahead);
                    stream_begin<1, D>(share(p0, p1), load(grp, p0));
                }
                built = true;
                __syncthreads();
            }
            stream<D>(share(p0, p1), load(grp, p0), [&](auto d, int k) {
                const int p = p0 + split + k * S;
                const uint8_t *base = img + (uint32_t)((p - p0) * SB) * block_bytes;
                multiply_quantum<WT, SS, QU, TG, HALF>(z[d.value], quantum(p), whole(p), nb, g, upper, TG, acc,
                                                       [&](int tg, int h, int step) {
                    return *reinterpret_cast<const rt_bf16x8 *>(base + (uint32_t)(h * QB + step) * block_bytes + frag_off[tg]);
                });
            });
            const int next = p1 < steps ? p1 : 0, next_end = next + pass < steps ? next + pass : steps;
            stream_begin<0, D>(share(next, next_end), load(p1 < steps ? grp : grp + wgs, next));
        }
        float *const mine = red + parity * waves * TG * 64;
#pragma unroll
        for (int tg = 0; tg < TG; ++tg) mine[(wave * TG + tg) * 64 + lane] = row_total(acc[tg], upper);
        __syncthreads();
        // the other parity's sums are read no more once every wave is here
        for (int i = threadIdx.x; i < T * TG * 64; i += threads) {
            const int l = i & 63, tg = (i >> 6) % TG, t = (i >> 6) / TG;
            const int col = l & 15, tok = 4 * tg + (l >> 4);
            const int64_t m = (int64_t)(grp * T + t) * ROWS + col;
            if (col >= ROWS || m >= M || tok >= N) continue;
            float s = 0.0f, u = 0.0f;
            for (int k = 0; k < S; ++k) {
                const float *part = mine + ((t * S + k) * TG + tg) * 64 + l;
                s += part[0];
                if constexpr (SW || HALF) u += part[8];
            }
            Y[(uint64_t)tok * y_pitch + m] = SW ? rt_swish(s) * u : HALF ? s + u : s;
        }
    }
}

typedef void (*Kernel)(MxArgs);
// depth: quanta of one wave and pass over K; with one or two there is nothing to
// load ahead.
template <int QU, int TG, bool SW, bool HALF>
Kernel pick_depth(int depth)
{
    constexpr int D = QU == 1 ? 4 : 3;
    return depth >= 3 ? gemv_mx_kernel<QU, TG, SW, HALF, D>
                      : depth == 2 ? gemv_mx_kernel<QU, TG, SW, HALF, 2> : gemv_mx_kernel<QU, TG, SW, HALF, 1>;
}
template <int TG, bool SW>
Kernel pick(int qu, int depth)
{
    return qu == 2 ? pick_depth<2, TG, SW, false>(depth) : pick_depth<1, TG, SW, false>(depth);
}

hipError_t launch(const GemvTask *tasks, const WeightView *up, int count, hipStream_t stream)
{
    const int64_t K = tasks[0].w.K, N = tasks[0].x.N;
    const bool sw = up != nullptr;
    int64_t full = 0, half = 0;
    for (int i = 0; i < count; ++i) {
        full += (tasks[i].w.M + 15) / 16;
        half += (tasks[i].w.M + 7) / 8;
    }
    if (half == 0 || N == 0) return hipSuccess;
    const RowPlan p = plan_rows((K + 127) / 128, 4, sw ? half : full, sw ? 0 : half, (int)N, (int)N);
    const int rows = sw || p.half ? 8 : 16, T = p.waves >> p.s_log2, tg = N > 4 ? 2 : 1;
    MxArgs a = {};
    a.N = (int32_t)N;
    a.nb = (int32_t)(K / 32);
    a.qoff = (int32_t)quant_offset(K, 1);
    a.steps = p.steps;
    a.s_log2 = p.s_log2;
    a.pass = pass_steps(p.image, p.step_bytes, (int)N, p.s_log2, p.steps);
    const int lds = 2 * p.waves * tg * 64 * 4 + p.image;
    // as many workgroups as the CUs hold at once stream the tiles between them
    const int per_cu = 16 / p.waves;
    const int64_t cap = (int64_t)per_cu * device_cus();
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
    const int depth = (a.pass + (1 << p.s_log2) - 1) >> p.s_log2;
    const Kernel k = p.half ? pick_depth<1, 1, false, true>(depth)
                     : sw   ? (tg == 1 ? pick<1, true>(p.qu, depth) : pick<2, true>(p.qu, depth))
                            : (tg == 1 ? pick<1, false>(p.qu, depth) : pick<2, false>(p.qu, depth));
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(k), 128 * 1024);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k, dim3((unsigned)widest, (unsigned)n), dim3(64 * p.waves), (unsigned)lds, stream, a);
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
