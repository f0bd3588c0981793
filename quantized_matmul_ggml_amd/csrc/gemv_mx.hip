// gemv_mx.hip -- decode GEMV for MXFP4 weights and 1 to 8 fp32 tokens on the
// bf16 matrix cores, alone, batched, or as the gate/up pair fused with SwiGLU.
//
// y[n][m] = sum_k W'[m][k] x[n][k] (A Complete Guide to llama.cpp and
// Customization with C++, §2.1: at one token per step every projection is a
// GEMV, bound by the weight stream), with the arithmetic of row_tiles.h: every
// product is exact and only the binary32 accumulation rounds.
//
// Work split: a workgroup of W waves covers W / S tiles of 16 weight rows, S
// waves sharing a tile's K, one run of 64-byte units each; where that leaves
// the chip idle a tile has eight rows and a wave takes two units of each at
// once (HALF, row_tiles.h).  The first units of every wave are in flight while
// the workgroup splits its tokens into the LDS image, and those of its next
// tile while the S partial sums of this one meet in LDS, where they are added
// in wave order.
//
// 32000 x 2048, one token: 8.3 us for 34.8 MB (a bare read of them: 7.7).
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
    int32_t N;                // tokens
};
static_assert(sizeof(MxItem) == 64, "one 64-byte record per item");

struct MxArgs {
    int32_t nb;               // 32-blocks per row
    int32_t qoff;
    int32_t steps;            // units (HALF: pairs of units) per row
    int32_t s_log2;           // waves per tile
    int32_t pass;             // steps per pass over K (a multiple of S, or all)
    int32_t pad[11];
    MxItem item[QMM_GEMV_BATCH_MAX];
};

template <int TG, bool SW, bool HALF, int D>
__global__ __launch_bounds__(1024) void gemv_mx_kernel(const MxArgs a)
{
    constexpr int WT = W_MXFP4, SS = 0;
    constexpr int QB = RowFmt<WT, SS>::MF;                 // blocks (and instructions) per unit
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
    const int N = it.N, nb = a.nb, qoff = a.qoff, steps = a.steps, s_log2 = a.s_log2, pass = a.pass;
    if ((int)blockIdx.x >= wgs) return;

    const int threads = blockDim.x, waves = threads >> 6;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, g = lane >> 4;
    const bool upper = j >= 8;
    const int S = 1 << s_log2, T = waves >> s_log2;
    const int split = wave & (S - 1), tile_in = wave >> s_log2;
    float *const red = reinterpret_cast<float *>(lds);     // [2][waves][TG][64]
    uint8_t *const scales = lds + 2 * waves * TG * 64 * 4 + wave * kScaleLds;
    uint8_t *const img = lds + waves * (2 * TG * 64 * 4 + kScaleLds);

    // ---- the rows of a tile: columns of the gate or up matrix; rows past M
    // repeat the last one and are not stored ----
    auto unit = [&](int p) { return HALF ? 2 * p + (upper ? 1 : 0) : p; };
    auto whole = [&](int p) { return (p + 1) * SB <= nb; };
    Unit<WT, SS> z[D];
    ScaleWindow<WT, SS, HALF, D> window;
    // The wave's run of steps in a pass of len steps from p0 on: its first, and
    // their number.
    auto per_wave = [&](int len) { return (len + S - 1) >> s_log2; };
    auto first = [&](int p0, int len) { return p0 + split * per_wave(len); };
    auto share = [&](int len) {
        const int left = len - split * per_wave(len);
        return left < 0 ? 0 : left < per_wave(len) ? left : per_wave(len);
    };
    auto pass_len = [&](int p0) { return p0 + pass < steps ? pass : steps - p0; };
    // the lane's row of a tile (HALF: columns j and j + 8 are halves of one)
    auto tile_row = [&](int grp) {
        const int64_t r = (int64_t)(grp * T + tile_in) * ROWS + (ROWS == 8 ? j & 7 : j);
        return (SW && upper ? W2 : W) + (uint64_t)(r < M ? r : M - 1) * (SW && upper ? pitch2 : pitch);
    };
    auto load = [&](const uint8_t *r, int from) {
        return [&, r, from](auto d, int k) { load_codes<WT, SS>(z[d.value], r, qoff, 16 * nb, unit(from + k), g); };
    };
    auto load_scales = [&](const uint8_t *r, int p) {
        window.load(r, qoff + 16 * nb, p, g, upper);
        __builtin_amdgcn_sched_barrier(0);
    };
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
    if (steps > 0) {
        const int len = pass_len(0), from = first(0, len);
        const uint8_t *const r = tile_row(grp);
        image_ahead<WT>(ahead, N, 0, len * SB, nb, threads, row);
        load_scales(r, from);
        stream_begin<0, 1>(share(len), load(r, from));
        build_image<WT, true>(img, N, 0, len * SB, nb, threads, row, ahead);
        stream_begin<1, D>(share(len), load(r, from));
        __syncthreads();
    }
    int parity = 0;
    for (const int grp0 = grp; grp < n_groups; grp += wgs, parity ^= 1) {
        RowAcc<WT, HALF> acc[TG];
        for (int p0 = 0, p1; p0 < steps; p0 = p1) {
            const int len = pass_len(p0), from = first(p0, len);
            p1 = p0 + len;
            if (pass < steps && (grp > grp0 || p0 > 0)) {
                __syncthreads();                   // the last pass's image is no longer read
                build_image<WT, false>(img, N, p0 * SB, len * SB, nb, threads, row, ahead);
                __syncthreads();
            }
            const uint8_t *const r = tile_row(grp);
            stream<D>(share(len), [&](auto more, int i) {
                window.put(scales, j, g);
                if constexpr (more.value) load_scales(r, from + i);
            }, load(r, from), [&](auto d, int k) {
                const int p = from + k;
                const uint8_t *base = img + (uint32_t)((p - p0) * SB) * block_bytes;
                window.get(z[d.value], scales, d.value, j);
                multiply_unit<WT, SS, TG, HALF>(z[d.value], unit(p), whole(p), nb, g, upper, TG, acc,
                                                       [&](int tg, int h, int step) {
                    return *reinterpret_cast<const rt_bf16x8 *>(base + (uint32_t)(h * QB + step) * block_bytes + frag_off[tg]);
                });
            });
            const bool same = p1 < steps;
            if (same || grp + wgs < n_groups) {
                const int p = same ? p1 : 0, next_len = pass_len(p), next = first(p, next_len);
                const uint8_t *const n = tile_row(same ? grp : grp + wgs);
                load_scales(n, next);
                stream_begin<0, D>(share(next_len), load(n, next));
            }
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
template <int TG, bool SW, bool HALF>
Kernel pick(int depth)
{
    if (depth == 1) return gemv_mx_kernel<TG, SW, HALF, 1>;
    if (depth == 2) return gemv_mx_kernel<TG, SW, HALF, 2>;
    if constexpr (!HALF) {
        if (depth == 8) return gemv_mx_kernel<TG, SW, HALF, 8>;
    }
    return gemv_mx_kernel<TG, SW, HALF, 4>;
}

hipError_t launch(const GemvTask *tasks, const WeightView *up, int count, hipStream_t stream)
{
    const int64_t K = tasks[0].w.K, all = tasks[0].x.N;
    const bool sw = up != nullptr;
    int64_t M[QMM_GEMV_BATCH_MAX], rows = 0;
    for (int i = 0; i < count; ++i) rows += M[i] = tasks[i].w.M;
    if (rows == 0 || all == 0) return hipSuccess;
    const MxPlan p = plan_mx(M, count, K, all, sw);
    MxArgs a = {};
    a.nb = (int32_t)(K / 32);
    a.qoff = (int32_t)quant_offset(K, 1);
    a.steps = p.rows.steps;
    a.s_log2 = p.rows.s_log2;
    a.pass = p.pass;
    int64_t widest = 0;
    int n = 0;
    for (int i = 0; i < p.parts * count; ++i) {
        const GemvTask &t = tasks[i / p.parts];
        const int64_t from = p.N * (i % p.parts);
        if (t.w.M == 0 || from >= all) continue;
        MxItem &it = a.item[n++];
        it.w = t.w.base;
        it.pitch = (uint32_t)t.w.pitch;
        it.w2 = sw ? up->base : it.w;
        it.pitch2 = sw ? (uint32_t)up->pitch : it.pitch;
        it.x = static_cast<const float *>(t.x.data) + (uint64_t)from * t.x.pitch_elems;
        it.x_pitch = (uint32_t)t.x.pitch_elems;
        it.y = t.y.data + (uint64_t)from * t.y.pitch_elems;
        it.y_pitch = (uint32_t)t.y.pitch_elems;
        it.M = (int32_t)t.w.M;
        it.N = (int32_t)(all - from < p.N ? all - from : p.N);
        it.n_groups = (int32_t)(((t.w.M + p.tile_rows - 1) / p.tile_rows + p.T - 1) / p.T);
        int64_t wgs = it.n_groups;
        if (p.groups > p.cap) {
            wgs = wgs * p.cap / p.groups;
            if (wgs < 1) wgs = 1;
        }
        it.wgs = (int32_t)wgs;
        if (wgs > widest) widest = wgs;
    }
    const Kernel k = p.rows.half ? pick<1, false, true>(p.depth)
                     : sw        ? (p.tg == 1 ? pick<1, true, false>(p.depth) : pick<2, true, false>(p.depth))
                                 : (p.tg == 1 ? pick<1, false, false>(p.depth) : pick<2, false, false>(p.depth));
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(k), kLdsMost);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k, dim3((unsigned)widest, (unsigned)n), dim3(64 * p.rows.waves), (unsigned)p.lds, stream, a);
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
