// moe.hip -- mixture-of-experts layer for a few tokens: the router's choice,
// and the chosen experts' SwiGLU feed-forward blocks.
//
// The feed-forward block of one expert is that of the Development Guide for
// Small AI Models (TinyLLaMA, etc.) Using C++, §4.4 (SwiGLU(x) =
// Swish(x W_gate) * (x W_up), then the down projection); a layer has E of them
// and each token uses the k its router chose:
//   y[n] = sum_s p[n][s] Wd_e (Swish(Wg_e x[n]) * (Wu_e x[n])),  e = ids[n][s].
//
// For one to eight tokens the run time is the time to stream the chosen
// experts' weights (A Complete Guide to llama.cpp and Customization with C++,
// §2.1), so each chosen expert is read once, whatever the number of tokens
// that share it, in two launches with the arithmetic of row_tiles.h:
//
//  * moe_up_kernel: grid (tile groups, pairs).  A pair is a (token, slot);
//    the first pair that names an expert is its leader and does the work of
//    all tokens that chose it, the workgroups of the others leave at once.
//    h = Swish(gate) * up, times the token's weight for the expert (so that
//    the second launch only adds), goes to the workspace as the three bf16
//    parts of row_tiles.h, in the order the matrix instructions read them.
//  * moe_down_kernel: one workgroup per 16 output rows.  Its sixteen waves
//    share the quanta of all leaders' down rows; since the weights are already
//    in h, the experts' products add up in the same accumulators.  The waves'
//    sums are added in wave order, so results do not depend on timing.
#include "row_tiles.h"

namespace qmm {
namespace {

constexpr int kWaves = 16;            // of moe_down_kernel's workgroups
constexpr int kThreads = 64 * kWaves;
constexpr int kPairs = QMM_MOE_MAX_TOKENS * QMM_MOE_MAX_TOP_K;
static_assert(kPairs == 128, "two pairs per lane of a wave");

// ---------------------------------------------------------------- router
//
// One wave per token: lane l holds the logits l, l + 64, ...  The k largest
// are taken one at a time (wave-wide maximum, then the lowest index that has
// it), so the order is by logit and ties go to the lowest expert.  The whole
// softmax needs one more wave sum.  Bound by launch latency for a few tokens
// and by the k dependent wave reductions for many.

__device__ inline float wave_max(float v)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
    return v;
}
__device__ inline float wave_sum(float v)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

template <int R>
__global__ __launch_bounds__(256) void moe_route_kernel(const float *logits, uint64_t pitch, int64_t N, int E, int k,
                                                        int all, int32_t *ids, float *weights)
{
    const int lane = threadIdx.x & 63;
    const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (n >= N) return;
    const float *l = logits + (uint64_t)n * pitch;
    float v[R];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int e = lane + 64 * i;
        const float x = e < E ? l[e] : -INFINITY;
        v[i] = x > -INFINITY ? x : -INFINITY;       // a NaN is masked too
        top = fmaxf(top, v[i]);
    }
    top = wave_max(top);
    // e^(v - top); an infinite largest logit weighs 1 against 0 for the rest
    auto weigh = [&](float x) { return x == top ? 1.0f : expf(x - top); };
    float total = 0.0f;
    if (all) {
#pragma unroll
        for (int i = 0; i < R; ++i) total += v[i] > -INFINITY ? weigh(v[i]) : 0.0f;
        total = wave_sum(total);
    }
    // lane s keeps slot s
    int my_id = -1;
    float my_w = 0.0f, chosen = 0.0f;
    float best = top;
    for (int s = 0; s < k && best > -INFINITY; ++s) {
        int e = -1;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const uint64_t m = __ballot(v[i] == best);
            if (e < 0 && m != 0) e = 64 * i + __builtin_ctzll(m);
        }
        const float w = weigh(best);
        chosen += w;
        if (lane == s) {
            my_id = e;
            my_w = w;
        }
        float next = -INFINITY;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (e == lane + 64 * i) v[i] = -INFINITY;
            next = fmaxf(next, v[i]);
        }
        best = wave_max(next);
    }
    if (lane < k) {
        ids[n * k + lane] = my_id;
        weights[n * k + lane] = my_id < 0 ? 0.0f : my_w / (all ? total : chosen);
    }
}

// ---------------------------------------------------------- the experts

struct MoeArgs {
    const uint8_t *gate, *up, *down;
    uint64_t gate_pitch, up_pitch, down_pitch;       // bytes between rows
    uint64_t gate_expert, up_expert, down_expert;    // bytes between experts
    const float *x;
    float *y;
    uint64_t x_pitch, y_pitch;                       // elements
    const int32_t *ids;
    const float *weights;
    uint8_t *h;               // workspace: h_pair bytes per pair
    uint64_t h_pair;          // kImageBytes per 32-block of F, whole groups of four blocks
    int32_t E, N, k, F, M;    // M: output rows
    int32_t nb1, qoff1;       // gate / up rows: blocks, code offset
    int32_t nb2, qoff2;       // down rows
    int32_t steps1;           // moe_up_kernel: quanta per row, waves per tile,
    int32_t s_log2;           //   LDS bytes of the image
    int32_t image;
    int32_t steps2;           // moe_down_kernel: quanta (or pairs) per row
};

template <int WT, int SS, int QU, int TG>
__global__ __launch_bounds__(1024) void moe_up_kernel(const MoeArgs a)
{
    using F = RowFmt<WT, SS>;
    constexpr int QB = QU * F::MF;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ float pair_weight[kPairs];
    __shared__ float psum[8];
    __shared__ int slot_tok[8], slot_pair[8];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int P = a.N * a.k;
    const int pair = blockIdx.y;
    const int e = a.ids[pair];
    if (e < 0 || e >= a.E) return;                   // an empty slot
    // every pair that names this expert; the first of them leads
    const int id0 = lane < P ? a.ids[lane] : -1, id1 = lane + 64 < P ? a.ids[lane + 64] : -1;
    const uint64_t m0 = __ballot(id0 == e), m1 = __ballot(id1 == e);
    const int leader = m0 ? __builtin_ctzll(m0) : 64 + __builtin_ctzll(m1);
    if (leader != pair) return;

    const int j = lane & 15, g = lane >> 4;
    const int threads = blockDim.x, waves = threads >> 6;
    const int S = 1 << a.s_log2, T = waves >> a.s_log2;
    const int split = wave & (S - 1), tile_in = wave >> a.s_log2;
    const int grp = blockIdx.x;
    float *const red = reinterpret_cast<float *>(lds);     // [waves][TG][64]
    uint8_t *const img = lds + waves * TG * 64 * 4;

    // the first quantum is in flight while the tokens are set up
    const bool upper = j >= 8;
    const uint8_t *const W = upper ? a.up + (uint64_t)e * a.up_expert : a.gate + (uint64_t)e * a.gate_expert;
    const int r = (grp * T + tile_in) * 8 + (j & 7);
    const uint8_t *const row = W + (uint64_t)(r < a.F ? r : a.F - 1) * (upper ? a.up_pitch : a.gate_pitch);
    const int code_bytes = F::BB * a.nb1;
    Quantum<WT, SS, QU> cur, nxt;
    auto whole = [&](int q) { return (q + 1) * QB <= a.nb1; };
    if (split < a.steps1) load_quantum<WT, SS, QU>(cur, row, a.qoff1, code_bytes, split, g, whole(split));

    // ---- the tokens: bit t of `toks`; thread t adds up the weights of token
    // t's slots in slot order (a token may name an expert twice) ----
    if (wave == 0) {
        if (lane < P) pair_weight[lane] = id0 == e ? a.weights[lane] : 0.0f;
        if (lane + 64 < P) pair_weight[lane + 64] = id1 == e ? a.weights[lane + 64] : 0.0f;
    }
    uint32_t toks = 0;
    for (int t = 0; t < a.N; ++t) {                  // N <= 8
        const int b = t * a.k, c = b + a.k;          // pairs b .. c - 1
        auto bits = [&](uint64_t m, int base) -> uint64_t {
            const int lo = b - base < 0 ? 0 : b - base, hi = c - base > 64 ? 64 : c - base;
            if (lo >= hi) return 0;
            return (m >> lo) & (hi - lo == 64 ? ~0ull : (1ull << (hi - lo)) - 1);
        };
        if (bits(m0, 0) | bits(m1, 64)) toks |= 1u << t;
    }
    const int cnt = __builtin_popcount(toks);
    __syncthreads();
    if (threadIdx.x < 8 && (toks >> threadIdx.x & 1)) {
        const int t = threadIdx.x, slot = __builtin_popcount(toks & ((1u << t) - 1));
        const int b = t * a.k;
        float p = 0.0f;
        for (int s = 0; s < a.k; ++s) p += pair_weight[b + s];
        psum[slot] = p;
        slot_tok[slot] = t;
        // the token's first pair: the lowest set bit from b on
        const uint64_t low = b < 64 ? m0 >> b : 0;
        slot_pair[slot] = low ? b + __builtin_ctzll(low)
                              : b > 64 ? b + __builtin_ctzll(m1 >> (b - 64)) : 64 + __builtin_ctzll(m1);
    }
    __syncthreads();

    uint32_t frag_off[TG];
#pragma unroll
    for (int tg = 0; tg < TG; ++tg) {
        const int tok = 4 * tg + (j >> 2), part = (j & 3) < 2 ? (j & 3) : 2;
        frag_off[tg] = (uint32_t)((tok < cnt ? tok : cnt - 1) * kImageBytes + 64 * part + 16 * g);
    }
    const uint32_t step_bytes = (uint32_t)cnt * kImageBytes;
    const int groups = __builtin_amdgcn_readfirstlane(cnt > 4 ? 2 : 1);

    RowAcc<WT, false> acc[TG];
    const int pass = pass_steps(a.image, QB * kImageBytes, cnt, a.s_log2, a.steps1);
    for (int q0 = 0; q0 < a.steps1; q0 += pass) {
        const int q1 = q0 + pass < a.steps1 ? q0 + pass : a.steps1;
        if (q0 > 0) __syncthreads();
        build_image<WT>(img, cnt, q0 * QB, (q1 - q0) * QB, a.nb1, threads,
                        [&](int t) { return a.x + (uint64_t)slot_tok[t] * a.x_pitch; });
        __syncthreads();
        for (int q = q0 + split; q < q1; q += S) {
            if (q + S < a.steps1) load_quantum<WT, SS, QU>(nxt, row, a.qoff1, code_bytes, q + S, g, whole(q + S));
            const uint8_t *base = img + (uint32_t)((q - q0) * QB) * step_bytes;
            multiply_quantum<WT, SS, QU, TG, false>(cur, q, whole(q), a.nb1, g, upper, groups, acc, [&](int tg, int, int step) {
                return *reinterpret_cast<const rt_bf16x8 *>(base + (uint32_t)step * step_bytes + frag_off[tg]);
            });
            cur = nxt;
        }
    }
#pragma unroll
    for (int tg = 0; tg < TG; ++tg) red[(wave * TG + tg) * 64 + lane] = row_total(acc[tg], upper);
    __syncthreads();
    // ---- h = Swish(gate) * up * weight, one thread per (row, token) ----
    for (int i = threadIdx.x; i < T * cnt * 8; i += threads) {
        const int rr = i & 7, t = (i >> 3) / cnt, slot = (i >> 3) % cnt;
        const int f = (grp * T + t) * 8 + rr;
        if (f >= a.F) continue;
        const int tg = slot >> 2, l = 16 * (slot & 3) + rr;
        float s = 0.0f, u = 0.0f;
        for (int w = 0; w < S; ++w) {
            const float *part = red + ((t * S + w) * TG + tg) * 64 + l;
            s += part[0];
            u += part[8];
        }
        const float hv = rt_swish(s) * u * psum[slot];
        // its place among the parts: block f / 32, element f % 32
        const int b = f >> 5, el = f & 31;
        int q, idx;
        if (WT == W_Q8_0) {
            const int o = el >> 3;                   // octets 0, 1, 2, 3 sit in quarters 0, 2, 1, 3
            q = o == 1 ? 2 : o == 2 ? 1 : o;
            idx = el & 7;
        } else {
            q = (el & 15) >> 2;
            idx = 2 * (el & 3) + (el >> 4);
        }
        const uint32_t hb = __builtin_bit_cast(uint32_t, hv);
        const bool special = (hb & 0x7F800000u) == 0x7F800000u;
        const uint32_t hi = (hb & 0x7FFFFFFFu) > 0x7F800000u ? 0x7FC00000u : hb & 0xFFFF0000u;
        float r1 = hv - __builtin_bit_cast(float, hb & 0xFFFF0000u);
        r1 = special ? 0.0f : r1;
        const uint32_t mid = __builtin_bit_cast(uint32_t, r1) & 0xFFFF0000u;
        const uint32_t lo = __builtin_bit_cast(uint32_t, r1 - __builtin_bit_cast(float, mid));
        uint16_t *dst = reinterpret_cast<uint16_t *>(a.h + (uint64_t)slot_pair[slot] * a.h_pair +
                                                     (uint64_t)image_step<WT>(b, q) * kImageBytes +
                                                     16 * image_group<WT>(b, q)) + idx;
        dst[0] = (uint16_t)(hi >> 16);
        dst[32] = (uint16_t)(mid >> 16);
        dst[64] = (uint16_t)(lo >> 16);
    }
}

template <int WT, int SS, int QU, int TG, bool HALF>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(const MoeArgs a)
{
    using F = RowFmt<WT, SS>;
    constexpr int QB = QU * F::MF, H = HALF ? 2 : 1, SB = QB * H;
    constexpr int ROWS = HALF ? 8 : 16;
    __shared__ float red[kWaves][TG][64];
    __shared__ __attribute__((aligned(16))) int ids[kPairs];
    __shared__ int lead_pos[kPairs];             // a leader pair's place in the list
    __shared__ int lead_id[kPairs];
    __shared__ int16_t tok_pair[kPairs][8];      // the pair that holds (leader, token)'s h, or -1
    __shared__ int n_lead;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int P = a.N * a.k;
    // ---- the chosen experts, in the order of their first pair ----
    if (tid < kPairs) {
        const int v = tid < P ? a.ids[tid] : -1;
        ids[tid] = v >= 0 && v < a.E ? v : -1;
    }
    reinterpret_cast<int *>(tok_pair)[tid & 511] = -1;      // 512 dwords
    static_assert(sizeof(tok_pair) == 4 * 512 && kThreads >= 512, "cleared in one go");
    __syncthreads();
    int first = -1, first_tok = -1;
    if (tid < P && ids[tid] >= 0) {
        const int v = ids[tid], t0 = tid / a.k * a.k;
        // from the last pair down, so that the lowest match stays
#pragma unroll 4
        for (int c = (P - 1) >> 2; c >= 0; --c) {
            const int4 w = reinterpret_cast<const int4 *>(ids)[c];
            const int m[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 3; i >= 0; --i)
                if (m[i] == v) {
                    first = 4 * c + i;
                    if (4 * c + i >= t0) first_tok = 4 * c + i;
                }
        }
    }
    if (wave < 2) {
        const uint64_t lead = __ballot(tid < P && first == tid);
        // wave 1 counts wave 0's leaders through LDS below
        if (lane == 0) lead_id[kPairs - 1 - wave] = __builtin_popcountll(lead);
        if (tid < P && first == tid) lead_pos[tid] = __builtin_popcountll(lead & ((1ull << lane) - 1));
    }
    __syncthreads();
    const int c0 = lead_id[kPairs - 1], c1 = lead_id[kPairs - 2];
    __syncthreads();
    if (tid < P && first >= 0) {
        const int pos = lead_pos[first] + (first >= 64 ? c0 : 0);
        if (first == tid) lead_id[pos] = ids[tid];
        if (first_tok == tid) tok_pair[pos][tid / a.k] = (int16_t)tid;
    }
    if (tid == 0) n_lead = c0 + c1;
    __syncthreads();

    const int j = lane & 15, g = lane >> 4;
    const bool upper = j >= 8;
    const int r = (int)blockIdx.x * ROWS + (j & (ROWS - 1));
    const uint64_t row_off = (uint64_t)(r < a.M ? r : a.M - 1) * a.down_pitch;
    const int code_bytes = F::BB * a.nb2;
    const int items = __builtin_amdgcn_readfirstlane(n_lead) * a.steps2;
    const int part = (j & 3) < 2 ? (j & 3) : 2;
    const __amdgpu_buffer_rsrc_t hres = __builtin_amdgcn_make_buffer_rsrc(
        a.h, 0, (int)((uint32_t)P * (uint32_t)a.h_pair), BUFFER_FLAGS);
    auto quantum = [&](int p) { return HALF ? 2 * p + (upper ? 1 : 0) : p; };
    auto whole = [&](int p) { return (p + 1) * SB <= a.nb2; };
    auto load = [&](Quantum<WT, SS, QU> &z, int i) {
        const int li = i / a.steps2, p = i - li * a.steps2;
        const uint8_t *w = a.down + (uint64_t)__builtin_amdgcn_readfirstlane(lead_id[li]) * a.down_expert + row_off;
        load_quantum<WT, SS, QU>(z, w, a.qoff2, code_bytes, quantum(p), g, whole(p));
    };
    RowAcc<WT, HALF> acc[TG];
    Quantum<WT, SS, QU> cur, nxt;
    if (wave < items) load(cur, wave);
    for (int i = wave; i < items; i += kWaves) {
        if (i + kWaves < items) load(nxt, i + kWaves);
        const int li = i / a.steps2, p = i - li * a.steps2;
        const int blk0 = p * SB;
        // one token group after the other (only those with a token of this
        // expert): its fragments, blocks past the row and tokens without this
        // expert as zeros
#pragma unroll
        for (int tg = 0; tg < TG; ++tg) {
            const int pr = tok_pair[li][4 * tg + (j >> 2)];
            if (__ballot(pr >= 0) == 0) continue;
            const uint32_t off = (uint32_t)pr * (uint32_t)a.h_pair + (uint32_t)(64 * part + 16 * g);
            rt_bf16x8 fr[SB];
#pragma unroll
            for (int s = 0; s < SB; ++s) {
                // the block whose values this lane group feeds to instruction s
                const int b = WT == W_MXFP4 ? blk0 + (s & ~3) + g : blk0 + s;
                const uint32_t o = pr >= 0 && b < a.nb2 ? off + (uint32_t)(blk0 + s) * kImageBytes : OUT_OF_RANGE;
                fr[s] = __builtin_bit_cast(rt_bf16x8, __builtin_amdgcn_raw_buffer_load_b128(hres, o, 0, 0));
            }
            RowAcc<WT, HALF> one[1] = {acc[tg]};
            multiply_quantum<WT, SS, QU, 1, HALF>(cur, quantum(p), whole(p), a.nb2, g, upper, 1, one,
                                                  [&](int, int h, int s) { return fr[h * QB + s]; });
            acc[tg] = one[0];
        }
        cur = nxt;
    }
#pragma unroll
    for (int tg = 0; tg < TG; ++tg) red[wave][tg][lane] = row_total(acc[tg], upper);
    __syncthreads();
    if (tid < TG * 64) {
        const int l = tid & 63, tg = tid >> 6, col = l & 15;
        const int m = (int)blockIdx.x * ROWS + col, t = 4 * tg + (l >> 4);
        if (col < ROWS && m < a.M && t < a.N) {
            float s = 0.0f;
            for (int w = 0; w < kWaves; ++w) s += HALF ? red[w][tg][l] + red[w][tg][l + 8] : red[w][tg][l];
            a.y[(uint64_t)t * a.y_pitch + m] = s;
        }
    }
}

typedef void (*Kernel)(MoeArgs);
template <int WT, int SS, int TG>
void pick(int qu, bool half, Kernel *up, Kernel *down)
{
    *up = qu == 4 ? moe_up_kernel<WT, SS, 4, TG> : qu == 2 ? moe_up_kernel<WT, SS, 2, TG> : moe_up_kernel<WT, SS, 1, TG>;
    *down = half ? moe_down_kernel<WT, SS, 1, TG, true> : moe_down_kernel<WT, SS, 2, TG, false>;
}
template <int WT, int SS>
void pick(int qu, int tg, bool half, Kernel *up, Kernel *down)
{
    if (tg == 1) pick<WT, SS, 1>(qu, half, up, down);
    else pick<WT, SS, 2>(qu, half, up, down);
}

}  // namespace

hipError_t launch_moe_route(const float *logits, uint64_t pitch, int64_t N, int E, int k, bool all, int32_t *ids,
                            float *weights, hipStream_t stream)
{
    if (N == 0) return hipSuccess;
    const dim3 grid((unsigned)((N + 3) / 4)), block(256);
#define QMM_ROUTE(R) hipLaunchKernelGGL(moe_route_kernel<R>, grid, block, 0, stream, logits, pitch, N, E, k, (int)all, ids, weights)
    if (E <= 64) QMM_ROUTE(1);
    else if (E <= 128) QMM_ROUTE(2);
    else if (E <= 256) QMM_ROUTE(4);
    else QMM_ROUTE(16);
#undef QMM_ROUTE
    return hipGetLastError();
}

// Workspace bytes of one (token, slot) pair.
static uint64_t h_pair_bytes(int64_t F) { return (uint64_t)((F + 127) / 128) * 4 * kImageBytes; }

uint64_t moe_workspace(int64_t N, int64_t k, int64_t F)
{
    return (uint64_t)(N * k) * h_pair_bytes(F);
}

hipError_t launch_moe_swiglu(const ExpertView &gate, const ExpertView &up, const ExpertView &down, const ActView &x,
                             const int32_t *ids, const float *weights, int k, const OutView &y, void *ws,
                             hipStream_t stream)
{
    const int type = gate.w.type, ss = type == W_MXFP4 ? 0 : gate.w.scale_shift;
    const int64_t N = x.N, F = gate.w.M, M = down.w.M;
    const int kpu = type == W_Q8_0 ? 64 : 128;
    MoeArgs a = {};
    a.gate = gate.w.base;
    a.up = up.w.base;
    a.down = down.w.base;
    a.gate_pitch = gate.w.pitch;
    a.up_pitch = up.w.pitch;
    a.down_pitch = down.w.pitch;
    a.gate_expert = gate.expert_pitch;
    a.up_expert = up.expert_pitch;
    a.down_expert = down.expert_pitch;
    a.x = static_cast<const float *>(x.data);
    a.x_pitch = x.pitch_elems;
    a.y = y.data;
    a.y_pitch = y.pitch_elems;
    a.ids = ids;
    a.weights = weights;
    a.h = static_cast<uint8_t *>(ws);
    a.h_pair = h_pair_bytes(F);
    a.E = (int32_t)gate.E;
    a.N = (int32_t)N;
    a.k = k;
    a.F = (int32_t)F;
    a.M = (int32_t)M;
    a.nb1 = (int32_t)(gate.w.K / 32);
    a.qoff1 = (int32_t)quant_offset(gate.w.K, gate.w.scale_shift);
    a.nb2 = (int32_t)(F / 32);
    a.qoff2 = (int32_t)quant_offset(F, down.w.scale_shift);
    const int64_t units1 = (gate.w.K + kpu - 1) / kpu, units2 = (F + kpu - 1) / kpu;
    // about how many experts several tokens choose between them
    const int64_t experts = N < 2 ? k : N * k / 2 + 1 < gate.E ? N * k / 2 + 1 : gate.E;
    const int tg = N > 4 ? 2 : 1;
    const RowPlan p = plan_rows(units1, kpu / 32, (F + 7) / 8 * experts, 0, (int)N);
    a.steps1 = p.steps;
    a.s_log2 = p.s_log2;
    a.image = p.image;
    const int T = p.waves >> p.s_log2;
    const int lds = p.waves * tg * 64 * 4 + p.image;
    // tiles of eight output rows while sixteen would leave CUs without one
    const bool half = (M + 15) / 16 < 2 * (int64_t)device_cus();
    a.steps2 = (int32_t)((units2 + 1) / 2);

    Kernel ku = nullptr, kd = nullptr;
    if (type == W_MXFP4) pick<W_MXFP4, 0>(p.qu, tg, half, &ku, &kd);
    else if (type == W_Q4_0) ss ? pick<W_Q4_0, 1>(p.qu, tg, half, &ku, &kd) : pick<W_Q4_0, 0>(p.qu, tg, half, &ku, &kd);
    else if (type == W_Q8_0) ss ? pick<W_Q8_0, 1>(p.qu, tg, half, &ku, &kd) : pick<W_Q8_0, 0>(p.qu, tg, half, &ku, &kd);
    else return hipErrorInvalidValue;
    hipError_t e = hipSuccess;
    if (F > 0) {
        e = allow_dynamic_lds(reinterpret_cast<const void *>(ku), 128 * 1024);
        if (e != hipSuccess) return e;
        const unsigned groups = (unsigned)(((F + 7) / 8 + T - 1) / T);
        hipLaunchKernelGGL(ku, dim3(groups, (unsigned)(N * k)), dim3(64 * p.waves), (unsigned)lds, stream, a);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const unsigned tiles = (unsigned)(half ? (M + 7) / 8 : (M + 15) / 16);
    hipLaunchKernelGGL(kd, dim3(tiles), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace qmm
