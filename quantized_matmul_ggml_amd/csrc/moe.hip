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
// §2.1), so tokens that share an expert share its reads, in two launches with
// the arithmetic of row_tiles.h.  A pair is a (token, slot); an entry is an
// expert and one or two of the pairs that name it.
//
//  * moe_up_kernel: grid (tile groups, pairs).  The first, third, ... pair that
//    names an expert does the work of its entry, the workgroups of the others
//    leave at once.
//    h = Swish(gate) * up, times the token's weight for the expert (so that
//    the second launch only adds), goes to the workspace as the three bf16
//    parts of row_tiles.h, in the order the matrix instructions read them.
//  * moe_down_kernel: one workgroup per 8 output rows.  Its sixteen waves share
//    the units of all entries' down rows; the weights are already in h, so the
//    experts' products only add up, in a fixed order: results do not depend
//    on timing.
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
    int32_t steps1;           // moe_up_kernel: units per row, waves per tile,
    int32_t s_log2;           //   LDS bytes of the image
    int32_t image;
    int32_t steps2;           // moe_down_kernel: pairs of units per row
};

// A workgroup takes T tiles of eight rows of one expert and one or two of its
// pairs; an expert with more makes several, whose weights then come from the
// caches (with four pairs a workgroup the few experts that have them needed
// twice the LDS, took several passes over K, and finished last).
//
// Bound by the weight stream's loads: 42 of 64 experts of 1024 x 2048 (gate and
// up, 94 MB of MXFP4) for eight tokens take 24 us, the same loads alone 18.4;
// two experts of 5632 x 2048 Q4_0 (26 MB) for one token 12 us, of which 3 pass
// before the first product.  Workgroups that walk over several tile groups
// with one image were slower (33 us): few, long workgroups end unevenly.
template <int WT, int SS, int D>
__global__ __launch_bounds__(1024) void moe_up_kernel(const MoeArgs a)
{
    using F = RowFmt<WT, SS>;
    constexpr int QB = F::MF;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int P = a.N * a.k;
    const int pair = blockIdx.y;
    // every pair's expert, pairs `lane` and `lane + 64`
    const int id0 = lane < P ? a.ids[lane] : -1, id1 = lane + 64 < P ? a.ids[lane + 64] : -1;
    const int e = pair < 64 ? __builtin_amdgcn_readlane(id0, pair) : __builtin_amdgcn_readlane(id1, pair - 64);
    if (e < 0 || e >= a.E) return;                   // an empty slot
    // The pairs that name this expert, in order (a token that names an expert
    // twice has two); every second one leads, the next one is its mate.
    const uint64_t m0 = __ballot(id0 == e), m1 = __ballot(id1 == e);
    const uint64_t from0 = pair < 63 ? ~0ull << (pair + 1) : 0, from1 = pair < 64 ? ~0ull : pair < 127 ? ~0ull << (pair - 63) : 0;
    const int later = __builtin_popcountll(m0 & from0) + __builtin_popcountll(m1 & from1);
    const int rank = __builtin_popcountll(m0) + __builtin_popcountll(m1) - 1 - later;
    if (rank & 1) return;
    const int now = later ? 2 : 1;
    const int mate = m0 & from0 ? __builtin_ctzll(m0 & from0) : later ? 64 + __builtin_ctzll(m1 & from1) : pair;

    const int j = lane & 15, g = lane >> 4;
    const int threads = blockDim.x, waves = threads >> 6;
    const int S = 1 << a.s_log2, T = waves >> a.s_log2;
    const int split = wave & (S - 1), tile_in = wave >> a.s_log2;
    const int grp = blockIdx.x;
    float *const red = reinterpret_cast<float *>(lds);     // [waves][64]
    uint8_t *const scales = lds + waves * 64 * 4 + wave * kScaleLds;
    uint8_t *const img = lds + waves * (64 * 4 + kScaleLds);

    // ---- the activations and the first units of weights ----
    const bool upper = j >= 8;
    const int r = (grp * T + tile_in) * 8 + (j & 7), rc = r < a.F ? r : a.F - 1;
    const uint8_t *const row = upper ? a.up + (uint64_t)e * a.up_expert + (uint64_t)rc * a.up_pitch
                                     : a.gate + (uint64_t)e * a.gate_expert + (uint64_t)rc * a.gate_pitch;
    const int code_bytes = F::BB * a.nb1;
    auto whole = [&](int q) { return (q + 1) * QB <= a.nb1; };
    const int pass = pass_steps(a.image, QB * kImageBytes, now, a.s_log2, a.steps1);
    const float *const x0 = a.x + (uint64_t)(pair / a.k) * a.x_pitch, *const x1 = a.x + (uint64_t)(mate / a.k) * a.x_pitch;
    const float w0 = a.weights[pair], w1 = a.weights[mate];
    auto rows = [&](int place) { return place ? x1 : x0; };
    ImageAhead ahead;
    Unit<WT, SS> z[D];
    ScaleWindow<WT, SS, false, D> window;
    // The wave's run of units in a pass of len steps from q0 on: its first, and
    // their number.
    auto per_wave = [&](int len) { return (len + S - 1) >> a.s_log2; };
    auto first = [&](int q0, int len) { return q0 + split * per_wave(len); };
    auto share = [&](int len) {
        const int left = len - split * per_wave(len);
        return left < 0 ? 0 : left < per_wave(len) ? left : per_wave(len);
    };
    auto pass_len = [&](int q0) { return q0 + pass < a.steps1 ? pass : a.steps1 - q0; };
    auto load = [&](int from) {
        return [&, from](auto d, int k) { load_codes<WT, SS>(z[d.value], row, a.qoff1, code_bytes, from + k, g); };
    };
    auto load_scales = [&](int p) {
        window.load(row, a.qoff1 + code_bytes, p, g, upper);
        __builtin_amdgcn_sched_barrier(0);
    };
    if (a.steps1 > 0) {
        const int len = pass_len(0), from = first(0, len);
        image_ahead<WT>(ahead, now, 0, len * QB, a.nb1, threads, rows);
        load_scales(from);
        stream_begin<0, D - 1>(share(len), load(from));
        build_image<WT, true>(img, now, 0, len * QB, a.nb1, threads, rows, ahead);
        stream_begin<D - 1, D>(share(len), load(from));
        __syncthreads();
    }
    // columns of the activations' operand: four each for two tokens, three
    // parts and the last again; with one token it stands in both
    const uint32_t step_bytes = (uint32_t)now * kImageBytes;
    const uint32_t frag_off = (uint32_t)((j >> 2 & now - 1) * kImageBytes + ((j & 3) < 2 ? (j & 3) : 2) * 64 + 16 * g);
    RowAcc<WT, false> acc[1];
    for (int q0 = 0; q0 < a.steps1; q0 += pass) {
        const int len = pass_len(q0), from = first(q0, len);
        if (q0 > 0) {
            __syncthreads();                       // the last image is no longer read
            build_image<WT, false>(img, now, q0 * QB, len * QB, a.nb1, threads, rows, ahead);
            __syncthreads();
        }
        stream<D>(share(len), [&](auto more, int i) {
            window.put(scales, j, g);
            if constexpr (more.value) load_scales(from + i);
        }, load(from), [&](auto d, int k) {
            const int q = from + k;
            const uint8_t *at = img + (uint32_t)((q - q0) * QB) * step_bytes + frag_off;
            window.get(z[d.value], scales, d.value, j);
            multiply_unit<WT, SS, 1, false>(z[d.value], q, whole(q), a.nb1, g, upper, 1, acc, [&](int, int, int step) {
                return *reinterpret_cast<const rt_bf16x8 *>(at + (uint32_t)step * step_bytes);
            });
        });
        if (q0 + pass < a.steps1) {
            const int next_len = pass_len(q0 + pass), next = first(q0 + pass, next_len);
            load_scales(next);
            stream_begin<0, D>(share(next_len), load(next));
        }
    }
    red[wave * 64 + lane] = row_total(acc[0], upper);
    __syncthreads();
    // ---- h = Swish(gate) * up * weight, one thread per (row, place); the last
    // workgroup also clears the parts of the rows after F in the last group of
    // four blocks, which moe_down_kernel reads ----
    const int f_begin = grp * T * 8;
    const int f_end = grp == (int)gridDim.x - 1 ? (a.F + 127) / 128 * 128 : f_begin + T * 8;
    for (int i = threadIdx.x; i < (f_end - f_begin) * 2; i += threads) {
        const int place = i & 1, ff = i >> 1, f = f_begin + ff;
        if (place >= now) continue;
        const int home = place ? mate : pair;
        float hv = 0.0f;
        if (f < a.F) {
            const float *part = red + (ff >> 3) * S * 64 + 16 * place + (ff & 7);
            float s = 0.0f, u = 0.0f;
            for (int w = 0; w < S; ++w) {
                s += part[64 * w];
                u += part[64 * w + 8];
            }
            hv = rt_swish(s) * u * (place ? w1 : w0);
        }
        // its place among the parts: block f / 32, element f % 32
        const int b = f >> 5, el = f & 31;
        int q, idx;
        if (WT == W_Q8_0) {
            const int o = el >> 3;         // octets 0, 1, 2, 3 sit in quarters 0, 2, 1, 3
            q = o == 1 ? 2 : o == 2 ? 1 : o;
            idx = el & 7;
        } else {
            q = (el & 15) >> 2;
            idx = 2 * (el & 3) + (el >> 4);
        }
        // the three parts, as split_parts makes them
        auto top = [](float x) { return __builtin_bit_cast(uint32_t, x) >> 16; };
        auto rest = [&](float x) { return x - __builtin_bit_cast(float, top(x) << 16); };
        const float mid = fabsf(hv) == INFINITY ? 0.0f : rest(hv);
        uint16_t *dst = reinterpret_cast<uint16_t *>(a.h + (uint64_t)home * a.h_pair +
                                                     (uint64_t)image_step<WT>(b, q) * kImageBytes +
                                                     16 * image_group<WT>(b, q)) + idx;
        dst[0] = (uint16_t)top(hv);
        dst[32] = (uint16_t)top(mid);
        dst[64] = (uint16_t)top(rest(mid));
    }
}


// A tile is eight rows: columns 0 .. 7 of the matrix instruction hold unit
// 2 p of the rows, columns 8 .. 15 unit 2 p + 1, and likewise matrix rows
// 0 .. 7 the parts of two tokens' activations of unit 2 p and rows 8 .. 15
// those of unit 2 p + 1: the two diagonal quarters of D are the sums wanted.
// An entry is an expert and one or two of its pairs (an expert with more
// makes several, whose weights then come from the caches).  An item,
// one entry's pair of units, is loaded while the item before is multiplied:
// its weights, and its tokens' parts, which lie together in the workspace and
// go through a piece of LDS of the wave's own to reach their lanes (loaded
// fragment by fragment they were four times the load instructions, on the load
// path, which is the busiest part of the kernel as it is).
//
// The same 42 experts' 2048 x 1024 (47 MB) take 20 us: 6 before the first and
// after the last item, and of the rest half are the loads and half the
// products, which do not overlap as they should (of a CU's busy cycles the
// texture data unit is busy for 74 %, half of them waiting for the caches, the
// LDS for 34 %, the matrix cores for 7 %).  Waves that take runs of items
// instead of every sixteenth were slower (21.5 us), and so was binary32 h cut
// into parts here (20.2).
template <int WT, int SS>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(const MoeArgs a)
{
    using F = RowFmt<WT, SS>;
    constexpr int QB = F::MF, SB = 2 * QB;
    constexpr int CHUNK = SB * kImageBytes;      // a token's parts of one item
    constexpr int HALF_LDS = CHUNK / 2 + 128, TOK_LDS = 2 * HALF_LDS + 64;   // strides that spread the banks
    constexpr int NA = (2 * CHUNK + 1023) / 1024;          // 16-byte loads per lane for two tokens
    __shared__ __attribute__((aligned(16))) uint8_t parts[kWaves][2 * TOK_LDS];
    __shared__ float sums[kWaves][8][16];
    __shared__ __attribute__((aligned(16))) int ids[kPairs];
    __shared__ int4 entry[kPairs + 1];           // expert, its two pairs (-1: one only)
    __shared__ int count[2];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int P = a.N * a.k;
    if (tid < kPairs) {
        const int v = tid < P ? a.ids[tid] : -1;
        ids[tid] = v >= 0 && v < a.E ? v : -1;
    }
    for (int i = lane; i < 128; i += 64) (&sums[wave][0][0])[i] = 0.0f;
    __syncthreads();
    // ---- entries: every second pair of an expert starts one ----
    int rank = 0, mate = kPairs;
    const int mine_id = tid < P ? ids[tid] : -1;
    if (wave < 2) {
#pragma unroll 4
        for (int c = 0; c < (P + 3) >> 2; ++c) {
            const int4 w = reinterpret_cast<const int4 *>(ids)[c];
            const int m[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = 4 * c + i;
                rank += m[i] == mine_id && p < tid ? 1 : 0;
                mate = min(mate, m[i] == mine_id && p > tid ? p : kPairs);
            }
        }
    }
    const bool starts = mine_id >= 0 && (rank & 1) == 0;
    const uint64_t starting = __ballot(starts);
    if (wave < 2 && lane == 0) count[wave] = __builtin_popcountll(starting);
    __syncthreads();
    if (starts)
        entry[(wave ? count[0] : 0) + __builtin_popcountll(starting & ((1ull << lane) - 1))] =
            make_int4(mine_id, tid, mate < kPairs ? mate : -1, tid / a.k | (mate < kPairs ? mate / a.k : 0) << 8);
    const int entries = __builtin_amdgcn_readfirstlane(count[0] + count[1]);
    __syncthreads();

    const int j = lane & 15, g = lane >> 4;
    const bool upper = j >= 8;
    const int r = (int)blockIdx.x * 8 + (j & 7);
    const uint64_t row_off = (uint64_t)(r < a.M ? r : a.M - 1) * a.down_pitch;
    const int code_bytes = F::BB * a.nb2;
    const int items = entries * a.steps2;
    const int last_q = (a.nb2 - 1) / QB;
    const __amdgpu_buffer_rsrc_t hres = __builtin_amdgcn_make_buffer_rsrc(
        a.h, 0, (int)((uint32_t)P * (uint32_t)a.h_pair), BUFFER_FLAGS);
    constexpr int D = 2;                         // items in flight (three or four: no faster)
    uint4 part[D][NA];
    Unit<WT, SS> z[D];
    // The wave takes items wave, wave + 16, ...: entry n, step p.  Two cursors
    // follow them, one for the loads and one for the products.
    struct Cursor {
        int n, p;
    };
    const int steps2 = a.steps2 > 0 ? a.steps2 : 1;
    const Cursor stride = {kWaves / steps2, kWaves % steps2};
    auto advance = [&](Cursor &c) {
        c.n += stride.n;
        c.p += stride.p;
        if (c.p >= steps2) {
            c.p -= steps2;
            ++c.n;
        }
    };
    Cursor loads = {wave / steps2, wave % steps2}, products = loads;
    // the wave's next item: its activations, then its weights, both in flight
    // (past the last item the last entry again, unused)
    auto load = [&](auto d, int) {
        const int n = loads.n < entries ? loads.n : entries - 1, p = loads.p;
        advance(loads);
        const int4 en = entry[n];
#pragma unroll
        for (int k = 0; k < NA; ++k) {
            const int at = 1024 * k + 16 * lane;             // within the two tokens' chunks
            const int tok = at >= CHUNK ? 1 : 0;
            const uint32_t off = (uint32_t)(p * CHUNK + at - tok * CHUNK);
            const int pr = tok ? en.z : en.y;
            const bool in = pr >= 0 && at < 2 * CHUNK && off < (uint32_t)a.h_pair;
            part[d.value][k] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                hres, in ? (uint32_t)pr * (uint32_t)a.h_pair + off : OUT_OF_RANGE, 0, 0));
        }
        const uint8_t *w = a.down + (uint64_t)__builtin_amdgcn_readfirstlane(en.x) * a.down_expert + row_off;
        load_unit<WT, SS>(z[d.value], w, a.qoff2, code_bytes, 2 * p + (upper ? 1 : 0), last_q, g);
    };
    const uint32_t frag_off = (uint32_t)((j >> 2 & 1) * TOK_LDS + (j >> 3) * HALF_LDS + ((j & 3) < 2 ? (j & 3) : 2) * 64 + 16 * g);
    uint8_t *const mine = parts[wave];
    const int share = wave < items ? (items - wave + kWaves - 1) / kWaves : 0;
    if (items > 0) stream_begin<0, D>(share, load);
    stream<D>(share, [](auto, int) {}, load, [&](auto d, int) {
        // this item's parts to their lanes (the wave's own LDS: its reads and
        // writes stay in order)
#pragma unroll
        for (int k = 0; k < NA; ++k) {
            const int at = 1024 * k + 16 * lane, tok = at >= CHUNK ? 1 : 0, in = at - tok * CHUNK;
            if (2 * CHUNK % 1024 == 0 || at < 2 * CHUNK)
                *reinterpret_cast<uint4 *>(mine + tok * TOK_LDS + (in >= CHUNK / 2 ? HALF_LDS - CHUNK / 2 : 0) + in) = part[d.value][k];
        }
        const int p = products.p;
        const int4 en = entry[products.n];
        advance(products);
        __builtin_amdgcn_wave_barrier();
        RowAcc<WT, false> acc[1];
        multiply_unit<WT, SS, 1, false>(z[d.value], 2 * p + (upper ? 1 : 0), (p + 1) * SB <= a.nb2, a.nb2, g, upper, 1, acc,
                                               [&](int, int, int s) {
            return *reinterpret_cast<const rt_bf16x8 *>(mine + (uint32_t)s * kImageBytes + frag_off);
        });
        __builtin_amdgcn_wave_barrier();
        // D's diagonal quarters: pair g & 1, half g >> 1.  One pair after the
        // other: both may be of one token.
        const float total = row_total(acc[0], upper);
        const bool mine_now = (g >> 1) == (j >> 3);
        if (mine_now && (g & 1) == 0) sums[wave][en.w & 255][j] += total;
        __builtin_amdgcn_wave_barrier();
        if (mine_now && (g & 1) == 1 && en.z >= 0) sums[wave][en.w >> 8][j] += total;
        __builtin_amdgcn_wave_barrier();
    });
    __syncthreads();
    if (tid < 64) {
        const int m = (int)blockIdx.x * 8 + (tid & 7), t = tid >> 3;
        if (m < a.M && t < a.N) {
            float s = 0.0f;
            for (int w = 0; w < kWaves; ++w) s += sums[w][t][tid & 7] + sums[w][t][8 + (tid & 7)];
            a.y[(uint64_t)t * a.y_pitch + m] = s;
        }
    }
}

typedef void (*Kernel)(MoeArgs);
template <int WT, int SS>
void pick(int depth, Kernel *up, Kernel *down)
{
    *up = depth == 8 ? moe_up_kernel<WT, SS, 8> : depth == 4 ? moe_up_kernel<WT, SS, 4> : moe_up_kernel<WT, SS, 2>;
    *down = moe_down_kernel<WT, SS>;
}

}  // namespace

hipError_t launch_moe_route(const float *logits, uint64_t pitch, int64_t N, int E, int k, bool all, int32_t *ids,
                            float *weights, hipStream_t stream)
{
    // 2^25 tokens (2^31 threads) per launch: see kMaxGridThreads
    constexpr int64_t MOST = 1ll << 25;
    for (; N > 0; N -= MOST, logits += MOST * pitch, ids += MOST * k, weights += MOST * k) {
        const int64_t n = N < MOST ? N : MOST;
        const dim3 grid((unsigned)((n + 3) / 4)), block(256);
#define QMM_ROUTE(R) hipLaunchKernelGGL(moe_route_kernel<R>, grid, block, 0, stream, logits, pitch, n, E, k, (int)all, ids, weights)
        if (E <= 64) QMM_ROUTE(1);
        else if (E <= 128) QMM_ROUTE(2);
        else if (E <= 256) QMM_ROUTE(4);
        else QMM_ROUTE(16);
#undef QMM_ROUTE
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
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
    const RowPlan p = plan_moe(gate.E, k, N, F, units1, kpu / 32);
    a.steps1 = p.steps;
    a.s_log2 = p.s_log2;
    a.image = p.image;
    const int T = p.waves >> p.s_log2;
    const int lds = moe_lds(p);
    a.steps2 = (int32_t)((units2 + 1) / 2);

    const int depth = moe_depth((p.steps + (1 << p.s_log2) - 1) >> p.s_log2);
    Kernel ku = nullptr, kd = nullptr;
    if (type == W_MXFP4) pick<W_MXFP4, 0>(depth, &ku, &kd);
    else if (type == W_Q4_0) ss ? pick<W_Q4_0, 1>(depth, &ku, &kd) : pick<W_Q4_0, 0>(depth, &ku, &kd);
    else if (type == W_Q8_0) ss ? pick<W_Q8_0, 1>(depth, &ku, &kd) : pick<W_Q8_0, 0>(depth, &ku, &kd);
    else return hipErrorInvalidValue;
    hipError_t e = hipSuccess;
    if (F > 0) {
        e = allow_dynamic_lds(reinterpret_cast<const void *>(ku), kLdsMost);
        if (e != hipSuccess) return e;
        const unsigned groups = (unsigned)(((F + 7) / 8 + T - 1) / T);
        hipLaunchKernelGGL(ku, dim3(groups, (unsigned)(N * k)), dim3(64 * p.waves), (unsigned)lds, stream, a);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kd, dim3((unsigned)((M + 7) / 8)), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace qmm
