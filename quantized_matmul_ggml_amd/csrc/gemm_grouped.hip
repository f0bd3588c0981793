// gemm_grouped.hip -- matrix products grouped by expert, with ragged sizes.
//
//   y[r] = W_e x[t(r)],   offsets[e] <= r < offsets[e + 1],
// and the fused gate/up pair h[r] = Swish(Wg_e x[t(r)]) * (Wu_e x[t(r)]) of the
// feed-forward block (Development Guide for Small AI Models (TinyLLaMA, etc.)
// Using C++, §4.4), for a mixture of experts whose tokens are grouped on the
// device: t(r) is r itself, or the token of slot order[r].
//
// Arithmetic: codes and bf16 activations multiply exactly on the bf16 matrix
// cores.  For the integer types the codes enter as whole numbers, a block's 32
// products add up in the matrix core's binary32 accumulators, and the block's
// fp16 scale multiplies that sum in binary32 (A Complete Guide to llama.cpp and
// Customization with C++, §2.2: each block has its scale); MXFP4 values are
// exact in bf16 with their scale.  So only binary32 sums round.
//
// A workgroup of four waves takes a tile of weight rows x grouped rows of one
// expert.  KP waves share each wave's tile and split K among them:
//   KP = 1: 128 weight rows x 128 grouped rows, K in steps of 64
//   KP = 2:  64 x 64, steps of 128
//   KP = 4:  32 x 32, steps of 256
// so that a step is 16 KB of activations and 128 x 64 weights in all three (of rows in
// two bf16 parts, P = 2, half as many weights),
// and a wave multiplies 32 weight rows by the tile's rows over 64 of K.  Steps
// go from memory to LDS with direct-to-LDS loads one or two steps ahead, one barrier
// each; two or three workgroups share a CU, so that one's matrix instructions run
// beside the other's waits, unpacking and epilogue.
//
// Bound by the vector work beside the matrix instructions (one multiply-add per
// output and block, and the unpacking) at the clock that it leaves: 8186 rows x
// 2048 x 5632 Q8_0 over 8 experts take 299 us a call (632 TFLOP/s; 307 to 345 under
// the profiler, 615 thousand cycles at 1.74 GHz, 2.3 GHz with operands of zeros), of
// which the matrix cores are busy 193 thousand and the vector units 326 thousand; a
// matrix instruction costs the waves of a SIMD about 8 issue cycles, other vector
// ones 4 to 5.
#include "gemm_common.h"
#include "grouped_tile.h"
#include "lds_load.h"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kTokBytes = 16 * 1024;       // of one stage
constexpr int kScaleBytes = 1024;

template <int WT> struct GrpFmt;
template <> struct GrpFmt<W_Q4_0> { static constexpr int QB = 16; };
template <> struct GrpFmt<W_MXFP4> { static constexpr int QB = 16; };
template <> struct GrpFmt<W_Q8_0> { static constexpr int QB = 32; };

template <int WT, int KP, int NST, int P>
struct GrpTile {
    static constexpr int QB = GrpFmt<WT>::QB;      // code bytes of a 32-block
    static constexpr int RG = 4 / KP;              // waves along the weight rows
    static constexpr int TT = 4 / KP;              // 32-row sub-tiles along the grouped rows
    static constexpr int BM = 32 * RG, BN = 32 * TT, BK = 64 * KP;
    static constexpr int UPR = BK / 32 * QB / 16;  // 16-byte code units per row and step
    static constexpr int CODE_BYTES = BM * UPR * 16;
    static constexpr int CODE_LOADS = CODE_BYTES / (16 * kThreads);
    static constexpr int TPR = BK * 2 / 16;        // 16-byte chunks per grouped row and step
    static constexpr int TOK_LOADS = kTokBytes / (16 * kThreads);
    static constexpr int LOADS = TOK_LOADS + CODE_LOADS + 1;   // per wave and step
    // With P = 2 a row's step of 64 KP values is of half as many weights, and the weights
    // of two such steps are loaded together, to one of two places of their own (loaded
    // with each step, the layer of 4096 tokens took 921 us, so 858).
    static constexpr int STAGE = kTokBytes + (P == 1 ? CODE_BYTES + kScaleBytes : 0);
    static constexpr int CODE_OFF = P == 1 ? kTokBytes : NST * kTokBytes, SCALE_OFF = CODE_OFF + CODE_BYTES;
    static constexpr int W_STAGE = P == 1 ? STAGE : CODE_BYTES + kScaleBytes;      // between weights' places
    // With two stages three workgroups share a CU, with three two.  Where there are
    // enough tiles the workgroup is worth more than the stage (gate and up of 4096 rows,
    // 5632 x 2048 Q4_0, two and three stages: 64-row tiles 349 and 376 us, 32-row ones
    // 565 and 670; 7372 rows, 128-row tiles 501 and 543); with few tiles a CU the
    // stage is (486 rows, pair of 321 x 3584 Q4_0 17.4 and 15.6, 137 rows, layer of
    // three Q8_0 experts 2176 -> 3648 48.9 and 45.4).
    static constexpr int STAGES = NST;
    static constexpr int LDS_BYTES = STAGES * STAGE + (P == 1 ? 0 : 2 * W_STAGE);
    static_assert(BN * BK * 2 == kTokBytes && CODE_BYTES == CODE_LOADS * 16 * kThreads, "whole loads");
    static_assert((KP == 1 ? 3 : 2) * LDS_BYTES <= 160 * 1024, "workgroups per CU");
    static_assert(KP == 1 || 4 * 64 * TT * 16 * 4 <= LDS_BYTES, "the waves' sums fit the ring");
};

// Byte E of w as a signed int8, converted to float (one SDWA conversion).
template <int E>
__device__ inline float sbyte(uint32_t w) { return (float)(int8_t)(w >> (8 * E)); }

// Pair P of one lane's 16 weights of a block as bf16: k = 8 h + 2 P, + 1 for P < 4
// and 16 + 8 h + 2 (P - 4), + 1 from there on (h: the lane's half of the wave).
//  Q4_0: a nibble with its top bit flipped, at the top of a byte, is the int8
//        16 (code - 8); the block's scale takes the 16 back.
//  Q8_0: the signed bytes themselves.
//  MXFP4: the value times its scale, exactly.
template <int WT, int P>
__device__ inline uint32_t unpack_pair(u32x2 c0, u32x2 c1, float scale)
{
    constexpr int i = P / 2 % 2, e = 2 * (P % 2);
    if constexpr (WT == W_Q4_0) {
        const uint32_t v = c0[i] ^ 0x88888888u, b = (P < 4 ? v << 4 : v) & 0xF0F0F0F0u;
        return pack_bf16(sbyte<e>(b), sbyte<e + 1>(b));
    } else if constexpr (WT == W_Q8_0) {
        const uint32_t b = P < 4 ? c0[i] : c1[i];
        return pack_bf16(sbyte<e>(b), sbyte<e + 1>(b));
    } else {
        // the even and odd bytes' nibbles side by side: a pair is neighbouring k
        const uint32_t n = (P < 4 ? c0[i] : c0[i] >> 4) & 0x0F0F0F0Fu;
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(n | (n >> 4), scale, e));
    }
}

__device__ inline float grp_swish(float z) { return z / (1.0f + expf(-z)); }

template <int WT, int SS, int KP, bool SW, int NST, int P>
__global__ __launch_bounds__(kThreads, NST == 2 ? 3 : 2) void gemm_grouped_kernel(const GrpArgs a)
{
    using T = GrpTile<WT, KP, NST, P>;
    static_assert(P == 1 || !SW, "split rows are the pair's own output");
    constexpr int TT = T::TT, BN = T::BN, BK = T::BK;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(lds);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    GroupTile tile;
    if (!find_tile<BN>(a, tile)) return;
    const int e = tile.e, n0 = tile.n0, toks = tile.rows;
    constexpr int MROWS = SW ? T::BM / 2 : T::BM;         // matrix rows per tile
    const int64_t m0 = (int64_t)tile.mt * MROWS;

    // ---- loads ----
    // Activations: load i of a thread is unit 256 i + thread of the tile's
    // TPR-chunk rows; chunk slot s of row t holds chunk s ^ (t's low bits), so
    // that rows read together fall in different banks.  Rows outside the
    // group, tokens outside x and chunks past K read zeros.
    const int steps = (P * a.K + BK - 1) / BK;
    const uint32_t x_bytes = (uint32_t)(((uint64_t)((a.order ? a.N : toks) - 1) * a.x_pitch + P * a.K) * 2);
    const ll_i32x4 xres = ll_rsrc(a.order ? a.x : a.x + (uint64_t)n0 * a.x_pitch, a.K > 0 ? x_bytes : 0);
    uint32_t xoff[T::TOK_LOADS];
    int xk[T::TOK_LOADS];
#pragma unroll
    for (int i = 0; i < T::TOK_LOADS; ++i) {
        const int u = kThreads * i + (int)threadIdx.x, t = u / T::TPR;
        const int q = u % T::TPR ^ (T::TPR >= 16 ? t & 15 : t >> 1 & 7);
        const int row = t >= toks ? -1 : a.order ? token_of(a, n0 + t) : t;
        xoff[i] = row >= 0 ? (uint32_t)((uint64_t)row * a.x_pitch * 2) + 16u * q : OUT_OF_RANGE;
        xk[i] = row >= 0 ? P * a.K - 8 * q : INT32_MIN;      // the chunk of step s is in K iff BK s < xk
    }
    // Codes: the same with the tile's weight rows; with SW rows 0 .. BM / 2 - 1
    // are of the gate matrix and the rest the same rows of the up matrix.
    // Scales: dword d of row r, whole dwords (a step of 64-weight or one-byte
    // scales with KP = 1 is half a dword, loaded in both steps).
    const int64_t rows = a.M - m0 < MROWS ? a.M - m0 : MROWS;
    const uint32_t row_bytes = (uint32_t)a.qoff + (uint32_t)(a.K / 32) * T::QB;
    auto matrix = [&](const uint8_t *w, uint64_t pitch, uint64_t expert) {
        return ll_rsrc(w + (uint64_t)e * expert + (uint64_t)m0 * pitch, (uint32_t)((uint64_t)(rows - 1) * pitch + row_bytes));
    };
    const ll_i32x4 wres = matrix(a.w, a.pitch, a.expert);
    const ll_i32x4 ures = SW ? matrix(a.w2, a.pitch2, a.expert2) : wres;
    // whether this wave's code load i, and its scale load, are of the up matrix
    auto code_upper = [&](int i) { return SW && (T::CODE_LOADS == 2 ? i == 1 : wave >= 2); };
    const bool scale_upper = SW && wave >= 2;
    uint32_t coff[T::CODE_LOADS];
    int ck[T::CODE_LOADS];
#pragma unroll
    for (int i = 0; i < T::CODE_LOADS; ++i) {
        const int u = kThreads * i + (int)threadIdx.x, r = u / T::UPR;
        const int unit = u % T::UPR ^ (r / (16 / T::UPR) & (T::UPR - 1));
        const bool up = code_upper(i);
        const int mr = up ? r - MROWS : r;
        coff[i] = mr < rows ? (uint32_t)(mr * (up ? a.pitch2 : a.pitch)) + (uint32_t)a.qoff + 16u * unit : OUT_OF_RANGE;
        ck[i] = (a.K / 32) * T::QB - 16 * unit;          // bytes of the row's codes from this unit of step 0 on
    }
    constexpr int STEP_SCALES = 4 * KP >> SS;            // scale bytes per row and step
    constexpr int DPR = STEP_SCALES < 4 ? 1 : STEP_SCALES / 4;
    constexpr int SROWS = T::BM / 4;                     // rows per wave's scale load
    const int sr = wave * SROWS + lane / DPR;
    const int smr = scale_upper ? sr - MROWS : sr;
    const uint32_t soff = lane < SROWS * DPR && smr < rows
                              ? (uint32_t)(smr * (scale_upper ? a.pitch2 : a.pitch)) + 4u * (lane % DPR) : OUT_OF_RANGE;
    const int sk = (a.K / 32 * 2 >> SS) - 4 * (lane % DPR);
    const int full = P * (a.K / BK);                     // steps wholly in K, with their weights
    // Load L of a wave for step s, weights (with P = 2 every other step has some) to
    // place w.  FAST: the step is wholly in K, its offset goes in as a scalar; else every
    // lane is checked against K (past the last step all read zeros).
    auto load = [&](auto FAST, auto L, int s, int stage) {
        constexpr int l = decltype(L)::value;
        constexpr bool fast = decltype(FAST)::value;
        const int ws = s / P, w = P == 1 ? stage : ws & 1;
        if (P == 2 && l >= T::TOK_LOADS && s % 2) return;
        if constexpr (l < T::TOK_LOADS) {
            const uint32_t dst = lds0 + (uint32_t)(stage * T::STAGE) + 1024u * wave + 4096u * l, o = 2u * BK * s;
            if constexpr (fast) ll_load_at<16>(xres, dst, xoff[l], o);
            else ll_load<16>(xres, dst, BK * s < xk[l] ? xoff[l] + o : OUT_OF_RANGE);
        } else if constexpr (l < T::TOK_LOADS + T::CODE_LOADS) {
            constexpr int i = l - T::TOK_LOADS;
            const uint32_t dst = lds0 + (uint32_t)(w * T::W_STAGE + T::CODE_OFF) + 1024u * wave + 4096u * i, o = 16u * T::UPR * ws;
            const ll_i32x4 &res = code_upper(i) ? ures : wres;
            if constexpr (fast) ll_load_at<16>(res, dst, coff[i], o);
            else ll_load<16>(res, dst, (int)o < ck[i] && coff[i] != OUT_OF_RANGE ? coff[i] + o : OUT_OF_RANGE);
        } else {
            const uint32_t dst = lds0 + (uint32_t)(w * T::W_STAGE + T::SCALE_OFF) + 256u * wave;
            const uint32_t o = (uint32_t)(STEP_SCALES * ws) & ~3u;
            const ll_i32x4 &res = scale_upper ? ures : wres;
            if constexpr (fast) ll_load_at<4>(res, dst, soff, o);
            else ll_load<4>(res, dst, (int)o < sk && soff != OUT_OF_RANGE ? soff + o : OUT_OF_RANGE);
        }
    };

    // ---- this wave's part of a step ----
    const int rg = wave % T::RG, par = wave / T::RG;     // weight rows 32 rg .., K 64 par .. of each step
    const int h = lane >> 5, l32 = lane & 31;
    // its weight row of the tile: with SW lanes 0 .. 15 hold gate rows and
    // lanes 16 .. 31 the same rows of the up matrix
    const int rl = SW ? (l32 < 16 ? 16 * rg + l32 : T::BM / 2 + 16 * rg + l32 - 16) : 32 * rg + l32;
    const uint32_t c_row = (uint32_t)(T::CODE_OFF + rl * T::UPR * 16), c_sw = rl / (16 / T::UPR) & (T::UPR - 1);
    auto code_at = [&](int unit) { return c_row + 16u * ((uint32_t)unit ^ c_sw) + 8u * h; };
    const uint32_t s_row = (uint32_t)(T::SCALE_OFF + 256 * (rl / SROWS) + 4 * DPR * (rl % SROWS));
    uint32_t t_row[TT], t_sw[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) {
        const int t = 32 * j + l32;
        t_row[j] = (uint32_t)(t * T::TPR * 16);
        t_sw[j] = T::TPR >= 16 ? t & 15 : t >> 1 & 7;
    }
    const int blocks = a.K / 32;
    f32x16 acc[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[j][r] = 0.0f;

    // ---- the steps ----
    // A unit is one tile's products with one block (two blocks that share a
    // scale): its matrix instructions start from zero and their sums are scaled
    // and added while the next unit's run.  Each matrix instruction is followed
    // by its share of that, of the second block's unpacking and of the fragment
    // and LDS loads, in this order: with the waves of a SIMD out of step, one's
    // vector work runs beside the other's matrix work (all loads of a step issued
    // together took 367 us instead of 354 for 8186 rows x 2048 x 5632 Q8_0).
    constexpr bool SCALED = WT != W_MXFP4;
    constexpr int PER = SCALED && (SS || P == 2) ? 2 : 1;       // blocks (or parts of one) of a unit
    constexpr int NB = P == 2 ? 1 : 2;                   // weight blocks of a step and wave
    constexpr int UNITS = 2 / PER * TT, PU = 2 * PER;    // units per step, instructions per unit
    constexpr int MI = UNITS * PU, AHEAD = MI < 4 ? MI : 4;
    f32x16 sum[2] = {};                                  // of the units at hand
    float pending = 0.0f;                                // the last unit's scale
    auto add = [&](auto U, int from, int to, float d) {  // unit U's sums, registers from .. to - 1
        constexpr int j = decltype(U)::value % TT;
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (r >= from && r < to) acc[j][r] = fmaf(sum[decltype(U)::value & 1][r], d, acc[j][r]);
    };
    // step s from its stage, and the loads of step s + T::STAGES - 1 into another
    auto multiply = [&](auto FAST, const uint8_t *st, int s, int next) {
        // its weights' step and place, and the first block there
        const int ws = s / P, first = P == 1 ? NB * par : KP * (s % P) + par;
        const uint8_t *const wst = P == 1 ? st : lds + (ws & 1) * T::W_STAGE;
        u32x2 c0[2], c1[2];
        float d[2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int bi = first + b;                    // block of the step
            if constexpr (T::QB == 16) {
                c0[b] = c1[b] = *reinterpret_cast<const u32x2 *>(wst + code_at(bi));
            } else {
                c0[b] = *reinterpret_cast<const u32x2 *>(wst + code_at(2 * bi));
                c1[b] = *reinterpret_cast<const u32x2 *>(wst + code_at(2 * bi + 1));
            }
        }
        uint32_t raw[2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int bi = first + b;
            if constexpr (WT == W_MXFP4) raw[b] = wst[s_row + (KP == 1 ? 2 * (ws & 1) : 0) + bi];
            else raw[b] = *reinterpret_cast<const uint16_t *>(wst + s_row + (SS ? (KP == 1 ? 2 * (ws & 1) : 2 * (bi >> 1)) : 2 * bi));
        }
        // instruction k: block b, tile j, chunk c of the block
        auto frag = [&](auto K) {
            constexpr int k = decltype(K)::value, u = k / PU, b = PER == 2 ? k % PU / 2 : u / TT, j = u % TT, c = k % 2;
            const uint32_t q = (uint32_t)(8 * par + 4 * b + 2 * c + h);
            return *reinterpret_cast<const bf16x8 *>(st + t_row[j] + 16u * (q ^ t_sw[j]));
        };
        bf16x8 x[AHEAD];
        static_for<AHEAD>([&](auto K) { x[decltype(K)::value] = frag(K); });
        if constexpr (SCALED && UNITS > 1) add(std::integral_constant<int, UNITS - 1>{}, 0, 16, pending);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            // a block past K gets a zero scale (a mask: no branch between the products)
            raw[b] &= 2 * KP * ws + first + b < blocks ? 0xFFFFu : 0u;
            if constexpr (WT == W_MXFP4) d[b] = __builtin_bit_cast(float, raw[b] << 23);
            else d[b] = (float)__builtin_bit_cast(_Float16, (uint16_t)raw[b]) * (WT == W_Q4_0 ? 0.0625f : 1.0f);
        }
        u32x4 w[2][2];
        static_for<8>([&](auto I) {
            constexpr int p = decltype(I)::value;
            w[0][p / 4][p % 4] = unpack_pair<WT, p>(c0[0], c1[0], d[0]);
        });
        static_for<MI>([&](auto K) {
            constexpr int k = decltype(K)::value, u = k / PU, b = PER == 2 ? k % PU / 2 : u / TT, j = u % TT, c = k % 2;
            const bf16x8 wf = __builtin_bit_cast(bf16x8, w[P == 2 ? 0 : b][c]), xf = x[k % AHEAD];
            if constexpr (!SCALED) acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xf, wf, acc[j], 0, 0, 0);
            else if constexpr (k % PU == 0) sum[u & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xf, wf, f32x16{}, 0, 0, 0);
            else sum[u & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xf, wf, sum[u & 1], 0, 0, 0);
            if constexpr (k + AHEAD < MI) x[k % AHEAD] = frag(std::integral_constant<int, k + AHEAD>{});
            // with one stage ahead a load behind each of the first instructions, so that
            // they have the rest of the step to land (spread over the step, a pair of
            // 5632 x 2048 MXFP4 for 4096 rows took 238 us instead of 230), else spread
            constexpr int per = (T::LOADS + MI - 1) / MI, gap = per > 1 || T::STAGES == 2 ? 1 : MI / T::LOADS;
            static_for<per>([&](auto I) {
                constexpr int l = k / gap * per + decltype(I)::value;
                if constexpr (k % gap == 0 && l < T::LOADS) load(FAST, std::integral_constant<int, l>{}, s + T::STAGES - 1, next);
            });
            __builtin_amdgcn_sched_barrier(0);
            // the second block's pairs, before the first instruction that takes them
            constexpr int B1 = PER == 2 ? 2 : MI / 2, n = (8 + B1 - 1) / B1;
            static_for<n>([&](auto I) {
                constexpr int p = k * n + decltype(I)::value;
                if constexpr (P == 1 && k < B1 && p < 8) w[1][p / 4][p % 4] = unpack_pair<WT, p>(c0[1], c1[1], d[1]);
            });
            // the unit before
            constexpr int share = 16 / PU;
            if constexpr (SCALED && u > 0)
                add(std::integral_constant<int, u - 1>{}, share * (k % PU), share * (k % PU + 1), d[PER == 2 ? 0 : (u - 1) / TT]);
            __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (SCALED) {
            pending = d[PER == 2 ? 0 : 1];
            if constexpr (UNITS == 1) add(std::integral_constant<int, 0>{}, 0, 16, pending);
        }
    };
    for (int s = 0; s < T::STAGES - 1; ++s)
        static_for<T::LOADS>([&](auto L) { load(std::false_type{}, L, s, s); });
    int stage = 0, next = T::STAGES - 1;
    auto run_steps = [&](auto FAST, int s, int to) {
        for (; s < to; ++s) {
            // this wave's loads of step s have landed (with three stages, those of the next
            // step may be pending, with or without weights)
            if (P == 1 || T::STAGES == 2 || s % 2) ll_wait<T::LOADS * (T::STAGES - 2)>();
            else ll_wait<T::TOK_LOADS * (T::STAGES - 2)>();
            // every wave's have, and the stage of step s - 1 is free
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            multiply(FAST, lds + stage * T::STAGE, s, next);
            next = stage;
            stage = stage + 1 == T::STAGES ? 0 : stage + 1;
        }
    };
    const int fast_to = full - (T::STAGES - 1) > 0 ? full - (T::STAGES - 1) : 0;
    run_steps(std::true_type{}, 0, fast_to);
    run_steps(std::false_type{}, fast_to, steps);
    if constexpr (SCALED && UNITS > 1) add(std::integral_constant<int, UNITS - 1>{}, 0, 16, pending);

    // ---- the KP waves of a sub-tile add their sums, each a part of them ----
    ll_wait<0>();                    // no load may still write the ring
    constexpr int FR = TT * 16 / KP;
    float fin[FR];
    if constexpr (KP == 1) {
#pragma unroll
        for (int i = 0; i < FR; ++i) fin[i] = acc[i / 16][i % 16];
    } else {
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        float *xch = reinterpret_cast<float *>(lds);     // [wave][TT * 16][64]
#pragma unroll
        for (int i = 0; i < TT * 16; ++i) xch[(wave * TT * 16 + i) * 64 + lane] = acc[i / 16][i % 16];
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int i = 0; i < FR; ++i) {
            fin[i] = 0.0f;
#pragma unroll
            for (int p = 0; p < KP; ++p) fin[i] += xch[((rg + T::RG * p) * TT * 16 + par * FR + i) * 64 + lane];
        }
    }
    // the tile's row that register i of this wave holds
    auto row_of = [&](int i) {
        const int reg = par * FR + i;
        return 32 * (reg / 16) + 8 * (reg % 16 / 4) + 4 * h + reg % 4;
    };
    auto store = [&](int t, int64_t m, float v) {
        if (t < toks && m < a.M) {
            const uint64_t p = (uint64_t)(n0 + t) * a.y_pitch + m;
            if (SW && a.split_out) store_split(static_cast<uint16_t *>(a.y) + (uint64_t)(n0 + t) * a.y_pitch, m, v);
            else if (a.bf16_out) static_cast<uint16_t *>(a.y)[p] = (uint16_t)pack_bf16(v, 0.0f);
            else static_cast<float *>(a.y)[p] = v;
        }
    };
    if constexpr (SW) {
        // swap the up half of register i with the gate half of register i + 1:
        // lanes 0 .. 15 then hold both of row i, lanes 16 .. 31 of row i + 1
        const int64_t m = m0 + 16 * rg + (l32 & 15);
#pragma unroll
        for (int i = 0; i < FR; i += 2) {
            const auto p = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, fin[i]),
                                                            __builtin_bit_cast(uint32_t, fin[i + 1]), false, false);
            const float g = __builtin_bit_cast(float, (uint32_t)p[0]), u = __builtin_bit_cast(float, (uint32_t)p[1]);
            store(l32 < 16 ? row_of(i) : row_of(i + 1), m, grp_swish(g) * u);
        }
    } else {
        const int64_t m = m0 + rl;
#pragma unroll
        for (int i = 0; i < FR; ++i) store(row_of(i), m, fin[i]);
    }
}

template <int WT, int SS, int KP, bool SW, int NST, int P>
hipError_t launch_tile(GrpArgs &a, hipStream_t stream)
{
    using T = GrpTile<WT, KP, NST, P>;
    a.m_tiles = (int32_t)((a.M + (SW ? T::BM / 2 : T::BM) - 1) / (SW ? T::BM / 2 : T::BM));
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&gemm_grouped_kernel<WT, SS, KP, SW, NST, P>), T::LDS_BYTES);
    if (e != hipSuccess) return e;
    const int64_t blocks = grouped_row_tiles(a.R, a.E, T::BN) * a.m_tiles;
    hipLaunchKernelGGL((gemm_grouped_kernel<WT, SS, KP, SW, NST, P>), dim3((unsigned)blocks), dim3(kThreads), T::LDS_BYTES, stream, a);
    return hipGetLastError();
}
template <int WT, int SS, bool SW, int P>
hipError_t launch_form(GrpArgs &a, GroupedForm f, hipStream_t stream)
{
    if (f.kp == 1) return launch_tile<WT, SS, 1, SW, 2, P>(a, stream);
    if (f.kp == 2) return f.deep ? launch_tile<WT, SS, 2, SW, 3, P>(a, stream) : launch_tile<WT, SS, 2, SW, 2, P>(a, stream);
    return f.deep ? launch_tile<WT, SS, 4, SW, 3, P>(a, stream) : launch_tile<WT, SS, 4, SW, 2, P>(a, stream);
}
template <int WT, int SS>
hipError_t launch_type(GrpArgs &a, GroupedForm f, bool sw, int parts, hipStream_t stream)
{
    if (sw) return launch_form<WT, SS, true, 1>(a, f, stream);
    return parts == 2 ? launch_form<WT, SS, false, 2>(a, f, stream) : launch_form<WT, SS, false, 1>(a, f, stream);
}

}  // namespace

hipError_t launch_gemm_grouped(const ExpertView &w, const ExpertView *up, const ActView &x, const int32_t *offsets,
                               const int32_t *order, int top_k, const GroupedOut &y, hipStream_t stream)
{
    if (y.R == 0 || w.w.M == 0) return hipSuccess;
    GrpArgs a = {};
    const ExpertView &u = up ? *up : w;
    a.w = w.w.base;
    a.w2 = u.w.base;
    a.pitch = w.w.pitch;
    a.pitch2 = u.w.pitch;
    a.expert = w.expert_pitch;
    a.expert2 = u.expert_pitch;
    a.x = static_cast<const uint16_t *>(x.data);
    a.x_pitch = x.pitch_elems;
    a.offsets = offsets;
    a.order = order;
    a.y = y.data;
    a.y_pitch = y.pitch_elems;
    a.M = w.w.M;
    a.K = x.N > 0 ? (int32_t)w.w.K : 0;         // without tokens every row is zeros
    a.qoff = (int32_t)quant_offset(w.w.K, w.w.scale_shift);
    a.E = (int32_t)w.E;
    a.top_k = top_k;
    a.N = (int32_t)x.N;
    a.R = (int32_t)y.R;
    a.bf16_out = y.bf16;
    a.split_out = y.split;
    const bool sw = up != nullptr;
    const int parts = x.split ? 2 : 1;
    if (sw && parts != 1) return hipErrorInvalidValue;
    const GroupedForm f = grouped_form(a.M, w.w.K, y.R, w.E, w.w.type, sw, device_cus(), parts);
    if (f.kp == 0) return launch_gemm_rows(a, w.w.type, w.w.scale_shift, sw, parts, stream);
    if (w.w.type == W_MXFP4) return launch_type<W_MXFP4, 1>(a, f, sw, parts, stream);
    if (w.w.type == W_Q4_0) return w.w.scale_shift ? launch_type<W_Q4_0, 1>(a, f, sw, parts, stream) : launch_type<W_Q4_0, 0>(a, f, sw, parts, stream);
    if (w.w.type == W_Q8_0) return w.w.scale_shift ? launch_type<W_Q8_0, 1>(a, f, sw, parts, stream) : launch_type<W_Q8_0, 0>(a, f, sw, parts, stream);
    return hipErrorInvalidValue;
}

}  // namespace qmm
