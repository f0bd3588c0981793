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
// so that a step is 16 KB of activations and 128 x 64 weights in all three,
// and a wave multiplies 32 weight rows by the tile's rows over 64 of K.  Steps
// go from memory to LDS with direct-to-LDS loads, kStages - 1 ahead, one barrier
// each; two workgroups share a CU, so that one's matrix instructions run
// beside the other's waits, unpacking and epilogue.
#include "gemm_common.h"
#include "lds_load.h"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kStages = 3;
constexpr int kTokBytes = 16 * 1024;       // of one stage
constexpr int kScaleBytes = 1024;

template <int WT> struct GrpFmt;
template <> struct GrpFmt<W_Q4_0> { static constexpr int QB = 16; };
template <> struct GrpFmt<W_MXFP4> { static constexpr int QB = 16; };
template <> struct GrpFmt<W_Q8_0> { static constexpr int QB = 32; };

template <int WT, int KP>
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
    static constexpr int CODE_OFF = kTokBytes, SCALE_OFF = CODE_OFF + CODE_BYTES;
    static constexpr int STAGE = SCALE_OFF + kScaleBytes;
    static constexpr int LDS_BYTES = kStages * STAGE;
    static_assert(BN * BK * 2 == kTokBytes && CODE_BYTES == CODE_LOADS * 16 * kThreads, "whole loads");
    static_assert(2 * LDS_BYTES <= 160 * 1024, "two workgroups per CU");
    static_assert(KP == 1 || 4 * 64 * TT * 16 * 4 <= LDS_BYTES, "the waves' sums fit the ring");
};

struct GrpArgs {
    const uint8_t *w, *w2;        // SW: the gate and the up matrices
    uint64_t pitch, pitch2;       // bytes between rows
    uint64_t expert, expert2;     // bytes between experts
    const uint16_t *x;
    uint64_t x_pitch;             // elements
    const int32_t *offsets, *order;
    void *y;
    uint64_t y_pitch;             // elements
    int64_t M;                    // weight rows
    int32_t K, qoff, E, top_k;
    int32_t N, R;                 // tokens, grouped rows
    int32_t m_tiles;
    int32_t bf16_out;
};

// Byte E of w as a signed int8, converted to float (one SDWA conversion).
template <int E>
__device__ inline float sbyte(uint32_t w) { return (float)(int8_t)(w >> (8 * E)); }

// One lane's 16 weights of a block as bf16 pairs, k = 8 h .. 8 h + 7 in b[0..3]
// and 16 + 8 h .. 16 + 8 h + 7 in b[4..7] (h: the lane's half of the wave).
//  Q4_0: a nibble with its top bit flipped, at the top of a byte, is the int8
//        16 (code - 8); the block's scale takes the 16 back.
//  Q8_0: the signed bytes themselves.
//  MXFP4: the value times its scale, exactly.
template <int WT>
__device__ inline void unpack(u32x2 c0, u32x2 c1, float scale, u32x4 &lo, u32x4 &hi)
{
    if constexpr (WT == W_Q4_0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t v = c0[i] ^ 0x88888888u;
            const uint32_t a = (v << 4) & 0xF0F0F0F0u, b = v & 0xF0F0F0F0u;
            lo[2 * i] = pack_bf16(sbyte<0>(a), sbyte<1>(a));
            lo[2 * i + 1] = pack_bf16(sbyte<2>(a), sbyte<3>(a));
            hi[2 * i] = pack_bf16(sbyte<0>(b), sbyte<1>(b));
            hi[2 * i + 1] = pack_bf16(sbyte<2>(b), sbyte<3>(b));
        }
    } else if constexpr (WT == W_Q8_0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            lo[2 * i] = pack_bf16(sbyte<0>(c0[i]), sbyte<1>(c0[i]));
            lo[2 * i + 1] = pack_bf16(sbyte<2>(c0[i]), sbyte<3>(c0[i]));
            hi[2 * i] = pack_bf16(sbyte<0>(c1[i]), sbyte<1>(c1[i]));
            hi[2 * i + 1] = pack_bf16(sbyte<2>(c1[i]), sbyte<3>(c1[i]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t a = c0[i] & 0x0F0F0F0Fu, b = (c0[i] >> 4) & 0x0F0F0F0Fu;
            const uint32_t p = a | (a >> 4), q = b | (b >> 4);
            auto cvt = [&](uint32_t v, auto SEL) {
                return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, decltype(SEL)::value));
            };
            lo[2 * i] = cvt(p, std::integral_constant<int, 0>{});
            lo[2 * i + 1] = cvt(p, std::integral_constant<int, 2>{});
            hi[2 * i] = cvt(q, std::integral_constant<int, 0>{});
            hi[2 * i + 1] = cvt(q, std::integral_constant<int, 2>{});
        }
    }
}

__device__ inline float grp_swish(float z) { return z / (1.0f + expf(-z)); }

__device__ inline int wave_inclusive_sum(int v, int lane)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int o = __shfl_up(v, m);
        v += lane >= m ? o : 0;
    }
    return v;
}

// A group of rows: expert e's [first, end), cut to the rows that there are,
// whatever the offsets hold.
__device__ inline void group_rows(const int32_t *offsets, int e, int R, int &first, int &end)
{
    const int a = offsets[e], b = offsets[e + 1];
    first = a < 0 ? 0 : a > R ? R : a;
    end = b < first ? first : b > R ? R : b;
}

template <int WT, int SS, int KP, bool SW>
__global__ __launch_bounds__(kThreads, 2) void gemm_grouped_kernel(const GrpArgs a)
{
    using T = GrpTile<WT, KP>;
    constexpr int TT = T::TT, BN = T::BN, BK = T::BK;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(lds);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // ---- this workgroup's tile ----
    // Each lane counts the row tiles of a run of experts; the launch has a
    // workgroup for every tile that R rows of E experts can need, in an order
    // (expert, weight tile, row tile) whose consecutive tiles share weights;
    // the eight XCDs take contiguous parts of the tiles that there are.
    const int run = (a.E + 63) / 64;
    int mine = 0;
    for (int i = 0; i < run; ++i) {
        const int e = lane * run + i;
        if (e < a.E) {
            int first, end;
            group_rows(a.offsets, e, a.R, first, end);
            mine += (end - first + BN - 1) / BN;
        }
    }
    const int upto = wave_inclusive_sum(mine, lane);
    const int64_t total = (int64_t)__builtin_amdgcn_readlane(upto, 63) * a.m_tiles;
    if ((int64_t)blockIdx.x >= total) return;
    const int nwg = (int)(total < (int64_t)gridDim.x ? total : (int64_t)gridDim.x);
    const int x8 = (int)blockIdx.x % 8, q8 = nwg / 8, r8 = nwg % 8;
    const int at = x8 * q8 + (x8 < r8 ? x8 : r8) + (int)blockIdx.x / 8;
    const int row_tile = at / a.m_tiles;
    const int owner = __builtin_ctzll(__ballot(upto > row_tile));
    int before = __builtin_amdgcn_readlane(upto, owner) - __builtin_amdgcn_readlane(mine, owner);
    int e = owner * run, first = 0, end = 0, tiles = 0;
    for (;; ++e) {
        group_rows(a.offsets, e, a.R, first, end);
        tiles = (end - first + BN - 1) / BN;
        if (row_tile < before + tiles) break;
        before += tiles;
    }
    e = __builtin_amdgcn_readfirstlane(e);
    first = __builtin_amdgcn_readfirstlane(first);
    end = __builtin_amdgcn_readfirstlane(end);
    tiles = __builtin_amdgcn_readfirstlane(tiles);
    const int local = at - __builtin_amdgcn_readfirstlane(before) * a.m_tiles;
    const int mt = __builtin_amdgcn_readfirstlane(local / tiles);
    const int nt = local - mt * tiles;
    constexpr int MROWS = SW ? T::BM / 2 : T::BM;         // matrix rows per tile
    const int64_t m0 = (int64_t)mt * MROWS;
    const int n0 = first + nt * BN;
    const int toks = end - n0 < BN ? end - n0 : BN;

    // ---- loads ----
    // Activations: load i of a thread is unit 256 i + thread of the tile's
    // TPR-chunk rows; chunk slot s of row t holds chunk s ^ (t's low bits), so
    // that rows read together fall in different banks.  Rows outside the
    // group, tokens outside x and chunks past K read zeros.
    const int steps = (a.K + BK - 1) / BK;
    const uint32_t x_bytes = a.order ? (uint32_t)(((uint64_t)(a.N > 0 ? a.N - 1 : 0) * a.x_pitch + a.K) * 2)
                                     : (uint32_t)(((uint64_t)(toks - 1) * a.x_pitch + a.K) * 2);
    const ll_i32x4 xres = ll_rsrc(a.order ? a.x : a.x + (uint64_t)n0 * a.x_pitch, a.N > 0 ? x_bytes : 0);
    uint32_t xoff[T::TOK_LOADS];
    int xk[T::TOK_LOADS];
#pragma unroll
    for (int i = 0; i < T::TOK_LOADS; ++i) {
        const int u = kThreads * i + (int)threadIdx.x, t = u / T::TPR;
        const int q = u % T::TPR ^ (T::TPR >= 16 ? t & 15 : t >> 1 & 7);
        int row = t < toks ? t : -1;
        if (a.order && row >= 0) {
            const int slot = a.order[n0 + t];
            row = slot >= 0 ? slot / a.top_k : -1;
            if (row >= a.N) row = -1;
        }
        xoff[i] = row >= 0 ? (uint32_t)((uint64_t)row * a.x_pitch * 2) + 16u * q : OUT_OF_RANGE;
        xk[i] = row >= 0 ? a.K - 8 * q : INT32_MIN;      // the chunk of step s is in K iff BK s < xk
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
    const int full = a.K / BK;                           // steps wholly in K
    auto issue = [&](int s, int stage) {
        const uint32_t base = lds0 + (uint32_t)(stage * T::STAGE) + 1024u * wave;
        const uint32_t sb = (uint32_t)(STEP_SCALES * s) & ~3u;
        const uint32_t sdst = lds0 + (uint32_t)(stage * T::STAGE + T::SCALE_OFF) + 256u * wave;
        if (s < full) {
#pragma unroll
            for (int i = 0; i < T::TOK_LOADS; ++i) ll_load_at<16>(xres, base + 4096u * i, xoff[i], 2u * BK * s);
#pragma unroll
            for (int i = 0; i < T::CODE_LOADS; ++i)
                ll_load_at<16>(code_upper(i) ? ures : wres, base + T::CODE_OFF + 4096u * i, coff[i], 16u * T::UPR * s);
            ll_load_at<4>(scale_upper ? ures : wres, sdst, soff, sb);
        } else {
#pragma unroll
            for (int i = 0; i < T::TOK_LOADS; ++i)
                ll_load<16>(xres, base + 4096u * i, BK * s < xk[i] ? xoff[i] + 2u * BK * s : OUT_OF_RANGE);
#pragma unroll
            for (int i = 0; i < T::CODE_LOADS; ++i)
                ll_load<16>(code_upper(i) ? ures : wres, base + T::CODE_OFF + 4096u * i,
                            16 * T::UPR * s < ck[i] && coff[i] != OUT_OF_RANGE ? coff[i] + 16u * T::UPR * s : OUT_OF_RANGE);
            ll_load<4>(scale_upper ? ures : wres, sdst, (int)sb < sk && soff != OUT_OF_RANGE ? soff + sb : OUT_OF_RANGE);
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

    auto multiply = [&](const uint8_t *st, int s) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int bi = 2 * par + b;                  // block of the step
            u32x2 c0, c1;
            if constexpr (T::QB == 16) {
                c0 = *reinterpret_cast<const u32x2 *>(st + code_at(bi));
                c1 = c0;
            } else {
                c0 = *reinterpret_cast<const u32x2 *>(st + code_at(2 * bi));
                c1 = *reinterpret_cast<const u32x2 *>(st + code_at(2 * bi + 1));
            }
            // a block past K gets a zero scale
            const bool live = 2 * KP * s + bi < blocks;
            float d;
            if constexpr (WT == W_MXFP4) {
                const uint32_t byte = st[s_row + (KP == 1 ? 2 * (s & 1) : 0) + bi];
                d = __builtin_bit_cast(float, live ? byte << 23 : 0u);
            } else {
                const uint32_t o = SS ? (KP == 1 ? 2 * (s & 1) : 2 * (bi >> 1)) : 2 * bi;
                d = live ? (float)*reinterpret_cast<const _Float16 *>(st + s_row + o) : 0.0f;
                if constexpr (WT == W_Q4_0) d *= 0.0625f;
            }
            u32x4 lo, hi;
            unpack<WT>(c0, c1, d, lo, hi);
            const bf16x8 b0 = __builtin_bit_cast(bf16x8, lo), b1 = __builtin_bit_cast(bf16x8, hi);
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                auto frag = [&](int c) {
                    const uint32_t q = (uint32_t)(8 * par + 4 * b + 2 * c + h);
                    return *reinterpret_cast<const bf16x8 *>(st + t_row[j] + 16u * (q ^ t_sw[j]));
                };
                if constexpr (WT == W_MXFP4) {
                    acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag(0), b0, acc[j], 0, 0, 0);
                    acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag(1), b1, acc[j], 0, 0, 0);
                } else {
                    f32x16 sum = {};
                    sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag(0), b0, sum, 0, 0, 0);
                    sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag(1), b1, sum, 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[j][r] = fmaf(sum[r], d, acc[j][r]);
                }
            }
        }
    };

    // ---- the steps ----
    for (int s = 0; s < kStages - 1; ++s) issue(s, s);
    int stage = 0, next = kStages - 1;
    for (int s = 0; s < steps; ++s) {
        ll_wait<T::LOADS * (kStages - 2)>();             // this wave's loads of step s have landed
        // every wave's have, and the stage of step s - 1 is free
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        issue(s + kStages - 1, next);                    // past the last step: zeros
        multiply(lds + stage * T::STAGE, s);
        next = stage;
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }

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
            if (a.bf16_out) static_cast<uint16_t *>(a.y)[p] = (uint16_t)pack_bf16(v, 0.0f);
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

template <int WT, int SS, int KP, bool SW>
hipError_t launch_tile(GrpArgs &a, hipStream_t stream)
{
    using T = GrpTile<WT, KP>;
    a.m_tiles = (int32_t)((a.M + (SW ? T::BM / 2 : T::BM) - 1) / (SW ? T::BM / 2 : T::BM));
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&gemm_grouped_kernel<WT, SS, KP, SW>), T::LDS_BYTES);
    if (e != hipSuccess) return e;
    const int64_t blocks = grouped_row_tiles(a.R, a.E, T::BN) * a.m_tiles;
    hipLaunchKernelGGL((gemm_grouped_kernel<WT, SS, KP, SW>), dim3((unsigned)blocks), dim3(kThreads), T::LDS_BYTES, stream, a);
    return hipGetLastError();
}
template <int WT, int SS>
hipError_t launch_type(GrpArgs &a, int kp, bool sw, hipStream_t stream)
{
    if (kp == 1) return sw ? launch_tile<WT, SS, 1, true>(a, stream) : launch_tile<WT, SS, 1, false>(a, stream);
    if (kp == 2) return sw ? launch_tile<WT, SS, 2, true>(a, stream) : launch_tile<WT, SS, 2, false>(a, stream);
    return sw ? launch_tile<WT, SS, 4, true>(a, stream) : launch_tile<WT, SS, 4, false>(a, stream);
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
    a.K = (int32_t)w.w.K;
    a.qoff = (int32_t)quant_offset(w.w.K, w.w.scale_shift);
    a.E = (int32_t)w.E;
    a.top_k = top_k;
    a.N = (int32_t)x.N;
    a.R = (int32_t)y.R;
    a.bf16_out = y.bf16;
    const int kp = grouped_k_waves(y.R, w.E);
    const bool sw = up != nullptr;
    if (w.w.type == W_MXFP4) return launch_type<W_MXFP4, 1>(a, kp, sw, stream);
    if (w.w.type == W_Q4_0) return w.w.scale_shift ? launch_type<W_Q4_0, 1>(a, kp, sw, stream) : launch_type<W_Q4_0, 0>(a, kp, sw, stream);
    if (w.w.type == W_Q8_0) return w.w.scale_shift ? launch_type<W_Q8_0, 1>(a, kp, sw, stream) : launch_type<W_Q8_0, 0>(a, kp, sw, stream);
    return hipErrorInvalidValue;
}

}  // namespace qmm
