// row_tiles.h -- device parts shared by the kernels that stream packed weight
// rows through the bf16 matrix cores against exactly represented binary32
// activations: the MXFP4 GEMV (gemv_mx.hip) and the mixture-of-experts layer
// (moe.hip).  Internal to the library.
//
// One matrix instruction, v_mfma_f32_16x16x32_bf16 (D 16 x 16 += A 16 x 32 *
// B 32 x 16), takes 32 values of k of 16 weight rows (B) and of up to four
// tokens (A).  The arithmetic is exact up to the binary32 accumulation:
//
//  * A, activations.  A binary32 value is cut into three bf16 parts of eight
//    significant bits each, x = hi + mid + lo exactly (the top 16 bits, the
//    top 16 bits of what is left, the rest); matrix row 4 t + p carries part p
//    of token t (p = 3 is not used: such rows repeat part 2 and their sums
//    are never read).  Products of two 8-bit significands are exact.
//  * B, weights.  Row j of a tile is matrix column j.  A lane holds 16 bytes
//    of its row, so the four lane groups g = lane / 16 cover one 64-byte
//    unit of the row (four 32-blocks of 4-bit codes, or two of 8-bit ones)
//    in one 128-bit register each, and the unit is used up by four (or two)
//    matrix instructions:
//     - MXFP4: instruction i takes dword i of every lane: eight values of block
//       4 u + g from lane group g.  Scale and value convert to bf16 together,
//       exactly (v_cvt_scalef32_pk_bf16_fp4), so sums run through whole rows.
//     - Q4_0, Q8_0: two cross-lane swaps regroup the dwords so that one
//       instruction sees one block; the signed codes enter as exact bf16
//       integers and the block's fp16 scale multiplies its sum in binary32.
//  * D: lane (j, g) receives the three partial sums of row j and token g.
//
// What bounds these kernels is the weight stream; the activations' parts sit
// in LDS in the order the matrix instructions read them (192 bytes per token
// and 32-block), or come from memory in the same order.
#pragma once

#include "row_plan.h"

#include <type_traits>

namespace qmm {

typedef __bf16 rt_bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 rt_bf16x2 __attribute__((ext_vector_type(2)));
typedef float rt_f32x4 __attribute__((ext_vector_type(4)));
typedef float rt_f32x2 __attribute__((ext_vector_type(2)));
// four floats at any 4-byte aligned address
typedef float rt_f32x4u __attribute__((ext_vector_type(4), aligned(4)));

// Calls f(std::integral_constant<int, 0>{}) .. f(std::integral_constant<int, N-1>{}).
template <int N, int I = 0, class F>
__device__ inline void static_steps(F &&f)
{
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        static_steps<N, I + 1>(f);
    }
}

constexpr int kTileCols = 16;          // weight rows per tile

// A row format: MF matrix instructions (32-blocks) per 64-byte unit and SPU
// scale bytes per unit.
template <int WT, int SS>
struct RowFmt {
    static constexpr int MF = WT == W_Q8_0 ? 2 : 4;
    static constexpr int KPU = 32 * MF;
    static constexpr int BB = 64 / MF;                   // code bytes of a block
    static constexpr int SPU = WT == W_MXFP4 ? 4 : (2 * MF) >> SS;
};

// Where the activation parts of (block, quarter) lie, in units of 64-byte
// (part, group) rows times the token count: the quarter q of a block is the
// eight values one lane group feeds to one matrix instruction.  MXFP4: lane
// group = block within the unit, instruction = quarter; otherwise the other
// way round.
template <int WT>
__device__ inline int image_step(int block, int q)
{
    return WT == W_MXFP4 ? (block & ~3) + q : block;
}
template <int WT>
__device__ inline int image_group(int block, int q)
{
    return WT == W_MXFP4 ? block & 3 : q;
}
// First elements (within the block) of the two runs of four that make up
// quarter q, and whether the runs interleave (4-bit codes: byte s holds
// elements 4 q + s and 16 + 4 q + s, values in that order; 8-bit codes: the
// swap leaves codes 0.., 16.., 8.., 24.. in lane groups 0..3).
template <int WT>
__device__ inline int run0(int q)
{
    return WT == W_Q8_0 ? (q == 0 ? 0 : q == 1 ? 16 : q == 2 ? 8 : 24) : 4 * q;
}
template <int WT>
__device__ inline int run1(int q)
{
    return WT == W_Q8_0 ? run0<WT>(q) + 4 : 16 + 4 * q;
}

// The exact three-way split of eight values (in matrix order) into bf16
// parts: the upper 16 bits, the upper 16 bits of the remainder, and the rest
// (eight significant bits each).  An infinity is its own first part; a NaN's
// remainder is a NaN.
__device__ inline void split_parts(const float (&v)[8], uint4 (&part)[3])
{
    // the upper halves of two dwords side by side
    auto pk = [](float a, float b) {
        return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u);
    };
    auto upper = [](float x) { return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & 0xFFFF0000u); };
    float mid[8], lo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        mid[i] = fabsf(v[i]) == INFINITY ? 0.0f : v[i] - upper(v[i]);
        lo[i] = mid[i] - upper(mid[i]);
    }
    part[0] = make_uint4(pk(v[0], v[1]), pk(v[2], v[3]), pk(v[4], v[5]), pk(v[6], v[7]));
    part[1] = make_uint4(pk(mid[0], mid[1]), pk(mid[2], mid[3]), pk(mid[4], mid[5]), pk(mid[6], mid[7]));
    part[2] = make_uint4(pk(lo[0], lo[1]), pk(lo[2], lo[3]), pk(lo[4], lo[5]), pk(lo[6], lo[7]));
}

// The two runs of four in matrix order.
template <int WT>
__device__ inline void matrix_order(const rt_f32x4 a, const rt_f32x4 b, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (WT == W_Q8_0) {
            v[i] = a[i];
            v[4 + i] = b[i];
        } else {
            v[2 * i] = a[i];
            v[2 * i + 1] = b[i];
        }
    }
}

// The LDS image of blocks [b0, b0 + nblk) of `ntok` tokens, filled by all
// `threads` threads in pieces of eight values; blocks from nb on are zeros.
// row(t) is token t's row.  A thread's first two pieces are loaded ahead of the
// workgroup's first weights (AHEAD: image_ahead, then build_image), since loads
// complete in order; the weights that follow the first unit are asked for
// after the conversion, because the memory takes them only as fast as it
// delivers, and a wave waiting to issue loads converts nothing.
struct ImageAhead {
    rt_f32x4 r[2][2];
};
// Piece i as (token, piece of the token): tokens are few, so no division.
struct ImagePiece {
    int t, i;
    __device__ inline void settle(int per_tok)
    {
#pragma nounroll
        while (i >= per_tok) {
            i -= per_tok;
            ++t;
        }
    }
};
template <int WT, class Row>
__device__ inline void image_load(const ImagePiece &p, int ntok, int b0, int nb, Row row, rt_f32x4 &r0, rt_f32x4 &r1)
{
    const int b = b0 + (p.i >> 2), q = p.i & 3;
    r0 = r1 = rt_f32x4{0, 0, 0, 0};
    if (p.t < ntok && b < nb) {
        const float *x = row(p.t) + (int64_t)b * 32;
        r0 = *reinterpret_cast<const rt_f32x4u *>(x + run0<WT>(q));
        r1 = *reinterpret_cast<const rt_f32x4u *>(x + run1<WT>(q));
    }
}
template <int WT, class Row>
__device__ inline void image_ahead(ImageAhead &a, int ntok, int b0, int nblk, int nb, int threads, Row row)
{
    ImagePiece p = {0, (int)threadIdx.x};
#pragma unroll
    for (int n = 0; n < 2; ++n, p.i += threads) {
        p.settle(4 * nblk);
        image_load<WT>(p, ntok, b0, nb, row, a.r[n][0], a.r[n][1]);
    }
    __builtin_amdgcn_sched_barrier(0);
}
template <int WT, bool AHEAD, class Row>
__device__ inline void build_image(uint8_t *img, int ntok, int b0, int nblk, int nb, int threads, Row row,
                                   const ImageAhead &ahead)
{
    auto put = [&](const ImagePiece &p, const rt_f32x4 r0, const rt_f32x4 r1) {
        const int b = p.i >> 2, q = p.i & 3;
        float v[8];
        matrix_order<WT>(r0, r1, v);
        uint4 part[3];
        split_parts(v, part);
        uint8_t *dst = img + (image_step<WT>(b, q) * ntok + p.t) * kImageBytes + 16 * image_group<WT>(b, q);
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4 *>(dst + 64 * k) = part[k];
    };
    ImagePiece p = {0, (int)threadIdx.x};
    p.settle(4 * nblk);
    if constexpr (AHEAD) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            if (p.t < ntok) put(p, ahead.r[n][0], ahead.r[n][1]);
            __builtin_amdgcn_sched_barrier(0);     // one after the other: fewer registers
            p.i += threads;
            p.settle(4 * nblk);
        }
    }
#pragma nounroll
    while (p.t < ntok) {
        rt_f32x4 r0, r1;
        image_load<WT>(p, ntok, b0, nb, row, r0, r1);
        put(p, r0, r1);
        p.i += threads;
        p.settle(4 * nblk);
    }
}

// One unit of a tile's rows in registers: codes, and the scales of the lane's
// row.
template <int WT, int SS>
struct Unit {
    static constexpr int SB = RowFmt<WT, SS>::SPU;
    uint4 q;
    uint32_t s[(SB + 3) / 4];
};

// Swap helpers: rows of 32 (or 16) lanes of two registers exchanged so that
// a keeps the lower ones of both and b the upper ones.
__device__ inline void rt_swap32(uint32_t &a, uint32_t &b)
{
    const auto p = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = p[0];
    b = p[1];
}
__device__ inline void rt_swap16(uint32_t &a, uint32_t &b)
{
    const auto p = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = p[0];
    b = p[1];
}

typedef uint32_t rt_u32x4 __attribute__((ext_vector_type(4)));

// The codes of unit qi of the lane's row: 16 bytes of it each, 64 bytes of
// sixteen rows per load.  (Two units of eight rows, whole cache lines, streamed
// no faster, and handing each lane its own row afterwards took registers that
// hold units in flight now.)
//
// Always the same loads in the same order, whatever the row's length: a
// branch around a load would make the compiler wait for every load in flight,
// the next unit's among them.  Every address lies inside the row: units past
// its end repeat its last 16 bytes (the activations there are zeros and
// multiply_unit zeroes the scales).
template <int WT, int SS>
__device__ inline void load_codes(Unit<WT, SS> &z, const uint8_t *row, int qoff, int code_bytes, int qi, int g)
{
    const int c = 64 * qi + 16 * g, top = code_bytes - 16;
    z.q = *reinterpret_cast<const uint4 *>(row + (uint32_t)(qoff + (c < top ? c : top)));
}

// SB bytes at an address aligned to SB.
template <int SB>
__device__ inline void scale_words(const uint8_t *s, uint32_t (&out)[(SB + 3) / 4])
{
    if constexpr (SB == 2) {
        out[0] = *reinterpret_cast<const uint16_t *>(s);
    } else if constexpr (SB == 4) {
        out[0] = *reinterpret_cast<const uint32_t *>(s);
    } else {
        static_assert(SB == 8, "scale bytes of a unit");
        const uint2 v = *reinterpret_cast<const uint2 *>(s);
        out[0] = v.x;
        out[1] = v.y;
    }
}

// Codes and scales of one unit.  A unit past the row's end (last_q) has the
// scales of its last; the scale bytes of a unit with any block of the row end
// at or before the row's end, because the row's codes follow its scales.
template <int WT, int SS>
__device__ inline void load_unit(Unit<WT, SS> &z, const uint8_t *row, int qoff, int code_bytes, int qi, int last_q, int g)
{
    constexpr int SB = Unit<WT, SS>::SB;
    load_codes<WT, SS>(z, row, qoff, code_bytes, qi, g);
    scale_words<SB>(row + (uint32_t)(SB * (qi < last_q ? qi : last_q)), z.s);
}

// The scales of D consecutive steps of a wave's rows, in one load: lane group
// g takes the g-th 16 bytes of its row (with HALF the eight lanes of a row one
// piece each), and a piece of LDS of the wave's own hands every lane the
// scales it multiplies by.  One load per unit for its scales, four lanes
// reading the same bytes, takes the texture units as long as 1 KB of codes:
// streaming 94 MB of MXFP4 rows took 21.9 us with it, 18.8 with one load per
// row, 18.4 with no scales at all.
template <int WT, int SS, bool HALF, int D>
struct ScaleWindow {
    static constexpr int SB = RowFmt<WT, SS>::SPU;
    static constexpr int STEP = SB * (HALF ? 2 : 1), PIECES = (D * STEP + 15) / 16;
    static constexpr int STRIDE = HALF ? 144 : 80;         // rows on different banks
    static_assert(PIECES <= (HALF ? 8 : 4), "one piece per lane");
    typedef uint32_t words __attribute__((ext_vector_type(4), aligned(2)));
    words next;

    // Steps p .. p + D - 1 of the lane's row of row_bytes bytes, clamped so that
    // every address lies in the row: its last 16 bytes are codes.
    __device__ inline void load(const uint8_t *row, int row_bytes, int p, int g, bool upper)
    {
        const int piece = HALF && upper ? 4 + g : g;
        const int at = STEP * p + 16 * (piece < PIECES ? piece : PIECES - 1), top = row_bytes - 16;
        next = *reinterpret_cast<const words *>(row + (uint32_t)(at < top ? at : top));
    }
    __device__ inline void put(uint8_t *lds, int j, int g) const
    {
        const int row = HALF ? j & 7 : j, piece = HALF && j >= 8 ? 4 + g : g;
        __builtin_amdgcn_wave_barrier();
        *reinterpret_cast<uint4 *>(lds + row * STRIDE + 16 * piece) = make_uint4(next.x, next.y, next.z, next.w);
        __builtin_amdgcn_wave_barrier();
    }
    __device__ inline void get(Unit<WT, SS> &z, const uint8_t *lds, int d, int j) const
    {
        const int row = HALF ? j & 7 : j;
        scale_words<SB>(lds + row * STRIDE + (HALF ? 2 * d + (j >= 8 ? 1 : 0) : d) * SB, z.s);
    }
};
static_assert(kScaleLds >= 16 * 80 && kScaleLds >= 8 * 144, "a wave's LDS for it");

// The sum of a lane's row and token over the instructions so far.  MXFP4 keeps
// the matrix instruction's own accumulators (one per part, added at the end;
// with HALF one set for each half of the columns).
template <int WT, bool HALF>
struct RowAcc {
    rt_f32x4 c[WT == W_MXFP4 && HALF ? 2 : 1] = {};
};
template <int WT, bool HALF>
__device__ inline float row_total(const RowAcc<WT, HALF> &a, bool upper)
{
    if constexpr (WT == W_MXFP4 && HALF) {
        const float lo = a.c[0][0] + a.c[0][1] + a.c[0][2], hi = a.c[1][0] + a.c[1][1] + a.c[1][2];
        return upper ? hi : lo;
    } else if constexpr (WT == W_MXFP4) {
        return a.c[0][0] + a.c[0][1] + a.c[0][2];
    } else {
        return a.c[0][0];
    }
}

// Byte E of w as a signed int8, converted to float (one SDWA conversion).
template <int E>
__device__ inline float rt_sbyte(uint32_t w) { return (float)(int8_t)(w >> (8 * E)); }
__device__ inline uint32_t rt_pack(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(rt_f32x2{a, b}, rt_bf16x2));
}

// Multiplies the units in z with the activation fragments of token groups
// tg < groups.  frag(tg, half, step) is the fragment of instruction `step` of
// the unit that columns 8 half .. 8 half + 7 hold.  Without HALF all
// sixteen columns are rows of the same unit (half is 0); with it columns
// 0 .. 7 are eight rows' unit 2 q and columns 8 .. 15 the same rows' unit
// 2 q + 1, so that a tile of eight rows still loads sixteen columns at once:
// each weight fragment meets both halves' activations, and each half of the
// columns keeps its own product.  qi: this lane's unit; whole: whether every
// column's unit lies in the row to its last block; nb: blocks of the row.
template <int WT, int SS, int TG, bool HALF, class Frag>
__device__ inline void multiply_unit(const Unit<WT, SS> &z, int qi, bool whole, int nb, int g, bool upper, int groups,
                                        RowAcc<WT, HALF> (&acc)[TG], Frag frag)
{
    using F = RowFmt<WT, SS>;
    constexpr int H = HALF ? 2 : 1;
    const int left = whole ? F::MF : nb - qi * F::MF;      // blocks of this unit in the row
    rt_bf16x8 fr[TG][H][F::MF];
#pragma unroll
    for (int t = 0; t < F::MF; ++t)
#pragma unroll
        for (int tg = 0; tg < TG; ++tg)
            if (tg < groups) {
#pragma unroll
                for (int h = 0; h < H; ++h) fr[tg][h][t] = frag(tg, h, t);
            }
    __builtin_amdgcn_sched_barrier(0);
    uint32_t d[4] = {z.q.x, z.q.y, z.q.z, z.q.w};
    if constexpr (WT == W_MXFP4) {
        // lane group g holds block g of the unit: its scale byte
        // as the exponent of a float (255 is NaN, 0 is 2^-127)
        uint32_t e = (z.s[0] >> (8 * g)) & 0xFFu;
        if (!whole) e = g < left ? e : 0u;
        const float f = __builtin_bit_cast(float, e << 23);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint4 bw = make_uint4(
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d[t], f, 0)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d[t], f, 1)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d[t], f, 2)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d[t], f, 3)));
            const rt_bf16x8 b = __builtin_bit_cast(rt_bf16x8, bw);
#pragma unroll
            for (int tg = 0; tg < TG; ++tg)
                if (tg < groups) {
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        acc[tg].c[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fr[tg][h][t], b, acc[tg].c[h], 0, 0, 0);
                }
        }
    } else {
        rt_swap32(d[0], d[2]);
        rt_swap32(d[1], d[3]);
        if constexpr (WT == W_Q4_0) {
            rt_swap16(d[0], d[1]);
            rt_swap16(d[2], d[3]);
        }
#pragma unroll
        for (int t = 0; t < F::MF; ++t) {
            uint4 bw;
            if constexpr (WT == W_Q4_0) {
                // a nibble n at the top of a byte with its top bit flipped
                // is the int8 value 16 (n - 8); the scale absorbs the 16
                const uint32_t x = d[t] ^ 0x88888888u;
                const uint32_t lo = (x << 4) & 0xF0F0F0F0u, hi = x & 0xF0F0F0F0u;
                bw = make_uint4(rt_pack(rt_sbyte<0>(lo), rt_sbyte<0>(hi)), rt_pack(rt_sbyte<1>(lo), rt_sbyte<1>(hi)),
                                rt_pack(rt_sbyte<2>(lo), rt_sbyte<2>(hi)), rt_pack(rt_sbyte<3>(lo), rt_sbyte<3>(hi)));
            } else {
                const uint32_t a = d[2 * t], c = d[2 * t + 1];
                bw = make_uint4(rt_pack(rt_sbyte<0>(a), rt_sbyte<1>(a)), rt_pack(rt_sbyte<2>(a), rt_sbyte<3>(a)),
                                rt_pack(rt_sbyte<0>(c), rt_sbyte<1>(c)), rt_pack(rt_sbyte<2>(c), rt_sbyte<3>(c)));
            }
            const rt_bf16x8 b = __builtin_bit_cast(rt_bf16x8, bw);
            const int sh = t >> SS;                        // the block's scale (a half) within the unit
            const uint32_t sb = (sh & 1) ? z.s[sh / 2] >> 16 : z.s[sh / 2] & 0xFFFFu;
            float f = (float)__builtin_bit_cast(_Float16, (uint16_t)sb);
            if constexpr (WT == W_Q4_0) f *= 0.0625f;
            if (!whole) f = t < left ? f : 0.0f;
#pragma unroll
            for (int tg = 0; tg < TG; ++tg)
                if (tg < groups) {
                    const rt_f32x4 zero = {0, 0, 0, 0};
                    const rt_f32x4 s0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fr[tg][0][t], b, zero, 0, 0, 0);
                    float sum = s0[0] + (s0[1] + s0[2]);
                    if constexpr (HALF) {
                        const rt_f32x4 s1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fr[tg][1][t], b, zero, 0, 0, 0);
                        const float other = s1[0] + (s1[1] + s1[2]);
                        sum = upper ? other : sum;
                    }
                    acc[tg].c[0][0] = fmaf(f, sum, acc[tg].c[0][0]);
                }
        }
    }
}

// A wave's run over its n units (or items) 0 .. n - 1 with D of them in
// registers: `stream_begin` loads the first D, `stream` multiplies each and
// loads the one D later into its place.  The places are fixed at compile time:
// moving a loaded register would wait for its load, so that only one unit
// were ever in flight.  load(d, i) fills place d; use(d, i) consumes it;
// head(more, i) is called before each D of them with the index of the next D
// and whether there are any.  Past the end the last one is loaded again (from
// the caches), so that every load is unconditional: a place loaded on one of
// two paths would be copied where they meet, and waited for there.  Every path
// into `stream` has to issue the loads in this order too, since the compiler
// waits for the fewest loads that may have followed on any of them.
template <int FROM, int TO, class Load>
__device__ inline void stream_begin(int n, Load load)
{
    static_steps<TO - FROM>([&](auto i) {
        constexpr int d = FROM + decltype(i)::value;
        load(std::integral_constant<int, d>{}, d < n ? d : n > 0 ? n - 1 : 0);
        __builtin_amdgcn_sched_barrier(0);
    });
}
template <int D, class Head, class Load, class Use>
__device__ inline void stream(int n, Head head, Load load, Use use)
{
    int i = 0;
    for (; n - i > D; i += D) {
        head(std::true_type{}, i + D);
        __builtin_amdgcn_sched_barrier(0);
        static_steps<D>([&](auto d) {
            const int k = i + (int)d.value;
            use(d, k);
            __builtin_amdgcn_sched_barrier(0);
            load(d, k + D < n ? k + D : n - 1);
            __builtin_amdgcn_sched_barrier(0);
        });
    }
    head(std::false_type{}, 0);
    static_steps<D>([&](auto d) {
        if (i + (int)d.value < n) use(d, i + (int)d.value);
    });
}

// Swish(z) = z * sigma(z) = z / (1 + e^{-z}) in binary32; for z far below
// zero e^{-z} overflows and the quotient is the limit -0.
__device__ inline float rt_swish(float z)
{
    return z / (1.0f + expf(-z));
}

}  // namespace qmm
