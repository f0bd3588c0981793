// grouped_tile.h -- how a workgroup of the grouped products finds its tile from
// the groups' offsets.  Internal to the library.
#pragma once

#include "qmm_internal.h"

namespace qmm {

// The operands of a launch of grouped products.
struct GrpArgs {
    const uint8_t *w, *w2;        // SwiGLU: the gate and the up matrices
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
    int32_t m_tiles;              // tiles along the weight rows
    int32_t bf16_out, split_out;  // split_out: GroupedOut's two parts
    int32_t tiles_per_wave;       // gemm_rows.hip
};

// A group of rows: expert e's [first, end), cut to the rows that there are,
// whatever the offsets hold.
__device__ inline void group_rows(const int32_t *offsets, int e, int R, int &first, int &end)
{
    const int a = offsets[e], b = offsets[e + 1];
    first = a < 0 ? 0 : a > R ? R : a;
    end = b < first ? first : b > R ? R : b;
}

// A workgroup's tile: expert e, grouped rows n0 .. n0 + rows - 1, weight tile mt.
struct GroupTile {
    int e, n0, rows, mt;
};

// Finds it, with all waves of the workgroup; false: there is none.  The launch has
// a workgroup for every tile of BN rows that R rows of E groups can need, in an
// order (expert, weight tile, row tile) whose consecutive tiles share weights;
// the eight XCDs (workgroup b runs on XCD b mod 8) take contiguous parts of the
// tiles that there are.  Each lane counts the row tiles of a run of experts, without
// sign: descending offsets can make groups that overlap, whose tiles the count may
// not hold; then too no tile lies outside the operands.
template <int BN>
__device__ inline bool find_tile(const GrpArgs &a, GroupTile &t)
{
    const int lane = threadIdx.x & 63;
    const int run = (a.E + 63) / 64;
    uint32_t counted = 0;
    for (int i = 0; i < run; ++i) {
        const int e = lane * run + i;
        if (e < a.E) {
            int first, end;
            group_rows(a.offsets, e, a.R, first, end);
            counted += (uint32_t)(end - first + BN - 1) / BN;
        }
    }
    const int mine = (int)counted;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const uint32_t o = __shfl_up(counted, m);
        counted += lane >= m ? o : 0;
    }
    const int upto = (int)counted;
    const int64_t total = (int64_t)__builtin_amdgcn_readlane(upto, 63) * a.m_tiles;
    if ((int64_t)blockIdx.x >= total) return false;
    const int nwg = (int)(total < (int64_t)gridDim.x ? total : (int64_t)gridDim.x);
    const int x8 = (int)blockIdx.x % 8, q8 = nwg / 8, r8 = nwg % 8;
    const int at = x8 * q8 + (x8 < r8 ? x8 : r8) + (int)blockIdx.x / 8;
    const int row_tile = at / a.m_tiles;
    const int owner = __builtin_ctzll(__ballot(upto > row_tile));
    int before = __builtin_amdgcn_readlane(upto, owner) - __builtin_amdgcn_readlane(mine, owner);
    if (before < 0 || before > row_tile) return false;
    int e = owner * run, first = 0, end = 0, tiles = 0;
    for (;; ++e) {
        if (e >= a.E) return false;
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
    t.e = e;
    t.mt = __builtin_amdgcn_readfirstlane(local / tiles);
    t.n0 = first + (local - t.mt * tiles) * BN;
    t.rows = end - t.n0 < BN ? end - t.n0 : BN;
    return true;
}

// Value m of a row, in two parts: rounded to bf16 (cut, where that gives an infinity),
// and what is left, rounded, so that their sum is within 2^-16 of it.  An infinity is
// its own first part.
__device__ inline void store_split(uint16_t *row, int64_t m, float v)
{
    const float near = (float)(__bf16)v, cut = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xFFFF0000u);
    const float first = fabsf(near) == INFINITY ? cut : near;
    const float rest = fabsf(first) == INFINITY ? 0.0f : v - first;
    uint16_t *const p = row + m + (m & ~31);
    p[0] = (uint16_t)(__builtin_bit_cast(uint32_t, first) >> 16);
    p[32] = __builtin_bit_cast(uint16_t, (__bf16)rest);
}

// The token of grouped row r, or -1 if it is none of x's.
__device__ inline int token_of(const GrpArgs &a, int r)
{
    if (!a.order) return r;
    const int slot = a.order[r];
    const int token = slot >= 0 ? slot / a.top_k : -1;
    return token < a.N ? token : -1;
}

hipError_t launch_gemm_rows(GrpArgs &a, int type, int scale_shift, bool swiglu, int parts, hipStream_t stream);

}  // namespace qmm
