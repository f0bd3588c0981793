// lora_plan.h -- how the two launches of an adapter call split their work: host
// code, apart from the kernels so that it can be built and checked alone.
// Internal to the library.
#pragma once

#include "qmm_internal.h"

namespace qmm {

constexpr int kShrinkWaves = 8;      // of a workgroup of the first launch, which share its part of K
constexpr int kMostParts = 4;        // of K

struct LoraPlan {
    int rt;              // 16-rank tiles: 1, 2, 4 or 8
    bool single;         // one launch, which needs no workspace
    bool tiled;          // the first launch: tiles of 32 tokens through LDS (else of 16, through registers)
    int chunk, chunks;   // K per workgroup of the first launch (a multiple of 64), and its parts
    int j1, j2;          // workgroups (of each launch) that share a tile's adapters
    int mt;              // output tiles per workgroup: of 128 in the second launch (1, 2, 4 or 8), of 512 in the one
    int64_t m_blocks;    // workgroups along the outputs of the second launch
    int64_t blocks1, blocks2;
};

inline bool lora_wide(const void *x, uint64_t pitch_elems, bool f32x)
{
    return (uintptr_t)x % 16 == 0 && pitch_elems % (f32x ? 4 : 8) == 0;
}

// wide: x's rows are 16-byte aligned, as the loads to LDS want them.
inline LoraPlan plan_lora(int64_t N, int64_t K, int64_t M, int64_t r, bool wide, int64_t cus)
{
    LoraPlan p = {};
    p.rt = r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8;
    // The one launch: a workgroup per CU where the tokens allow it (64 tokens of rank
    // 16, 2048 x 5632: 6.5 us, 11.6 with a workgroup for each 512 outputs, 14.0 with two
    // launches).  Each token's workgroups read all of its A, so that its time goes
    // with r K and the rounds of tokens; two launches read a matrix once for the
    // tokens of a tile that share it, but go through a tile's adapters one after
    // the other, and which tokens share one is not known here.  us in a graph, one
    // launch, then two with 24 adapters in turn / with four prompts:
    //   256 tokens, rank 16, 2048 x 2048    6.9   17.4 / 12.3
    //   256 tokens, rank 64, 2048 x 2048   19.7   31.3 / 14.0
    //   256 tokens, rank 64, 5632 x 4096   43.1   61.3 / 17.7
    //  1024 tokens, rank 16, 2048 x 2048   18.3   80.1 / 13.8
    //  1024 tokens, rank 64, 2048 x 2048   69.1  126.4 / 19.0
    //    16 tokens, rank 64, 2048 x 2048   12.6   14.2
    //     1 token,  rank 64, 2048 x 2048   12.3   11.0
    //     1 token,  rank 16, 5632 x 2048    9.7    8.2
    //     1 token,  rank 16, 2048 x 2048    5.3    7.9
    p.single = N <= 4 * cus && r * K * ((N + cus - 1) / cus) <= (N < 16 ? 1 << 16 : 1 << 17);
    if (p.single) {
        const int64_t tiles = (M + 511) / 512, groups = N < cus ? cus / N : 1;
        p.mt = (int)((tiles + groups - 1) / groups);
        return p;
    }
    // Few tokens are decoded ones, which may all have different adapters:
    // workgroups share a tile's until there are `want` of them.  Prompts' tiles
    // have one, or two where one prompt ends: with one workgroup for both such a
    // tile took twice as long as all others (1021 tokens of three prompts, rank
    // 128: 16.8 and 19.5 us for the two launches, 10.9 and 12.7 without ends).
    auto share = [](int64_t groups, int64_t want, int64_t tokens) {
        int j = 1;
        while (j < tokens && groups * j < want) j *= 2;
        return j;
    };
    // Tiles of 32 tokens through LDS want tokens that share an adapter, tiles of 16
    // through registers take different ones better, and more tokens are prompts more
    // often.  us in a graph, registers then tiles, four prompts / 24 adapters in turn:
    //   512 tokens, rank 64, 2048 x 2048, bf16 x    15.8 and 12.7 / 41.7 and 55.5
    //   640 tokens                                  20.2 and 13.6 / 53.8 and 60.7
    //  1024 tokens                                  21.1 and 14.6 / 67.7 and 65.5
    //   640 tokens, rank 128, 2048 x 5632           51.6 and 22.8 / 171 and 123
    //   640 tokens, rank 64, 2048 x 2048, fp32 x    22.1 and 17.7 / 60.1 and 103
    p.tiled = wide && N > 512;
    const int64_t tile1 = p.tiled ? 32 : 16, tiles1 = (N + tile1 - 1) / tile1;
    int64_t parts = (p.tiled ? 2 : 1) * cus / tiles1;
    if (parts > kMostParts) parts = kMostParts;
    if (parts > K / 1024) parts = K / 1024;              // four steps of 32 for each of eight waves
    if (parts < 1) parts = 1;
    p.chunk = (int)((K + 64 * parts - 1) / (64 * parts) * 64);
    p.chunks = K > 0 ? (int)((K + p.chunk - 1) / p.chunk) : 0;
    p.j1 = p.tiled ? 2 : share(tiles1 * p.chunks, 2 * cus, N < tile1 ? N : tile1);
    p.blocks1 = tiles1 * p.chunks * p.j1;
    const int64_t tiles2 = (N + 31) / 32, m_tiles = (M + 127) / 128;
    p.mt = 1;
    // As many as leave a workgroup with work per CU: each first joins the parts of
    // u, which takes longer for high ranks (both launches, us in a graph, with 1, 2, 4
    // and 8 tiles each: 1021 tokens, rank 128, 2048 outputs 25.4, 21.4, 22.6, 29.3;
    // 4093 tokens, rank 128 61.4, 45.8, 38.7, 35.2, rank 16 26.4, 23.0, 21.9, 24.6).
    while (p.mt < (p.rt < 4 ? 4 : 8) && tiles2 * ((m_tiles + 2 * p.mt - 1) / (2 * p.mt)) >= cus) p.mt *= 2;
    p.m_blocks = (m_tiles + p.mt - 1) / p.mt;
    p.j2 = p.tiled ? 2 : share(tiles2 * p.m_blocks, 2 * cus, N < 32 ? N : 32);
    p.blocks2 = tiles2 * p.m_blocks * p.j2;
    return p;
}

}  // namespace qmm
