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
    int mt;              // 128-output tiles per workgroup of the second launch: 1, 2, 4 or 8
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
    // Every workgroup of the one launch (a token and 512 outputs) reads all of its
    // token's A: worth it while that is little (us in a graph, one launch against two;
    // rank 16, 2048 x 2048: one token 5.2 / 7.8, 64 tokens 5.6 / 12.2, 128 tokens
    // 8.4 / 12.7; 2048 x 5632: 64 tokens 11.4 / 13.9, 128 tokens 19.3 / 16.7; rank 16
    // of 5632 for one token 9.6 / 8.3, rank 64 of 2048 12.2 / 11.0).
    p.single = N <= 256 && r * K <= 1 << 16 && N * ((M + 511) / 512) * r * K <= 1 << 25;
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
    while (p.mt < 8 && tiles2 * ((m_tiles + 2 * p.mt - 1) / (2 * p.mt)) >= 2 * cus) p.mt *= 2;
    p.m_blocks = (m_tiles + p.mt - 1) / p.mt;
    p.j2 = p.tiled ? 2 : share(tiles2 * p.m_blocks, 2 * cus, N < 32 ? N : 32);
    p.blocks2 = tiles2 * p.m_blocks * p.j2;
    return p;
}

}  // namespace qmm
