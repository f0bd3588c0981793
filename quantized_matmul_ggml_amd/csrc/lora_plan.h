// lora_plan.h -- how the two launches of an adapter call split their work: host
// code, apart from the kernels so that it can be built and checked alone.
// Internal to the library.
#pragma once

#include "qmm_internal.h"

namespace qmm {

struct LoraPlan {
    int rt;              // 16-rank tiles: 1, 2, 4 or 8
    int chunk, chunks;   // K per wave of the first launch (a multiple of 32), and its parts
    int j1, j2;          // waves (first launch) or workgroups (second) that share a tile's adapters
    int mt;              // 32-output tiles per wave of the second launch
    int64_t tasks1;      // waves of the first launch
    int64_t m_blocks;    // workgroups along the outputs of the second launch
    int64_t blocks2;     // its workgroups
};

// The first launch has a wave per 16 tokens, part of K and share of the tile's
// adapters; the second a workgroup per 32 tokens, 4 mt tiles of 32 outputs and
// share of the adapters.
inline LoraPlan plan_lora(int64_t N, int64_t K, int64_t M, int64_t r, int64_t cus)
{
    LoraPlan p = {};
    p.rt = r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8;
    const int64_t want = 8 * cus;                        // two waves on every SIMD
    const int64_t tiles1 = (N + 15) / 16;
    int64_t parts = (want + tiles1 - 1) / tiles1;
    if (parts > 16) parts = 16;
    int64_t chunk = (K + 32 * parts - 1) / (32 * parts) * 32;
    if (chunk < 128) chunk = 128;
    p.chunk = (int)chunk;
    p.chunks = K > 0 ? (int)((K + chunk - 1) / chunk) : 0;
    auto share = [](int64_t waves, int64_t target, int64_t most) {
        int j = 1;
        while (j < most && waves * j < target) j *= 2;
        return j;
    };
    const int64_t tokens1 = N < 16 ? N : 16, tokens2 = N < 32 ? N : 32;
    p.j1 = share(tiles1 * p.chunks, want, tokens1);
    p.tasks1 = tiles1 * p.chunks * p.j1;
    const int64_t tiles2 = (N + 31) / 32, m_tiles = (M + 31) / 32;
    p.mt = 1;
    while (p.mt < 8 && tiles2 * ((m_tiles + 8 * p.mt - 1) / (8 * p.mt)) >= 2 * cus) p.mt *= 2;
    p.m_blocks = (m_tiles + 4 * p.mt - 1) / (4 * p.mt);
    p.j2 = share(tiles2 * p.m_blocks, 2 * cus, tokens2);
    p.blocks2 = tiles2 * p.m_blocks * p.j2;
    return p;
}

}  // namespace qmm
