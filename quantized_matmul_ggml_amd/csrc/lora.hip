// lora.hip -- low-rank adapters of many requests at once, beside a projection
// that all of them share:
//   y[n] = base[n] + s_a B_a (A_a x[n]),   a = ids[n],
// A_a: r x K, B_a: M x r (bf16), for tokens of any mix of adapters.
//
// Two launches.  The first makes u = A_a x: a workgroup takes 16 or 32 tokens
// and a part of K (all of it where the tokens alone fill the chip) and goes
// through the different adapters among its tokens (a prompt's are all the same
// one; decoded tokens' may be sixteen); the parts' sums go to the workspace.  The
// second makes base + B_a (s_a u) for 32 tokens and tiles of 128 outputs.  In
// both, each adapter's products are made for all tokens of the tile and kept for
// its own, so no token's values meet another's; where there are few tiles,
// workgroups share a tile's adapters.  One or a few tokens take one launch.
//
// Arithmetic: binary32 values (x when it is F32, and s_a u) enter the matrix
// cores as three bf16 parts whose sum is exact (row_tiles.h), so every product
// is exact and only binary32 sums and s_a u round.
//
// Bound by memory: decoding by the adapters' matrices (read once per tile of
// tokens that uses them) and the launches' latency, prompts by base and y.
#include "lds_load.h"
#include "lora_plan.h"
#include "row_tiles.h"

namespace qmm {
namespace {

typedef float lr_f32x16 __attribute__((ext_vector_type(16)));

struct LoraArgs {
    const uint16_t *a, *b;
    uint64_t a_pitch, b_pitch;         // elements between rows
    uint64_t a_adapter, b_adapter;     // elements between adapters
    const void *x;
    uint64_t x_pitch;
    const int32_t *ids;
    const float *scales;               // NULL: 1
    const float *base;                 // NULL: 0
    uint64_t base_pitch;
    float *y;
    uint64_t y_pitch;
    float *u;                          // [part][token][rp]
    int64_t N, M;
    int32_t L, K, r, rp;
    int32_t chunk, chunks;             // K per part, parts
    int32_t j1, j2;                    // workgroups that share a tile's adapters
    int32_t mt;                        // output tiles per workgroup: 128 (second launch), 512 (the one launch)
    int64_t m_blocks;                  // workgroups along M of the second launch
};

// Calls f(adapter, tokens of the tile that use it) for the adapters j, j + J, ..
// among the tile's tokens (lane t holds token t's, or a negative number).
template <class F>
__device__ inline void for_adapters(int id, uint64_t tokens, int j, int J, F f)
{
    uint64_t left = __ballot(id >= 0) & tokens;
    for (int i = 0; left; i = i + 1 == J ? 0 : i + 1) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t m = __ballot(id == a) & left;
        left &= ~m;
        if (i == j) f(a, m);
    }
}

// This workgroup's place in an order of which each of the eight XCDs (workgroup
// b runs on XCD b mod 8, each with its own L2) takes a contiguous part: a
// prompt's tiles, which read the same adapter, then share an L2.
__device__ inline uint32_t xcd_place()
{
    const uint32_t b = blockIdx.x, n = gridDim.x, x = b % 8, q = n / 8, r = n % 8;
    return x * q + (x < r ? x : r) + b / 8;
}

__device__ inline rt_bf16x8 load8(const uint16_t *p)
{
    return __builtin_bit_cast(rt_bf16x8, *reinterpret_cast<const uint4 *>(p));
}

// A wave's part k_from .. k_to - 1 of u for the sixteen tokens whose rows (elements
// from x on) its lanes hold: token c, rank 16 t + c of the adapter at `rows`.
template <bool F32X, int RT>
__device__ inline void shrink_steps(const LoraArgs &a, uint64_t row, const uint16_t *rows, int k_from, int k_to, int c, int g,
                                    rt_f32x4 (&acc)[RT])
{
    constexpr int PARTS = F32X ? 3 : 1, U = RT == 8 ? 2 : 4;
    // S steps of 32 from k0 on: all loads, then all products
    auto steps = [&](auto count, int k0) {
        constexpr int S = decltype(count)::value;
        rt_f32x4u v[S][F32X ? 2 : 1];
        rt_bf16x8 w[S][RT];
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int k = k0 + 32 * i + 8 * g;
            if constexpr (F32X) {
                const float *p = static_cast<const float *>(a.x) + row + k;
                v[i][0] = *reinterpret_cast<const rt_f32x4u *>(p);
                v[i][1] = *reinterpret_cast<const rt_f32x4u *>(p + 4);
            } else {
                v[i][0] = __builtin_bit_cast(rt_f32x4, load8(static_cast<const uint16_t *>(a.x) + row + k));
            }
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const int r = 16 * t + c < a.r ? 16 * t + c : a.r - 1;
                w[i][t] = load8(rows + (uint64_t)r * a.a_pitch + k);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < S; ++i) {
            uint4 xp[PARTS];
            if constexpr (F32X) {
                const float f[8] = {v[i][0][0], v[i][0][1], v[i][0][2], v[i][0][3], v[i][1][0], v[i][1][1], v[i][1][2], v[i][1][3]};
                split_parts(f, xp);
            } else {
                xp[0] = __builtin_bit_cast(uint4, (rt_f32x4)v[i][0]);
            }
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(rt_bf16x8, xp[p]), w[i][t], acc[t], 0, 0, 0);
        }
    };
    int k0 = k_from;
    for (; k0 + 32 * U <= k_to; k0 += 32 * U) steps(std::integral_constant<int, U>{}, k0);
    for (; k0 < k_to; k0 += 32) steps(std::integral_constant<int, 1>{}, k0);
}

// The first launch for few tokens: a tile of 16, each wave a part of K, loads
// straight to registers (they are few, and all in flight at once).  The waves'
// sums lie in LDS in register order, [wave][rank tile][register][lane].
template <bool F32X, int RT>
__global__ __launch_bounds__(512) void lora_shrink_kernel(const LoraArgs a)
{
    constexpr int REGS = RT * 4;
    extern __shared__ __attribute__((aligned(16))) float red[];
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t place = xcd_place();
    const int j = (int)(place % a.j1), chunk = (int)(place / a.j1 % a.chunks);
    const int64_t n0 = (int64_t)(place / a.j1 / a.chunks) * 16;
    const int64_t n = n0 + c < a.N ? n0 + c : a.N - 1;
    int id = a.ids[n];
    if (n0 + c >= a.N || id >= a.L) id = -1;
    const uint64_t row = (uint64_t)n * a.x_pitch;        // elements from x on
    const int c_to = (chunk + 1) * a.chunk < a.K ? (chunk + 1) * a.chunk : a.K;
    const int per = (a.chunk / 32 + kShrinkWaves - 1) / kShrinkWaves * 32;
    const int k_from = chunk * a.chunk + wave * per, k_to = k_from + per < c_to ? k_from + per : c_to;
    bool again = false;
    for_adapters(id, 0xFFFF, j, a.j1, [&](int ad, uint64_t mask) {
        const uint16_t *rows = a.a + (uint64_t)ad * a.a_adapter;
        rt_f32x4 acc[RT] = {};
        shrink_steps<F32X, RT>(a, row, rows, k_from, k_to, c, g, acc);
        if (again) __syncthreads();            // the last adapter's sums are no longer read
        again = true;
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[(wave * REGS + t * 4 + i) * 64 + lane] = acc[t][i];
        __syncthreads();
        // D: token 4 g + i, rank 16 t + c; the waves' sums in order
        for (int e = tid; e < REGS * 64; e += 512) {
            const int i = e >> 6 & 3, t = e >> 8, token = 4 * g + i;
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < kShrinkWaves; ++q) s += red[q * REGS * 64 + e];
            if ((mask >> token & 1) && 16 * t + c < a.r) a.u[((uint64_t)chunk * a.N + n0 + token) * a.rp + 16 * t + c] = s;
        }
    });
}

// The first launch for many tokens: a tile of 32 tokens and all ranks, K in
// steps of 64 that go through LDS (whole lines, kTileStages - 1 steps ahead).  A
// wave takes 32 ranks with v_mfma_f32_32x32x16_bf16; where the ranks have fewer
// than four such tiles, WK waves share one and split each step's K.
constexpr int kTileStages = 4;
template <bool F32X, int RT>
struct ShrinkTile {
    static constexpr int RG = RT < 2 ? 1 : RT / 2, WK = 4 / RG;      // rank tiles, waves of each
    static constexpr int XB = F32X ? 256 : 128;                      // bytes of a token's step
    static constexpr int X_BYTES = 32 * XB, A_BYTES = RG * 32 * 128;
    static constexpr int X_LOADS = X_BYTES / 4096, LOADS = X_LOADS + RG;
    static constexpr int STAGE = X_BYTES + A_BYTES;
    static constexpr int LDS = kTileStages * STAGE;
    static_assert(4 * 16 * 64 * 4 <= LDS, "the waves' sums fit the ring");
};
template <bool F32X, int RT>
__global__ __launch_bounds__(256) void lora_shrink_tile_kernel(const LoraArgs a)
{
    using T = ShrinkTile<F32X, RT>;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(lds);
    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t place = xcd_place();
    const int j = (int)(place % a.j1), chunk = (int)(place / a.j1 % a.chunks);
    const int64_t n0 = (int64_t)(place / a.j1 / a.chunks) * 32;
    int id = n0 + l32 < a.N ? a.ids[n0 + l32] : -1;
    if (id >= a.L) id = -1;
    const int toks = a.N - n0 < 32 ? (int)(a.N - n0) : 32;
    const int k_from = chunk * a.chunk, k_to = k_from + a.chunk < a.K ? k_from + a.chunk : a.K;
    const int steps = (k_to - k_from + 63) / 64;
    constexpr int ES = F32X ? 4 : 2, XU = T::XB / 16;        // bytes of an element, units of a token's step
    // 16-byte units of a row are placed by an XOR with bits of the row, so that
    // rows read together lie in different banks
    const ll_i32x4 xres = ll_rsrc(static_cast<const uint8_t *>(a.x) + (uint64_t)n0 * a.x_pitch * ES + (uint64_t)k_from * ES,
                                  (uint32_t)(((uint64_t)(toks - 1) * a.x_pitch + (uint64_t)(k_to - k_from)) * ES));
    uint32_t xoff[T::X_LOADS];
    int xk[T::X_LOADS];                                      // unit of step s in K iff XB s < xk
#pragma unroll
    for (int i = 0; i < T::X_LOADS; ++i) {
        const int u = 256 * i + tid, t = u / XU, unit = u % XU ^ (F32X ? t & 15 : t >> 1 & 7);
        xoff[i] = t < toks ? (uint32_t)((uint64_t)t * a.x_pitch * ES) + 16u * unit : OUT_OF_RANGE;
        xk[i] = t < toks ? (k_to - k_from) * ES - 16 * unit : INT32_MIN;
    }
    uint32_t aoff[T::RG];
    int ak[T::RG];
#pragma unroll
    for (int i = 0; i < T::RG; ++i) {
        const int u = 256 * i + tid, r = u / 8, unit = u % 8 ^ (r >> 1 & 7);
        aoff[i] = r < a.r ? (uint32_t)((uint64_t)r * a.a_pitch * 2) + 16u * unit : OUT_OF_RANGE;
        ak[i] = r < a.r ? (k_to - k_from) * 2 - 16 * unit : INT32_MIN;
    }
    const int rg = wave % T::RG, par = wave / T::RG;
    bool again = false;
    for_adapters(id, 0xFFFFFFFF, j, a.j1, [&](int ad, uint64_t mask) {
        const ll_i32x4 ares = ll_rsrc(a.a + (uint64_t)ad * a.a_adapter + k_from,
                                      (uint32_t)(((uint64_t)(a.r - 1) * a.a_pitch + (uint64_t)(k_to - k_from)) * 2));
        auto load = [&](int s, int stage) {                  // past the last step: zeros
            const uint32_t base = lds0 + (uint32_t)(stage * T::STAGE) + 1024u * wave;
#pragma unroll
            for (int i = 0; i < T::X_LOADS; ++i)
                ll_load<16>(xres, base + 4096u * i, T::XB * s < xk[i] ? xoff[i] + (uint32_t)(T::XB * s) : OUT_OF_RANGE);
#pragma unroll
            for (int i = 0; i < T::RG; ++i)
                ll_load<16>(ares, base + T::X_BYTES + 4096u * i, 128 * s < ak[i] ? aoff[i] + 128u * s : OUT_OF_RANGE);
        };
        if (again) __syncthreads();            // the last adapter's sums are no longer read
        again = true;
        lr_f32x16 acc = {};
        for (int s = 0; s < kTileStages - 1; ++s) load(s, s);
        int stage = 0, next = kTileStages - 1;
        for (int s = 0; s < steps; ++s) {
            ll_wait<T::LOADS * (kTileStages - 2)>();
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            load(s + kTileStages - 1, next);
            const uint8_t *st = lds + stage * T::STAGE;
#pragma unroll
            for (int q = 0; q < 4 / T::WK; ++q) {
                const int cu = 4 / T::WK * par + q;          // 16 of the step's 64 k
                const int ar = 32 * rg + l32;
                const rt_bf16x8 w = *reinterpret_cast<const rt_bf16x8 *>(st + T::X_BYTES + ar * 128 + 16 * ((2 * cu + h) ^ (ar >> 1 & 7)));
                if constexpr (F32X) {
                    const int u = 4 * cu + 2 * h;
                    const float4 lo = *reinterpret_cast<const float4 *>(st + l32 * 256 + 16 * (u ^ (l32 & 15)));
                    const float4 hi = *reinterpret_cast<const float4 *>(st + l32 * 256 + 16 * ((u + 1) ^ (l32 & 15)));
                    const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    uint4 xp[3];
                    split_parts(f, xp);
#pragma unroll
                    for (int p = 0; p < 3; ++p)
                        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(rt_bf16x8, xp[p]), w, acc, 0, 0, 0);
                } else {
                    const rt_bf16x8 x = *reinterpret_cast<const rt_bf16x8 *>(st + l32 * 128 + 16 * ((2 * cu + h) ^ (l32 >> 1 & 7)));
                    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, w, acc, 0, 0, 0);
                }
            }
            next = stage;
            stage = stage + 1 == kTileStages ? 0 : stage + 1;
        }
        // D: token 8 (i / 4) + 4 h + i % 4, rank 32 rg + l32; the WK waves' sums in
        // order, each wave a part of the registers
        ll_wait<0>();                          // no load may still write the ring
        constexpr int FR = 16 / T::WK;
        float fin[FR];
        if constexpr (T::WK > 1) {
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            float *red = reinterpret_cast<float *>(lds);
#pragma unroll
            for (int i = 0; i < 16; ++i) red[(wave * 16 + i) * 64 + lane] = acc[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < FR; ++i) {
                fin[i] = 0.0f;
#pragma unroll
                for (int q = 0; q < T::WK; ++q) fin[i] += red[((rg + T::RG * q) * 16 + FR * par + i) * 64 + lane];
            }
        } else {
#pragma unroll
            for (int i = 0; i < FR; ++i) fin[i] = acc[i];
        }
        const int rank = 32 * rg + l32;
#pragma unroll
        for (int i = 0; i < FR; ++i) {
            const int reg = FR * par + i, token = 8 * (reg / 4) + 4 * h + reg % 4;
            if ((mask >> token & 1) && rank < a.r) a.u[((uint64_t)chunk * a.N + n0 + token) * a.rp + rank] = fin[i];
        }
    });
}

// The second launch.  Its work is a list of items, an adapter's rows for one
// tile of 128 outputs: their B goes through LDS (whole lines), the next item's
// while this one is multiplied; u lies in the second buffer until it is in
// registers.
template <int RT>
__global__ __launch_bounds__(256) void lora_expand_kernel(const LoraArgs a)
{
    constexpr int RP = 16 * RT, LDU = RP + 4, UPR = RP / 8;         // 16-byte units of a row of B
    constexpr int B_BYTES = 128 * RP * 2, B_LOADS = B_BYTES / 4096;
    static_assert(32 * LDU * 4 <= B_BYTES, "u fits a buffer");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * B_BYTES];
    __shared__ int ad_list[32];
    __shared__ uint32_t mask_list[32];
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(lds);
    float *const us = reinterpret_cast<float *>(lds + B_BYTES);
    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t place = xcd_place();
    const int j = (int)(place % a.j2);
    const int64_t block = place / a.j2 % a.m_blocks, n0 = (int64_t)(place / a.j2 / a.m_blocks) * 32;
    int id = n0 + l32 < a.N ? a.ids[n0 + l32] : -1;
    if (id >= a.L) id = -1;
    // the rows that this workgroup writes: its adapters' tokens, and for one of
    // the workgroups the tokens without one
    uint32_t mine = 0;
    int n_ad = 0, first_ad = 0;
    for_adapters(id, 0xFFFFFFFF, j, a.j2, [&](int ad, uint64_t m) {
        if (n_ad == 0) first_ad = ad;
        if (tid == 0) {
            ad_list[n_ad] = ad;
            mask_list[n_ad] = (uint32_t)m;
        }
        ++n_ad;
        mine |= (uint32_t)m;
    });
    const uint32_t rows = mine | (j == 0 ? (uint32_t)__ballot(id < 0 && n0 + l32 < a.N) : 0);
    if (!rows) return;
    // B of adapter ad for outputs m0 .. m0 + 127
    uint32_t boff[B_LOADS];
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i) {
        const int u = 256 * i + tid, r = u / UPR, unit = u % UPR ^ (r / (16 / UPR) & (UPR - 1));
        boff[i] = 8 * unit < a.r ? (uint32_t)((uint64_t)r * a.b_pitch * 2) + 16u * unit : OUT_OF_RANGE;
    }
    auto load = [&](int ad, int64_t m0, int buf) {
        const int64_t left = a.M - m0 < 128 ? a.M - m0 : 128;
        const ll_i32x4 res = ll_rsrc(a.b + (uint64_t)ad * a.b_adapter + (uint64_t)m0 * a.b_pitch,
                                     (uint32_t)(((uint64_t)(left - 1) * a.b_pitch + a.r) * 2));
#pragma unroll
        for (int i = 0; i < B_LOADS; ++i) ll_load<16>(res, lds0 + (uint32_t)(buf * B_BYTES) + 4096u * i + 1024u * wave, boff[i]);
    };
    const int64_t m_first = block * a.mt * 128;
    const int tiles = a.M - m_first > (int64_t)(a.mt - 1) * 128 ? a.mt : (int)((a.M - m_first + 127) / 128);
    if (n_ad) load(first_ad, m_first, 0);
    // ---- s_a u of those tokens, the parts added in order: four ranks a thread at
    // a time, all loads in flight together ----
    constexpr int QUADS = 32 * RP / 4, PER = (QUADS + 255) / 256;
    rt_f32x4 v[PER][kMostParts] = {};
    float scale[PER] = {};
    const uint64_t part = (uint64_t)a.N * a.rp;
    if (a.chunks > 0) {                                  // without K there is no u
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = 256 * i + tid, t = e / (RP / 4), q = e % (RP / 4) * 4;
            const bool live = e < QUADS && (mine >> (t & 31) & 1) && q < a.r;
            const float *p = a.u + (live ? (uint64_t)(n0 + t) * a.rp + q : 0);
#pragma unroll
            for (int c = 0; c < kMostParts; ++c) v[i][c] = *reinterpret_cast<const rt_f32x4 *>(p + (c < a.chunks ? c : 0) * part);
            scale[i] = live && a.scales ? a.scales[a.ids[n0 + t]] : 1.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = 256 * i + tid, t = e / (RP / 4), q = e % (RP / 4) * 4;
        const bool live = (mine >> (t & 31) & 1) && q < a.r;
        rt_f32x4 s = v[i][0];
#pragma unroll
        for (int c = 1; c < kMostParts; ++c)
            if (c < a.chunks) s += v[i][c];
#pragma unroll
        for (int c = 0; c < 4; ++c) s[c] = live ? s[c] * scale[i] : 0.0f;
        if (e < QUADS) *reinterpret_cast<rt_f32x4 *>(us + t * LDU + q) = s;
    }
    __syncthreads();
    uint4 up[RT][3];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
        const float4 *p = reinterpret_cast<const float4 *>(us + l32 * LDU + 16 * q + 8 * h);
        const float4 lo = p[0], hi = p[1];
        const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        split_parts(v, up[q]);
    }
    // ---- the tiles ----
    // base and y go through buffers of the tile's rows; what is not this
    // workgroup's to read or write gets an offset out of range.
    const int64_t toks = a.N - n0 < 32 ? a.N - n0 : 32;
    auto buffer = [&](const float *p, uint64_t pitch) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(p) + (uint64_t)n0 * pitch, 0,
                                                 (int)(((uint64_t)(toks - 1) * pitch + a.M) * 4), BUFFER_FLAGS);
    };
    const __amdgpu_buffer_rsrc_t yres = buffer(a.y, a.y_pitch), bres = buffer(a.base ? a.base : a.y, a.base ? a.base_pitch : a.y_pitch);
    const uint32_t my_rows = rows >> (4 * h);
    auto offset = [&](int r, int64_t m, uint64_t pitch) {
        const int t = 8 * (r / 4) + r % 4;               // and 4 h
        return my_rows >> t & 1 && m < a.M ? (uint32_t)(t + 4 * h) * (uint32_t)(4 * pitch) + 4u * (uint32_t)m : OUT_OF_RANGE;
    };
    const int br = 32 * wave + l32;                      // its row of a tile of B
    const uint32_t b_row = (uint32_t)(br * RP * 2), b_sw = br / (16 / UPR) & (UPR - 1);
    int buf = 0;
    for (int i = 0; i < tiles; ++i) {
        const int64_t m0 = m_first + i * 128, m = m0 + br;
        float out[16];
#pragma unroll
        for (int r = 0; r < 16; ++r)
            out[r] = !a.base ? 0.0f
                             : __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(bres, offset(r, m, a.base_pitch), 0, 0));
        for (int k = 0; k < n_ad; ++k) {
            ll_wait<0>();
            // this item's B is there, and the other buffer (first: u) no longer read
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            if (k + 1 < n_ad) load(__builtin_amdgcn_readfirstlane(ad_list[k + 1]), m0, buf ^ 1);
            else if (i + 1 < tiles) load(first_ad, m0 + 128, buf ^ 1);
            const uint8_t *st = lds + buf * B_BYTES + b_row;
            buf ^= 1;
            lr_f32x16 d = {};
#pragma unroll
            for (int q = 0; q < RT; ++q) {
                const rt_bf16x8 w = *reinterpret_cast<const rt_bf16x8 *>(st + 16 * ((uint32_t)(2 * q + h) ^ b_sw));
#pragma unroll
                for (int s = 0; s < 3; ++s)
                    d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(rt_bf16x8, up[q][s]), w, d, 0, 0, 0);
            }
            const uint32_t my_mask = (uint32_t)__builtin_amdgcn_readfirstlane(mask_list[k]) >> (4 * h);
#pragma unroll
            for (int r = 0; r < 16; ++r) out[r] = my_mask >> (8 * (r / 4) + r % 4) & 1 ? out[r] + d[r] : out[r];
        }
#pragma unroll
        for (int r = 0; r < 16; ++r)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, out[r]), yres, offset(r, m, a.y_pitch), 0, 0);
    }
    ll_wait<0>();
}

// One launch for few tokens: a workgroup takes one token and mt tiles of 512
// outputs.  It makes all of the token's u for itself (its adapter's A then comes
// from the L2 for all workgroups but the first) and has its first rows of B in
// flight meanwhile.  The outputs are one thread's sums over the ranks, exact
// products in binary32.
template <bool F32X, int RT>
__global__ __launch_bounds__(512) void lora_token_kernel(const LoraArgs a)
{
    __shared__ float part[kShrinkWaves][16 * RT];
    __shared__ __attribute__((aligned(16))) float us[16 * RT];
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t n = blockIdx.y, m_first = (int64_t)blockIdx.x * a.mt * 512 + tid;
    const int tiles = a.M - (m_first - tid) > (int64_t)(a.mt - 1) * 512 ? a.mt : (int)((a.M - (m_first - tid) + 511) / 512);
    const int ad = __builtin_amdgcn_readfirstlane(a.ids[n]);
    const bool live = ad >= 0 && ad < a.L;
    const uint16_t *const b = a.b + (live ? (uint64_t)ad * a.b_adapter : 0);
    uint4 w[2 * RT];
    float out = 0.0f;
    auto load = [&](int64_t m) {
        const uint16_t *const p = b + (uint64_t)(m < a.M ? m : a.M - 1) * a.b_pitch;
        if (live)
#pragma unroll
            for (int q = 0; q < 2 * RT; ++q) w[q] = *reinterpret_cast<const uint4 *>(p + (8 * q < a.r ? 8 * q : 0));
        out = a.base && m < a.M ? a.base[(uint64_t)n * a.base_pitch + m] : 0.0f;
    };
    load(m_first);
    if (live) {
        const int per = (a.K / 32 + kShrinkWaves - 1) / kShrinkWaves * 32;
        const int k_from = wave * per, k_to = k_from + per < a.K ? k_from + per : a.K;
        rt_f32x4 acc[RT] = {};
        shrink_steps<F32X, RT>(a, (uint64_t)n * a.x_pitch, a.a + (uint64_t)ad * a.a_adapter, k_from, k_to, c, g, acc);
        // all sixteen tokens of D are this one
        if (g == 0) {
#pragma unroll
            for (int t = 0; t < RT; ++t) part[wave][16 * t + c] = acc[t][0];
        }
        __syncthreads();
        if (tid < 16 * RT) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < kShrinkWaves; ++q) s += part[q][tid];
            if (a.scales) s *= a.scales[ad];
            us[tid] = s;
        }
        __syncthreads();
    }
    for (int i = 0; i < tiles; ++i) {
        const int64_t m = m_first + 512 * i;
        float y = out;
        if (live) {
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < 2 * RT; ++q) {
                if (8 * q >= a.r) break;
                const uint32_t d[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum = fmaf(__builtin_bit_cast(float, d[j] << 16), us[8 * q + 2 * j], sum);
                    sum = fmaf(__builtin_bit_cast(float, d[j] & 0xFFFF0000u), us[8 * q + 2 * j + 1], sum);
                }
            }
            y += sum;
        }
        if (i + 1 < tiles) load(m + 512);
        if (m < a.M) a.y[(uint64_t)n * a.y_pitch + m] = y;
    }
}

template <bool F32X, int RT>
hipError_t launch_shrink(const LoraArgs &a, const LoraPlan &p, hipStream_t stream)
{
    const void *fn = p.tiled ? reinterpret_cast<const void *>(&lora_shrink_tile_kernel<F32X, RT>)
                             : reinterpret_cast<const void *>(&lora_shrink_kernel<F32X, RT>);
    const int bytes = p.tiled ? ShrinkTile<F32X, RT>::LDS : kShrinkWaves * RT * 4 * 64 * 4;
    const hipError_t e = allow_dynamic_lds(fn, bytes);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)p.blocks1);
    if (p.tiled) hipLaunchKernelGGL((lora_shrink_tile_kernel<F32X, RT>), grid, dim3(256), bytes, stream, a);
    else hipLaunchKernelGGL((lora_shrink_kernel<F32X, RT>), grid, dim3(64 * kShrinkWaves), bytes, stream, a);
    return hipGetLastError();
}
template <int RT>
hipError_t launch_rank(const LoraArgs &a, const LoraPlan &p, bool f32x, hipStream_t stream)
{
    if (p.single) {
        const dim3 grid((unsigned)((a.M + 512 * a.mt - 1) / (512 * a.mt)), (unsigned)a.N);
        if (f32x) hipLaunchKernelGGL((lora_token_kernel<true, RT>), grid, dim3(512), 0, stream, a);
        else hipLaunchKernelGGL((lora_token_kernel<false, RT>), grid, dim3(512), 0, stream, a);
        return hipGetLastError();
    }
    if (p.blocks1) {                   // without K every sum is empty
        const hipError_t e = f32x ? launch_shrink<true, RT>(a, p, stream) : launch_shrink<false, RT>(a, p, stream);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(lora_expand_kernel<RT>, dim3((unsigned)p.blocks2), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(const LoraTask &t, hipStream_t stream)
{
    const LoraPlan p = plan_lora(t.N, t.K, t.M, t.r, lora_wide(t.x, t.x_pitch, t.f32x), device_cus());
    LoraArgs a = {};
    a.a = t.a;
    a.b = t.b;
    a.a_pitch = t.a_pitch;
    a.b_pitch = t.b_pitch;
    a.a_adapter = t.a_adapter;
    a.b_adapter = t.b_adapter;
    a.x = t.x;
    a.x_pitch = t.x_pitch;
    a.ids = t.ids;
    a.scales = t.scales;
    a.base = t.base;
    a.base_pitch = t.base_pitch;
    a.y = t.y;
    a.y_pitch = t.y_pitch;
    a.u = static_cast<float *>(t.ws);
    a.N = t.N;
    a.M = t.M;
    a.L = (int32_t)t.L;
    a.K = (int32_t)t.K;
    a.r = (int32_t)t.r;
    a.rp = 16 * p.rt;
    a.chunk = p.chunk;
    a.chunks = p.chunks;
    a.j1 = p.j1;
    a.j2 = p.j2;
    a.mt = p.mt;
    a.m_blocks = p.m_blocks;
    switch (p.rt) {
    case 1: return launch_rank<1>(a, p, t.f32x, stream);
    case 2: return launch_rank<2>(a, p, t.f32x, stream);
    case 4: return launch_rank<4>(a, p, t.f32x, stream);
    default: return launch_rank<8>(a, p, t.f32x, stream);
    }
}

}  // namespace qmm
