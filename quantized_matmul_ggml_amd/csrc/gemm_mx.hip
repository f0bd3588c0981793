// gemm_mx.hip -- prefill GEMM of MXFP4 weights and MXFP4 activations on the
// scaled matrix instructions.
//
// Y[n][m] = sum_k W'[m][k] X'[n][k] (No Python! Building an AI Inference Engine
// Exclusively in C++, §6: C_ij = sum_k A_ik B_kj), both operands packed rows of
// 32-blocks with a power-of-two scale.  v_mfma_scale_f32_32x32x64_f8f6f4 takes
// the four-bit codes as they lie in memory: a lane feeds one block (16 bytes,
// 32 values of k) of one row together with the block's scale byte, and the
// instruction multiplies the codes, scales by 2^(s_w + s_x - 254) and adds in
// binary32.  The order of the codes within a block does not matter, since both
// operands have the same one, so nothing is unpacked.  Four times the bf16
// rate per instruction: 9.8 PFLOP/s of zeros and 6.8 of random codes, for which
// the clock falls to 1.7 GHz (all CUs, registers only; 6.0 and 1.5 GHz on another
// card).
//
// Work split: a workgroup of WR x WC waves computes BM weight rows x BN tokens,
// each wave TM x TN tiles of 32 x 32, so that a fragment read from LDS feeds TM
// or TN instructions.  K advances 256 (128 code bytes, whole cache lines, and 8
// scale bytes of each row) per step.  Codes and scales go from memory to LDS
// with direct-to-LDS loads into a ring of NST stages, NST - 1 of them in
// flight; one barrier per step.  The fragments of one depth of 64 are read
// while those of the depth before are multiplied, across the barrier too, so
// that the matrix cores do not wait for LDS.  Every 16-byte unit of a row is
// placed by an XOR of its index with bits of the row, so that the rows read
// together fall in different banks.
//
// 11008 x 4096 x 4096: 122 us (3.0 PFLOP/s).  Its 688 tiles are 2.7 rounds of
// the chip; in copies of the kernel that left parts out, the matrix instructions
// and their LDS reads alone took 90 us, the loads alone 74, and the stores of y
// added 20.  Of the cycles that a CU is busy its matrix cores are for 39 %, its
// texture data unit, through which the direct-to-LDS loads go, for 86 % (56 %
// waiting for the caches), LDS reads for 17 %.  5632 x 2048 x 512: 10.5 us, of
// which 4 pass before the first products and after the last.  (K steps of 128, four stages
// deep, were slower: 64-byte pieces of lines need twice the L2's requests.  So
// were four waves of 128 x 128 each, and fetching later steps' lines into the L2
// changed nothing.)
#include "gemm_common.h"
#include "lds_load.h"

namespace qmm {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct GemmMxArgs {
    const uint8_t *w, *x;
    float *y;
    uint64_t w_pitch, x_pitch;    // bytes
    uint64_t y_pitch;             // elements
    int64_t M, N;
    int32_t nb;                   // 32-blocks per row
    int32_t qoff;
    int32_t m_tiles, n_tiles;     // tiles of weight rows and of tokens
    int32_t steps;                // K steps of 256
};

constexpr int kBandTiles = 5;     // token tiles of a band: 32 CUs of an XCD work on about 6 x 5 tiles

template <int TM, int TN, int WR, int WC, int NST>
struct MxTile {
    static constexpr int BM = 32 * TM * WR, BN = 32 * TN * WC, NW = WR * WC, THREADS = 64 * NW;
    static constexpr int W_OFF = 0, X_OFF = BM * 128, WS_OFF = X_OFF + BN * 128, XS_OFF = WS_OFF + BM * 8;
    static constexpr int STAGE = XS_OFF + BN * 8;
    static constexpr int LDS = NST * STAGE;
    static_assert(LDS <= 160 * 1024, "one workgroup's LDS");
    // code loads (8 rows each) and scale loads (32 rows) per wave and step
    static constexpr int WL = BM / 8 / NW, XL = BN / 8 / NW, SL = (BM + BN) / 32 / NW;
    static_assert(BM % (16 * NW) == 0 && BN % (16 * NW) == 0, "an even number of whole code loads per wave");
    static_assert(SL * 32 * NW == BM + BN, "whole scale loads per wave");
    static constexpr int LOADS = WL + XL + SL;
    static_assert(LOADS * (NST - 1) <= 63, "vmcnt range");
};

template <int TM, int TN, int WR, int WC, int NST>
__global__ __launch_bounds__((MxTile<TM, TN, WR, WC, NST>::THREADS)) void gemm_mx_kernel(const GemmMxArgs a)
{
    using L = MxTile<TM, TN, WR, WC, NST>;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(lds);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = wave % WR, wc = wave / WR;
    const int h = lane >> 5;

    // ---- the tile: bands of token tiles, weight tiles within a band, so that
    // the tiles an XCD works on together share both operands in its L2 ----
    const int order = xcd_order_index(), per_band = kBandTiles * a.m_tiles;
    const int band = __builtin_amdgcn_readfirstlane(order / per_band), in_band = order - band * per_band;
    const int left = a.n_tiles - band * kBandTiles, wide_of = left < kBandTiles ? left : kBandTiles;
    const int mt = __builtin_amdgcn_readfirstlane(in_band / wide_of);
    const int nt = __builtin_amdgcn_readfirstlane(band * kBandTiles + in_band - mt * wide_of);
    const int64_t m0 = (int64_t)mt * L::BM, n0 = (int64_t)nt * L::BN;
    const int rows = (int)(a.M - m0 < L::BM ? a.M - m0 : L::BM);
    const int toks = (int)(a.N - n0 < L::BN ? a.N - n0 : L::BN);
    const uint32_t row_bytes = (uint32_t)(a.qoff + 16 * a.nb);
    const uint32_t wp = (uint32_t)a.w_pitch, xp = (uint32_t)a.x_pitch;
    const ll_i32x4 wres = ll_rsrc(a.w + (uint64_t)m0 * a.w_pitch, (uint32_t)(rows - 1) * wp + row_bytes);
    const ll_i32x4 xres = ll_rsrc(a.x + (uint64_t)n0 * a.x_pitch, (uint32_t)(toks - 1) * xp + row_bytes);

    // ---- loads: lane slot e of a row holds its unit e ^ ((row >> 1) & 7).  Rows
    // that do not exist lie past the buffers' ends, and blocks that do not
    // are sent there: both read zeros.  Of a wave's code loads the even ones
    // and the odd ones hold the same units. ----
    const int nb = a.nb;
    const int lrow = lane >> 3, unit0 = (lane & 7) ^ (lrow >> 1), unit1 = unit0 ^ 4;
    const uint32_t woff = (uint32_t)(8 * L::WL * wave + lrow) * wp + (uint32_t)a.qoff;
    const uint32_t xoff = (uint32_t)(8 * L::XL * wave + lrow) * xp + (uint32_t)a.qoff;
    const uint32_t woff0 = woff + 16u * unit0, woff1 = woff + 16u * unit1, xoff0 = xoff + 16u * unit0, xoff1 = xoff + 16u * unit1;
    // scale loads: the weights', then the activations', in turn over the waves
    const uint32_t wsoff = (uint32_t)(lane >> 1) * wp + 4u * (lane & 1), xsoff = (uint32_t)(lane >> 1) * xp + 4u * (lane & 1);
    auto issue = [&](int step) {
        const uint32_t st = lds0 + (uint32_t)(step % NST) * L::STAGE, k = 128u * step;
        const bool in0 = 8 * step + unit0 < nb, in1 = 8 * step + unit1 < nb, ins = 8 * step + 4 * (lane & 1) < nb;
#pragma unroll
        for (int i = 0; i < L::WL; ++i) {
            const uint32_t off = (i & 1 ? woff1 : woff0) + (8u * i * wp + k);
            ll_load<16>(wres, st + L::W_OFF + 1024u * (L::WL * wave + i), (i & 1 ? in1 : in0) ? off : OUT_OF_RANGE);
        }
#pragma unroll
        for (int i = 0; i < L::XL; ++i) {
            const uint32_t off = (i & 1 ? xoff1 : xoff0) + (8u * i * xp + k);
            ll_load<16>(xres, st + L::X_OFF + 1024u * (L::XL * wave + i), (i & 1 ? in1 : in0) ? off : OUT_OF_RANGE);
        }
#pragma unroll
        for (int i = 0; i < L::SL; ++i) {
            const int n = L::SL * wave + i, nx = n - L::BM / 32;
            const bool of_w = nx < 0;
            const uint32_t off = (of_w ? wsoff : xsoff) + ((of_w ? 32u * n * wp : 32u * nx * xp) + 8u * step);
            ll_load<4>(of_w ? wres : xres, st + (of_w ? L::WS_OFF + 256u * n : L::XS_OFF + 256u * nx), ins ? off : OUT_OF_RANGE);
        }
    };

    // ---- fragments: depth s of a stage is blocks 2 s + h ----
    const int wrow = 32 * TM * wr + (lane & 31), xrow = 32 * TN * wc + (lane & 31);
    auto slot = [&](int s) { return 16u * (uint32_t)((2 * s + h) ^ ((lane >> 1) & 7)); };
    struct Frags {
        u32x4 w[TM], x[TN];
    };
    struct RawScales {
        u32x2 w[TM], x[TN];
    };
    struct Scales {
        int w[TM], x[TN];
    };
    auto wide = [](u32x4 v) { return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0}; };
    auto read = [&](Frags &f, const uint8_t *st, int s) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
            f.w[i] = *reinterpret_cast<const u32x4 *>(st + L::W_OFF + (wrow + 32 * i) * 128 + slot(s));
#pragma unroll
        for (int j = 0; j < TN; ++j)
            f.x[j] = *reinterpret_cast<const u32x4 *>(st + L::X_OFF + (xrow + 32 * j) * 128 + slot(s));
    };
    auto read_scales = [&](RawScales &c, const uint8_t *st) {
#pragma unroll
        for (int i = 0; i < TM; ++i) c.w[i] = *reinterpret_cast<const u32x2 *>(st + L::WS_OFF + (wrow + 32 * i) * 8);
#pragma unroll
        for (int j = 0; j < TN; ++j) c.x[j] = *reinterpret_cast<const u32x2 *>(st + L::XS_OFF + (xrow + 32 * j) * 8);
    };
    // scale bytes of blocks h, 2 + h, 4 + h, 6 + h of a row's step; those of
    // blocks past the row may be any bytes, NaN among them, and become zeros
    // (no branch: across one the compiler sinks the matrix instructions before it)
    auto order_scales = [&](Scales &c, const RawScales &raw, int t) {
        const int in = (nb - h - 8 * t + 1) >> 1;                     // blocks in the row
        const uint32_t cut = in >= 4 ? 0u : in <= 0 ? ~0u : ~0u << (8 * in);
        const uint32_t sel = ((h ? 0x07050301u : 0x06040200u) & ~cut) | (0x0C0C0C0Cu & cut);    // 12: a zero byte
#pragma unroll
        for (int i = 0; i < TM; ++i) c.w[i] = (int)__builtin_amdgcn_perm(raw.w[i][1], raw.w[i][0], sel);
#pragma unroll
        for (int j = 0; j < TN; ++j) c.x[j] = (int)__builtin_amdgcn_perm(raw.x[j][1], raw.x[j][0], sel);
    };

    f32x16 acc[TN][TM];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;
    auto multiply = [&](const Frags &f, const Scales &c, auto S) {
        constexpr int s = decltype(S)::value;
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int i = 0; i < TM; ++i)
                acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(f.x[j]), wide(f.w[i]), acc[j][i], 4, 4, s, c.x[j],
                                                                           s, c.w[i]);
    };
    // this wave's loads of the next step have landed and its reads of this one
    // too, then every wave's
    auto meet = [&] {
        ll_wait<L::LOADS *(NST - 2)>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };

#pragma unroll
    for (int s = 0; s < NST - 1; ++s) issue(s);
    meet();
    issue(NST - 1);
    Frags f[2];
    RawScales raw;
    Scales c;
    read(f[0], lds, 0);
    read_scales(raw, lds);
    for (int t = 0; t < a.steps; ++t) {
        const uint8_t *const st = lds + (t % NST) * L::STAGE, *const next = lds + ((t + 1) % NST) * L::STAGE;
        order_scales(c, raw, t);
        static_for<4>([&](auto S) {
            constexpr int s = decltype(S)::value;
            if constexpr (s < 3) {
                read(f[(s + 1) % 2], st, s + 1);
            } else {
                // every wave has read step t's stage: the step NST later takes it
                meet();
                issue(t + NST);
                read(f[(s + 1) % 2], next, 0);
                read_scales(raw, next);
            }
            __builtin_amdgcn_sched_barrier(0);
            multiply(f[s % 2], c, S);
            __builtin_amdgcn_sched_barrier(0);
        });
    }
    ll_wait<0>();                  // no load may still write the LDS of a finished workgroup

    // ---- D: column lane % 32 is a weight row, register r token 8 (r / 4) +
    // 4 h + r % 4.  Streaming stores: nothing here reads y again. ----
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t m = m0 + wrow + 32 * i;
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int64_t n = n0 + 32 * (TN * wc + j) + 8 * (r / 4) + 4 * h + (r % 4);
                if (n < a.N) __builtin_nontemporal_store(acc[j][i][r], a.y + (uint64_t)n * a.y_pitch + m);
            }
    }
}

template <int TM, int TN, int WR, int WC, int NST>
hipError_t launch_tile(GemmMxArgs a, hipStream_t stream)
{
    using L = MxTile<TM, TN, WR, WC, NST>;
    const int64_t mt = (a.M + L::BM - 1) / L::BM, nt = (a.N + L::BN - 1) / L::BN;
    // (64 x 64 tiles are taken for a few hundred of them only)
    static_assert((L::BM >= 128 && L::BN >= 128 && L::THREADS == 512) || L::BM == 64, "no more threads than gemm_tiles counts");
    a.m_tiles = (int32_t)mt;
    a.n_tiles = (int32_t)nt;
    const void *fn = reinterpret_cast<const void *>(&gemm_mx_kernel<TM, TN, WR, WC, NST>);
    const hipError_t e = allow_dynamic_lds(fn, L::LDS);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((gemm_mx_kernel<TM, TN, WR, WC, NST>), dim3((unsigned)(mt * nt)), dim3(L::THREADS), L::LDS, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_mx(const WeightView &w, const ActView &x, const OutView &y, hipStream_t stream)
{
    GemmMxArgs a = {};
    a.w = w.base;
    a.x = static_cast<const uint8_t *>(x.data);
    a.y = y.data;
    a.w_pitch = w.pitch;
    a.x_pitch = x.pitch_elems;
    a.y_pitch = y.pitch_elems;
    a.M = w.M;
    a.N = x.N;
    a.nb = (int32_t)(w.K / 32);
    a.steps = (a.nb + 7) / 8;
    a.qoff = (int32_t)quant_offset(w.K, w.scale_shift);
    
    // 256 x 256 tiles read half the bytes of 128 x 128 ones per product, but one
    // takes a little over twice as long: they win where the small ones need more
    // than two rounds on the chip's CUs for each of theirs (2048-deep, us, large
    // and small: 2048 x 2048 23.4, 12.6; 5632 x 1024 23.6, 21.2; 5632 x 2048
    // 26.9, 33.0; 5632 x 4096 52.8, 60.2).  A step of a 64 x 64 tile takes half a
    // step of a 128 x 128 one, and three fit a CU: they win up to two a CU (us, 64
    // and 128: 2048 x 5632 x 512 13.9, 23.6; 2048 x 2048 x 100 5.7, 8.7;
    // 5632 x 2048 x 256 9.1, 10.3; 5632 x 2048 x 512 14.0, 11.4).
    const int64_t cus = device_cus();
    auto tiles = [&](int64_t size) { return ((a.M + size - 1) / size) * ((a.N + size - 1) / size); };
    auto rounds = [&](int64_t size) { return (tiles(size) + cus - 1) / cus; };
    if (tiles(64) <= 2 * cus) return launch_tile<1, 1, 2, 2, 3>(a, stream);
    const bool offsets = 256ull * a.w_pitch < (1ull << 31) && 256ull * a.x_pitch < (1ull << 31);
    if (offsets && rounds(128) > 2 * rounds(256)) return launch_tile<2, 4, 4, 2, 2>(a, stream);
    return launch_tile<2, 1, 2, 4, 3>(a, stream);
}

}  // namespace qmm
