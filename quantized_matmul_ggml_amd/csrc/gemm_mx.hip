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
// rate per instruction, so what bounds large products is feeding it.
//
// Work split: a workgroup of WR x WC waves computes BM weight rows x BN tokens,
// each wave TM x TN tiles of 32 x 32, so that a fragment read from LDS feeds TM
// or TN instructions.  K advances 256 (128 code bytes and 8 scale bytes of each
// row) per step.  Codes and scales go from memory to LDS with direct-to-LDS
// loads, NST - 1 steps ahead, into a ring of NST stages; one barrier per step.
// Every 16-byte unit of a row is placed by an XOR of its index with bits of the
// row, so that the rows read together fall in different banks.
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
    int32_t n_tiles;              // token tiles
    int32_t steps;                // K steps of 256
};

template <int TM, int TN, int WR, int WC, int NST>
struct MxTile {
    static constexpr int BM = 32 * TM * WR, BN = 32 * TN * WC, NW = WR * WC, THREADS = 64 * NW;
    static constexpr int W_CODES = BM * 128, X_CODES = BN * 128;
    static constexpr int W_OFF = 0, X_OFF = W_CODES, WS_OFF = X_OFF + X_CODES, XS_OFF = WS_OFF + BM * 8;
    static constexpr int STAGE = XS_OFF + BN * 8;
    static constexpr int LDS = NST * STAGE;
    static_assert(LDS <= 160 * 1024, "one workgroup's LDS");
    static constexpr int WL = BM / 8 / NW, XL = BN / 8 / NW;       // code loads per wave and step
    static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole code loads per wave");
    // scale loads: one covers 32 rows (two dwords each); the waves share
    // them, waves without one repeat the last
    static constexpr int WSL = (BM / 32 + NW - 1) / NW, XSL = (BN / 32 + NW - 1) / NW;
    static constexpr int LOADS = WL + XL + WSL + XSL;
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

    const int tile = xcd_order_index();
    const int mt = __builtin_amdgcn_readfirstlane(tile / a.n_tiles);
    const int nt = __builtin_amdgcn_readfirstlane(tile - mt * a.n_tiles);
    const int64_t m0 = (int64_t)mt * L::BM, n0 = (int64_t)nt * L::BN;
    const int rows = (int)(a.M - m0 < L::BM ? a.M - m0 : L::BM);
    const int toks = (int)(a.N - n0 < L::BN ? a.N - n0 : L::BN);
    const uint32_t row_bytes = (uint32_t)(a.qoff + 16 * a.nb);
    const uint32_t wp = (uint32_t)a.w_pitch, xp = (uint32_t)a.x_pitch;
    const ll_i32x4 wres = ll_rsrc(a.w + (uint64_t)m0 * a.w_pitch, (uint32_t)(rows - 1) * wp + row_bytes);
    const ll_i32x4 xres = ll_rsrc(a.x + (uint64_t)n0 * a.x_pitch, (uint32_t)(toks - 1) * xp + row_bytes);

    // ---- loads: lane slot e of a row holds its unit e ^ ((row >> 1) & 7);
    // rows and blocks that do not exist read zeros ----
    const int nb = a.nb, qoff = a.qoff;
    auto codes = [&](const ll_i32x4 &res, uint32_t pitch, int nrows, uint32_t dst, int i, int step) {
        const int row = 8 * i + (lane >> 3), unit = (lane & 7) ^ ((row >> 1) & 7);
        const int blk = 8 * step + unit;
        ll_load<16>(res, dst + 1024u * i,
                    row < nrows && blk < nb ? (uint32_t)row * pitch + (uint32_t)(qoff + 16 * blk) : OUT_OF_RANGE);
    };
    auto scales = [&](const ll_i32x4 &res, uint32_t pitch, int nrows, uint32_t dst, int i, int step) {
        const int row = 32 * i + (lane >> 1), blk = 8 * step + 4 * (lane & 1);
        ll_load<4>(res, dst + 256u * i, row < nrows && blk < nb ? (uint32_t)row * pitch + (uint32_t)blk : OUT_OF_RANGE);
    };
    auto issue = [&](int step) {
        const uint32_t st = lds0 + (uint32_t)(step % NST) * L::STAGE;
#pragma unroll
        for (int i = 0; i < L::WL; ++i) codes(wres, wp, rows, st + L::W_OFF, L::WL * wave + i, step);
#pragma unroll
        for (int i = 0; i < L::XL; ++i) codes(xres, xp, toks, st + L::X_OFF, L::XL * wave + i, step);
#pragma unroll
        for (int i = 0; i < L::WSL; ++i) {
            const int k = L::WSL * wave + i;
            scales(wres, wp, rows, st + L::WS_OFF, k < L::BM / 32 ? k : L::BM / 32 - 1, step);
        }
#pragma unroll
        for (int i = 0; i < L::XSL; ++i) {
            const int k = L::XSL * wave + i;
            scales(xres, xp, toks, st + L::XS_OFF, k < L::BN / 32 ? k : L::BN / 32 - 1, step);
        }
    };

    // ---- fragment addresses within a stage ----
    const int wrow = 32 * TM * wr + (lane & 31), xrow = 32 * TN * wc + (lane & 31);
    auto frag = [&](const uint8_t *base, int row, int s) {
        const int unit = (2 * s + h) ^ ((row >> 1) & 7);
        return *reinterpret_cast<const u32x4 *>(base + row * 128 + 16 * unit);
    };
    // scale bytes of blocks h, 2 + h, 4 + h, 6 + h of a row's step
    const uint32_t sel = h ? 0x07050301u : 0x06040200u;
    auto scale4 = [&](const uint8_t *base, int row, uint32_t mask) {
        const u32x2 v = *reinterpret_cast<const u32x2 *>(base + row * 8);
        return (int)(__builtin_amdgcn_perm(v[1], v[0], sel) & mask);
    };
    auto wide = [](u32x4 v) { return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0}; };

    f32x16 acc[TN][TM];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;

#pragma unroll
    for (int s = 0; s < NST - 1; ++s) issue(s);
    for (int t = 0; t < a.steps; ++t) {
        // this wave's loads of step t have landed, then every wave's; and
        // every wave is done with step t - 1, whose stage the next loads take
        ll_wait<L::LOADS *(NST - 2)>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        issue(t + NST - 1);
        const uint8_t *st = lds + (t % NST) * L::STAGE;
        // scales of blocks past the row may be any bytes, NaN among them
        uint32_t mask = 0xFFFFFFFFu;
        if (8 * t + 8 > nb) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (8 * t + 2 * s + h >= nb) mask &= ~(0xFFu << (8 * s));
        }
        int ws[TM], xs[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) ws[i] = scale4(st + L::WS_OFF, wrow + 32 * i, mask);
#pragma unroll
        for (int j = 0; j < TN; ++j) xs[j] = scale4(st + L::XS_OFF, xrow + 32 * j, mask);
        static_for<4>([&](auto S) {
            constexpr int s = decltype(S)::value;
            i32x8 wf[TM], xf[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) wf[i] = wide(frag(st + L::W_OFF, wrow + 32 * i, s));
#pragma unroll
            for (int j = 0; j < TN; ++j) xf[j] = wide(frag(st + L::X_OFF, xrow + 32 * j, s));
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xf[j], wf[i], acc[j][i], 4, 4, s, xs[j],
                                                                               s, ws[i]);
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
    if (mt * nt >= (1ll << 31)) return hipErrorInvalidValue;
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
    a.qoff = (int32_t)quant_offset(w.K, w.scale_shift);
    a.steps = (int32_t)((w.K + 255) / 256);
    const int64_t large = ((a.M + 255) / 256) * ((a.N + 255) / 256);
    const bool offsets = 256ull * a.w_pitch < (1ull << 31) && 256ull * a.x_pitch < (1ull << 31);
    if (offsets && large >= device_cus()) return launch_tile<2, 4, 4, 2, 2>(a, stream);
    return launch_tile<2, 2, 2, 2, 4>(a, stream);
}

}  // namespace qmm
