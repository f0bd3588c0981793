// gemm_rows.hip -- grouped products (gemm_grouped.hip) for experts with few rows:
// the time is the time to stream the chosen experts' weights (A Complete Guide to
// llama.cpp and Customization with C++, §2.1), so the weights go from memory to
// registers in 64-byte units of sixteen rows (row_tiles.h), several in flight per
// wave, and up to sixteen grouped rows' activations lie in LDS in the order that
// the matrix instructions read them.
//
// One v_mfma_f32_16x16x32_bf16 takes 32 values of k of 16 weight rows (columns)
// and of 16 grouped rows.  The activations are bf16 as they are, so every product
// is exact; a block's sum starts from zero and its scale multiplies it in binary32
// (MXFP4: the scale is in the values, and sums run through whole rows).
//
// A workgroup of eight waves takes one row tile of an expert and 8 C tiles of
// sixteen weight rows (SwiGLU: eight gate rows and the same eight up rows), C to a
// wave, one after the other without a gap in the loads.  Rows in two bf16 parts (P = 2,
// GroupedOut) take two instructions and twice the image per 32 of k.
//
// 32 experts, gate and up 1408 x 2048 MXFP4, 33 tokens of four: 21.6 us, 4.5 TB/s of
// weights; 64 experts with eight rows each, 142 MB of MXFP4: 30.3 us, 4.7 TB/s (34.3
// where nothing is left in a cache).  Q4_0 takes about four times MXFP4's vector
// work per byte, which shows where few experts leave one workgroup per CU: 16
// experts of 2048 x 2048 with eight rows 14.7 us, MXFP4 10.5.
#include "grouped_tile.h"
#include "row_tiles.h"

namespace qmm {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 16;                       // grouped rows of a tile
constexpr int kBlockBytes = kRows * 64;         // LDS bytes of a 32-block's activations
constexpr int kImage = 64 * 1024;               // LDS of the activations: 2048 / P of K at a time
constexpr int kScales = kImage;                 // the waves' scales
constexpr int kLds = kScales + kWaves * kScaleLds;
static_assert(2 * kLds <= 160 * 1024, "two workgroups per CU");

// Multiplies unit q of the rows (as multiply_unit of row_tiles.h) with the fragments
// at img, adds to acc: columns are the 16 weight rows, rows the grouped ones.
template <int WT, int SS, int P>
__device__ inline void multiply_rows(const Unit<WT, SS> &z, const uint8_t *img, int left, int g, rt_f32x4 &acc)
{
    using F = RowFmt<WT, SS>;
    rt_bf16x8 fr[F::MF][P];
#pragma unroll
    for (int t = 0; t < F::MF; ++t)
#pragma unroll
        for (int p = 0; p < P; ++p) fr[t][p] = *reinterpret_cast<const rt_bf16x8 *>(img + (t * P + p) * kBlockBytes);
    uint32_t d[4] = {z.q.x, z.q.y, z.q.z, z.q.w};
    if constexpr (WT == W_MXFP4) {
        uint32_t e = (z.s[0] >> (8 * g)) & 0xFFu;
        e = g < left ? e : 0u;                          // blocks past the row
        const float f = __builtin_bit_cast(float, e << 23);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint4 bw = make_uint4(
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d[t], f, 0)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d[t], f, 1)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d[t], f, 2)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d[t], f, 3)));
#pragma unroll
            for (int p = 0; p < P; ++p)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fr[t][p], __builtin_bit_cast(rt_bf16x8, bw), acc, 0, 0, 0);
        }
    } else {
        rt_swap32(d[0], d[2]);
        rt_swap32(d[1], d[3]);
        if constexpr (WT == W_Q4_0) {
            rt_swap16(d[0], d[1]);
            rt_swap16(d[2], d[3]);
        }
        constexpr int PER = 1 << SS;                    // blocks under one scale
#pragma unroll
        for (int t0 = 0; t0 < F::MF; t0 += PER) {
            rt_f32x4 sum = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int t = t0 + i;
                uint4 bw;
                if constexpr (WT == W_Q4_0) {
                    const uint32_t x = d[t] ^ 0x88888888u;
                    const uint32_t lo = (x << 4) & 0xF0F0F0F0u, hi = x & 0xF0F0F0F0u;
                    bw = make_uint4(rt_pack(rt_sbyte<0>(lo), rt_sbyte<0>(hi)), rt_pack(rt_sbyte<1>(lo), rt_sbyte<1>(hi)),
                                    rt_pack(rt_sbyte<2>(lo), rt_sbyte<2>(hi)), rt_pack(rt_sbyte<3>(lo), rt_sbyte<3>(hi)));
                } else {
                    const uint32_t p = d[2 * t], q = d[2 * t + 1];
                    bw = make_uint4(rt_pack(rt_sbyte<0>(p), rt_sbyte<1>(p)), rt_pack(rt_sbyte<2>(p), rt_sbyte<3>(p)),
                                    rt_pack(rt_sbyte<0>(q), rt_sbyte<1>(q)), rt_pack(rt_sbyte<2>(q), rt_sbyte<3>(q)));
                }
#pragma unroll
                for (int p = 0; p < P; ++p)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fr[t][p], __builtin_bit_cast(rt_bf16x8, bw), sum, 0, 0, 0);
            }
            const int sh = t0 >> SS;                    // the scale (a half) within the unit
            const uint32_t sb = (sh & 1) ? z.s[sh / 2] >> 16 : z.s[sh / 2] & 0xFFFFu;
            float f = (float)__builtin_bit_cast(_Float16, (uint16_t)sb);
            if constexpr (WT == W_Q4_0) f *= 0.0625f;
            f = t0 < left ? f : 0.0f;                   // blocks past the row
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[r] = fmaf(f, sum[r], acc[r]);
        }
    }
}

// D: units in flight.  A wave walks over C tiles' units in groups of D, a tile's
// units filled up to whole groups (of the row's last bytes and zero scales).  With
// several passes over K (rows longer than the image) C is 1.  The group after the
// one at hand is loaded place by place as the units are multiplied; MXFP4, whose
// unpacking is light, at once behind them: then D * 64 bytes of each row stand
// together in the stream, which memory serves better, and other waves cover the
// wait (64 experts, 142 MB with 8 rows each: 32.2 us place by place, 30.3 at once;
// Q4_0, 16 experts of 37 MB: 14.7 and 15.5).
// P: the parts of x's rows, or with SW those of h's values.
template <int WT, int SS, bool SW, int D, int P>
__global__ __launch_bounds__(kThreads, 4) void gemm_rows_kernel(const GrpArgs a)
{
    using F = RowFmt<WT, SS>;
    constexpr int MF = F::MF, XP = SW ? 1 : P;
    constexpr bool AT_ONCE = WT == W_MXFP4;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, j = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint8_t *const scales = lds + kScales + wave * kScaleLds;
    GroupTile tile;
    if (!find_tile<kRows>(a, tile)) return;
    const int blocks = a.K / 32, code_bytes = F::BB * blocks, row_bytes = a.qoff + code_bytes;
    const int C = a.tiles_per_wave;
    constexpr int TILE = SW ? 8 : 16;                   // weight rows (of each matrix) of a tile
    const bool upper = SW && j >= 8;
    const int64_t tile0 = ((int64_t)tile.mt * kWaves + wave) * C;
    // the lane's matrix and weight row of tile c
    const uint8_t *const matrix = upper ? a.w2 + (uint64_t)tile.e * a.expert2 : a.w + (uint64_t)tile.e * a.expert;
    const uint64_t pitch = upper ? a.pitch2 : a.pitch;
    auto row_of = [&](int c) {
        const int64_t r = (tile0 + c) * TILE + (SW ? j & 7 : j);
        return matrix + (uint64_t)(r < a.M ? r : a.M - 1) * pitch;
    };
    // this thread's share of the activations: of one grouped row, every 32nd piece
    // of eight values
    constexpr int PIECES = kImage / (kThreads * 16);
    const int xt = tid / 32, xp = tid % 32;
    const int token = xt < tile.rows ? token_of(a, tile.n0 + xt) : -1;
    const uint16_t *const x = a.x + (uint64_t)(token > 0 ? token : 0) * a.x_pitch;
    const int units = (blocks + MF - 1) / MF, pass_units = kImage / (MF * XP * kBlockBytes);
    static_assert(kImage / (MF * XP * kBlockBytes) % D == 0, "whole groups fit the image");
    Unit<WT, SS> z[D];
    ScaleWindow<WT, SS, false, D> window;
    rt_f32x4 acc = {0, 0, 0, 0};
    auto finish = [&](int c) {
        const int64_t m = (tile0 + c) * TILE + (SW ? j & 7 : j);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float v = acc[r];
            if constexpr (SW) {
                // the up row's sum, from the lane eight further on
                const float u = __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x128, 0xF, 0xF, false));
                v = rt_swish(v) * u;
            }
            const int t = 4 * g + r;
            if (t < tile.rows && m < a.M && !upper) {
                const uint64_t p = (uint64_t)(tile.n0 + t) * a.y_pitch + m;
                if constexpr (SW && P == 2) store_split(static_cast<uint16_t *>(a.y) + (uint64_t)(tile.n0 + t) * a.y_pitch, m, v);
                else if (a.bf16_out) static_cast<uint16_t *>(a.y)[p] = (uint16_t)rt_pack(v, 0.0f);
                else static_cast<float *>(a.y)[p] = v;
            }
            acc[r] = 0.0f;
        }
    };
    for (int u0 = 0; u0 < units; u0 += pass_units) {
        const int len = units - u0 < pass_units ? units - u0 : pass_units;
        const int groups = (len + D - 1) / D, total = groups * C;
        // ---- the activations, then the first units of weights: loads complete in
        // order, and the activations are needed first ----
        uint2 v0[PIECES], v1[PIECES];
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int b = u0 * MF + 8 * (i / XP) + (xp >> 2);
            // without a branch, at a place that is there
            const uint16_t *const p = x + 32 * (XP * (b < blocks ? b : 0) + i % XP);
            v0[i] = *reinterpret_cast<const uint2 *>(p + run0<WT>(xp & 3));
            v1[i] = *reinterpret_cast<const uint2 *>(p + run1<WT>(xp & 3));
        }
        __builtin_amdgcn_sched_barrier(0);
        const uint8_t *row = row_of(0);
        window.load(row, row_bytes, u0, g, false);
        __builtin_amdgcn_sched_barrier(0);
        static_steps<D>([&](auto d) {
            load_codes<WT, SS>(z[d.value], row, a.qoff, code_bytes, u0 + (int)d.value, g);
            __builtin_amdgcn_sched_barrier(0);
        });
        if (u0 > 0) __syncthreads();                    // the last image is no longer read
        if (xt < tile.rows) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                uint4 v;
                if (WT == W_Q8_0) {
                    v = make_uint4(v0[i].x, v0[i].y, v1[i].x, v1[i].y);
                } else {                                // the two runs' values in turn
                    v.x = __builtin_amdgcn_perm(v1[i].x, v0[i].x, 0x05040100u);
                    v.y = __builtin_amdgcn_perm(v1[i].x, v0[i].x, 0x07060302u);
                    v.z = __builtin_amdgcn_perm(v1[i].y, v0[i].y, 0x05040100u);
                    v.w = __builtin_amdgcn_perm(v1[i].y, v0[i].y, 0x07060302u);
                }
                const int lb = 8 * (i / XP) + (xp >> 2), q = xp & 3; // block within the image, quarter
                if (token < 0 || u0 * MF + lb >= blocks) v = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(lds + (image_step<WT>(lb, q) * XP + i % XP) * kBlockBytes + image_group<WT>(lb, q) * (kRows * 16) + xt * 16) = v;
            }
        }
        __syncthreads();
        // ---- the units ----
        const uint8_t *const img = lds + 16 * lane;     // group g, row j
        int q = 0, c = 0;                               // this group's first unit and tile
        for (int i = 0; i < total; ++i) {
            window.put(scales, j, g);
            // the next group: of this tile, of the next, or (unused) this one again
            int qn = q + D, cn = c;
            if (qn >= groups * D) {
                qn = 0;
                ++cn;
                if (cn == C) {
                    cn = c;
                    qn = q;
                }
                row = row_of(cn);
            }
            window.load(row, row_bytes, u0 + qn, g, false);
            __builtin_amdgcn_sched_barrier(0);
            static_steps<D>([&](auto d) {
                const int u = q + (int)d.value;
                window.get(z[d.value], scales, d.value, j);
                // units past the pass: zero activations and scales (whole groups fit the
                // image, which is zeros past the row)
                multiply_rows<WT, SS, XP>(z[d.value], img + u * MF * XP * kBlockBytes, u < len ? blocks - (u0 + u) * MF : 0, g, acc);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (!AT_ONCE) load_codes<WT, SS>(z[d.value], row, a.qoff, code_bytes, u0 + qn + (int)d.value, g);
                __builtin_amdgcn_sched_barrier(0);
            });
            if constexpr (AT_ONCE) {
                static_steps<D>([&](auto d) {
                    load_codes<WT, SS>(z[d.value], row, a.qoff, code_bytes, u0 + qn + (int)d.value, g);
                    __builtin_amdgcn_sched_barrier(0);
                });
            }
            if (cn != c || i + 1 == total) {
                if (u0 + pass_units >= units) finish(c);
            }
            q = qn;
            c = cn;
        }
    }
    if (units == 0)
        for (int c = 0; c < C; ++c) finish(c);
}

template <int WT, int SS, bool SW, int P>
hipError_t launch_rows(GrpArgs &a, int depth, hipStream_t stream)
{
    const void *fn = depth == 8 ? reinterpret_cast<const void *>(&gemm_rows_kernel<WT, SS, SW, 8, P>)
                                : reinterpret_cast<const void *>(&gemm_rows_kernel<WT, SS, SW, 4, P>);
    const hipError_t e = allow_dynamic_lds(fn, kLds);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(grouped_row_tiles(a.R, a.E, kRows) * a.m_tiles)), block(kThreads);
    if (depth == 8) hipLaunchKernelGGL((gemm_rows_kernel<WT, SS, SW, 8, P>), grid, block, kLds, stream, a);
    else hipLaunchKernelGGL((gemm_rows_kernel<WT, SS, SW, 4, P>), grid, block, kLds, stream, a);
    return hipGetLastError();
}
template <int WT, int SS>
hipError_t launch_rows(GrpArgs &a, int depth, bool sw, int parts, hipStream_t stream)
{
    if (sw) return a.split_out ? launch_rows<WT, SS, true, 2>(a, depth, stream) : launch_rows<WT, SS, true, 1>(a, depth, stream);
    return parts == 2 ? launch_rows<WT, SS, false, 2>(a, depth, stream) : launch_rows<WT, SS, false, 1>(a, depth, stream);
}

}  // namespace

hipError_t launch_gemm_rows(GrpArgs &a, int type, int scale_shift, bool swiglu, int parts, hipStream_t stream)
{
    const RowsPlan p = plan_grouped_rows(a.M, a.K, a.R, a.E, type, swiglu, device_cus(), parts);
    a.tiles_per_wave = p.tiles_per_wave;
    a.m_tiles = (int32_t)p.m_tiles;
    if (type == W_MXFP4) return launch_rows<W_MXFP4, 0>(a, p.depth, swiglu, parts, stream);
    if (type == W_Q4_0) return scale_shift ? launch_rows<W_Q4_0, 1>(a, p.depth, swiglu, parts, stream) : launch_rows<W_Q4_0, 0>(a, p.depth, swiglu, parts, stream);
    if (type == W_Q8_0) return scale_shift ? launch_rows<W_Q8_0, 1>(a, p.depth, swiglu, parts, stream) : launch_rows<W_Q8_0, 0>(a, p.depth, swiglu, parts, stream);
    return hipErrorInvalidValue;
}

}  // namespace qmm
