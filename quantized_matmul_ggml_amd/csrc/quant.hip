// quant.hip -- load-time Q8_0 / Q4_0 quantization and dequantization on the GPU.
//
// Block rule (A Complete Guide to llama.cpp and Customization with C++, §2.2:
// w_i ~= Delta * q_i with Delta from the block's largest |w|; Development Guide
// for Small AI Models (TinyLLaMA, etc.) Using C++, §6.1: 32 values per block,
// one FP16 scale):
//   amax = max |w_i|;  Delta = fp16_rne(amax / 127) (Q8_0) or fp16_rne(amax / 8) (Q4_0)
//   q_i  = roundf(w_i / Delta)  -- one correctly rounded binary32 division by the
//          stored scale, then round half away from zero;
//   Q8_0 clamps q to [-127, 127]; Q4_0 stores q + 8 clamped to [0, 15].
// The library is built without fast-math, so '/' is the IEEE division and
// the fp16 / bf16 conversions round to nearest even: the codes are bit-exact.
//
// A second Q4 rule is the pages' own (A Complete Guide to llama.cpp ...,
// §2.2: Delta = max|w| / 7, q_i in [-8, 7]): the same steps with 7 as the
// divisor, stored the same way (clamp(q + 8, 0, 15) = clamp(q, -8, 7) + 8).
//
// 64-weight blocks (same page: the block length is usually 32 or 64) take
// the same steps over 64 values; their codes are stored as two runs of 32
// laid out like a 32-block's.
//
// These kernels run once per weight at load time, so they favour clarity:
// one thread per block.
#include "qmm_internal.h"

namespace qmm {
namespace {

__device__ inline uint16_t f32_to_f16_bits(float f)
{
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
}

__device__ inline float f16_bits_to_f32(uint16_t h)
{
    return static_cast<float>(__builtin_bit_cast(_Float16, h));
}

template <int TYPE, int DIV, int BS>
__global__ __launch_bounds__(256) void quantize_kernel(const float *__restrict__ src,
                                                       uint64_t src_pitch, int64_t K, int64_t M,
                                                       uint8_t *__restrict__ dst, uint64_t dst_pitch)
{
    constexpr int RUNS = BS / 32;          // 32-code runs per block, laid out as in the 32-blocks
    const int64_t nblk = K / BS;
    const int64_t total = M * nblk;
    const int64_t qoff = quant_offset(K, BS == 64 ? 1 : 0);
    const int64_t qbytes = (TYPE == W_Q8_0) ? K : K / 2;
    const int64_t row_bytes = qoff + ((qbytes + 15) / 16) * 16;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / nblk;
        const int64_t b = i - r * nblk;
        const float *w = src + r * src_pitch + b * BS;
        float v[BS];
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < BS; ++j) {
            v[j] = w[j];
            amax = fmaxf(amax, fabsf(v[j]));
        }
        const float s = amax / (float)DIV;
        const uint16_t sb = f32_to_f16_bits(s);
        const float d = f16_bits_to_f32(sb);
        uint8_t *row = dst + r * dst_pitch;
        *reinterpret_cast<uint16_t *>(row + 2 * b) = sb;
#pragma unroll
        for (int h = 0; h < RUNS; ++h) {
            const float *vr = v + 32 * h;
            const int64_t run = b * RUNS + h;          // 32-code run within the row
            if (TYPE == W_Q8_0) {
                uint32_t words[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) words[j] = 0;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float q = 0.0f;
                    if (d != 0.0f) q = fminf(fmaxf(roundf(vr[j] / d), -127.0f), 127.0f);
                    words[j / 4] |= (uint32_t)(uint8_t)(int8_t)q << (8 * (j % 4));
                }
                uint4 *out = reinterpret_cast<uint4 *>(row + qoff + 32 * run);
                out[0] = make_uint4(words[0], words[1], words[2], words[3]);
                out[1] = make_uint4(words[4], words[5], words[6], words[7]);
            } else {
                uint32_t nib[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float q = 8.0f;
                    if (d != 0.0f) q = fminf(fmaxf(roundf(vr[j] / d) + 8.0f, 0.0f), 15.0f);
                    nib[j] = (uint32_t)q;
                }
                uint32_t words[4] = {0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    words[j / 4] |= (nib[j] | (nib[j + 16] << 4)) << (8 * (j % 4));
                *reinterpret_cast<uint4 *>(row + qoff + 16 * run) =
                    make_uint4(words[0], words[1], words[2], words[3]);
            }
        }
        if (b == 0) {
            for (int64_t p = 2 * nblk; p < qoff; ++p) row[p] = 0;
            for (int64_t p = qoff + qbytes; p < row_bytes; ++p) row[p] = 0;
        }
    }
}

template <int TYPE, int BS>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint8_t *__restrict__ src,
                                                         uint64_t src_pitch, int64_t K, int64_t M,
                                                         float *__restrict__ dst, uint64_t dst_pitch)
{
    constexpr int RUNS = BS / 32;
    const int64_t nblk = K / BS;
    const int64_t total = M * nblk;
    const int64_t qoff = quant_offset(K, BS == 64 ? 1 : 0);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / nblk;
        const int64_t b = i - r * nblk;
        const uint8_t *row = src + r * src_pitch;
        const float d = f16_bits_to_f32(*reinterpret_cast<const uint16_t *>(row + 2 * b));
#pragma unroll
        for (int h = 0; h < RUNS; ++h) {
            const int64_t run = b * RUNS + h;
            float *out = dst + r * dst_pitch + run * 32;
            if (TYPE == W_Q8_0) {
                const int8_t *q = reinterpret_cast<const int8_t *>(row + qoff + 32 * run);
#pragma unroll
                for (int j = 0; j < 32; ++j) out[j] = d * (float)q[j];
            } else {
                const uint8_t *q = row + qoff + 16 * run;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    out[j] = d * (float)((int)(q[j] & 0x0F) - 8);
                    out[j + 16] = d * (float)((int)(q[j] >> 4) - 8);
                }
            }
        }
    }
}

__global__ __launch_bounds__(256) void f16_to_f32_kernel(const uint8_t *__restrict__ src,
                                                         uint64_t src_pitch, int64_t K, int64_t M,
                                                         float *__restrict__ dst, uint64_t dst_pitch)
{
    const int64_t total = M * K;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / K;
        const int64_t k = i - r * K;
        const uint16_t *row = reinterpret_cast<const uint16_t *>(src + r * src_pitch);
        dst[r * dst_pitch + k] = f16_bits_to_f32(row[k]);
    }
}

// MXFP4 (microscaled e2m1 values: 32 weights share one power-of-two scale).
// Scale 2^e with e = floor(log2 amax) - 2, so that amax lands in [4, 8), where
// e2m1's largest value 6 is; stored as the byte e + 127, e at least -127.  The
// codes are w / 2^e rounded to e2m1 (nearest even, above 6 to 6, the sign of
// w kept): v_cvt_scalef32_pk_fp4_f32 divides by the scale and rounds two
// values at once.  A block holding an infinity or a NaN stores the scale byte
// 255 (not a number) and zero codes.
//
// Bound by memory (4 or 2 bytes read per weight, 17/32 written).  Four lanes
// share a block, eight neighbouring weights each, so a wave's loads are
// contiguous; amax comes by two DPP exchanges within the four.  Byte j holds
// codes j and j + 16, so lane pairs (0, 2) and (1, 3) exchange their packed
// nibbles and lanes 0 and 1 store 8 code bytes each.
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(const void *__restrict__ src, uint64_t src_pitch,
                                                             int64_t K, int64_t M, uint8_t *__restrict__ dst,
                                                             uint64_t dst_pitch)
{
    const int64_t nblk = K / 32;
    const int64_t total = M * nblk * 4;
    const int64_t qoff = quant_offset(K, 1);
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    // total and step are multiples of 4: a block's four lanes stay together
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t bi = i >> 2;
        const int part = (int)(i & 3);
        const int64_t r = bi / nblk;
        const int64_t b = bi - r * nblk;
        float v[8];
        if constexpr (BF16) {
            const uint4 h = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + r * src_pitch + b * 32 + 8 * part);
            const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __builtin_bit_cast(float, w[j] << 16);
                v[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
            }
        } else {
            const float *w = static_cast<const float *>(src) + r * src_pitch + b * 32 + 8 * part;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = w[j];
        }
        // the largest magnitude as bits: an infinity or NaN compares above
        // every finite value
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t m = __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu;
            amax = m > amax ? m : amax;
        }
        // quad_perm [1, 0, 3, 2], then [2, 3, 0, 1]
        uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0xB1, 0xF, 0xF, true);
        amax = o > amax ? o : amax;
        o = (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0x4E, 0xF, 0xF, true);
        amax = o > amax ? o : amax;
        // the exponent field of amax is floor(log2 amax) + 127 (0 below 2^-126,
        // where e would be under -127 anyway)
        const uint32_t field = amax >> 23;
        const bool bad = field == 255u;
        const uint32_t se = field > 2u ? field - 2u : 0u;
        const float scale = __builtin_bit_cast(float, se << 23);
        uint32_t code = 0;
        code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[0], v[1], scale, 0);
        code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[2], v[3], scale, 1);
        code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[4], v[5], scale, 2);
        code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(code, v[6], v[7], scale, 3);
        code = bad ? 0u : code;
        // nibble j of `code` is code 8 part + j; lanes 0, 1 take the matching
        // nibbles of lanes 2, 3 (codes 16 further) as high nibbles
        const uint32_t high = (uint32_t)__builtin_amdgcn_mov_dpp((int)code, 0x4E, 0xF, 0xF, true);
        uint8_t *row = dst + r * dst_pitch;
        if (part < 2) {
            auto spread = [](uint32_t n) {          // nibbles 0..3 to the low halves of four bytes
                n = (n | (n << 8)) & 0x00FF00FFu;
                return (n | (n << 4)) & 0x0F0F0F0Fu;
            };
            const uint32_t w0 = spread(code & 0xFFFFu) | (spread(high & 0xFFFFu) << 4);
            const uint32_t w1 = spread(code >> 16) | (spread(high >> 16) << 4);
            *reinterpret_cast<uint2 *>(row + qoff + 16 * b + 8 * part) = make_uint2(w0, w1);
        }
        if (part == 0) row[b] = (uint8_t)(bad ? 255u : se);
        if (b == 0 && part == 3)
            for (int64_t p = nblk; p < qoff; ++p) row[p] = 0;
    }
}

// W' = 2^e * value: two values of a byte per conversion, exact (a scale byte
// of 255 gives NaN).  Four lanes per block, as above: lane `part` expands the
// four code bytes 4 part .. 4 part + 3 into two runs of four floats.
__global__ __launch_bounds__(256) void dequantize_mxfp4_kernel(const uint8_t *__restrict__ src, uint64_t src_pitch,
                                                               int64_t K, int64_t M, float *__restrict__ dst,
                                                               uint64_t dst_pitch)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const int64_t nblk = K / 32;
    const int64_t total = M * nblk * 4;
    const int64_t qoff = quant_offset(K, 1);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t bi = i >> 2;
        const int part = (int)(i & 3);
        const int64_t r = bi / nblk;
        const int64_t b = bi - r * nblk;
        const uint8_t *row = src + r * src_pitch;
        const float scale = __builtin_bit_cast(float, (uint32_t)row[b] << 23);
        const uint32_t w = *reinterpret_cast<const uint32_t *>(row + qoff + 16 * b + 4 * part);
        const f32x2 a0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
        const f32x2 a1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
        const f32x2 a2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
        const f32x2 a3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
        float *out = dst + r * dst_pitch + b * 32 + 4 * part;
        out[0] = a0.x;
        out[1] = a1.x;
        out[2] = a2.x;
        out[3] = a3.x;
        out[16] = a0.y;
        out[17] = a1.y;
        out[18] = a2.y;
        out[19] = a3.y;
    }
}

unsigned grid_for(int64_t items)
{
    const int64_t blocks = (items + 255) / 256;
    return (unsigned)(blocks < 65536 ? (blocks > 0 ? blocks : 1) : 65536);
}

}  // namespace

hipError_t launch_quantize(const float *src, uint64_t src_pitch_elems, int64_t K, int64_t M,
                           uint8_t *dst, uint64_t dst_pitch, int type, hipStream_t stream,
                           bool q4_amax7, int scale_shift)
{
    if ((type & ~kSrcBf16) == W_MXFP4) {
        const int64_t lanes = M * (K / 32) * 4;
        if (lanes == 0) return hipSuccess;
        if (type & kSrcBf16)
            hipLaunchKernelGGL(quantize_mxfp4_kernel<true>, dim3(grid_for(lanes)), dim3(256), 0, stream,
                               (const void *)src, src_pitch_elems, K, M, dst, dst_pitch);
        else
            hipLaunchKernelGGL(quantize_mxfp4_kernel<false>, dim3(grid_for(lanes)), dim3(256), 0, stream,
                               (const void *)src, src_pitch_elems, K, M, dst, dst_pitch);
        return hipGetLastError();
    }
    const int64_t items = M * (K / (scale_shift ? 64 : 32));
    if (items == 0) return hipSuccess;
    const dim3 grid(grid_for(items)), block(256);
#define QMM_QUANT(T, D, B) hipLaunchKernelGGL((quantize_kernel<T, D, B>), grid, block, 0, stream, \
                                              src, src_pitch_elems, K, M, dst, dst_pitch)
    if (scale_shift == 0) {
        if (type == W_Q8_0) QMM_QUANT(W_Q8_0, 127, 32);
        else if (q4_amax7) QMM_QUANT(W_Q4_0, 7, 32);
        else QMM_QUANT(W_Q4_0, 8, 32);
    } else {
        if (type == W_Q8_0) QMM_QUANT(W_Q8_0, 127, 64);
        else if (q4_amax7) QMM_QUANT(W_Q4_0, 7, 64);
        else QMM_QUANT(W_Q4_0, 8, 64);
    }
#undef QMM_QUANT
    return hipGetLastError();
}

hipError_t launch_dequantize(const uint8_t *src, uint64_t src_pitch, int64_t K, int64_t M,
                             int type, float *dst, uint64_t dst_pitch_elems, hipStream_t stream,
                             int scale_shift)
{
    if (type == W_F16) {
        if (M * K == 0) return hipSuccess;
        hipLaunchKernelGGL(f16_to_f32_kernel, dim3(grid_for(M * K)), dim3(256), 0, stream,
                           src, src_pitch, K, M, dst, dst_pitch_elems);
        return hipGetLastError();
    }
    if (type == W_MXFP4) {
        const int64_t lanes = M * (K / 32) * 4;
        if (lanes == 0) return hipSuccess;
        hipLaunchKernelGGL(dequantize_mxfp4_kernel, dim3(grid_for(lanes)), dim3(256), 0, stream,
                           src, src_pitch, K, M, dst, dst_pitch_elems);
        return hipGetLastError();
    }
    const int64_t items = M * (K / (scale_shift ? 64 : 32));
    if (items == 0) return hipSuccess;
    const dim3 grid(grid_for(items)), block(256);
    if (type == W_Q8_0) {
        if (scale_shift) hipLaunchKernelGGL((dequantize_kernel<W_Q8_0, 64>), grid, block, 0, stream, src, src_pitch, K, M, dst, dst_pitch_elems);
        else hipLaunchKernelGGL((dequantize_kernel<W_Q8_0, 32>), grid, block, 0, stream, src, src_pitch, K, M, dst, dst_pitch_elems);
    } else {
        if (scale_shift) hipLaunchKernelGGL((dequantize_kernel<W_Q4_0, 64>), grid, block, 0, stream, src, src_pitch, K, M, dst, dst_pitch_elems);
        else hipLaunchKernelGGL((dequantize_kernel<W_Q4_0, 32>), grid, block, 0, stream, src, src_pitch, K, M, dst, dst_pitch_elems);
    }
    return hipGetLastError();
}

}  // namespace qmm
