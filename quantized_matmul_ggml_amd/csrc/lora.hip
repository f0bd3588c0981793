// lora.hip -- low-rank adapters of many requests at once, beside a projection
// that all of them share:
//   y[n] = base[n] + s_a B_a (A_a x[n]),   a = ids[n],
// A_a: r x K, B_a: M x r (bf16), for tokens of any mix of adapters.
//
// Two launches.  lora_shrink_kernel makes u = A_a x: a wave takes 16 tokens and
// a part of K, and goes through the different adapters among its tokens (a
// prompt's are all the same one; decoded tokens' may be sixteen) with
// v_mfma_f32_16x16x32_bf16; the parts' sums go to the workspace.
// lora_expand_kernel adds them up in order and makes base + B_a (s_a u): a wave
// takes 32 tokens and tiles of 32 outputs, with v_mfma_f32_32x32x16_bf16.  In
// both, each adapter's products are made for all tokens of the tile and kept
// for its own, so no token's values meet another's.
//
// Arithmetic: binary32 values (x when it is F32, and s_a u) enter the matrix
// cores as three bf16 parts whose sum is exact (row_tiles.h), so every product
// is exact and only binary32 sums and s_a u round.
//
// Bound by memory: decoding by the adapters' matrices (read once per tile of
// tokens that uses them) and the launches' latency, prompts by base and y.
#include "row_tiles.h"
#include "lora_plan.h"

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
    float *u;                          // [chunk][token][rp]
    int64_t N, M;
    int32_t L, K, r, rp;
    int32_t chunk, chunks;             // K per part, parts
    int32_t j1, j2;                    // waves that share a tile's adapters
    int32_t mt;                        // 32-output tiles per wave
    int64_t tasks1;                    // waves of the first launch
    int64_t m_blocks;                  // workgroups along M of the second
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

__device__ inline rt_bf16x8 load8(const uint16_t *p)
{
    return __builtin_bit_cast(rt_bf16x8, *reinterpret_cast<const uint4 *>(p));
}

template <bool F32X, int RT>
__global__ __launch_bounds__(256) void lora_shrink_kernel(const LoraArgs a)
{
    constexpr int PARTS = F32X ? 3 : 1, U = RT >= 8 ? 2 : 4;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int64_t task = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (task >= a.tasks1) return;
    const int j = (int)(task % a.j1), chunk = (int)(task / a.j1 % a.chunks);
    const int64_t n0 = task / a.j1 / a.chunks * 16;
    const int64_t n = n0 + c < a.N ? n0 + c : a.N - 1;
    int id = a.ids[n];
    if (n0 + c >= a.N || id >= a.L) id = -1;
    const int k_from = chunk * a.chunk, k_to = k_from + a.chunk < a.K ? k_from + a.chunk : a.K;
    for_adapters(id, 0xFFFF, j, a.j1, [&](int ad, uint64_t mask) {
        const uint16_t *rows = a.a + (uint64_t)ad * a.a_adapter;
        rt_f32x4 acc[RT] = {};
        for (int k0 = k_from; k0 < k_to; k0 += 32 * U) {
            uint4 xp[U][PARTS];
            rt_bf16x8 w[U][RT];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                // past the part's end its last step again, unused
                const int k = (k0 + 32 * i < k_to ? k0 + 32 * i : k_to - 32) + 8 * g;
                if constexpr (F32X) {
                    const float *p = static_cast<const float *>(a.x) + (uint64_t)n * a.x_pitch + k;
                    const rt_f32x4u lo = *reinterpret_cast<const rt_f32x4u *>(p), hi = *reinterpret_cast<const rt_f32x4u *>(p + 4);
                    const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                    split_parts(v, xp[i]);
                } else {
                    xp[i][0] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + (uint64_t)n * a.x_pitch + k);
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const int row = 16 * t + c < a.r ? 16 * t + c : a.r - 1;
                    w[i][t] = load8(rows + (uint64_t)row * a.a_pitch + k);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (k0 + 32 * i < k_to) {
#pragma unroll
                    for (int t = 0; t < RT; ++t)
#pragma unroll
                        for (int p = 0; p < PARTS; ++p)
                            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(rt_bf16x8, xp[i][p]), w[i][t], acc[t], 0, 0, 0);
                }
        }
        // D: tokens 4 g .. 4 g + 3, rank 16 t + c
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if ((mask >> (4 * g + i) & 1) && 16 * t + c < a.r)
                    a.u[((uint64_t)chunk * a.N + n0 + 4 * g + i) * a.rp + 16 * t + c] = acc[t][i];
    });
}

template <int RT>
__global__ __launch_bounds__(256) void lora_expand_kernel(const LoraArgs a)
{
    constexpr int RP = 16 * RT, LDU = RP + 4;
    __shared__ __attribute__((aligned(16))) float us[32 * LDU];
    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = (int)(blockIdx.x % a.j2);
    const int64_t block = blockIdx.x / a.j2 % a.m_blocks, n0 = blockIdx.x / a.j2 / a.m_blocks * 32;
    auto adapter = [&](int t) {
        const int id = n0 + t < a.N ? a.ids[n0 + t] : -1;
        return id < a.L ? id : -1;
    };
    // ---- s_a u of the tile's tokens, the parts added in order ----
    for (int i = tid; i < 32 * RP; i += 256) {
        const int t = i / RP, q = i % RP, ad = adapter(t);
        float s = 0.0f;
        if (ad >= 0 && q < a.r) {
            const float *p = a.u + (uint64_t)(n0 + t) * a.rp + q;
            for (int ch = 0; ch < a.chunks; ++ch) s += p[(uint64_t)ch * a.N * a.rp];
            if (a.scales) s *= a.scales[ad];
        }
        us[t * LDU + q] = s;
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
    const int id = adapter(l32);
    // the rows that this workgroup writes: its adapters' tokens, and for one of
    // the workgroups the tokens without one
    uint64_t rows = 0;
    for_adapters(id, 0xFFFFFFFF, j, a.j2, [&](int, uint64_t m) { rows |= m; });
    if (j == 0) rows |= __ballot(id < 0 && n0 + l32 < a.N) & 0xFFFFFFFF;
    if (!rows) return;
    for (int i = 0; i < a.mt; ++i) {
        const int64_t m0 = ((block * 4 + wave) * a.mt + i) * 32;
        if (m0 >= a.M) break;
        const int64_t m = m0 + l32, mr = m < a.M ? m : a.M - 1;
        float out[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int t = 8 * (r / 4) + 4 * h + r % 4;
            out[r] = a.base && (rows >> t & 1) && m < a.M ? a.base[(uint64_t)(n0 + t) * a.base_pitch + m] : 0.0f;
        }
        for_adapters(id, 0xFFFFFFFF, j, a.j2, [&](int ad, uint64_t mask) {
            const uint16_t *p = a.b + (uint64_t)ad * a.b_adapter + (uint64_t)mr * a.b_pitch + 8 * h;
            lr_f32x16 d = {};
#pragma unroll
            for (int q = 0; q < RT; ++q) {
                const uint4 zero = make_uint4(0, 0, 0, 0);
                const rt_bf16x8 w = 16 * q + 8 * h < a.r ? load8(p + 16 * q) : __builtin_bit_cast(rt_bf16x8, zero);
#pragma unroll
                for (int s = 0; s < 3; ++s)
                    d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(rt_bf16x8, up[q][s]), w, d, 0, 0, 0);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) out[r] = mask >> (8 * (r / 4) + 4 * h + r % 4) & 1 ? out[r] + d[r] : out[r];
        });
        if (m < a.M) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int t = 8 * (r / 4) + 4 * h + r % 4;
                if (rows >> t & 1) a.y[(uint64_t)(n0 + t) * a.y_pitch + m] = out[r];
            }
        }
    }
}

template <int RT>
hipError_t launch_rank(const LoraArgs &a, bool f32x, hipStream_t stream)
{
    const unsigned first = (unsigned)((a.tasks1 + 3) / 4);
    if (first == 0) {}                 // no K: every sum is empty
    else if (f32x) hipLaunchKernelGGL((lora_shrink_kernel<true, RT>), dim3(first), dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((lora_shrink_kernel<false, RT>), dim3(first), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const unsigned second = (unsigned)((a.N + 31) / 32 * a.m_blocks * a.j2);
    hipLaunchKernelGGL(lora_expand_kernel<RT>, dim3(second), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(const LoraTask &t, hipStream_t stream)
{
    const LoraPlan p = plan_lora(t.N, t.K, t.M, t.r, device_cus());
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
    a.tasks1 = p.tasks1;
    a.m_blocks = p.m_blocks;
    switch (p.rt) {
    case 1: return launch_rank<1>(a, t.f32x, stream);
    case 2: return launch_rank<2>(a, t.f32x, stream);
    case 4: return launch_rank<4>(a, t.f32x, stream);
    default: return launch_rank<8>(a, t.f32x, stream);
    }
}

}  // namespace qmm
