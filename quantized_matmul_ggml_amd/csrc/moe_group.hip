// moe_group.hip -- slots (token, choice) grouped by expert, and the weighted
// sum over each token's slots: what stands before and after the grouped
// products of a mixture-of-experts layer for many tokens (gemm_grouped.hip).
//
// Grouping is a stable counting sort by expert on the device, so that a layer
// needs no host in between.  Wave w of a workgroup counts a contiguous run of
// slots per expert in LDS; a scan over (expert, wave) turns the counts into
// places; the wave walks its run again, 64 slots at a time, and lanes with the
// same expert find their ranks by balloting the bits of the expert's number.
// No place depends on which wave is faster.  Up to kGroupSlots slots go to
// one workgroup in one launch; more to several, which count in a first launch
// and find their places from all workgroups' counts in a second one.
// Bound by latency: a few dependent passes over 4 bytes per slot.
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kWaves = 16;
constexpr int kThreads = 64 * kWaves;

struct GroupArgs {
    const int32_t *ids;
    int32_t *offsets, *order, *place;
    int32_t *counts;          // several workgroups: [workgroup][bucket]
    int32_t S, E, chunk;      // slots, experts, slots per workgroup (a multiple of kThreads)
    int32_t bits;             // of a bucket's number (0 .. E: E for empty slots)
};

enum { kWhole = 0, kCount = 1, kPlace = 2 };

template <int STEP>
__global__ __launch_bounds__(kThreads) void moe_group_kernel(const GroupArgs a)
{
    extern __shared__ int32_t lds[];
    const int NB = a.E + 1;
    int32_t *const cnt = lds;                     // [kWaves][NB]
    int32_t *const base = lds + kWaves * NB;      // [NB]
    __shared__ int32_t wave_total[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int i = tid; i < kWaves * NB; i += kThreads) cnt[i] = 0;
    __syncthreads();
    const int64_t from = (int64_t)blockIdx.x * a.chunk + (int64_t)wave * (a.chunk / kWaves);
    const int64_t to = from + a.chunk / kWaves < a.S ? from + a.chunk / kWaves : a.S;
    auto bucket = [&](int64_t s) {
        const int32_t id = a.ids[s];
        return id >= 0 && id < a.E ? id : a.E;
    };
    for (int64_t s = from + lane; s < to; s += 64) atomicAdd(&cnt[wave * NB + bucket(s)], 1);
    __syncthreads();
    // each bucket's counts of the waves before, and its total
    for (int b = tid; b < NB; b += kThreads) {
        int run = 0;
        for (int w = 0; w < kWaves; ++w) {
            const int c = cnt[w * NB + b];
            cnt[w * NB + b] = run;
            run += c;
        }
        if constexpr (STEP == kCount) {
            a.counts[(int64_t)blockIdx.x * NB + b] = run;
        } else if constexpr (STEP == kPlace) {
            int all = 0, before = 0;
            for (int g = 0; g < (int)gridDim.x; ++g) {
                const int c = a.counts[(int64_t)g * NB + b];
                before += g < (int)blockIdx.x ? c : 0;
                all += c;
            }
            for (int w = 0; w < kWaves; ++w) cnt[w * NB + b] += before;
            base[b] = all;
        } else {
            base[b] = run;
        }
    }
    if constexpr (STEP == kCount) return;
    __syncthreads();
    // the buckets' first places: a scan of the totals, thread t of bucket t (E
    // is at most kThreads, so that only bucket kThreads may be left over)
    const int mine = tid < NB ? base[tid] : 0;
    int upto = mine;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int o = __shfl_up(upto, m);
        upto += lane >= m ? o : 0;
    }
    if (lane == 63) wave_total[wave] = upto;
    __syncthreads();
    int first = upto - mine;
    for (int w = 0; w < wave; ++w) first += wave_total[w];
    if (tid < NB) base[tid] = first;
    if (NB > kThreads && tid == kThreads - 1) base[kThreads] = first + mine;
    __syncthreads();
    if (blockIdx.x == 0)
        for (int b = tid; b < NB; b += kThreads) a.offsets[b] = base[b];
    // a bucket's counter is its wave's own from here on; volatile, as other
    // lanes' writes change what a lane reads
    volatile int32_t *const at = cnt + wave * NB;
    for (int64_t s0 = from; s0 < to; s0 += 64) {
        const int64_t s = s0 + lane;
        const bool in = s < to;
        const int b = in ? bucket(s) : 0;
        uint64_t same = __ballot(in);
        for (int i = 0; i < a.bits; ++i) {
            const uint64_t m = __ballot(b >> i & 1);
            same &= b >> i & 1 ? m : ~m;
        }
        if (in) {
            const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
            const int c = at[b];
            const int pos = base[b] + c + rank;
            a.order[pos] = (int32_t)s;
            a.place[s] = b < a.E ? pos : -1;
            __builtin_amdgcn_wave_barrier();
            if (rank == 0) at[b] = c + __builtin_popcountll(same);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// y[n] = sum_s weights[n][s] d[place[n][s]], in slot order; slots without a
// place count for nothing, whatever their weight.  Four outputs per thread; d's
// rows are a multiple of four floats apart.
struct CombineArgs {
    const float *d;
    uint64_t d_pitch;
    const int32_t *place;
    const float *weights;
    void *y;
    uint64_t y_pitch;
    int64_t N, M, tasks;
    int32_t k, quads, vec, bf16_out;
};
__global__ __launch_bounds__(256) void moe_combine_kernel(const CombineArgs a)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.tasks; i += (int64_t)gridDim.x * 256) {
        const int64_t n = i / a.quads;
        const int64_t m = (i - n * a.quads) * 4;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int c = 0; c < a.k; ++c) {
            const int32_t p = a.place[n * a.k + c];
            if (p < 0) continue;
            const float w = a.weights[n * a.k + c];
            const float4 v = *reinterpret_cast<const float4 *>(a.d + (uint64_t)p * a.d_pitch + m);
            s.x = fmaf(w, v.x, s.x);
            s.y = fmaf(w, v.y, s.y);
            s.z = fmaf(w, v.z, s.z);
            s.w = fmaf(w, v.w, s.w);
        }
        const uint64_t o = (uint64_t)n * a.y_pitch + m;
        const float v[4] = {s.x, s.y, s.z, s.w};
        if (a.bf16_out) {
            __bf16 *y = static_cast<__bf16 *>(a.y) + o;
            if (a.vec && m + 4 <= a.M) {
                typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                *reinterpret_cast<bf16x4 *>(y) = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
            } else {
                for (int c = 0; c < 4; ++c)
                    if (m + c < a.M) y[c] = (__bf16)v[c];
            }
        } else {
            float *y = static_cast<float *>(a.y) + o;
            if (a.vec && m + 4 <= a.M) {
                *reinterpret_cast<float4 *>(y) = s;
            } else {
                for (int c = 0; c < 4; ++c)
                    if (m + c < a.M) y[c] = v[c];
            }
        }
    }
}

template <int STEP>
hipError_t launch_step(const GroupArgs &a, unsigned groups, hipStream_t stream)
{
    const int bytes = (kWaves + 1) * (a.E + 1) * 4;
    constexpr int most = (kWaves + 1) * (QMM_MOE_MAX_ROUTED + 1) * 4;
    static_assert(QMM_MOE_MAX_ROUTED <= kThreads, "one thread per expert");
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&moe_group_kernel<STEP>), most);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(moe_group_kernel<STEP>, dim3(groups), dim3(kThreads), bytes, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_group(const int32_t *ids, int64_t S, int64_t E, int32_t *offsets, int32_t *order, int32_t *place,
                            void *ws, hipStream_t stream)
{
    const int64_t groups = moe_group_chunks(S);
    GroupArgs a = {ids, offsets, order, place, static_cast<int32_t *>(ws), (int32_t)S, (int32_t)E, 0, 0};
    const int64_t per = (S + groups - 1) / groups;
    a.chunk = (int32_t)((per + kThreads - 1) / kThreads * kThreads);
    while (E >> a.bits) ++a.bits;
    if (groups == 1) return launch_step<kWhole>(a, 1, stream);
    const hipError_t e = launch_step<kCount>(a, (unsigned)groups, stream);
    return e != hipSuccess ? e : launch_step<kPlace>(a, (unsigned)groups, stream);
}

hipError_t launch_moe_combine(const float *d, uint64_t d_pitch, const int32_t *place, const float *weights, int k,
                              int64_t N, int64_t M, const GroupedOut &y, hipStream_t stream)
{
    CombineArgs a = {d, d_pitch, place, weights, y.data, y.pitch_elems, N, M, 0, k, (int32_t)((M + 3) / 4), 0, y.bf16};
    const uintptr_t wide = y.bf16 ? 8 : 16;
    a.vec = (uintptr_t)y.data % wide == 0 && y.pitch_elems % 4 == 0;
    a.tasks = N * a.quads;
    if (a.tasks == 0) return hipSuccess;
    const int64_t want = (a.tasks + 255) / 256;
    hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)(want < (1 << 20) ? want : (1 << 20))), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace qmm
