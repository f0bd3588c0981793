// moe_group.hip -- slots (token, choice) grouped by expert, and the weighted
// sum over each token's slots: what stands before and after the grouped
// products of a mixture-of-experts layer for many tokens (gemm_grouped.hip).
//
// Grouping is a stable counting sort by expert on the device, so that a layer
// needs no host in between.  Lanes of a wave with the same expert find each other
// by balloting the bits of the expert's number, 64 slots at a time: a slot's rank
// in its wave is the wave's count of that expert so far (in LDS, its own) and
// the lanes before.  A scan over (expert, wave) turns the counts into places, and
// no place depends on which wave is faster.
//
// One launch, of a workgroup up to kGroupWhole slots and of one for 1024 slots up
// to kGroupAll; each of those counts all the others' slots too, with LDS
// additions spread over eight counters per expert, which costs less than the
// second launch, the workspace and the wait between (32744 slots over 128 experts
// through the binding: 9.4 us, 14.5 with two launches; the kernel 9.6, and 10.6 with
// workgroups of 2048 slots, of which 4 are the count of the others' slots).  More
// slots go to 64 workgroups which count in a first launch and add up the workgroups
// before them in a second one (70000 slots of 8 experts 20 us, 524288 of 128 28, 2^24
// 731).  Bound by launches and a few dependent passes over LDS.
#include "qmm_internal.h"

namespace qmm {
namespace {

constexpr int kWaves = 16;
constexpr int kThreads = 64 * kWaves;

struct GroupArgs {
    const int32_t *ids;
    int32_t *offsets, *order, *place;
    int32_t *counts;          // several workgroups: [workgroup][bucket]
    int32_t S, E, chunk;      // slots, experts, slots per workgroup (a multiple of R kThreads)
    int32_t bits;             // of a bucket's number (0 .. E: E for empty slots)
};

enum { kWhole = 0, kCount = 1, kPlace = 2, kAll = 3 };
constexpr int kSpread = 8;        // kAll: counters per bucket, by lane

// R: slots per thread and round.  ONE: a workgroup's slots are one round, whose
// buckets and ranks stay in registers; else it walks over its rounds twice.
template <int STEP, int R, bool ONE>
__global__ __launch_bounds__(kThreads) void moe_group_kernel(const GroupArgs a)
{
    extern __shared__ int32_t lds[];
    const int NB = a.E + 1;
    int32_t *const base = lds + kWaves * NB;      // [NB]
    __shared__ int32_t wave_total[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // [kWaves][NB]; volatile, as other lanes' writes change what a lane reads
    volatile int32_t *const cnt = lds;
    volatile int32_t *const mine = cnt + wave * NB;
    for (int i = tid; i < kWaves * NB; i += kThreads) cnt[i] = 0;
    if constexpr (STEP == kAll)
        for (int i = tid; i < 2 * kSpread * NB; i += kThreads) base[NB + i] = 0;
    __syncthreads();
    const int64_t from = (int64_t)blockIdx.x * a.chunk + (int64_t)wave * (a.chunk / kWaves);
    const int64_t to = from + a.chunk / kWaves < a.S ? from + a.chunk / kWaves : a.S;
    // a round: the buckets of the slots s0 + 64 i + lane (-1: none), and their
    // ranks among the wave's slots of that bucket
    int32_t bucket[R], rank[R];
    auto walk = [&](int64_t s0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t s = s0 + 64 * i + lane;
            const int32_t id = s < to ? a.ids[s] : -1;
            bucket[i] = s >= to ? -1 : id >= 0 && id < a.E ? id : a.E;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int b = bucket[i];
            uint64_t same = __ballot(b >= 0);
            for (int k = 0; k < a.bits; ++k) {
                const uint64_t m = __ballot(b >> k & 1);
                same &= b >> k & 1 ? m : ~m;
            }
            if (b >= 0) {
                const int before = __builtin_popcountll(same & ((1ull << lane) - 1));
                const int c = mine[b];
                rank[i] = c + before;
                __builtin_amdgcn_wave_barrier();
                if (before == 0) mine[b] = c + __builtin_popcountll(same);
            }
            __builtin_amdgcn_wave_barrier();
        }
    };
    for (int64_t s0 = from; s0 < to; s0 += 64 * R) walk(s0);
    if constexpr (STEP == kAll) {
        // the slots of the workgroups before this one, and all others
        int32_t *const before = base + NB, *const after = before + kSpread * NB;     // [NB][kSpread]
        const int64_t start = (int64_t)blockIdx.x * a.chunk;
        for (int64_t s0 = tid; s0 < a.S; s0 += 8 * kThreads) {
            int32_t id[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) id[i] = s0 + i * kThreads < a.S ? a.ids[s0 + i * kThreads] : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t s = s0 + i * kThreads;
                const int b = id[i] >= 0 && id[i] < a.E ? id[i] : a.E;
                if (s < a.S) atomicAdd((s < start ? before : after) + b * kSpread + (lane & (kSpread - 1)), 1);
            }
        }
    }
    __syncthreads();
    // each bucket's first rank of each wave, and its total
    for (int b = tid; b < NB; b += kThreads) {
        int run = 0, all = 0, before = 0;
        if constexpr (STEP == kPlace) {
#pragma unroll 8
            for (int g = 0; g < (int)gridDim.x; ++g) {
                const int c = a.counts[(int64_t)g * NB + b];
                before += g < (int)blockIdx.x ? c : 0;
                all += c;
            }
            run = before;
        }
        if constexpr (STEP == kAll) {
#pragma unroll
            for (int i = 0; i < kSpread; ++i) {
                run += base[NB + b * kSpread + i];
                all += base[NB + (NB + b) * kSpread + i];
            }
            all += run;
        }
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int c = cnt[w * NB + b];
            cnt[w * NB + b] = run;
            run += c;
        }
        if constexpr (STEP == kCount) a.counts[(int64_t)blockIdx.x * NB + b] = run;
        else base[b] = STEP == kWhole ? run : all;
    }
    if constexpr (STEP == kCount) return;
    __syncthreads();
    // the buckets' first places: a scan of the totals, thread t of bucket t (E
    // is at most kThreads, so that only bucket kThreads may be left over)
    const int total = tid < NB ? base[tid] : 0;
    int upto = total;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int o = __shfl_up(upto, m);
        upto += lane >= m ? o : 0;
    }
    if (lane == 63) wave_total[wave] = upto;
    __syncthreads();
    int first = upto - total;
    for (int w = 0; w < wave; ++w) first += wave_total[w];
    if (tid < NB) base[tid] = first;
    if (NB > kThreads && tid == kThreads - 1) base[kThreads] = first + total;
    __syncthreads();
    if (blockIdx.x == 0)
        for (int b = tid; b < NB; b += kThreads) a.offsets[b] = base[b];
    auto put = [&](int64_t s0, bool again) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t s = s0 + 64 * i + lane;
            const int b = bucket[i];
            if (b >= 0) {
                // in a second walk the counters go on from the first ranks
                const int pos = base[b] + rank[i] + (again ? 0 : mine[b]);
                a.order[pos] = (int32_t)s;
                a.place[s] = b < a.E ? pos : -1;
            }
        }
    };
    if constexpr (ONE) {
        if (from < to) put(from, false);
    } else {
        for (int64_t s0 = from; s0 < to; s0 += 64 * R) {
            walk(s0);
            put(s0, true);
        }
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
        // eight slots at a time, their loads in flight together (one after the other
        // 64 tokens of eight slots took 5.2 us, so 4.7)
        for (int c0 = 0; c0 < a.k; c0 += 8) {
            int32_t p[8];
            float w[8];
            float4 v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int64_t at = n * a.k + (c0 + c < a.k ? c0 + c : c0);
                p[c] = c0 + c < a.k ? a.place[at] : -1;
                w[c] = a.weights[at];
            }
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (p[c] >= 0) v[c] = *reinterpret_cast<const float4 *>(a.d + (uint64_t)p[c] * a.d_pitch + m);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if (p[c] < 0) continue;
                s.x = fmaf(w[c], v[c].x, s.x);
                s.y = fmaf(w[c], v[c].y, s.y);
                s.z = fmaf(w[c], v[c].z, s.z);
                s.w = fmaf(w[c], v[c].w, s.w);
            }
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

template <int STEP, int R, bool ONE>
hipError_t launch_step(const GroupArgs &a, unsigned groups, hipStream_t stream)
{
    constexpr int ints = kWaves + 1 + (STEP == kAll ? 2 * kSpread : 0), most = ints * (QMM_MOE_MAX_ROUTED + 1) * 4;
    const int bytes = ints * (a.E + 1) * 4;
    static_assert(QMM_MOE_MAX_ROUTED <= kThreads, "one thread per expert");
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&moe_group_kernel<STEP, R, ONE>), most);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((moe_group_kernel<STEP, R, ONE>), dim3(groups), dim3(kThreads), bytes, stream, a);
    return hipGetLastError();
}
template <int R, bool ONE>
hipError_t launch_both(const GroupArgs &a, unsigned groups, hipStream_t stream)
{
    const hipError_t e = launch_step<kCount, R, ONE>(a, groups, stream);
    return e != hipSuccess ? e : launch_step<kPlace, R, ONE>(a, groups, stream);
}

}  // namespace

hipError_t launch_moe_group(const int32_t *ids, int64_t S, int64_t E, int32_t *offsets, int32_t *order, int32_t *place,
                            void *ws, hipStream_t stream)
{
    GroupArgs a = {ids, offsets, order, place, static_cast<int32_t *>(ws), (int32_t)S, (int32_t)E, 0, 0};
    while (E >> a.bits) ++a.bits;
    constexpr int64_t few = 2 * kThreads, many = 8 * kThreads;
    if (S <= kGroupAll) {
        a.chunk = S <= few ? few : S <= kGroupWhole ? many : kThreads;
        if (S <= few) return launch_step<kWhole, 2, true>(a, 1, stream);
        if (S <= kGroupWhole) return launch_step<kWhole, 8, true>(a, 1, stream);
        return launch_step<kAll, 1, true>(a, (unsigned)((S + kThreads - 1) / kThreads), stream);
    }
    const int64_t per = (S + kGroupChunks - 1) / kGroupChunks;
    a.chunk = (int32_t)((per + many - 1) / many * many);
    return per <= many ? launch_both<8, true>(a, kGroupChunks, stream) : launch_both<8, false>(a, kGroupChunks, stream);
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
