// Before and after the prompt-chunk attention: the work plan and the join of units that several
// ranges shared. Both are bound by latency. A short call is three launches and in each its first instructions and loads: 5 rows of
// 16 heads over 300 tokens 17.4 us. The join reads 128 KB of each piece, from the L2 cache mostly.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "prefill.cuh"
#include "ptx.cuh"

namespace dsa {
namespace prefill {
namespace {

constexpr int kFewThreads = 256, kManyThreads = 1024;  // of a plan's block
constexpr float kNegInf = -__builtin_huge_valf();

// Sum of v over the threads before this one; *total over all. A lane for each warp.
template <int kWarps>
__device__ __forceinline__ int64_t scan(int64_t v, int64_t* sums, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    __syncthreads();  // the previous scan's sums are read
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int64_t mine = lane < kWarps ? sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, mine, o);
        if (lane >= o) mine += x;
    }
    *total = __shfl_sync(0xffffffffu, mine, 31);
    const int64_t before = __shfl_sync(0xffffffffu, mine, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : 0) + inc - v;
}

// One block. Threads share the requests (a scan gives each its first row, another its first unit),
// then the units in equal parts, whatever request they belong to.
template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) prefill_plan_kernel(const __grid_constant__ Params p) {
    extern __shared__ int32_t mem[];
    constexpr int kWarps = kPlanThreads / 32;
    __shared__ int64_t sums[kWarps];
    __shared__ int32_t joins;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int32_t n = p.num_seqs, tid = threadIdx.x;
    int32_t* row0 = mem;              // [n + 1] first rows, cut to the rows there are
    int32_t* unit0 = row0 + n + 1;    // [n + 1] first units
    int32_t* range_k = unit0 + n + 1; // [clusters] unit that each range starts in
    if (tid == 0) {
        atomicExch(p.status, 0);
        joins = 0;
    }
    for (int32_t j = tid; j < p.most_joins; j += kPlanThreads) p.joins[j].pieces = 0;

    const int32_t per = (n + kPlanThreads - 1) / kPlanThreads;
    const int32_t lo = min(n, tid * per), hi = min(n, lo + per);
    bool bad = false;
    int64_t mine = 0, total;
    for (int32_t s = lo; s < hi; ++s) {
        const int32_t k = p.new_lens[s];
        bad |= k < 0;
        mine += max(k, 0);
    }
    int64_t at = scan<kWarps>(mine, sums, &total);
    bad |= total > p.max_rows;
    auto cut = [&](int64_t row) { return static_cast<int32_t>(row < p.max_rows ? row : p.max_rows); };
    mine = 0;
    for (int32_t s = lo; s < hi; ++s) {
        const int32_t row = cut(at), base = p.base_lens[s];
        at += max(p.new_lens[s], 0);
        const int32_t k = cut(at) - row;
        row0[s] = row;
        bad |= base < 0 || (k > 0 && static_cast<int64_t>(base) + k > p.room);
        mine += (static_cast<int64_t>(k) * p.heads + kPairs - 1) / kPairs;
    }
    int64_t unit = scan<kWarps>(mine, sums, &total);
    for (int32_t s = lo; s < hi; ++s) {
        unit0[s] = static_cast<int32_t>(unit);
        const int32_t end = s + 1 < hi ? row0[s + 1] : cut(at);
        unit += (static_cast<int64_t>(end - row0[s]) * p.heads + kPairs - 1) / kPairs;
    }
    if (hi == n && lo < n) row0[n] = cut(at);
    if (tid == 0) unit0[n] = static_cast<int32_t>(total);
    __syncthreads();

    const int32_t units = unit0[n], each = (units + kPlanThreads - 1) / kPlanThreads;
    const int32_t u0 = min(units, tid * each), u1 = min(units, u0 + each);
    int32_t s0 = 0;
    if (u0 < u1) {  // the last request whose first unit is at most u0
        int32_t top = n;
        while (top - s0 > 1) {
            const int32_t mid = (s0 + top) >> 1;
            if (unit0[mid] <= u0) s0 = mid; else top = mid;
        }
    }
    auto walk = [&](auto&& visit) {
        int32_t s = s0, seen = -1, base = 0;
        for (int32_t u = u0; u < u1; ++u) {
            while (u >= unit0[s + 1]) ++s;
            if (s != seen) base = max(p.base_lens[s], 0);
            seen = s;
            const int32_t first = (u - unit0[s]) * kPairs;
            const int32_t valid = min(kPairs, (row0[s + 1] - row0[s]) * p.heads - first);
            visit(u, s, base, first, valid, (pair_len(p, base, first + valid - 1) + kTile - 1) / kTile);
        }
    };
    int64_t tiles = 0;
    walk([&](int32_t, int32_t, int32_t, int32_t, int32_t, int32_t t) { tiles += t; });
    int64_t all;
    int64_t before = scan<kWarps>(tiles, sums, &all);
    const full::Line line = full::make_line(all, units, p.clusters, kGap);
    walk([&](int32_t u, int32_t s, int32_t base, int32_t first, int32_t valid, int32_t t) {
        const int64_t b = before + line.gap * u, e = b + t;
        before += t;
        p.units[u] = Unit{b, static_cast<int64_t>(row0[s]) * p.heads + first, s, first, valid, base};
        int32_t c0, c1;
        const full::UnitPieces q = full::unit_pieces(line, u, b, e, &c0, &c1);
        for (int32_t c = c0; c < c1; ++c) range_k[c] = u;
        if (q.pieces > 1) p.joins[atomicAdd(&joins, 1)] = Join{u, q.slot_lo, q.pieces, q.c_lo};
    });
    __syncthreads();
    for (int32_t c = tid; c < p.clusters; c += kPlanThreads) {
        Start st{};
        if (c < line.ctas) {
            st.begin = full::range_begin(line, c);
            st.end = full::range_begin(line, c + 1);
            st.gap = static_cast<int32_t>(line.gap);
            st.k = range_k[c];
            st.unit = p.units[st.k];
        }
        p.starts[c] = st;
    }
    if (bad) report(p, kStatusBounds);  // cleared before the scans' barriers
}

// ------------------------------------------------------------------------------------
// Join of the pieces of split units
// ------------------------------------------------------------------------------------
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kDims = 32;   // dims of a block: the lanes of a warp
constexpr int kFlight = 4;  // pieces whose loads a warp has in flight

// Partial k holds O_k / l_k (f16, E4M3 code units) and lse_k = m_k + log2 l_k; out = v_scale *
// sum_k 2^(lse_k - M) O_k / sum_k 2^(lse_k - M). A warp folds pieces of 8 pairs x 32 dims, with
// a running maximum per pair, kFlight pieces at a time.
//   kSplit = 1: block (join, 32 dims, 64 pairs), a warp per 8-pair group, each over all pieces
//   kSplit = 8: block (join, 32 dims, 8-pair group), the warps share the pieces and join
//               through shared memory; for few units, which the most pieces come with
template <int kSplit>
__global__ void __launch_bounds__(kJoinThreads, 5) prefill_join_kernel(const __grid_constant__ Params p) {
    constexpr int kGroups = kJoinWarps / kSplit;  // 8-pair groups of a block
    static_assert(kSplit == 1 || kGroups == 1, "one group, or one warp per group");
    __shared__ float w_s[kJoinWarps][kFlight][8];
    __shared__ __align__(16) float a_s[kJoinWarps][8];
    __shared__ float m_s[kJoinWarps][8], sum_s[kJoinWarps][8];
    __shared__ float o_s[kSplit > 1 ? kSplit : 1][8][kDims + 1];
    __shared__ __align__(16) __nv_bfloat16 out_s[8 * kGroups][kDims];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int group = kSplit > 1 ? blockIdx.z : blockIdx.z * kGroups + warp;  // of 8 pairs
    const int part = kSplit > 1 ? warp : 0;                                   // this warp's share of the pieces
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Join q = p.joins[blockIdx.x];
    const int pieces = q.pieces;
    if (pieces < 2) return;
    const Unit u = p.units[q.unit];
    auto slot = [&](int i) { return static_cast<int64_t>(i == 0 ? q.slot_lo : 2 * (q.c + i)); };
    constexpr int64_t kPartVecs = kPairs * kLatent / 8;
    const uint4* po = reinterpret_cast<const uint4*>(p.part_o) + (static_cast<int64_t>(blockIdx.y) * (kPairs / 8) + group) * kDims + lane;
    float acc[8] = {};
    float m_run = kNegInf, s_run = 0.0f;  // lanes 0..7: pair 8*group + lane
    for (int k0 = part; k0 < pieces; k0 += kSplit * kFlight) {
        uint4 raw[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            raw[i] = make_uint4(0, 0, 0, 0);
            if (k0 + i * kSplit < pieces) raw[i] = po[slot(k0 + i * kSplit) * kPartVecs];
        }
        __syncwarp();  // the previous turn's weights are read
        if (lane < 8) {
            float lse[kFlight], top = m_run;
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                lse[i] = k0 + i * kSplit < pieces ? p.part_lse[slot(k0 + i * kSplit) * kPairs + group * 8 + lane] : kNegInf;
                top = fmaxf(top, lse[i]);
            }
            const float a = m_run != kNegInf ? exp2f(m_run - top) : 0.0f;
            s_run *= a;
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                const float w = lse[i] != kNegInf ? exp2f(lse[i] - top) : 0.0f;
                s_run += w;
                w_s[warp][i][lane] = w;
            }
            a_s[warp][lane] = a;
            m_run = top;
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= a_s[warp][e];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const __half2* hv = reinterpret_cast<const __half2*>(&raw[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = __half22float2(hv[e]);
                acc[2 * e] = fmaf(w_s[warp][i][2 * e], f.x, acc[2 * e]);
                acc[2 * e + 1] = fmaf(w_s[warp][i][2 * e + 1], f.y, acc[2 * e + 1]);
            }
        }
    }
    if (lane < 8) {
        m_s[warp][lane] = m_run;
        sum_s[warp][lane] = s_run;
    }
    if constexpr (kSplit > 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o_s[part][e][lane] = acc[e];
        __syncthreads();
        // Warp w joins pair w over the parts.
        float top = kNegInf, sum = 0.0f, o = 0.0f;
#pragma unroll
        for (int i = 0; i < kSplit; ++i) top = fmaxf(top, m_s[i][warp]);
#pragma unroll
        for (int i = 0; i < kSplit; ++i) {
            const float w = m_s[i][warp] != kNegInf ? exp2f(m_s[i][warp] - top) : 0.0f;
            sum = fmaf(w, sum_s[i][warp], sum);
            o = fmaf(w, o_s[i][warp][lane], o);
        }
        out_s[warp][lane] = __float2bfloat16_rn(sum == 0.0f ? 0.0f : o * (p.v_scale / sum));
    } else {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float sum = sum_s[warp][e];
            out_s[warp * 8 + e][lane] = __float2bfloat16_rn(sum == 0.0f ? 0.0f : acc[e] * (p.v_scale / sum));
        }
    }
    __syncthreads();
    const int hl = t / 4, c = (t % 4) * 8, pair = blockIdx.z * 8 * kGroups + hl;
    if (hl < 8 * kGroups && pair < u.valid)
        *reinterpret_cast<uint4*>(p.out + (u.pair0 + pair) * kLatent + blockIdx.y * kDims + c) =
            *reinterpret_cast<const uint4*>(&out_s[hl][c]);
}

}  // namespace
}  // namespace prefill

cudaError_t prefill_plan_setup(int clusters) {
    const int smem = 2 * (DSA_MAX_PLAN_SEQS + 1) * 4 + clusters * 4;
    cudaError_t e = cudaFuncSetAttribute(prefill::prefill_plan_kernel<prefill::kManyThreads>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(prefill::prefill_join_kernel<1>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(prefill::prefill_join_kernel<8>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
}

cudaError_t launch_prefill_plan(const prefill::Params& p, cudaStream_t stream) {
    const int smem = 2 * (p.num_seqs + 1) * 4 + p.clusters * 4;
    if (p.small_plan) prefill::prefill_plan_kernel<prefill::kFewThreads><<<1, prefill::kFewThreads, smem, stream>>>(p);
    else prefill::prefill_plan_kernel<prefill::kManyThreads><<<1, prefill::kManyThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_prefill_join(const prefill::Params& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.most_joins, kLatent / prefill::kDims, p.few_units ? prefill::kPairs / 8 : 2);
    cfg.blockDim = dim3(prefill::kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return p.few_units ? cudaLaunchKernelEx(&cfg, prefill::prefill_join_kernel<8>, p)
                       : cudaLaunchKernelEx(&cfg, prefill::prefill_join_kernel<1>, p);
}

}  // namespace dsa
