// Before and after the full-cache decode kernel: the prologue (work plan and query operands)
// and the join of units that several CTAs shared.
//
// Both are bound by latency. The prologue (one block plans, four per unit make its operand)
// ends some 4 us after its start, much of that instruction fetches of code that runs once: the
// plan's loops are kept rolled and its divisions out of line, and 512 threads beat 256 (32 units of
// 16384 tokens 71.7 against 72.3 us a call). The join takes 5 to 10 us alone and cold, by how
// many pieces the units have, 1.5 to 4 in a call; it starts when the last block of the decode is
// at its end, and its partials come from L2.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "full.cuh"
#include "ptx.cuh"

namespace dsa {
namespace full {
namespace {

constexpr int kPrologueThreads = 512;
constexpr int kWarps = kPrologueThreads / 32;
constexpr int kQuarterPairs = kHeadsPerCta / 4;
static_assert(kWarps == kQuarterPairs, "a warp per pair");
constexpr int kStageBytes = kQImageBytes / 4;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ void scan2(int64_t& a, int32_t& b, int64_t* sa, int32_t* sb, int64_t* ta, int32_t* tb) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t ia = a;
    int32_t ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, ia, o);
        const int32_t y = __shfl_up_sync(0xffffffffu, ib, o);
        if (lane >= o) {
            ia += x;
            ib += y;
        }
    }
    __syncthreads();  // the previous round's sums are read
    if (lane == 31) {
        sa[warp] = ia;
        sb[warp] = ib;
    }
    __syncthreads();
    int64_t pa = 0;
    int32_t pb = 0;
    *ta = 0;
    *tb = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            pa += sa[w];
            pb += sb[w];
        }
        *ta += sa[w];
        *tb += sb[w];
    }
    a = pa + ia - a;
    b = pb + ib - b;
}

// One block: the line of tiles (see full.cuh). Thread t has units [t*per, (t+1)*per): a sweep
// sums their tiles, one scan gives every unit its place, a second sweep writes the units'
// entries and which unit each range starts in (cta_k, shared memory), and thread c then writes
// range c's.
__device__ void make_plan(const Params& p, int32_t* cta_k) {
    __shared__ int64_t sa[kWarps];
    __shared__ int32_t sb[kWarps];
    if (threadIdx.x == 0) atomicExch(p.status, 0);
    bool any_over = false;
    // Longest and shortest length of a unit's rows.
    auto lengths = [&](int32_t u, int32_t* top, int32_t* low) {
        const int32_t seq = u / p.groups, first = (u - seq * p.groups) * kHeadsPerCta;
        const int32_t r0 = first / p.heads, r1 = (min(first + kHeadsPerCta, p.pairs) - 1) / p.heads;
        *top = 0;
        *low = INT32_MAX;
        // Verify rows grow by one from the first to the last.
#pragma unroll 1
        for (int32_t i = r0; i <= r1; i += p.verify_rows && i < r1 ? r1 - r0 : 1) {
            bool over;
            const int32_t n = row_len(p, seq, i, &over);
            any_over |= over;
            *top = max(*top, n);
            *low = min(*low, n);
        }
    };
    const int32_t per = (p.units + kPrologueThreads - 1) / kPrologueThreads;
    const int32_t lo = static_cast<int32_t>(min(static_cast<int64_t>(p.units), static_cast<int64_t>(threadIdx.x) * per));
    const int32_t hi = min(p.units, lo + per);
    int64_t at = 0;
    int32_t k = 0, top = 0, low = 0;
#pragma unroll 1
    for (int32_t u = lo; u < hi; ++u) {
        lengths(u, &top, &low);
        at += (top + kTile - 1) / kTile;
        k += top > 0 ? 1 : 0;
    }
    int64_t tiles;
    int32_t live;
    scan2(at, k, sa, sb, &tiles, &live);
    const Line line = make_line(tiles, live, p.max_ctas);
#pragma unroll 1
    for (int32_t c = line.ctas + threadIdx.x; c < p.max_ctas; c += kPrologueThreads) p.plan.cta[c].begin = p.plan.cta[c].end = 0;
#pragma unroll 1
    for (int32_t u = lo; u < hi; ++u) {
        if (hi - lo > 1) lengths(u, &top, &low);
        UnitPieces q{0, 0, 0, 0};
        if (top > 0) {
            const int64_t b = at + line.gap * k, e = b + (top + kTile - 1) / kTile;
            p.plan.start[k] = b;
            p.plan.unit[k] = u;
            p.plan.max_len[k] = top;
            p.plan.min_len[k] = low;
            int32_t c0, c1;
            q = unit_pieces(line, k, b, e, &c0, &c1);
#pragma unroll 1
            for (int32_t c = c0; c < c1; ++c) cta_k[c] = k;
            at += e - b;
            ++k;
        }
        p.plan.pieces[u] = q;
    }
    __syncthreads();
#pragma unroll 1
    for (int32_t c = threadIdx.x; c < line.ctas; c += kPrologueThreads) {
        const int32_t first = cta_k[c];
        const int64_t begin = range_begin(line, c), end = range_begin(line, c + 1);
        p.plan.cta[c] = CtaStart{begin, end, segment(begin, end, line.gap, c, true, first, p.plan.unit[first], p.plan.start[first],
                                                     p.plan.max_len[first], p.plan.min_len[first]), line.gap, 0};
    }
    // The status was cleared before the scan's barriers.
    if (any_over) report(p, kStatusBounds);
}

// Query operand of a lane quarter of one unit, 16 of its pairs, as the selected decode's prologue
// makes it: a warp per pair, lane l dims [16l, 16l+16); a head's bf16 query as two E4M3 terms
// after a scaling by a power of two (exact for elements from 2^-9 of its largest, smaller ones off
// by 2^-16 of it at most), rows 2k and 2k+1 of the quarter the two terms of its pair k, stored
// chunk-major. The head's scale of its dots is positive (the decode takes maxima of the dots): a
// negative score scale turns the codes' signs, a zero one zeroes the codes. A head with a NaN or
// an infinity gets zero codes and a NaN scale, which makes all its scores NaN. A unit without a
// token writes its zeros here. (A block per unit, four pairs a warp, ended a microsecond later
// than the plan does.)
__device__ void prepare(const Params& p, int32_t unit, int quarter, uint8_t* stage) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hl = kQuarterPairs * quarter + warp;
    const int32_t seq = unit / p.groups, first = (unit % p.groups) * kHeadsPerCta;
    const int32_t valid = min(kHeadsPerCta, p.pairs - first);
    const int64_t pair = static_cast<int64_t>(seq) * p.pairs + first + hl;
    uint4 raw[2] = {};
    if (hl < valid) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + pair * kLatent + lane * 16);
        raw[0] = src[0];
        raw[1] = src[1];
    }
    bool none = true;  // checked while the queries are on their way
#pragma unroll 1
    for (int32_t i = first / p.heads; i <= (first + valid - 1) / p.heads; ++i) {
        bool over;
        none &= row_len(p, seq, i, &over) == 0;
    }
    if (none) {
        if (hl < valid) {
            uint4* o = reinterpret_cast<uint4*>(p.out + pair * kLatent + lane * 16);
            o[0] = o[1] = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
    uint32_t amax = 0;  // magnitudes as bits: NaN and infinity are the largest
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = max(amax, max((w[k] << 16) & 0x7FFFFFFFu, w[k] & 0x7FFF0000u));
    amax = __reduce_max_sync(0xffffffffu, amax);
    const int E = static_cast<int>(amax >> 23);
    const bool broken = E == 255;
    int e = amax > 0u ? 134 - E : 0;  // amax * 2^e in [128, 256)
    e = e > 126 ? 126 : (e < -126 ? -126 : e);
    const float back = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    const float sign = p.score_scale > 0.0f ? 1.0f : (p.score_scale < 0.0f ? -1.0f : 0.0f);
    const float sc = __uint_as_float(static_cast<uint32_t>(e + 127) << 23) * sign;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float vh[4], vl[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const uint32_t bits = m & 1 ? w[2 * k + m / 2] & 0xFFFF0000u : w[2 * k + m / 2] << 16;
            const float v = broken ? 0.0f : __uint_as_float(bits) * sc;
            vh[m] = __uint_as_float(__float_as_uint(v) & 0xFFF00000u);
            vl[m] = v - vh[m];
        }
        hi[k] = f32x2_to_e4m3x2(vh[0], vh[1]) | (f32x2_to_e4m3x2(vh[2], vh[3]) << 16);
        lo[k] = f32x2_to_e4m3x2(vl[0], vl[1]) | (f32x2_to_e4m3x2(vl[2], vl[3]) << 16);
    }
    const int r = 2 * warp;
    *reinterpret_cast<uint4*>(stage + r * 512 + ((lane ^ r) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(stage + (r + 1) * 512 + ((lane ^ (r + 1)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (lane == 0)
        p.qscale[static_cast<int64_t>(unit) * kHeadsPerCta + hl] =
            broken || p.score_scale != p.score_scale ? __uint_as_float(0x7FC00000u)
                                                     : fmaxf(fabsf(p.score_scale) * back, 0x1p-120f);
    __syncthreads();
    uint8_t* img = p.qimg + static_cast<int64_t>(unit) * kQImageBytes + quarter * 32 * 16;
    for (int k = threadIdx.x; k < kQImageBytes / 4 / 16; k += kPrologueThreads) {
        const int c = k >> 5, row = k & 31;
        *reinterpret_cast<uint4*>(img + c * 2048 + row * 16) = *reinterpret_cast<const uint4*>(stage + row * 512 + ((c ^ row) << 4));
    }
}

__global__ void __launch_bounds__(kPrologueThreads) full_prologue_kernel(const Params p) {
    extern __shared__ __align__(16) uint8_t stage[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x - 1;
    if (b < 0) make_plan(p, reinterpret_cast<int32_t*>(stage));
    else prepare(p, b >> 2, b & 3, stage);
}

// ------------------------------------------------------------------------------------
// Join of the pieces of split units
// ------------------------------------------------------------------------------------
constexpr int kCombineThreads = 256;
constexpr int kCombineWarps = kCombineThreads / 32;
constexpr int kDims = 32;   // dims of a block: the lanes of a warp
constexpr int kFlight = 4;  // pieces whose loads a warp has in flight

// Partial k holds O_k / l_k (f16, E4M3 code units) and lse_k = m_k + log2 l_k; out = v_scale *
// sum_k 2^(lse_k - M) O_k / sum_k 2^(lse_k - M). A warp folds pieces of 8 pairs x 32 dims, with
// a running maximum per pair, kFlight pieces at a time.
//   kSplit = 1: block (unit, 32 dims), a warp per 8-pair group, each over all pieces
//   kSplit = 8: block (unit, 32 dims, 8-pair group), the warps share the pieces and join
//               through shared memory; for few units, which the most pieces come with
template <int kSplit>
__global__ void __launch_bounds__(kCombineThreads, 5) full_combine_kernel(const Params p) {
    constexpr int kGroups = kCombineWarps / kSplit;  // 8-pair groups of a block
    static_assert(kSplit == 1 || kGroups == 1, "one group, or one warp per group");
    __shared__ float w_s[kCombineWarps][kFlight][8];
    __shared__ __align__(16) float a_s[kCombineWarps][8];
    __shared__ float m_s[kCombineWarps][8], sum_s[kCombineWarps][8];
    __shared__ float o_s[kSplit > 1 ? kSplit : 1][8][kDims + 1];
    __shared__ __align__(16) __nv_bfloat16 out_s[8 * kGroups][kDims];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int32_t unit = blockIdx.x;
    const int group = kSplit > 1 ? blockIdx.z : warp;  // of 8 pairs
    const int part = kSplit > 1 ? warp : 0;            // this warp's share of the pieces
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const UnitPieces q = p.plan.pieces[unit];
    const int pieces = q.pieces;
    if (pieces < 2) return;  // written whole, or zeros already
    auto slot = [&](int i) { return static_cast<int64_t>(i == 0 ? q.slot_lo : 2 * (q.c_lo + i)); };
    const uint4* po = reinterpret_cast<const uint4*>(p.part_o) + (static_cast<int64_t>(blockIdx.y) * 8 + group) * kDims + lane;
    constexpr int64_t kPartVecs = kHeadsPerCta * kLatent / 8;
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
                lse[i] = k0 + i * kSplit < pieces ? p.part_lse[slot(k0 + i * kSplit) * kHeadsPerCta + group * 8 + lane] : kNegInf;
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
    const int32_t seq = unit / p.groups, first = (unit % p.groups) * kHeadsPerCta;
    const int hl = t / 4, c = (t % 4) * 8, pair = first + (kSplit > 1 ? group * 8 : 0) + hl;
    if (hl < 8 * kGroups && pair < p.pairs)
        *reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(seq) * p.pairs + pair) * kLatent + blockIdx.y * kDims + c) =
            *reinterpret_cast<const uint4*>(&out_s[hl][c]);
}

}  // namespace
}  // namespace full

cudaError_t full_plan_setup() {
    cudaError_t e = cudaFuncSetAttribute(full::full_prologue_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(full::full_combine_kernel<1>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(full::full_combine_kernel<8>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
}

cudaError_t launch_full_plan(const full::Params& p, cudaStream_t stream) {
    full::full_prologue_kernel<<<4 * p.units + 1, full::kPrologueThreads, full::kStageBytes, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_full_combine(const full::Params& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    // With fewer units than an eighth of the CTAs a unit comes in more than eight pieces.
    const bool split = p.units * 8 <= p.max_ctas;
    cfg.gridDim = dim3(p.units, kLatent / full::kDims, split ? kHeadsPerCta / 8 : 1);
    cfg.blockDim = dim3(full::kCombineThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return split ? cudaLaunchKernelEx(&cfg, full::full_combine_kernel<8>, p) : cudaLaunchKernelEx(&cfg, full::full_combine_kernel<1>, p);
}

}  // namespace dsa
