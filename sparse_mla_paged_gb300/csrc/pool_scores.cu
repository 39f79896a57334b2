// Pooled index scores: the cheap score by which the selector ranks the pools of each row.
//
//   I[r,j]     = s_j * sum_h w[r,h] * max(0, q[r,h,:] . k_j)       (k_j, s_j: index cache)
//   score[r,p] = max over the kpool tokens j of pool p of I[r,j], and -inf unless the whole
//                pool lies at or before the row's position q_pos[r]
//
// The dots are a matrix product, tokens x (rows x heads), on tcgen05 tensor cores: the keys'
// E4M3 codes are the A operand as they lie in the cache (M = 128 tokens of a tile), the
// queries of up to 128/heads rows of one sequence the B operand (N = rows x heads). A BF16
// query is two E4M3 terms (hi = its top 4 significant bits after scaling its head by a power
// of two, lo = the rest), both accumulated into the same FP32 columns, so the product is
// exact but for elements below 2^-9.9 of their head's largest (they may be off by 2^-16.9 of it:
// a third term would cost half as many MMAs again). With tokens as rows of D, a token's heads
// lie in one thread's columns: the relu, the weighted sum over heads and the key's scale need no
// exchange between threads, and the maximum over a pool's tokens is a few shuffles between
// neighbouring lanes. The power of two goes into the head's weight.
//
// A unit is a group of rows of one sequence; its 128-token tiles up to the last pool that one
// of its rows sees stand on a line, unit after unit with gaps between (kGap), that is cut into
// equal ranges, one per persistent block (scores of different tokens are independent: nothing to
// join). Each block sums the units' tiles for itself, 4 bytes a row from L2, which costs less than
// a launch or a workspace for a plan. Warps of a block: epilogue (four per 128 tokens, TMEM lane
// quarters; they also write the queries' operand of each unit), two that issue the MMAs, two that
// load key tiles into a ring in the 128-byte-swizzled operand layout and run ahead over units:
// with tensor-map boxes of a page's rows when pages, pools and tiles fit each other, else with
// 16-byte copies.
//
// Shared memory's bandwidth is what the tile loop competes for (a tile is written once and
// read twice, by the hi and the lo product, with the queries each time): the weights therefore
// stay in registers, a warp's columns being the same in every tile. Read from shared memory
// for every tile they cost as much of it as the MMAs (pooled 128k 413 us, prefill 588).
//
// Measured, 64 heads: 128 rows over 131072 tokens each (pooled 128k) 327 us, 6.8 TB/s, what a
// copy of the keys would take. 1024 rows over one cache of 32768 tokens (prefill) 378 us in
// bursts, 1490 TFLOP/s with the two terms counted once, 0.78 of the rate of a BF16 product (403 us
// in a long loop, at the power limit); there the issue
// slots are 62 % busy, the tensor pipe 58 %, and shared memory about three quarters (an MMA of
// N = 128 reads its operands for as long as it computes, and tiles are written beside it). 64
// rows over 8 to 32 thousand tokens 34 us, 25.4 of them at the HBM's rate; the rest is the
// launch, the shares, the queries' operand and the first tiles, one after another, which is all
// of a small call's 8 us. One MMA warp for 128 columns: prefill 440 us.
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128;                       // tokens of a tile: MMA M
constexpr int kLoadWarps = 2;                    // copies: 64 tokens of a tile each
constexpr int kLoadTurns = 2;                    // of 32 tokens
constexpr int kTileBytes = kTile * kIndexDim;    // 16 KB of codes
constexpr int kBarEpilogue = 1;
// Starting a unit (queries, weights, an empty pipeline) costs its block the time of several
// tiles; so many places of the line after each unit hold none, so that the block that starts one
// has fewer tiles. With less than two tiles a block (by the pools that there are room for) the
// starts run side by side anyway and gaps would only crowd the tiles. 64 rows of 64 heads
// over 8 to 32 thousand tokens 35.4 -> 33.6 us, 17 rows of 48 heads over 6 to 20 thousand 14.9 ->
// 12.6; with gaps also below, 23 rows over 1 to 2 thousand would take 9.0 instead of 8.4.
constexpr int kGap = 6;
constexpr int kFillPools = 1024;                 // pools of one piece of the fill with -inf

// Variants by the columns (rows x padded heads) that one unit's MMAs take: MMA N.
template <int kCols>
struct Shape {
    static constexpr int kCtas = kCols == 64 ? 2 : 1;  // blocks per SM
    static constexpr int kStages = kCols == 64 ? 4 : 10;
    static constexpr int kEpiWarps = kCols / 16;       // 64 columns, whose weights fit its registers, a warp
    static constexpr int kSets = kEpiWarps / 4;        // warps that share a lane quarter
    static constexpr int kWeights = kCols / kSets;     // columns of a warp: 64
    static constexpr int kChunk = kCols == 64 ? 8 : 16;  // columns of a tensor-memory load, as registers allow
    static constexpr int kDBufs = 4;
    // MMA warps, and load warps of boxes, that take tiles in turn. Each has to meet every phase of
    // its barriers (a wait for a phase that has not begun passes as the one before it), so the
    // ring and the D buffers are a multiple of them: a slot is always the same warp's.
    static constexpr int kMmaWarps = 2;
    static_assert(kStages % kMmaWarps == 0 && kDBufs % kMmaWarps == 0, "slots belong to warps");
    static constexpr int kMmaWarp0 = kEpiWarps;
    static constexpr int kLoadWarp0 = kMmaWarp0 + kMmaWarps;
    static constexpr int kThreads = (kLoadWarp0 + kLoadWarps) * 32;
    static constexpr int kMaxRows = kCols / 16;
    // A scale slot is written again kScaleSlots tiles later: by then the MMA kStages tiles before
    // that has run, hence the epilogue kDBufs tiles before it has read its scales.
    static constexpr int kScaleSlots = 16;
    static_assert(kScaleSlots >= kStages + kDBufs, "scale slots");
    static constexpr int kOffQ = kStages * kTileBytes;                      // [2 terms][cols][128 codes]
    static constexpr int kOffScale = kOffQ + 2 * kCols * kIndexDim;         // float [slots][128]
    static constexpr int kOffW = kOffScale + kScaleSlots * kTile * 4;       // float [cols]
    static constexpr int kOffToken = kOffW + kCols * 4;                     // float [rows][128] token scores
    static constexpr int kOffVis = kOffToken + kMaxRows * kTile * 4;        // int32 [rows] visible pools of a row
    static constexpr int kOffScan = kOffVis + kMaxRows * 4;                 // int64 [16] warp sums, then what they find
    static constexpr int kOffBars = kOffScan + 20 * 8;
    static constexpr int BAR_FULL = 0, BAR_EMPTY = kStages, BAR_DFULL = 2 * kStages, BAR_DEMPTY = BAR_DFULL + kDBufs,
                         BAR_QFULL = BAR_DEMPTY + kDBufs, BAR_QSEEN = BAR_QFULL + 1, BAR_DRAIN = BAR_QSEEN + 1, kNumBars = BAR_DRAIN + 1;
    static constexpr int kOffTmem = kOffBars + kNumBars * 8;
    static constexpr int kOffAbort = kOffTmem + 4;
    static constexpr int kSmem = kOffAbort + 4 + 1024;                      // slack for the 1024-byte alignment
    static constexpr uint32_t kTmemCols = kDBufs * kCols;
    static_assert(kCtas * (kSmem + 1024) <= 228 * 1024 && kCtas * kTmemCols <= 512, "blocks per SM");
};

constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// acc[k] += w[k] * relu(x[k]) of four columns. Two as max(x, 0) on the compare pipe (half
// rate), two as x + |x| on the FMA pipe, so that neither is what the epilogue waits for; the
// weights of the latter are stored halved. Both keep a NaN. (Packed two-wide FMAs need moves
// to pair their operands up and come to more instructions.)
__device__ __forceinline__ void fma_relu4(float (&acc)[4], const float* w, const uint32_t* x) {
    const float x2 = __uint_as_float(x[2]), x3 = __uint_as_float(x[3]);
    acc[0] = fmaf(w[0], max_nan(__uint_as_float(x[0]), 0.0f), acc[0]);
    acc[1] = fmaf(w[1], max_nan(__uint_as_float(x[1]), 0.0f), acc[1]);
    acc[2] = fmaf(w[2], x2 + fabsf(x2), acc[2]);
    acc[3] = fmaf(w[3], x3 + fabsf(x3), acc[3]);
}

// Columns of a lane in two steps: the load, and the wait that makes its registers valid (they
// are operands of the wait so that no use moves ahead of it).
__device__ __forceinline__ void load_columns(uint32_t at, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(at));
}
__device__ __forceinline__ void load_columns(uint32_t at, uint32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(at));
}
__device__ __forceinline__ void wait_columns(uint32_t (&v)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7])
                 :: "memory");
}
__device__ __forceinline__ void wait_columns(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :: "memory");
}
__device__ __forceinline__ void tma_box3(uint32_t dst, const void* tmap, int32_t y, int32_t z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst), "l"(tmap), "r"(0), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// One unit as a block sees it.
struct Unit {
    int32_t seq, row0, rows;  // rows [row0, row0 + rows) of sequence seq
    int32_t seen;             // pools that some of them sees: [0, seen)
    int64_t tiles;
};

template <int kCols>
struct Block {
    using S = Shape<kCols>;
    const PoolScoresParams& p;
    uint8_t* smem;
    uint32_t sbase;
    volatile int* abort_flag;
    int32_t groups, group_rows, units, per_tile;  // units of a sequence, rows of a unit, units, pools of a tile
    int32_t gap;                                  // places on the line after each unit that hold no tile
    int64_t begin, end;                           // this block's range of the line
    int32_t unit0;                                // unit that it starts in, and where that unit starts
    int64_t start0;

    __device__ uint32_t bar(int i) const { return sbase + S::kOffBars + 8 * i; }
    __device__ void fail(int code) const {
        atomicCAS(p.status, 0, code);
        *abort_flag = 1;
    }
    __device__ void wait(int b, uint32_t parity) const {
        if (!mbar_wait(bar(b), parity, abort_flag, p.wait_limit_ns)) fail(kStatusTimeout);
        __syncwarp();
    }
    // The epilogue's: the longest limit, or less once another warp gave up (the call's own limit
    // between its FMAs makes 1024 rows over 32768 tokens 390 to 405 us, 378 without).
    __device__ void epilogue_wait(int b, uint32_t parity) const {
        if (!mbar_wait(bar(b), parity, abort_flag, kDefaultWaitLimitNs)) fail(kStatusTimeout);
        __syncwarp();
    }
    __device__ int32_t visible(int32_t row) const {
        const int32_t q = __ldg(p.q_pos + row);  // (q + 1) / kpool in 32 bits: q + 1 <= 2^31
        return q < 0 ? 0 : min(static_cast<int32_t>(divide(static_cast<uint32_t>(q) + 1u, p.by_kpool)), p.n_pools);
    }
    __device__ Unit unit(int32_t u) const {
        Unit x;
        x.seq = u / groups;
        const int32_t first = (u - x.seq * groups) * group_rows;
        x.row0 = x.seq * p.rows_per_seq + first;
        x.rows = min(group_rows, p.rows_per_seq - first);
        x.seen = 0;
        for (int r = 0; r < x.rows; ++r) x.seen = max(x.seen, visible(x.row0 + r));
        x.tiles = x.seen / per_tile + (x.seen % per_tile != 0 ? 1 : 0);
        return x;
    }
    // Calls f(unit, first tile, last tile + 1 of the unit) for the stretches of this block's
    // range, in order; the whole warp calls it (units without tiles are passed 32 at a time).
    template <typename F>
    __device__ void stretches(F&& f) const {
        int64_t at = start0;
        int32_t u = unit0;
        while (at < end && u < units) {
            const Unit x = unit(u);
            if (x.tiles > 0) {
                const int64_t t0 = begin > at ? begin - at : 0, t1 = min(end - at, x.tiles);
                if (t0 < t1) f(x, static_cast<int32_t>(t0), static_cast<int32_t>(t1));
                at += x.tiles + gap;
                ++u;
            } else {
                const int32_t v = u + 1 + static_cast<int32_t>(threadIdx.x & 31);
                const uint32_t some = __ballot_sync(0xffffffffu, v < units && unit(v).tiles > 0);
                u += some ? __ffs(some) : 33;
            }
        }
    }
};

// This block's equal share of the line of tiles and gaps.
template <int kCols>
__device__ void share(Block<kCols>& b) {
    using S = Shape<kCols>;
    constexpr int kWarps = S::kThreads / 32;
    int64_t* sum_s = reinterpret_cast<int64_t*>(b.smem + S::kOffScan);
    int64_t* found = sum_s + 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t per = (b.units + S::kThreads - 1) / S::kThreads;
    const int32_t lo = min(static_cast<int64_t>(b.units), static_cast<int64_t>(threadIdx.x) * per), hi = min(b.units, lo + per);
    int64_t mine = 0;
#pragma unroll 4
    for (int32_t u = lo; u < hi; ++u) {
        const int64_t n = b.unit(u).tiles;
        mine += n > 0 ? n + b.gap : 0;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) sum_s[warp] = incl;
    if (threadIdx.x == 0) found[0] = b.units;
    __syncthreads();
    int64_t at = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at += sum_s[w];
        total += sum_s[w];
    }
    const int64_t ctas = gridDim.x, c = blockIdx.x;
    b.begin = c * total / ctas;
    b.end = (c + 1) * total / ctas;
    if (b.begin < b.end && at <= b.begin && b.begin < at + mine) {  // the one thread whose units hold the first tile
        int32_t u = lo;
        for (;; ++u) {
            const int64_t n = b.unit(u).tiles, w = n > 0 ? n + b.gap : 0;
            if (b.begin < at + w) break;
            at += w;
        }
        found[0] = u;
        found[1] = at;
    }
    __syncthreads();
    b.unit0 = static_cast<int32_t>(found[0]);
    b.start0 = found[1];
}

// A unit's queries as two E4M3 terms, its weights with the heads' powers of two; a half-warp
// per (row, head), eight dims a lane, eight loads in flight. Columns past the heads are zero.
template <int kHeads, int kCols>
__device__ void load_queries(const Block<kCols>& b, const Unit& x) {
    using S = Shape<kCols>;
    constexpr int kStep = 2 * S::kEpiWarps;  // columns per turn of the epilogue warps
    const int sub = threadIdx.x & 15;
    float* w_s = reinterpret_cast<float*>(b.smem + S::kOffW);
    const int cols = x.rows * kHeads;        // a multiple of 16, hence of kStep or half of it
    for (int c0 = threadIdx.x >> 4; c0 - static_cast<int>(threadIdx.x >> 4 & 1) < cols; c0 += 8 * kStep) {
        uint4 raw[8];
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int col = c0 + i * kStep, h = col % kHeads;
            const int64_t rh = static_cast<int64_t>(x.row0 + col / kHeads) * b.p.heads + h;
            raw[i] = make_uint4(0, 0, 0, 0);
            w[i] = 0.0f;
            if (col < cols && h < b.p.heads) {
                raw[i] = __ldg(reinterpret_cast<const uint4*>(b.p.q + rh * kIndexDim) + sub);
                w[i] = __ldg(b.p.w + rh);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int col = c0 + i * kStep;
            const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            uint32_t top = 0;  // magnitudes as bits: NaN and infinity are the largest
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max(top, max((u[k] << 16) & 0x7FFFFFFFu, u[k] & 0x7FFF0000u));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            // e with top * 2^e in [240, 480), whose first four bits are E4M3 numbers; a head with a NaN
            // or an infinity gets zero codes and a NaN weight, which makes all its row's scores NaN.
            const int E = static_cast<int>(top >> 23);
            const bool broken = E == 255;
            int e = top > 0u ? ((top & 0x7FFFFFu) < 0x700000u ? 135 : 134) - E : 0;
            e = e > 126 ? 126 : (e < -126 ? -126 : e);
            const float sc = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float vh[4], vl[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const uint32_t bits = m & 1 ? u[2 * k + m / 2] & 0xFFFF0000u : u[2 * k + m / 2] << 16;
                    const float v = broken ? 0.0f : __uint_as_float(bits) * sc;
                    vh[m] = __uint_as_float(__float_as_uint(v) & 0xFFF00000u);
                    vl[m] = v - vh[m];
                }
                hi[k] = f32x2_to_e4m3x2(vh[0], vh[1]) | (f32x2_to_e4m3x2(vh[2], vh[3]) << 16);
                lo[k] = f32x2_to_e4m3x2(vl[0], vl[1]) | (f32x2_to_e4m3x2(vl[2], vl[3]) << 16);
            }
            if (col < cols) {
                uint8_t* at = b.smem + S::kOffQ + col * kIndexDim + (((sub >> 1) ^ (col & 7)) << 4) + (sub & 1) * 8;
                *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2*>(at + kCols * kIndexDim) = make_uint2(lo[0], lo[1]);
                if (sub == 0)
                    w_s[col] = broken ? __uint_as_float(0x7FC00000u)  // halved in every second pair: fma_relu4
                                      : w[i] * __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * (col & 2 ? 0.5f : 1.0f);
            }
        }
    }
}

// -inf past the tiles of each unit: pieces of kFillPools pools of a row, over all blocks' load
// warps, which are done before the rest of their block.
template <int kCols>
__device__ void fill(const Block<kCols>& b) {
    using S = Shape<kCols>;
    const PoolScoresParams& p = b.p;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - S::kLoadWarp0;
    const int32_t pieces = (p.n_pools + kFillPools - 1) / kFillPools;
    const int64_t items = static_cast<int64_t>(p.num_seqs) * p.rows_per_seq * pieces, step = static_cast<int64_t>(gridDim.x) * kLoadWarps;
    // Each lane looks for one piece's part to fill; the warp then fills what its lanes found.
    for (int64_t first = blockIdx.x + static_cast<int64_t>(gridDim.x) * w; first < items; first += 32 * step) {
        const int64_t i = first + lane * step;
        int64_t lo = 0, hi = 0;  // as offsets into scores
        if (i < items) {
            const int32_t row = static_cast<int32_t>(i / pieces), piece = static_cast<int32_t>(i % pieces);
            const int32_t seq = row / p.rows_per_seq, g = (row - seq * p.rows_per_seq) / b.group_rows;
            const int64_t done = b.unit(seq * b.groups + g).tiles * b.per_tile, at = static_cast<int64_t>(row) * p.n_pools;
            lo = at + max(static_cast<int64_t>(piece) * kFillPools, done);
            hi = at + min(static_cast<int64_t>(piece + 1) * kFillPools, static_cast<int64_t>(p.n_pools));
        }
        for (uint32_t some = __ballot_sync(0xffffffffu, lo < hi); some; some &= some - 1) {
            const int from = __ffs(some) - 1;
            const int64_t end = __shfl_sync(0xffffffffu, hi, from);
            for (int64_t k = __shfl_sync(0xffffffffu, lo, from) + lane; k < end; k += 32) p.scores[k] = kNegInf;
        }
    }
}

// Load by tensor-map boxes: load warp w takes every kMmaWarps-th tile from its w-th on; lane l
// has box l, p.box_rows rows of one page (looked up a tile of its own ahead): the codes by the
// map, the scales by a plain bulk copy. (One lane issuing all boxes in turn was slower: pooled
// 128k 414 us.)
template <int kCols>
__device__ void run_load_boxes(const Block<kCols>& b, const CUtensorMap* tmap) {
    using S = Shape<kCols>;
    const PoolScoresParams& p = b.p;
    const int lane = threadIdx.x & 31;
    const uint32_t w = (threadIdx.x >> 5) - S::kLoadWarp0;
    const int tokens = b.per_tile * p.kpool;
    const bool mine = lane * p.box_rows < tokens;
    const uint32_t box_codes = static_cast<uint32_t>(p.box_rows) * kIndexDim, box_scales = static_cast<uint32_t>(p.box_rows) * 4u;
    uint32_t tau = 0, issued = 0;  // tiles so far, and past the last one that this warp asked for
    bool stop = false;
    b.stretches([&](const Unit& x, int32_t t0, int32_t t1) {
        const int32_t limit = x.seen * p.kpool;
        const int32_t* table = p.block_tables + static_cast<int64_t>(x.seq) * p.max_blocks_per_seq;
        // This lane's page of tile t (-1: bad, -2: nothing that a row sees) and the row its box starts at.
        auto look = [&](int32_t t, int32_t* row) -> int32_t {
            const int32_t pos = t * tokens + lane * p.box_rows;
            *row = 0;
            if (!mine || t >= t1 || pos >= limit) return -2;
            const int32_t blk = static_cast<int32_t>(divide(static_cast<uint32_t>(pos), p.by_block));
            *row = pos - blk * p.block_size;
            return p.max_blocks_per_seq == 0 || blk < p.max_blocks_per_seq ? max(__ldg(table + blk), -1) : -1;
        };
        const int32_t own = t0 + static_cast<int32_t>((w - tau) & (S::kMmaWarps - 1));  // this warp's first tile here
        int32_t row_next, page_next = look(own, &row_next);
        for (int32_t t = own; t < t1 && !stop; t += S::kMmaWarps) {
            const uint32_t ta = tau + static_cast<uint32_t>(t - t0);
            const int32_t page = page_next, row = row_next;
            page_next = look(t + S::kMmaWarps, &row_next);
            const uint32_t e = ta % S::kStages;
            if (ta >= S::kStages) b.wait(S::BAR_EMPTY + e, (ta / S::kStages - 1) & 1);
            // After a failed wait nothing more is issued (the drain below finds what is in flight).
            if (__shfl_sync(0xffffffffu, *b.abort_flag, 0)) {
                stop = true;
                break;
            }
            float* scales = reinterpret_cast<float*>(b.smem + S::kOffScale) + (ta % S::kScaleSlots) * kTile;
            if (page == -1) {  // tokens without a page score -inf
                for (int i = 0; i < p.box_rows; ++i) scales[lane * p.box_rows + i] = kNegInf;
                atomicCAS(p.status, 0, kStatusBounds);
            }
            __syncwarp();  // lane 0's arrival releases these stores too
            const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, page >= 0));
            const uint32_t full = b.bar(S::BAR_FULL + e);
            if (lane == 0) mbar_arrive_expect_tx(full, boxes * (box_codes + box_scales));
            __syncwarp();
            if (page >= 0) {
                tma_box3(b.sbase + e * kTileBytes + lane * box_codes, tmap, row, page, full);
                bulk_g2s(smem_u32(scales) + lane * box_scales,
                         p.cache + page * p.page_stride + static_cast<int64_t>(p.block_size) * kIndexDim + static_cast<int64_t>(row) * 4, box_scales, full);
            }
            __syncwarp();
            issued = ta + 1;
        }
        tau += static_cast<uint32_t>(t1 - t0);
    });
    fill(b);
    // No copy into shared memory is in flight when the block exits: the bytes of the last tiles
    // that were asked for. (Waited for by the tiles of the whole range, which an abort leaves
    // unasked, a slot's wait could have been for a phase of the other parity and passed at once.)
    if (lane == 0) {
        for (uint32_t i = issued > S::kStages ? issued - S::kStages : 0; i < issued; ++i) {
            if ((i & (S::kMmaWarps - 1)) != w) continue;
            const uint64_t since = globaltimer_ns();
            while (!mbar_try_wait(b.bar(S::BAR_FULL + static_cast<int>(i % S::kStages)), (i / S::kStages) & 1) &&
                   globaltimer_ns() - since < kDrainLimitNs) {
            }
        }
    }
    __syncwarp();
}

// Copy warps: warp w takes tokens 64w .. 64w+63 of every tile; lane l resolves the pages of
// tokens 64w + l and 64w + 32 + l (a tile ahead of their copies) and copies their scales.
template <int kCols>
__device__ void run_load(const Block<kCols>& b) {
    using S = Shape<kCols>;
    const PoolScoresParams& p = b.p;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - S::kLoadWarp0;
    const int tokens = b.per_tile * p.kpool;
    const int tk0 = 64 * w + lane;
    constexpr int64_t kNone = -1, kBad = -2;
    uint32_t tau = 0;
    b.stretches([&](const Unit& x, int32_t t0, int32_t t1) {
        const int32_t limit = x.seen * p.kpool;
        const int32_t* table = p.block_tables + static_cast<int64_t>(x.seq) * p.max_blocks_per_seq;
        // Page and row there of this lane's token of turn i, tile t (row -1: none). What is made of
        // them is left to the next turn: using the page here would wait for its load.
        auto look = [&](int32_t t, int i, int32_t& page, int32_t& row) {
            row = -1;
            const int tk = tk0 + 32 * i;
            const int32_t pos = t * tokens + tk;
            if (t >= t1 || tk >= tokens || pos >= limit) return;
            const int32_t blk = static_cast<int32_t>(divide(static_cast<uint32_t>(pos), p.by_block));
            row = pos - blk * p.block_size;
            page = (p.max_blocks_per_seq == 0 || blk < p.max_blocks_per_seq) ? __ldg(table + blk) : -1;
        };
        int64_t code[kLoadTurns], to_scale[kLoadTurns];  // offset of a token's codes, and from there to its scale
        int32_t next_page[kLoadTurns] = {}, next_row[kLoadTurns];
#pragma unroll
        for (int i = 0; i < kLoadTurns; ++i) look(t0, i, next_page[i], next_row[i]);
        for (int32_t t = t0; t < t1; ++t, ++tau) {
#pragma unroll
            for (int i = 0; i < kLoadTurns; ++i) {
                const int64_t row = next_row[i];
                code[i] = row < 0 ? kNone : (next_page[i] < 0 ? kBad : next_page[i] * p.page_stride + row * kIndexDim);
                to_scale[i] = static_cast<int64_t>(p.block_size) * kIndexDim - row * (kIndexDim - 4);
                look(t + 1, i, next_page[i], next_row[i]);
            }
            const int e = static_cast<int>(tau % S::kStages);
            if (tau >= S::kStages) b.wait(S::BAR_EMPTY + e, (tau / S::kStages - 1) & 1);
            const uint32_t dst = b.sbase + e * kTileBytes + 64 * w * kIndexDim;
#pragma unroll
            for (int i = 0; i < kLoadTurns; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int row = 4 * j + (lane >> 3), c = lane & 7;
                    const int64_t at = __shfl_sync(0xffffffffu, code[i], row);
                    const uint32_t d = (32 * i + row) * kIndexDim + ((c ^ (row & 7)) << 4);
                    cp_async_16_zfill(dst + d, p.cache + (at >= 0 ? at + c * 16 : 0), at >= 0 ? 16u : 0u);
                }
                float* slot = reinterpret_cast<float*>(b.smem + S::kOffScale) + (tau % S::kScaleSlots) * kTile + tk0 + 32 * i;
                if (code[i] >= 0) {
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(slot)),
                                 "l"(p.cache + code[i] + to_scale[i]) : "memory");
                } else {
                    *slot = kNegInf;  // a token without a page scores -inf
                    if (code[i] == kBad) atomicCAS(p.status, 0, kStatusBounds);
                }
            }
            cp_async_arrive_noinc(b.bar(S::BAR_FULL + e));
            __syncwarp();
            if (lane == 0) mbar_arrive(b.bar(S::BAR_FULL + e));  // releases the slots written by plain stores
        }
    });
    fill(b);
    cp_async_wait_all();
}

// MMA warp w issues every kMmaWarps-th tile from its w-th on: a tile's waits, fence, issue and
// commits are one chain of some 900 cycles, more than the MMAs of 128 columns take.
template <int kHeads, int kCols>
__device__ void run_mma(const Block<kCols>& b, uint32_t tmem) {
    using S = Shape<kCols>;
    const uint32_t w = (threadIdx.x >> 5) - S::kMmaWarp0;
    const uint32_t el = elect_one();
    const uint64_t q = smem_desc(b.sbase + S::kOffQ, 16, 1024, kSwizzle128B);
    uint32_t tau = 0, entered = 0;
    b.stretches([&](const Unit& x, int32_t t0, int32_t t1) {
        const uint32_t idesc = idesc_e4m3(kTile, 16, false, false) +
                               (static_cast<uint32_t>(x.rows * kHeads - 16) >> 3 << 17);  // N = rows x heads
        b.wait(S::BAR_QFULL, entered++ & 1);
        if (el) mbar_arrive(b.bar(S::BAR_QSEEN));  // a warp without a tile here must not miss the phase
        for (int32_t t = t0 + static_cast<int32_t>((w - tau) & (S::kMmaWarps - 1)); t < t1; t += S::kMmaWarps) {
            const uint32_t ta = tau + static_cast<uint32_t>(t - t0);
            const int e = static_cast<int>(ta % S::kStages), d = static_cast<int>(ta % S::kDBufs);
            b.wait(S::BAR_FULL + e, (ta / S::kStages) & 1);
            if (ta >= S::kDBufs) b.wait(S::BAR_DEMPTY + d, (ta / S::kDBufs - 1) & 1);
            fence_proxy_async_smem();
            tc_fence_after();
            const uint64_t k = smem_desc(b.sbase + e * kTileBytes, 16, 1024, kSwizzle128B);
            const uint32_t dst = tmem + d * kCols;
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t bq = q + static_cast<uint64_t>((term * kCols * kIndexDim + ks * 32) >> 4);
                    mma_e4m3_el(dst, k + static_cast<uint64_t>((ks * 32) >> 4), bq, idesc, term + ks > 0 ? 1u : 0u, el);
                }
            tc_commit_el(b.bar(S::BAR_EMPTY + e), el);
            tc_commit_el(b.bar(S::BAR_DFULL + d), el);
            if (el) mbar_arrive(b.bar(S::BAR_DFULL + d));
        }
        tau += static_cast<uint32_t>(t1 - t0);
    });
    // Every MMA has completed before the block gives its tensor memory back.
    tc_commit_el(b.bar(S::BAR_DRAIN), el);
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(b.bar(S::BAR_DRAIN), 0) && globaltimer_ns() - t0 < kDrainLimitNs) {
    }
    __syncwarp();
}

template <int kHeads, int kCols>
__device__ void run_epilogue(const Block<kCols>& b, uint32_t tmem) {
    using S = Shape<kCols>;
    const PoolScoresParams& p = b.p;
    constexpr bool kHalves = kHeads > S::kWeights;                // two warps have half of a row each
    constexpr int kRows = kHalves ? 1 : S::kWeights / kHeads;     // rows of a warp
    constexpr int kChunk = S::kChunk;
    constexpr int kRowChunks = (kHalves ? S::kWeights : kHeads) / kChunk, kChunks = S::kWeights / kChunk;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tk = threadIdx.x & 127, set = threadIdx.x >> 7;
    const float* w_s = reinterpret_cast<const float*>(b.smem + S::kOffW);
    const float* scale_s = reinterpret_cast<const float*>(b.smem + S::kOffScale);
    float* token_s = reinterpret_cast<float*>(b.smem + S::kOffToken);
    int32_t* vis_s = reinterpret_cast<int32_t*>(b.smem + S::kOffVis);
    const bool in_lanes = p.kpool <= 32 && (p.kpool & (p.kpool - 1)) == 0;  // a pool's tokens in one warp
    constexpr int kSteps = 5;  // exchanges for the maximum over a pool's lanes, those past its width without effect
    const int pool_tk = tk / p.kpool;
    const bool writer = tk % p.kpool == 0;
    const int row_first = kHalves ? 0 : set * kRows;
    uint32_t tau = 0, entered = 0;
    b.stretches([&](const Unit& x, int32_t t0, int32_t t1) {
        if (entered > 0) b.epilogue_wait(S::BAR_QSEEN, (entered - 1) & 1);
        ++entered;
        // The unit before is done with: its last D buffer was full, so its MMAs have read the
        // queries, and every epilogue warp has its weights.
        named_bar_sync<kBarEpilogue, S::kEpiWarps * 32>();
        load_queries<kHeads, kCols>(b, x);
        if (threadIdx.x < x.rows) vis_s[threadIdx.x] = b.visible(x.row0 + threadIdx.x);
        fence_proxy_async_smem();
        named_bar_sync<kBarEpilogue, S::kEpiWarps * 32>();
        if (lane == 0) mbar_arrive(b.bar(S::BAR_QFULL));
        const int mine = min(max(x.rows - row_first, 0), kRows);  // rows of this warp in the unit
        // This lane's pool of the tile at pool p is out[p], there for p < room and seen by row r
        // for p < vis[r].
        float* out = p.scores + static_cast<int64_t>(x.row0 + row_first) * p.n_pools + pool_tk;
        const int32_t room = in_lanes && writer && !(kHalves && set == 1) ? p.n_pools - pool_tk : 0;
        int32_t vis[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) vis[r] = r < mine ? vis_s[row_first + r] - pool_tk : 0;
        float w[S::kWeights];
#pragma unroll
        for (int i = 0; i < S::kWeights; ++i) w[i] = w_s[set * S::kWeights + i];
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + set * S::kWeights;
        // The tile before, whose pools' maxima are taken and stored between this one's FMAs, as
        // the next tile's barrier is polled and its first columns fetched before the last FMAs:
        // nothing that an epilogue warp waits for then stands alone (1024 rows of 64 heads over
        // 32768 tokens: 465 -> 405 us, then; two tiles at once or twice the warps were slower).
        float held[kRows] = {};
        int32_t held_at = p.n_pools;
        auto exchange = [&](int k) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float other = __shfl_xor_sync(0xffffffffu, held[r], 1 << k);
                if (p.kpool > 1 << k) held[r] = max_nan(held[r], other);
            }
        };
        auto store = [&]() {
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (r < mine && held_at < room) out[static_cast<int64_t>(r) * p.n_pools + held_at] = held_at < vis[r] ? held[r] : kNegInf;
        };
        b.epilogue_wait(S::BAR_DFULL + static_cast<int>(tau % S::kDBufs), (tau / S::kDBufs) & 1);
        tc_fence_after();
        uint32_t v[2][kChunk];
        load_columns(lanes + tau % S::kDBufs * kCols, v[0]);
        for (int32_t t = t0; t < t1; ++t, ++tau) {
            const uint32_t d = tau % S::kDBufs, d_next = (tau + 1) % S::kDBufs, turn_next = (tau + 1) / S::kDBufs & 1;
            const int32_t pool_t = t * b.per_tile;
            const float scale = scale_s[(tau % S::kScaleSlots) * kTile + tk];
            // Chunks of columns, the next one's load in flight while one is summed. The columns
            // of rows that the unit lacks hold anything; their sums are not used.
            float sums[kRows];
            bool ready = false;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = r * kRowChunks; i < (r + 1) * kRowChunks; ++i) {
                    wait_columns(v[i & 1]);
                    if (i + 1 < kChunks) {
                        load_columns(lanes + d * kCols + (i + 1) * kChunk, v[(i + 1) & 1]);
                        if (i + 2 == kChunks) ready = mbar_test_wait(b.bar(S::BAR_DFULL + static_cast<int>(d_next)), turn_next) || t + 1 >= t1;
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(b.bar(S::BAR_DEMPTY + static_cast<int>(d)));
                        // Past the last tile the columns hold anything; they are not used. (Branches
                        // between the FMAs cost more: one around three exchanges made prefill 514 us.)
                        if (!__all_sync(0xffffffffu, ready)) b.epilogue_wait(S::BAR_DFULL + static_cast<int>(d_next), turn_next);
                        tc_fence_after();
                        load_columns(lanes + d_next * kCols, v[0]);
                    }
#pragma unroll
                    for (int c = 0; c < kChunk; c += 4) {
                        constexpr int kEvery = kChunks * kChunk / 4 / (kSteps + 1) + 1;  // fours of columns between exchanges
                        const int four = (i * kChunk + c) / 4;
                        if (four % kEvery == 0 && four / kEvery < kSteps) exchange(four / kEvery);
                        fma_relu4(acc, w + i * kChunk + c, v[i & 1] + c);
                    }
                }
                sums[r] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
            }
            store();
            if constexpr (kHalves) {
                // The second half's sums, double-buffered: written again two tiles on, past the next barrier.
                float* half_s = token_s + (tau & 1) * kTile;
                if (set == 1) half_s[tk] = sums[0];
                named_bar_sync<kBarEpilogue, S::kEpiWarps * 32>();
                if (set == 0) sums[0] += half_s[tk];
            }
            held_at = pool_t;
#pragma unroll
            for (int r = 0; r < kRows; ++r) held[r] = scale == kNegInf ? kNegInf : sums[r] * scale;
            if (!in_lanes) {
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    if (r < mine && !(kHalves && set == 1)) token_s[(kHalves ? 2 : row_first + r) * kTile + tk] = held[r];
                named_bar_sync<kBarEpilogue, S::kEpiWarps * 32>();
                // Pools that do not lie in one warp's lanes. A warp takes one of more than 16 tokens
                // (of 64, 234 rows of 20 heads over 90 thousand tokens: 273 us, 404 with a thread
                // each), a thread one of fewer. (Read a tile later, with one barrier, they took
                // 1.5 % less, but the code beside the tile loop cost all others 1.5 % more.)
                const bool wide = p.kpool > 16;
                const int step = wide ? 32 : 1;
                for (int i = wide ? warp : threadIdx.x; i < x.rows * b.per_tile; i += S::kEpiWarps * 32 / step) {
                    const int r = static_cast<int>(divide(static_cast<uint32_t>(i), p.by_tile)), k = i - r * b.per_tile;
                    const int32_t pool = pool_t + k;
                    if (pool >= p.n_pools) continue;
                    float s = kNegInf;
                    if (pool < vis_s[r]) {
                        const float* from = token_s + (kHalves ? 2 : r) * kTile + k * p.kpool;
                        for (int j = wide ? lane : 0; j < p.kpool; j += step) s = max_nan(s, from[j]);
                        if (wide)
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1) s = max_nan(s, __shfl_xor_sync(0xffffffffu, s, o));
                    }
                    if (!wide || lane == 0) p.scores[static_cast<int64_t>(x.row0 + r) * p.n_pools + pool] = s;
                }
                named_bar_sync<kBarEpilogue, S::kEpiWarps * 32>();
            }
        }
        wait_columns(v[0]);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) exchange(k);
        store();
    });
}

template <int kHeads, int kCols>
__global__ void __launch_bounds__(Shape<kCols>::kThreads, Shape<kCols>::kCtas)
    pool_scores_kernel(const PoolScoresParams p, const __grid_constant__ CUtensorMap tmap, int32_t groups, int32_t group_rows, int32_t gap) {
    using S = Shape<kCols>;
    extern __shared__ uint8_t smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Block<kCols> b{p, smem, smem_u32(smem), reinterpret_cast<volatile int*>(smem + S::kOffAbort)};
    b.groups = groups;
    b.group_rows = group_rows;
    b.gap = gap;
    b.units = p.num_seqs * groups;
    b.per_tile = p.per_tile;
    if (tid == 0) {
        for (int e = 0; e < S::kStages; ++e) {
            // boxes: one arrival with the bytes to come; copies: every lane's, and a plain one per warp
            mbar_init(b.bar(S::BAR_FULL + e), p.box_rows > 0 ? 1 : kLoadWarps * 33);
            mbar_init(b.bar(S::BAR_EMPTY + e), 1);
        }
        for (int d = 0; d < S::kDBufs; ++d) {
            mbar_init(b.bar(S::BAR_DFULL + d), 2);  // the MMAs' commit, and the MMA warp passing on the scales
            mbar_init(b.bar(S::BAR_DEMPTY + d), S::kEpiWarps);
        }
        mbar_init(b.bar(S::BAR_QFULL), S::kEpiWarps);
        mbar_init(b.bar(S::BAR_QSEEN), S::kMmaWarps);
        mbar_init(b.bar(S::BAR_DRAIN), S::kMmaWarps);
        *b.abort_flag = 0;
        fence_mbar_init();
        if (p.box_rows > 0) prefetch_tmap(&tmap);
    }
    if (warp == S::kMmaWarp0) {
        tmem_alloc(b.sbase + S::kOffTmem, S::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    share(b);  // two block barriers
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + S::kOffTmem);
    if (warp < S::kEpiWarps) {
        run_epilogue<kHeads, kCols>(b, tmem);
    } else {
        if (warp < S::kLoadWarp0) run_mma<kHeads, kCols>(b, tmem);
        else if (p.box_rows == 0) run_load(b);
        else if (warp < S::kLoadWarp0 + S::kMmaWarps) run_load_boxes(b, &tmap);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == S::kMmaWarp0) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kTmemCols);
    }
}

// Runs f with the kernel of a padded head count and its columns.
template <int kHeads, typename F>
cudaError_t with_cols(int cols, F&& f) {
    if constexpr (kHeads <= 64)
        if (cols <= 64) return f(pool_scores_kernel<kHeads, 64>, Shape<64>{});
    return f(pool_scores_kernel<kHeads, 128>, Shape<128>{});
}
template <typename F>
cudaError_t with_kernel(int padded, int cols, F&& f) {
    switch (padded) {
        case 16: return with_cols<16>(cols, f);
        case 32: return with_cols<32>(cols, f);
        case 64: return with_cols<64>(cols, f);
        default: return with_cols<128>(cols, f);
    }
}

}  // namespace

cudaError_t pool_scores_kernel_setup() {
    for (int heads = 16; heads <= 128; heads *= 2)
        for (int cols = heads < 128 ? 64 : 128; cols <= 128; cols *= 2) {
            const cudaError_t e = with_kernel(heads, cols, [](auto* kernel, auto shape) {
                using S = decltype(shape);
                const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
                if (r != cudaSuccess) return r;
                return cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
            });
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

cudaError_t launch_pool_scores(const PoolScoresParams& p, const CUtensorMap& tmap, int sms, cudaStream_t stream) {
    // Heads are padded to 16, 32, 64 or 128 columns; a unit takes as many rows as its columns
    // hold, 128 when there are rows (or heads) enough: a key tile is then read from memory once
    // for all of them, and an MMA of N = 128 takes 64 cycles, one of N = 64 48 of which its
    // arithmetic fills 32.
    const int padded = p.heads <= 16 ? 16 : (p.heads <= 32 ? 32 : (p.heads <= 64 ? 64 : 128));
    const int64_t all = static_cast<int64_t>(p.rows_per_seq) * padded;
    const int cols = all <= 64 ? 64 : 128;
    const int32_t group_rows = cols / padded, groups = (p.rows_per_seq + group_rows - 1) / group_rows;
    return with_kernel(padded, cols, [&](auto* kernel, auto shape) {
        using S = decltype(shape);
        const int64_t ctas = static_cast<int64_t>(sms) * S::kCtas, unit_tiles = p.n_pools / p.per_tile + 1;
        const int32_t gap = static_cast<int64_t>(p.num_seqs) * groups >= 2 * ctas / unit_tiles ? kGap : 0;
        kernel<<<sms * S::kCtas, S::kThreads, S::kSmem, stream>>>(p, tmap, groups, group_rows, gap);
        return cudaGetLastError();
    });
}

}  // namespace dsa
