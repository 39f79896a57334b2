// Attention of each decode row over its whole paged latent cache (no selection):
//
//   out[r,h,:] = sum_{j < len(r)} softmax_j(sm_scale * q[r,h,:] . (k_scale*K_j)) (v_scale*V_j)
//
// One persistent CTA per SM over the line of 128-token tiles that the prologue planned (see
// full.cuh). Arithmetic as in the selected decode: keys and values are the cached E4M3 codes
// themselves, the operands of both products as they lie in the ring; a query is two E4M3
// terms (M = 128 query rows: 64 (row, head) pairs x {hi, lo}, in tensor memory); S[128 x 128
// tokens] goes to tensor memory, P' = 2^(x - m + kPBias) back to shared memory as two E4M3
// terms; O^T[512 x 64 pairs] accumulates in tensor memory in FP32, rescaled only when a
// pair's reference maximum m moves (kRescale* in common.cuh).
//
//   load     tiles into a ring of three, [16 groups of 8 tokens][4 blocks of 128 dims][8 tokens]
//            [128 bytes] with the 128-byte swizzle, each in four quarters of 32 tokens that are
//            refilled as soon as their P.V is done: two warps with tensor-map boxes of a page's
//            rows when pages and tiles fit each other, else four warps with 16-byte copies
//   MMA      one warp for Q.K^T, one for P.V
//   softmax  eight warps, two per TMEM lane quarter; the same warps write the output
//
// A tile that holds tokens which some row of the unit does not see ("edge" tile: the last
// ones, or those past a shorter row) is masked per pair, and its V bytes are made safe
// before P.V reads them: a hidden token's zero weight would not silence a NaN code. Tokens
// past every row are cleared, a partly visible token with a NaN code is cleared and its
// score made NaN for the pairs that see it.
//
// What bounds it is the tensor core with its operands from shared memory: a tile's Q.K^T takes 16
// MMAs of 64 cycles, its P.V 32 of 48 (N = 64 computes for 32, but reads 6 KB of operands), 2560
// cycles, and the softmax chain of a tile 2200 beside it; a tile takes some 2900. On long work
// the GPU runs at its power limit, at 1640 to 1790 MHz. Measured (plan and join included, in
// bursts): two contexts of 512 thousand tokens with 128 heads 200 us, 1350 TFLOP/s (each product
// counted once; 141 us at the rate of a BF16 product; 218 at the power limit); 64 rows of 64
// heads over 8 to 32 thousand tokens 134 us (143), 4.9 TB/s in all and 6 in the middle; 32
// sequences of four rows of 16 heads over 16384 tokens 68 us, 9 of them before the first scores
// and 10 after the first CTAs' last; one row over 777 tokens 16 us; 128 requests of 200 to 2048
// tokens 46 us, most of it unit changes. With K and V apart the ring holds one tile of both, and
// the ragged rows take 326 us. One warp issuing both products took 15 % more (10 % with V's tile
// kept in the collector for the second term of P'); sixteen softmax warps were slower too.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "full.cuh"
#include "ptx.cuh"

namespace dsa {
namespace full {
namespace {

constexpr int kTileBytes = kTile * kLatent;  // 64 KB
constexpr int kGroupBytes = 8 * kLatent;     // 8 tokens: four 1 KB swizzle atoms, one per 128 dims
constexpr int kRingTiles = 3;
// Quarters of a tile. A slot is held from its load until its P.V is done, and three slots over
// that time are the most tiles that pass: loading and releasing quarters takes three quarters
// of a P.V and most of the load's 64 KB out of it.
constexpr int kQuarters = 4;
constexpr int kQuarterTokens = kTile / kQuarters;  // 32: K of one MMA of P.V
constexpr int kQuarterBytes = kTileBytes / kQuarters;
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
constexpr int kHalfCols = kTile / 2;         // S columns per softmax warp
constexpr int kScores = kHalfCols / 2;       // scores per softmax thread: 32, one bit each of a word
constexpr int kPTermBytes = kHeadsPerCta * kTile;

constexpr int kBarSoftmax = 1;
constexpr int kBarPair0 = 2;  // 2..5: the two softmax warps of a lane quarter

constexpr int kOffP = kRingTiles * kTileBytes;               // P' [2 buffers][hi, lo]; epilogue staging
constexpr int kOffHm = kOffP + 4 * kPTermBytes;              // float [2 token halves][64] tile maxima; row sums at the end
constexpr int kOffAlpha = kOffHm + 2 * kHeadsPerCta * 4;     // float [2 tile parities][64] rescale factors; accounts in passing
constexpr int kOffF = kOffAlpha + 2 * kHeadsPerCta * 4;      // float [64] output factors; accounts in passing
constexpr int kOffFlags = kOffF + kHeadsPerCta * 4;          // u32 [2 tile parities][4 lane quarters]
constexpr int kOffBroken = kOffFlags + 2 * 4 * 4;            // 128 bits: an edge tile's tokens with a NaN code
constexpr int kOffBars = kOffBroken + kTile / 8;
enum {
    BAR_FULL0 = 0,                        // ring slot loaded
    BAR_EMPTY0 = BAR_FULL0 + kRingTiles,  // quarter of a ring slot free: its P.V is done
    BAR_SFULL = BAR_EMPTY0 + kRingTiles * kQuarters,  // S written
    BAR_SEMPTY,                           // S read
    BAR_PFULL0,                           // 2: P' buffer written
    BAR_PVDONE0 = BAR_PFULL0 + 2,         // 2: the P.V reading it is done
    BAR_QFULL = BAR_PVDONE0 + 2,
    BAR_QEMPTY,
    BAR_OEMPTY,
    BAR_DRAIN,
    BAR_DONE,
    kNumBars
};
constexpr int kOffTmem = kOffBars + kNumBars * 8;
constexpr int kOffAbort = kOffTmem + 4;
constexpr int kSmem = kOffAbort + 4 + 1024;  // slack for the 1024-byte alignment
static_assert(kSmem <= 227 * 1024, "shared memory");
static_assert(kSoftmaxWarps * 2048 <= 4 * kPTermBytes, "epilogue staging fits the P buffers");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0;    // O^T: dims 128c.. of all 64 pairs at column 64c
constexpr uint32_t kTmemQ = 256;  // query operand
constexpr uint32_t kTmemS = 384;

// A reference is this much above its tile's maximum. Each move costs the CTA about a
// microsecond (the pipeline drains): with normal scores of deviation 1, 8 of 106 tiles of 64
// pairs moved at the selected decode's 1 octave and moves of the asking pairs only (two contexts
// of 512 thousand tokens: 205 us, 199 with them). The lowest tile maximum that a reference serves,
// kRescaleDrop below it, is the same.
constexpr float kSlack = 2.0f;
// What the two E4M3 terms of a P' lose: 2^-10 at most (it itself when below), beside 1.2 * 2^-9 of
// it. The row sum takes P' whole, so a tile far below its pair's reference would be counted but not
// added: 128 terms of 2^-11 weigh 2^-4, as much as a 512th of a row whose sum is the 2^5 of one
// maximum. Each thread therefore keeps an account per pair, kLostShare (common.cuh) of its P'
// less what their terms may lose. While the four threads of a pair have one in credit together,
// less than kLostShare of the row is lost; a thread that sees its own run out asks, and a pair that
// could not pay for one more tile moves its reference down to that tile. (A tile that holds 2^5
// pays for itself: 2^5 * kLostShare = 128 * 2^-10.) Scores of deviation 1 never ask; of
// deviation 2 in natural units, 56 of 128 tiles of 64 pairs move a reference, 25 without it.
constexpr float kMostLost = kScores * 0x1p-10f;  // by a thread in a tile
constexpr float kNegInf = -__builtin_huge_valf();

// Warps of the two variants.
template <bool kTma>
struct Roles {
    static constexpr int kLoadWarps = kTma ? 2 : 4;
    static constexpr int kMmaWarp = kLoadWarps;  // Q.K^T; the next one P.V
    static constexpr int kSoftmax0 = kMmaWarp + 2;
    static constexpr int kThreads = (kSoftmax0 + kSoftmaxWarps) * 32;
};

// Box of whole 8-token groups of one page ([group][128-dim block][8 rows][128 bytes]).
__device__ __forceinline__ void tma_groups(uint32_t dst, const void* tmap, int32_t group, int32_t page, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], [%5];" ::
            "r"(dst), "l"(tmap), "r"(0), "r"(group), "r"(page), "r"(bar)
        : "memory");
}

// What every role of a CTA has in hand.
struct Cta {
    const Params& p;
    uint8_t* smem;
    uint32_t sbase, tmem;
    volatile int* abort_flag;
    CtaStart start;      // range and first segment

    __device__ uint32_t bar(int i) const { return sbase + kOffBars + 8 * i; }
    __device__ void fail(int code) const {
        report(p, code);
        *abort_flag = 1;
    }
    __device__ void wait(int b, uint32_t parity) const {
        if (!mbar_wait(bar(b), parity, abort_flag, p.wait_limit_ns)) fail(kStatusTimeout);
        __syncwarp();
    }
    // The stretch after s (not its last).
    __device__ Segment next(const Segment& s) const {
        const int32_t k = s.k + 1;
        return segment(start.begin, start.end, start.gap, blockIdx.x, false, k, p.plan.unit[k], p.plan.start[k], p.plan.max_len[k],
                       p.plan.min_len[k]);
    }
};

// Page of the block that holds position pos (negative: the caller reports it), and its row there.
__device__ __forceinline__ int32_t page_of(const Params& p, int32_t seq, int32_t pos, int32_t* row) {
    const int32_t blk = static_cast<int32_t>(divide(static_cast<uint32_t>(pos), p.by_block));
    *row = pos - blk * p.block_size;
    return __ldg(p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq + blk);
}

// ------------------------------------------------------------------------------------
// load: tensor-map boxes (warps 0 and 1, two quarters of every tile each: one warp's chain of
// waits and issues, some 2300 cycles a tile, would be what the ring waits for; lane l has box
// l of a tile, p.box_rows <= 32 tokens)
// ------------------------------------------------------------------------------------
__device__ void run_load_tma(const Cta& c, const CUtensorMap* kmap, const CUtensorMap* vmap) {
    const Params& p = c.p;
    const int lane = threadIdx.x & 31, q0 = 2 * (threadIdx.x >> 5);
    const int quarter = lane * p.box_rows / kQuarterTokens;  // kQuarters and up: no box
    const uint32_t box_bytes = static_cast<uint32_t>(p.box_rows) * kLatent;
    const int slots = p.kv_same ? kRingTiles : kRingTiles / 2;
    const uint32_t slot_bytes = p.kv_same ? kTileBytes : 2 * kTileBytes;
    uint32_t tau = 0;
    bool stop = false;
    for (Segment s = c.start.first; !stop; s = c.next(s)) {
        const int32_t seq = s.unit / p.groups;
        // This lane's page of tile t (requested a tile ahead), its first row there, and
        // whether any row of the unit sees the box.
        auto look = [&](int32_t t, int32_t* row, bool* live) {
            const int32_t pos = t * kTile + lane * p.box_rows;
            *live = (quarter == q0 || quarter == q0 + 1) && t < s.t1 && pos < s.max_len;
            return *live ? page_of(p, seq, pos, row) : -1;
        };
        int32_t row = 0, row_next = 0;
        bool live, live_next;
        int32_t page_next = look(s.t0, &row_next, &live_next);
        for (int32_t t = s.t0; t < s.t1 && !stop; ++t, ++tau) {
            const int32_t page = page_next;
            row = row_next;
            live = live_next;
            page_next = look(t + 1, &row_next, &live_next);
            if (live && page < 0) report(p, kStatusBounds);
            const int e = static_cast<int>(tau % slots);
            const uint32_t full = c.bar(BAR_FULL0 + e);
            const uint32_t lives = __ballot_sync(0xffffffffu, live);
#pragma unroll 1
            for (int j = q0; j < q0 + 2; ++j) {
                if (tau >= static_cast<uint32_t>(slots)) c.wait(BAR_EMPTY0 + e * kQuarters + j, (tau / slots - 1) & 1);
                // After a failed wait nothing more is issued (the drain below finds what is in flight).
                if (__shfl_sync(0xffffffffu, *c.abort_flag, 0)) {
                    stop = true;
                    break;
                }
                const uint32_t boxes = __popc(lives & __ballot_sync(0xffffffffu, quarter == j)) * (p.kv_same ? 1 : 2);
                if (lane == 0) mbar_arrive_expect_tx(full, boxes * box_bytes);
                __syncwarp();
                if (live && quarter == j) {  // a negative page lies outside the map: zeros
                    const uint32_t dst = c.sbase + e * slot_bytes + lane * box_bytes;
                    tma_groups(dst, kmap, row >> 3, page, full);
                    if (!p.kv_same) tma_groups(dst + kTileBytes, vmap, row >> 3, page, full);
                }
                __syncwarp();
            }
        }
        if (s.last) break;
    }
    // No copy into shared memory is in flight when the CTA exits: the last tiles' bytes (after
    // an abort a quarter may never have been asked for: its wait ends at the limit).
    if (lane == 0) {
        for (uint32_t i = tau > static_cast<uint32_t>(slots) ? tau - slots : 0; i < tau; ++i) {
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(c.bar(BAR_FULL0 + static_cast<int>(i % slots)), (i / slots) & 1) &&
                   globaltimer_ns() - t0 < kDrainLimitNs / (stop ? kRingTiles : 1)) {
            }
        }
    }
    __syncwarp();
}

// ------------------------------------------------------------------------------------
// load: 16-byte copies (warps 0-3, a quarter of a tile each; lane l resolves token l's page)
// ------------------------------------------------------------------------------------
__device__ void run_load_copies(const Cta& c) {
    const Params& p = c.p;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int slots = p.kv_same ? kRingTiles : kRingTiles / 2;
    const uint32_t slot_bytes = p.kv_same ? kTileBytes : 2 * kTileBytes;
    uint32_t tau = 0;
    for (Segment s = c.start.first;; s = c.next(s)) {
        const int32_t seq = s.unit / p.groups;
        // This lane's page and row there (-1: no token). What is made of them is left to the next
        // tile: using the page here would wait for its load.
        auto look = [&](int32_t t, int32_t* row) -> int32_t {
            const int32_t pos = t * kTile + kQuarterTokens * w + lane;
            *row = -1;
            return t < s.t1 && pos < s.max_len ? page_of(p, seq, pos, row) : 0;
        };
        int32_t row_next, page_next = look(s.t0, &row_next);
        for (int32_t t = s.t0; t < s.t1; ++t, ++tau) {
            const int32_t page = page_next, row = row_next;
            page_next = look(t + 1, &row_next);
            if (page < 0) report(p, kStatusBounds);
            const int64_t mine = page < 0 || row < 0 ? -1 : page * p.cache_stride + static_cast<int64_t>(row) * kLatent;
            const int e = static_cast<int>(tau % slots);
            if (tau >= static_cast<uint32_t>(slots)) c.wait(BAR_EMPTY0 + e * kQuarters + w, (tau / slots - 1) & 1);
            const uint32_t dst = c.sbase + e * slot_bytes + w * kQuarterBytes + (lane >> 3) * 1024;
#pragma unroll 8
            for (int j = 0; j < kQuarterTokens; ++j) {
                const int64_t at = __shfl_sync(0xffffffffu, mine, j);
                const uint32_t d = dst + (j >> 3) * kGroupBytes + (j & 7) * 128 + (((lane & 7) ^ (j & 7)) << 4);
                const uint64_t src = at >= 0 ? static_cast<uint64_t>(at) + lane * 16 : 0;
                cp_async_16_zfill(d, p.k_cache + src, at >= 0 ? 16u : 0u);
                if (!p.kv_same) cp_async_16_zfill(d + kTileBytes, p.v_cache + src, at >= 0 ? 16u : 0u);
            }
            cp_async_arrive_noinc(c.bar(BAR_FULL0 + e));
        }
        if (s.last) break;
    }
    cp_async_wait_all();
}

// ------------------------------------------------------------------------------------
// MMA warps, one for Q.K^T and one for P.V (converged, one elected lane issues). The issue of
// an MMA blocks while the tensor core's queue is full, so one warp for both products left the
// core idle during its waits, fences and commits, some 800 of 3350 cycles a tile.
// ------------------------------------------------------------------------------------
__device__ void run_qk(const Cta& c) {
    const Params& p = c.p;
    const int slots = p.kv_same ? kRingTiles : kRingTiles / 2;
    const uint32_t slot_bytes = p.kv_same ? kTileBytes : 2 * kTileBytes;
    const uint32_t idesc = idesc_e4m3(128, kTile, false, false);
    const uint32_t el = elect_one();
    uint32_t tau = 0, units = 0;
    for (Segment s = c.start.first;; s = c.next(s)) {
        c.wait(BAR_QFULL, units++ & 1);
        for (int32_t t = s.t0; t < s.t1; ++t, ++tau) {
            c.wait(BAR_FULL0 + static_cast<int>(tau % slots), (tau / slots) & 1);
            if (tau > 0) c.wait(BAR_SEMPTY, (tau - 1) & 1);
            fence_proxy_async_smem();
            tc_fence_after();
            const uint64_t kdesc = smem_desc(c.sbase + static_cast<uint32_t>(tau % slots) * slot_bytes, 16, kGroupBytes, kSwizzle128B);
            const uint32_t d = c.tmem + kTmemS;
            mma_e4m3_ta_el(d, c.tmem + kTmemQ, kdesc, idesc, 0u, el);
#pragma unroll
            for (int ks = 1; ks < 16; ++ks)
                mma_e4m3_ta_acc_el(d, c.tmem + kTmemQ + ks * 8,
                                   kdesc + static_cast<uint64_t>(((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), idesc, el);
            tc_commit_el(c.bar(BAR_SFULL), el);
            if (t == s.t1 - 1) tc_commit_el(c.bar(BAR_QEMPTY), el);
        }
        if (s.last) break;
    }
    tc_commit_el(c.bar(BAR_DRAIN), el);
}

__device__ void run_pv(const Cta& c) {
    const Params& p = c.p;
    const int slots = p.kv_same ? kRingTiles : kRingTiles / 2;
    const uint32_t slot_bytes = p.kv_same ? kTileBytes : 2 * kTileBytes;
    const uint32_t idesc = idesc_e4m3(128, kHeadsPerCta, true, false);
    const uint32_t el = elect_one();
    const uint64_t pdesc0 = smem_desc(c.sbase + kOffP, 1024, 128, kSwizzleNone);
    uint32_t tau = 0, units = 0;
    for (Segment s = c.start.first;; s = c.next(s), ++units) {
        for (int32_t t = s.t0; t < s.t1; ++t, ++tau) {
            const int pb = tau & 1, e = static_cast<int>(tau % slots);
            c.wait(BAR_PFULL0 + pb, (tau >> 1) & 1);
            if (t == s.t0 && units > 0) c.wait(BAR_OEMPTY, (units - 1) & 1);
            tc_fence_after();
            // V^T: 128 dims of block mc x the 32 tokens of a quarter (four 8-token swizzle groups),
            // MN-major. P'^T: 64 pairs x 32 tokens, K-major core matrices.
            const uint64_t vdesc = smem_desc(c.sbase + e * slot_bytes + (p.kv_same ? 0u : kTileBytes), 1024, kGroupBytes, kSwizzle128B);
            const uint64_t pdesc = pdesc0 + static_cast<uint64_t>((pb * 2 * kPTermBytes) >> 4);
#pragma unroll
            for (int j = 0; j < kQuarters; ++j) {
                const uint64_t bh = pdesc + static_cast<uint64_t>((j * 2048) >> 4);
                const uint64_t bl = pdesc + static_cast<uint64_t>((kPTermBytes + j * 2048) >> 4);
#pragma unroll
                for (int mc = 0; mc < 4; ++mc) {
                    const uint64_t a = vdesc + static_cast<uint64_t>((j * kQuarterBytes + mc * 1024) >> 4);
                    const uint32_t d = c.tmem + kTmemO + mc * 64;
                    if (j == 0) mma_e4m3_el(d, a, bh, idesc, t == s.t0 ? 0u : 1u, el);
                    else mma_e4m3_acc_el(d, a, bh, idesc, el);
                    mma_e4m3_acc_el(d, a, bl, idesc, el);
                }
                if (j == kQuarters - 1) tc_commit_el(c.bar(BAR_PVDONE0 + pb), el);
                tc_commit_el(c.bar(BAR_EMPTY0 + e * kQuarters + j), el);
            }
        }
        if (s.last) break;
    }
    tc_commit_el(c.bar(BAR_DRAIN), el);
}

// ------------------------------------------------------------------------------------
// softmax / output warps
// ------------------------------------------------------------------------------------
// Two probabilities as two E4M3 terms each (hi: rounded to nearest; lo: what is left of the
// float16 value, whose own rounding of 2^-12 is far below lo's 2^-9 of P'; kMostLost has what small
// ones lose). Through float16 pairs this takes five instructions where single floats take eight.
__device__ __forceinline__ void split2(float p0, float p1, uint32_t& hi, uint32_t& lo) {
    uint16_t h, l;
    asm("{\n\t.reg .b32 v, r, d;\n\t"
        "cvt.rn.f16x2.f32 v, %3, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 %0, v;\n\t"
        "cvt.rn.f16x2.e4m3x2 r, %0;\n\t"
        "sub.rn.f16x2 d, v, r;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 %1, d;\n\t}"
        : "=&h"(h), "=h"(l)
        : "f"(p0), "f"(p1));
    hi = h;
    lo = l;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Makes one token's V bytes of an edge tile safe; returns whether it held a NaN code. Lanes
// l and l + 16 share a token, 256 bytes each.
__device__ __forceinline__ bool clean_token(uint8_t* v_tile, int token, int part, bool hidden) {
    uint4* at[16];
    uint32_t nan = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        // blocks 2*part and 2*part + 1 of 128 dims, all eight 16-byte pieces of the token's row
        at[i] = reinterpret_cast<uint4*>(v_tile + (token >> 3) * kGroupBytes + (2 * part + (i >> 3)) * 1024 + (token & 7) * 128 +
                                         (i & 7) * 16);
        if (!hidden) {
            const uint4 v = *at[i];
            nan |= ((v.x & 0x7F7F7F7Fu) + 0x01010101u) | ((v.y & 0x7F7F7F7Fu) + 0x01010101u) |
                   ((v.z & 0x7F7F7F7Fu) + 0x01010101u) | ((v.w & 0x7F7F7F7Fu) + 0x01010101u);
        }
    }
    const bool broken = ((nan | __shfl_xor_sync(0xffffffffu, nan, 16)) & 0x80808080u) != 0u;
    if (hidden || broken)
#pragma unroll
        for (int i = 0; i < 16; ++i) *at[i] = make_uint4(0, 0, 0, 0);
    return broken;
}

// A warp's 32 dims x 32 pairs block (dims on lanes) scaled and written to bf16 rows through
// the warp's 2 KB staging area with 16-byte stores.
__device__ __forceinline__ void store_block(__nv_bfloat16* rows, int h0, int hvalid, int dim0, const uint32_t* v, const float* f,
                                            uint8_t* stage, int lane) {
    __nv_bfloat16* stg = reinterpret_cast<__nv_bfloat16*>(stage);  // [32 pairs][32 dims]
#pragma unroll
    for (int k = 0; k < 32; ++k) stg[k * 32 + lane] = __float2bfloat16_rn(__uint_as_float(v[k]) * f[k]);
    __syncwarp();
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
        const int hk = pass * 8 + lane / 4, col = (lane % 4) * 8;
        const uint4 val = *reinterpret_cast<const uint4*>(stg + hk * 32 + col);
        if (h0 + hk < hvalid) *reinterpret_cast<uint4*>(rows + static_cast<int64_t>(h0 + hk) * kLatent + dim0 + col) = val;
    }
    __syncwarp();
}

template <bool kTma>
__device__ void run_softmax(const Cta& c) {
    const Params& p = c.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sw = warp - Roles<kTma>::kSoftmax0;  // 0..7
    const int q4 = warp & 3;                       // TMEM lane quarter
    const int half = sw >> 2;                      // token half of each tile
    const int term = lane & 1;                     // 0: hi row, 1: lo row
    const int hq = 16 * q4 + (lane >> 1);          // pair of this thread within the unit
    float* hm_s = reinterpret_cast<float*>(c.smem + kOffHm);
    float* alpha_s = reinterpret_cast<float*>(c.smem + kOffAlpha);
    float* f_s = reinterpret_cast<float*>(c.smem + kOffF);
    uint32_t* flag_s = reinterpret_cast<uint32_t*>(c.smem + kOffFlags);
    uint16_t* broken_s = reinterpret_cast<uint16_t*>(c.smem + kOffBroken);
    uint8_t* stage = c.smem + kOffP + sw * 2048;
    const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
    // This thread's first 16-byte row in a P' term: K-major core matrices of 8 pairs x 16 tokens.
    const uint32_t p_off = (((half * kHalfCols + term * kScores) / 16) * 8 + (hq >> 3)) * 128 + (hq & 7) * 16;
    const int slots = p.kv_same ? kRingTiles : kRingTiles / 2;
    const uint32_t slot_bytes = p.kv_same ? kTileBytes : 2 * kTileBytes;
    uint32_t tau = 0;
    int units = 0;

    auto load_q = [&](int32_t unit) {
        const uint4* src = reinterpret_cast<const uint4*>(p.qimg + static_cast<int64_t>(unit) * kQImageBytes + half * 16 * 2048 +
                                                          (q4 * 32 + lane) * 16);
        uint32_t a[2][32];
#pragma unroll
        for (int hc = 0; hc < 2; ++hc)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 v = src[(hc * 8 + i) * (2048 / 16)];
                a[hc][4 * i] = v.x;
                a[hc][4 * i + 1] = v.y;
                a[hc][4 * i + 2] = v.z;
                a[hc][4 * i + 3] = v.w;
            }
#pragma unroll
        for (int hc = 0; hc < 2; ++hc) tmem_st_x32(c.tmem + lane_base + kTmemQ + half * 64 + hc * 32, a[hc]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(c.bar(BAR_QFULL));
    };
    // Length that this thread's pair sees.
    auto pair_len = [&](int32_t unit) -> int32_t {
        const int32_t pair = (unit % p.groups) * kHeadsPerCta + hq;
        bool over;
        return pair < p.pairs ? row_len(p, unit / p.groups, pair / p.heads, &over) : 0;
    };

    // What turns its dots into log2 scores. A broken query's is NaN, which would also reach the
    // -inf of hidden tokens: a pair that sees none (a padding row) takes 1 and stays at zero.
    auto pair_scale = [&](int32_t unit, int32_t len) {
        const float given = p.qscale[static_cast<int64_t>(unit) * kHeadsPerCta + hq];  // beside the length's load
        return len > 0 ? given : 1.0f;
    };

    Segment next = c.start.first;
    int32_t len_next = pair_len(next.unit);
    float c_next = pair_scale(next.unit, len_next);
    bool q_loaded = false;  // the unit's query operand was loaded during the unit before
    bool pv_seen = false;   // the P.V two tiles back was already waited for
    for (;;) {
        const Segment s = next;
        const float qs = c_next;
        const int32_t len = len_next;
        if (!s.last) {
            next = c.next(s);
            len_next = pair_len(next.unit);
            c_next = pair_scale(next.unit, len_next);
        }
        if (!q_loaded) {
            if (units > 0) c.wait(BAR_QEMPTY, (units - 1) & 1);
            load_q(s.unit);
        }
        q_loaded = false;
        float m_ref = kNegInf;  // reference max of the pair (log2 units)
        float m_top = kNegInf;  // highest reference so far
        float l_part = 0.0f;    // this thread's share of the sum of P'
        float credit = 0.0f;    // and its account of what the terms may have lost of it

        for (int32_t t = s.t0; t < s.t1; ++t, ++tau) {
            c.wait(BAR_SFULL, tau & 1);
            tc_fence_after();
            uint32_t v[kHalfCols];
            tmem_ld_x64(c.tmem + lane_base + kTmemS + half * kHalfCols, v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar(BAR_SEMPTY));

            // Dots of pair hq with tokens tok0 .. tok0+31 of the tile: this lane's term plus the
            // neighbouring lane's other one; the score in log2 units is qs (> 0) times that.
            const int tok0 = half * kHalfCols + term * kScores;
            float x[kScores];
#pragma unroll
            for (int j = 0; j < kScores; ++j) {
                const float send = __uint_as_float(term ? v[j] : v[kScores + j]);
                const float mine = __uint_as_float(term ? v[kScores + j] : v[j]);
                x[j] = mine + __shfl_xor_sync(0xffffffffu, send, 1);
            }
            if ((t + 1) * kTile > s.min_len) {  // an edge tile
                uint8_t* v_tile = c.smem + static_cast<uint32_t>(tau % slots) * slot_bytes + (p.kv_same ? 0 : kTileBytes);
                const int token = 16 * sw + (lane & 15);
                const int32_t pos = t * kTile + token;
                bool broken = false;
                c.wait(BAR_FULL0 + static_cast<int>(tau % slots), (tau / slots) & 1);  // passed: the copied bytes
                if (__any_sync(0xffffffffu, pos >= s.min_len))
                    broken = clean_token(v_tile, token, lane >> 4, pos >= s.max_len) && pos < s.max_len;
                const uint32_t bits = __ballot_sync(0xffffffffu, broken);
                if (lane == 0) broken_s[sw] = static_cast<uint16_t>(bits);
                named_bar_sync<kBarSoftmax, kSoftmaxThreads>();
                const int32_t lim = len - t * kTile;
                const uint32_t nan = reinterpret_cast<const uint32_t*>(broken_s)[tok0 / kScores];
#pragma unroll
                for (int j = 0; j < kScores; ++j) {
                    if (tok0 + j >= lim) x[j] = kNegInf;
                    else if (nan >> j & 1u) x[j] = __uint_as_float(0x7FC00000u);
                }
            }
            float hm4[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
            for (int j = 0; j < kScores; j += 2) hm4[(j >> 1) & 3] = max3(hm4[(j >> 1) & 3], x[j], x[j + 1]);
            float hmax = fmaxf(fmaxf(hm4[0], hm4[1]), fmaxf(hm4[2], hm4[3]));
            hmax = fmaxf(hmax, __shfl_xor_sync(0xffffffffu, hmax, 1)) * qs;
            // A tile mostly leaves every pair's reference where it is, so P' is formed with it at
            // once (but for a unit's first tile, which finds none); one barrier then tells whether
            // any half of any pair's scores asks for a move (the maximum exceeds the reference by
            // more than the margin, or lies far below it, or the account runs out). Only then the
            // halves are compared, references move and P' is formed again.
            const bool ask = hmax > m_ref + kRescaleMargin ||
                             (hmax < m_ref - kRescaleDrop && m_ref > m_top - kRescaleFloor && hmax != kNegInf);
            uint32_t hw[kScores / 4], lw[kScores / 4];
            float fresh, earned = 0.0f;
            bool resc[2] = {false, false};
            const float* alpha_t = alpha_s + (tau & 1) * kHeadsPerCta;
#pragma unroll 1
            for (bool again = false;; again = true) {
                if (again || t > s.t0) {
                    float ls4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    const float off = m_ref == kNegInf ? 0.0f : kPBias - m_ref;  // nothing seen so far: every x is -inf
#pragma unroll
                    for (int g = 0; g < kScores / 4; ++g) {
                        float pp[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            pp[e] = ex2_approx(fmaf(x[4 * g + e], qs, off));
                            ls4[e] += pp[e];
                        }
                        uint32_t h0, l0, h1, l1;
                        split2(pp[0], pp[1], h0, l0);
                        split2(pp[2], pp[3], h1, l1);
                        hw[g] = h0 | h1 << 16;
                        lw[g] = l0 | l1 << 16;
                    }
                    fresh = (ls4[0] + ls4[1]) + (ls4[2] + ls4[3]);
                    earned = fmaf(fresh, kLostShare, -fminf(fresh, kMostLost));
                    if (again || !named_bar_any<kBarSoftmax, kSoftmaxThreads>(
                                     ask || (credit + earned < 0.0f && m_ref > m_top - kRescaleFloor)))
                        break;
                }
                // The halves' accounts go through words that are free here: the output factors,
                // and the rescale factors of the tile before, which every warp has applied.
                float* const credit_s = alpha_s + ((tau + 1) & 1) * kHeadsPerCta;
                const float credit2 = credit + earned + __shfl_xor_sync(0xffffffffu, credit + earned, 1);
                if (term == 0) {
                    hm_s[half * kHeadsPerCta + hq] = hmax;
                    (half == 0 ? f_s : credit_s)[hq] = credit2;
                }
                named_bar_sync_id(kBarPair0 + q4, 64);
                const float tm = fmaxf(hm_s[hq], hm_s[kHeadsPerCta + hq]);
                const float credit4 = f_s[hq] + credit_s[hq];
                // The move is paid for once any pair needs it: every pair whose reference rises with
                // this tile takes its new one too, and seldom asks for a move of its own.
                const bool rise = tm + kSlack > m_ref;
                const bool change = rise || ((tm < m_ref - kRescaleDrop || (tm < m_ref - kSlack && credit4 < 4.0f * kMostLost)) &&
                                             m_ref > m_top - kRescaleFloor && tm != kNegInf);
                float alpha = 1.0f;
                if (change) {
                    const float m_new = fmaxf(tm + (rise ? kSlack : kRescaleSlack), m_top - kRescaleFloor);
                    alpha = m_ref == kNegInf ? 0.0f : ex2_approx(m_ref - m_new);
                    l_part *= alpha;
                    credit *= alpha;
                    m_ref = m_new;
                    m_top = fmaxf(m_top, m_new);
                } else {
                    credit = fmaf(0.25f, credit4, -earned);  // in equal parts: who asked gets what the others do not need
                }
                if (term == 0 && half == 0) alpha_s[(tau & 1) * kHeadsPerCta + hq] = alpha;
                const uint32_t changed = __ballot_sync(0xffffffffu, change);
                if (half == 0 && lane == 0) flag_s[(tau & 1) * 4 + q4] = changed;
                // Also keeps the next tile's maxima from overwriting these.
                const bool any_change = named_bar_any<kBarSoftmax, kSoftmaxThreads>(change);
                if (!any_change && t > s.t0) break;
                if (t > s.t0) {
                    const uint4 f = *reinterpret_cast<const uint4*>(flag_s + (tau & 1) * 4);
                    resc[0] = (f.x | f.y) != 0u;
                    resc[1] = (f.z | f.w) != 0u;
                }
            }
            l_part += fresh;
            credit += earned;
            if (tau >= 2 && !pv_seen) c.wait(BAR_PVDONE0 + (tau & 1), ((tau >> 1) - 1) & 1);
            pv_seen = false;
            const uint32_t pb = c.sbase + kOffP + (tau & 1) * 2 * kPTermBytes;
#pragma unroll
            for (int i = 0; i < kScores / 16; ++i) {
                st_shared_v4(pb + p_off + i * 1024, hw[4 * i], hw[4 * i + 1], hw[4 * i + 2], hw[4 * i + 3]);
                st_shared_v4(pb + kPTermBytes + p_off + i * 1024, lw[4 * i], lw[4 * i + 1], lw[4 * i + 2], lw[4 * i + 3]);
            }
            fence_proxy_async_smem();
            if (resc[0] || resc[1]) {
                // After the P.V before this tile, and before this tile's (P-full below): the
                // changed 32-pair blocks of this warp's two dim chunks.
                c.wait(BAR_PVDONE0 + ((tau - 1) & 1), ((tau - 1) >> 1) & 1);
                pv_seen = true;
                tc_fence_after();
#pragma unroll 1
                for (int hh = 0; hh < 2; ++hh) {
                    if (!resc[hh]) continue;
                    const uint32_t ta = c.tmem + lane_base + kTmemO + 2 * half * 64 + hh * 32;
                    uint32_t o0[32], o1[32];
                    tmem_ld_2x32(ta, ta + 64, o0, o1);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float f = alpha_t[hh * 32 + i];
                        o0[i] = __float_as_uint(__uint_as_float(o0[i]) * f);
                        o1[i] = __float_as_uint(__uint_as_float(o1[i]) * f);
                    }
                    tmem_st_x32(ta, o0);
                    tmem_st_x32(ta + 64, o1);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar(BAR_PFULL0 + (tau & 1)));
        }

        // The next unit's query operand goes in while this unit's last P.V runs.
        if (!s.last) {
            c.wait(BAR_QEMPTY, units & 1);
            load_q(next.unit);
            q_loaded = true;
        }

        // ---- output of the unit ----
        c.wait(BAR_PVDONE0 + ((tau - 1) & 1), ((tau - 1) >> 1) & 1);
        pv_seen = true;
        tc_fence_after();
        const float lpair = l_part + __shfl_xor_sync(0xffffffffu, l_part, 1);
        if (term == 0) hm_s[half * kHeadsPerCta + hq] = lpair;
        named_bar_sync<kBarSoftmax, kSoftmaxThreads>();
        const bool whole = s.part < 0;
        if (term == 0 && half == 0) {
            const float l = hm_s[hq] + hm_s[kHeadsPerCta + hq];
            f_s[hq] = l == 0.0f ? 0.0f : (whole ? p.v_scale : 1.0f) / l;  // nothing seen: zero; NaN stays
            if (!whole) p.part_lse[s.part * kHeadsPerCta + hq] = l == 0.0f ? kNegInf : m_ref + __log2f(l);
        }
        named_bar_sync<kBarSoftmax, kSoftmaxThreads>();
        const int32_t seq = s.unit / p.groups, first = (s.unit % p.groups) * kHeadsPerCta;
        const int hvalid = min(kHeadsPerCta, p.pairs - first);
        const int64_t pair0 = static_cast<int64_t>(seq) * p.pairs + first;
#pragma unroll 1
        for (int mc2 = 0; mc2 < 2; ++mc2) {
            const int mc = 2 * half + mc2;
            const int dim0 = mc * 128 + q4 * 32;
            uint32_t v64[64];
            tmem_ld_x64(c.tmem + lane_base + kTmemO + mc * 64, v64);
            if (whole) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
                    store_block(reinterpret_cast<__nv_bfloat16*>(p.out) + pair0 * kLatent, hh * 32, hvalid, dim0, v64 + hh * 32,
                                f_s + hh * 32, stage, lane);
            } else {
                __half* part = reinterpret_cast<__half*>(p.part_o) + static_cast<int64_t>(s.part) * kHeadsPerCta * kLatent;
#pragma unroll
                for (int i = 0; i < kHeadsPerCta; i += 8) {
                    uint32_t h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __half2 hv = __floats2half2_rn(__uint_as_float(v64[i + 2 * e]) * f_s[i + 2 * e],
                                                             __uint_as_float(v64[i + 2 * e + 1]) * f_s[i + 2 * e + 1]);
                        h[e] = *reinterpret_cast<const uint32_t*>(&hv);
                    }
                    *reinterpret_cast<uint4*>(part + ((static_cast<int64_t>(dim0 / 32) * 8 + i / 8) * 32 + lane) * 8) =
                        make_uint4(h[0], h[1], h[2], h[3]);
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(c.bar(BAR_OEMPTY));
        // The staging area is the P buffer; hm_s and f_s are used again.
        named_bar_sync<kBarSoftmax, kSoftmaxThreads>();
        ++units;
        if (s.last) break;
    }
}

template <bool kTma>
__global__ void __launch_bounds__(Roles<kTma>::kThreads, 1)
    full_kernel(const Params p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using R = Roles<kTma>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Cta c{p, smem, smem_u32(smem), 0u, reinterpret_cast<volatile int*>(smem + kOffAbort)};

    if (tid == 0) {
        // boxes: one arrival per quarter, with the bytes to come; copies: one per lane
        for (int e = 0; e < kRingTiles; ++e) mbar_init(c.bar(BAR_FULL0 + e), kTma ? kQuarters : 32 * R::kLoadWarps);
        for (int e = 0; e < kRingTiles * kQuarters; ++e) mbar_init(c.bar(BAR_EMPTY0 + e), 1);
        mbar_init(c.bar(BAR_SFULL), 1);
        mbar_init(c.bar(BAR_SEMPTY), kSoftmaxWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(c.bar(BAR_PFULL0 + i), kSoftmaxWarps);
            mbar_init(c.bar(BAR_PVDONE0 + i), 1);
        }
        mbar_init(c.bar(BAR_QFULL), kSoftmaxWarps);
        mbar_init(c.bar(BAR_QEMPTY), 1);
        mbar_init(c.bar(BAR_OEMPTY), kSoftmaxWarps);
        mbar_init(c.bar(BAR_DRAIN), 2);
        mbar_init(c.bar(BAR_DONE), kSoftmaxWarps);
        *c.abort_flag = 0;
        fence_mbar_init();
        if (kTma) {
            prefetch_tmap(&kmap);
            if (!p.kv_same) prefetch_tmap(&vmap);
        }
    }
    if (warp == R::kMmaWarp) {
        tmem_alloc(c.sbase + kOffTmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    c.tmem = *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem);
    // Everything above overlaps the prologue; its plan is read only after this.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    c.start = p.plan.cta[blockIdx.x];
    if (c.start.begin < c.start.end) {
        if (warp < R::kLoadWarps) {
            if constexpr (kTma) run_load_tma(c, &kmap, &vmap);
            else run_load_copies(c);
        } else if (warp < R::kSoftmax0) {
            if (warp == R::kMmaWarp) run_qk(c);
            else run_pv(c);
            // Until every MMA has completed and the softmax warps have read tensor memory.
            uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(c.bar(BAR_DRAIN), 0) && globaltimer_ns() - t0 < kDrainLimitNs) {
            }
            t0 = globaltimer_ns();
            while (!mbar_try_wait(c.bar(BAR_DONE), 0) && globaltimer_ns() - t0 < kDrainLimitNs) {
            }
            __syncwarp();
        } else {
            run_softmax<kTma>(c);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar(BAR_DONE));
        }
    }
    tc_fence_before();
    __syncthreads();
    // The join's blocks, let in while others compute, would take issue slots from them.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == R::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(c.tmem, kTmemCols);
    }
}

template <bool kTma>
cudaError_t setup() {
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, full_kernel<kTma>);
    if (e != cudaSuccess) return e;
    if (attr.maxThreadsPerBlock < Roles<kTma>::kThreads) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(full_kernel<kTma>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(full_kernel<kTma>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
}

}  // namespace
}  // namespace full

cudaError_t full_setup() {
    const cudaError_t e = full::setup<true>();
    return e != cudaSuccess ? e : full::setup<false>();
}

cudaError_t launch_full(const full::Params& p, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.max_ctas);
    cfg.blockDim = dim3(p.box_rows > 0 ? full::Roles<true>::kThreads : full::Roles<false>::kThreads);
    cfg.dynamicSmemBytes = full::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return p.box_rows > 0 ? cudaLaunchKernelEx(&cfg, full::full_kernel<true>, p, kmap, vmap)
                          : cudaLaunchKernelEx(&cfg, full::full_kernel<false>, p, kmap, vmap);
}

}  // namespace dsa
