// Attention of packed prompt chunks over their paged latent caches: row t, the i-th new token of
// request s, sees the positions below base[s] + i + 1.
//
//   out[t,h,:] = sum_{j < base[s]+i+1} softmax_j(sm_scale * q[t,h,:] . (k_scale*K_j)) (v_scale*V_j)
//
// A cluster of two CTAs works on one unit of 128 (row, head) pairs at a time (see prefill.cuh), and
// both products are MMAs of the pair of SMs (cta_group::2). Arithmetic as in the full decode: the
// cached E4M3 codes are the operands, a query is two E4M3 terms, P' = 2^(x - m + kPBias) two more.
//
//   S[256 query rows x 128 tokens] = Q K^T   each CTA holds the rows of its 64 pairs x {hi, lo} in
//       tensor memory and brings 64 of the tile's tokens, all dims
//   O^T[512 dims x 128 pairs] += V^T P'^T    each CTA accumulates 256 dims of all 128 pairs, brings
//       those dims of the tile's tokens and the P' of its 64 pairs
//
// so that a CTA softmaxes its own pairs and no probability leaves it, while the second product has
// N = 128 (full.cu: 64): 6 KB of operands for 64 cycles of arithmetic, not for 32.
//
//   warp 0, 1    load K tiles into a ring of two and V tiles into one of four ([16 groups of 8
//                tokens][blocks of 128 dims][8 tokens][128 bytes], 128-byte swizzle): tensor-map
//                boxes of a page's rows when pages and tiles fit each other, else 16-byte copies
//   warp 2, 3    issue Q K^T and P V (rank 0); tell rank 0 of the loaded K tiles (rank 1)
//   warps 4-11   softmax, two per TMEM lane quarter; after a unit's last tile they put the next
//                unit's query operand in place
//   warps 12-15  make the next unit's query operand, rescale O when a reference moves, write a unit's
//                output
//
// Bound by the tensor pipe, and on long calls by the power that it may take: Q K^T counts twice for
// the two query terms and P V twice for those of P', 4 x 128 x 128 x 512 multiply-adds of E4M3 per
// unit and tile. 1024 rows of 64 heads after 31.7k cached tokens (4.5 TFLOP of bf16 arithmetic):
// 2.28 ms in short bursts, 1960 TFLOP/s (a bf16 matrix product of the library: 1924), 2.54 in a long
// loop, at the power limit, 1760 (1725); one prompt of 4096 rows, 732 us, 1500; 512 rows over 4096
// tokens, 168 us, 1530. There a change of unit is what is lost: some 7000 cycles between products
// with V, where tiles follow at 2500. (9500 with the operand put in place by warps 12-15 once the last
// product is issued; by them, earlier, on an event of its own: 3 % more on short units, for one
// wait more.) Every instruction less in the softmax also saves power, and so time on long calls.
// Short units are bound by the fetching of instructions: sixteen warps run nine programs, so loops
// stay rolled and warps that do the same run the same code.
//
// Measured beside this split: three K and three V slots, 1 to 4 % more (a value tile is held until
// its softmax is done, a key tile is not); the queries by four warps of their own, at 96 registers
// a thread instead of 128, 4 % more on long units and on short ones; O's dims as the outer
// loop of P V, with either half let go early, 10 %; the next tile's scores read ahead, 5 %
// (the registers); softmax loops with any test more, 2 to 7 %.
//
// A reference that moves in one CTA rescales columns of O in both. The CTA that asks writes the
// factors into both; the warp that issues P V finds its mark before the tile's product, has
// warps 12-15 of both CTAs rescale, and goes on. Tiles that no pair asks in pay nothing for it.
//
// A tile that holds tokens which some row of the unit does not see is masked per pair, and its V
// bytes are made safe before P V reads them: a hidden token's zero weight would not silence a NaN
// code. Tokens past every row are cleared; of one that only later rows see the NaN codes are cleared,
// and the warps that write the unit's output put a NaN into their dims of the rows that see it.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "prefill.cuh"
#include "ptx.cuh"
#include "softmax.cuh"

namespace dsa {
namespace prefill {
namespace {

constexpr int kCtaPairs = kPairs / 2;
constexpr int kKeySlots = 2, kValueSlots = 4;       // of the rings
constexpr int kKeyTokens = kTile / 2;               // tokens of a tile that a CTA brings as keys
constexpr int kDims = kLatent / 2;                  // dims that it brings as values
constexpr int kSlotBytes = kKeyTokens * kLatent;    // 32 KB
static_assert(kSlotBytes == kTile * kDims, "both halves of a tile");
constexpr int kKGroup = 8 * kLatent;                // bytes of 8 tokens
constexpr int kVGroup = 8 * kDims;
constexpr int kSoftmax0 = 4, kSoftmaxWarps = 8;
constexpr int kEpilogue0 = 12, kEpilogueWarps = 4;
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
constexpr int kThreads = (kEpilogue0 + kEpilogueWarps) * 32;
constexpr int kHalfCols = kTile / 2;                // S columns per softmax warp
static_assert(kScores == kHalfCols / 2, "scores per softmax thread: 32, one bit each of a word");
constexpr int kPTermBytes = kCtaPairs * kTile;

constexpr int kBarSoftmax = 1;
constexpr int kBarPair0 = 2;  // 2..5: the two softmax warps of a lane quarter
constexpr int kBarFirst = 6;  // the first unit's query operand is made

constexpr int kOffV = kKeySlots * kSlotBytes;
constexpr int kOffP = (kKeySlots + kValueSlots) * kSlotBytes;  // P' [2 buffers][hi, lo]
constexpr int kOffHm = kOffP + 4 * kPTermBytes;              // float2 [2 token halves][64] tile maximum, account; row sums at the end
constexpr int kOffAlpha = kOffHm + 2 * kCtaPairs * 8;        // float [2 tile parities][128] rescale factors, of both CTAs
constexpr int kOffF = kOffAlpha + 2 * kPairs * 4;            // float [128] output factors, of both CTAs
constexpr int kOffScale = kOffF + kPairs * 4;                // u8 [2 unit parities][64] exponents of the queries' scales
constexpr int kOffFlags = kOffScale + 2 * kCtaPairs;         // u32 [2 tile parities][2 CTAs][4 lane quarters] tile that moved a reference
// u32 [3 units in turn][4] tokens from the unit's shortest row on with a NaN code. (Not two in turn: an
// epilogue warp may be at the next unit but one's when another still writes the output. One unit
// further it is not, as P V waits for that output.)
constexpr int kOffBroken = kOffFlags + 2 * 2 * 4 * 4;
static_assert(kOffBroken % 16 == 0, "read as one piece");
constexpr int kOffEvent = kOffBroken + 3 * 4 * 4;            // u32: a tile's number + 1 to rescale before, 0: the unit is done
constexpr int kOffProgress = kOffEvent + 4;                  // u32: key tiles asked for
constexpr int kOffSent = kOffProgress + 4;                   // u32 [2] units whose factors this CTA sent, events that it sent
constexpr int kOffTmem = kOffSent + 2 * 4;
constexpr int kOffAbort = kOffTmem + 4;
constexpr int kOffBars = (kOffAbort + 4 + 7) / 8 * 8;
// (both): in either CTA; (0): in rank 0, both CTAs arrive.
enum {
    BAR_KFULL0 = 0,                          // own half of a K slot loaded
    BAR_VFULL0 = BAR_KFULL0 + kKeySlots,     // own half of a V slot loaded
    BAR_KPEER0 = BAR_VFULL0 + kValueSlots,   // (0) rank 1's half of a K slot loaded
    BAR_KEMPTY0 = BAR_KPEER0 + kKeySlots,    // (both) its Q K^T is done
    BAR_VEMPTY0 = BAR_KEMPTY0 + kKeySlots,   // (both) its P V is done
    BAR_PFULL0 = BAR_VEMPTY0 + kValueSlots,  // (0) 2: P' buffers written, V there
    BAR_PVDONE0 = BAR_PFULL0 + 2,            // (both) 2: the P V reading it is done
    BAR_SFULL = BAR_PVDONE0 + 2,             // (both) S written
    BAR_SEMPTY,                              // (0) S read
    BAR_QFULL,                               // (0) query operands in place
    BAR_QEMPTY,                              // (both) the unit's last Q K^T is done
    BAR_QMADE0,                              // 2: query operand made, by the unit's parity
    BAR_EVENT = BAR_QMADE0 + 2,              // (both) something for the epilogue warps
    BAR_OFREE,                               // (0) they did it
    BAR_FFULL,                               // (both) output factors written
    BAR_FEMPTY,                              // (both) and used
    BAR_UDONE0,                              // 2: the softmax warps are done with a unit (by its parity)
    BAR_DRAIN = BAR_UDONE0 + 2,              // (both) every MMA is done
    kNumBars
};
constexpr int kSmem = kOffBars + kNumBars * 8;
static_assert(kSmem <= 227 * 1024, "shared memory");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0;    // O^T: dims 128c.. of this CTA's 256, all pairs, at column 128c
constexpr uint32_t kTmemQ = 256;  // query operand
constexpr uint32_t kTmemS = 384;
constexpr float kSlack = 2.0f;  // a reference above its tile's maximum, as in the full decode: a move stops both products
constexpr float kNegInf = -__builtin_huge_valf();

// A cluster's stretch of one unit.
struct Segment {
    int32_t k, t0, t1;  // unit's number, tiles of it
    int32_t part;       // partial slot, -1: the whole unit
    int32_t max_len, min_len;
    bool last;
    Unit u;
};

// What every role of a CTA has in hand.
struct Cta {
    const Params& p;
    uint8_t* smem;
    uint32_t sbase, rank, cluster;
    volatile int* abort_flag;
    uint32_t tmem;
    int64_t begin, end;
    int32_t gap;

    __device__ uint32_t bar(int i) const { return sbase + kOffBars + 8 * i; }
    __device__ void fail(int code) const {
        report(p, code);
        *abort_flag = 1;
        st_cluster(map_rank(sbase + kOffAbort, rank ^ 1u), 1u);
    }
    __device__ void wait(int b, uint32_t parity) const {
        if (!mbar_wait(bar(b), parity, abort_flag, p.wait_limit_ns)) fail(kStatusTimeout);
        __syncwarp();
    }
    __device__ volatile uint32_t* progress() const { return reinterpret_cast<volatile uint32_t*>(smem + kOffProgress); }
    __device__ volatile uint32_t* sent() const { return reinterpret_cast<volatile uint32_t*>(smem + kOffSent); }
    // As wait, for what may take longer than a wait is allowed (a unit of very many tiles): the limit
    // runs anew while tiles come in.
    __device__ void wait_long(int b, uint32_t parity) const {
        for (uint32_t seen = ~0u; *progress() != seen && !*abort_flag;) {
            seen = *progress();
            if (mbar_wait(bar(b), parity, abort_flag, p.wait_limit_ns) || p.wait_limit_ns < kPollHintNs) break;
        }
        wait(b, parity);
    }
    // Says nothing of shared memory that the other CTA's threads have written (fence_cluster).
    __device__ void arrive(int b, uint32_t to) const { mbar_arrive_cluster(map_rank(bar(b), to)); }

    __device__ Segment segment(int32_t k, const Unit& u, bool first) const {
        Segment s;
        s.u = u;
        s.k = k;
        s.max_len = pair_len(p, u.base, u.first + u.valid - 1);
        s.min_len = pair_len(p, u.base, u.first);
        const int64_t e = u.start + (s.max_len + kTile - 1) / kTile;
        s.t0 = static_cast<int32_t>((begin > u.start ? begin : u.start) - u.start);
        s.t1 = static_cast<int32_t>((end < e ? end : e) - u.start);
        s.part = begin <= u.start && e <= end ? -1 : 2 * static_cast<int32_t>(cluster) + (first ? 0 : 1);
        s.last = e + gap >= end;
        return s;
    }
};

// A role's way through its cluster's units; records are brought into L1 a unit or more ahead.
struct Walk {
    const Cta& c;
    Segment s;
    __device__ explicit Walk(const Cta& cta) : c(cta) {
        const Start& st = c.p.starts[c.cluster];
        s = c.segment(st.k, st.unit, true);
        prefetch();
    }
    __device__ void advance() {
        s = c.segment(s.k + 1, c.p.units[s.k + 1], false);
        prefetch();
    }
    __device__ void prefetch() const { asm volatile("prefetch.global.L1 [%0];" ::"l"(c.p.units + s.k + 1)); }
};

// Page of the block that holds position pos (negative: the caller reports it), and its row there.
__device__ __forceinline__ int32_t page_of(const Params& p, int32_t seq, int32_t pos, int32_t* row) {
    const int32_t blk = static_cast<int32_t>(divide(static_cast<uint32_t>(pos), p.by_block));
    *row = pos - blk * p.block_size;
    return __ldg(p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq + blk);
}

// Box of whole 8-token groups of one page, from 128-byte block `block` on.
__device__ __forceinline__ void tma_groups(uint32_t dst, const void* tmap, int32_t block, int32_t group, int32_t page, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4, %5}], [%6];" ::
            "r"(dst), "l"(tmap), "r"(0), "r"(block), "r"(group), "r"(page), "r"(bar)
        : "memory");
}

// ------------------------------------------------------------------------------------
// load: warp 0 keys (64 tokens of a tile), warp 1 values (256 dims)
// ------------------------------------------------------------------------------------
template <bool kValues>
__device__ void run_load_tma(const Cta& c, const CUtensorMap* tmap) {
    constexpr int kTokens = kValues ? kTile : kKeyTokens;
    constexpr int kFull = kValues ? BAR_VFULL0 : BAR_KFULL0, kEmpty = kValues ? BAR_VEMPTY0 : BAR_KEMPTY0;
    constexpr int kSlots = kValues ? kValueSlots : kKeySlots;
    const Params& p = c.p;
    const int lane = threadIdx.x & 31;
    const uint32_t box_bytes = static_cast<uint32_t>(p.box_rows) * (kValues ? kDims : kLatent);
    const uint32_t ring = c.sbase + (kValues ? kOffV : 0);
    const int32_t block = kValues ? static_cast<int32_t>(c.rank) * (kDims / 128) : 0;
    const int32_t pos0 = lane * p.box_rows + (kValues ? 0 : static_cast<int32_t>(c.rank) * kKeyTokens);
    const bool have = lane * p.box_rows < kTokens;  // a box of this lane's in every tile
    uint32_t tau = 0;
    bool stop = false;
    for (Walk w(c); !stop; w.advance()) {
        const Segment& s = w.s;
        // This lane's page of tile t (requested a tile ahead), its first row there, and whether any
        // row of the unit sees the box.
        auto look = [&](int32_t t, int32_t* row, bool* live) {
            const int32_t pos = t * kTile + pos0;
            *live = have && t < s.t1 && pos < s.max_len;
            return *live ? page_of(p, s.u.seq, pos, row) : -1;
        };
        int32_t row_next = 0;
        bool live_next;
        int32_t page_next = look(s.t0, &row_next, &live_next);
        for (int32_t t = s.t0; t < s.t1; ++t, ++tau) {
            const int32_t page = page_next, row = row_next;
            const bool live = live_next;
            page_next = look(t + 1, &row_next, &live_next);
            if (live && page < 0) report(p, kStatusBounds);
            const int e = static_cast<int>(tau % kSlots);
            if (tau >= kSlots) c.wait(kEmpty + e, (tau / kSlots - 1) & 1);
            if (!kValues && lane == 0) *c.progress() = tau;
            // After a failed wait nothing more is issued (the drain below finds what is in flight).
            if (__any_sync(0xffffffffu, *c.abort_flag != 0)) {
                stop = true;
                break;
            }
            const uint32_t full = c.bar(kFull + e), boxes = __popc(__ballot_sync(0xffffffffu, live));
            if (lane == 0) mbar_arrive_expect_tx(full, boxes * box_bytes);
            __syncwarp();
            if (live) tma_groups(ring + e * kSlotBytes + lane * box_bytes, tmap, block, row >> 3, page, full);  // a negative page lies outside the map: zeros
            __syncwarp();
        }
        if (s.last) break;
    }
    // No copy into shared memory is in flight when the CTA exits.
    if (lane == 0) {
        for (uint32_t i = tau > kSlots ? tau - kSlots : 0; i < tau; ++i) {
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(c.bar(kFull + static_cast<int>(i % kSlots)), (i / kSlots) & 1) && globaltimer_ns() - t0 < kDrainLimitNs) {
            }
        }
    }
    __syncwarp();
}

// The same by 16-byte copies: an instruction brings 128 bytes of each of four rows. Both warps run one
// code, for what they bring of a tile has one shape: four half rows of 256 bytes for each lane to
// look up, of two tokens' keys or of four tokens' values. (2000 rows of 20 heads over pages of 100
// tokens 113 us; when it took 134, a code each took 165, and more the more it was unrolled: the
// instruction cache holds the softmax as well. Boxes, where a page takes them: 107 to 112.)
__device__ void run_load_copies(const Cta& c, bool values) {
    constexpr int kEach = 4;
    const Params& p = c.p;
    const int lane = threadIdx.x & 31, sub = lane >> 3, piece = lane & 7;
    const int keys = values ? 0 : 1;
    const uint32_t slots = values ? kValueSlots : kKeySlots, group = values ? kVGroup : kKGroup;
    const int full = values ? BAR_VFULL0 : BAR_KFULL0, empty = values ? BAR_VEMPTY0 : BAR_KEMPTY0;
    const uint8_t* cache = values ? p.v_cache + c.rank * kDims : p.k_cache;
    const uint32_t ring = c.sbase + (values ? kOffV : 0) + sub * 128 + ((piece ^ sub) << 4);
    const int32_t pos0 = lane + (values ? 0 : static_cast<int32_t>(c.rank) * kKeyTokens);
    uint32_t e = 0, round = 0, tau = 0;
    for (Walk w(c);; w.advance()) {
        const Segment& s = w.s;
        int32_t row_next[kEach], page_next[kEach];
        // Pages and rows there (row -1: no token). What is made of them is left to the next tile:
        // using a page here would wait for its load.
        auto look = [&](int32_t t) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int32_t pos = t * kTile + pos0 + 32 * (i >> keys);
                row_next[i] = -1;
                page_next[i] = t < s.t1 && pos < s.max_len ? page_of(p, s.u.seq, pos, &row_next[i]) : 0;
            }
        };
        look(s.t0);
        for (int32_t t = s.t0; t < s.t1; ++t, ++tau) {
            const uint8_t* mine[kEach];
            uint32_t live[kEach];  // lanes whose token there is
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                if (page_next[i] < 0) report(p, kStatusBounds);
                const bool there = page_next[i] >= 0 && row_next[i] >= 0;
                live[i] = __ballot_sync(0xffffffffu, there) >> sub;
                mine[i] = cache;
                if (there) mine[i] += page_next[i] * p.cache_stride + static_cast<int64_t>(row_next[i]) * kLatent + (i & keys) * 256;
            }
            look(t + 1);
            if (round > 0) c.wait(empty + e, (round - 1) & 1);
            if (!values && lane == 0) *c.progress() = tau;
            const uint32_t slot = ring + e * kSlotBytes;
#pragma unroll 2
            for (int j = 0; j < 32; j += 4) {
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    // Rows j and j + 4 of an 8-row group in turn.
                    const uint32_t dst = slot + 4 * (i >> keys) * group + (i & keys) * 2048;
                    const auto half = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine[i]), j + sub);
                    const uint8_t* src = reinterpret_cast<const uint8_t*>(half) + piece * 16;
                    const uint32_t size = (live[i] >> j & 1u) * 16u;
                    const uint32_t d = (dst + (j >> 3) * group + (j & 4) * 128) ^ ((j & 4) << 4);
                    cp_async_16_zfill(d, src, size);
                    cp_async_16_zfill(d + 1024, src + 128, size);
                }
            }
            cp_async_arrive_noinc(c.bar(full + e));
            if (++e == slots) e = 0, ++round;
        }
        if (s.last) break;
    }
    cp_async_wait_all();
}

// ------------------------------------------------------------------------------------
// MMA warps of rank 0 (converged, one elected lane issues)
// ------------------------------------------------------------------------------------
__device__ void run_qk(const Cta& c) {
    constexpr int kSlots = kKeySlots;
    const uint32_t idesc = idesc_e4m3(256, kTile, false, false);
    const uint32_t el = elect_one();
    uint32_t tau = 0, units = 0;
    for (Walk w(c);; w.advance()) {
        const Segment& s = w.s;
        c.wait(BAR_QFULL, units++ & 1);
        for (int32_t t = s.t0; t < s.t1; ++t, ++tau) {
            const int e = static_cast<int>(tau % kSlots);
            c.wait(BAR_KFULL0 + e, (tau / kSlots) & 1);
            c.wait(BAR_KPEER0 + e, (tau / kSlots) & 1);
            if (tau > 0) c.wait(BAR_SEMPTY, (tau - 1) & 1);
            fence_proxy_async_smem();
            tc_fence_after();
            const uint64_t kdesc = smem_desc(c.sbase + e * kSlotBytes, 16, kKGroup, kSwizzle128B);
            const uint32_t d = c.tmem + kTmemS;
#pragma unroll
            for (int ks = 0; ks < 16; ++ks)
                mma_pair_ts_el(d, c.tmem + kTmemQ + ks * 8, kdesc + static_cast<uint64_t>(((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), idesc,
                               ks > 0 ? 1u : 0u, el);
            commit_both_el(c.bar(BAR_SFULL), el);
            commit_both_el(c.bar(BAR_KEMPTY0 + e), el);
            if (t == s.t1 - 1) commit_both_el(c.bar(BAR_QEMPTY), el);
        }
        if (s.last) break;
    }
    commit_both_el(c.bar(BAR_DRAIN), el);
}

// Returns the events that were sent.
__device__ uint32_t run_pv(const Cta& c) {
    constexpr int kSlots = kValueSlots;
    const int lane = threadIdx.x & 31;
    const uint32_t idesc = idesc_e4m3(256, kPairs, true, false);
    const uint32_t el = elect_one();
    const uint64_t pdesc0 = smem_desc(c.sbase + kOffP, 1024, 128, kSwizzleNone);
    const volatile uint32_t* flags = reinterpret_cast<const volatile uint32_t*>(c.smem + kOffFlags);
    uint32_t tau = 0, events = 0, sent = 0;
    // Has the epilogue warps of both CTAs do what `event` says.
    auto post = [&](uint32_t event) {
        ++events;
        if (__any_sync(0xffffffffu, *c.abort_flag != 0)) return;  // nobody waits for one event before the next then
        ++sent;
        if (lane < 2) {
            const uint32_t bar = map_rank(c.bar(BAR_EVENT), lane);
            mbar_arrive_expect_cluster(bar, 4);
            st_async(map_rank(c.sbase + kOffEvent, lane), event, bar);
        }
        __syncwarp();
    };
    for (Walk w(c);; w.advance()) {
        const Segment& s = w.s;
        for (int32_t t = s.t0; t < s.t1; ++t, ++tau) {
            const int pb = tau & 1, e = static_cast<int>(tau % kSlots);
            c.wait(BAR_PFULL0 + pb, (tau >> 1) & 1);
            fence_acquire_shared_cluster();  // the other CTA's marks and factors: a wait alone acquires from this CTA only
            if (t == s.t0) {
                if (events > 0) c.wait(BAR_OFREE, (events - 1) & 1);  // the unit before has been read
            } else if (__any_sync(0xffffffffu, flags[pb * 8 + (lane & 7)] == tau + 1)) {
                post(tau + 1);
                c.wait(BAR_OFREE, (events - 1) & 1);
            }
            fence_proxy_async_smem();
            tc_fence_after();
            // V^T: 128 dims of block mc x 32 tokens (four 8-token swizzle groups), MN-major.
            // P'^T: 64 pairs of each CTA x 32 tokens, K-major core matrices.
            const uint64_t vdesc = smem_desc(c.sbase + kOffV + e * kSlotBytes, 1024, kVGroup, kSwizzle128B);
            const uint64_t pdesc = pdesc0 + static_cast<uint64_t>((pb * 2 * kPTermBytes) >> 4);
// (Rolled: 1 to 3 % less than four copies of the code.)
#pragma unroll 1
            for (int j = 0; j < kTile / 32; ++j) {
                const uint64_t bh = pdesc + static_cast<uint64_t>((j * 2048) >> 4);
                const uint64_t bl = pdesc + static_cast<uint64_t>((kPTermBytes + j * 2048) >> 4);
#pragma unroll
                for (int mc = 0; mc < kDims / 128; ++mc) {
                    const uint64_t a = vdesc + static_cast<uint64_t>((j * 4 * kVGroup + mc * 1024) >> 4);
                    const uint32_t d = c.tmem + kTmemO + mc * kPairs;
                    mma_pair_ss_el(d, a, bh, idesc, j > 0 || t > s.t0 ? 1u : 0u, el);
                    mma_pair_ss_el(d, a, bl, idesc, 1u, el);
                }
            }
            commit_both_el(c.bar(BAR_PVDONE0 + pb), el);
            commit_both_el(c.bar(BAR_VEMPTY0 + e), el);
        }
        post(0);
        if (s.last) break;
    }
    commit_both_el(c.bar(BAR_DRAIN), el);
    return sent;
}

// Rank 1: its half of each K slot, to rank 0.
__device__ void run_forward(const Cta& c) {
    constexpr int kSlots = kKeySlots;
    const int lane = threadIdx.x & 31;
    uint32_t tau = 0;
    for (Walk w(c);; w.advance()) {
        const Segment& s = w.s;
        for (int32_t t = s.t0; t < s.t1; ++t, ++tau) {
            const int e = static_cast<int>(tau % kSlots);
            c.wait(BAR_KFULL0 + e, (tau / kSlots) & 1);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) c.arrive(BAR_KPEER0 + e, 0);
        }
        if (s.last) break;
    }
}

// ------------------------------------------------------------------------------------
// softmax warps
// ------------------------------------------------------------------------------------
__device__ __forceinline__ uint8_t* query_image(const Cta& c, int parity) {
    return c.p.qimg + (static_cast<int64_t>(blockIdx.x) * 2 + parity) * kQImageBytes;
}
// Half of a lane quarter of unit number `units`' query operand into tensor memory, once it is made and
// the unit before has no more use for the place.
__device__ __forceinline__ void place_query(const Cta& c, uint32_t units, int half) {
    const int lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3;
    const uint32_t place = c.tmem + (static_cast<uint32_t>(q4 * 32) << 16) + kTmemQ + half * 64;
    const int row = 2 * (16 * q4 + (lane & 15)) + (lane >> 4);  // 16 pairs' hi rows, then their lo rows
    const uint4* src = reinterpret_cast<const uint4*>(query_image(c, units & 1) + half * (16 * 2048) + row * 16);
    c.wait(BAR_QMADE0 + (units & 1), (units >> 1) & 1);
    if (units > 0) c.wait(BAR_QEMPTY, (units - 1) & 1);
    tc_fence_after();
    uint32_t a[2][32];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint4 v = __ldcg(src + i * (2048 / 16));
        a[i >> 3][4 * (i & 7)] = v.x;
        a[i >> 3][4 * (i & 7) + 1] = v.y;
        a[i >> 3][4 * (i & 7) + 2] = v.z;
        a[i >> 3][4 * (i & 7) + 3] = v.w;
    }
    tmem_st_x32(place, a[0]);
    tmem_st_x32(place + 32, a[1]);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) c.arrive(BAR_QFULL, 0);
}

__device__ __forceinline__ uint32_t* broken_of(const Cta& c, uint32_t units) {
    return reinterpret_cast<uint32_t*>(c.smem + kOffBroken) + units % 3 * 4;
}
// Bytes that are NaN codes: 128; and the word with zeros for them.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t without_nan(uint32_t w) { return w & ~((nan_codes(w) >> 7) * 0xFFu); }

// Returns the units whose factors were sent.
__device__ uint32_t run_softmax(const Cta& c) {
    constexpr int kSlots = kValueSlots;
    const Params& p = c.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sw = warp - kSoftmax0;               // 0..7
    const int q4 = warp & 3;                       // TMEM lane quarter
    const int half = sw >> 2;                      // token half of each tile
    const int side = lane >> 4;                    // half of those tokens
    const int hq = 16 * q4 + (lane & 15);          // pair of this thread within the CTA
    const int pair = static_cast<int>(c.rank) * kCtaPairs + hq;  // and within the unit
    float2* hm_s = reinterpret_cast<float2*>(c.smem + kOffHm);
    const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
    // This thread's first 16-byte row in a P' term: K-major core matrices of 8 pairs x 16 tokens.
    const uint32_t p_off = (((half * kHalfCols + side * kScores) / 16) * 8 + (hq >> 3)) * 128 + (hq & 7) * 16;
    uint32_t tau = 0, units = 0;
    bool pv_seen = false;  // the P.V two tiles back was already waited for

    const int32_t k0 = p.starts[c.cluster].k;
    place_query(c, 0, half);
    for (;; ++units) {
        // The tile loop keeps few of the unit's numbers (registers are short here); what else it needs,
        // seldom, it takes from the record again, which stays in L1.
        auto unit = [&] { return c.segment(k0 + units, p.units[k0 + units], units == 0); };
        auto seen_by = [&](const Segment& s) { return pair < s.u.valid ? pair_len(p, s.u.base, s.u.first + pair) : 0; };
        int32_t t, t1, edge;  // tiles; the first with tokens that some row does not see
        bool none;            // the pair sees nothing
        {
            const Segment s = unit();
            t = s.t0;
            t1 = s.t1;
            edge = s.min_len / kTile;
            none = seen_by(s) == 0;
            asm volatile("prefetch.global.L1 [%0];" ::"l"(p.units + k0 + units + 1));
        }
        bool first = true;      // tile of the unit here
        float qs = 0.0f;        // what turns dots into log2 scores, known with the first tile
        float m_ref = kNegInf;  // reference max of the pair (log2 units)
        float m_top = kNegInf;  // highest reference so far
        float l_part = 0.0f;    // this thread's share of the sum of P'
        float credit = 0.0f;    // and its account of what the terms may have lost of it

        for (; t < t1; ++t, ++tau, first = false) {
            c.wait(BAR_SFULL, tau & 1);
            tc_fence_after();
            // Dots of pair hq with tokens tok0 .. tok0+31 of the tile: the hi term's row plus the lo
            // term's, 16 lanes further on, both in this thread by the load's own shape. (By 32-lane loads
            // of neighbouring rows and an exchange between their threads 7 % more, on calls at the power
            // limit too.) The score in log2 units is qs (> 0) times that.
            const int tok0 = half * kHalfCols + side * kScores;
            float x[kScores];
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                uint32_t a[16], b[16];
                const uint32_t at = c.tmem + lane_base + kTmemS + half * kHalfCols + 16 * part;
                tmem_ld_halves_2x16(at, at + (16u << 16), a, b);
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float2 r = add_two({__uint_as_float(a[j]), __uint_as_float(a[j + 1])}, {__uint_as_float(b[j]), __uint_as_float(b[j + 1])});
                    x[16 * part + j] = r.x;
                    x[16 * part + j + 1] = r.y;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) c.arrive(BAR_SEMPTY, 0);
            if (first) {
                // A broken query's scale is NaN, which would also reach the -inf of hidden tokens: a
                // pair that sees none (behind the unit's last) takes 1 and stays at zero.
                const uint32_t e = c.smem[kOffScale + (units & 1) * kCtaPairs + hq];
                qs = e == 255 || p.score_scale != p.score_scale ? __uint_as_float(0x7FC00000u)
                                                                : fmaxf(fabsf(p.score_scale) * __uint_as_float(e << 23), 0x1p-120f);
                if (none) qs = 1.0f;
            }
            const int v_slot = static_cast<int>(tau % kSlots);
            if (t >= edge) {
                const Segment s = unit();
                uint8_t* v_tile = c.smem + kOffV + v_slot * kSlotBytes;
                const uint32_t* broken = broken_of(c, units);
                // 32 of those marks from position pos on.
                auto marks = [&](int32_t pos) -> uint32_t {
                    const int32_t i = pos - s.min_len;
                    if (i <= -32 || i >= kPairs) return 0;
                    const uint32_t lo = i >= 0 ? broken[i >> 5] : 0, hi = i < kPairs - 32 ? broken[(i + 32) >> 5] : 0;
                    return __funnelshift_r(lo, hi, i & 31);
                };
                // The warp's sixteen tokens: 256 of their dims are here, 8 lanes to 128 of them.
                const int32_t pos0 = t * kTile + 16 * sw;
                const uint32_t past = pos0 + 16 <= s.max_len ? 0u : ~0u << max(s.max_len - pos0, 0), nan = marks(pos0);
                if (((past | nan) & 0xFFFFu) != 0u) {
                    c.wait(BAR_VFULL0 + v_slot, (tau / kSlots) & 1);
// (Unrolled: 250 requests of up to 8 rows 123 -> 128.5 us.)
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        const int token = (4 * i + (lane >> 3)) & 15, block = i >> 2;
                        uint4* at = reinterpret_cast<uint4*>(v_tile + ((16 * sw + token) >> 3) * kVGroup + block * 1024 + (token & 7) * 128 +
                                                             (lane & 7) * 16);
                        if (past >> token & 1u) {
                            *at = make_uint4(0, 0, 0, 0);
                        } else if (nan >> token & 1u) {
                            const uint4 v = *at;
                            *at = make_uint4(without_nan(v.x), without_nan(v.y), without_nan(v.z), without_nan(v.w));
                        }
                    }
                }
                const int32_t lim = seen_by(s) - t * kTile - tok0;  // this thread's scores before it are seen
                const uint32_t hidden = lim >= 32 ? 0u : lim <= 0 ? ~0u : ~0u << lim;
#pragma unroll
                for (int j = 0; j < kScores; ++j) x[j] = hidden >> j & 1u ? kNegInf : x[j];
            }
            float hm4[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
            for (int j = 0; j < kScores; j += 2) hm4[(j >> 1) & 3] = max3(hm4[(j >> 1) & 3], x[j], x[j + 1]);
            float hmax = fmaxf(fmaxf(hm4[0], hm4[1]), fmaxf(hm4[2], hm4[3]));
            hmax = fmaxf(hmax, __shfl_xor_sync(0xffffffffu, hmax, 16)) * qs;
            // As in the full decode: P' is formed with the reference as it is (but for a unit's first
            // tile), one barrier tells whether any half of any pair's scores asks for a move, and
            // only then the halves are compared, references move and P' is formed again. A tile far
            // below its reference asks when the account runs out, not before: the last tile of a unit
            // often holds few tokens that are seen.
            const bool ask = hmax > m_ref + kRescaleMargin;
            uint32_t hw[kScores / 4], lw[kScores / 4];
            float fresh, earned = 0.0f;
#pragma unroll 1
            for (bool again = false;; again = true) {
                if (again || !first) {
                    float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
                    const float off = m_ref == kNegInf ? 0.0f : kPBias - m_ref;  // nothing seen so far: every x is -inf
#pragma unroll
                    for (int g = 0; g < kScores / 4; ++g) {
                        uint32_t h[2], l[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 y = fma_two({x[4 * g + 2 * e], x[4 * g + 2 * e + 1]}, {qs, qs}, {off, off});
                            const float2 pp = {ex2_approx(y.x), ex2_approx(y.y)};
                            sum[e] = add_two(sum[e], pp);
                            split2(pp.x, pp.y, h[e], l[e]);
                        }
                        hw[g] = h[0] | h[1] << 16;
                        lw[g] = l[0] | l[1] << 16;
                    }
                    fresh = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    earned = fmaf(fresh, kLostShare, -fminf(fresh, kMostLost));
                    if (again || !named_bar_any<kBarSoftmax, kSoftmaxThreads>(
                                     ask || (credit + earned < 0.0f && m_ref > m_top - kRescaleFloor)))
                        break;
                }
                const float credit2 = credit + earned + __shfl_xor_sync(0xffffffffu, credit + earned, 16);
                if (side == 0) hm_s[half * kCtaPairs + hq] = make_float2(hmax, credit2);
                named_bar_sync_id(kBarPair0 + q4, 64);
                const float2 h0 = hm_s[hq], h1 = hm_s[kCtaPairs + hq];
                const float tm = fmaxf(h0.x, h1.x), credit4 = h0.y + h1.y;
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
                if (!first && half == 0) {
                    // Factors and the tile's mark into both CTAs (the words' last readers were done
                    // before the P.V two tiles back).
                    if (tau >= 2 && !pv_seen) c.wait(BAR_PVDONE0 + (tau & 1), ((tau >> 1) - 1) & 1);
                    pv_seen = true;
                    const uint32_t changed = __ballot_sync(0xffffffffu, change);
                    const uint32_t to = map_rank(c.sbase, side);  // a lane of each pair per CTA
                    st_cluster(to + kOffAlpha + ((tau & 1) * kPairs + pair) * 4, __float_as_uint(alpha));
                    if ((lane & 15) == 0 && changed != 0u)
                        st_cluster(to + kOffFlags + (((tau & 1) * 2 + c.rank) * 4 + q4) * 4, tau + 1);
                    __syncwarp();
                    fence_cluster();  // of all lanes' words, by the lane that arrives
                }
                // Also keeps the next tile's maxima from overwriting these.
                if (!named_bar_any<kBarSoftmax, kSoftmaxThreads>(change) && !first) break;
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
            c.wait(BAR_VFULL0 + v_slot, (tau / kSlots) & 1);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) c.arrive(BAR_PFULL0 + (tau & 1), 0);
        }

        const Segment s = unit();
        if (!s.last) place_query(c, units + 1, half);  // while the last P.V runs

        // ---- the unit's output factors, to both CTAs ----
        const float lpair = l_part + __shfl_xor_sync(0xffffffffu, l_part, 16);
        if (side == 0) hm_s[half * kCtaPairs + hq].x = lpair;
        if (half == 0 && units > 0) c.wait(BAR_FEMPTY, (units - 1) & 1);
        // All eight warps end together, and send nothing before what they sent last has been used.
        if (named_bar_any<kBarSoftmax, kSoftmaxThreads>(*c.abort_flag != 0)) return units;
        if (half == 0) {
            const float l = hm_s[hq].x + hm_s[kCtaPairs + hq].x;
            const bool whole = s.part < 0;
            const float f = l == 0.0f ? 0.0f : (whole ? p.v_scale : 1.0f) / l;  // nothing seen: zero; NaN stays
            if (sw == 0 && lane == 0) mbar_arrive_expect_tx(c.bar(BAR_FFULL), kPairs * 4);
            st_async(map_rank(c.sbase, side) + kOffF + pair * 4, __float_as_uint(f), map_rank(c.bar(BAR_FFULL), side));
            if (!whole && side == 0) p.part_lse[s.part * kPairs + pair] = l == 0.0f ? kNegInf : m_ref + __log2f(l);
        }
        if (lane == 0) mbar_arrive(c.bar(BAR_UDONE0 + (units & 1)));
        named_bar_sync<kBarSoftmax, kSoftmaxThreads>();  // the sums are read
        if (s.last) return units + 1;
    }
}

// After an aborted call, when both CTAs have ended: what they sent and nobody waited for has arrived here.
// A CTA sends neither an event nor a unit's factors before the last were used, so that each barrier has
// one phase open at most, and the CTAs' factors are one unit apart at most: what a barrier was told to
// expect and what comes are then brought into line.
// (Out of line: at the kernel's end, which every call runs through, its code took 0.2 us.)
__device__ __noinline__ void receive_rest(uint32_t sbase, uint32_t rank) {
    auto count = [&](int i, uint32_t of) { return ld_cluster(map_rank(sbase + kOffSent + 4 * i, of)); };
    auto bar = [&](int b) { return sbase + kOffBars + 8 * b; };
    const uint32_t mine = count(0, rank), other = count(0, rank ^ 1u), events = count(1, 0);
    constexpr uint32_t kBytes = kCtaPairs * 4;  // of a unit's factors from either CTA
    if (mine > other) mbar_complete_tx(bar(BAR_FFULL), kBytes);
    if (mine < other) mbar_arrive_expect_tx(bar(BAR_FFULL), kBytes);
    const uint64_t t0 = globaltimer_ns();
    auto wait = [&](int b, uint32_t phases) {
        while (phases > 0 && !mbar_try_wait(bar(b), (phases - 1) & 1) && globaltimer_ns() - t0 < kDrainLimitNs) {
        }
    };
    wait(BAR_FFULL, max(mine, other));
    wait(BAR_EVENT, events);
}

// ------------------------------------------------------------------------------------
// query operands (epilogue warps)
// ------------------------------------------------------------------------------------
constexpr int kPrepPairs = 4;                         // pairs whose loads are in flight together
constexpr int kOwnPairs = kCtaPairs / kEpilogueWarps; // pairs of a warp
constexpr int kFirstPairs = (kCtaPairs - kPrepPairs * kSoftmaxWarps) / kEpilogueWarps;  // of the first unit
static_assert(kFirstPairs % kPrepPairs == 0 && kOwnPairs % kPrepPairs == 0, "whole turns");

// Query operand rows of a warp's kPrepPairs or more pairs: lane l has dims [16l, 16l+16). A
// head's bf16 query becomes two E4M3 terms after a scaling by a power of two (exact for elements from
// 2^-9 of its largest, smaller ones off by 2^-16 of it at most), rows 2k and 2k+1 of the image the terms of pair
// k, stored chunk-major. The scale of its dots is positive (maxima are taken of the dots): a
// negative score scale turns the codes' signs, a zero one zeroes the codes. A head with a NaN or an
// infinity gets zero codes and a NaN scale (exponent 255), which makes all its scores NaN.
// The loop over pairs stays rolled: unrolled, its code is fetched anew for each unit, which took
// longer than all else here (18700 cycles for 16 pairs against 10600; 8500 now, with the terms
// formed as packed halves, which hold a query's eight bits exactly from 2^-14 on: below, both are 0).
struct Query {
    uint4 a, b;
};
__device__ __forceinline__ Query ask_query(const Cta& c, const Unit& u, int h) {
    const int pair = static_cast<int>(c.rank) * kCtaPairs + h;
    Query x{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (pair < u.valid) {
        const uint4* src = reinterpret_cast<const uint4*>(c.p.q + (u.pair0 + pair) * kLatent + (threadIdx.x & 31) * 16);
        x.a = __ldcs(src);
        x.b = __ldcs(src + 1);
    }
    return x;
}
struct Ahead {  // pairs whose loads are in flight
    Query x[kPrepPairs];
};
__device__ __forceinline__ Ahead ask_queries(const Cta& c, const Unit& u, int h0) {
    Ahead q;
#pragma unroll
    for (int i = 0; i < kPrepPairs; ++i) q.x[i] = ask_query(c, u, h0 + i);
    return q;
}
__device__ __forceinline__ void make_operand(const Cta& c, const Unit& u, Ahead q, int parity, int h0, int count, uint8_t* img) {
    constexpr int kTurn = 2;  // pairs side by side: one's instructions alone wait for one another
    const Params& p = c.p;
    const int lane = threadIdx.x & 31;
    const float sign = p.score_scale > 0.0f ? 1.0f : (p.score_scale < 0.0f ? -1.0f : 0.0f);
#pragma unroll 1
    for (int i = 0; i < count; i += kTurn) {
        uint32_t w[kTurn][8], amax[kTurn];
#pragma unroll
        for (int j = 0; j < kTurn; ++j) {
            const uint4 a = q.x[j].a, b = q.x[j].b;
            const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            amax[j] = 0;  // magnitudes as bits: NaN and infinity are the largest
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                w[j][k] = v[k];
                amax[j] = __vmaxu2(amax[j], v[k] & 0x7FFF7FFFu);
            }
            amax[j] = max(amax[j] << 16, amax[j] & 0xFFFF0000u);
        }
#pragma unroll
        for (int k = kTurn; k < kPrepPairs; ++k) q.x[k - kTurn] = q.x[k];
#pragma unroll
        for (int j = 0; j < kTurn; ++j)
            if (i + kPrepPairs + j < count) q.x[kPrepPairs - kTurn + j] = ask_query(c, u, h0 + i + kPrepPairs + j);
        float sc[kTurn];
#pragma unroll
        for (int j = 0; j < kTurn; ++j) amax[j] = __reduce_max_sync(0xffffffffu, amax[j]);
#pragma unroll
        for (int j = 0; j < kTurn; ++j) {
            const int E = static_cast<int>(amax[j] >> 23);
            int e = amax[j] > 0u ? 134 - E : 0;  // amax * 2^e in [128, 256)
            e = e > 126 ? 126 : (e < -126 ? -126 : e);
            sc[j] = __uint_as_float(static_cast<uint32_t>(e + 127) << 23) * sign;
            if (E == 255) {
#pragma unroll
                for (int k = 0; k < 8; ++k) w[j][k] = 0;
            }
            if (lane == 0) c.smem[kOffScale + parity * kCtaPairs + h0 + i + j] = E == 255 ? 255 : static_cast<uint8_t>(127 - e);
        }
        uint32_t hi[kTurn][4], lo[kTurn][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < kTurn; ++j) {
                uint32_t h2[2], l2[2];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t two = w[j][2 * k + m];
                    const __half2 v = __floats2half2_rn(__uint_as_float(two << 16) * sc[j], __uint_as_float(two & 0xFFFF0000u) * sc[j]);
                    h2[m] = *reinterpret_cast<const uint32_t*>(&v) & 0xFF80FF80u;
                    const __half2 r = __hsub2(v, *reinterpret_cast<const __half2*>(&h2[m]));
                    l2[m] = *reinterpret_cast<const uint32_t*>(&r);
                }
                hi[j][k] = f16x4_to_e4m3x4(h2[0], h2[1]);
                lo[j][k] = f16x4_to_e4m3x4(l2[0], l2[1]);
            }
#pragma unroll
        for (int j = 0; j < kTurn; ++j) {  // both rows' 16 bytes, one sector, one store
            auto two = [](uint32_t a, uint32_t b) { return static_cast<unsigned long long>(b) << 32 | a; };
            *reinterpret_cast<ulonglong4_32a*>(img + lane * 2048 + 2 * (h0 + i + j) * 16) =
                ulonglong4_32a{two(hi[j][0], hi[j][1]), two(hi[j][2], hi[j][3]), two(lo[j][0], lo[j][1]), two(lo[j][2], lo[j][3])};
        }
    }
    __syncwarp();
}

// Which of the tokens from the unit's shortest row on to its longest one's end hold a NaN code; both
// CTAs find out for themselves. One word of 32 tokens per warp.
__device__ uint32_t find_broken(const Cta& c, const Segment& s) {
    const Params& p = c.p;
    const int lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3;
    const int32_t first = s.min_len + 32 * q4, count = min(32, s.max_len - first);
    uint32_t word = 0;
    if (count > 0) {
        int32_t row = 0;
        const int32_t page = lane < count ? page_of(p, s.u.seq, first + lane, &row) : -1;
        const int64_t mine = page < 0 ? -1 : page * p.cache_stride + static_cast<int64_t>(row) * kLatent;
#pragma unroll 4
        for (int i = 0; i < count; ++i) {
            const int64_t at = __shfl_sync(0xffffffffu, mine, i);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (at >= 0) v = *reinterpret_cast<const uint4*>(p.v_cache + at + lane * 16);
            const uint32_t nan = nan_codes(v.x) | nan_codes(v.y) | nan_codes(v.z) | nan_codes(v.w);
            if (__any_sync(0xffffffffu, nan != 0u)) word |= 1u << i;
        }
    }
    return word;
}

// The first unit's operand is made by all warps that have nothing to do yet: kPrepPairs pairs by each
// softmax warp, the others by the epilogue warps.
__device__ void prepare_first(const Cta& c, int sw) {
    const Unit& u = c.p.starts[c.cluster].unit;
    const int h0 = sw * kPrepPairs;
    make_operand(c, u, ask_queries(c, u, h0), 0, h0, kPrepPairs, query_image(c, 0));
    named_bar_sync<kBarFirst, kThreads - kSoftmax0 * 32>();
}

// This warp's pairs of unit number `units` of the cluster, s: scales, marks and operand image.
__device__ void prepare_query(const Cta& c, const Segment& s, uint32_t units) {
    const int lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3, parity = units & 1;
    // The next unit's queries, one after another in memory, into L2.
    if (!s.last && lane == 0) {
        const Unit& u = c.p.units[s.k + 1];
        const int first = static_cast<int>(c.rank) * kCtaPairs + q4 * kOwnPairs, count = min(kOwnPairs, u.valid - first);
        if (count > 0) bulk_prefetch_l2(c.p.q + (u.pair0 + first) * kLatent, count * kLatent * 2);
    }
    const int count = units > 0 ? kOwnPairs : kFirstPairs, h0 = (units > 0 ? 0 : kSoftmaxWarps * kPrepPairs) + q4 * count;
    const Ahead x = ask_queries(c, s.u, h0);
    const uint32_t broken = find_broken(c, s);
    // The scales of the unit before the last are read. (One barrier for both parities
    // could pass two phases meanwhile.)
    if (units > 1) c.wait(BAR_UDONE0 + parity, ((units >> 1) - 1) & 1);
    make_operand(c, s.u, x, parity, h0, count, query_image(c, parity));
    if (lane == 0) broken_of(c, units)[q4] = broken;
    __syncwarp();
    if (units == 0) named_bar_sync<kBarFirst, kThreads - kSoftmax0 * 32>();
    if (lane == 0) mbar_arrive(c.bar(BAR_QMADE0 + parity));
}

// ------------------------------------------------------------------------------------
// epilogue warps: O's rescales and output
// ------------------------------------------------------------------------------------
__device__ void run_epilogue(const Cta& c) {
    const Params& p = c.p;
    const int lane = threadIdx.x & 31, q4 = (threadIdx.x >> 5) & 3;
    const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
    uint32_t tau = 0, units = 0, events = 0;
    Walk w(c), ahead(c);
    prepare_query(c, w.s, 0);
    for (;; w.advance(), ++units) {
        const Segment& s = w.s;
        tau += s.t1 - s.t0;
        if (!s.last) {
            ahead.advance();
            prepare_query(c, ahead.s, units + 1);
        }
        for (;;) {
            c.wait_long(BAR_EVENT, events++ & 1);
            const uint32_t event = *reinterpret_cast<volatile uint32_t*>(c.smem + kOffEvent);
            if (event == 0u || __any_sync(0xffffffffu, *c.abort_flag != 0)) break;
            // Tile event - 1 moved references: rescale O after the product before it.
            fence_cluster();
            const uint32_t at = event - 1;
            c.wait(BAR_PVDONE0 + ((at - 1) & 1), ((at - 1) >> 1) & 1);
            tc_fence_after();
            const volatile uint32_t* flags = reinterpret_cast<const volatile uint32_t*>(c.smem + kOffFlags) + (at & 1) * 8;
            const float* alpha = reinterpret_cast<const float*>(c.smem + kOffAlpha) + (at & 1) * kPairs;
#pragma unroll 1
            for (int b = 0; b < kPairs / 32; ++b) {  // 32 pairs of two lane quarters
                if (flags[2 * b] != event && flags[2 * b + 1] != event) continue;
                const uint32_t ta = c.tmem + lane_base + kTmemO + b * 32;
                uint32_t o0[32], o1[32];
                tmem_ld_2x32(ta, ta + kPairs, o0, o1);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float f = alpha[b * 32 + i];
                    o0[i] = __float_as_uint(__uint_as_float(o0[i]) * f);
                    o1[i] = __float_as_uint(__uint_as_float(o1[i]) * f);
                }
                tmem_st_x32(ta, o0);
                tmem_st_x32(ta + kPairs, o1);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) c.arrive(BAR_OFREE, 0);
        }

        // ---- output of the unit ----
        c.wait(BAR_PVDONE0 + ((tau - 1) & 1), ((tau - 1) >> 1) & 1);
        c.wait(BAR_FFULL, units & 1);
        tc_fence_after();
        const float* f_s = reinterpret_cast<const float*>(c.smem + kOffF);
        const bool whole = s.part < 0;
#pragma unroll 1
        for (int g = 0; g < kPairs / 32; ++g) {
            uint32_t v[2][32];  // of both blocks of 128 dims
            tmem_ld_2x32(c.tmem + lane_base + kTmemO + 32 * g, c.tmem + lane_base + kTmemO + kPairs + 32 * g, v[0], v[1]);
            const int dim0 = static_cast<int>(c.rank) * kDims + q4 * 32;
            if (whole) {
                // Neighbouring lanes exchange pairs and dims, so that a store has two dims of a pair.
                const int odd = lane & 1;
                const uint32_t pick = odd ? 0x3276u : 0x5410u;
                uint16_t* at = p.out + (s.u.pair0 + 32 * g + odd) * kLatent + dim0 + (lane & ~1);
                const int left = s.u.valid - 32 * g - odd;
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float2 f = *reinterpret_cast<const float2*>(f_s + 32 * g + i);
#pragma unroll
                    for (int mc = 0; mc < 2; ++mc) {
                        const __nv_bfloat162 r = __floats2bfloat162_rn(__uint_as_float(v[mc][i]) * f.x, __uint_as_float(v[mc][i + 1]) * f.y);
                        const uint32_t mine = *reinterpret_cast<const uint32_t*>(&r);
                        const uint32_t two = __byte_perm(mine, __shfl_xor_sync(0xffffffffu, mine, 1), pick);
                        if (i < left) *reinterpret_cast<uint32_t*>(at + i * kLatent + mc * 128) = two;
                    }
                }
            } else {
                uint16_t* part = p.part_o + static_cast<int64_t>(s.part) * kPairs * kLatent;
#pragma unroll
                for (int mc = 0; mc < 2; ++mc)
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = *reinterpret_cast<const float2*>(f_s + 32 * g + i + 2 * e);
                            const __half2 hv = __floats2half2_rn(__uint_as_float(v[mc][i + 2 * e]) * f.x, __uint_as_float(v[mc][i + 2 * e + 1]) * f.y);
                            h[e] = *reinterpret_cast<const uint32_t*>(&hv);
                        }
                        *reinterpret_cast<uint4*>(part + ((static_cast<int64_t>(dim0 / 32 + 4 * mc) * (kPairs / 8) + 4 * g + i / 8) * 32 + lane) * 8) =
                            make_uint4(h[0], h[1], h[2], h[3]);
                    }
            }
        }
        // NaN codes that were taken out of their tiles, into the dims of the rows that see them (in one
        // piece of a split unit: the join carries them on whatever the piece weighs).
        const uint4 broken = *reinterpret_cast<const uint4*>(broken_of(c, units));
        if ((broken.x | broken.y | broken.z | broken.w) != 0u) {
            __syncwarp();  // a lane's output was stored by its neighbour
#pragma unroll 1
            for (int i = 0; i < kPairs; ++i) {
                const int32_t pos = s.min_len + i, t = pos / kTile;
                if ((broken_of(c, units)[i >> 5] >> (i & 31) & 1u) == 0u || t < s.t0 || t >= s.t1 || pos >= s.max_len) continue;
                int32_t row;
                const int32_t page = page_of(p, s.u.seq, pos, &row);
                if (page < 0) continue;  // (after an abort the marks may be anything)
                const int64_t before = static_cast<int64_t>(pos - s.u.base) * p.heads - s.u.first;  // pairs that do not see it
#pragma unroll 1
                for (int mc = 0; mc < 2; ++mc) {
                    const int dim = static_cast<int>(c.rank) * kDims + q4 * 32 + mc * 128 + lane;
                    const uint8_t code = p.v_cache[page * p.cache_stride + static_cast<int64_t>(row) * kLatent + dim];
                    if ((code & 0x7F) != 0x7F) continue;
#pragma unroll 1
                    for (int pair = before > 0 ? static_cast<int>(before) : 0; pair < s.u.valid; ++pair) {
                        uint16_t* at = whole ? p.out + (s.u.pair0 + pair) * kLatent + dim
                                             : p.part_o + static_cast<int64_t>(s.part) * kPairs * kLatent +
                                                   ((dim / 32 * (kPairs / 8) + pair / 8) * 32 + lane) * 8 + pair % 8;
                        *at = 0x7FFF;  // a NaN in BF16 and in FP16
                    }
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) c.arrive(BAR_OFREE, 0);
        if (lane < 2) c.arrive(BAR_FEMPTY, lane);
        if (s.last) break;
    }
}

template <bool kTma>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap kmap,
                                                              const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5;
    Cta c{p, smem, smem_u32(smem), cluster_rank(), blockIdx.x >> 1, reinterpret_cast<volatile int*>(smem + kOffAbort)};

    if (tid == 0) {
        for (int e = 0; e < kKeySlots; ++e) {
            mbar_init(c.bar(BAR_KFULL0 + e), kTma ? 1 : 32);
            mbar_init(c.bar(BAR_KPEER0 + e), 1);
            mbar_init(c.bar(BAR_KEMPTY0 + e), 1);
        }
        for (int e = 0; e < kValueSlots; ++e) {
            mbar_init(c.bar(BAR_VFULL0 + e), kTma ? 1 : 32);
            mbar_init(c.bar(BAR_VEMPTY0 + e), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(c.bar(BAR_PFULL0 + i), 2 * kSoftmaxWarps);
            mbar_init(c.bar(BAR_PVDONE0 + i), 1);
            mbar_init(c.bar(BAR_UDONE0 + i), kSoftmaxWarps);
            mbar_init(c.bar(BAR_QMADE0 + i), kEpilogueWarps);
        }
        mbar_init(c.bar(BAR_SFULL), 1);
        mbar_init(c.bar(BAR_SEMPTY), 2 * kSoftmaxWarps);
        mbar_init(c.bar(BAR_QFULL), 2 * kSoftmaxWarps);
        mbar_init(c.bar(BAR_QEMPTY), 1);
        mbar_init(c.bar(BAR_EVENT), 1);
        mbar_init(c.bar(BAR_OFREE), 2 * kEpilogueWarps);
        mbar_init(c.bar(BAR_FFULL), 1);  // and the factors' bytes
        mbar_init(c.bar(BAR_FEMPTY), 2 * kEpilogueWarps);
        mbar_init(c.bar(BAR_DRAIN), 2);
        for (int i = 0; i < 16; ++i) reinterpret_cast<uint32_t*>(smem + kOffFlags)[i] = 0;
        for (int i = 0; i < 2; ++i) c.sent()[i] = 0;
        *c.progress() = 0;
        *c.abort_flag = 0;
        fence_mbar_init();
        if (kTma) {
            prefetch_tmap(&kmap);
            prefetch_tmap(&vmap);
        }
    }
    if (warp == 2) {
        tmem_alloc_pair(c.sbase + kOffTmem, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
    c.tmem = *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem);
    // Everything above overlaps the plan; it is read only after this.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    c.begin = p.starts[c.cluster].begin;
    c.end = p.starts[c.cluster].end;
    c.gap = p.starts[c.cluster].gap;
    if ((c.sbase & 1023u) != 0u) {  // the swizzled operands count on it
        if (tid == 0) report(p, DSA_ERR_UNSUPPORTED);
    } else if (c.begin < c.end) {
        if (warp < 2) {
            if constexpr (!kTma) run_load_copies(c, warp == 1);
            else if (warp == 0) run_load_tma<false>(c, &kmap);
            else run_load_tma<true>(c, &vmap);
        } else if (warp < kSoftmax0) {
            if (warp == 2) {
                if (c.rank == 0) run_qk(c);
                else run_forward(c);
            } else if (c.rank == 0) {
                c.sent()[1] = run_pv(c);
            }
            // In both CTAs: products arrive at barriers of both, and for the last arrivals nobody else waits.
            if (warp == 2 || c.rank == 0) {
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(c.bar(BAR_DRAIN), 0) && globaltimer_ns() - t0 < kDrainLimitNs) {
                }
                __syncwarp();
            }
        } else if (warp < kEpilogue0) {
            prepare_first(c, warp - kSoftmax0);
            const uint32_t sent = run_softmax(c);
            if (warp == kSoftmax0) c.sent()[0] = sent;
        } else {
            run_epilogue(c);
        }
    }
    tc_fence_before();
    __syncthreads();
    // Neither CTA leaves while the other may still reach into it.
    cluster_arrive();
    cluster_wait();
    if (*c.abort_flag != 0) {  // as both CTAs find by now
        if (tid == 0) receive_rest(c.sbase, c.rank);
        __syncthreads();
        cluster_arrive();  // the counts are read
        cluster_wait();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(c.tmem, kTmemCols);
    }
}

template <bool kTma>
cudaError_t setup() {
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, prefill_kernel<kTma>);
    if (e != cudaSuccess) return e;
    if (attr.maxThreadsPerBlock < kThreads) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(prefill_kernel<kTma>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(prefill_kernel<kTma>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
}

}  // namespace
}  // namespace prefill

cudaError_t prefill_setup() {
    const cudaError_t e = prefill::setup<true>();
    return e != cudaSuccess ? e : prefill::setup<false>();
}

cudaError_t launch_prefill(const prefill::Params& p, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * p.clusters);
    cfg.blockDim = dim3(prefill::kThreads);
    cfg.dynamicSmemBytes = prefill::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return p.box_rows > 0 ? cudaLaunchKernelEx(&cfg, prefill::prefill_kernel<true>, p, kmap, vmap)
                          : cudaLaunchKernelEx(&cfg, prefill::prefill_kernel<false>, p, kmap, vmap);
}

}  // namespace dsa
