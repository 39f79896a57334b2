// Shared by the kernels of the full-cache decode (full_plan.cu, full.cu): geometry, workspace
// layout, parameters and the device-side work plan.
//
// A sequence's rows_per_seq*heads (row, head) pairs all read the same cache, so they are cut
// into groups of 64 whatever their rows, and a work unit is (sequence, group): few heads and
// several verify rows fill one unit together. A unit's tokens are [0, max of its rows'
// lengths); rows that see fewer mask theirs. The units with any token, in order, form a line
// of 128-token tiles with a gap of up to kGap tiles between units, T long, that is cut into
// `ctas` equal ranges: CTA c takes the tiles in [c*T/ctas, (c+1)*T/ctas). A gap stands for what
// a change of unit costs the CTA whose range holds it (output, query operand, first tile):
// without it those CTAs finish last. The lengths are on the device, so the plan is made there.
// A unit inside one range is written straight to the output; one that several ranges share
// leaves a partial per CTA (slot 2c for the CTA's first unit, 2c+1 for its last) that the
// combine kernel joins.
#pragma once

#include "common.cuh"

namespace dsa {
namespace full {

constexpr int kTile = 128;
constexpr int kGap = 5;      // tiles that a unit change costs, at most a quarter of a range
constexpr int64_t kMaxLen = (int64_t{1} << 31) - 2 * kTile;  // positions stay in 32 bits

// One CTA's stretch of one unit.
struct Segment {
    int32_t k, unit;           // live unit's number, its unit
    int32_t t0, t1;            // tiles of the unit
    int32_t max_len, min_len;  // of the unit's rows
    int32_t part;              // partial slot, -1: the whole unit
    int32_t last;              // the CTA's last unit
};

// What a CTA starts with, in one load: its range (empty: begin = end) and its first segment.
struct alignas(16) CtaStart {
    int64_t begin, end;
    Segment first;
    int64_t gap;
    int64_t pad;
};

// Where a unit's pieces are: ranges c_lo .. c_lo + pieces - 1, all in slot 2c but the first
// one, in slot_lo (its CTA may have started in the unit before). Nothing to join below two.
struct alignas(16) UnitPieces {
    int32_t c_lo, slot_lo, pieces, pad;
};

struct PlanArrays {
    CtaStart* cta;        // [max_ctas]
    UnitPieces* pieces;   // [units]
    // by a live unit's number k:
    int64_t* start;       // [units] its first tile on the line
    int32_t* unit;        // [units]
    int32_t* max_len;     // [units] longest length of its rows
    int32_t* min_len;     // [units] shortest
};

// ------------------------------------------------------------------------------------
// The plan's arithmetic (host and device: the tests run it on the host).
// ------------------------------------------------------------------------------------
// n / d for n >= 0, d > 0. They fit 32 bits but for the longest caches, and a 64-bit division
// is a long sequence. Out of line: the plan runs once, and what its code weighs in instruction
// fetches is most of its time.
#ifdef __CUDACC__
__host__ __device__ __noinline__
#endif
static int64_t quotient(int64_t n, int64_t d) {
    if (n >> 32 == 0 && d >> 32 == 0) return static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
    return n / d;
}

struct Line {
    int64_t length, gap;
    int32_t ctas;  // ranges; none is empty
};
__host__ __device__ inline Line make_line(int64_t tiles, int32_t live, int32_t max_ctas) {
    Line l;
    l.ctas = static_cast<int32_t>(tiles < max_ctas ? tiles : max_ctas);
    // At most a quarter of a range, so that no range lies inside a gap.
    l.gap = tiles / (4 * max_ctas);
    if (l.gap > kGap) l.gap = kGap;
    l.length = tiles + l.gap * (live > 0 ? live - 1 : 0);
    return l;
}
// Range c is [floor(c*T/C), floor((c+1)*T/C)).
__host__ __device__ inline int64_t range_begin(const Line& l, int64_t c) { return quotient(c * l.length, l.ctas); }
// Pieces of live unit k, at [b, e) of the line: the range that holds tile x is
// floor(((x + 1)*C - 1) / T). The unit is the first of the ranges [*c0, *c1), which start
// after the unit before it ended and before it ends itself.
__host__ __device__ inline UnitPieces unit_pieces(const Line& l, int32_t k, int64_t b, int64_t e, int32_t* c0, int32_t* c1) {
    UnitPieces q;
    q.c_lo = static_cast<int32_t>(quotient((b + 1) * l.ctas - 1, l.length));
    q.pieces = static_cast<int32_t>(quotient(e * l.ctas - 1, l.length)) - q.c_lo + 1;
    *c0 = static_cast<int32_t>(quotient((k > 0 ? b - l.gap : 0) * l.ctas + l.length - 1, l.length));
    *c1 = static_cast<int32_t>(quotient(e * l.ctas + l.length - 1, l.length));
    q.slot_lo = 2 * q.c_lo + (*c0 <= q.c_lo ? 0 : 1);
    q.pad = 0;
    return q;
}
// CTA's stretch of live unit k, whose first tile is b on the line, given the CTA's range.
__host__ __device__ inline Segment segment(int64_t begin, int64_t end, int64_t gap, int32_t cta, bool first, int32_t k, int32_t unit,
                                           int64_t b, int32_t max_len, int32_t min_len) {
    const int64_t e = b + (max_len + kTile - 1) / kTile;
    Segment s;
    s.k = k;
    s.unit = unit;
    s.t0 = static_cast<int32_t>((begin > b ? begin : b) - b);
    s.t1 = static_cast<int32_t>((end < e ? end : e) - b);
    s.max_len = max_len;
    s.min_len = min_len;
    s.part = begin <= b && e <= end ? -1 : 2 * cta + (first ? 0 : 1);
    s.last = e + gap >= end;
    return s;
}

struct Layout {
    size_t status, cta, pieces, start, unit, max_len, min_len, qimg, qscale, part_o, part_lse, total;
};

inline Layout layout(int64_t units, int64_t ctas) {
    Layout L;
    size_t o = 0;
    auto put = [&](size_t bytes) {
        const size_t at = o;
        o = align256(o + bytes);
        return at;
    };
    L.status = put(256);
    L.cta = put(static_cast<size_t>(ctas) * sizeof(CtaStart));
    L.pieces = put(static_cast<size_t>(units) * sizeof(UnitPieces));
    L.start = put(static_cast<size_t>(units) * 8);
    L.unit = put(static_cast<size_t>(units) * 4);
    L.max_len = put(static_cast<size_t>(units) * 4);
    L.min_len = put(static_cast<size_t>(units) * 4);
    L.qimg = put(static_cast<size_t>(units) * kQImageBytes);
    L.qscale = put(static_cast<size_t>(units) * kHeadsPerCta * 4);
    L.part_o = put(static_cast<size_t>(2 * ctas) * kHeadsPerCta * kLatent * 2);
    L.part_lse = put(static_cast<size_t>(2 * ctas) * kHeadsPerCta * 4);
    L.total = o;
    return L;
}

struct Params {
    const uint16_t* q;         // bf16 bits [R, heads, 512]
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const int32_t* block_tables;
    const int32_t* seq_lens;   // [R], or [num_seqs] before the verify rows
    uint16_t* out;             // bf16 bits [R, heads, 512]
    int* status;               // of the call, in its workspace
    int* step_status;          // of the device, see dsa_step_device_status
    PlanArrays plan;
    uint8_t* qimg;             // [units, 64 KB]
    float* qscale;             // [units, 64]
    uint16_t* part_o;          // f16 bits [2*ctas, 64, 512], laid out as the selected decode's partials
    float* part_lse;           // [2*ctas, 64]
    int64_t cache_stride;
    int32_t num_seqs, rows_per_seq, heads, pairs, groups, units, max_ctas;
    int32_t block_size, max_blocks_per_seq, verify_rows;
    FastDiv by_block;          // block_size
    int32_t box_rows;          // tokens of a tensor-map box (8, 16 or 32), 0: per-thread copies
    int32_t kv_same;
    float score_scale;         // sm_scale * k_scale * log2(e)
    float v_scale;
    uint64_t wait_limit_ns;
};

#ifdef __CUDACC__
__device__ __forceinline__ void report(const Params& p, int code) {
    atomicCAS(p.status, 0, code);
    atomicCAS(p.step_status, 0, code);
}
// Tokens that a row sees. `given` may pass the block table's room: *over says so.
__device__ __forceinline__ int32_t row_len(const Params& p, int64_t seq, int32_t i, bool* over) {
    int64_t n = p.verify_rows ? static_cast<int64_t>(p.seq_lens[seq]) + i + 1 : p.seq_lens[seq * p.rows_per_seq + i];
    int64_t room = p.max_blocks_per_seq > 0 ? static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size : kMaxLen;
    if (room > kMaxLen) room = kMaxLen;
    *over = n > room;
    if (n > room) n = room;
    return n > 0 ? static_cast<int32_t>(n) : 0;
}
#endif

}  // namespace full

cudaError_t full_setup();
// kmap / vmap: 5-D tensor maps of the caches ([page][group of 8 rows][128-byte block][row]
// [128 bytes], boxes of whole groups, p.box_rows rows), read only when p.box_rows > 0.
cudaError_t launch_full(const full::Params& p, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream);
cudaError_t full_plan_setup();
cudaError_t launch_full_plan(const full::Params& p, cudaStream_t stream);
cudaError_t launch_full_combine(const full::Params& p, cudaStream_t stream);

}  // namespace dsa
