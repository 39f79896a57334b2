// Shared by the kernels of the prompt-chunk attention (prefill_plan.cu, prefill.cu): geometry,
// workspace layout, parameters and the device-side work plan.
//
// A request's new tokens times the heads, its (row, head) pairs, lie one after another in the packed
// queries and all read the same cache, so they are cut into units of 128 pairs whatever their rows.
// Rows of a unit see one token more from each to the next; its tokens are those that its last row
// sees. As in the full decode (full.cuh) the units' 128-token tiles form a line, with a gap between
// units for what a change of unit costs, that is cut into equal ranges, here one per pair of CTAs;
// a unit that several ranges share leaves a partial in each, which are joined afterwards.
#pragma once

#include "full.cuh"

namespace dsa {
namespace prefill {

constexpr int kPairs = 128;  // (row, head) pairs of a unit, 64 in each CTA of a cluster
constexpr int kTile = full::kTile;
// Tiles that a unit change costs, at most a quarter of a range. (One prompt of 4096 rows of 64 heads with
// gaps of 3, 4, 5, 6 and 8 tiles: 1003, 882, 796, 734 and 735 us; 128 short requests: 99, 96, 95, 95, 95; a mixed
// batch: 1953, 1934, 1949, 1949, 1973.)
constexpr int kGap = 6;

struct alignas(16) Unit {
    int64_t start;  // its first tile on the line
    int64_t pair0;  // its first pair among all packed ones
    int32_t seq, first, valid, base;  // request; first pair among the request's, pairs; cached tokens
};
// What a cluster starts with (an empty range: begin = end).
struct alignas(16) Start {
    int64_t begin, end;
    int32_t gap, k, pad[2];
    Unit unit;  // number k
};
// Pieces of a unit that range c starts and others go on with (0: none): in the partial slots 2c or
// 2c + 1 (slot_lo), then 2(c + 1), 2(c + 2), ...
struct alignas(16) Join {
    int32_t unit, slot_lo, pieces, c;
};

struct Layout {
    size_t status, starts, joins, units, qimg, part_o, part_lse, total;
};
inline Layout layout(int64_t units, int64_t clusters) {
    Layout L;
    size_t o = 0;
    auto put = [&](size_t bytes) {
        const size_t at = o;
        o = align256(o + bytes);
        return at;
    };
    L.status = put(256);
    L.starts = put(static_cast<size_t>(clusters) * sizeof(Start));
    L.joins = put(static_cast<size_t>(clusters) * sizeof(Join));
    L.units = put(static_cast<size_t>(units + 1) * sizeof(Unit));  // read one ahead
    L.qimg = put(static_cast<size_t>(2 * 2 * clusters) * kQImageBytes);
    L.part_o = put(static_cast<size_t>(2 * clusters) * kPairs * kLatent * 2);
    L.part_lse = put(static_cast<size_t>(2 * clusters) * kPairs * 4);
    L.total = o;
    return L;
}
// Units of a call at most: all rows' pairs, and a unit that is not full for each request.
inline int64_t max_units(int64_t num_seqs, int64_t max_rows, int64_t heads) {
    return max_rows * heads / kPairs + (num_seqs < max_rows ? num_seqs : max_rows);
}

struct Params {
    const uint16_t* q;         // bf16 bits [max_rows, heads, 512]
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const int32_t* block_tables;
    const int32_t* base_lens;  // [num_seqs]
    const int32_t* new_lens;   // [num_seqs]
    uint16_t* out;             // bf16 bits [max_rows, heads, 512]
    int* status;               // of the call, in its workspace
    int* step_status;          // of the device, see dsa_step_device_status
    Start* starts;             // [clusters]
    Join* joins;               // [most_joins], in any order
    Unit* units;               // [units]
    uint8_t* qimg;             // [2 * clusters CTAs][2 units in turn][64 KB] query operands
    uint16_t* part_o;          // f16 bits [2 * clusters][16 blocks of 32 dims][16 groups of 8 pairs][32 dims][8 pairs]
    float* part_lse;           // [2 * clusters][128]
    int64_t cache_stride;
    int32_t num_seqs, max_rows, heads, block_size, max_blocks_per_seq, clusters;
    int32_t most_joins;        // units, or ranges, whichever are fewer
    int32_t few_units;         // units may come in many pieces each
    int32_t small_plan;        // few requests and units
    int32_t box_rows;          // tokens of a tensor-map box (8, 16 or 32), 0: per-thread copies
    FastDiv by_block, by_heads;
    int32_t room;              // tokens that a table holds
    float score_scale;         // sm_scale * k_scale * log2(e)
    float v_scale;
    uint64_t wait_limit_ns;
};

#ifdef __CUDACC__
__device__ __forceinline__ void report(const Params& p, int code) {
    atomicCAS(p.status, 0, code);
    atomicCAS(p.step_status, 0, code);
}
// Tokens that pair `pair` of a request sees.
__device__ __forceinline__ int32_t pair_len(const Params& p, int32_t base, int32_t pair) {
    const int64_t n = static_cast<int64_t>(base) + divide(static_cast<uint32_t>(pair), p.by_heads) + 1;
    return static_cast<int32_t>(n < p.room ? n : p.room);
}
#endif

}  // namespace prefill

cudaError_t prefill_setup();
cudaError_t prefill_plan_setup(int clusters);
// kmap, vmap: 5-D tensor maps of the caches ([page][group of 8 rows][128-byte block][row][128 bytes]),
// boxes of p.box_rows rows and all blocks (K) or two of them (V); read only when p.box_rows > 0.
cudaError_t launch_prefill_plan(const prefill::Params& p, cudaStream_t stream);
cudaError_t launch_prefill(const prefill::Params& p, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream);
cudaError_t launch_prefill_join(const prefill::Params& p, cudaStream_t stream);

}  // namespace dsa
