// The step plan: from every request's cached and new token counts, the physical pages of the
// new tokens (written into the block tables) and each new token's cache slot, position,
// visible length and request, as the cache writers, the selector and the decode take them
// (decode_k.rs, decode_k: slot = physical*block_size + pos % block_size).
//
//   have(s) = ceil(base(s)/bs), want(s) = ceil((base(s)+new(s))/bs), both at most the table's width
//   table[s][have(s)+i] = free[g0(s)+i] (or -1 past the free list), g0 = exclusive sum of want - have
//   row of token i of s: pos = base(s)+i, slot = table[s][pos/bs]*bs + pos%bs, len = pos+1
//
// Lengths and positions fit 32 bits (the table's room does), divisions are 32-bit, and a lane
// works on four rows at once, 32 apart, so that their searches and page loads overlap and
// their stores stay coalesced.
//
// One launch. Both prefix sums (tokens, pages) over the requests are made by every block for
// itself in shared memory: 8 bytes a request, served by L2 after the first block, cost less
// than a second launch. Rows and new table entries are then spread over all blocks. A packed
// row finds its request by a binary search of the token prefix sums in shared memory. A new
// page's id is read from the free list, not from the table entry that another block writes,
// so no block waits for another. Block 0 alone reports what it finds wrong.
//
// Bound by latency and instruction issue, not by bytes: one token of each of 64 requests takes
// 3.2 us; 256 packed prompts with 528 000 tokens 7.3 us (1.5 TB/s of the 20 bytes that a row has
// written, 1.6 us at the HBM's rate; 55 % of the issue slots under a profiler). Four rows a lane,
// one search for a warp's 128 rows where one prompt fills them, and divisions through a
// multiplier made on the host were each a step from 11.4 us. More blocks repeat the prefix
// sums, fewer leave SMs idle.
#include <climits>

#include "common.cuh"

namespace dsa {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kTurns = 4;                    // rows that a lane works on at once
constexpr int kRowsPerWarp = 32 * kTurns;

__device__ __forceinline__ int32_t saturate(int64_t x) { return x > INT_MAX ? INT_MAX : static_cast<int32_t>(x); }

// Token counts of a request as the plan uses them; `bad` when they had to be cut.
struct Request {
    uint32_t base, fresh;  // cached and new tokens
    uint32_t have, want;   // pages before and after, at most the table's width
    bool bad;
};
__device__ __forceinline__ uint32_t pages_of(const PlanParams& p, uint32_t tokens) {
    const uint32_t q = divide(tokens, p.by_block);
    return min(q + (tokens != q * p.by_block.d ? 1u : 0u), static_cast<uint32_t>(p.max_blocks));
}
__device__ __forceinline__ Request request(const PlanParams& p, int32_t s) {
    Request r;
    const int32_t b = p.base_lens[s], n = p.new_lens[s];
    r.base = b < 0 ? 0 : b;
    r.fresh = n < 0 ? 0 : n;
    r.bad = b < 0 || n < 0;
    if (p.rows_per_seq > 0 && r.fresh > static_cast<uint32_t>(p.rows_per_seq)) {
        r.fresh = p.rows_per_seq;
        r.bad = true;
    }
    const uint32_t all = r.base + r.fresh;  // below 2^32
    r.bad |= all > static_cast<uint32_t>(p.max_blocks) * static_cast<uint32_t>(p.block_size);
    r.have = pages_of(p, r.base);
    r.want = pages_of(p, all);
    return r;
}

// Index of the last entry of the ascending array a[0..n] that is <= x (a[0] = 0 <= x < a[n]).
__device__ __forceinline__ int32_t last_at_most(const int32_t* a, int32_t n, int32_t x) {
    int32_t lo = 0, hi = n;
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
    extern __shared__ int32_t prefix[];  // tokens t0[0..n], then pages g0[0..n]
    __shared__ int64_t warp_tokens[kPlanWarps], warp_pages[kPlanWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t n = p.num_seqs;
    int32_t* t0 = prefix;
    int32_t* g0 = prefix + n + 1;

    // Thread t sums requests [t*per, (t+1)*per), a block scan gives its start, and a second
    // sweep writes the prefix sums (saturated: rows and pages past 2^31 - 1 do not exist).
    const int32_t per = (n + kPlanThreads - 1) / kPlanThreads;
    const int32_t lo = min(n, tid * per), hi = min(n, lo + per);
    int64_t tokens = 0, pages = 0;
    for (int32_t s = lo; s < hi; ++s) {
        const Request r = request(p, s);
        tokens += r.fresh;
        pages += r.want - r.have;
    }
    int64_t it = tokens, ip = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, it, o), b = __shfl_up_sync(0xffffffffu, ip, o);
        if (lane >= o) {
            it += a;
            ip += b;
        }
    }
    if (lane == 31) {
        warp_tokens[warp] = it;
        warp_pages[warp] = ip;
    }
    __syncthreads();
    int64_t ct = it - tokens, cp = ip - pages;
    for (int w = 0; w < warp; ++w) {
        ct += warp_tokens[w];
        cp += warp_pages[w];
    }
    bool bad = false;
    for (int32_t s = lo; s < hi; ++s) {
        const Request r = request(p, s);
        t0[s] = saturate(ct);
        g0[s] = saturate(cp);
        ct += r.fresh;
        cp += r.want - r.have;
        bad |= r.bad;
        // The page that the first new token shares with cached ones has to be there already.
        if (blockIdx.x == 0 && r.fresh > 0) {
            const uint32_t blk = divide(r.base, p.by_block);
            if (blk < r.have) bad |= p.tables[static_cast<int64_t>(s) * p.max_blocks + blk] < 0;
        }
    }
    if (hi == n && (lo < n || (n == 0 && tid == 0))) {  // the last thread with a request; no request: thread 0
        t0[n] = saturate(ct);
        g0[n] = saturate(cp);
    }
    bad = __syncthreads_or(bad);
    const int32_t all_tokens = t0[n], all_pages = g0[n];
    if (blockIdx.x == 0 && tid == 0) {
        bad |= all_pages > p.num_free || (p.rows_per_seq == 0 && all_tokens > p.rows);
        p.info[0] = p.rows_per_seq == 0 ? min(all_tokens, p.rows) : all_tokens;
        p.info[1] = min(all_pages, p.num_free);
        p.info[2] = bad ? DSA_ERR_DEVICE_BOUNDS : DSA_OK;
        p.info[3] = 0;
    }

    const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid; e < all_pages; e += step) {
        const int32_t s = last_at_most(g0, n, static_cast<int32_t>(e));
        const int64_t have = request(p, s).have;
        p.tables[static_cast<int64_t>(s) * p.max_blocks + have + (e - g0[s])] = e < p.num_free ? p.free_pages[e] : -1;
    }
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kPlanWarps;
    for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) * kPlanWarps + warp) * kRowsPerWarp; r0 < p.rows; r0 += warps * kRowsPerWarp) {
        uint32_t pos[kTurns], off[kTurns];
        int32_t seq[kTurns], page[kTurns];
        // Where token i of request s goes.
        auto place = [&](int j, int32_t s, const Request& r, uint32_t i) {
            const uint32_t at = r.base + i, blk = divide(at, p.by_block);
            if (i >= r.fresh || blk >= static_cast<uint32_t>(p.max_blocks)) return;
            seq[j] = s;
            pos[j] = at;
            off[j] = at - blk * p.by_block.d;
            const int64_t g = static_cast<int64_t>(g0[s]) + blk - r.have;
            if (blk < r.have) page[j] = p.tables[static_cast<int64_t>(s) * p.max_blocks + blk];
            else if (g < p.num_free) page[j] = p.free_pages[g];
        };
#pragma unroll
        for (int j = 0; j < kTurns; ++j) {
            seq[j] = page[j] = -1;
            pos[j] = 0xFFFFFFFFu;
            off[j] = 0;
        }
        if (p.rows_per_seq > 0) {
#pragma unroll
            for (int j = 0; j < kTurns; ++j) {
                const int64_t row = r0 + 32 * j + lane;
                if (row >= p.rows) continue;
                const int32_t s = static_cast<int32_t>(row) / p.rows_per_seq;
                place(j, s, request(p, s), static_cast<uint32_t>(static_cast<int32_t>(row) - s * p.rows_per_seq));
            }
        } else if (r0 < all_tokens) {
            // A prompt's tokens mostly fill the warp's rows: one search then does for all.
            const int32_t s0 = last_at_most(t0, n, static_cast<int32_t>(r0));
            if (t0[s0 + 1] - r0 >= kRowsPerWarp) {
                const Request r = request(p, s0);
#pragma unroll
                for (int j = 0; j < kTurns; ++j) {
                    const int64_t row = r0 + 32 * j + lane;
                    if (row < p.rows) place(j, s0, r, static_cast<uint32_t>(static_cast<int32_t>(row) - t0[s0]));
                }
            } else {
#pragma unroll
                for (int j = 0; j < kTurns; ++j) {
                    const int64_t row = r0 + 32 * j + lane;
                    if (row >= p.rows || row >= all_tokens) continue;
                    const int32_t s = last_at_most(t0, n, static_cast<int32_t>(row));
                    place(j, s, request(p, s), static_cast<uint32_t>(static_cast<int32_t>(row) - t0[s]));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kTurns; ++j) {
            const int64_t row = r0 + 32 * j + lane;
            if (row >= p.rows) continue;
            p.slots[row] = page[j] >= 0 ? static_cast<int64_t>(page[j]) * p.block_size + off[j] : -1;
            p.positions[row] = static_cast<int32_t>(pos[j]);
            p.row_lens[row] = static_cast<int32_t>(pos[j] + 1u);
            p.row_seqs[row] = seq[j];
        }
    }
}

}  // namespace

cudaError_t plan_kernel_setup() {
    return cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                2 * (DSA_MAX_PLAN_SEQS + 1) * 4);
}

cudaError_t launch_plan(const PlanParams& p, int sms, cudaStream_t stream) {
    // Four rows a thread before another block is worth its own prefix sums, and no more blocks
    // than run at once.
    const int64_t want = (static_cast<int64_t>(p.rows) + kTurns * kPlanThreads - 1) / (kTurns * kPlanThreads);
    const int most = (p.num_seqs <= 4096 ? 4 : 1) * sms;
    const int blocks = static_cast<int>(want < 1 ? 1 : (want > most ? most : want));
    plan_kernel<<<blocks, kPlanThreads, 2 * (p.num_seqs + 1) * 4, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dsa
