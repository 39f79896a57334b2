// Pages of a paged cache: copied, forked (shared by a further request), released to the free list
// and compacted to the pool's front. Whatever runs side by side here is sums, minima and bits of
// whole numbers, so results do not depend on an order: pages are listed by their number.
//
// The books (tables, shares, free list) are bound by latency: a launch each for what every block
// has to know of the others', the launches overlapped, and within each a few dependent loads and
// barriers. 64 requests that give back their drafts 6.9 us (two launches), half of 256 requests with
// 1.2 thousand pages each 17.7, a fork of four ways 4.6 (two launches), a pool of 380 pages compacted
// 8.9 (three launches), each measured with a copy of the books in front: 1.2 us, 4.0 in the second.
// Page data is bound by HBM: 1024 pages of two pools in four layers, 338 MB read and written, 53 us,
// 6.4 TB/s, 94 % of a plain copy's rate. Blocks of 256 threads with four 16-byte pieces in flight
// each, eight blocks to an SM, are what it takes; pieces pass the caches by, as they are not read again.
#include "pages.cuh"
#include "ptx.cuh"

namespace dsa {
namespace pages {
namespace {

constexpr int kMarkThreads = 256;
constexpr int kListThreads = 1024;
constexpr int kListWarps = kListThreads / 32;
// Up to kFewForks forks are planned by a block of kForkThreads, whose barriers are cheaper (4 forks 4.4
// us, 5.8 with kManyForkThreads; 240 forks 7.2 and 8.4; 512 forks 10.3 and 10.6; 1024 forks 16.2 and 14.9).
constexpr int kFewForks = 512, kForkThreads = 256, kManyForkThreads = 1024;

__device__ __forceinline__ void report(int* status) { atomicCAS(status, 0, DSA_ERR_DEVICE_BOUNDS); }
__device__ __forceinline__ void wait_prior() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Length of request s, cut to what its table holds.
__device__ __forceinline__ int32_t clamped(const Tables& t, int32_t n, bool* bad) {
    const int64_t room = static_cast<int64_t>(t.max_blocks) * t.block_size;
    *bad |= n < 0 || n > room;
    if (n > room) n = static_cast<int32_t>(room);
    return n < 0 ? 0 : n;
}
__device__ __forceinline__ int32_t pages_of(const Tables& t, int32_t n) {
    return static_cast<int32_t>(divide(static_cast<uint32_t>(n) + static_cast<uint32_t>(t.block_size) - 1u, t.by_block));
}

// One chunk of one page: item of pair (src, dst).
__device__ __forceinline__ void copy_chunk(const Pools& pools, uint32_t rest, int32_t src, int32_t dst) {
    int j = 0;
    while (j + 1 < pools.count && rest >= pools.pool[j + 1].first) ++j;
    const Pool& pool = pools.pool[j];
    rest -= pool.first;
    const uint32_t layer = divide(rest, pool.by_chunks), chunk = rest - layer * pool.by_chunks.d;
    const int64_t at = static_cast<int64_t>(layer) * pool.layer_stride + static_cast<int64_t>(chunk) * kChunkVecs * 16;
    const uint4* s = reinterpret_cast<const uint4*>(pool.base + src * pool.page_stride + at);
    uint4* d = reinterpret_cast<uint4*>(pool.base + dst * pool.page_stride + at);
    const uint32_t n = min(kChunkVecs, pool.vecs - chunk * kChunkVecs);
    uint4 v[kCopyVecs];
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i)
        if (threadIdx.x + i * kCopyThreads < n) v[i] = __ldcs(s + threadIdx.x + i * kCopyThreads);
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i)
        if (threadIdx.x + i * kCopyThreads < n) __stcs(d + threadIdx.x + i * kCopyThreads, v[i]);
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
    const uint32_t items = static_cast<uint32_t>(p.count) * p.pools.items;
    for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const uint32_t pair = divide(static_cast<uint32_t>(it), p.pools.by_items);
        const int32_t src = p.src[pair], dst = p.dst[pair];
        if (src < 0 || dst < 0) continue;
        if (src >= p.num_pages || dst >= p.num_pages) {
            if (threadIdx.x == 0) report(p.status);
            continue;
        }
        if (src != dst) copy_chunk(p.pools, static_cast<uint32_t>(it) - pair * p.pools.items, src, dst);
    }
}

// ------------------------------------------------------------------------------------
// fork
// ------------------------------------------------------------------------------------
// Sum of v over the block's threads before this one; *total over all. Ends with the sums read.
template <int kWarps>
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t* sums, int32_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int32_t x = sums[w];
        if (w < warp) before += x;
        all += x;
    }
    __syncthreads();
    *total = all;
    return before + inc - v;
}

// One block: which forks are made (its child is named by no earlier fork and is nobody's parent),
// how many pages each shares and which fresh page takes its last, partly filled one.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) fork_plan_kernel(const __grid_constant__ ForkParams p) {
    extern __shared__ int32_t first_child[];  // [num_seqs] first fork that names the child
    __shared__ int32_t sums[kThreads / 32];
    uint32_t* parent_bits = reinterpret_cast<uint32_t*>(first_child + p.t.num_seqs);
    let_next();
    const int tid = threadIdx.x;
    const int32_t n = p.t.num_seqs;
    for (int32_t i = tid; i < n; i += kThreads) first_child[i] = INT32_MAX;
    for (int32_t i = tid; i < (n + 31) / 32; i += kThreads) parent_bits[i] = 0;
    __syncthreads();
    bool bad = false;
    for (int32_t f = tid; f < p.forks; f += kThreads) {
        const int32_t a = p.parents[f], c = p.children[f];
        if (a < 0 || c < 0) continue;
        if (a >= n || c >= n) {
            bad = true;
            continue;
        }
        atomicMin(first_child + c, f);
        atomicOr(parent_bits + (a >> 5), 1u << (a & 31));
    }
    __syncthreads();
    int32_t taken = 0, made_here = 0;
    for (int32_t f0 = 0; f0 < p.forks; f0 += kThreads) {
        const int32_t f = f0 + tid;
        int32_t src = -1, whole = -1;
        if (f < p.forks) {
            const int32_t a = p.parents[f], c = p.children[f];
            if (a >= 0 && c >= 0 && a < n && c < n) {
                if (first_child[c] != f || (parent_bits[c >> 5] >> (c & 31) & 1u)) {
                    bad = true;
                } else {
                    const int32_t len = clamped(p.t, p.t.lens[a], &bad);
                    whole = static_cast<int32_t>(divide(static_cast<uint32_t>(len), p.t.by_block));
                    ++made_here;
                    if (len > whole * p.t.block_size) {
                        src = p.t.entries[static_cast<int64_t>(a) * p.t.max_blocks + whole];
                        int32_t* mine = p.t.entries + static_cast<int64_t>(c) * p.t.max_blocks + whole;
                        if (src < 0 || src >= p.t.num_pages) {
                            *mine = src = -1;
                            bad = true;
                        }
                    }
                }
            }
        }
        int32_t total;
        const int32_t at = taken + block_scan<kThreads / 32>(src >= 0 ? 1 : 0, sums, &total);
        taken += total;
        if (f < p.forks) {
            int32_t dst = -1;
            if (src >= 0) {
                if (at < p.num_free) dst = p.free_pages[at];
                if (dst < 0 || dst >= p.t.num_pages) {
                    dst = -1;
                    bad = true;
                }
                p.t.entries[static_cast<int64_t>(p.children[f]) * p.t.max_blocks + whole] = dst;
            }
            p.src[f] = src;
            p.dst[f] = dst;
            p.whole[f] = whole;
        }
    }
    int32_t made;
    block_scan<kThreads / 32>(made_here, sums, &made);
    bad = __syncthreads_or(bad);
    if (tid == 0) {
        p.info[0] = made;
        p.info[1] = min(taken, p.num_free);
        p.info[2] = bad ? DSA_ERR_DEVICE_BOUNDS : DSA_OK;
        p.info[3] = 0;
    }
}

// Table entries of the forks' whole pages (a chunk of a row per turn), then the copied pages.
__global__ void __launch_bounds__(kCopyThreads) fork_kernel(const __grid_constant__ ForkParams p) {
    wait_prior();
    constexpr int kRow = kCopyThreads;  // entries of a turn
    const int32_t row_turns = static_cast<int32_t>((static_cast<uint32_t>(p.t.max_blocks) + kRow - 1u) / kRow);
    const int64_t turns = static_cast<int64_t>(p.forks) * row_turns;
    const uint32_t items = static_cast<uint32_t>(p.forks) * p.pools.items;
    for (int64_t it = blockIdx.x; it < turns + items; it += gridDim.x) {
        if (it < turns) {
            const int32_t f = static_cast<int32_t>(it / row_turns);
            const int32_t col = static_cast<int32_t>(it - static_cast<int64_t>(f) * row_turns) * kRow + threadIdx.x;
            if (col >= p.whole[f]) continue;
            const int32_t page = p.t.entries[static_cast<int64_t>(p.parents[f]) * p.t.max_blocks + col];
            const bool good = page >= 0 && page < p.t.num_pages;
            p.t.entries[static_cast<int64_t>(p.children[f]) * p.t.max_blocks + col] = good ? page : -1;
            if (good) atomicAdd(p.shares + page, 1);
            else report(p.info + 2);
            continue;
        }
        const uint32_t at = static_cast<uint32_t>(it - turns), f = divide(at, p.pools.by_items);
        const int32_t src = p.src[f], dst = p.dst[f];
        if (src >= 0 && dst >= 0 && src != dst) copy_chunk(p.pools, at - f * p.pools.items, src, dst);
    }
}

// ------------------------------------------------------------------------------------
// release, compact: marks
// ------------------------------------------------------------------------------------
// A warp per chunk of a request's table.
template <class F>
__device__ __forceinline__ void for_entries(const Tables& t, F&& each) {
    const int lane = threadIdx.x & 31;
    const int64_t turn = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (turn >= static_cast<int64_t>(t.num_seqs) * t.chunks) return;
    const int32_t s = static_cast<int32_t>(divide(static_cast<uint32_t>(turn), t.by_chunks));
    each(s, static_cast<int32_t>(turn - static_cast<int64_t>(s) * t.chunks) * kEntries, lane);
}

// Every reference that goes lowers its page's shares; the one that finds none left marks the page.
__global__ void __launch_bounds__(kMarkThreads) release_mark_kernel(const __grid_constant__ ReleaseParams p) {
    let_next();
    for_entries(p.t, [&](int32_t s, int32_t col0, int lane) {
        bool bad = false;
        const int32_t len = clamped(p.t, p.t.lens[s], &bad);
        int32_t keep = p.keep_lens[s];
        bad |= keep < 0;
        keep = min(max(keep, 0), len);
        const int32_t lo = pages_of(p.t, keep), hi = pages_of(p.t, len);
        int32_t* row = p.t.entries + static_cast<int64_t>(s) * p.t.max_blocks;
        int32_t refs = 0;
        if (col0 < hi && lo - col0 < kEntries) {
            int32_t page[kEntries / 32], before[kEntries / 32];
#pragma unroll
            for (int i = 0; i < kEntries / 32; ++i) {
                const int32_t col = col0 + 32 * i + lane;
                page[i] = col >= lo && col < hi ? row[col] : -1;
            }
#pragma unroll
            for (int i = 0; i < kEntries / 32; ++i) {
                const int32_t col = col0 + 32 * i + lane;
                if (col >= lo && col < hi) row[col] = -1;
                before[i] = 1;
                if (page[i] >= p.t.num_pages) {
                    bad = true;
                } else if (page[i] >= 0) {
                    ++refs;
                    before[i] = atomicSub(p.shares + page[i], 1);
                }
            }
#pragma unroll
            for (int i = 0; i < kEntries / 32; ++i) {
                if (before[i] == 0) atomicOr(p.marks + mark_at(page[i] >> 5), 1u << (page[i] & 31));
                bad |= before[i] < 0;
            }
            refs = __reduce_add_sync(0xffffffffu, refs);
            if (lane == 0 && refs > 0) atomicAdd(&p.head->refs, refs);
        }
        if (bad) report(&p.head->status);
    });
}

__global__ void __launch_bounds__(kMarkThreads) compact_mark_kernel(const __grid_constant__ CompactParams p) {
    let_next();
    for_entries(p.t, [&](int32_t s, int32_t col0, int lane) {
        bool bad = false;
        const int32_t hi = pages_of(p.t, clamped(p.t, p.t.lens[s], &bad));
        const int32_t* row = p.t.entries + static_cast<int64_t>(s) * p.t.max_blocks;
#pragma unroll
        for (int i = 0; i < kEntries / 32; ++i) {
            const int32_t col = col0 + 32 * i + lane;
            const int32_t page = col < hi ? row[col] : -1;
            if (page >= p.t.num_pages) bad = true;
            else if (page >= 0) atomicOr(p.marks + mark_at(page >> 5), 1u << (page & 31));
        }
        if (bad) report(&p.head->status);
    });
}

// ------------------------------------------------------------------------------------
// release, compact: pages in order
// ------------------------------------------------------------------------------------
// The marks of all pages are counted by every block (a bit per page: 32 KB for 262144 pages),
// which takes less time than a launch between counting and listing; a block then lists the pages
// of its own words, kBlockWords a turn, a warp eight of them. (Blocks of 1024 words, with a warp's
// words visited whether they had marks or not, took 10.9 us for 64 requests' drafts, not 6.7.)
constexpr int kBlockWords = 256;
constexpr int kWarpWords = kBlockWords / kListWarps;

// Sums of two values over the block.
__device__ __forceinline__ int2 block_sums(int a, int b, int2* sums) {
    a = __reduce_add_sync(0xffffffffu, a);
    b = __reduce_add_sync(0xffffffffu, b);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = make_int2(a, b);
    __syncthreads();
    const int2 mine = sums[threadIdx.x & 31];  // a lane for each of the 32 warps
    const int2 r = make_int2(__reduce_add_sync(0xffffffffu, mine.x), __reduce_add_sync(0xffffffffu, mine.y));
    __syncthreads();
    return r;
}
static_assert(kListWarps == 32, "a lane for each warp");

// Marked pages: x all, y those of the words before w0.
__device__ __forceinline__ int2 count_marks(const uint32_t* marks, int32_t words, int32_t w0, int2* sums) {
    int all = 0, before = 0;
    for (int32_t w = 4 * threadIdx.x; w < words; w += 4 * kListThreads) {
        const uint4 v = *reinterpret_cast<const uint4*>(marks + mark_at(w));
        const int n = __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
        all += n;
        if (w < w0) before += n;  // both multiples of 4
    }
    return block_sums(all, before, sums);
}
// Marked pages below page `limit`.
__device__ __forceinline__ int32_t count_below(const uint32_t* marks, int32_t limit, int2* sums) {
    int n = 0;
    for (int32_t w = 4 * threadIdx.x; w < (limit + 31) / 32; w += 4 * kListThreads) {
        const uint4 v = *reinterpret_cast<const uint4*>(marks + mark_at(w));
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t left = limit - (w + i) * 32;
            if (left > 0) n += __popc(left >= 32 ? x[i] : x[i] & ((1u << left) - 1u));
        }
    }
    return block_sums(n, 0, sums).x;
}

// This block's turns.
__device__ __forceinline__ int2 block_turns(int32_t words) {
    const int32_t turns = (words + kBlockWords - 1) / kBlockWords, each = (turns + gridDim.x - 1) / gridDim.x;
    const int32_t first = min(turns, static_cast<int32_t>(blockIdx.x) * each);
    return make_int2(first, min(turns, first + each));
}
// each(page, is it marked, marked pages before it) for the pages of words [w0, w0 + kBlockWords), a
// page a lane; `before` marked pages precede them. Returns the marked pages up to their end. With
// kMarked only words with marked pages are visited.
template <bool kMarked, class F>
__device__ __forceinline__ int32_t for_pages(const uint32_t* marks, int32_t w0, int32_t words, int32_t num_pages, int32_t before, F&& each) {
    __shared__ int32_t firsts[kListWarps];
    __syncthreads();  // the turn before has read them
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t base = w0 + warp * kWarpWords;
    const uint32_t mine = lane < kWarpWords && base + lane < words ? marks[mark_at(base + lane)] : 0u;
    int32_t inc = __popc(mine);
#pragma unroll
    for (int o = 1; o < kWarpWords; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == kWarpWords - 1) firsts[warp] = inc;
    __syncthreads();
    const int32_t of_warp = firsts[lane];
    const int32_t at = before + __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0) + inc - __popc(mine);
    uint32_t visit = kMarked ? __ballot_sync(0xffffffffu, mine != 0u) : (1u << kWarpWords) - 1u;
    while (visit != 0u) {
        const int j = __ffs(visit) - 1;
        visit &= visit - 1u;
        const uint32_t bits = __shfl_sync(0xffffffffu, mine, j);
        const int32_t first = __shfl_sync(0xffffffffu, at, j);
        const int32_t page = (base + j) * 32 + lane;
        if (page < num_pages) each(page, (bits >> lane & 1u) != 0u, first + __popc(bits & ((1u << lane) - 1u)));
    }
    return before + __reduce_add_sync(0xffffffffu, of_warp);
}

// Whether this block is the last one to come here.
__device__ __forceinline__ bool last_block(int32_t* ticket) {
    __shared__ bool last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(ticket, 1) == static_cast<int32_t>(gridDim.x) - 1;
        __threadfence();
    }
    __syncthreads();
    return last;
}

__global__ void __launch_bounds__(kListThreads) release_list_kernel(const __grid_constant__ ReleaseParams p) {
    __shared__ int2 sums[kListWarps];
    wait_prior();
    const int32_t words = static_cast<int32_t>((static_cast<int64_t>(p.t.num_pages) + 127) / 128 * 4);
    const int2 turns = block_turns(words);
    const int32_t had = *p.num_free, want = p.taken ? *p.taken : 0;  // on their way beside the marks
    const int2 counts = count_marks(p.marks, words, turns.x * kBlockWords, sums);
    const int32_t freed = counts.x;
    int32_t before = counts.y;
    const int32_t count = min(max(had, 0), p.t.num_pages), taken = min(max(want, 0), count);
    bool bad = had != count || want != taken;
    const int64_t after = static_cast<int64_t>(count) - taken + freed;
    const int32_t now = static_cast<int32_t>(min(after, static_cast<int64_t>(p.t.num_pages)));
    bad |= now != after;
    for (int32_t turn = turns.x; turn < turns.y; ++turn)
        before = for_pages<true>(p.marks, turn * kBlockWords, words, p.t.num_pages, before, [&](int32_t page, bool mine, int32_t k) {
            if (!mine) return;
            p.shares[page] = 0;
            const int64_t at = k < taken ? k : static_cast<int64_t>(count) - taken + k;
            if (at < p.t.num_pages) p.free_pages[at] = page;
        });
    if (blockIdx.x == 0) {
        const int32_t gap = max(0, taken - freed), moved = min(gap, count - taken);
        for (int32_t i = threadIdx.x; i < moved; i += kListThreads) p.free_pages[freed + i] = p.free_pages[count - moved + i];
        __syncthreads();
        for (int32_t i = now + threadIdx.x; i < count; i += kListThreads) p.free_pages[i] = -1;
    }
    if (!last_block(&p.head->ticket)) return;
    for (int32_t w = 4 * threadIdx.x; w < words; w += 4 * kListThreads) *reinterpret_cast<uint4*>(p.marks + mark_at(w)) = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) {
        p.info[0] = p.head->refs;
        p.info[1] = freed;
        p.info[2] = bad || p.head->status != 0 ? DSA_ERR_DEVICE_BOUNDS : DSA_OK;
        p.info[3] = now;
        *p.num_free = now;
        p.head->refs = p.head->status = p.head->ticket = 0;
    }
}

// Pages from the number of live ones on that are live move, in order, to the dead ones below it.
__global__ void __launch_bounds__(kListThreads) compact_list_kernel(const __grid_constant__ CompactParams p) {
    __shared__ int2 sums[kListWarps];
    wait_prior();
    let_next();
    const int32_t words = static_cast<int32_t>((static_cast<int64_t>(p.t.num_pages) + 127) / 128 * 4);
    const int2 turns = block_turns(words);
    const int2 counts = count_marks(p.marks, words, turns.x * kBlockWords, sums);
    const int32_t live = counts.x, low = count_below(p.marks, live, sums);  // of them, those that stay
    int32_t before = counts.y;
    for (int32_t turn = turns.x; turn < turns.y; ++turn)
        before = for_pages<false>(p.marks, turn * kBlockWords, words, p.t.num_pages, before, [&](int32_t page, bool mine, int32_t k) {
            if (page >= live) {
                if (mine) {
                    p.rank[entry_at(page)] = k - low;
                    p.src[entry_at(k - low)] = page;
                } else {
                    p.shares[page] = 0;
                }
            } else if (!mine) {
                p.dst[entry_at(page - k)] = page;
            }
            p.free_pages[page] = page < p.t.num_pages - live ? page + live : -1;
        });
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.head->live = live;
        p.head->moved = live - low;
        p.info[0] = live;
        p.info[1] = live - low;
        p.info[2] = p.head->status;
        p.head->status = 0;
        p.info[3] = p.t.num_pages - live;
        *p.num_free = p.t.num_pages - live;
    }
}

// Shares, table entries and data of the pages that move; the marks are cleared for the next call.
__global__ void __launch_bounds__(kCopyThreads) compact_kernel(const __grid_constant__ CompactParams p) {
    wait_prior();
    const int32_t live = p.head->live, moved = p.head->moved;
    const int64_t tid = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x, threads = static_cast<int64_t>(gridDim.x) * kCopyThreads;
    const int64_t words = (static_cast<int64_t>(p.t.num_pages) + 127) / 128 * 4;
    for (int64_t w = tid; w < words; w += threads) p.marks[mark_at(w)] = 0;
    for (int64_t k = tid; k < moved; k += threads) {
        const int32_t src = p.src[entry_at(k)];
        p.shares[p.dst[entry_at(k)]] = p.shares[src];
        p.shares[src] = 0;
    }
    if (moved > 0) {
        const int64_t turns = static_cast<int64_t>(p.t.num_seqs) * p.t.chunks;
        const int lane = threadIdx.x & 31;
        for (int64_t turn = tid >> 5; turn < turns; turn += threads >> 5) {
            const int32_t s = static_cast<int32_t>(divide(static_cast<uint32_t>(turn), p.t.by_chunks));
            const int32_t col0 = static_cast<int32_t>(turn - static_cast<int64_t>(s) * p.t.chunks) * kEntries;
            bool bad = false;
            const int32_t hi = pages_of(p.t, clamped(p.t, p.t.lens[s], &bad));
            int32_t* row = p.t.entries + static_cast<int64_t>(s) * p.t.max_blocks;
#pragma unroll
            for (int i = 0; i < kEntries / 32; ++i) {
                const int32_t col = col0 + 32 * i + lane;
                const int32_t page = col < hi ? row[col] : -1;
                if (page >= live && page < p.t.num_pages) row[col] = p.dst[entry_at(p.rank[entry_at(page)])];
            }
        }
        const uint64_t items = static_cast<uint64_t>(moved) * p.pools.items;
        for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
            const uint32_t k = divide(static_cast<uint32_t>(it), p.pools.by_items);
            copy_chunk(p.pools, static_cast<uint32_t>(it) - k * p.pools.items, p.src[entry_at(k)], p.dst[entry_at(k)]);
        }
    }
}

template <class P>
cudaError_t launch_after(void (*kernel)(P), int blocks, int threads, const P& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

int at_most(int64_t want, int most) { return static_cast<int>(want < 1 ? 1 : (want < most ? want : most)); }
int mark_blocks(const Tables& t) {
    return at_most((static_cast<int64_t>(t.num_seqs) * t.chunks + kMarkThreads / 32 - 1) / (kMarkThreads / 32), INT32_MAX);
}
// No more blocks than run at once: each reads all marks.
int list_blocks(const Tables& t, int sms) { return at_most((mark_words(t.num_pages) + kBlockWords - 1) / kBlockWords, sms); }

}  // namespace
}  // namespace pages

cudaError_t pages_setup() {
    const int smem = DSA_MAX_PLAN_SEQS * 4 + DSA_MAX_PLAN_SEQS / 8;
    const cudaError_t e = cudaFuncSetAttribute(pages::fork_plan_kernel<pages::kManyForkThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(pages::fork_plan_kernel<pages::kForkThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

cudaError_t launch_copy_pages(const pages::CopyParams& p, int sms, cudaStream_t stream) {
    const int blocks = pages::at_most(static_cast<int64_t>(p.count) * p.pools.items, 8 * sms);
    pages::copy_kernel<<<blocks, pages::kCopyThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_fork_pages(const pages::ForkParams& p, int sms, cudaStream_t stream) {
    const int smem = p.t.num_seqs * 4 + (p.t.num_seqs + 31) / 32 * 4;
    if (p.forks <= pages::kFewForks) pages::fork_plan_kernel<pages::kForkThreads><<<1, pages::kForkThreads, smem, stream>>>(p);
    else pages::fork_plan_kernel<pages::kManyForkThreads><<<1, pages::kManyForkThreads, smem, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t turns = (static_cast<int64_t>(p.t.max_blocks) + pages::kCopyThreads - 1) / pages::kCopyThreads;
    return pages::launch_after(pages::fork_kernel, pages::at_most(p.forks * (turns + p.pools.items), 8 * sms), pages::kCopyThreads, p, stream);
}

cudaError_t launch_release_pages(const pages::ReleaseParams& p, int sms, cudaStream_t stream) {
    pages::release_mark_kernel<<<pages::mark_blocks(p.t), pages::kMarkThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return pages::launch_after(pages::release_list_kernel, pages::list_blocks(p.t, sms), pages::kListThreads, p, stream);
}

cudaError_t launch_compact_pages(const pages::CompactParams& p, int sms, cudaStream_t stream) {
    pages::compact_mark_kernel<<<pages::mark_blocks(p.t), pages::kMarkThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        e = pages::launch_after(pages::compact_list_kernel, pages::list_blocks(p.t, sms), pages::kListThreads, p, stream);
    if (e != cudaSuccess) return e;
    return pages::launch_after(pages::compact_kernel, 8 * sms, pages::kCopyThreads, p, stream);
}

}  // namespace dsa
