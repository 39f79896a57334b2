// Shared by the page operators (pages.cu, api_pages.cu): pools, workspace and parameters.
//
// A page is named by one number in every pool (latent cache, index cache, ...) and every layer. A
// request's references to pages are its block-table entries; page_shares[p] counts the requests
// that share page p beyond the one that an unshared page belongs to, so the step plan, which takes
// pages that nobody shares, has nothing to write there.
#pragma once

#include "common.cuh"

namespace dsa {
namespace pages {

constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;                                // 16-byte pieces in flight per thread
constexpr uint32_t kChunkVecs = kCopyThreads * kCopyVecs;   // of a page: 16 KB
constexpr int kEntries = 128;                               // table entries of a warp's turn

struct Pool {
    uint8_t* base;
    int64_t page_stride, layer_stride;
    uint32_t vecs;       // 16-byte pieces of a page
    uint32_t first;      // its first item among a page's
    FastDiv by_chunks;   // chunks of a page in one layer
};
struct Pools {
    Pool pool[DSA_MAX_PAGE_POOLS];
    int32_t count;
    uint32_t items;      // chunks of one page in all pools and layers
    FastDiv by_items;
};

// Words at the workspace's start. refs, status, ticket and the marks are 0 between calls.
struct Head {
    int32_t refs;        // references given back
    int32_t status;
    int32_t ticket;      // blocks that are done
    int32_t live, moved;
};

// Workspace: the head, then segments of kSegment pages each: their marks, then their entries of three
// lists. Where a page's mark and entries lie does not depend on how many pages a call has, so that
// calls on pools of different sizes may take turns with one workspace: no list's entry ever lies
// where a mark is expected to be zero.
constexpr uint32_t kSegment = 1 << 14;
constexpr uint32_t kSegmentMarks = kSegment / 32;
constexpr uint32_t kSegmentWords = kSegmentMarks + 3 * kSegment;
static_assert(kSegment >= DSA_MAX_PLAN_SEQS, "a fork's lists lie in the first segment");
static_assert(kSegmentMarks % 4 == 0 && kSegmentWords % 4 == 0, "whole 16-byte pieces");

// Place of mark word w behind the first one, and of a list's entry i behind its first (below 2^32 for 2^30 pages).
__host__ __device__ inline uint32_t mark_at(uint32_t w) { return w / kSegmentMarks * kSegmentWords + w % kSegmentMarks; }
__host__ __device__ inline uint32_t entry_at(uint32_t i) { return i / kSegment * kSegmentWords + i % kSegment; }

// Marks are a bit per page, in whole 16-byte pieces.
inline int64_t mark_words(int64_t pages) { return (pages + 127) / 128 * 4; }
struct Layout {
    size_t marks, rank, src, dst, total;
};
inline Layout layout(int64_t pages) {
    Layout L;
    L.marks = 256;
    L.rank = L.marks + kSegmentMarks * 4;
    L.src = L.rank + kSegment * 4;
    L.dst = L.src + kSegment * 4;
    L.total = L.marks + static_cast<size_t>((pages + kSegment - 1) / kSegment) * kSegmentWords * 4;
    return L;
}

// The requests' tables, as every operator takes them.
struct Tables {
    int32_t* entries;      // [num_seqs, max_blocks]
    const int32_t* lens;   // [num_seqs]
    int32_t num_seqs, max_blocks, block_size, chunks;  // chunks of kEntries in a row
    int32_t num_pages;
    FastDiv by_block, by_chunks;
};

struct CopyParams {
    Pools pools;
    const int32_t* src;    // [count]
    const int32_t* dst;
    int32_t count, num_pages;
    int* status;
};

struct ForkParams {
    Pools pools;
    Tables t;
    const int32_t* parents;   // [forks]
    const int32_t* children;
    const int32_t* free_pages;
    int32_t* shares;          // [num_pages]
    int32_t* info;
    int32_t* src;             // workspace: each fork's copied page (-1: none), [forks] by src and dst
    int32_t* dst;
    int32_t* whole;           // workspace: shared pages of each fork, -1: not made
    int32_t forks, num_free;
};

struct ReleaseParams {
    Tables t;
    const int32_t* keep_lens;
    const int32_t* taken;     // or null
    int32_t* shares;
    int32_t* free_pages;      // [num_pages]
    int32_t* num_free;
    int32_t* info;
    Head* head;
    uint32_t* marks;          // mark_at
};

struct CompactParams {
    Pools pools;
    Tables t;
    int32_t* shares;
    int32_t* free_pages;
    int32_t* num_free;
    int32_t* info;
    Head* head;
    uint32_t* marks;          // mark_at
    int32_t* rank;            // [num_pages] number of a page that moves (entry_at, as the next two)
    int32_t* src;             // [moved]
    int32_t* dst;
};

}  // namespace pages

cudaError_t pages_setup();
cudaError_t launch_copy_pages(const pages::CopyParams& p, int sms, cudaStream_t stream);
cudaError_t launch_fork_pages(const pages::ForkParams& p, int sms, cudaStream_t stream);
cudaError_t launch_release_pages(const pages::ReleaseParams& p, int sms, cudaStream_t stream);
cudaError_t launch_compact_pages(const pages::CompactParams& p, int sms, cudaStream_t stream);

}  // namespace dsa
