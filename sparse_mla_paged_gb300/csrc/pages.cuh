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

struct Layout {
    size_t marks, rank, src, dst, total;
};
// Marks are a bit per page, in whole 16-byte pieces.
inline int64_t mark_words(int64_t pages) { return (pages + 127) / 128 * 4; }
inline Layout layout(int64_t pages) {
    Layout L;
    size_t o = 256;
    auto put = [&](size_t bytes) {
        const size_t at = o;
        o = align256(o + bytes);
        return at;
    };
    L.marks = put(static_cast<size_t>(mark_words(pages)) * 4);
    // Lists by page or by fork.
    const size_t list = static_cast<size_t>(pages > DSA_MAX_PLAN_SEQS ? pages : DSA_MAX_PLAN_SEQS) * 4;
    L.rank = put(list);
    L.src = put(list);
    L.dst = put(list);
    L.total = o;
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
    uint32_t* marks;
};

struct CompactParams {
    Pools pools;
    Tables t;
    int32_t* shares;
    int32_t* free_pages;
    int32_t* num_free;
    int32_t* info;
    Head* head;
    uint32_t* marks;
    int32_t* rank;            // [num_pages] number of a page that moves
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
