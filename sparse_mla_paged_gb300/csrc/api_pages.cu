// Host side of the page operators declared in include/dsa_mla.h: argument checks and launches.
#include "pages.cuh"

using namespace dsa;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int32_t from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return DSA_OK;
    return e == cudaErrorNoKernelImageForDevice || e == cudaErrorInvalidDeviceFunction ? DSA_ERR_NO_KERNEL : DSA_ERR_CUDA;
}

// pairs: the most pages that one call copies.
int32_t make_pools(const dsa_page_pool* given, int32_t count, int64_t pairs, pages::Pools* out) {
    if (!given || count < 1) return DSA_ERR_INVALID_ARGUMENT;
    if (count > DSA_MAX_PAGE_POOLS) return DSA_ERR_UNSUPPORTED;
    uint64_t items = 0;
    for (int32_t i = 0; i < count; ++i) {
        const dsa_page_pool& g = given[i];
        if (!g.base || !aligned(g.base, 16) || g.layers < 1 || g.reserved != 0 || g.page_bytes < 16 || g.page_bytes % 16 != 0 ||
            g.page_stride_bytes % 16 != 0 || g.page_stride_bytes < g.page_bytes)
            return DSA_ERR_INVALID_ARGUMENT;
        if (g.layers > 1 && (g.layer_stride_bytes % 16 != 0 || g.layer_stride_bytes < g.page_bytes)) return DSA_ERR_INVALID_ARGUMENT;
        if (g.page_bytes / 16 > INT32_MAX) return DSA_ERR_UNSUPPORTED;
        pages::Pool& p = out->pool[i];
        p.base = static_cast<uint8_t*>(g.base);
        p.page_stride = g.page_stride_bytes;
        p.layer_stride = g.layers > 1 ? g.layer_stride_bytes : 0;
        p.vecs = static_cast<uint32_t>(g.page_bytes / 16);
        p.first = static_cast<uint32_t>(items);
        const uint32_t chunks = (p.vecs + pages::kChunkVecs - 1) / pages::kChunkVecs;
        p.by_chunks = fast_div(chunks);
        items += static_cast<uint64_t>(chunks) * static_cast<uint32_t>(g.layers);
        if (items > UINT32_MAX) return DSA_ERR_UNSUPPORTED;
    }
    if (pairs > 0 && items > UINT32_MAX / static_cast<uint64_t>(pairs)) return DSA_ERR_UNSUPPORTED;
    out->count = count;
    out->items = static_cast<uint32_t>(items);
    out->by_items = fast_div(out->items);
    return DSA_OK;
}

constexpr int32_t kMaxPages = 1 << 30;

int32_t make_tables(int32_t* entries, int32_t max_blocks, const int32_t* lens, int32_t num_seqs, int32_t block_size, int32_t num_pages,
                    pages::Tables* t) {
    if (num_seqs < 0 || block_size < 1 || max_blocks < 1 || num_pages < 1) return DSA_ERR_INVALID_ARGUMENT;
    if (num_seqs > 0 && (!entries || !lens)) return DSA_ERR_INVALID_ARGUMENT;
    if (!aligned(entries, 4) || !aligned(lens, 4)) return DSA_ERR_INVALID_ARGUMENT;
    const int64_t chunks = (static_cast<int64_t>(max_blocks) + pages::kEntries - 1) / pages::kEntries;
    if (num_seqs > DSA_MAX_PLAN_SEQS || num_pages > kMaxPages || static_cast<int64_t>(max_blocks) * block_size > INT32_MAX ||
        chunks * num_seqs > INT32_MAX)
        return DSA_ERR_UNSUPPORTED;
    t->entries = entries;
    t->lens = lens;
    t->num_seqs = num_seqs;
    t->max_blocks = max_blocks;
    t->block_size = block_size;
    t->chunks = static_cast<int32_t>(chunks);
    t->num_pages = num_pages;
    t->by_block = fast_div(static_cast<uint32_t>(block_size));
    t->by_chunks = fast_div(static_cast<uint32_t>(chunks));
    return DSA_OK;
}

int32_t check_workspace(const void* workspace, size_t bytes, int32_t num_pages) {
    if (!workspace || !aligned(workspace, 256)) return DSA_ERR_INVALID_ARGUMENT;
    return bytes < pages::layout(num_pages).total ? DSA_ERR_WORKSPACE : DSA_OK;
}

}  // namespace

extern "C" {

size_t dsa_pages_workspace_bytes(int32_t num_pages) {
    return num_pages < 1 || num_pages > kMaxPages ? 0 : pages::layout(num_pages).total;
}

int32_t dsa_copy_pages(const dsa_page_pool* pools, int32_t num_pools, const int32_t* src_pages, const int32_t* dst_pages,
                       int32_t count, int32_t num_pages, void* stream) {
    pages::CopyParams p{};
    if (count < 0 || num_pages < 1 || (count > 0 && (!src_pages || !dst_pages)) || !aligned(src_pages, 4) || !aligned(dst_pages, 4))
        return DSA_ERR_INVALID_ARGUMENT;
    int32_t st = make_pools(pools, num_pools, count, &p.pools);
    if (st != DSA_OK || count == 0) return st;
    int sms = 0;
    st = device_info(&sms, &p.status);
    if (st != DSA_OK) return st;
    p.src = src_pages;
    p.dst = dst_pages;
    p.count = count;
    p.num_pages = num_pages;
    return from_cuda(launch_copy_pages(p, sms, static_cast<cudaStream_t>(stream)));
}

int32_t dsa_fork_pages(const dsa_page_pool* pools, int32_t num_pools, const int32_t* parents, const int32_t* children,
                       int32_t num_forks, const int32_t* lens, int32_t num_seqs, int32_t block_size, int32_t* block_tables,
                       int32_t max_blocks_per_seq, const int32_t* free_pages, int32_t num_free, int32_t* page_shares,
                       int32_t num_pages, int32_t* info, void* workspace, size_t workspace_bytes, void* stream) {
    pages::ForkParams p{};
    if (num_forks < 0 || num_free < 0 || !info || !page_shares || (num_forks > 0 && (!parents || !children)) ||
        (num_free > 0 && !free_pages))
        return DSA_ERR_INVALID_ARGUMENT;
    if (!aligned(parents, 4) || !aligned(children, 4) || !aligned(free_pages, 4) || !aligned(page_shares, 4) || !aligned(info, 4))
        return DSA_ERR_INVALID_ARGUMENT;
    int32_t st = make_tables(block_tables, max_blocks_per_seq, lens, num_seqs, block_size, num_pages, &p.t);
    if (st == DSA_OK && num_forks > DSA_MAX_PLAN_SEQS) st = DSA_ERR_UNSUPPORTED;
    if (st == DSA_OK) st = make_pools(pools, num_pools, num_forks, &p.pools);
    if (st == DSA_OK) st = check_workspace(workspace, workspace_bytes, num_pages);
    int sms = 0;
    int* unused = nullptr;
    if (st == DSA_OK) st = device_info(&sms, &unused);
    if (st != DSA_OK) return st;
    const pages::Layout L = pages::layout(num_pages);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.parents = parents;
    p.children = children;
    p.free_pages = free_pages;
    p.shares = page_shares;
    p.info = info;
    p.src = reinterpret_cast<int32_t*>(ws + L.src);
    p.dst = reinterpret_cast<int32_t*>(ws + L.dst);
    p.whole = reinterpret_cast<int32_t*>(ws + L.rank);
    p.forks = num_forks;
    p.num_free = num_free;
    return from_cuda(launch_fork_pages(p, sms, static_cast<cudaStream_t>(stream)));
}

int32_t dsa_release_pages(int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* lens, const int32_t* keep_lens,
                          int32_t num_seqs, int32_t block_size, int32_t* page_shares, int32_t num_pages, int32_t* free_pages,
                          int32_t* num_free, const int32_t* taken, int32_t* info, void* workspace, size_t workspace_bytes,
                          void* stream) {
    pages::ReleaseParams p{};
    if (!page_shares || !free_pages || !num_free || !info || (num_seqs > 0 && !keep_lens)) return DSA_ERR_INVALID_ARGUMENT;
    if (!aligned(keep_lens, 4) || !aligned(page_shares, 4) || !aligned(free_pages, 4) || !aligned(num_free, 4) ||
        !aligned(taken, 4) || !aligned(info, 4))
        return DSA_ERR_INVALID_ARGUMENT;
    int32_t st = make_tables(block_tables, max_blocks_per_seq, lens, num_seqs, block_size, num_pages, &p.t);
    if (st == DSA_OK) st = check_workspace(workspace, workspace_bytes, num_pages);
    int sms = 0;
    int* unused = nullptr;
    if (st == DSA_OK) st = device_info(&sms, &unused);
    if (st != DSA_OK) return st;
    const pages::Layout L = pages::layout(num_pages);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.keep_lens = keep_lens;
    p.taken = taken;
    p.shares = page_shares;
    p.free_pages = free_pages;
    p.num_free = num_free;
    p.info = info;
    p.head = reinterpret_cast<pages::Head*>(ws);
    p.marks = reinterpret_cast<uint32_t*>(ws + L.marks);
    return from_cuda(launch_release_pages(p, sms, static_cast<cudaStream_t>(stream)));
}

int32_t dsa_compact_pages(const dsa_page_pool* pools, int32_t num_pools, int32_t* block_tables, int32_t max_blocks_per_seq,
                          const int32_t* lens, int32_t num_seqs, int32_t block_size, int32_t* page_shares, int32_t num_pages,
                          int32_t* free_pages, int32_t* num_free, int32_t* info, void* workspace, size_t workspace_bytes,
                          void* stream) {
    pages::CompactParams p{};
    if (!page_shares || !free_pages || !num_free || !info) return DSA_ERR_INVALID_ARGUMENT;
    if (!aligned(page_shares, 4) || !aligned(free_pages, 4) || !aligned(num_free, 4) || !aligned(info, 4))
        return DSA_ERR_INVALID_ARGUMENT;
    int32_t st = make_tables(block_tables, max_blocks_per_seq, lens, num_seqs, block_size, num_pages, &p.t);
    if (st == DSA_OK) st = make_pools(pools, num_pools, num_pages, &p.pools);
    if (st == DSA_OK) st = check_workspace(workspace, workspace_bytes, num_pages);
    int sms = 0;
    int* unused = nullptr;
    if (st == DSA_OK) st = device_info(&sms, &unused);
    if (st != DSA_OK) return st;
    const pages::Layout L = pages::layout(num_pages);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.shares = page_shares;
    p.free_pages = free_pages;
    p.num_free = num_free;
    p.info = info;
    p.head = reinterpret_cast<pages::Head*>(ws);
    p.marks = reinterpret_cast<uint32_t*>(ws + L.marks);
    p.rank = reinterpret_cast<int32_t*>(ws + L.rank);
    p.src = reinterpret_cast<int32_t*>(ws + L.src);
    p.dst = reinterpret_cast<int32_t*>(ws + L.dst);
    return from_cuda(launch_compact_pages(p, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
