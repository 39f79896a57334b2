// Shared by the prompt-chunk attention's kernels and its host side.
#pragma once

#include "common.cuh"

namespace dsa {
namespace prefill {

struct Layout {
    size_t status, total;
};
inline Layout layout() { return {0, 256}; }

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
    int64_t cache_stride;
    int32_t num_seqs, max_rows, heads, block_size, max_blocks_per_seq;
    FastDiv by_block;          // block_size
    float score_scale;         // sm_scale * k_scale * log2(e)
    float v_scale;
    uint64_t wait_limit_ns;
};

}  // namespace prefill

cudaError_t launch_prefill(const prefill::Params& p, cudaStream_t stream);

}  // namespace dsa
