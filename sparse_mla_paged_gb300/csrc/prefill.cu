// Attention of packed prompt chunks over their paged latent caches: row t of request s, its i-th
// new token, sees the positions below base[s] + i + 1.
//
//   out[t,h,:] = sum_{j < base[s]+i+1} softmax_j(sm_scale * q[t,h,:] . (k_scale*K_j)) (v_scale*V_j)
//
// A block per row and eight heads, a warp per head, a lane per 16 dims; one pass over the tokens
// with a running maximum and sum in FP32.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "prefill.cuh"

namespace dsa {
namespace prefill {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void report(const Params& p) {
    atomicCAS(p.status, 0, kStatusBounds);
    atomicCAS(p.step_status, 0, kStatusBounds);
}

__device__ __forceinline__ void decode16(const uint4& c, float (&v)[16]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        __nv_fp8_e4m3 f;
        f.__x = static_cast<__nv_fp8_storage_t>(w[i >> 2] >> (8 * (i & 3)));
        v[i] = static_cast<float>(f);
    }
}

__global__ void __launch_bounds__(kThreads) prefill_kernel(const Params p) {
    __shared__ int32_t seq_s, row_s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x;
    if (threadIdx.x == 0) {
        int64_t at = 0;
        int32_t s = 0;
        for (; s < p.num_seqs; ++s) {
            const int32_t n = max(p.new_lens[s], 0);
            if (row < at + n) break;
            at += n;
        }
        seq_s = s;
        row_s = static_cast<int32_t>(row - at);
        if (blockIdx.y == 0) {
            if (s < p.num_seqs) {
                if (p.base_lens[s] < 0 || p.new_lens[s] < 0) report(p);
            } else if (row == 0 || row == p.max_rows - 1) {
                for (int32_t i = 0; i < p.num_seqs; ++i)
                    if (p.new_lens[i] < 0) report(p);
            }
            if (row == p.max_rows - 1) {
                int64_t all = 0;
                for (int32_t i = 0; i < p.num_seqs; ++i) all += max(p.new_lens[i], 0);
                if (all > p.max_rows) report(p);
            }
        }
    }
    __syncthreads();
    const int32_t seq = seq_s, h = blockIdx.y * (kThreads / 32) + warp;
    if (seq >= p.num_seqs || h >= p.heads) return;
    int64_t len = static_cast<int64_t>(max(p.base_lens[seq], 0)) + row_s + 1;
    const int64_t room = p.max_blocks_per_seq > 0 ? static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size : INT32_MAX - 256;
    if (len > room) {
        len = room;
        if (lane == 0) report(p);
    }
    const int64_t at = (row * p.heads + h) * kLatent + lane * 16;
    float q[16], o[16] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = __uint_as_float(static_cast<uint32_t>(p.q[at + i]) << 16);
    float m = -INFINITY, l = 0.0f;
    for (int32_t j = 0; j < len; ++j) {
        const uint32_t blk = divide(j, p.by_block);
        const int32_t page = p.block_tables[static_cast<int64_t>(seq) * p.max_blocks_per_seq + blk];
        uint4 kc = make_uint4(0, 0, 0, 0), vc = kc;
        if (page >= 0) {
            const int64_t off = page * p.cache_stride + static_cast<int64_t>(j - blk * p.block_size) * kLatent + lane * 16;
            kc = *reinterpret_cast<const uint4*>(p.k_cache + off);
            vc = *reinterpret_cast<const uint4*>(p.v_cache + off);
        } else if (lane == 0) {
            report(p);
        }
        float k[16], dot = 0.0f;
        decode16(kc, k);
#pragma unroll
        for (int i = 0; i < 16; ++i) dot = fmaf(q[i], k[i], dot);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
        const float s = dot * p.score_scale, top = fmaxf(m, s);
        const float a = exp2f(m - top), e = exp2f(s - top);
        m = top;
        l = fmaf(l, a, e);
        decode16(vc, k);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = fmaf(o[i], a, e * k[i]);
    }
    const float f = p.v_scale / l;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const __nv_bfloat16 b = __float2bfloat16_rn(len > 0 ? o[i] * f : 0.0f);
        p.out[at + i] = __bfloat16_as_ushort(b);
    }
}

}  // namespace
}  // namespace prefill

cudaError_t launch_prefill(const prefill::Params& p, cudaStream_t stream) {
    cudaError_t e = cudaMemsetAsync(p.status, 0, 4, stream);
    if (e != cudaSuccess) return e;
    const dim3 grid(p.max_rows, (p.heads + prefill::kThreads / 32 - 1) / (prefill::kThreads / 32));
    prefill::prefill_kernel<<<grid, prefill::kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dsa
