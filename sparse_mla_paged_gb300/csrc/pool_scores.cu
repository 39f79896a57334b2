// Pooled index scores: the cheap score by which the selector ranks the pools of each row.
//
//   I[r,j]     = s_j * sum_h w[r,h] * max(0, q[r,h,:] . k_j)       (k_j, s_j: index cache)
//   score[r,p] = max over the kpool tokens j of pool p of I[r,j], and -inf unless the whole
//                pool lies at or before the row's position q_pos[r]
//
// One block per (row, stretch of whole pools, at most 128 tokens): a thread takes a token,
// its key in registers, the row's queries as float32 in shared memory; the pools' maxima are
// formed in shared memory.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace dsa {
namespace {

constexpr int kScoreThreads = 128;

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__global__ void __launch_bounds__(kScoreThreads) pool_scores_kernel(const PoolScoresParams p, int32_t chunks) {
    extern __shared__ __align__(16) float q_s[];  // [heads][128], then w[heads]
    __shared__ float token_s[kScoreThreads];
    const int tid = threadIdx.x;
    const int32_t r = static_cast<int32_t>(blockIdx.x / chunks), chunk = static_cast<int32_t>(blockIdx.x % chunks);
    const int32_t seq = r / p.rows_per_seq;
    const int32_t per = kScoreThreads / p.kpool;  // pools of a stretch
    const int32_t pool0 = chunk * per;
    const int64_t q_pos = p.q_pos[r];
    const int64_t n = q_pos < 0 ? 0 : min((q_pos + 1) / p.kpool, static_cast<int64_t>(p.n_pools));  // visible pools: [0, n)
    const int32_t seen = static_cast<int32_t>(min(max(n - pool0, int64_t{0}), static_cast<int64_t>(per)));
    float* w_s = q_s + p.heads * kIndexDim;
    if (seen > 0) {
        for (int i = tid; i < p.heads * kIndexDim; i += kScoreThreads) {
            const float x = __uint_as_float(static_cast<uint32_t>(p.q[static_cast<int64_t>(r) * p.heads * kIndexDim + i]) << 16);
            q_s[i] = isinf(x) ? __uint_as_float(0x7FC00000u) : x;
        }
        for (int i = tid; i < p.heads; i += kScoreThreads) w_s[i] = p.w[static_cast<int64_t>(r) * p.heads + i];
    }
    __syncthreads();
    float score = -__builtin_huge_valf();
    if (tid < seen * p.kpool) {
        const int64_t pos = static_cast<int64_t>(pool0) * p.kpool + tid;
        const int64_t blk = pos / p.block_size, off = pos % p.block_size;
        const int32_t page = (p.max_blocks_per_seq == 0 || blk < p.max_blocks_per_seq)
                                 ? p.block_tables[static_cast<int64_t>(seq) * p.max_blocks_per_seq + blk] : -1;
        if (page < 0) {
            if (p.status) atomicCAS(p.status, 0, kStatusBounds);
        } else {
            const uint8_t* at = p.cache + page * p.page_stride;
            float k[kIndexDim];
#pragma unroll
            for (int i = 0; i < kIndexDim / 16; ++i) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(at + off * kIndexDim) + i);
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int b = 0; b < 16; ++b)
                    k[16 * i + b] = __half2float(__half(__nv_cvt_fp8_to_halfraw((u[b >> 2] >> (8 * (b & 3))) & 255u, __NV_E4M3)));
            }
            float sum = 0.0f;
            for (int h = 0; h < p.heads; ++h) {
                float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
                for (int i = 0; i < kIndexDim; i += 2) {
                    d0 = fmaf(q_s[h * kIndexDim + i], k[i], d0);
                    d1 = fmaf(q_s[h * kIndexDim + i + 1], k[i + 1], d1);
                }
                sum = fmaf(w_s[h], max_nan(d0 + d1, 0.0f), sum);
            }
            score = sum * reinterpret_cast<const float*>(at + static_cast<int64_t>(p.block_size) * kIndexDim)[off];
        }
    }
    token_s[tid] = score;
    __syncthreads();
    if (tid < per && pool0 + tid < p.n_pools) {
        float best = -__builtin_huge_valf();
        for (int i = 0; i < p.kpool; ++i) best = max_nan(best, token_s[tid * p.kpool + i]);
        p.scores[static_cast<int64_t>(r) * p.n_pools + pool0 + tid] = best;
    }
}

}  // namespace

cudaError_t pool_scores_kernel_setup() {
    return cudaFuncSetAttribute(pool_scores_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                DSA_MAX_INDEX_HEADS * (kIndexDim + 1) * 4);
}

cudaError_t launch_pool_scores(const PoolScoresParams& p, cudaStream_t stream) {
    const int32_t per = kScoreThreads / p.kpool;
    const int32_t chunks = (p.n_pools + per - 1) / per;
    const int64_t blocks = static_cast<int64_t>(chunks) * p.num_seqs * p.rows_per_seq;
    pool_scores_kernel<<<static_cast<unsigned>(blocks), kScoreThreads, p.heads * (kIndexDim + 1) * 4, stream>>>(p, chunks);
    return cudaGetLastError();
}

}  // namespace dsa
