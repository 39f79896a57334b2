// Attention of each decode row over its whole paged latent cache (no selection):
//
//   out[r,h,:] = sum_{j < len(r)} softmax_j(sm_scale * q[r,h,:] . (k_scale*K_j)) (v_scale*V_j)
//
// One warp per (row, head): lane l holds dims 16l .. 16l+15 of the query and of the running
// weighted sum, and walks the row's tokens with a running maximum and sum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace dsa {
namespace {

constexpr int kFullWarps = 4;

__device__ __forceinline__ void decode16(const uint4 v, float* f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int b = 0; b < 16; ++b)
        f[b] = __half2float(__half(__nv_cvt_fp8_to_halfraw((u[b >> 2] >> (8 * (b & 3))) & 255u, __NV_E4M3)));
}

__global__ void __launch_bounds__(kFullWarps * 32) full_kernel(const FullParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t rh = static_cast<int64_t>(blockIdx.x) * kFullWarps + (threadIdx.x >> 5);
    if (rh >= static_cast<int64_t>(p.num_seqs) * p.rows_per_seq * p.heads) return;
    const int64_t r = rh / p.heads, seq = r / p.rows_per_seq;
    const int64_t given = p.verify_rows ? static_cast<int64_t>(p.seq_lens[seq]) + r % p.rows_per_seq + 1 : p.seq_lens[r];
    const int64_t room = p.max_blocks_per_seq > 0 ? static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size : given;
    const int64_t len = min(given, room);
    bool bad = given > room;
    float q[16], o[16] = {}, m = -__builtin_huge_valf(), l = 0.0f;
    const uint16_t* qp = p.q + rh * kLatent + lane * 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = __uint_as_float(static_cast<uint32_t>(qp[i]) << 16) * p.score_scale;
    for (int64_t j = 0; j < len; ++j) {
        const int32_t page = p.block_tables[seq * p.max_blocks_per_seq + j / p.block_size];
        if (page < 0) {
            bad = true;
            continue;
        }
        const int64_t at = page * p.cache_stride + (j % p.block_size) * kLatent + lane * 16;
        float k[16], x = 0.0f;
        decode16(__ldg(reinterpret_cast<const uint4*>(p.k_cache + at)), k);
#pragma unroll
        for (int i = 0; i < 16; ++i) x = fmaf(q[i], k[i], x);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
        if (p.v_cache != p.k_cache) decode16(__ldg(reinterpret_cast<const uint4*>(p.v_cache + at)), k);
        const float top = fmaxf(m, x), a = exp2f(m - top), e = exp2f(x - top);
        m = top;
        l = l * a + e;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = fmaf(e, k[i], o[i] * a);
    }
    const float f = l > 0.0f ? p.v_scale / l : 0.0f;
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + rh * kLatent + lane * 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) out[i] = __float2bfloat16_rn(o[i] * f);
    if (bad && lane == 0) atomicCAS(p.status, 0, kStatusBounds);
}

}  // namespace

cudaError_t launch_full(const FullParams& p, cudaStream_t stream) {
    cudaError_t e = cudaMemsetAsync(p.status, 0, 4, stream);
    if (e != cudaSuccess) return e;
    const int64_t warps = static_cast<int64_t>(p.num_seqs) * p.rows_per_seq * p.heads;
    full_kernel<<<static_cast<unsigned>((warps + kFullWarps - 1) / kFullWarps), kFullWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dsa
