// The index-key writer: each new token's 128-wide index key, layer-normalised when a weight
// is given, quantised to E4M3 with a scale of its own and stored in its slot of the paged
// index cache that the pool scores read.
//
//   y = (x - mean x) / sqrt(mean (x - mean x)^2 + eps) * w + b      (or y = x)
//   s = max(max|y|, 2^-100) / 448,   code = E4M3(y / s)
//
// Page p of the cache holds block_size rows of 128 codes, then block_size float32 scales.
//
// Sixteen lanes take one row, eight consecutive dims (one 16-byte load) each: both sums of
// the norm and the maximum stay in registers and four shuffles. HBM-bound: 264 bytes read
// and 132 written a row.
#include "common.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kIndexWriteThreads = 256;
constexpr int kRowsPerBlock = kIndexWriteThreads / 16;

__device__ __forceinline__ void unpack8(const uint4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The larger of two, NaN when either is (fmaxf would drop it, and with it a broken key).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__global__ void __launch_bounds__(kIndexWriteThreads) index_write_kernel(const IndexWriteParams p) {
    const int sub = threadIdx.x & 15;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 4);
    const bool in = row < p.rows;  // both half-warps stay for the shuffles
    const long long slot = in ? p.slots[row] : -1;
    float y[8] = {};
    if (slot >= 0) unpack8(__ldg(reinterpret_cast<const uint4*>(p.x + row * kIndexDim) + sub), y);
    if (p.weight) {
        float w[8], b[8] = {};
        unpack8(__ldg(reinterpret_cast<const uint4*>(p.weight) + sub), w);
        if (p.bias) unpack8(__ldg(reinterpret_cast<const uint4*>(p.bias) + sub), b);
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += y[k];
        const float mean = sum16(s) * (1.0f / kIndexDim);
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            y[k] -= mean;
            ss = fmaf(y[k], y[k], ss);
        }
        const float inv = 1.0f / sqrtf(sum16(ss) * (1.0f / kIndexDim) + p.eps);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = fmaf(y[k] * inv, w[k], b[k]);
    }
    float top = 0x1p-100f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max_nan(top, fabsf(y[k]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (slot < 0) return;
    const float inv = 448.0f / top;
    uint32_t c[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        c[k] = f32x2_to_e4m3x2(y[4 * k] * inv, y[4 * k + 1] * inv) |
               (f32x2_to_e4m3x2(y[4 * k + 2] * inv, y[4 * k + 3] * inv) << 16);
    uint8_t* page = p.cache + (slot / p.block_size) * p.page_stride;
    const int64_t off = slot % p.block_size;
    reinterpret_cast<uint2*>(page + off * kIndexDim)[sub] = make_uint2(c[0], c[1]);
    if (sub == 0) reinterpret_cast<float*>(page + static_cast<int64_t>(p.block_size) * kIndexDim)[off] = top / 448.0f;
}

}  // namespace

cudaError_t launch_index_write(const IndexWriteParams& p, cudaStream_t stream) {
    const int64_t blocks = (static_cast<int64_t>(p.rows) + kRowsPerBlock - 1) / kRowsPerBlock;
    index_write_kernel<<<static_cast<unsigned>(blocks), kIndexWriteThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dsa
