// The index-key writer: each new token's 128-wide index key, layer-normalised when a weight
// is given, quantised to E4M3 with a scale of its own and stored in its slot of the paged
// index cache that the pool scores read.
//
//   y = (x - mean x) / sqrt(mean (x - mean x)^2 + eps) * w + b      (or y = x)
//   s = max(max|y|, 2^-100) / 448,   code = E4M3(y / s), midpoints to the even code
//
// Page p of the cache holds block_size rows of 128 codes, then block_size float32 scales.
//
// Eight lanes take one row, sixteen consecutive dims each (the norm's sums and the maximum
// are three shuffles), and persistent blocks keep the weights in registers, a row's loads in
// flight while the one before is written. A row's chain of dependent instructions bounds it
// rather than bytes: 262144 rows with the norm take 22 us (4.7 TB/s of the 104 MB read and
// written, which the HBM moves in 15.5 us; 61 % of the issue slots under a profiler), without it
// 23, 64 rows 1.9 us. With sixteen lanes a row, 64-bit divisions of the slot and no reuse of the
// weights it took 41 us; two dims an instruction in the norm were the last step, from 24. More
// blocks per SM with fewer registers each were no faster.
#include "common.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kIndexWriteThreads = 256;
constexpr int kLanes = 8;                  // of a row
constexpr int kDims = kIndexDim / kLanes;  // of a lane: 16
constexpr int kRowsPerBlock = kIndexWriteThreads / kLanes;

__device__ __forceinline__ void unpack8(const uint4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The larger of two, NaN when either is (fmaxf would drop it, and with it a broken key).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <bool kNorm>
__global__ void __launch_bounds__(kIndexWriteThreads) index_write_kernel(const IndexWriteParams p) {
    const int sub = threadIdx.x % kLanes;
    float w[kDims], b[kDims];
    if constexpr (kNorm) {
        const uint4* ws = reinterpret_cast<const uint4*>(p.weight) + 2 * sub;
        unpack8(__ldg(ws), w);
        unpack8(__ldg(ws + 1), w + 8);
#pragma unroll
        for (int k = 0; k < kDims; ++k) b[k] = 0.0f;
        if (p.bias) {
            const uint4* bs = reinterpret_cast<const uint4*>(p.bias) + 2 * sub;
            unpack8(__ldg(bs), b);
            unpack8(__ldg(bs + 1), b + 8);
        }
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRowsPerBlock;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + threadIdx.x / kLanes;
    long long slot = -1;
    uint4 raw[2] = {};
    auto fetch = [&](int64_t r) {
        slot = r < p.rows ? p.slots[r] : -1;
        if (r < p.rows) {
            const uint4* x = reinterpret_cast<const uint4*>(p.x + r * kIndexDim) + 2 * sub;
            raw[0] = __ldg(x);
            raw[1] = __ldg(x + 1);
        }
    };
    fetch(row);
    // The whole warp stays while any of its rows is left (the shuffles need it).
    while (__any_sync(0xffffffffu, row < p.rows)) {
        float y[kDims];
        unpack8(raw[0], y);
        unpack8(raw[1], y + 8);
        const long long at = slot;
        row += step;
        fetch(row);
        if constexpr (kNorm) {
            // Two dims an instruction.
            float2* y2 = reinterpret_cast<float2*>(y);
            const float2 *w2 = reinterpret_cast<const float2*>(w), *b2 = reinterpret_cast<const float2*>(b);
            float2 s = make_float2(0.0f, 0.0f), ss = s;
#pragma unroll
            for (int k = 0; k < kDims / 2; ++k) s = __fadd2_rn(s, y2[k]);
            const float2 mean = both(row_sum(s.x + s.y) * (-1.0f / kIndexDim));
#pragma unroll
            for (int k = 0; k < kDims / 2; ++k) {
                y2[k] = __fadd2_rn(y2[k], mean);
                ss = __ffma2_rn(y2[k], y2[k], ss);
            }
            const float2 inv = both(rsqrtf(row_sum(ss.x + ss.y) * (1.0f / kIndexDim) + p.eps));
#pragma unroll
            for (int k = 0; k < kDims / 2; ++k) y2[k] = __ffma2_rn(__fmul2_rn(y2[k], inv), w2[k], b2[k]);
        }
        float top = 0x1p-100f;
#pragma unroll
        for (int k = 0; k < kDims; ++k) top = max_nan(top, fabsf(y[k]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        // Without a norm a key's y / s = 448 y / top often lies exactly between two codes (both are
        // bf16 numbers); a reciprocal's rounding would then choose for the even code. One correction
        // with the remainder of 7/8 y (exact in float32) by top / 512 finds the midpoint itself; none
        // with an infinite top, whose remainders would be NaN. A norm's y has no such ties, and
        // the correction would cost 0.8 us of 262144 rows' 21.9.
        const float2 inv = both((kNorm ? 448.0f : 512.0f) / top);
        const float2 back = both(top < __builtin_huge_valf() ? top * (-1.0f / 512.0f) : 0.0f);
        uint32_t c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t pair[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float2 x = reinterpret_cast<const float2*>(y)[2 * k + m];
                if constexpr (kNorm) {
                    x = __fmul2_rn(x, inv);
                } else {
                    const float2 z = __fmul2_rn(x, both(0.875f)), q = __fmul2_rn(z, inv);
                    x = __ffma2_rn(__ffma2_rn(q, back, z), inv, q);
                }
                pair[m] = f32x2_to_e4m3x2(x.x, x.y);
            }
            c[k] = pair[0] | pair[1] << 16;
        }
        if (at >= 0) {
            int64_t page, off;
            if (at >> 32 == 0) {  // a 64-bit division is a long sequence
                const uint32_t u = static_cast<uint32_t>(at), q = divide(u, p.by_block);
                page = q;
                off = u - q * p.by_block.d;
            } else {
                page = at / p.block_size;
                off = at % p.block_size;
            }
            uint8_t* dst = p.cache + page * p.page_stride;
            reinterpret_cast<uint4*>(dst + off * kIndexDim)[sub] = make_uint4(c[0], c[1], c[2], c[3]);
            if (sub == 0) reinterpret_cast<float*>(dst + static_cast<int64_t>(p.block_size) * kIndexDim)[off] = top / 448.0f;
        }
    }
}

}  // namespace

cudaError_t launch_index_write(const IndexWriteParams& p, int sms, cudaStream_t stream) {
    const int64_t all = (static_cast<int64_t>(p.rows) + kRowsPerBlock - 1) / kRowsPerBlock;
    const unsigned blocks = static_cast<unsigned>(all < 3 * sms ? all : 3 * sms);  // resident at once
    if (p.weight) index_write_kernel<true><<<blocks, kIndexWriteThreads, 0, stream>>>(p);
    else index_write_kernel<false><<<blocks, kIndexWriteThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace dsa
