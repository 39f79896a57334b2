// Pooled index scores: the cheap score by which the selector ranks the pools of each row.
//
//   I[r,j]     = s_j * sum_h w[r,h] * max(0, q[r,h,:] . k_j)       (k_j, s_j: index cache)
//   score[r,p] = max over the kpool tokens j of pool p of I[r,j], and -inf unless the whole
//                pool lies at or before the row's position q_pos[r]
//
// The dots are a matrix product, tokens x (rows x heads), on tcgen05 tensor cores: the keys'
// E4M3 codes are the A operand as they lie in the cache (M = 128 tokens of a tile), the
// queries of up to 128/heads rows of one sequence the B operand (N = rows x heads). A BF16
// query is two E4M3 terms (hi = its top 4 significant bits after scaling its head by a power
// of two, lo = the rest), both accumulated into the same FP32 columns, so the product is
// exact but for elements below 2^-10 of their head's largest. With tokens as rows of D, a
// token's heads lie in one thread's columns: the relu, the weighted sum over heads and the
// key's scale need no exchange between threads, and the maximum over a pool's tokens is a few
// shuffles between neighbouring lanes. The power of two goes into the head's weight.
//
// One block per (row group of a sequence, stretch of token tiles): warps 0-3 epilogue (one
// TMEM lane quarter each), warp 4 issues the MMAs, warps 5-8 copy 16-byte pieces of the key
// rows into a ring of tiles in the 128-byte-swizzled operand layout. Scores of different
// tokens are independent, so a long cache is split over blocks with nothing to join.
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128;                       // tokens of a tile: MMA M
constexpr int kMaxCols = 128;                    // rows x padded heads of a block: MMA N
constexpr int kStages = 4;
constexpr int kEpiWarps = 4;
constexpr int kMmaWarp = kEpiWarps;
constexpr int kLoadWarp0 = kMmaWarp + 1;
constexpr int kLoadWarps = 4;                    // 32 tokens of a tile each
constexpr int kThreads = (kLoadWarp0 + kLoadWarps) * 32;
constexpr int kTileBytes = kTile * kIndexDim;    // 16 KB of codes
// A scale slot is written again 2*kStages tiles later: by then the MMA of the tile kStages
// before it has run, hence the epilogue two tiles before that one has read its scales.
constexpr int kScaleSlots = 2 * kStages;
constexpr int kBarEpilogue = 1;

constexpr int kOffQ = kStages * kTileBytes;                    // [2 terms][cols][128 codes]
constexpr int kOffScale = kOffQ + 2 * kMaxCols * kIndexDim;    // float [slots][128]
constexpr int kOffW = kOffScale + kScaleSlots * kTile * 4;     // float [cols]
constexpr int kOffToken = kOffW + kMaxCols * 4;                // float [8 rows][128] token scores
constexpr int kOffVis = kOffToken + 8 * kTile * 4;             // int32 [8] visible pools of a row
constexpr int kOffBars = kOffVis + 8 * 4;
enum { BAR_FULL = 0, BAR_EMPTY = kStages, BAR_DFULL = 2 * kStages, BAR_DEMPTY = BAR_DFULL + 2, BAR_DRAIN = BAR_DEMPTY + 2, kNumBars };
constexpr int kOffTmem = kOffBars + kNumBars * 8;
constexpr int kOffAbort = kOffTmem + 4;
constexpr int kSmem = kOffAbort + 4 + 1024;      // 1 KB of slack for the 1024-byte alignment
constexpr uint32_t kTmemCols = 2 * kMaxCols;     // two D buffers; two blocks fill an SM's 512
static_assert(2 * kSmem <= 227 * 1024, "two blocks per SM");

constexpr uint64_t kWaitNs = 1000ull * 1000ull * 1000ull;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// acc += w * (max(x0, 0), max(x1, 0)), both halves in one instruction.
__device__ __forceinline__ void fma_relu2(uint64_t& acc, uint64_t w, uint32_t x0, uint32_t x1) {
    const uint32_t a = __float_as_uint(max_nan(__uint_as_float(x0), 0.0f));
    const uint32_t b = __float_as_uint(max_nan(__uint_as_float(x1), 0.0f));
    asm("{\n\t.reg .b64 x;\n\tmov.b64 x, {%2, %3};\n\tfma.rn.f32x2 %0, x, %1, %0;\n\t}" : "+l"(acc) : "l"(w), "r"(a), "r"(b));
}
__device__ __forceinline__ float sum2(uint64_t a) {
    return __uint_as_float(static_cast<uint32_t>(a)) + __uint_as_float(static_cast<uint32_t>(a >> 32));
}

struct Block {
    const PoolScoresParams& p;
    uint8_t* smem;
    uint32_t sbase;
    volatile int* abort_flag;
    int32_t seq, row0, rows;       // rows [row0, row0 + rows) of sequence seq
    int32_t per_tile;              // pools of a tile; its tokens are per_tile*kpool
    int32_t pool0;                 // first pool of the stretch
    int32_t tiles;                 // tiles with a pool that some row sees
    int32_t seen;                  // pools that some row sees: [0, seen)

    __device__ uint32_t bar(int i) const { return sbase + kOffBars + 8 * i; }
    __device__ void fail(int code) const {
        if (p.status) atomicCAS(p.status, 0, code);
        *abort_flag = 1;
    }
    __device__ void wait(int b, uint32_t parity) const {
        if (!mbar_wait(bar(b), parity, abort_flag, kWaitNs)) fail(kStatusTimeout);
        __syncwarp();
    }
};

// Queries of the block's rows as two E4M3 terms, weights with the heads' powers of two; a
// half-warp per (row, head), eight dims a lane. Columns past the heads are zero.
template <int kHeads>
__device__ void load_queries(const Block& b) {
    const int sub = threadIdx.x & 15;
    float* w_s = reinterpret_cast<float*>(b.smem + kOffW);
    const int cols = b.rows * kHeads;
    // Both half-warps of a warp take the same number of turns (the shuffles need them).
    for (int c0 = threadIdx.x >> 5; 2 * c0 < cols; c0 += kThreads / 32) {
        const int col = 2 * c0 + ((threadIdx.x >> 4) & 1);
        const int r = col / kHeads, h = col % kHeads;
        const bool real = h < b.p.heads;
        const int64_t rh = static_cast<int64_t>(b.row0 + r) * b.p.heads + h;
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (real) raw = __ldg(reinterpret_cast<const uint4*>(b.p.q + rh * kIndexDim) + sub);
        const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
        float x[8], top = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = __uint_as_float(u[k] << 16);
            x[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max_nan(top, fabsf(x[k]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        // e with top * 2^e in [128, 256); a head with a NaN or an infinity gets zero codes and
        // a NaN weight, which makes all its row's scores NaN.
        const int E = static_cast<int>((__float_as_uint(top) >> 23) & 0xFF);
        const bool broken = E == 255;
        int e = top > 0.0f ? 134 - E : 0;
        e = e > 126 ? 126 : (e < -126 ? -126 : e);
        const float sc = broken ? 0.0f : __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float vh[4], vl[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float v = broken ? 0.0f : x[4 * k + m] * sc;
                vh[m] = __uint_as_float(__float_as_uint(v) & 0xFFF00000u);
                vl[m] = v - vh[m];
            }
            hi[k] = f32x2_to_e4m3x2(vh[0], vh[1]) | (f32x2_to_e4m3x2(vh[2], vh[3]) << 16);
            lo[k] = f32x2_to_e4m3x2(vl[0], vl[1]) | (f32x2_to_e4m3x2(vl[2], vl[3]) << 16);
        }
        uint8_t* at = b.smem + kOffQ + col * kIndexDim + (((sub >> 1) ^ (col & 7)) << 4) + (sub & 1) * 8;
        *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(at + kMaxCols * kIndexDim) = make_uint2(lo[0], lo[1]);
        if (sub == 0) {
            const float w = real ? b.p.w[rh] : 0.0f;
            w_s[col] = broken ? __uint_as_float(0x7FC00000u) : w * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        }
    }
}

// Copy warps: warp w takes tokens 32w .. 32w+31 of every tile; lane l resolves the page of
// token 32w + l (a tile ahead of its copies) and copies its scale.
__device__ void run_load(const Block& b) {
    const PoolScoresParams& p = b.p;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - kLoadWarp0;
    const int tokens = b.per_tile * p.kpool;
    const int tk = 32 * w + lane;
    const int64_t limit = static_cast<int64_t>(b.seen) * p.kpool;
    const int32_t* table = p.block_tables + static_cast<int64_t>(b.seq) * p.max_blocks_per_seq;
    constexpr int64_t kNone = -1, kBad = -2;
    // Page and row of this lane's token of tile t, as the byte offsets of its codes and scale.
    auto resolve = [&](int t, int64_t& code, int64_t& scale) {
        code = scale = kNone;
        const int64_t pos = (static_cast<int64_t>(b.pool0) + static_cast<int64_t>(t) * b.per_tile) * p.kpool + tk;
        if (t >= b.tiles || tk >= tokens || pos >= limit) return;
        const int32_t blk = static_cast<int32_t>(pos) / p.block_size, off = static_cast<int32_t>(pos) - blk * p.block_size;
        const int32_t page = (p.max_blocks_per_seq == 0 || blk < p.max_blocks_per_seq) ? __ldg(table + blk) : -1;
        if (page < 0) {
            code = kBad;
            return;
        }
        const int64_t at = page * p.page_stride;
        code = at + static_cast<int64_t>(off) * kIndexDim;
        scale = at + static_cast<int64_t>(p.block_size) * kIndexDim + off * 4;
    };
    int64_t code, scale, next_code, next_scale;
    resolve(0, next_code, next_scale);
    for (int t = 0; t < b.tiles; ++t) {
        code = next_code;
        scale = next_scale;
        resolve(t + 1, next_code, next_scale);
        const int e = t % kStages;
        if (t >= kStages) b.wait(BAR_EMPTY + e, (t / kStages - 1) & 1);
        const uint32_t dst = b.sbase + e * kTileBytes;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = 4 * i + (lane >> 3), c = lane & 7;
            const int64_t at = __shfl_sync(0xffffffffu, code, row);
            const uint32_t d = (32 * w + row) * kIndexDim + ((c ^ (row & 7)) << 4);
            cp_async_16_zfill(dst + d, p.cache + (at >= 0 ? at + c * 16 : 0), at >= 0 ? 16u : 0u);
        }
        float* slot = reinterpret_cast<float*>(b.smem + kOffScale) + (t % kScaleSlots) * kTile + tk;
        if (scale >= 0) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(slot)), "l"(p.cache + scale) : "memory");
        } else {
            *slot = kNegInf;  // a token without a page scores -inf
            if (code == kBad && p.status) atomicCAS(p.status, 0, kStatusBounds);
        }
        cp_async_arrive_noinc(b.bar(BAR_FULL + e));
        __syncwarp();
        if (lane == 0) mbar_arrive(b.bar(BAR_FULL + e));  // releases the slots written by plain stores
    }
    cp_async_wait_all();
}

__device__ void run_mma(const Block& b, uint32_t tmem, int cols) {
    const uint32_t idesc = idesc_e4m3(kTile, cols, false, false);
    const uint32_t el = elect_one();
    const uint64_t q = smem_desc(b.sbase + kOffQ, 16, 1024, kSwizzle128B);
    for (int t = 0; t < b.tiles; ++t) {
        const int e = t % kStages, d = t & 1;
        b.wait(BAR_FULL + e, (t / kStages) & 1);
        if (t >= 2) b.wait(BAR_DEMPTY + d, ((t >> 1) - 1) & 1);
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t k = smem_desc(b.sbase + e * kTileBytes, 16, 1024, kSwizzle128B);
        const uint32_t dst = tmem + d * kMaxCols;
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                const uint64_t bq = q + static_cast<uint64_t>((term * kMaxCols * kIndexDim + ks * 32) >> 4);
                mma_e4m3_el(dst, k + static_cast<uint64_t>((ks * 32) >> 4), bq, idesc, term + ks > 0 ? 1u : 0u, el);
            }
        tc_commit_el(b.bar(BAR_EMPTY + e), el);
        tc_commit_el(b.bar(BAR_DFULL + d), el);
        if (el) mbar_arrive(b.bar(BAR_DFULL + d));
    }
    // Every MMA has completed before the block gives its tensor memory back.
    tc_commit_el(b.bar(BAR_DRAIN), el);
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(b.bar(BAR_DRAIN), 0) && globaltimer_ns() - t0 < kDrainLimitNs) {
    }
    __syncwarp();
}

template <int kHeads>
__device__ void run_epilogue(const Block& b, uint32_t tmem) {
    const PoolScoresParams& p = b.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tk = threadIdx.x;
    const float* w_s = reinterpret_cast<const float*>(b.smem + kOffW);
    const float* scale_s = reinterpret_cast<const float*>(b.smem + kOffScale);
    float* token_s = reinterpret_cast<float*>(b.smem + kOffToken);
    const int32_t* vis_s = reinterpret_cast<const int32_t*>(b.smem + kOffVis);
    const bool in_lanes = p.kpool <= 32 && (p.kpool & (p.kpool - 1)) == 0;  // a pool's tokens in one warp
    constexpr int kChunk = kHeads < 32 ? kHeads : 32;
    for (int t = 0; t < b.tiles; ++t) {
        const int d = t & 1;
        const int32_t pool_t = b.pool0 + t * b.per_tile;
        b.wait(BAR_DFULL + d, (t >> 1) & 1);
        tc_fence_after();
        const float scale = scale_s[(t % kScaleSlots) * kTile + tk];
        for (int r = 0; r < b.rows; ++r) {
            uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
            for (int c0 = 0; c0 < kHeads; c0 += kChunk) {
                uint32_t x[kChunk];
                const uint32_t at = tmem + (static_cast<uint32_t>(warp * 32) << 16) + d * kMaxCols + r * kHeads + c0;
                if constexpr (kChunk == 32) tmem_ld_x32(at, x); else tmem_ld_x16(at, x);
#pragma unroll
                for (int c = 0; c < kChunk; c += 4) {
                    const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(w_s + r * kHeads + c0 + c);
                    fma_relu2(acc[(c >> 1) & 3], w.x, x[c], x[c + 1]);
                    fma_relu2(acc[((c >> 1) + 1) & 3], w.y, x[c + 2], x[c + 3]);
                }
            }
            if (r == b.rows - 1) {  // the buffer's last values are in registers
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b.bar(BAR_DEMPTY + d));
            }
            float s = ((sum2(acc[0]) + sum2(acc[1])) + (sum2(acc[2]) + sum2(acc[3]))) * scale;
            if (scale == kNegInf) s = kNegInf;
            float* out = p.scores + static_cast<int64_t>(b.row0 + r) * p.n_pools;
            if (in_lanes) {
                for (int o = 1; o < p.kpool; o <<= 1) s = max_nan(s, __shfl_xor_sync(0xffffffffu, s, o));
                const int32_t pool = pool_t + tk / p.kpool;
                if (tk % p.kpool == 0 && pool < p.n_pools) out[pool] = pool < vis_s[r] ? s : kNegInf;
            } else {
                token_s[r * kTile + tk] = s;
            }
        }
        if (!in_lanes) {
            named_bar_sync<kBarEpilogue, kEpiWarps * 32>();
            for (int i = tk; i < b.rows * b.per_tile; i += kEpiWarps * 32) {
                const int r = i / b.per_tile, k = i % b.per_tile;
                const int32_t pool = pool_t + k;
                if (pool >= p.n_pools) continue;
                float s = kNegInf;
                if (pool < vis_s[r])
                    for (int j = 0; j < p.kpool; ++j) s = max_nan(s, token_s[r * kTile + k * p.kpool + j]);
                p.scores[static_cast<int64_t>(b.row0 + r) * p.n_pools + pool] = s;
            }
            named_bar_sync<kBarEpilogue, kEpiWarps * 32>();
        }
    }
}

template <int kHeads>
__global__ void __launch_bounds__(kThreads, 2)
    pool_scores_kernel(const PoolScoresParams p, int32_t groups, int32_t chunks, int32_t chunk_tiles) {
    extern __shared__ uint8_t smem_raw[];
    constexpr int kRows = kMaxCols / kHeads;
    static_assert(kRows <= 8, "rows of a block");
    const int tid = threadIdx.x, warp = tid >> 5;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int32_t unit = static_cast<int32_t>(blockIdx.x / chunks), chunk = static_cast<int32_t>(blockIdx.x % chunks);
    Block b{p, smem, smem_u32(smem), reinterpret_cast<volatile int*>(smem + kOffAbort)};
    b.seq = unit / groups;
    const int32_t first = (unit % groups) * kRows;
    b.row0 = b.seq * p.rows_per_seq + first;
    b.rows = min(kRows, p.rows_per_seq - first);
    b.per_tile = kTile / p.kpool;
    b.pool0 = chunk * chunk_tiles * b.per_tile;
    int32_t* vis_s = reinterpret_cast<int32_t*>(smem + kOffVis);
    b.seen = 0;
    for (int r = 0; r < b.rows; ++r) {
        const int64_t q = p.q_pos[b.row0 + r];
        const int32_t n = q < 0 ? 0 : static_cast<int32_t>(min((q + 1) / p.kpool, static_cast<int64_t>(p.n_pools)));
        if (tid == 0) vis_s[r] = n;
        b.seen = max(b.seen, n);
    }
    const int32_t end = static_cast<int32_t>(min(static_cast<int64_t>(b.pool0) + static_cast<int64_t>(chunk_tiles) * b.per_tile,
                                                 static_cast<int64_t>(p.n_pools)));
    const int32_t left = min(b.seen, end) - b.pool0;
    b.tiles = left > 0 ? (left + b.per_tile - 1) / b.per_tile : 0;
    // Pools of the stretch past the last tile that is computed.
    for (int r = 0; r < b.rows; ++r)
        for (int64_t k = static_cast<int64_t>(b.pool0) + static_cast<int64_t>(b.tiles) * b.per_tile + tid; k < end; k += kThreads)
            p.scores[static_cast<int64_t>(b.row0 + r) * p.n_pools + k] = kNegInf;
    if (b.tiles == 0) return;

    if (tid == 0) {
        for (int e = 0; e < kStages; ++e) {
            mbar_init(b.bar(BAR_FULL + e), kLoadWarps * 33);  // 32 lanes' copies and a plain arrival per warp
            mbar_init(b.bar(BAR_EMPTY + e), 1);
        }
        for (int d = 0; d < 2; ++d) {
            mbar_init(b.bar(BAR_DFULL + d), 2);  // the MMAs' commit, and the MMA warp passing on the scales
            mbar_init(b.bar(BAR_DEMPTY + d), kEpiWarps);
        }
        mbar_init(b.bar(BAR_DRAIN), 1);
        *b.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(b.sbase + kOffTmem, kTmemCols);
        tmem_relinquish();
    }
    load_queries<kHeads>(b);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem);
    if (warp < kEpiWarps) run_epilogue<kHeads>(b, tmem);
    else if (warp == kMmaWarp) run_mma(b, tmem, b.rows * kHeads);
    else run_load(b);
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

using Kernel = void (*)(const PoolScoresParams, int32_t, int32_t, int32_t);

// Heads are padded to 16, 32, 64 or 128 columns.
Kernel pick(int heads, int* padded) {
    *padded = heads <= 16 ? 16 : (heads <= 32 ? 32 : (heads <= 64 ? 64 : 128));
    switch (*padded) {
        case 16: return pool_scores_kernel<16>;
        case 32: return pool_scores_kernel<32>;
        case 64: return pool_scores_kernel<64>;
        default: return pool_scores_kernel<128>;
    }
}

}  // namespace

cudaError_t pool_scores_kernel_setup() {
    for (int heads = 16; heads <= 128; heads *= 2) {
        int padded;
        const Kernel k = pick(heads, &padded);
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_pool_scores(const PoolScoresParams& p, int sms, cudaStream_t stream) {
    int padded;
    const Kernel k = pick(p.heads, &padded);
    const int32_t rows = kMaxCols / padded, groups = (p.rows_per_seq + rows - 1) / rows;
    const int64_t units = static_cast<int64_t>(p.num_seqs) * groups;
    const int32_t per_tile = kTile / p.kpool;
    const int64_t tiles = (p.n_pools + static_cast<int64_t>(per_tile) - 1) / per_tile;
    // Tiles of a block: about four waves of two blocks per SM, at least two tiles (a block's
    // set-up costs about as much as one) and at most 64.
    int64_t chunk = (units * tiles + 8 * sms - 1) / (8 * sms);
    chunk = chunk < 2 ? 2 : (chunk > 64 ? 64 : chunk);
    if (chunk > tiles) chunk = tiles;
    int64_t chunks = (tiles + chunk - 1) / chunk;
    while (units * chunks > INT32_MAX) {  // the grid's limit: longer stretches
        chunk *= 2;
        chunks = (tiles + chunk - 1) / chunk;
    }
    k<<<static_cast<unsigned>(units * chunks), kThreads, kSmem, stream>>>(p, groups, static_cast<int32_t>(chunks),
                                                                      static_cast<int32_t>(chunk));
    return cudaGetLastError();
}

}  // namespace dsa
