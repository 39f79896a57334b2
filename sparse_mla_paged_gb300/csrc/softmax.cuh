// The softmax of the decodes whose probabilities become two E4M3 terms (full.cu, prefill.cu).
#pragma once

#include "common.cuh"

namespace dsa {

// What the two E4M3 terms of a P' lose: 2^-10 at most (it itself when below), beside 1.2 * 2^-9 of
// it. The row sum takes P' whole, so a tile far below its pair's reference would be counted but not
// added: 128 terms of 2^-11 weigh 2^-4, as much as a 512th of a row whose sum is the 2^5 of one
// maximum. Each thread therefore keeps an account per pair, kLostShare (common.cuh) of its P'
// less what their terms may lose. While the four threads of a pair have one in credit together,
// less than kLostShare of the row is lost; a thread that sees its own run out asks, and a pair that
// could not pay for one more tile moves its reference down to that tile. (A tile that holds 2^5
// pays for itself: 2^5 * kLostShare = 128 * 2^-10.) Scores of deviation 1 never ask; of
// deviation 2 in natural units, 56 of 128 tiles of 64 pairs move a reference, 25 without it.
constexpr int kScores = 32;                      // of a thread in a tile
constexpr float kMostLost = kScores * 0x1p-10f;  // by a thread in a tile

// Two probabilities as two E4M3 terms each (hi: rounded to nearest; lo: what is left of the
// float16 value, whose own rounding of 2^-12 is far below lo's 2^-9 of P'; kMostLost has what small
// ones lose). Through float16 pairs this takes five instructions where single floats take eight.
__device__ __forceinline__ void split2(float p0, float p1, uint32_t& hi, uint32_t& lo) {
    uint16_t h, l;
    asm("{\n\t.reg .b32 v, r, d;\n\t"
        "cvt.rn.f16x2.f32 v, %3, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 %0, v;\n\t"
        "cvt.rn.f16x2.e4m3x2 r, %0;\n\t"
        "sub.rn.f16x2 d, v, r;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 %1, d;\n\t}"
        : "=&h"(h), "=h"(l)
        : "f"(p0), "f"(p1));
    hi = h;
    lo = l;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

}  // namespace dsa
