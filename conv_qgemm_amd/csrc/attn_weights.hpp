// attn_weights.hpp -- what a run of cached tokens' key and value scales make of
// scores, softmax weights and their sum in attention over the int8 cache: plain
// binary32 arithmetic that also builds for the host.
//
// Every factor here is finite for every scale that a cache may hold, 0 (a block
// of zeros) included, and scores' factors are above 0, so that neither 0 *
// infinity nor infinity - infinity occurs: the attention kernels are compiled on
// the promise that no operation makes a NaN.
#pragma once

namespace qg {

// A row's maximum before it has seen a token: finite, so that the difference of
// two such is 0 and with any other score a power of 2 that vanishes.
constexpr float kNothing = -0x1.fffffep127f;
// Weights are 2^6 times larger: small ones keep bits.
constexpr float kLift = 6.0f;
// Scales of blocks with any other code than 0 are 2^-100 or more, so those of
// zeros are told from them: their logarithm and reciprocal are finite.
constexpr float kLeastScale = 0x1p-101f;

// Scores' factor: key scale * (softmax scale * log2 e).  A masked score,
// -infinity, stays that after it.
__device__ __forceinline__ float score_factor(float ks, float c2)
{
    return __builtin_fminf(__builtin_fmaxf(ks * c2, 0x1p-126f), 3.4e38f);
}

__device__ __forceinline__ float held_scale(float s) { return __builtin_fmaxf(s, kLeastScale); }

// log2 of the factor s / R of a weight, lifted (R: the row's largest weight
// times scale).  Under 2^-80 it stays there: the values vanish beside the
// others, but the sum still needs the weights.
__device__ __forceinline__ float run_shift(float log2s, float log2R)
{
    return __builtin_fmaxf(log2s - log2R, -80.0f) + kLift;
}

// What takes that factor out of the weight again, for the sum; rs = 1 / s.  It
// may underflow: the row's weight is no more then.
__device__ __forceinline__ float run_back(float R, float rs)
{
    return __builtin_fminf(R * rs, 0x1p80f) * 0x1p-6f;
}

}  // namespace qg
