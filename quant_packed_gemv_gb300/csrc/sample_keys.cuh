// Logits as whole numbers in their order ("keys"), and ranges of them cut into
// bins (the sampler, csrc/sample.cu).
#pragma once

#include <cstdint>
#include <cstring>

namespace plm {

constexpr int BINS = 2560;
constexpr uint32_t LOWEST = 0x007FFFFFu;       // the key of -inf
constexpr uint32_t MINUS_ZERO = 0x7FFFFFFFu;   // of -0: no logit has it, as they are added to 0 first

// (-0 is added to 0 before)
__host__ __device__ __forceinline__ uint32_t key_of(float x) {
    uint32_t b;
    memcpy(&b, &x, sizeof b);
    return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__host__ __device__ __forceinline__ float logit_of(uint32_t key) {
    const uint32_t b = key ^ ((uint32_t)((int)~key >> 31) | 0x80000000u);
    float x;
    memcpy(&x, &b, sizeof x);
    return x;
}

// Where a range of keys may end so that the logits in it are those that are no larger as
// f32.  As f32, -0 is no less than 0, whose key is one above: a range that ended at its key
// would let the zeros in, outside all bins.
__host__ __device__ __forceinline__ uint32_t range_end(uint32_t key) { return key == MINUS_ZERO ? key - 1 : key; }

// Keys lo .. hi in bins of 2^shift keys from hi downwards.
struct KeyBins {
    uint32_t lo, hi;
    int shift;
    __host__ __device__ KeyBins(uint32_t l, uint32_t h) : lo(l), hi(h), shift(0) {
        while (((hi - lo) >> shift) >= (uint32_t)BINS) ++shift;
    }
    __host__ __device__ __forceinline__ int bin(uint32_t key) const {   // (in the histogram whatever the key is)
        const uint32_t b = (hi - key) >> shift;
        return b < (uint32_t)BINS ? (int)b : BINS - 1;
    }
    __host__ __device__ __forceinline__ uint32_t first(int b) const { return hi - ((uint32_t)b << shift); }   // the highest of a bin
    __host__ __device__ __forceinline__ uint32_t last(int b) const {
        const uint32_t k = first(b);
        return (k - lo) >> shift ? k - (1u << shift) + 1 : lo;
    }
};

}  // namespace plm
