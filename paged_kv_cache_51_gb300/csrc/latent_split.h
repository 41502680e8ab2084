// The arithmetic of the latent attention's split: `total` steps, one after the other, are
// cut into `teams` stretches, stretch t beginning at step floor(t total / teams).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define PKV_SPLIT_FN __host__ __device__ __forceinline__
#else
#define PKV_SPLIT_FN inline
#endif

namespace pkv {

// floor(a b / c) for a product below 2^63; in 32 bits where all of it fits
PKV_SPLIT_FN int64_t mul_div(int64_t a, int64_t b, int64_t c) {
    const uint64_t x = uint64_t(a) * uint64_t(b);
    return ((x | uint64_t(c)) >> 32) == 0 ? int64_t(uint32_t(x) / uint32_t(c)) : int64_t(x / uint64_t(c));
}

PKV_SPLIT_FN int64_t stretch_begin(int64_t t, int64_t total, int teams) { return mul_div(t, total, teams); }

// the last t that begins at or before `step`
PKV_SPLIT_FN int stretch_of(int64_t step, int64_t total, int teams) {
    const int t = int(mul_div(step + 1, teams, total));
    return t < teams && stretch_begin(t, total, teams) <= step ? t : t - 1;
}

}  // namespace pkv
