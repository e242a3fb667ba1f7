// Where the cache in 4 bits holds what: tiles of 16 positions of one head (the
// layout is given in codec.h).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace codec {

template <int D>
struct Q4Tile {
    static constexpr int G = D / 32;                // groups of a head
    static constexpr int kBytes = 10 * D;           // codes 8 D, scales and lows 2 D
    static constexpr int kParams = 8 * D;

    // Keys.  The word of values 8 t .. 8 t + 7 of group g, and its (scale, low).
    static __host__ __device__ constexpr int k_word(int p, int t, int g) { return p * (D / 2) + (t * G + g) * 4; }
    static __host__ __device__ constexpr int k_param(int p, int g) { return kParams + (p * G + g) * 4; }

    // Values.  The two bytes of values 4 r .. 4 r + 3 of group g; scale (low: D bytes further).
    static __host__ __device__ constexpr int v_pair(int p, int r, int g)
    {
        return (p >> 3) * 4 * D + (r * 4 + ((p & 7) >> 1)) * 4 * G + g * 4 + (p & 1) * 2;
    }
    static __host__ __device__ constexpr int v_scale(int p, int g)
    {
        return kParams + ((((p & 7) >> 1) * G + g) * 4 + (p >> 3) * 2 + (p & 1)) * 2;
    }
};

// Queries as halves: times 2^lift, which brings a head's largest element to 2^14 ..
// 2^15, so exact but for what lies 2^24 below (what is not finite stays so); and
// the factor that undoes it with the scale.
__device__ __forceinline__ int q4_query_lift(float top)
{
    const int e = (int)(__float_as_uint(top) >> 23);
    return e == 255 ? 0 : min(127 + 14 - e, 100);
}
// Neither bound is met by scores that differ.
__device__ __forceinline__ float q4_query_factor(float c, int lift)
{
    return fmaxf(fminf(c * __int_as_float((127 - lift) << 23), 1e31f), 1e-30f);
}

}  // namespace codec
