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

}  // namespace codec
