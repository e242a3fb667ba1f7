// Joining partial attention results of one row: o = sum w_i o_i / sum w_i with
// w_i = exp(lse_i - max lse), in the parts' order.  One warp, D / 32 columns
// per lane.
#pragma once

#include <cuda_runtime.h>

namespace codec {

// lse_of(i): a part's lse; part_of(i, x): this lane's columns of a part.
// empty: the row sees nothing (v = 0, lse = -inf).  kAhead: parts that are read
// before their weights are known.  kValues: every part has finite values or NaN, one
// without keys zeros, so that one of no weight is added like others (0 times NaN is NaN);
// else it is left out, whatever it holds.
template <int kE, int kAhead, bool kValues = false, typename Lse, typename Part>
__device__ __forceinline__ void join_row(int parts, bool empty, Lse lse_of, Part part_of, float* v, float& lse)
{
    const int lane = threadIdx.x & 31;
    // the first parts are on their way while the weights are worked out
    const float mine = lane < parts ? lse_of(lane) : -INFINITY;
    float ahead[kAhead][kE];
#pragma unroll
    for (int i = 0; i < kAhead; i++)
        if (i < parts) part_of(i, ahead[i]);
    float m = -INFINITY;
    bool nan = false;
    for (int i = lane; i < parts; i += 32) {
        const float x = i < 32 ? mine : lse_of(i);
        m = fmaxf(m, x);
        nan |= x != x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (__any_sync(0xffffffffu, nan)) m = NAN;
    const float ref = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < kE; e++) v[e] = 0.f;
    float w = lane < parts ? expf(mine - ref) : 0.f;
    auto add = [&](float f, const float* x) {
        sum += f;
#pragma unroll
        for (int e = 0; e < kE; e++) v[e] = kValues || f != 0.f ? fmaf(f, x[e], v[e]) : v[e];
    };
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
        const float f = __shfl_sync(0xffffffffu, w, i);
        if (i < parts) add(f, ahead[i]);
    }
    for (int i0 = 0; i0 < parts; i0 += 32) {
        if (i0 > 0) w = i0 + lane < parts ? expf(lse_of(i0 + lane) - ref) : 0.f;
        const int cnt = min(32, parts - i0);
#pragma unroll 8
        for (int i = i0 == 0 ? kAhead : 0; i < cnt; i++) {
            float x[kE];
            part_of(i0 + i, x);
            add(__shfl_sync(0xffffffffu, w, i), x);
        }
    }
    const float inv = empty ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < kE; e++) v[e] *= inv;
    lse = empty ? -INFINITY : m + logf(sum);
}

// This lane's columns of a row of D = 32 kE fp32 values, past L1.
template <int kE>
__device__ __forceinline__ void row_part(const float* row, float* x)
{
    const int lane = threadIdx.x & 31;
    if constexpr (kE == 4) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(row) + lane);
        x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
    } else {
        const float2 y = __ldcg(reinterpret_cast<const float2*>(row) + lane);
        x[0] = y.x; x[1] = y.y;
    }
}

}  // namespace codec
