// Attention of one token per request over the cache in 4 bits.
//
// A CTA per (request, query head); each warp takes every fourth tile of 16
// positions with a running maximum and sum of its own, and the four are joined
// at the end.  All in fp32.
#include "lm.h"
#include "lm_q4.cuh"

namespace codec {

namespace {

constexpr int kWarps = 4;

struct Params {
    const void* q;
    long long qs;
    const uint8_t *k, *v;
    const int *tables, *kv_len, *shared_table;
    int table_blocks, bs_shift, n_blocks, shared_len;
    int hq, hk, group;
    float scale;
    void* o;
    long long os;
    float* lse;
    unsigned* err;
};

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void from_float(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) lm_step_q4_kernel(const Params p)
{
    using Tile = Q4Tile<D>;
    __shared__ float qs[D], part[kWarps][D], stat[kWarps][2];
    const int b = blockIdx.x / p.hq, h = blockIdx.x - b * p.hq, kh = h / p.group;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_launch();
    for (int i = tid; i < D; i += 32 * kWarps)
        qs[i] = to_float(static_cast<const T*>(p.q)[b * p.qs + (long long)h * D + i]);
    int len = __ldg(p.kv_len + b);
    if (!lm_clamp_len(len, (long long)p.table_blocks << p.bs_shift) && tid == 0 && h == 0)
        atomicOr(p.err, CODEC_LM_ERR_LENGTH);
    __syncthreads();
    float m = -INFINITY, l = 0.f, acc[D / 32] = {};
    for (int t0 = warp * 16; t0 < len; t0 += 16 * kWarps) {
        const int j = t0 >> p.bs_shift;
        const int id = __ldg(t0 < p.shared_len ? p.shared_table + j : p.tables + (long long)b * p.table_blocks + j);
        const bool good = id >= 0 && id < p.n_blocks;
        if (!good && lane == 0) atomicOr(p.err, CODEC_LM_ERR_BLOCK);
        const int tiles = 1 << (p.bs_shift - 4);
        const long long at = good ? (((long long)id * p.hk + kh) * tiles + ((t0 & ((1 << p.bs_shift) - 1)) >> 4)) * Tile::kBytes : 0;
        const int left = min(16, len - t0);
        // two lanes a position, each half of the words
        const int pos = lane >> 1;
        float s = 0.f;
        if (good)
            for (int w = lane & 1; w < 4 * Tile::G; w += 2) {
                const int t = w & 3, g = w >> 2;
                const uint32_t word = *reinterpret_cast<const uint32_t*>(p.k + at + Tile::k_word(pos, t, g));
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(p.k + at + Tile::k_param(pos, g)));
                float dot = 0.f, sum = 0.f;
                for (int e = 0; e < 8; e++) {
                    const float q = qs[g * 32 + t * 8 + e];
                    dot += q * (float)(word >> (4 * e) & 15u);
                    sum += q;
                }
                s += f.x * dot + f.y * sum;
            }
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s = pos < left ? s * p.scale : -INFINITY;
        float top = s;
        for (int o = 2; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float now = fmaxf(m, top), ref = now == -INFINITY ? 0.f : now;
        const float f = expf(m - ref), e = expf(s - ref);
        m = now;
        float sum = lane & 1 ? 0.f : e;
        for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = l * f + sum;
#pragma unroll
        for (int i = 0; i < D / 32; i++) acc[i] *= f;
        for (int x = 0; x < left; x++) {
            const float w = __shfl_sync(0xffffffffu, e, 2 * x);
            if (!good) continue;
#pragma unroll
            for (int g = 0; g < D / 32; g++) {
                const int r = lane >> 2, k = lane & 3;
                const uint32_t two = *reinterpret_cast<const uint16_t*>(p.v + at + Tile::v_pair(x, r, g));
                const float sc = __half2float(*reinterpret_cast<const __half*>(p.v + at + Tile::v_scale(x, g)));
                const float lo = __half2float(*reinterpret_cast<const __half*>(p.v + at + Tile::v_scale(x, g) + D));
                acc[g] += w * fmaf(sc, (float)(two >> (4 * k) & 15u), lo);
            }
        }
    }
#pragma unroll
    for (int g = 0; g < D / 32; g++) part[warp][g * 32 + lane] = acc[g];
    if (lane == 0) {
        stat[warp][0] = m;
        stat[warp][1] = l;
    }
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; w++) top = fmaxf(top, stat[w][0]);
    for (int w = 0; w < kWarps; w++)
        if (stat[w][1] != stat[w][1]) top = NAN;
    float f[kWarps];
    for (int w = 0; w < kWarps; w++) {
        f[w] = stat[w][0] == -INFINITY && stat[w][1] == 0.f ? 0.f : expf(stat[w][0] - top);
        sum += f[w] * stat[w][1];
    }
    const float inv = len > 0 ? 1.f / sum : 0.f;
    for (int d = tid; d < D; d += 32 * kWarps) {
        float v = 0.f;
        for (int w = 0; w < kWarps; w++)
            if (f[w] != 0.f) v += f[w] * part[w][d];
        from_float(static_cast<T*>(p.o) + b * p.os + (long long)h * D + d, v * inv);
    }
    if (p.lse && tid == 0) p.lse[(long long)b * p.hq + h] = len > 0 ? top + logf(sum) : -INFINITY;
}

}  // namespace

cudaError_t launch_lm_step_q4(const LmShape& sh, const LmStepArgs& a, cudaStream_t s)
{
    const LmKeys& ks = a.keys;
    const Params p{a.q, a.qs, static_cast<const uint8_t*>(ks.k), static_cast<const uint8_t*>(ks.v), ks.tables,
                   ks.kv_len, a.shared_table, ks.table_blocks, ks.bs_shift, ks.n_blocks,
                   a.shared_blocks << ks.bs_shift, sh.hq, sh.hk, sh.group, sh.scale, a.o, a.os, a.lse, sh.err};
    const dim3 grid((unsigned)(a.B * sh.hq)), block(32 * kWarps);
    if (sh.type == CODEC_LM_BF16)
        return launch_pdl(sh.D == 128 ? lm_step_q4_kernel<__nv_bfloat16, 128> : lm_step_q4_kernel<__nv_bfloat16, 64>,
                          grid, block, 0, s, p);
    return launch_pdl(sh.D == 128 ? lm_step_q4_kernel<__half, 128> : lm_step_q4_kernel<__half, 64>, grid, block, 0, s,
                      p);
}

}  // namespace codec
