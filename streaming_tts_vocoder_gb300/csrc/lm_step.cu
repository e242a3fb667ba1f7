// Attention of the codec LM for single tokens.
//
// o = softmax(scale q K^T) V by one pass over the keys with the running
// maximum m and sum l: a key of score x rescales the sums by exp(m - m') and
// adds exp(x - m') v.  One warp per (row, query head), lanes over the head's
// elements.
#include "lm.h"

namespace codec {

namespace {

constexpr int kWarps = 4;

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

struct Sources {
    const int* shared_table;
    int shared_blocks;
};

// Row `row` of request b sees keys 0 .. n - 1.
template <typename T, int D>
__device__ void attend(const LmShape& sh, const LmKeys& ks, Sources src, const T* q, int b, long long packed0, int n,
                       int h, T* o, float* lse)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, hk = h / sh.group;
    float x[E], acc[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < E; i++) x[i] = to_f(q[lane + 32 * i]) * sh.scale;
    for (int j = 0; j < n; j++) {
        const T *k, *v;
        bool held = true;
        if (ks.tables) {
            const int blk = j >> ks.bs_shift;
            const int id = blk < src.shared_blocks ? __ldg(src.shared_table + blk)
                                                   : __ldg(ks.tables + (long long)b * ks.table_blocks + blk);
            held = id >= 0 && id < ks.n_blocks;
            if (!held && lane == 0) atomicOr(sh.err, CODEC_LM_ERR_BLOCK);
            const long long r = ((long long)(held ? id : 0) << ks.bs_shift) + (j & ((1 << ks.bs_shift) - 1));
            k = static_cast<const T*>(ks.k) + (r * sh.hk + hk) * D;
            v = static_cast<const T*>(ks.v) + (r * sh.hk + hk) * D;
        } else {
            k = static_cast<const T*>(ks.k) + (packed0 + j) * ks.k_stride + (long long)hk * D;
            v = static_cast<const T*>(ks.v) + (packed0 + j) * ks.v_stride + (long long)hk * D;
        }
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < E; i++) dot = fmaf(x[i], held ? to_f(k[lane + 32 * i]) : 0.f, dot);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        const float m2 = fmaxf(m, dot), f = expf(m - m2), p = expf(dot - m2);
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < E; i++) acc[i] = fmaf(p, held ? to_f(v[lane + 32 * i]) : 0.f, acc[i] * f);
        m = m2;
    }
#pragma unroll
    for (int i = 0; i < E; i++) o[lane + 32 * i] = from_f<T>(n > 0 ? acc[i] / l : 0.f);
    if (lse && lane == 0) *lse = n > 0 ? m + logf(l) : -INFINITY;
}

template <typename T, int D>
__global__ void lm_step_kernel(const LmShape sh, const LmStepArgs a)
{
    const long long w = blockIdx.x * (long long)kWarps + (threadIdx.x >> 5);
    const int b = (int)(w / sh.hq), h = (int)(w - (long long)b * sh.hq);
    if (b >= a.B) return;
    int keys = __ldg(a.keys.kv_len + b);
    if (!lm_clamp_len(keys, (long long)a.keys.table_blocks << a.keys.bs_shift)) atomicOr(sh.err, CODEC_LM_ERR_LENGTH);
    attend<T, D>(sh, a.keys, Sources{a.shared_table, a.shared_blocks},
                 static_cast<const T*>(a.q) + b * a.qs + (long long)h * D, b, 0, keys, h,
                 static_cast<T*>(a.o) + b * a.os + (long long)h * D,
                 a.lse ? a.lse + (long long)b * sh.hq + h : nullptr);
}

template <typename T, int D>
cudaError_t step(const LmShape& sh, const LmStepArgs& a, cudaStream_t s)
{
    const long long n = ((long long)a.B * sh.hq + kWarps - 1) / kWarps;
    lm_step_kernel<T, D><<<(unsigned)n, 32 * kWarps, 0, s>>>(sh, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lm_step(const LmShape& sh, const LmStepArgs& a, cudaStream_t s)
{
    if (sh.type == CODEC_LM_BF16) return sh.D == 128 ? step<__nv_bfloat16, 128>(sh, a, s) : step<__nv_bfloat16, 64>(sh, a, s);
    return sh.D == 128 ? step<__half, 128>(sh, a, s) : step<__half, 64>(sh, a, s);
}

}  // namespace codec
