// Per-head RMSNorm of queries and keys, position rotation, and the store of
// keys and values into their cache slots, in one pass over a projection's
// output.
//
// y = x / sqrt(mean(x^2) + eps) * gain, then pair (a, b) -> (a c - b s, b c + a s)
// with the cosine and sine of the row's angle, from a table that is computed
// in fp64 (at position 60,000 an fp32 angle would be off by 2^-9).  All in
// fp32, one rounding at the store.
//
// Bound by memory: every value is read and written once.  A head is the work
// of D / 16 lanes; each holds 8 elements of the first half and the 8 elements
// D / 2 further, so that both rotation forms stay inside a lane, every access
// is 16 bytes, and the norm is 2 or 3 shuffles.  A warp takes a row (or a part
// of its heads, when there are few rows): cosines, sines and a gain stay in
// registers over its heads, and kUnroll groups of heads are loaded (and kept
// as they lie in memory) before the first is worked on.  32,768 rows of 48
// heads of 128: 127 us, 6.35 TB/s; with two groups ahead 153, with eight 202,
// at three CTAs of 256 threads 129, at eight of 128 (registers spilled) 169.
#include "lm.h"

namespace codec {

namespace {

constexpr int kRotThreads = 128;

template <typename T> struct Pack;      // 8 values of 16 bits
template <> struct Pack<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t two(float a, float b)
    {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    static __device__ __forceinline__ float2 un(uint32_t w)
    {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
    }
};
template <> struct Pack<__half> {
    static __device__ __forceinline__ uint32_t two(float a, float b)
    {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    static __device__ __forceinline__ float2 un(uint32_t w)
    {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
};

// Eight values as they lie in memory (a projection's output may be q_out
// itself, so not by the read-only path), and in fp32.
template <typename T> struct Raw {
    uint4 w;
    __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float* x) const
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = Pack<T>::un(u[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = *reinterpret_cast<const float4*>(p);
        b = *(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void get(float* x) const
    {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float* x)
{
    *reinterpret_cast<uint4*>(p) = make_uint4(Pack<T>::two(x[0], x[1]), Pack<T>::two(x[2], x[3]),
                                              Pack<T>::two(x[4], x[5]), Pack<T>::two(x[6], x[7]));
}

// Heads first, first + kGroups step, .. of a row: norm (gain not null) and
// rotation (turn).  src, dst: the row's heads back to back.
template <typename T, typename TI, int D, bool kTurn>
__device__ __forceinline__ void heads_of(const TI* src, T* dst, int heads, int part, int parts, const float* gain,
                                         float eps, int pairs, const float* cs, const float* sn)
{
    constexpr int kLanes = D / 16, kGroups = 32 / kLanes, kUnroll = sizeof(TI) == 4 ? 2 : 4;
    const int lane = threadIdx.x & 31, g = lane / kLanes, c = (lane % kLanes) * 8;
    float gx[8], gy[8];
    if (kTurn && gain) {
        Raw<float> r;
        r.load(gain + c);
        r.get(gx);
        r.load(gain + D / 2 + c);
        r.get(gy);
    }
    for (int h0 = part * kGroups + g; h0 - g < heads; h0 += parts * kGroups * kUnroll) {
        Raw<TI> rx[kUnroll], ry[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const int h = h0 + u * parts * kGroups;
            const TI* at = src + (long long)min(h, heads - 1) * D + c;
            rx[u].load(at);
            ry[u].load(at + D / 2);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const int h = h0 + u * parts * kGroups;
            if (u > 0 && h - g >= heads) break;
            float x[8], y[8];
            rx[u].get(x);
            ry[u].get(y);
            if (kTurn && gain) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; i++) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float r = 1.f / sqrtf(ss * (1.f / D) + eps);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    x[i] = x[i] * r * gx[i];
                    y[i] = y[i] * r * gy[i];
                }
            }
            if (kTurn && pairs) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float p = x[2 * i], q = x[2 * i + 1], v = y[2 * i], w = y[2 * i + 1];
                    x[2 * i] = p * cs[i] - q * sn[i];
                    x[2 * i + 1] = q * cs[i] + p * sn[i];
                    y[2 * i] = v * cs[4 + i] - w * sn[4 + i];
                    y[2 * i + 1] = w * cs[4 + i] + v * sn[4 + i];
                }
            } else if (kTurn) {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float p = x[i], q = y[i];
                    x[i] = p * cs[i] - q * sn[i];
                    y[i] = q * cs[i] + p * sn[i];
                }
            }
            if (h < heads) {
                store8(dst + (long long)h * D + c, x);
                store8(dst + (long long)h * D + D / 2 + c, y);
            }
        }
    }
}

// Warp w of the grid: row w / parts, and every parts-th group of heads of it.
template <typename T, typename TI, int D>
__global__ void __launch_bounds__(kRotThreads, 5) lm_rotate_kernel(const LmRotateArgs a, int hq, int hk, int parts,
                                                                unsigned* err)
{
    constexpr int kLanes = D / 16;
    const int warp = (int)((blockIdx.x * (long long)kRotThreads + threadIdx.x) >> 5);
    const int row = parts == 1 ? warp : warp / parts, part = warp - row * parts;
    pdl_wait();
    pdl_launch();
    if (row >= a.rows) return;
    const int lane = threadIdx.x & 31, c = (lane % kLanes) * 8;
    const int pos = __ldg(a.positions + row);
    long long slot = row;
    if (a.slots) {
        slot = __ldg(a.slots + row);
        if (slot == -1) return;
        if (slot < 0 || slot >= a.n_slots) {
            if (lane == 0) atomicOr(err, CODEC_LM_ERR_SLOT);
            return;
        }
    }
    if (pos < 0 || pos >= a.max_positions) {
        if (lane == 0) atomicOr(err, CODEC_LM_ERR_POSITION);
        return;
    }
    // queries, keys and values: all here, or one of them by blockIdx.y
    const bool all = gridDim.y == 1;
    // cos, sin of this lane's eight rotations: pair index c + i (halves), or
    // c / 2 + i and D / 4 + c / 2 + i (pairs)
    float cs[8] = {}, sn[8] = {};
    if (blockIdx.y < 2) {
        const float2* t = a.turn + (long long)pos * (D / 2);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const int at = a.pairs ? (i < 4 ? c / 2 + i : D / 4 + c / 2 + i - 4) : c + i;
            const float4 v = __ldg(reinterpret_cast<const float4*>(t + at));
            cs[i] = v.x;
            sn[i] = v.y;
            cs[i + 1] = v.z;
            sn[i + 1] = v.w;
        }
    }
    if (blockIdx.y == 0)
        heads_of<T, TI, D, true>(static_cast<const TI*>(a.q) + row * a.qs,
                                 static_cast<T*>(a.q_out) + (long long)row * hq * D, hq, part, parts, a.q_gain, a.eps,
                                 a.pairs, cs, sn);
    if (all || blockIdx.y == 1)
        heads_of<T, TI, D, true>(static_cast<const TI*>(a.k) + row * a.ks, static_cast<T*>(a.k_dst) + slot * hk * D,
                                 hk, part, parts, a.k_gain, a.eps, a.pairs, cs, sn);
    if (a.v && (all || blockIdx.y == 2))
        heads_of<T, TI, D, false>(static_cast<const TI*>(a.v) + row * a.vs, static_cast<T*>(a.v_dst) + slot * hk * D,
                                  hk, part, parts, nullptr, 0.f, 0, cs, sn);
}

// The angle p theta^(-2 i / D) and its cosine and sine in fp64, rounded once.
__global__ void lm_turn_table_kernel(float2* turn, long long n, int half, double log2_theta)
{
    const long long u = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (u >= n) return;
    const int p = (int)(u / half), i = (int)(u - (long long)p * half);
    double s, c;
    sincos((double)p * exp2(-log2_theta * i / half), &s, &c);
    turn[u] = make_float2((float)c, (float)s);
}

template <typename T, typename TI, int D>
cudaError_t launch(const LmShape& sh, const LmRotateArgs& a, cudaStream_t s)
{
    constexpr int kGroups = 32 / (D / 16);
    // few rows: spread a row's heads over warps until there are about 16 warps per SM
    const int most = (sh.hq + kGroups - 1) / kGroups;
    int parts = 1;
    while (parts < most && (long long)a.rows * parts < 152 * 16) parts++;
    const long long warps = (long long)a.rows * parts;
    const unsigned ctas = (unsigned)((warps + kRotThreads / 32 - 1) / (kRotThreads / 32));
    // While every group of heads has a warp of its own, queries, keys and values go
    // to different warps: 64 rows of 16 / 16 heads of 64 2.4 us (in turn 3.2), of 32 / 8
    // of 128 2.9 (3.2), 500 rows of 16 / 16 3.1 (3.6).  Beyond that the warps' set-up
    // costs more than it spreads: 500 rows of 32 / 8 6.2 (5.2), 2,000 rows 10.4 (10.1)
    // and 8.0 (7.4), 16,000 70 (65) and 41 (38); 4,097 rows 17.0 (18.9) and 9.6 (9.3).
    const unsigned kinds = (long long)a.rows * most <= 152 * 16 ? (a.v ? 3 : 2) : 1;
    return launch_pdl(lm_rotate_kernel<T, TI, D>, dim3(ctas, kinds), dim3(kRotThreads), 0, s, a, sh.hq, sh.hk, parts,
                      sh.err);
}

template <typename T>
cudaError_t launch_t(const LmShape& sh, const LmRotateArgs& a, bool in32, cudaStream_t s)
{
    if (sh.D == 128) return in32 ? launch<T, float, 128>(sh, a, s) : launch<T, T, 128>(sh, a, s);
    return in32 ? launch<T, float, 64>(sh, a, s) : launch<T, T, 64>(sh, a, s);
}

}  // namespace

cudaError_t launch_lm_rotate(const LmShape& sh, const LmRotateArgs& a, int in_type, cudaStream_t s)
{
    const bool in32 = in_type == CODEC_LM_FP32;
    return sh.type == CODEC_LM_BF16 ? launch_t<__nv_bfloat16>(sh, a, in32, s) : launch_t<__half>(sh, a, in32, s);
}

cudaError_t launch_lm_turn_table(float2* turn, int max_positions, int D, double theta, cudaStream_t s)
{
    const long long n = (long long)max_positions * (D / 2);
    lm_turn_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(turn, n, D / 2, log2(theta));
    return cudaGetLastError();
}

}  // namespace codec
