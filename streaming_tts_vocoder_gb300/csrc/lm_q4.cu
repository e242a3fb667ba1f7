// Keys and values into the cache in 4 bits, and blocks of it back in 16.
//
// Element by element: a row's group of 32 is four lanes' (least and largest by two
// shuffles), a tile of 16 positions goes through shared memory on the way back, and
// every byte is read and written once.  24 prompts of 700 to 2,000 tokens (8 heads of 128,
// bf16), stored and read back: 70 us, 4.9 TB/s (71 %).  Storing is 42 of it and bound by
// instructions (77 % of the issue slots); codes of values go out by two bytes, as two
// positions share a word of the layout that the attention reads.
// Reading back is 28, bound by both (64 % of the issue slots, 51 % of the memory).  64
// rows: 6 us for both, launches.
#include "lm.h"
#include "lm_q4.cuh"

namespace codec {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float2 unpack2(uint32_t w, const __half*)
{
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, const __nv_bfloat16*)
{
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

// Eight values as they lie in memory, and in fp32.
template <typename T> struct Raw {
    uint4 w;
    __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float* x) const
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = unpack2(u[i], static_cast<const T*>(nullptr));
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

// NaN if one is.
__device__ __forceinline__ float min_nan(float a, float b, float c)
{
    float y;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b, float c)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Codes of 8 values, four lanes a group.  The steps and their roundings are the
// format's: no contraction, no approximate reciprocal.  A value below -65504 needs no cut
// of its own: low is -65504 then and its code 0 as that one's is.  One above 65504 gets no
// code above that one's, as the steps keep the order (low may have been rounded up to
// near it, and then that is not 15).  kPast: inputs that may lie there and need it,
// fp32; bf16's least value of such a group is a half already, and fp16 has none.
// What is not finite shows in the least and the largest.
template <bool kPast>
__device__ __forceinline__ uint32_t encode(const float* x, __half& scale, __half& low)
{
    float lo = min_nan(min_nan(x[0], x[1], x[2]), min_nan(x[3], x[4], x[5]), min_nan(x[6], x[6], x[7]));
    float hi = max_nan(max_nan(x[0], x[1], x[2]), max_nan(x[3], x[4], x[5]), max_nan(x[6], x[6], x[7]));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        lo = min_nan(lo, lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max_nan(hi, hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const bool good = fabsf(lo) < INFINITY && fabsf(hi) < INFINITY;
    lo = fminf(fmaxf(lo, -65504.f), 65504.f);
    hi = fminf(fmaxf(hi, -65504.f), 65504.f);
    scale = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), 1.f / 15.f));
    low = __float2half_rn(lo);
    const float s = __half2float(scale), l = __half2float(low);
    const float inv = __frcp_rn(s);
    const float most = kPast ? fminf(__fmul_rn(__fsub_rn(65504.f, l), inv), 15.f) : 15.f;
    // a number of 0 .. 15 plus 1.5 x 2^23 is rounded to a whole one, which then stands in
    // the last bits; what the others' bits add to the word is taken off at the end
    constexpr float kWhole = 12582912.f;
    const float2 minus = make_float2(-l, -l), by = make_float2(inv, inv), whole = make_float2(kWhole, kWhole);
    uint32_t word = 0, rest = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float2 c = __fmul2_rn(__fadd2_rn(make_float2(x[i], x[i + 1]), minus), by);
        c = __fadd2_rn(make_float2(fminf(fmaxf(c.x, 0.f), most), fminf(fmaxf(c.y, 0.f), most)), whole);
        word += __float_as_uint(c.x) << (4 * i);
        word += __float_as_uint(c.y) << (4 * i + 4);
        rest += (0x4b400000u << (4 * i)) + (0x4b400000u << (4 * i + 4));
    }
    if (!good) scale = low = __ushort_as_half(0x7fff);
    return good && s > 0.f ? word - rest : 0u;
}

struct StoreArgs {
    const void *k, *v;
    long long ks, vs;
    int rows, hk, bs_shift, parts;
    const int* slots;
    long long n_slots;
    uint8_t *k_cache, *v_cache;
    unsigned* err;
};

// Warp w of the grid: row w / parts, and every parts-th set of 256 / D heads of
// it; keys or values by blockIdx.y.
template <typename TI, int D>
__global__ void __launch_bounds__(kThreads) lm_store_q4_kernel(const StoreArgs a)
{
    using Tile = Q4Tile<D>;
    constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
    const int warp = (int)((blockIdx.x * (long long)kThreads + threadIdx.x) >> 5);
    const int row = warp / a.parts, part = warp - row * a.parts;
    pdl_wait();
    pdl_launch();
    if (row >= a.rows) return;
    const int lane = threadIdx.x & 31, c = lane % kLanes, g = c >> 2, t = c & 3;
    const int slot = __ldg(a.slots + row);
    if (slot == -1) return;
    if (slot < 0 || slot >= a.n_slots) {
        if (lane == 0) atomicOr(a.err, CODEC_LM_ERR_SLOT);
        return;
    }
    const bool values = blockIdx.y == 1;
    const TI* src = static_cast<const TI*>(values ? a.v : a.k) + row * (values ? a.vs : a.ks) + c * 8;
    const int block = slot >> a.bs_shift, pos = slot & ((1 << a.bs_shift) - 1), p = pos & 15;
    const long long head_bytes = (long long)Tile::kBytes << (a.bs_shift - 4);
    uint8_t* base = (values ? a.v_cache : a.k_cache) + (long long)block * a.hk * head_bytes + (pos >> 4) * Tile::kBytes;
    // kUnroll sets of heads are loaded before the first is worked on
    constexpr int kUnroll = sizeof(TI) == 4 ? 2 : 4;
    const int step = a.parts * kHeads;
    for (int h0 = part * kHeads; h0 < a.hk; h0 += kUnroll * step) {
        Raw<TI> raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; u++) raw[u].load(src + (long long)min(h0 + u * step + lane / kLanes, a.hk - 1) * D);
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const int h = h0 + u * step + lane / kLanes;
            if (u > 0 && h0 + u * step >= a.hk) break;
            float x[8];
            raw[u].get(x);
            __half scale, low;
            const uint32_t word = encode<sizeof(TI) == 4>(x, scale, low);
            if (h >= a.hk) continue;
            uint8_t* tile = base + h * head_bytes;
            if (!values) {
                *reinterpret_cast<uint32_t*>(tile + Tile::k_word(p, t, g)) = word;
                if (t == 0) *reinterpret_cast<__half2*>(tile + Tile::k_param(p, g)) = __halves2half2(scale, low);
            } else {
                *reinterpret_cast<uint16_t*>(tile + Tile::v_pair(p, 2 * t, g)) = (uint16_t)word;
                *reinterpret_cast<uint16_t*>(tile + Tile::v_pair(p, 2 * t + 1, g)) = (uint16_t)(word >> 16);
                if (t == 0) {
                    *reinterpret_cast<__half*>(tile + Tile::v_scale(p, g)) = scale;
                    *reinterpret_cast<__half*>(tile + Tile::v_scale(p, g) + D) = low;
                }
            }
        }
    }
}

struct LoadArgs {
    const uint8_t *k_cache, *v_cache;
    const int *src, *dst;
    int n, hk, bs_shift, n_blocks, dst_blocks;
    void *k_dst, *v_dst;
    unsigned* err;
};

__device__ __forceinline__ uint32_t pack2(float a, float b, const __nv_bfloat16*)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __half*)
{
    // low + 15 scale may pass fp16's largest by the scale's rounding (NaN stays)
    const __half2 v = __floats2half2_rn(a > 65504.f ? 65504.f : a, b > 65504.f ? 65504.f : b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// A tile of 16 positions (null: zeros) to rows of the same head `stride` elements
// apart; row: this lane's eight elements of the first.  A whole warp; buf: a tile's
// bytes of its own in shared memory.  Codes as they lie at the lowest bits of halves
// are that many times 2^-24, four bits further 2^-20, and the scale makes up for it.
template <typename T, int D>
__device__ __forceinline__ void decode(const uint8_t* at, bool values, T* row, long long stride, uint4* buf)
{
    using Tile = Q4Tile<D>;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kVectors = Tile::kBytes / 16;
    const int lane = threadIdx.x & 31, c = lane % kLanes, g = c >> 2, t = c & 3;
    uint4 v[(kVectors + 31) / 32];
#pragma unroll
    for (int i = 0; i < (kVectors + 31) / 32; i++) {
        const int x = lane + 32 * i;
        v[i] = at && x < kVectors ? __ldg(reinterpret_cast<const uint4*>(at) + x) : uint4{};
    }
    __syncwarp();                       // buf may still be read
#pragma unroll
    for (int i = 0; i < (kVectors + 31) / 32; i++)
        if (lane + 32 * i < kVectors) buf[lane + 32 * i] = v[i];
    __syncwarp();
    const uint8_t* tile = reinterpret_cast<const uint8_t*>(buf);
#pragma unroll
    for (int p0 = 0; p0 < 16; p0 += kRows) {
        const int p = p0 + lane / kLanes;
        uint32_t word;
        float scale, low;
        if (!values) {
            word = *reinterpret_cast<const uint32_t*>(tile + Tile::k_word(p, t, g));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(tile + Tile::k_param(p, g)));
            scale = f.x;
            low = f.y;
        } else {
            word = *reinterpret_cast<const uint16_t*>(tile + Tile::v_pair(p, 2 * t, g)) |
                   (uint32_t)*reinterpret_cast<const uint16_t*>(tile + Tile::v_pair(p, 2 * t + 1, g)) << 16;
            scale = __half2float(*reinterpret_cast<const __half*>(tile + Tile::v_scale(p, g)));
            low = __half2float(*reinterpret_cast<const __half*>(tile + Tile::v_scale(p, g) + D));
        }
        const float s0 = scale * 0x1p24f, s1 = scale * 0x1p20f;
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; j++) {   // codes j and j + 4
            const uint32_t two = (j < 2 ? word : word >> 8) & (j & 1 ? 0x00f000f0u : 0x000f000fu);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
            x[j] = fmaf(j & 1 ? s1 : s0, f.x, low);
            x[j + 4] = fmaf(j & 1 ? s1 : s0, f.y, low);
        }
        *reinterpret_cast<uint4*>(row + p * stride) =
            make_uint4(pack2(x[0], x[1], row), pack2(x[2], x[3], row), pack2(x[4], x[5], row), pack2(x[6], x[7], row));
    }
}

// A warp per tile of 16 positions; keys or values by blockIdx.y.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) lm_load_q4_kernel(const LoadArgs a)
{
    __shared__ uint4 buf[kThreads / 32][Q4Tile<D>::kBytes / 16];
    const int lane = threadIdx.x & 31;
    const bool values = blockIdx.y == 1;
    const uint8_t* cache = values ? a.v_cache : a.k_cache;
    T* out = static_cast<T*>(values ? a.v_dst : a.k_dst);
    pdl_wait();
    pdl_launch();
    const int tiles = 1 << (a.bs_shift - 4);
    const long long all = (long long)a.n * a.hk * tiles;
    for (long long w = (blockIdx.x * (long long)kThreads + threadIdx.x) >> 5; w < all;
         w += gridDim.x * (long long)(kThreads / 32)) {
        const int tile = (int)(w % tiles), i = (int)(w / tiles / a.hk), h = (int)(w / tiles - (long long)i * a.hk);
        const int from = __ldg(a.src + i), to = __ldg(a.dst + i);
        if (from == -1) continue;
        if (from < 0 || from >= a.n_blocks || to < 0 || to >= a.dst_blocks) {
            if (lane == 0) atomicOr(a.err, CODEC_LM_ERR_BLOCK);
            continue;
        }
        decode<T, D>(cache + (((long long)from * a.hk + h) * tiles + tile) * Q4Tile<D>::kBytes, values,
                     out + ((((long long)to << a.bs_shift) + tile * 16) * a.hk + h) * D + lane % (D / 8) * 8,
                     (long long)a.hk * D, buf[threadIdx.x >> 5]);
    }
}

// See LmHalvesArgs.  blockIdx.y: keys, values, queries (a warp per row and head).
template <int D>
__global__ void __launch_bounds__(kThreads) lm_halves_q4_kernel(const LmHalvesArgs a, int hq, int hk, float scale, unsigned* err)
{
    __shared__ uint4 buf[kThreads / 32][Q4Tile<D>::kBytes / 16];
    const int lane = threadIdx.x & 31;
    const long long first = (blockIdx.x * (long long)kThreads + threadIdx.x) >> 5, step = gridDim.x * (long long)(kThreads / 32);
    pdl_wait();
    pdl_launch();
    if (blockIdx.y < 2) {
        const bool values = blockIdx.y == 1;
        const uint8_t* cache = static_cast<const uint8_t*>(values ? a.v_cache : a.k_cache);
        __half* out = static_cast<__half*>(values ? a.v16 : a.k16);
        const int tiles = 1 << (a.bs_shift - 4);
        for (long long w = first; w < (long long)a.n * hk * tiles; w += step) {
            const int tile = (int)(w % tiles), i = (int)(w / tiles / hk), h = (int)(w / tiles - (long long)i * hk);
            const int from = __ldg(a.table + i);
            const bool good = from >= 0 && from < a.n_blocks;
            if (!good && lane == 0) atomicOr(err, CODEC_LM_ERR_BLOCK);
            decode<__half, D>(good ? cache + (((long long)from * hk + h) * tiles + tile) * Q4Tile<D>::kBytes : nullptr, values,
                              out + ((((long long)i << a.bs_shift) + tile * 16) * hk + h) * D + lane % (D / 8) * 8,
                              (long long)hk * D, buf[threadIdx.x >> 5]);
        }
        return;
    }
    constexpr int kE = D / 32;
    for (long long w = first; w < (long long)a.B * hq; w += step) {
        const int b = (int)(w / hq), h = (int)(w - (long long)b * hq);
        const uint32_t* row = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + b * a.qs + (long long)h * D) +
                              lane * (kE / 2);
        float2 x[kE / 2];
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < kE / 2; e++) {
            const uint32_t u = row[e];
            x[e] = unpack2(u, static_cast<const __nv_bfloat16*>(nullptr));
            top = fmaxf(top, fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int lift = q4_query_lift(top);
        const float m = __int_as_float((127 + lift) << 23);
        uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<__half*>(a.q16) + w * D) + lane * (kE / 2);
#pragma unroll
        for (int e = 0; e < kE / 2; e++) {
            const __half2 v = __floats2half2_rn(x[e].x * m, x[e].y * m);
            to[e] = *reinterpret_cast<const uint32_t*>(&v);
        }
        if (lane == 0) a.row_c[w] = q4_query_factor(scale, lift);
    }
}

__global__ void lm_count_kernel(int* count, int n)
{
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) count[i] = i;
}

template <typename TI>
cudaError_t store_t(const LmShape& sh, StoreArgs& a, cudaStream_t s)
{
    const int most = (sh.hk * sh.D + 255) / 256;    // sets of heads
    a.parts = 1;
    while (a.parts < most && (long long)a.rows * a.parts < 152 * 16) a.parts++;
    const long long warps = (long long)a.rows * a.parts;
    const dim3 grid((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)), 2);
    return launch_pdl(sh.D == 128 ? lm_store_q4_kernel<TI, 128> : lm_store_q4_kernel<TI, 64>, grid, dim3(kThreads), 0,
                      s, a);
}

template <typename T>
cudaError_t load_t(const LmShape& sh, const LoadArgs& a, cudaStream_t s)
{
    const long long warps = ((long long)a.n * sh.hk) << (a.bs_shift - 4);
    const dim3 grid((unsigned)std::min<long long>((warps + kThreads / 32 - 1) / (kThreads / 32), 152 * 32), 2);
    return launch_pdl(sh.D == 128 ? lm_load_q4_kernel<T, 128> : lm_load_q4_kernel<T, 64>, grid, dim3(kThreads), 0, s,
                      a);
}

}  // namespace

cudaError_t launch_lm_store_q4(const LmShape& sh, const LmStoreQ4Args& x, int in_type, cudaStream_t s)
{
    StoreArgs a{x.k, x.v, x.ks, x.vs, x.rows, sh.hk, x.bs_shift, 1, x.slots, x.n_slots,
                static_cast<uint8_t*>(x.k_cache), static_cast<uint8_t*>(x.v_cache), sh.err};
    return in_type == CODEC_LM_FP32   ? store_t<float>(sh, a, s)
           : in_type == CODEC_LM_BF16 ? store_t<__nv_bfloat16>(sh, a, s)
                                      : store_t<__half>(sh, a, s);
}

cudaError_t launch_lm_load_q4(const LmShape& sh, const LmLoadQ4Args& x, cudaStream_t s)
{
    const LoadArgs a{static_cast<const uint8_t*>(x.k_cache), static_cast<const uint8_t*>(x.v_cache), x.src, x.dst, x.n,
                     sh.hk, x.bs_shift, x.n_blocks, x.dst_blocks, x.k_dst, x.v_dst, sh.err};
    return sh.type == CODEC_LM_BF16 ? load_t<__nv_bfloat16>(sh, a, s) : load_t<__half>(sh, a, s);
}

cudaError_t launch_lm_halves_q4(const LmShape& sh, const LmHalvesArgs& a, cudaStream_t s)
{
    const long long warps = std::max(((long long)a.n * sh.hk) << (a.bs_shift - 4), (long long)a.B * sh.hq);
    const dim3 grid((unsigned)std::min<long long>((warps + kThreads / 32 - 1) / (kThreads / 32), 152 * 16), 3);
    return launch_pdl(sh.D == 128 ? lm_halves_q4_kernel<128> : lm_halves_q4_kernel<64>, grid, dim3(kThreads), 0, s, a, sh.hq,
                      sh.hk, (float)(sh.scale * 1.4426950408889634), sh.err);
}

cudaError_t launch_lm_count(int* count, int n, cudaStream_t s)
{
    lm_count_kernel<<<(n + 255) / 256, 256, 0, s>>>(count, n);
    return cudaGetLastError();
}

}  // namespace codec
