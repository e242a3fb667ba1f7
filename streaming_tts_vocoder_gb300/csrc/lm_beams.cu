// Beam search's selection: log-softmax of each beam's logits, and of each
// group's candidates the best.
//
// Two launches.  The first reads the logits once: a part of a row gives its
// log(sum(exp(x))) and its best `beams` tokens; inside a row the order of
// candidates is that of the logits themselves.  A warp holds 4 KB of a row in
// registers: maxima (packed), sums of 2^(x log2 e - C) with a whole number C, and
// then a search of the lanes' maxima, largest first, for values that belong into
// the list of the best; a lane's values are read once more for it, 64 by the
// whole warp.  The second launch joins the parts and picks among a group's rows by
// sums + x - log(sum), in fp64: lists are sorted, so a warp looks at their heads
// alone for each candidate, as whole numbers of the same order (three reductions).
//
// What decides between rows is the logarithm, and sums of exponentials in fp32
// are off by up to kNear.  Where two neighbours of the result come from different
// rows and lie closer, or the last one and any candidate of another row do, the
// logarithms of those rows are worked out again to about 1e-9, and the choice is made
// once more.
//
// 1,024 rows of 65,537 in bf16 (60 of them ended): 38.2 us, 3.3 TB/s; 30 of it before the
// search.  Neither the memory nor the issue slots bound it: a chunk's loads, maxima and
// sums follow one another in each warp, and all rows are one wave of CTAs, whose last
// stretch is the search.  The next chunk in registers meanwhile (spills), prefetches two
// chunks ahead (+1.5 us), six CTAs an SM (two waves, 54 us), ten (48), twice as many parts
// of a row (43) were slower.  4 x 4 of 2,048: 9.9 us, two launches and the second one's
// chain of steps.
//
// Logarithms that are worked out again are a CTA's for each group, a row after the other:
// 35 us each for 65,537 logits in bf16.  Beams with the same logits and sums always need
// it (8 of them 282 us where 8 of their own take 16, 32 1,134 and 71; 128 x 8 571 and 38;
// 4 x 4 of 2,048 25 and 10), and so do rows masked from end to end (8 304); a search that
// begins with one beam whose sum is finite, and the others' at -inf, does not.
#include <climits>

#include "lm.h"

namespace codec {

namespace {

constexpr int kThreads = 256;
// A row's logarithm is off by 2.1e-6 at most, and two rows' difference by twice that; the
// terms have one sign where few different logits fill a row, so they are added as they
// are.  Relative to the sum: the exponent's argument rounded once, 2^-20 ln 2 where it
// lies in 16 .. 32 below the largest (what lies further has no weight: 2^24 tokens), 6.6e-7;
// log2 e as a float, 1.33e-8 times the 17 that such a logit lies below, 2.2e-7; ex2 2^-22,
// 2.4e-7; up to 15 additions to one number and two that join those, 2^-24 each, 1.0e-6.
// The rest is kept or fp64.
constexpr float kNear = 5e-6f;
// A row whose largest logit is as far from zero (one masked by its type's lowest value
// from end to end) has its logarithm worked out from the differences to that one: the
// powers' whole numbers would not hold it.
constexpr float kFar = 1048576.f;
constexpr double kLog2eOff = 1.4426950408889634f / 1.4426950408889634074 - 1.;    // of log2 e as a float, relative
constexpr int kLists = 256;                 // of a group: beams x parts of a row

constexpr int kRowWarps = 4;
constexpr int kRowThreads = 32 * kRowWarps;
constexpr int kVectors = 8;                 // of 16 bytes a lane: a chunk of a row is 4 KB
constexpr int kWindow = 16;                 // chunks of each warp whose best are looked for at once

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// A row that offers tokens.
__device__ __forceinline__ bool offers(const LmBeamArgs& a, int row)
{
    return __ldg(a.ended + row) == 0 && fabsf(__ldg(a.sums + row)) < INFINITY;
}

// Candidate (value, index): the first before the second.
template <typename V>
__device__ __forceinline__ bool ahead(V x, int i, V y, int j) { return x > y || (x == y && i < j); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The values of 16 bytes.
template <typename T> struct Vector;
template <> struct Vector<float> {
    static constexpr int N = 4;
    // the largest (NaN if one is) of vectors: pairwise, then of the last
    using Two = float2;
    static __device__ __forceinline__ Two top(uint4 v)
    {
        return make_float2(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ Two max(Two a, Two b) { return make_float2(max_nan(a.x, b.x), max_nan(a.y, b.y)); }
    static __device__ __forceinline__ float2 split(Two a) { return a; }
    static __device__ __forceinline__ void get(uint4 v, float* x)
    {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
};
template <> struct Vector<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ __nv_bfloat162 two(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
    using Two = __nv_bfloat162;
    static __device__ __forceinline__ Two top(uint4 v)
    {
        return __hmax2_nan(__hmax2_nan(two(v.x), two(v.y)), __hmax2_nan(two(v.z), two(v.w)));
    }
    static __device__ __forceinline__ Two max(Two a, Two b) { return __hmax2_nan(a, b); }
    static __device__ __forceinline__ float2 split(Two a) { return __bfloat1622float2(a); }
    static __device__ __forceinline__ void get(uint4 v, float* x)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <> struct Vector<__half> {
    static constexpr int N = 8;
    static __device__ __forceinline__ __half2 two(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
    using Two = __half2;
    static __device__ __forceinline__ Two top(uint4 v)
    {
        return __hmax2_nan(__hmax2_nan(two(v.x), two(v.y)), __hmax2_nan(two(v.z), two(v.w)));
    }
    static __device__ __forceinline__ Two max(Two a, Two b) { return __hmax2_nan(a, b); }
    static __device__ __forceinline__ float2 split(Two a) { return __half22float2(a); }
    static __device__ __forceinline__ void get(uint4 v, float* x)
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = __half22float2(two(w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};
template <typename T> __device__ __forceinline__ T minus_infinity();
template <> __device__ __forceinline__ float minus_infinity() { return -INFINITY; }
template <> __device__ __forceinline__ __half minus_infinity() { return __ushort_as_half(0xfc00); }
template <> __device__ __forceinline__ __nv_bfloat16 minus_infinity() { return __ushort_as_bfloat16(0xff80); }

// A float as a whole number of the same order (not NaN).
__device__ __forceinline__ int ordered(float x)
{
    const int i = __float_as_int(x);
    return i >= 0 ? i : i ^ 0x7fffffff;
}

// 2^(c - most), 0 where c is none or far below.
__device__ __forceinline__ float power_of_two(int c, int most)
{
    return c == INT_MIN || c < most - 126 ? 0.f : __int_as_float((127 + c - most) << 23);
}

// hi + lo += y with the rounding error kept.
__device__ __forceinline__ void add_kept(float& hi, float& lo, float y)
{
    const float t = __fadd_rn(hi, y), b = __fsub_rn(t, hi);
    lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(y, b));
    hi = t;
}

// Row blockIdx.x, part blockIdx.y of it: windows of chunks, of which a warp takes
// every kRowWarps-th.
template <typename T>
__global__ void __launch_bounds__(kRowThreads, 8) lm_beam_rows_kernel(const LmBeamArgs a)
{
    using V = Vector<T>;
    constexpr int kChunk = kVectors * 32 * V::N;
    constexpr float kLog2e = 1.4426950408889634f;
    __shared__ float tops[kRowWarps][kWindow][33];      // (33: a lane's of all chunks lie in different banks)
    __shared__ float part_hi[kRowWarps], part_lo[kRowWarps], part_top[kRowWarps];
    __shared__ int part_c[kRowWarps];
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = a.beams;
    pdl_wait();
    pdl_launch();
    if (!offers(a, row)) return;
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    // vectors lie on 16 bytes: the first starts `lead` values before the row
    const int lead = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int end = lead + a.vocab, chunks = (end + kChunk - 1) / kChunk;
    const int each = (chunks + gridDim.y - 1) / gridDim.y;
    const int last = min(chunks, ((int)blockIdx.y + 1) * each);
    const T* base = x - lead;

    // of the first warp: lane i < K has the i-th best so far; the K-th
    float best_x = -INFINITY, least = -INFINITY;
    int best_i = INT_MAX, least_i = INT_MAX;
    float top = -INFINITY, hi = 0.f, lo = 0.f;  // of the warp; this lane's sum
    int C = INT_MIN;
    bool bad = false;
    for (int c0 = blockIdx.y * each; c0 < last; c0 += kRowWarps * kWindow) {
        for (int n = 0; n < kWindow; n++) tops[warp][n][lane] = -INFINITY;
        for (int n = 0, c = c0 + warp; n < kWindow && c < last && !bad; c += kRowWarps, n++) {
            const int v0 = c * kChunk + lane * V::N;
            // the warp's next chunk to L2: a line of 128 bytes a lane
            if (c + kRowWarps < last)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(
                    base + min((c + kRowWarps) * kChunk + lane * (128 / (int)sizeof(T)), end - 1)));
            uint4 raw[kVectors];
            if (c * kChunk >= lead && (c + 1) * kChunk <= end) {
#pragma unroll
                for (int i = 0; i < kVectors; i++)
                    raw[i] = __ldg(reinterpret_cast<const uint4*>(base + v0 + i * 32 * V::N));
            } else {
                // the row's first or last: vectors that pass its ends value by value
#pragma unroll
                for (int i = 0; i < kVectors; i++) {
                    const int v1 = v0 + i * 32 * V::N;
                    if (v1 >= lead && v1 + V::N <= end) {
                        raw[i] = __ldg(reinterpret_cast<const uint4*>(base + v1));
                    } else {
                        alignas(16) T e[V::N];
#pragma unroll
                        for (int j = 0; j < V::N; j++) e[j] = v1 + j >= lead && v1 + j < end ? base[v1 + j] : minus_infinity<T>();
                        raw[i] = *reinterpret_cast<const uint4*>(e);
                    }
                }
            }
            typename V::Two pair = V::top(raw[0]);
#pragma unroll
            for (int i = 1; i < kVectors; i++) pair = V::max(pair, V::top(raw[i]));
            const float mine = max_nan(V::split(pair).x, V::split(pair).y);
            bad = __any_sync(0xffffffffu, !(mine < INFINITY));
            if (bad) break;
            tops[warp][n][lane] = mine;
            const int most = __reduce_max_sync(0xffffffffu, ordered(mine));
            const float chunk_top = __int_as_float(most >= 0 ? most : most ^ 0x7fffffff);
            if (chunk_top == -INFINITY) continue;
            if (chunk_top > top) {
                top = chunk_top;
                const int now = (int)ceilf(top * kLog2e);
                const float f = power_of_two(C, now);
                hi *= f;
                lo *= f;
                C = now;
            }
            const float2 c2 = make_float2(-(float)C, -(float)C), log2e = make_float2(kLog2e, kLog2e);
            float2 sum[2] = {};
#pragma unroll
            for (int i = 0; i < kVectors; i++) {
                float y[V::N];
                V::get(raw[i], y);
#pragma unroll
                for (int j = 0; j < V::N; j += 2) {
                    float2 e = __ffma2_rn(make_float2(y[j], y[j + 1]), log2e, c2);
                    e = make_float2(exp2_fast(e.x), exp2_fast(e.y));
                    sum[j / 2 & 1] = __fadd2_rn(sum[j / 2 & 1], e);
                }
            }
            add_kept(hi, lo, (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
        }
        if (__syncthreads_or(bad)) {
            bad = true;
            break;
        }
        // The first warp takes the window's places (lane, chunk) with the largest values first,
        // until none can hold one that belongs into the list: K of them at a time, whose
        // last one's largest is below the list's last already, so that of their values, read
        // together, few are put in.
        float mx[kRowWarps];                    // of this lane's chunks of each warp, and which
        int of[kRowWarps];
        if (warp == 0) {
#pragma unroll
            for (int w = 0; w < kRowWarps; w++) {
                mx[w] = tops[w][0][lane];
                of[w] = 0;
#pragma unroll
                for (int j = 1; j < kWindow; j++) {
                    const float y = tops[w][j][lane];
                    of[w] = y > mx[w] ? j : of[w];
                    mx[w] = fmaxf(mx[w], y);
                }
            }
        }
        __syncwarp();
        constexpr int kPlaces = 32 * kRowWarps * kWindow;
        bool more = warp == 0;
        for (int round = 0; round <= kPlaces && more; round++) {
            int n = 0, place = 0;               // lane i: the i-th place
            float y = 0.f;
            for (int turn = 0; turn <= kPlaces && n < K; turn++) {
                float mine = mx[0];
                int at_w = 0, at_j = of[0];
#pragma unroll
                for (int w = 1; w < kRowWarps; w++) {
                    at_j = mx[w] > mine ? of[w] : at_j;
                    at_w = mx[w] > mine ? w : at_w;
                    mine = fmaxf(mine, mx[w]);
                }
                const int key = ordered(mine), k = __reduce_max_sync(0xffffffffu, key);
                y = __int_as_float(k >= 0 ? k : k ^ 0x7fffffff);
                more = y > -INFINITY && y >= least;
                if (!more) break;
                const int from = __ffs(__ballot_sync(0xffffffffu, key == k)) - 1;
                const int w = __shfl_sync(0xffffffffu, at_w, from), j0 = __shfl_sync(0xffffffffu, at_j, from);
                const int c = c0 + w + kRowWarps * j0;
                // that lane's next one of the warp's chunks: a chunk a lane
                float left = lane < kWindow && lane != j0 ? tops[w][lane][from] : -INFINITY;
                if (lane == j0) tops[w][j0][from] = -INFINITY;
                const int left_key = ordered(left), left_k = __reduce_max_sync(0xffffffffu, left_key);
                const int left_j = __ffs(__ballot_sync(0xffffffffu, left_key == left_k)) - 1;
                left = __int_as_float(left_k >= 0 ? left_k : left_k ^ 0x7fffffff);
#pragma unroll
                for (int i = 0; i < kRowWarps; i++)
                    if (i == w && lane == from) {
                        mx[i] = left;
                        of[i] = left_j;
                    }
                if (y == least && c * kChunk - lead > least_i) continue;    // equal ones only before those of the list
                if (lane == n) place = c * 32 + from;
                n++;
            }
            if (n == K && y > least) {          // K values are as large
                least = y;
                least_i = INT_MAX;
            }
            // their values: V::N / 4 for each lane, of kRead places at once
            constexpr int kE = V::N / 4, kRead = 4;
            for (int first = 0; first < n; first += kRead) {
                float z[kRead][kE];
                int at[kRead];
#pragma unroll
                for (int q = 0; q < kRead; q++) {
                    const int pl = __shfl_sync(0xffffffffu, place, min(first + q, n - 1));
                    at[q] = pl / 32 * kChunk + ((lane >> 2) * 32 + pl % 32) * V::N + (lane & 3) * kE;
#pragma unroll
                    for (int j = 0; j < kE; j++)
                        z[q][j] = first + q < n && at[q] + j >= lead && at[q] + j < end ? to_float(base[at[q] + j]) : -INFINITY;
                }
#pragma unroll
                for (int q = 0; q < kRead; q++)
#pragma unroll
                    for (int j = 0; j < kE; j++) {
                        unsigned in = __ballot_sync(0xffffffffu, z[q][j] > -INFINITY && ahead(z[q][j], at[q] + j - lead, least, least_i));
                        if (in == 0) continue;
                        while (in) {
                            const int who = __ffs(in) - 1;
                            in &= in - 1;
                            const float nx = __shfl_sync(0xffffffffu, z[q][j], who);
                            const int ni = __shfl_sync(0xffffffffu, at[q] + j - lead, who);
                            const int to = __popc(__ballot_sync(0xffffffffu, ahead(best_x, best_i, nx, ni)));
                            const float ux = __shfl_up_sync(0xffffffffu, best_x, 1);
                            const int ui = __shfl_up_sync(0xffffffffu, best_i, 1);
                            if (lane >= to) {
                                best_x = lane == to ? nx : ux;
                                best_i = lane == to ? ni : ui;
                            }
                        }
                        const float kx = __shfl_sync(0xffffffffu, best_x, K - 1);
                        const int ki = __shfl_sync(0xffffffffu, best_i, K - 1);
                        if (ahead(kx, ki, least, least_i)) {
                            least = kx;
                            least_i = ki;
                        }
                    }
            }
        }
        __syncthreads();                        // tops are written again
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo += __shfl_xor_sync(0xffffffffu, lo, o);
        add_kept(hi, lo, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (lane == 0) {
        part_hi[warp] = hi;
        part_lo[warp] = lo;
        part_c[warp] = C;
        part_top[warp] = bad ? NAN : top;
    }
    __syncthreads();
    const long long at = (long long)row * gridDim.y + blockIdx.y;
    if (tid < K) a.ws.best[at * K + tid] = make_uint2(__float_as_uint(best_x), (unsigned)best_i);
    if (tid == 0) {
        int most = part_c[0];
        float m = part_top[0];
        for (int w = 1; w < kRowWarps; w++) {
            m = max_nan(m, part_top[w]);
            most = max(most, part_c[w]);
        }
        double sum = 0.;
        for (int w = 0; w < kRowWarps; w++)
            sum += ((double)part_hi[w] + (double)part_lo[w]) * power_of_two(part_c[w], most);
        a.ws.part[at] = LmBeamPart{sum, m, most};
    }
}

// exp(d + e) by a table and a series (P. T. P. Tang, "Table-driven implementation of the
// exponential function in IEEE floating-point arithmetic", ACM TOMS 15, 1989) as 2^k 2^(j / 64)
// (1 + p): k, the power of two of the table (two floats), and p, a short series of what
// is left (at most ln 2 / 128).  e: a small rest of d.
__device__ __forceinline__ float2 exp_parts(float d, float e, const float2* table, float& p, float& scale)
{
    constexpr float kInv = 92.332482616893656f;             // 64 / ln 2
    constexpr float kHi = 0x1.62cp-7f;                      // ln 2 / 64: 11 bits, and the rest
    constexpr float kLo = (float)(0.010830424696249145 - (double)kHi);
    const float m = rintf(d * kInv);
    const float r = fmaf(-m, kLo, fmaf(-m, kHi, d)) + e;
    p = r * fmaf(r, fmaf(r, fmaf(r, 1.f / 24.f, 1.f / 6.f), 0.5f), 1.f);
    const int im = (int)m;
    scale = __int_as_float(((im >> 6) + 127) << 23);
    return table[im & 63];
}

// log(s) to about 1e-9, s in 2^-64 .. 2^64: fp32's, and how far s is from its exponential, a
// step of Newton's method (log() itself takes some 2 us, fp64 being slow).
__device__ __forceinline__ double log_of(double s, const float2* table)
{
    const float y = logf((float)s);
    float p, scale;
    const float2 t = exp_parts(-y, 0.f, table, p, scale);
    const double off = fma(s, ((double)t.x + (double)t.y) * (1. + (double)p) * (double)scale, -1.);
    return (double)y + off * (1. - 0.5 * off);
}

// log(sum(exp(x - top))) of a row to about 1e-9, by the whole CTA: terms added with
// their rounding errors kept.
template <typename T>
__device__ double exact_log_sum(const T* x, int n, float top, const float2* table, double* sm)
{
    const int tid = threadIdx.x;
    float s = 0.f, c = 0.f;
    for (int v = tid; v < n; v += kThreads) {
        const float y = to_float(x[v]);
        const float d = __fsub_rn(y, top);
        if (!(d > -80.f)) continue;                         // nothing beside the maximum's 1
        const float u = __fsub_rn(d, y), w = __fsub_rn(d, u);
        const float e = __fadd_rn(__fsub_rn(y, w), __fsub_rn(-top, u));     // what d was rounded by
        float p, scale;
        const float2 t = exp_parts(d, e, table, p, scale);
        const float h = t.x * scale, l = fmaf(t.x, p, t.y) * scale;
        const float now = __fadd_rn(s, h), b = __fsub_rn(now, s);
        c += __fadd_rn(__fsub_rn(s, __fsub_rn(now, b)), __fsub_rn(h, b)) + l;
        s = now;
    }
    double sum = (double)s + (double)c;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if ((tid & 31) == 0) sm[tid >> 5] = sum;
    __syncthreads();
    sum = 0.;
    for (int w = 0; w < kThreads / 32; w++) sum += sm[w];
    return log_of(sum, table);
}

// A score as a whole number of the same order, and back.  Zeros of both signs are one.
__device__ __forceinline__ unsigned long long key_of(double s)
{
    const long long bits = __double_as_longlong(__dadd_rn(s, 0.));
    return bits < 0 ? ~(unsigned long long)bits : (unsigned long long)bits | 1ULL << 63;
}
__device__ __forceinline__ double score_of(unsigned long long key)
{
    return __longlong_as_double((long long)(key >> 63 ? key & ~(1ULL << 63) : ~key));
}

// One group.  Dynamic shared memory: the lists' scores as whole numbers of the same
// order and their indexes (row of the group, token), [K x parts][K] each.
template <typename T>
__global__ void __launch_bounds__(kThreads) lm_beam_pick_kernel(const LmBeamArgs a, int parts)
{
    extern __shared__ unsigned long long keys[];
    __shared__ double base[kLmMaxBeams];        // sums - log(sum(exp(x - top))), or the sum of an ended beam
    __shared__ float top[kLmMaxBeams];
    __shared__ int power[kLmMaxBeams];
    __shared__ int kind[kLmMaxBeams];           // 0: offers nothing, 1: tokens, 2: itself
    __shared__ double sums[kThreads / 32], got[kLmMaxBeams + 1];
    __shared__ int got_i[kLmMaxBeams + 1];
    __shared__ float2 table[64];
    __shared__ unsigned again, far;
    const int K = a.beams, row0 = blockIdx.x * K, lists = K * parts;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int* index = reinterpret_cast<int*>(keys + lists * K);
    if (tid < 64) {
        const double t = exp2(tid / 64.);
        table[tid] = make_float2((float)t, (float)(t - (double)(float)t));
    }
    pdl_wait();
    pdl_launch();
    const uint2* best = a.ws.best + (long long)row0 * parts * K;
    // on their way meanwhile
    const uint2 ahead_of = tid < lists * K ? __ldcg(best + tid) : uint2{};
    const float sum = tid < K ? __ldg(a.sums + row0 + tid) : 0.f;
    const bool itself = tid < K && __ldg(a.ended + row0 + tid) != 0;
    for (int r = warp; r < K; r += kThreads / 32) {
        const int row = row0 + r;
        // (a row that offers nothing wrote nothing: what is found there is not used)
        float m = -INFINITY;
        double l = 0.;
        int most = INT_MIN;
        const LmBeamPart* part = a.ws.part + (long long)row * parts;
        for (int i = lane; i < parts; i += 32) {
            m = max_nan(m, __ldcg(&part[i].top));
            most = max(most, __ldcg(&part[i].c));
        }
        most = __reduce_max_sync(0xffffffffu, most);
        for (int i = lane; i < parts; i += 32) l += __ldcg(&part[i].sum) * power_of_two(__ldcg(&part[i].c), most);
        for (int o = parts > 1 ? 16 : 0; o > 0; o >>= 1) {
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            l += __shfl_xor_sync(0xffffffffu, l, o);
        }
        if (lane == 0) {
            top[r] = m;
            base[r] = l;
            power[r] = most;
        }
    }
    if (tid == 0) again = far = 0;
    __syncthreads();
    if (tid < K) {
        const float m = top[tid];
        const bool there = fabsf(sum) < INFINITY;
        kind[tid] = !there ? 0 : itself ? 2 : fabsf(m) < INFINITY ? 1 : 0;
        // sums of 2^(x log2 e - c), with a log2 e that is 1.33e-8 of itself too small or large
        base[tid] = kind[tid] != 1 ? (double)sum
                                   : (double)sum - ((log_of(base[tid], table) + power[tid] * 0.69314718055994531) -
                                                    kLog2eOff * (double)m - (double)m);
        if (kind[tid] == 1 && fabsf(m) >= kFar) atomicOr(&far, 1u << tid);
    }
    __syncthreads();
    auto work_out = [&](unsigned rows) {
        for (int q = 0; q < K; q++)
            if (rows >> q & 1 && kind[q] == 1) {
                const double l = exact_log_sum(static_cast<const T*>(a.logits) + (row0 + q) * a.stride, a.vocab, top[q],
                                               table, sums);
                if (tid == 0) base[q] = (double)__ldg(a.sums + row0 + q) - l;
            }
        __syncthreads();
    };
    if (far != 0) work_out(far);
    for (int round = 0; round < 2; round++) {
        for (int e = tid; e < lists * K; e += kThreads) {
            const uint2 c = e == tid ? ahead_of : __ldcg(best + e);
            const int l = e / K, r = l / parts;
            const float x = __uint_as_float(c.x);
            int i = INT_MAX;
            double s = 0.;
            if (kind[r] == 1 && x > -INFINITY) {
                s = base[r] + ((double)x - (double)top[r]);
                i = r * a.vocab + (int)c.y;
            } else if (kind[r] == 2 && e == r * parts * K) {
                s = base[r];
                i = r * a.vocab + max(a.end_token, 0);
            }
            keys[e] = key_of(s);
            index[e] = i;
        }
        __syncthreads();
        // The first warp picks: lane l has lists l, l + 32, .., each at its `at`-th
        // entry, and the best of their heads.
        if (warp == 0) {
            int at[kLists / 32] = {};
            unsigned hi = 0, lo = 0;
            int best_i = INT_MAX, which = 0;
            auto look = [&]() {
                unsigned long long key = 0;
                best_i = INT_MAX;
#pragma unroll
                for (int j = 0; j < kLists / 32; j++) {
                    if (32 * j >= lists) break;
                    const int l = lane + 32 * j;
                    if (l >= lists || at[j] == K) continue;
                    const int i = index[l * K + at[j]];
                    const unsigned long long k = keys[l * K + at[j]];
                    if (i != INT_MAX && (best_i == INT_MAX || k > key || (k == key && i < best_i))) {
                        key = k;
                        best_i = i;
                        which = j;
                    }
                }
                hi = (unsigned)(key >> 32);
                lo = (unsigned)key;
            };
            look();
            // one more than are wanted, to see how near it is
            for (int k = 0; k <= K; k++) {
                const unsigned top_hi = __reduce_max_sync(0xffffffffu, best_i == INT_MAX ? 0u : hi);
                const unsigned top_lo = __reduce_max_sync(0xffffffffu, best_i != INT_MAX && hi == top_hi ? lo : 0u);
                const int winner = __reduce_min_sync(0xffffffffu, hi == top_hi && lo == top_lo ? best_i : INT_MAX);
                if (lane == 0) {
                    got[k] = score_of((unsigned long long)top_hi << 32 | top_lo);
                    got_i[k] = winner;
                }
                if (winner != INT_MAX && best_i == winner) {
#pragma unroll
                    for (int j = 0; j < kLists / 32; j++)
                        if (j == which) at[j]++;
                    look();
                }
            }
        }
        __syncthreads();
        if (round == 1) break;
        if (tid < K && got_i[tid + 1] != INT_MAX) {
            const int p = got_i[tid] / a.vocab, q = got_i[tid + 1] / a.vocab;
            if (p != q && got[tid] - got[tid + 1] < kNear) atomicOr(&again, 1u << p | 1u << q);
        }
        // and other rows' that lie as near to the last one: what comes first behind it may be its own row's
        if (got_i[K - 1] != INT_MAX) {
            const int p = got_i[K - 1] / a.vocab;
            const double cut = got[K - 1];
            for (int e = tid; e < lists * K; e += kThreads) {
                const int q = e / K / parts;
                if (index[e] != INT_MAX && q != p && fabs(score_of(keys[e]) - cut) < kNear) atomicOr(&again, 1u << p | 1u << q);
            }
        }
        __syncthreads();
        if (again == 0) break;
        work_out(again & ~far);                 // (those far from zero are done)
    }
    if (tid < K) {
        const int c = got_i[tid], row = row0 + tid;
        const bool there = c != INT_MAX;
        const int p = there ? c / a.vocab : 0, token = there ? c - p * a.vocab : -1;
        const bool itself = there && kind[p] == 2;
        a.sums_out[row] = there ? itself ? __ldg(a.sums + row0 + p) : (float)got[tid] : -INFINITY;
        a.parents[row] = there ? row0 + p : -1;
        a.tokens[row] = itself ? a.end_token : token;
        a.ended_out[row] = !there || itself || token == a.end_token;
    }
}

template <typename T>
cudaError_t launch(const LmBeamArgs& a, cudaStream_t s)
{
    // parts of a row: about eight CTAs per SM, a chunk for each warp at least, and lists
    // for the second kernel's threads
    const int rows = a.groups * a.beams;
    const long long chunks = (a.vocab * (long long)sizeof(T) + 4095) / 4096;
    const int parts = (int)std::max<long long>(1, std::min<long long>({152 * 8 / rows, chunks / kRowWarps, kLists / a.beams}));
    const cudaError_t e = launch_pdl(lm_beam_rows_kernel<T>, dim3(rows, parts), dim3(kRowThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    const size_t smem = (sizeof(unsigned long long) + sizeof(int)) * a.beams * parts * a.beams;
    return launch_pdl(lm_beam_pick_kernel<T>, dim3(a.groups), dim3(kThreads), smem, s, a, parts);
}

template <typename T>
cudaError_t configure()
{
    return cudaFuncSetAttribute(lm_beam_pick_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(sizeof(unsigned long long) + sizeof(int)) * kLists * kLmMaxBeams);
}

}  // namespace

cudaError_t configure_lm_beams()
{
    for (const cudaError_t e : {configure<float>(), configure<__half>(), configure<__nv_bfloat16>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

cudaError_t launch_lm_beams(const LmBeamArgs& a, cudaStream_t s)
{
    return a.type == CODEC_LM_FP32   ? launch<float>(a, s)
           : a.type == CODEC_LM_BF16 ? launch<__nv_bfloat16>(a, s)
                                     : launch<__half>(a, s);
}

}  // namespace codec
